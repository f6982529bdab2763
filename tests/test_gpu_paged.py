"""GPU parity of the paged-cache operators against plain fp64 ones: ragged
batches, every head layout, pages that end inside tiles, shared prefixes,
padding, rows without keys, and what a step leaves alone."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

import paged_ref  # noqa: E402
from paged_ref import Batch, check_attention  # noqa: E402


@pytest.fixture(scope="module")
def cpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import context_long_sequence_gb300 as m
    return m


def run_attention(cpa, b, stream=None, q=None, **kw):
    plan = b.plan(cpa, **kw)
    cache, batch, qg, _, _ = b.to_gpu(cpa)
    q = qg if q is None else q
    o = torch.full((b.N, b.Hq, b.d), float("nan"), dtype=plan.o_dtype, device="cuda")
    lse = torch.full((b.Hq, b.N), float("nan"), device="cuda")
    cpa.cp_attn_paged(plan, cache, batch, q, o, lse, cpa.alloc_paged_workspace(plan), stream=stream)
    torch.cuda.synchronize()
    return o, lse


BF, FP = torch.bfloat16, torch.float16
ATTENTION = {
    # name: (Batch arguments, plan arguments)
    "one_key": (dict(past=[0], new=[1]), {}),
    "one_token_short": (dict(past=[16], new=[1], d=128, Hq=8, Hkv=2), {}),
    "decode_ragged_d128": (dict(past=[0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 999], new=[1] * 13, d=128, Hq=8, Hkv=2), {}),
    "decode_ragged_d64_fp16": (dict(past=[5, 63, 64, 200, 1023], new=[1] * 5, d=64, Hq=4, Hkv=4, dtype=FP, heads_first=True, page_size=32), {}),
    "decode_long_one": (dict(past=[5000], new=[1], d=128, Hq=8, Hkv=1, page_size=64), {}),
    "decode_many_heads": (dict(past=[70, 700], new=[1, 1], d=64, Hq=28, Hkv=4), {}),          # 7 heads a group
    "group_of_71": (dict(past=[100, 33], new=[1, 2], d=64, Hq=71, Hkv=1), {}),
    "group_of_128": (dict(past=[150], new=[1], d=128, Hq=128, Hkv=1), {}),
    "drafts": (dict(past=[0, 3, 64, 511], new=[5, 1, 7, 4], d=128, Hq=8, Hkv=2), {}),
    "drafts_padded_rows": (dict(past=[10, 20], new=[3, 2], pad=6, d=64, Hq=4, Hkv=2), {}),
    "prompts": (dict(past=[0, 0, 0], new=[129, 1, 300], d=128, Hq=4, Hkv=2, page_size=64), {}),
    "chunk_after_past": (dict(past=[333, 1000], new=[200, 65], d=128, Hq=8, Hkv=4, page_size=128), {}),
    "chunk_d64_fp16": (dict(past=[77, 0], new=[140, 257], d=64, Hq=6, Hkv=2, dtype=FP, page_size=16), {}),
    "mixed_empty_sequences": (dict(past=[40, 0, 7, 0], new=[1, 0, 0, 3], d=64, Hq=4, Hkv=2), {}),
    "no_keys_yet": (dict(past=[0, 0], new=[0, 2], d=64), {}),
    "not_causal": (dict(past=[100, 0, 55], new=[3, 4, 70], d=128, Hq=4, Hkv=2), dict(causal=False)),
    "not_causal_cross": (dict(past=[1490, 17], new=[10, 10], d=64, Hq=8, Hkv=8), dict(causal=False)),
    "one_large_page": (dict(past=[500, 3], new=[2, 1], page_size=1024, d=128, Hq=4, Hkv=1), {}),
    "out_fp32": (dict(past=[100, 700], new=[1, 3], d=128, Hq=8, Hkv=2), dict(out_fp32=True)),
    "scale": (dict(past=[100], new=[2], d=64), dict(softmax_scale=0.3)),
    "prefix_small": (dict(past=[0, 3, 20], new=[1, 1, 1], prefixes=[(3, 100)], d=64, Hq=4, Hkv=2), {}),
    "prefix_d128_g4": (dict(past=[1, 30, 64, 65, 200, 0, 7], new=[1] * 7, prefixes=[(7, 1000)], d=128, Hq=8, Hkv=2), {}),
    "prefix_two_groups": (dict(past=[5] * 12, new=[1] * 12, prefixes=[(5, 333), (7, 64)], d=128, Hq=16, Hkv=2, page_size=32), {}),
    "prefix_some_without": (dict(past=[9, 90, 1, 40, 3], new=[1] * 5, prefixes=[(2, 130), (0, 50), (1, 17)], first=1, d=64, Hq=8, Hkv=4), {}),
    "prefix_empty": (dict(past=[9, 0], new=[1, 1], prefixes=[(1, 0), (1, 0)], d=64), {}),
    "prefix_and_no_own_keys_but_new": (dict(past=[0, 0], new=[1, 2], prefixes=[(2, 48)], d=128, Hq=8, Hkv=2), {}),
    "prefix_drafts": (dict(past=[5, 0, 33], new=[4, 2, 5], prefixes=[(3, 700)], d=128, Hq=8, Hkv=2, dtype=FP), {}),
    "prefix_many_rows": (dict(past=[3] * 70, new=[1] * 70, prefixes=[(70, 900)], d=128, Hq=8, Hkv=1), {}),  # 560 rows
    "prefix_prompts": (dict(past=[0, 0], new=[90, 150], prefixes=[(2, 260)], d=64, Hq=4, Hkv=2), {}),
    "prefix_no_multiple_of_group": (dict(past=[3] * 20, new=[1] * 20, prefixes=[(20, 259)], d=128, Hq=14, Hkv=2), {}),
}


@pytest.mark.parametrize("name", list(ATTENTION))
def test_attention_matches_fp64(cpa, name):
    kw, plan_kw = ATTENTION[name]
    b = Batch(seed=len(name) + 7, **kw)
    o, lse = run_attention(cpa, b, **plan_kw)
    n = b.N - b.pad
    ref = b.attention(causal=plan_kw.get("causal", True), scale=plan_kw.get("softmax_scale", 0.0))
    check_attention(o, lse, ref, b.dtype, b.d, n, name)
    # Rows behind the last sequence stay as they were.
    assert torch.isnan(o[n:]).all() and torch.isnan(lse[:, n:]).all()


MORE = {
    # The ways in which parts are joined, by the batch's size (a block, a head,
    # a KV head or a token to a warp), beyond the small batches above.
    "rows_1000": (dict(past=[300] * 64, new=[1] * 64, d=64, Hq=16, Hkv=2), {}),
    "groups_2800": (dict(past=[0, 500], new=[300, 400], d=64, Hq=8, Hkv=4), {}),
    "tokens_4200": (dict(past=[0] * 14, new=[300] * 14, d=64, Hq=4, Hkv=2), {}),
    "forty_kv_heads": (dict(past=[0, 90], new=[150, 100], d=64, Hq=40, Hkv=40), {}),
    # Few rows, light and not: by the small workers in several tiles, or by CTAs
    # because a token has more than 8 rows or the keys are many.
    "light_prefix": (dict(past=[3, 0, 40, 7, 300], new=[1, 2, 1, 5, 1], prefixes=[(3, 200), (2, 1000)], d=128, Hq=8, Hkv=2), {}),
    "light_prefix_d64": (dict(past=[3] * 25, new=[1] * 25, prefixes=[(25, 300)], d=64, Hq=20, Hkv=4), {}),
    "light_chunk": (dict(past=[50, 100], new=[30, 9], d=128, Hq=6, Hkv=2, dtype=FP), {}),
    "light_but_one": (dict(past=[50, 100, 0], new=[1, 9, 40], d=128, Hq=8, Hkv=2), {}),
    "drafts_group_9": (dict(past=[50, 100, 700], new=[2, 3, 1], d=128, Hq=18, Hkv=2), {}),
    "prefix_group_16": (dict(past=[5, 0, 90], new=[1, 2, 1], prefixes=[(3, 500)], d=128, Hq=32, Hkv=2, dtype=FP), {}),
    "prefix_group_12_d64": (dict(past=[5, 0, 90], new=[1, 2, 1], prefixes=[(3, 500)], d=64, Hq=24, Hkv=2), {}),
    "chunk_long_few_rows": (dict(past=[60000], new=[20], d=64, Hq=8, Hkv=2, page_size=256), {}),
    "prefix_tokens": (dict(past=[0] * 6, new=[200] * 6, prefixes=[(4, 300)], first=1, d=64, Hq=8, Hkv=8), {}),
}
for page in (16, 32, 64, 128, 256):
    for dtype, d in ((BF, 128), (FP, 64)):
        MORE[f"few_page{page}_d{d}"] = (dict(past=[page - 1, 2 * page, 300 + page], new=[1, 2, 1], page_size=page, d=d, dtype=dtype,
                                             Hq=8, Hkv=2, heads_first=page == 32), {})
        MORE[f"many_page{page}_d{d}"] = (dict(past=[page - 1, 5, 300 + page], new=[40, 129, 70], page_size=page, d=d, dtype=dtype,
                                              Hq=8, Hkv=2, heads_first=page == 64), {})


@pytest.mark.parametrize("name", list(MORE))
def test_attention_more_shapes(cpa, name):
    kw, plan_kw = MORE[name]
    b = Batch(seed=len(name), **kw)
    o, lse = run_attention(cpa, b, **plan_kw)
    check_attention(o, lse, b.attention(), b.dtype, b.d, b.N, name)


APPEND = {
    "one_token": (dict(past=[100], new=[1], d=128, Hq=8, Hkv=2), dict(rope_dim=128)),
    "decode_ragged": (dict(past=[0, 15, 16, 31, 500], new=[1] * 5, d=64, Hq=4, Hkv=4), dict(rope_dim=64)),
    "prompts_fp16": (dict(past=[0, 7, 0], new=[50, 1, 33], d=128, Hq=4, Hkv=2, dtype=FP, heads_first=True, page_size=32), dict(rope_dim=128)),
    "interleaved_partial": (dict(past=[3, 60], new=[4, 2], d=64, Hq=6, Hkv=3), dict(rope_dim=32, rope_interleaved=True)),
    "halves_partial": (dict(past=[3, 60], new=[4, 2], d=128, Hq=7, Hkv=1), dict(rope_dim=48)),
    "no_rotation": (dict(past=[3, 60], new=[4, 2], d=64, Hq=4, Hkv=2), dict(rope_dim=0)),
    "with_prefix": (dict(past=[2, 0, 9, 4], new=[1, 2, 1, 1], prefixes=[(2, 77), (1, 500)], d=64, Hq=4, Hkv=2), dict(rope_dim=64)),
    "padded_and_empty": (dict(past=[2, 0, 9], new=[1, 0, 3], pad=5, d=64, Hq=4, Hkv=2), dict(rope_dim=64)),
    "partial_with_prefix": (dict(past=[2, 0, 9, 4], new=[1, 2, 1, 1], prefixes=[(2, 77), (1, 500)], d=128, Hq=4, Hkv=2), dict(rope_dim=32)),
    "no_rotation_with_prefix": (dict(past=[2, 0], new=[1, 2], prefixes=[(2, 77)], d=64, Hq=4, Hkv=2), dict(rope_dim=0)),
}


def run_append(cpa, b, positions=None, with_q=True, in_place=False, **kw):
    plan = b.plan(cpa, **kw)
    cache, batch, q, k, v = b.to_gpu(cpa, positions)
    q_out = q if in_place else torch.full((b.N, b.Hq, b.d), float("nan"), dtype=b.dtype, device="cuda")
    cpa.cp_cache_append(plan, cache, batch, q if with_q else None, k, v, q_out if with_q else None)
    torch.cuda.synchronize()
    return q_out, cache


def check_append(b, q_out, cache, rope_dim, interleaved, freqs, positions=None):
    """Rows written: half a step of the result, and the fp32 work before it.
    The half-turns are off by 2^-25 (one fp32 rounding below 1, and 2^-32 of
    the fraction's cut), so the angle by pi 2^-25; sine and cosine by two fp32
    steps more; two products and a sum by three half-steps: together less than
    2^-21 (|a| + |b|).  Rows not written: bit for bit."""
    q_ref, k_ref, v_ref, q_size, k_size = b.append(rope_dim, freqs, interleaved, positions)
    n, u = b.N - b.pad, paged_ref.HALF_STEP[b.dtype]
    tiny = 2.0 ** -25 if b.dtype == torch.float16 else 0.0
    got = q_out.double().cpu().numpy()
    err = np.abs(got[:n] - q_ref[:n])
    assert np.all(err <= u * np.abs(q_ref[:n]) + 2.0 ** -21 * q_size[:n] + tiny), err.max()
    kc, vc = cache.k.cpu(), cache.v.cpu()
    written = k_size.any(axis=-1) | np.zeros(k_size.shape[:-1], bool)
    written[:] = False
    for s in range(b.B):
        for i in range(b.new[s]):
            at = b.past[s] + i
            written[b.page_table[s][at // b.ps], at % b.ps] = True
    err = np.abs(kc.double().numpy() - k_ref)[written]
    assert np.all(err <= (u * np.abs(k_ref) + 2.0 ** -21 * k_size + tiny)[written]), err.max()
    assert np.array_equal(vc.double().numpy()[written], v_ref[written])
    same = torch.from_numpy(~written)
    assert torch.equal(kc[same].view(torch.int16), b.k_cache[same].view(torch.int16))
    assert torch.equal(vc[same].view(torch.int16), b.v_cache[same].view(torch.int16))


@pytest.mark.parametrize("name", list(APPEND))
def test_append_matches_fp64(cpa, name):
    kw, plan_kw = APPEND[name]
    b = Batch(seed=len(name), appended=False, **kw)
    rd = plan_kw["rope_dim"]
    freqs = 10000.0 ** (-2.0 * np.arange(rd // 2) / max(1, rd))
    q_out, cache = run_append(cpa, b, **plan_kw)
    check_append(b, q_out, cache, rd, plan_kw.get("rope_interleaved", False), freqs)
    assert torch.isnan(q_out[b.N - b.pad:]).all()


@pytest.mark.parametrize("far", [0, 123456, 1048575, 2 ** 31 - 40])
def test_append_far_positions(cpa, far):
    b = Batch(past=[5, 100], new=[30, 2], d=128, Hq=4, Hkv=2, dtype=FP, seed=3, appended=False)
    positions = far + np.arange(b.N)
    freqs = np.linspace(1.0, 1e-6, 64)
    q_out, cache = run_append(cpa, b, positions=positions, rope_dim=128, rope_freqs=list(freqs))
    check_append(b, q_out, cache, 128, False, freqs, positions)


def test_append_backward_frequencies(cpa):
    """Negative numbers turn the other way; -1e-20 is no turn at all."""
    b = Batch(past=[5, 100], new=[30, 2], d=128, Hq=4, Hkv=2, dtype=FP, seed=5, appended=False)
    freqs = np.concatenate([np.linspace(-1.0, -1e-3, 60), [-1e-20, 0.0, 7.5, -100.0]])
    q_out, cache = run_append(cpa, b, rope_dim=128, rope_freqs=list(freqs))
    check_append(b, q_out, cache, 128, False, freqs)


def test_append_in_place_and_without_queries(cpa):
    b = Batch(past=[5, 100], new=[3, 2], d=64, Hq=4, Hkv=2, seed=4, appended=False)
    freqs = 10000.0 ** (-2.0 * np.arange(32) / 64)
    q_out, cache = run_append(cpa, b, in_place=True, rope_dim=64)
    check_append(b, q_out, cache, 64, False, freqs)
    _, other = run_append(cpa, b, with_q=False, rope_dim=64)
    assert torch.equal(other.k.view(torch.int16), cache.k.view(torch.int16))
    assert torch.equal(other.v.view(torch.int16), cache.v.view(torch.int16))
