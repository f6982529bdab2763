"""Forms of the paged-cache calls beside those of test_gpu_paged.py: one batch
rotated and attended, plans with room to spare, fp32 output and padding in every
kernel, strides with gaps, and the ends of the documented ranges."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

from paged_ref import Batch, check_attention  # noqa: E402
from test_gpu_paged import check_append, run_attention  # noqa: E402
from test_gpu_paged_use import ints, outputs  # noqa: E402

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import context_long_sequence_gb300 as m
    return m


STEPS = {
    "decode": (dict(past=[0, 15, 16, 300, 999], new=[1] * 5, d=128, Hq=8, Hkv=2), dict(rope_dim=128)),
    "drafts_far": (dict(past=[3, 64, 511], new=[5, 1, 4], d=64, Hq=8, Hkv=2, dtype=FP, heads_first=True), dict(rope_dim=32, rope_interleaved=True)),
    "prompts": (dict(past=[0, 333], new=[150, 65], d=128, Hq=8, Hkv=4, page_size=64), dict(rope_dim=64)),
    "prefix": (dict(past=[2, 0, 90], new=[1, 3, 1], prefixes=[(2, 700)], d=128, Hq=8, Hkv=2, pad=3), dict(rope_dim=128)),
    "prefix_many_rows": (dict(past=[4] * 50, new=[2] * 50, prefixes=[(30, 300), (15, 77)], d=64, Hq=8, Hkv=2), dict(rope_dim=64)),
}


@pytest.mark.parametrize("name", list(STEPS))
def test_step_rotates_and_attends(cpa, name):
    """A step as a model makes it: the append's queries and cache against fp64
    rotations, and the attention over what the append wrote against fp64."""
    kw, rope = STEPS[name]
    b = Batch(seed=31 + len(name), appended=False, **kw)
    rd = rope["rope_dim"]
    positions = 900000 + np.arange(b.N) if name == "drafts_far" else None
    plan = b.plan(cpa, **rope)
    cache, batch, q, k, v = b.to_gpu(cpa, positions)
    q_out, (o, lse) = torch.full((b.N, b.Hq, b.d), float("nan"), dtype=b.dtype, device="cuda"), outputs(plan, b.N)
    cpa.cp_cache_append(plan, cache, batch, q, k, v, q_out)
    cpa.cp_attn_paged(plan, cache, batch, q_out, o, lse, cpa.alloc_paged_workspace(plan))
    check_append(b, q_out, cache, rd, rope.get("rope_interleaved", False), 10000.0 ** (-2.0 * np.arange(rd // 2) / rd), positions)
    b.k_cache, b.v_cache = cache.k.cpu(), cache.v.cpu()
    n = b.N - b.pad
    check_attention(o, lse, b.attention(q=q_out.cpu()), b.dtype, b.d, n, name)
    assert torch.isnan(o[n:]).all() and torch.isnan(lse[:, n:]).all()


SPARE = {
    "decode": dict(past=[(37 * i) % 900 for i in range(40)], new=[1] * 40, d=128, Hq=8, Hkv=2),
    "decode_d64_fp16": dict(past=[(37 * i) % 900 for i in range(40)], new=[1] * 40, d=64, Hq=8, Hkv=2, dtype=FP),
    "decode_group_16": dict(past=[5, 800, 63], new=[1] * 3, d=128, Hq=32, Hkv=2),
    "drafts_d64": dict(past=[(53 * i) % 700 for i in range(12)], new=[5] * 12, d=64, Hq=16, Hkv=4, dtype=FP),
    "drafts": dict(past=[(53 * i) % 700 for i in range(12)], new=[1 + i % 5 for i in range(12)], d=128, Hq=8, Hkv=2),
    "one_token": dict(past=[3000], new=[1], d=128, Hq=8, Hkv=2),
    "prefix": dict(past=[5, 3, 40], new=[1, 2, 1], prefixes=[(3, 300)], d=128, Hq=8, Hkv=2),
}


@pytest.mark.parametrize("name", list(SPARE))
def test_one_plan_for_all_steps(cpa, name):
    """A plan with room to spare in every bound gives what one that fits gives,
    within the rounding of both; its tables are wider and hold anything there."""
    b = Batch(seed=41, **SPARE[name])
    ref = b.attention()
    wide = np.full((b.B, b.page_table.shape[1] + 70), 2 ** 30, np.int32)
    wide[:, :b.page_table.shape[1]] = b.page_table
    pre = np.full((len(b.plen), b.prefix_table.shape[1] + 9), -5, np.int32) if b.plen else None
    if b.plen:
        pre[:, :b.prefix_table.shape[1]] = b.prefix_table
        b.prefix_table = pre
    b.page_table = wide
    o, lse = run_attention(cpa, b, max_seqs=200, max_tokens=1024, max_new=128, max_prefixes=6,
                           max_prefix_pages=pre.shape[1] if b.plen else 40)
    check_attention(o, lse, ref, b.dtype, b.d, b.N, name)


FP32 = {
    "chunk": dict(past=[333, 100], new=[200, 65], d=128, Hq=8, Hkv=4),
    "chunk_d64_fp16": dict(past=[77, 0], new=[140, 257], d=64, Hq=6, Hkv=2, dtype=FP),
    "prefix": dict(past=[5] * 60, new=[1] * 60, prefixes=[(60, 900)], d=128, Hq=8, Hkv=1),
    "prefix_some": dict(past=[9, 90, 1, 40, 3], new=[1, 2, 1, 30, 1], prefixes=[(2, 130), (1, 17)], first=1, d=64, Hq=8, Hkv=4, dtype=FP),
    "rows_1000": dict(past=[300] * 64, new=[1] * 64, d=64, Hq=16, Hkv=2),
    "tokens_4200": dict(past=[0] * 14, new=[300] * 14, d=64, Hq=4, Hkv=2),
    "prefix_tokens": dict(past=[0] * 6, new=[200] * 6, prefixes=[(4, 300)], first=1, d=64, Hq=8, Hkv=8),
}


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "whole"])
@pytest.mark.parametrize("name", list(FP32))
def test_fp32_output_and_padding(cpa, name, causal):
    b = Batch(seed=51, pad=5, **FP32[name])
    o, lse = run_attention(cpa, b, out_fp32=True, causal=causal)
    n = b.N - 5
    check_attention(o, lse, b.attention(causal=causal), b.dtype, b.d, n, name)
    assert torch.isnan(o[n:]).all() and torch.isnan(lse[:, n:]).all()


@pytest.mark.parametrize("new", [1, 50], ids=["few_rows", "many_rows"])
@pytest.mark.parametrize("d", [64, 128])
def test_strides_with_gaps(cpa, new, d):
    """Rows of the cache and of the inputs 8 elements apart and more, q at an odd
    multiple of 16 bytes; what lies in the gaps stays as it was."""
    b = Batch(past=[100, 35], new=[new, 2], d=d, Hq=6, Hkv=2, seed=61, appended=False, prefixes=[(1, 60)])
    gap = 8

    def spread(x):  # [pages][tokens][heads][d] with a gap behind each head and token
        whole = torch.full((x.shape[0], x.shape[1], x.shape[2] * (d + gap) + gap), 7.0, dtype=x.dtype, device="cuda")
        view = whole[..., :x.shape[2] * (d + gap)].unflatten(-1, (x.shape[2], d + gap))[..., :d]
        view.copy_(x)
        return whole, view
    (kw, kc), (vw, vc) = spread(b.k_cache), spread(b.v_cache)
    rows = torch.full((b.N, 10 * d + 3 * gap), 7.0, dtype=BF, device="cuda")
    q, k, v = (rows[:, at:at + n * d].unflatten(-1, (n, d)) for at, n in ((gap, 6), (6 * d + 2 * gap, 2), (8 * d + 3 * gap, 2)))
    for x, y in ((q, b.q), (k, b.k), (v, b.v)):
        x.copy_(y)
    out = torch.full((b.N, 6 * d + gap), 7.0, dtype=BF, device="cuda")
    q2 = out[:, :6 * d].unflatten(-1, (6, d))
    plan, cache = b.plan(cpa, rope_dim=d), cpa.PagedCache(kc, vc)
    _, batch, _, _, _ = b.to_gpu(cpa)
    o, lse = outputs(plan, b.N)
    cpa.cp_cache_append(plan, cache, batch, q, k, v, q2)
    cpa.cp_attn_paged(plan, cache, batch, q2, o, lse, cpa.alloc_paged_workspace(plan))
    check_append(b, q2, cache, d, False, 10000.0 ** (-2.0 * np.arange(d // 2) / d))
    b.k_cache, b.v_cache = kc.cpu(), vc.cpu()
    check_attention(o, lse, b.attention(q=q2.cpu()), BF, d, b.N, "gaps")
    assert (out[:, 6 * d:] == 7).all()
    for whole in (kw, vw):
        assert (whole[..., 2 * (d + gap):] == 7).all()
        assert (whole[..., :2 * (d + gap)].unflatten(-1, (2, d + gap))[..., d:] == 7).all()


ENDS = {
    "largest_page": dict(past=[70000, 5], new=[1, 1], page_size=65536, d=64, Hq=2, Hkv=1, spare=0),
    "largest_page_many_rows": dict(past=[66000, 5], new=[40, 1], page_size=65536, d=64, Hq=2, Hkv=1, spare=0),
    "most_entries": dict(past=[i % 19 for i in range(8000)], new=[1] * 8000, prefixes=[(40, 1 + i) for i in range(192)], first=11,
                         d=64, Hq=1, Hkv=1),
    "group_of_128_with_prefix": dict(past=[5, 40, 0], new=[1, 3, 1], prefixes=[(2, 150)], d=64, Hq=128, Hkv=1, dtype=FP),
    "one_head": dict(past=[500, 40, 0], new=[1, 300, 20], d=128, Hq=1, Hkv=1),
    "many_kv_heads_with_prefix": dict(past=[3] * 130, new=[1] * 130, prefixes=[(130, 64)], d=64, Hq=64, Hkv=64),  # 8320 groups
    "many_kv_heads": dict(past=[3] * 130, new=[1] * 130, prefixes=[(129, 64)], first=1, d=64, Hq=66, Hkv=66, pad=2),
}


@pytest.mark.parametrize("name", list(ENDS))
def test_ends_of_the_ranges(cpa, name):
    b = Batch(seed=71, **ENDS[name])
    o, lse = run_attention(cpa, b)
    n = b.N - b.pad
    b.k_cache, b.v_cache = b.k_cache.double(), b.v_cache.double()  # once, not a sequence at a time
    check_attention(o, lse, b.attention(), b.dtype, b.d, n, name)
    assert torch.isnan(o[n:]).all() and torch.isnan(lse[:, n:]).all()


FEW = {
    "rows_4": dict(past=[47, 20, 300], new=[1] * 3, Hq=8, Hkv=2),
    "rows_8_drafts": dict(past=[37, 20], new=[2, 1], Hq=8, Hkv=2),
    "rows_16": dict(past=[47, 20], new=[1] * 2, Hq=32, Hkv=2),
    "rows_14_drafts": dict(past=[35, 20], new=[2, 1], Hq=14, Hkv=2),
    "light_prefix": dict(past=[3, 9, 20], new=[1] * 3, prefixes=[(3, 60)], Hq=32, Hkv=8),
    "beside_ctas": dict(past=[33] * 300, new=[1] * 300, prefixes=[(1, 90), (40, 3000)], first=250, Hq=4, Hkv=1),
}


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 128), (BF, 64), (FP, 64)], ids=["bf16-128", "fp16-128", "bf16-64", "fp16-64"])
@pytest.mark.parametrize("name", list(FEW))
def test_few_rows_keep_their_weights(cpa, name, dtype, d):
    """Entries of up to 16 rows by single warps: a weight's two halves leave 2^-15
    of it (bf16) or 2^-21 and 2^-34 of the largest (fp16, whose second half may be
    a subnormal number), not the half step of the type: with u the half step, the
    second is at most (2 u + s) of the weight, s 2^-14 or 2^-13, and rounded to u.  Queries are small, so that
    the scores' own error (d + 4) 2^-24 scale |q| |k| is; the sums of up to 24
    products of 16 keys and of the parts add 2^-24 each, the merge's weights 2^-21."""
    b = Batch(seed=81, dtype=dtype, d=d, **FEW[name])
    b.qkv[:, :b.Hq] *= 0.05
    o, lse = run_attention(cpa, b, out_fp32=True)
    O, LSE, A, W = b.attention()
    n = 250 if name == "beside_ctas" else b.N    # the others' prefix is the CTAs'
    ds = (d + 4) * 2.0 ** -24 * W + 2.0 ** -21
    left = (2.0 ** -7 + 2.0 ** -14) * 2.0 ** -8 if dtype == BF else (2.0 ** -10 + 2.0 ** -13) * 2.0 ** -11
    most = 2.0 ** -34 * 400 * max(float(b.v_cache.nan_to_num().abs().max()), 1.0) if dtype == FP else 0.0
    bound = 2.0 ** -24 * np.abs(O) + 1.02 * (left + 2 * ds[:, :, None] + 32 * 2.0 ** -24 + 2.0 ** -21) * A + most
    err = np.abs(o.double().cpu().numpy() - O)
    assert np.all(err[:n] <= bound[:n]), (name, (err[:n] / bound[:n]).max())


INFINITE = {
    "rows_4": (dict(past=[47, 300], new=[1, 1], Hq=8, Hkv=2), 5),
    "rows_16": (dict(past=[47, 20], new=[1, 1], Hq=32, Hkv=2), 5),
    "rows_20": (dict(past=[47, 20], new=[5, 1], Hq=8, Hkv=2), 5),
    "many_rows": (dict(past=[300, 20], new=[60, 1], Hq=8, Hkv=2), 140),
    "only_key": (dict(past=[0, 20], new=[1, 1], Hq=8, Hkv=2), 0),
}


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 128), (BF, 64), (FP, 64)], ids=["bf16-128", "fp16-128", "bf16-64", "fp16-64"])
@pytest.mark.parametrize("name", list(INFINITE))
def test_a_seen_infinity_in_v_stays_one(cpa, name, dtype, d):
    """A weight times an infinite value is that infinity, as in the formula: the
    columns that hold it, and no others, are infinite in every row that sees it."""
    kw, at = INFINITE[name]
    b = Batch(seed=91, dtype=dtype, d=d, **kw)
    page, row = int(b.page_table[0][at // 16]), at % 16
    b.v_cache[page, row, :, 3], b.v_cache[page, row, :, d - 1] = float("inf"), float("-inf")
    n = int(b.start[1])
    O, LSE, A, W = b.attention()
    assert np.isposinf(O[:n, :, 3]).all() and np.isneginf(O[:n, :, d - 1]).all()
    o, lse = run_attention(cpa, b)
    got = o.double().cpu().numpy()
    assert np.array_equal(np.isposinf(got), np.isposinf(O)) and np.array_equal(np.isneginf(got), np.isneginf(O))
    o[:n, :, 3], o[:n, :, d - 1] = 0, 0
    for x in (O, A):
        x[:n, :, 3], x[:n, :, d - 1] = 0, 0
    check_attention(o, lse, (O, LSE, A, W), dtype, d, b.N, name)
