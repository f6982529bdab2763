"""What the paged-cache operators make of the data they are given: prefixes
and pages that are not there, and frequencies of every size at far positions."""
import math
import os
import sys
from fractions import Fraction

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

import paged_ref  # noqa: E402
from paged_ref import Batch, check_attention  # noqa: E402
from test_gpu_paged import check_append, run_append  # noqa: E402
from test_gpu_paged_use import ints, outputs  # noqa: E402

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import context_long_sequence_gb300 as m
    return m


# prefix_first, prefix_len and the keys that a bad prefix leaves to each of
# four sequences of a batch with prefixes of 77 and 500 keys.
BAD_PREFIXES = {
    "negative": ([0, 2, 3], [-7, 500], [0, 0, 500, 0]),
    "too_long": ([0, 2, 3], [77, 10 ** 9], [77, 77, 0, 0]),
    "longest_int": ([0, 2, 3], [2 ** 31 - 1, 500], [0, 0, 500, 0]),
    "backwards": ([0, 3, 1], [77, 500], [77, 0, 0, 0]),       # 1 and 2 fall to a prefix of 3 .. 1
    "behind_the_batch": ([0, 2, 9], [77, 500], [77, 77, 0, 0]),
    "before_the_batch": ([-1, 2, 3], [77, 500], [0, 0, 500, 0]),
}


@pytest.mark.parametrize("name", list(BAD_PREFIXES))
def test_append_beside_a_bad_prefix(cpa, name):
    """The sequences of a bad prefix have their own keys alone, in the append
    as in the attention: their tokens are turned by their own places, the
    others' as ever, and both calls record it."""
    first, plen, before = BAD_PREFIXES[name]
    kw = dict(past=[2, 0, 9, 4], new=[1, 2, 1, 1], prefixes=[(2, 77), (1, 500)], d=64, Hq=4, Hkv=2)
    b = Batch(seed=21, appended=False, **kw)
    freqs = 10000.0 ** (-2.0 * np.arange(32) / 64)
    plan = b.plan(cpa, rope_dim=64)
    cache, _, q, k, v = b.to_gpu(cpa)
    batch = cpa.PagedBatch(ints(b.start), ints(b.kv), ints(b.page_table), n_tokens=b.N, prefix_first=ints(first),
                           prefix_len=ints(plen), prefix_table=ints(b.prefix_table))
    q_out, (o, lse) = torch.full((b.N, 4, 64), float("nan"), dtype=BF, device="cuda"), outputs(plan, b.N)
    cpa.cp_cache_append(plan, cache, batch, q, k, v, q_out)
    rec = cpa.cp_get_status_detail()
    assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 6
    positions = np.concatenate([before[s] + b.past[s] + np.arange(b.new[s]) for s in range(4)])
    check_append(b, q_out, cache, 64, False, freqs, positions)
    cpa.cp_attn_paged(plan, cache, batch, q_out, o, lse, cpa.alloc_paged_workspace(plan))
    rec = cpa.cp_get_status_detail()
    assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 7
    b.of = [-1 if n == 0 else [77, 500].index(n) for n in before]
    ref = b.attention(q=q_out.cpu(), k_cache=cache.k.cpu(), v_cache=cache.v.cpu())
    check_attention(o, lse, ref, BF, 64, b.N, name)


def test_append_with_positions_asks_no_prefix(cpa):
    """Tokens that are placed by the caller, or not turned, need no prefix."""
    b = Batch(past=[2, 0], new=[1, 2], prefixes=[(2, 77)], d=64, Hq=4, Hkv=2, seed=22, appended=False)
    b.plen = [-7]
    freqs = 10000.0 ** (-2.0 * np.arange(32) / 64)
    positions = np.array([5, 900, 901])
    q_out, cache = run_append(cpa, b, positions=positions, rope_dim=64)
    check_append(b, q_out, cache, 64, False, freqs, positions)
    run_append(cpa, b, rope_dim=0)
    assert cpa.cp_get_status_detail()[0] == 0


WITHOUT_PAGES = {
    "few_rows": dict(past=[200, 60], new=[1, 1], d=128, Hq=8, Hkv=2),
    "many_rows": dict(past=[200, 60], new=[30, 1], d=64, Hq=8, Hkv=2),
    "many_rows_d128": dict(past=[300, 9], new=[70, 5], d=128, Hq=8, Hkv=2, page_size=32),
    "prefix": dict(past=[3, 4, 5], new=[1, 1, 1], prefixes=[(3, 200)], d=128, Hq=32, Hkv=2),
}


@pytest.mark.parametrize("page", [-1, -2, -3, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("name", list(WITHOUT_PAGES))
def test_every_page_that_is_not_there_is_recorded(cpa, name, page):
    """A page number outside the cache takes its keys out of the softmax and is
    recorded, whatever the number."""
    b = Batch(seed=23, **WITHOUT_PAGES[name])
    table = b.prefix_table if b.plen else b.page_table
    table[0][2] = page
    plan = b.plan(cpa)
    cache, batch, q, _, _ = b.to_gpu(cpa)
    o, lse = outputs(plan, b.N)
    cpa.cp_attn_paged(plan, cache, batch, q, o, lse, cpa.alloc_paged_workspace(plan))
    rec = cpa.cp_get_status_detail()
    assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 7
    table[0][2] = 0
    gone = range(2 * b.ps, 3 * b.ps)
    keys = b.prefix_keys(0) if b.plen else b.keys_of(0)
    left = [np.delete(x, gone, axis=0) for x in keys]
    if b.plen:
        b.prefix_keys = lambda p: left
    else:
        full, of = list(b.kv), Batch.keys_of
        b.kv = [full[0] - b.ps] + full[1:]
        b.keys_of = lambda s, *a: left if s == 0 else of(b, s, *a)
    check_attention(o, lse, b.attention(), BF, b.d, b.N, name)


# pi to 77 decimal places.
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620, 10 ** 77)


@pytest.mark.parametrize("far", [1000, 1048575, 2 ** 31 - 40])
def test_append_far_positions_of_any_frequency(cpa, far):
    """Angles of frequencies from 1e-30 to 2^40 at far positions, against
    fractions of a turn in whole numbers.  A pair's share of a turn is held to
    2^-63 or better (two roundings of 2^-64 each), times the position less than
    2^-32 of a turn; the bound is check_append's, whose largest part is the
    conversion to fp32."""
    b = Batch(past=[5, 100], new=[30, 2], d=128, Hq=4, Hkv=2, dtype=FP, seed=24, appended=False)
    positions = far + np.arange(b.N)
    freqs = np.concatenate([np.geomspace(1.0, 1e4, 30), -np.geomspace(1.0, 300.0, 20), np.geomspace(1e4, 2.0 ** 40, 9),
                            [1e-30, -1e-30, 0.25, 0.5, 2 * math.pi]])
    q_out, cache = run_append(cpa, b, positions=positions, rope_dim=128, rope_freqs=[float(f) for f in freqs])
    turns = np.array([[float(Fraction(int(p)) * Fraction(float(f)) / (2 * PI) % 1) for f in freqs] for p in positions])
    c, s = np.cos(2 * math.pi * turns), np.sin(2 * math.pi * turns)
    u = paged_ref.HALF_STEP[FP]

    def check(got, x, t):
        a, z = x[:, :64], x[:, 64:]
        ref = np.concatenate([a * c[t] - z * s[t], z * c[t] + a * s[t]], axis=1)
        size = np.tile(np.abs(a) + np.abs(z), (1, 2))
        err = np.abs(got.double().cpu().numpy() - ref)
        bound = u * np.abs(ref) + 2.0 ** -21 * size + 2.0 ** -25
        assert np.all(err <= bound), (t, (err / bound).max(), np.argwhere(err > bound)[:3].tolist())
    for sq in range(2):
        for i in range(b.new[sq]):
            t, at = int(b.start[sq]) + i, b.past[sq] + i
            check(q_out[t], b.q[t].double().numpy(), t)
            check(cache.k[int(b.page_table[sq][at // 16]), at % 16], b.k[t].double().numpy(), t)
