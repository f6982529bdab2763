"""The paged-cache operators as a serving program uses them: prompts and
tokens step by step against the whole-sequence forward, context-parallel
shares merged, captured and replayed steps, streams, bad data, far offsets,
scores that jump, and bitwise repeatability."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

import paged_ref  # noqa: E402
from paged_ref import Batch, check_attention  # noqa: E402
from test_gpu_paged import run_attention  # noqa: E402

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import context_long_sequence_gb300 as m
    return m


def ints(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def outputs(plan, b_tokens):
    return (torch.full((b_tokens, plan.Hq, plan.d), float("nan"), dtype=plan.o_dtype, device="cuda"),
            torch.full((plan.Hq, b_tokens), float("nan"), device="cuda"))


def test_prompt_and_steps_equal_the_whole_forward(cpa):
    """A prompt, a chunk, and single tokens appended and attended one after
    another give the rows of cp_attn_fwd over the whole sequence (no rotation
    there, so none here).  Both round P and O once: twice the bound of one."""
    L, Hq, Hkv, d, ps = 700, 8, 2, 128, 16
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(L, h, d, generator=gen).to(BF).cuda() for h in (Hq, Hkv, Hkv))
    whole = cpa.Plan(L, Hq, Hkv, d)
    o_ref = torch.empty_like(q)
    lse_ref = torch.empty(1, Hq, L, device="cuda")
    cpa.cp_attn_fwd(whole, q, k, v, o_ref, lse_ref, cpa.alloc_workspace(whole))
    pages = -(-L // ps)
    plan = cpa.PagedPlan(Hq, Hkv, d, page_size=ps, dtype=BF, max_seqs=1, max_tokens=L, max_new=L, max_pages=pages)
    cache = cpa.PagedCache(*(torch.full((pages + 2, ps, Hkv, d), float("nan"), dtype=BF, device="cuda") for _ in range(2)))
    table = ints(np.random.default_rng(0).permutation(pages + 2)[:pages][None])
    ws = cpa.alloc_paged_workspace(plan)
    o, lse = torch.empty_like(q), torch.empty(Hq, L, device="cuda")
    at = 0
    for n in [300, 1, 1, 5, 200] + [1] * 193:
        b = cpa.PagedBatch(ints([0, n]), ints([at + n]), table, n_tokens=n)
        os_, ls = outputs(plan, n)
        cpa.cp_cache_append(plan, cache, b, None, k[at:at + n], v[at:at + n])
        cpa.cp_attn_paged(plan, cache, b, q[at:at + n], os_, ls, ws)
        o[at:at + n], lse[:, at:at + n] = os_, ls
        at += n
    assert at == L
    assert torch.equal(cache.k[table[0].long()].reshape(-1, Hkv, d)[:L], k)
    A = torch.stack([v[:i + 1].float().abs().mean(0) for i in (0, L - 1)]).max()
    assert (o.float() - o_ref.float()).abs().max() <= 2 * 2.0 ** -8 * (o_ref.float().abs().max() + A) * 1.1
    assert (lse - lse_ref[0]).abs().max() <= 1e-3


def test_context_parallel_shares_merge(cpa):
    """Four ranks hold pieces of a sequence's keys; each attends its share
    (fp32, not causal but for the last) and cp_merge_lse joins them."""
    Hq, Hkv, d, ps, n = 8, 2, 64, 32, 3
    b = Batch(past=[997], new=[n], page_size=ps, Hq=Hq, Hkv=Hkv, d=d, seed=11)
    cuts = [0, 256, 512, 800, 1000]
    k, v = b.keys_of(0)
    q = b.q.cuda()
    parts, lses = [], []
    for r in range(4):
        keys = cuts[r + 1] - cuts[r]
        pages = -(-keys // ps)
        cache = []
        for x in (k, v):
            c = torch.full((pages, ps, Hkv, d), float("nan"), dtype=BF)
            c.reshape(-1, Hkv, d)[:keys] = torch.from_numpy(x[cuts[r]:cuts[r + 1]]).to(BF)
            cache.append(c.cuda())
        plan = cpa.PagedPlan(Hq, Hkv, d, page_size=ps, dtype=BF, max_seqs=1, max_tokens=n, max_new=n, max_pages=pages,
                             causal=r == 3, out_fp32=True)
        batch = cpa.PagedBatch(ints([0, n]), ints([keys]), ints(np.arange(pages)[None]), n_tokens=n)
        o, lse = outputs(plan, n)
        cpa.cp_attn_paged(plan, cpa.PagedCache(*cache), batch, q, o, lse, cpa.alloc_paged_workspace(plan))
        parts.append(o)
        lses.append(lse)
    out = torch.empty(n, Hq, d, dtype=BF, device="cuda")
    lse = torch.empty(Hq, n, device="cuda")
    cpa.cp_merge_lse(4, n, Hq, d, torch.stack(parts), torch.stack(lses), out, lse)
    check_attention(out, lse, b.attention(), BF, d, n, "shares")


def test_shared_prefix_equals_its_copies(cpa):
    """A prefix held once gives what copies of it before each sequence give,
    within the rounding of P (both sides)."""
    kw = dict(d=128, Hq=8, Hkv=2, seed=3)
    b = Batch(past=[10, 0, 77], new=[1, 2, 1], prefixes=[(3, 650)], **kw)
    o, lse = run_attention(cpa, b)
    ref = b.attention()
    check_attention(o, lse, ref, BF, 128, b.N, "shared")
    alone = Batch(past=[660, 650, 727], new=[1, 2, 1], **kw)
    for s in range(3):
        rows = alone.page_table[s]
        j = np.arange(alone.kv[s])
        for c, pre, own in zip((alone.k_cache, alone.v_cache), b.prefix_keys(0), b.keys_of(s)):
            c[torch.from_numpy(rows[j // 16].astype(np.int64)), torch.from_numpy(j % 16)] = torch.from_numpy(np.concatenate([pre, own])).to(BF)
    o2, lse2 = run_attention(cpa, alone, q=b.qkv.cuda()[:, :8])
    check_attention(o2, lse2, ref, BF, 128, b.N, "copies")
    assert (lse - lse2).abs().max() < 1e-5


MANY = {
    "decode": dict(past=[(i * 37) % 400 for i in range(300)], new=[1] * 300, d=64, Hq=4, Hkv=2),
    "drafts": dict(past=[(i * 53) % 200 for i in range(70)], new=[1 + i % 4 for i in range(70)], d=128, Hq=8, Hkv=2),
    "prefixes": dict(past=[(i * 37) % 90 for i in range(130)], new=[1] * 130, d=128, Hq=8, Hkv=2,
                     prefixes=[(5 + i % 3, 40 * i) for i in range(20)], first=3),
}


@pytest.mark.parametrize("name", list(MANY))
def test_many_sequences(cpa, name):
    """More entries than a warp's window of 32."""
    b = Batch(seed=1, **MANY[name])
    o, lse = run_attention(cpa, b)
    check_attention(o, lse, b.attention(), b.dtype, b.d, b.N, name)


def test_rows_that_see_nothing(cpa):
    """Fewer keys than new tokens: the first rows see none, in both kernels."""
    for new, G in ((5, 2), (150, 4)):
        b = Batch(past=[-(new - 2), 3], new=[new, 1], d=64, Hq=2 * G, Hkv=2, seed=2)
        o, lse = run_attention(cpa, b)
        check_attention(o, lse, b.attention(), b.dtype, b.d, b.N, "nothing")
        assert (o[:new - 2] == 0).all() and torch.isneginf(lse[:, :new - 2]).all()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("new", [1, 40], ids=["few_rows", "many_rows"])
def test_scores_that_jump(cpa, dtype, new):
    """Keys whose scores exceed all before them by up to 2^30 and more, in a
    tile's first or second half, and scores that fall off again."""
    b = Batch(past=[900, 300], new=[new, new], d=128, Hq=8, Hkv=2, dtype=dtype, seed=4)
    q = b.qkv[:, :8]
    q[:] = q * 0.2 + 1.0
    for s in range(2):
        for at, size in ((3, 0.5), (70, 1.0), (140, 1.7), (200, 2.6), (299, 0.2), (650, 3.5)):
            if at < b.past[s]:
                page, row = b.page_table[s][at // 16], at % 16
                b.k_cache[page, row] = (b.k_cache[page, row].float() * 0.1 + size).to(dtype)
    o, lse = run_attention(cpa, b)
    check_attention(o, lse, b.attention(), dtype, 128, b.N, "jumps")


@pytest.mark.parametrize("new", [1, 40], ids=["few_rows", "many_rows"])
def test_fp16_flat_tail(cpa, new):
    """One key far above thousands of equal ones: in fp16 the many small
    weights must not vanish beside the large one."""
    b = Batch(past=[20000], new=[new], d=64, Hq=4, Hkv=1, dtype=FP, seed=9, page_size=64)
    rows = b.page_table[0]
    j = np.arange(b.kv[0])
    page, row = torch.from_numpy(rows[j // 64].astype(np.int64)), torch.from_numpy(j % 64)
    b.k_cache[page, row] = 0.0
    b.k_cache[rows[0], 0] = 1.4                     # score 1.4 * 64 / 8 = 11.2 over the tail's: e^11.2 = 73,000
    b.v_cache[page, row] = 1.0 + 0.01 * b.v_cache[page, row].float().half()
    b.v_cache[rows[0], 0] = -1.0
    b.qkv[:, :4] = 1.0
    o, lse = run_attention(cpa, b)
    check_attention(o, lse, b.attention(), FP, 64, b.N, "flat tail")


def test_deterministic(cpa):
    for kw in (dict(past=[5000, 100, 0, 777], new=[1] * 4, d=128, Hq=8, Hkv=2),
               dict(past=[3] * 40, new=[1] * 40, prefixes=[(40, 2000)], d=128, Hq=8, Hkv=2),
               dict(past=[500, 0], new=[130, 300], d=64, Hq=8, Hkv=4)):
        b = Batch(seed=8, **kw)
        first = run_attention(cpa, b)
        for _ in range(3):
            again = run_attention(cpa, b)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_interleaved_caches_and_strided_queries(cpa):
    """K and V side by side in one buffer, queries as a slice of a projection."""
    b = Batch(past=[100, 35], new=[2, 1], d=64, Hq=4, Hkv=2, seed=6)
    both = torch.empty(b.pages, 2, 16, 2, 64, dtype=BF, device="cuda")
    both[:, 0], both[:, 1] = b.k_cache.cuda(), b.v_cache.cuda()
    _, batch, q, _, _ = b.to_gpu(cpa)
    plan = b.plan(cpa)
    o, lse = outputs(plan, b.N)
    cpa.cp_attn_paged(plan, cpa.PagedCache(both[:, 0], both[:, 1]), batch, q, o, lse, cpa.alloc_paged_workspace(plan))
    check_attention(o, lse, b.attention(), BF, 64, b.N, "interleaved")


def test_captured_step_follows_its_arrays(cpa):
    """One graph of append + attention, replayed while lengths, pages and
    tokens change under it; a second graph shares the workspace."""
    Hq, Hkv, d, ps, B = 8, 2, 128, 16, 5
    rng = np.random.default_rng(1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    pages = 100
    plan = cpa.PagedPlan(Hq, Hkv, d, page_size=ps, dtype=BF, max_seqs=B, max_tokens=B, max_new=1, max_pages=20, max_prefixes=1,
                         max_prefix_pages=20, rope_dim=128)
    kc, vc = (torch.randn(pages, ps, Hkv, d, generator=gen, device="cuda").to(BF) for _ in range(2))
    cache = cpa.PagedCache(kc, vc)
    table = ints(rng.permutation(pages)[:B * 10].reshape(B, 10).repeat(2, 1))
    kv, start = ints([1] * B), ints(np.arange(B + 1))
    batch = cpa.PagedBatch(start, kv, table, n_tokens=B, prefix_first=ints([0, 3]), prefix_len=ints([33]),
                           prefix_table=ints(rng.permutation(pages)[:20][None]))
    qkv = torch.empty(B, Hq + 2 * Hkv, d, dtype=BF, device="cuda")
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    q2, (o, lse) = torch.empty(B, Hq, d, dtype=BF, device="cuda"), outputs(plan, B)
    ws = cpa.alloc_paged_workspace(plan)

    def step():
        cpa.cp_cache_append(plan, cache, batch, q, k, v, q2)
        cpa.cp_attn_paged(plan, cache, batch, q2, o, lse, ws)
    qkv.normal_(generator=gen)
    step()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for i in range(6):
        kv.copy_(ints(rng.integers(1, 150, B)))
        table.copy_(ints(rng.permutation(pages)[:B * 10].reshape(B, 10).repeat(2, 1)))
        qkv.normal_(generator=gen)
        saved = kc.clone(), vc.clone()
        graphs[i % 2].replay()
        got = o.clone(), lse.clone(), kc.clone(), vc.clone(), q2.clone()
        kc.copy_(saved[0])
        vc.copy_(saved[1])
        step()
        for x, y in zip(got, (o, lse, kc, vc, q2)):
            assert torch.equal(x, y), i


def test_streams(cpa):
    """Two calls at once, each with a stream and a workspace of its own, and
    one on a stream that its tensors were not made on."""
    bs = [Batch(past=[3000, 50], new=[1, 1], d=128, Hq=8, Hkv=2, seed=s) for s in (1, 2)]
    ready = []
    for b in bs:
        plan = b.plan(cpa)
        cache, batch, q, _, _ = b.to_gpu(cpa)
        ready.append((plan, cache, batch, q, outputs(plan, b.N), cpa.alloc_paged_workspace(plan)))
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (plan, cache, batch, q, (o, lse), ws) in zip(streams, ready):
            cpa.cp_attn_paged(plan, cache, batch, q, o, lse, ws, stream=st)
    torch.cuda.synchronize()
    for b, (_, _, _, _, (o, lse), _) in zip(bs, ready):
        check_attention(o, lse, b.attention(), BF, 128, b.N, "streams")


def test_offsets_beyond_32_bits(cpa):
    """Pages whose element offsets pass 2^31 and byte offsets 2^32."""
    ps, Hkv, d, Hq = 64, 8, 128, 32
    pages = (1 << 31) // (ps * Hkv * d) + 300      # 2.15e9 elements
    kc = torch.zeros(pages, ps, Hkv, d, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    b = Batch(past=[200, 130], new=[2, 1], page_size=ps, Hq=Hq, Hkv=Hkv, d=d, seed=7, spare=0)
    move = pages - 1 - np.arange(b.pages)          # the batch's pages at the far end
    kc[torch.from_numpy(move).cuda()] = b.k_cache.cuda()
    vc[torch.from_numpy(move).cuda()] = b.v_cache.cuda()
    table = np.where(b.page_table >= 0, move[b.page_table], -1)
    plan = b.plan(cpa, rope_dim=128)
    batch = cpa.PagedBatch(ints(b.start), ints(b.kv), ints(table), n_tokens=b.N)
    qkv = b.qkv.cuda()
    o, lse = outputs(plan, b.N)
    cache = cpa.PagedCache(kc, vc)
    cpa.cp_attn_paged(plan, cache, batch, qkv[:, :Hq], o, lse, cpa.alloc_paged_workspace(plan))
    check_attention(o, lse, b.attention(), BF, d, b.N, "far")
    q2 = torch.empty_like(o)
    cpa.cp_cache_append(plan, cache, batch, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], q2)
    for s in range(2):
        at = b.past[s]
        assert torch.equal(vc[int(table[s][at // ps]), at % ps].cpu(), b.v[int(b.start[s])])
    assert kc[:1000].abs().max() == 0


def test_bad_pages_are_left_out(cpa):
    """Page numbers that are not the cache's: their keys take no part, nothing
    is read or written through them, and the record says so."""
    for kw in (dict(past=[200, 60], new=[1, 1], d=128, Hq=8, Hkv=2), dict(past=[200, 60], new=[30, 1], d=64, Hq=8, Hkv=2),
               dict(past=[3, 4, 5], new=[1, 1, 1], prefixes=[(3, 200)], d=128, Hq=32, Hkv=2)):
        b = Batch(seed=12, **kw)
        table = b.prefix_table if b.plen else b.page_table
        table[0][2], table[0][5] = b.pages, -7        # 32 keys of entry 0
        gone = np.r_[32:48, 80:96]
        plan = b.plan(cpa)
        cache, batch, q, _, _ = b.to_gpu(cpa)
        o, lse = outputs(plan, b.N)
        assert cpa.cp_get_status_detail()[0] == 0
        cpa.cp_attn_paged(plan, cache, batch, q, o, lse, cpa.alloc_paged_workspace(plan))
        rec = cpa.cp_get_status_detail()
        assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 7
        table[0][2] = table[0][5] = 0
        keep_of = lambda n: np.setdiff1d(np.arange(n), gone)  # noqa: E731
        own, pre = Batch.keys_of, Batch.prefix_keys
        # The reference without those keys: drop them, keep the causal places.
        if b.plen:
            b.prefix_keys = lambda p: [x[keep_of(b.plen[p])] for x in pre(b, p)]
            ref = b.attention()
        else:
            saved = list(b.kv), list(b.past)
            b.keys_of = lambda s, *a: [x[keep_of(len(x))] if s == 0 else x for x in _full(own, b, s, saved[0])]
            b.kv = [b.kv[0] - 32] + b.kv[1:]
            b.past = [b.past[0] - 32] + b.past[1:]
            ref = b.attention()
        check_attention(o, lse, ref, BF, b.d, b.N, "bad pages")


def _full(own, b, s, kv):
    held, b.kv = b.kv, kv
    try:
        return own(b, s)
    finally:
        b.kv = held


@pytest.mark.parametrize("what", ["backwards", "too_long", "too_many_new", "negative"])
def test_bad_sequences_are_skipped(cpa, what):
    b = Batch(past=[20, 30, 40], new=[1, 2, 1], d=64, Hq=4, Hkv=2, seed=13, appended=True)
    ref = b.attention()
    start, kv = b.start.copy(), np.array(b.kv)
    plan = b.plan(cpa, rope_dim=64, max_new=1 if what == "too_many_new" else 2)
    if what == "too_long":
        kv[1] = b.page_table.shape[1] * 16 + 1
    elif what == "negative":
        kv[1] = -1
    elif what == "backwards":
        start = np.array([0, 3, 2, 4], dtype=np.int32)    # sequence 0 takes three rows, 1 none that exist, 2 the last two
    cache, _, q, k, v = b.to_gpu(cpa)
    batch = cpa.PagedBatch(ints(start), ints(kv), ints(b.page_table), n_tokens=b.N)
    o, lse = outputs(plan, b.N)
    cpa.cp_attn_paged(plan, cache, batch, q, o, lse, cpa.alloc_paged_workspace(plan))
    rec = cpa.cp_get_status_detail()
    assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 7
    before = cache.k.clone(), cache.v.clone()
    if what == "backwards":
        return
    assert torch.isnan(o[1:3]).all() and torch.isnan(lse[:, 1:3]).all()
    for t in (0, 3):
        got = o[t:t + 1], lse[:, t:t + 1]
        check_attention(*got, tuple(x[t:t + 1] if i != 1 else x[:, t:t + 1] for i, x in enumerate(ref)), BF, 64, 1, what)
    q2 = torch.full_like(o, float("nan"))
    cpa.cp_cache_append(plan, cache, batch, q, k, v, q2)
    rec = cpa.cp_get_status_detail()
    assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 6
    assert torch.isnan(q2[1:3]).all() and not torch.isnan(q2[0]).any() and not torch.isnan(q2[3]).any()
    mine = torch.from_numpy(b.page_table[1][b.page_table[1] >= 0].astype(np.int64)).cuda()
    for x, y in zip(before, (cache.k, cache.v)):
        assert torch.equal(x[mine].view(torch.int16), y[mine].view(torch.int16))


@pytest.mark.parametrize("new", [1, 20, 70])
def test_overlapping_entries(cpa, new):
    """Prefixes or sequences out of order, so that some overlap and some rows
    have no part of this call's: nothing outside the workspace is read (it
    holds other numbers before), and whatever stands apart is right."""
    b = Batch(past=[20, 3, 64] * 4, new=[new] * 12, prefixes=[(2, 100), (3, 50), (2, 300), (3, 20)], d=64, Hq=4, Hkv=2, seed=15)
    ref = b.attention()
    plan = b.plan(cpa, max_new=2 * new)
    cache, _, q, _, _ = b.to_gpu(cpa)
    pre = ints([100, 50, 300, 20]), ints(b.prefix_table)
    for first, start in (([0, 9, 1, 2, 10], b.start), ([0, 10, 3, 5, 10], b.start),
                         (b.first, np.r_[0, new + new // 2, new, b.start[3:]])):
        batch = cpa.PagedBatch(ints(start), ints(b.kv), ints(b.page_table), n_tokens=b.N, prefix_first=ints(first),
                               prefix_len=pre[0], prefix_table=pre[1])
        o, lse = outputs(plan, b.N)
        ws = cpa.alloc_paged_workspace(plan)
        for fill in (0x7f, 0xff, 0x81):
            ws.fill_(fill)
            cpa.cp_attn_paged(plan, cache, batch, q, o, lse, ws)
            rec = cpa.cp_get_status_detail()
            assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS or (new == 1 and first is b.first)  # those rows are in order
        at = 10 * new                                    # sequences 10 and 11 have no prefix in any of these
        check_attention(o[at:], lse[:, at:], tuple(x[at:] if i != 1 else x[:, at:] for i, x in enumerate(ref)), BF, 64, 2 * new, "apart")


@pytest.mark.parametrize("where", ["few_rows", "one_part", "many_rows", "prefix", "many_rows_prefix"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_seen_nan_reaches_the_result(cpa, where, bad):
    """A key that is not a number makes the rows that see it so, O and LSE, in
    whichever part of a row it lies; no other sequence's."""
    kw = {"few_rows": dict(past=[2000, 300], new=[1, 1], Hq=8, Hkv=2), "one_part": dict(past=[20, 30], new=[1, 1], Hq=4, Hkv=2),
          "many_rows": dict(past=[900, 100], new=[60, 1], Hq=8, Hkv=2),
          "prefix": dict(past=[5, 3, 7], new=[1, 1, 1], prefixes=[(2, 400)], Hq=8, Hkv=2),
          "many_rows_prefix": dict(past=[5] * 20 + [7], new=[1] * 21, prefixes=[(20, 400)], Hq=16, Hkv=2)}[where]
    b = Batch(d=128, seed=16, **kw)
    if b.plen:
        hit, row = int(b.start[b.first[1]]), (b.prefix_table[0][6], 3)
    else:
        hit, row = int(b.start[1]), (b.page_table[0][1], 3)
    ref = b.attention()
    b.k_cache[int(row[0]), int(row[1])] = bad
    plan = b.plan(cpa)
    cache, batch, q, _, _ = b.to_gpu(cpa)
    o, lse = outputs(plan, b.N)
    o.zero_(), lse.zero_()
    cpa.cp_attn_paged(plan, cache, batch, q, o, lse, cpa.alloc_paged_workspace(plan))
    assert torch.isnan(o[:hit]).all() and torch.isnan(lse[:, :hit]).all()
    check_attention(o[hit:], lse[:, hit:], tuple(x[hit:] if i != 1 else x[:, hit:] for i, x in enumerate(ref)), BF, 128, b.N - hit, where)


def test_append_beyond_the_pages_and_before_the_first(cpa):
    """A new token whose page is not the cache's, and one that would lie before
    the sequence's first key, are not written."""
    b = Batch(past=[16, 5], new=[1, 1], d=64, Hq=4, Hkv=2, seed=14)
    b.page_table[0][1] = b.pages + 5
    plan = b.plan(cpa, rope_dim=64, max_new=3)
    cache, _, q, k, v = b.to_gpu(cpa)
    before = cache.k.clone()
    batch = cpa.PagedBatch(ints(b.start), ints([17, 0]), ints(b.page_table), n_tokens=2)
    q2 = torch.full((2, 4, 64), float("nan"), dtype=BF, device="cuda")
    cpa.cp_cache_append(plan, cache, batch, q, k, v, q2)
    assert cpa.cp_get_status_detail()[0] == cpa.CP_ERR_DEVICE_BOUNDS
    assert torch.equal(cache.k.view(torch.int16), before.view(torch.int16)) and torch.isnan(q2).all()


def test_empty_calls(cpa):
    plan = cpa.PagedPlan(4, 2, 64, page_size=16, dtype=BF, max_seqs=2, max_tokens=4, max_new=2, max_pages=3)
    cache = cpa.PagedCache(*(torch.zeros(3, 16, 2, 64, dtype=BF, device="cuda") for _ in range(2)))
    none = cpa.PagedBatch(ints([0]), ints(np.zeros(0)), torch.zeros(0, 3, dtype=torch.int32, device="cuda"), n_tokens=0)
    o, lse = outputs(plan, 0)
    cpa.cp_attn_paged(plan, cache, none, torch.empty(0, 4, 64, dtype=BF, device="cuda"), o, lse, cpa.alloc_paged_workspace(plan))
    pad = cpa.PagedBatch(ints([0, 0]), ints([0]), torch.zeros(1, 3, dtype=torch.int32, device="cuda"), n_tokens=4)
    q = torch.randn(4, 4, 64, device="cuda").to(BF)
    o, lse = outputs(plan, 4)
    cpa.cp_attn_paged(plan, cache, pad, q, o, lse, cpa.alloc_paged_workspace(plan))
    assert torch.isnan(o).all() and torch.isnan(lse).all()
