"""Host-side checks of the paged-cache ABI that need no GPU: plan validation,
refusals, workspace size, and how a batch is shared out among the workers,
with good data and bad."""
import ctypes
import os

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def cpa():
    if not os.path.exists(os.path.join(ROOT, "context_long_sequence_gb300", "libcpattn.so")):
        from context_long_sequence_gb300 import build as b
        b.build()
    import context_long_sequence_gb300 as m
    return m


def make_plan(cpa, **kw):
    o = dict(Hq=8, Hkv=2, d=128, page_size=16, dtype=torch.bfloat16, max_seqs=4, max_tokens=64, max_new=16, max_pages=100)
    o.update(kw)
    return cpa.PagedPlan(**o)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), -2), (dict(d=256), -2), (dict(Hq=9), -1), (dict(Hkv=0), -1), (dict(Hq=0), -1),
    (dict(Hq=258, Hkv=2), -2),                                   # 129 query heads to a KV head
    (dict(page_size=8), -2), (dict(page_size=24), -2), (dict(page_size=131072), -2), (dict(page_size=0), -1),
    (dict(max_seqs=0), -1), (dict(max_tokens=0), -1), (dict(max_new=0), -1), (dict(max_pages=0), -1),
    (dict(max_seqs=8193), -1), (dict(max_seqs=8000, max_prefixes=193, max_prefix_pages=1), -1),
    (dict(max_pages=1 << 26), -1), (dict(max_prefixes=1, max_prefix_pages=1 << 26), -1),
    (dict(max_prefixes=1), -1), (dict(max_prefix_pages=1), -1), (dict(max_prefixes=-1), -1),
    (dict(max_tokens=1 << 27), -1),
    (dict(softmax_scale=-1.0), -1), (dict(softmax_scale=float("inf")), -1), (dict(softmax_scale=float("nan")), -1),
    (dict(rope_dim=24), -2), (dict(rope_dim=144), -1), (dict(rope_dim=-16), -1),
    (dict(rope_dim=32, rope_base=0.0), -1), (dict(rope_dim=32, rope_base=float("nan")), -1),
    (dict(rope_dim=32, rope_freqs=[float("inf")] * 16), -1), (dict(rope_dim=32, rope_freqs=[1.0] * 15), -1),
    (dict(dtype=torch.float32), -1),
])
def test_plan_validation(cpa, kw, code):
    with pytest.raises(cpa.CPError) as e:
        make_plan(cpa, **kw)
    assert e.value.code == code


def test_plan_null_and_version(cpa):
    L = cpa._L()
    h = ctypes.c_void_p()
    assert L.cp_paged_create(None, ctypes.byref(h)) == cpa.CP_ERR_INVALID_ARG
    assert L.cp_paged_create(ctypes.byref(cpa.cp_paged_desc_t()), ctypes.byref(h)) == cpa.CP_ERR_INVALID_ARG  # version 0
    L.cp_paged_destroy(None)


def test_workspace_size(cpa):
    def size(Hq, Hkv, d, tokens, prefixes):
        rows = 2 * 1216 * 32 + 2 * 152 * 256 + (2 * tokens * Hq if prefixes else 0)
        al = lambda x: (x + 255) // 256 * 256  # noqa: E731
        return al(2 * tokens * Hkv * 16) + al(rows * 4) + rows * d * 4
    assert make_plan(cpa).workspace_size() == size(8, 2, 128, 64, False)
    assert make_plan(cpa, d=64, max_tokens=1000, max_prefixes=2, max_prefix_pages=3).workspace_size() == size(8, 2, 64, 1000, True)


FAKE = 1 << 36


def c_args(cpa, plan, cache=None, batch=None):
    """A cache and batch of fake addresses (the checks come before any use)."""
    c = cpa.cp_paged_cache_t(FAKE, FAKE + (1 << 30), 50, 16 * 2 * 128, 2 * 128, 128)
    b = cpa.cp_paged_batch_t(2, 10, FAKE, FAKE + 64, FAKE + 128, 0, None, None, None, None)
    for k, v in (cache or {}).items():
        setattr(c, k, v)
    for k, v in (batch or {}).items():
        setattr(b, k, v)
    return c, b


BAD = [
    (dict(k=None), {}, -1), (dict(v=FAKE + 8), {}, -3), (dict(num_pages=0), {}, -1),
    (dict(head_stride=64), {}, -1), (dict(token_stride=252), {}, -1), (dict(page_stride=-4096), {}, -1),
    (dict(page_stride=4096 - 8), {}, -1),            # pages overlap
    (dict(token_stride=128, head_stride=128), {}, -1),
    (dict(token_stride=1 << 36), {}, -1),
    ({}, dict(n_seqs=5), -1), ({}, dict(n_seqs=-1), -1), ({}, dict(n_tokens=65), -1), ({}, dict(n_tokens=-1), -1),
    ({}, dict(q_start=None), -1), ({}, dict(kv_len=None), -1), ({}, dict(page_table=None), -1),
    ({}, dict(kv_len=FAKE + 2), -3), ({}, dict(positions=FAKE + 1), -3),
    ({}, dict(n_prefixes=1), -1),                    # the plan has none
]


@pytest.mark.parametrize("cache,batch,code", BAD)
def test_refusals(cpa, cache, batch, code):
    plan = make_plan(cpa, rope_dim=128)
    c, b = c_args(cpa, plan, cache, batch)
    L, A = cpa._L(), ctypes.addressof
    ws = plan.workspace_size()
    assert L.cp_attn_paged(plan.handle, A(c), A(b), FAKE, 1024, FAKE, FAKE, FAKE, ws, None) == code
    assert L.cp_cache_append(plan.handle, A(c), A(b), FAKE, 1024, FAKE, 256, FAKE, 256, FAKE, 1024, None) == code


def test_refusals_of_tensors(cpa):
    plan = make_plan(cpa, rope_dim=128)
    c, b = c_args(cpa, plan)
    L, A = cpa._L(), ctypes.addressof
    ws = plan.workspace_size()

    def attn(q=FAKE, qs=1024, o=FAKE, lse=FAKE, w=FAKE, n=ws):
        return L.cp_attn_paged(plan.handle, A(c), A(b), q, qs, o, lse, w, n, None)
    assert attn(q=None) == -1 and attn(qs=1016) == -1 and attn(qs=1028) == -1 and attn(q=FAKE + 8) == -3
    assert attn(o=None) == -1 and attn(lse=None) == -1 and attn(o=FAKE + 4) == -3 and attn(lse=FAKE + 4) == -3
    assert attn(w=None) == cpa.CP_ERR_WORKSPACE and attn(n=ws - 1) == cpa.CP_ERR_WORKSPACE and attn(w=FAKE + 8) == -3

    def append(q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, o=FAKE, os_=1024):
        return L.cp_cache_append(plan.handle, A(c), A(b), q, qs, k, ks, v, vs, o, os_, None)
    assert append(k=None) == -1 and append(v=None) == -1 and append(o=None) == -1
    assert append(ks=128) == -1 and append(vs=260) == -1 and append(k=FAKE + 2) == -3
    assert append(os_=2048) == -1                    # in place with another stride
    assert L.cp_attn_paged(None, A(c), A(b), FAKE, 1024, FAKE, FAKE, FAKE, ws, None) == -1
    assert L.cp_cache_append(plan.handle, None, A(b), None, 0, FAKE, 256, FAKE, 256, None, 0, None) == -1


def ints(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32)


def host_batch(cpa, start, kv, pages, n_tokens, first=None, plen=None, prefix_pages=0):
    pre = {} if first is None else dict(prefix_first=ints(first), prefix_len=ints(plen),
                                        prefix_table=torch.zeros(len(plen), prefix_pages, dtype=torch.int32))
    return cpa.PagedBatch(ints(start), ints(kv), torch.zeros(len(kv), pages, dtype=torch.int32), n_tokens=n_tokens, **pre)


def shares(cpa, start, kv, first=None, plen=None, Hq=8, Hkv=2, ps=16, pages=4096, prefix_pages=4096, max_new=4096, ctas=152,
           causal=True, max_tokens=None):
    B, N = len(kv), int(max(start[-1], 1))
    plan = make_plan(cpa, Hq=Hq, Hkv=Hkv, page_size=ps, max_seqs=max(B, 1), max_tokens=max_tokens or N, max_new=max_new,
                     max_pages=pages, max_prefixes=len(plen) if plen else 0, max_prefix_pages=prefix_pages if plen else 0,
                     causal=causal)
    b = host_batch(cpa, start, kv, pages, N, first, plen, prefix_pages)
    return plan, cpa.cp_paged_shares(plan, b, ctas)


def check_shares(table, start, kv, first, plen, Hq, Hkv, max_tokens, causal=True, skipped=()):
    """Every key of every entry that some token sees is in exactly one run for
    each KV head and token tile; runs of one tile follow each other; parts are
    where the records say; no two runs share a slot; the rows of the workspace
    are inside it."""
    B, G = len(kv), Hq // Hkv
    covered = set(range(first[0], first[-1])) if plen else set()
    small_rows, large_rows = 2 * 1216 * 32, 2 * 152 * 256
    home = small_rows + large_rows
    runs, slots = {}, set()
    for large, worker, e, h, t0, nt, k0, k1, mode, row, parts, r1, r2, stride in table.tolist():
        runs.setdefault((large, e, h, t0), []).append((k0, k1, worker, nt, mode, row, parts, r1, r2, stride))
        assert e not in skipped
        if mode == 2:
            assert row not in slots
            slots.add(row)
            assert row == (small_rows if large else 0) + (2 * worker + (1 if k0 == 0 else 0)) * (256 if large else 32)
            assert nt * G <= (256 if large else 32) and row < home
            assert worker < (152 if large else 1216)
        elif mode == 1:
            assert row == home + (max_tokens * Hq if e >= B else 0)
            assert e >= B or e in covered
        else:
            assert e < B and e not in covered
    seen = {}
    for (large, e, h, t0), rs in runs.items():
        rs.sort()
        nt = rs[0][3]
        a, n, keys = (start[e], start[e + 1] - start[e], kv[e]) if e < B else \
            (start[first[e - B]], start[first[e - B + 1]] - start[first[e - B]], plen[e - B])
        assert a <= t0 and t0 + nt <= a + n
        last = keys if e >= B or not causal else min(keys, keys - n + (t0 - a) + nt)
        assert rs[0][0] == 0 and rs[-1][1] >= last and all(x[1] == y[0] for x, y in zip(rs, rs[1:]))
        assert all(x[1] <= keys for x in rs)
        assert [x[2] for x in rs] == list(range(rs[0][2], rs[0][2] + len(rs)))  # consecutive workers
        assert rs[0][6] == len(rs) and all(x[6] == 0 for x in rs[1:])
        k0, k1, worker, nt, mode, row, parts, r1, r2, stride = rs[0]
        assert r1 == (row if mode == 2 else row + t0 * Hq + h * G)
        for i, x in enumerate(rs[1:]):
            assert x[4] == 2 and x[5] == r2 + i * stride
        for t in range(t0, t0 + nt):
            assert (e, h, t) not in seen
            seen[e, h, t] = True
    for e in range(B + (len(plen) if plen else 0)):
        if e in skipped:
            continue
        a, n, keys = (start[e], start[e + 1] - start[e], kv[e]) if e < B else \
            (start[first[e - B]], start[first[e - B + 1]] - start[first[e - B]], plen[e - B])
        for h in range(Hkv):
            for i in range(n):
                sees = keys if e >= B or not causal else min(keys, keys - n + i + 1)
                if sees > 0:
                    assert (e, h, a + i) in seen, (e, h, i)


def rand_batch(rng, B, new, past, P=0, plen_max=0):
    n = rng.integers(0 if new > 1 else 1, new + 1, B)
    kv = n + rng.integers(0, past + 1, B)
    start = np.concatenate([[0], np.cumsum(n)])
    first = np.sort(rng.integers(0, B + 1, P + 1)) if P else None
    return start.tolist(), kv.tolist(), (first.tolist() if P else None), (rng.integers(0, plen_max + 1, P).tolist() if P else None)


@pytest.mark.parametrize("seed", range(24))
def test_shares_cover_everything_once(cpa, seed):
    rng = np.random.default_rng(seed)
    B = int(rng.choice([1, 2, 7, 31, 32, 33, 65, 150]))
    new, past = int(rng.choice([1, 1, 3, 40, 300])), int(rng.choice([0, 5, 700, 9000]))
    if new >= 40:
        B = min(B, 7)
    P = int(rng.choice([0, 0, 1, 2, 5]))
    Hkv = int(rng.choice([1, 2, 3]))
    G = int(rng.choice([1, 4, 7, 16, 71]))
    start, kv, first, plen = rand_batch(rng, B, new, past, P, 3000)
    causal = bool(rng.random() < 0.8)
    ctas = int(rng.choice([152, 148, 5]))
    plan, t = shares(cpa, start, kv, first, plen, Hq=G * Hkv, Hkv=Hkv, causal=causal, ctas=ctas)
    check_shares(t, start, kv, first, plen, G * Hkv, Hkv, plan.max_tokens, causal)
    # Equal shares: no worker has more than its part of the units and one more.
    for large in (0, 1):
        w = t[t[:, 0] == large]
        if len(w):
            size, lead = (128, 4) if large else (16, 3)
            cost = {}
            for r in w.tolist():
                cost[r[1]] = cost.get(r[1], 0) + -(-(r[7] - r[6]) // size)
            assert max(cost.values()) <= -(-(sum(cost.values()) + (lead + 1) * len(w)) // len(cost)) + 3 * lead + 4


@pytest.mark.parametrize("Hq,new,prefix,light", [
    (8, [1] * 7, 2000, True), (8, [1] * 32, 500, True), (8, [1] * 33, 500, False), (8, [1] * 7, 80000, False),
    (18, [1] * 7, 2000, False), (8, [1] * 20 + [40], 0, False), (8, [20], 0, True)])
def test_shares_of_light_batches(cpa, Hq, new, prefix, light):
    """A batch with entries of more rows than the small workers' tiles is theirs
    all the same when it is light: few rows, few units, 8 rows a token at most."""
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    kv = [n + 30 for n in new]
    first, plen = ([0, len(new)], [prefix]) if prefix else (None, None)
    plan, t = shares(cpa, start, kv, first, plen, Hq=Hq, Hkv=2, prefix_pages=8192)
    check_shares(t, start, kv, first, plen, Hq, 2, plan.max_tokens)
    assert (t[:, 0] == 0).all() == light


def test_shares_of_a_million_keys(cpa):
    start, kv = [0, 1], [1 << 20]
    plan, t = shares(cpa, start, kv, Hq=32, Hkv=8, ps=64, pages=1 << 14)
    check_shares(t, start, kv, None, None, 32, 8, plan.max_tokens)
    assert len(set(t[:, 1])) == 1216


@pytest.mark.parametrize("what,skipped", [
    (dict(start=[0, 3, 2, 5]), {1}),                 # sequence 1 goes backwards
    (dict(start=[-1, 3, 4, 5]), {0}),
    (dict(start=[0, 3, 4, 99]), {2}),                # behind the batch's rows
    (dict(kv=[5, -1, 7]), {1}),
    (dict(kv=[5, 10 ** 9, 7]), {1}),                 # more keys than its pages hold
    (dict(max_new=2), {0}),                          # more new tokens than the plan allows
    (dict(first=[0, 5], plen=[40]), {3}),            # a prefix of sequences that are not there
    (dict(first=[2, 1], plen=[40]), {3}),
    (dict(first=[-1, 2], plen=[40]), {3}),
    (dict(first=[0, 3], plen=[-7]), {3}),
    (dict(first=[0, 3], plen=[10 ** 9]), {3}),
])
def test_shares_skip_bad_data(cpa, what, skipped):
    b = dict(start=[0, 3, 4, 5], kv=[5, 20, 700], first=None, plen=None, max_new=8)
    b.update(what)
    N = 5
    P = len(b["plen"]) if b["plen"] else 0
    plan = make_plan(cpa, max_seqs=3, max_tokens=N, max_new=b["max_new"], max_pages=64, max_prefixes=P, max_prefix_pages=64 if P else 0)
    t = cpa.cp_paged_shares(plan, host_batch(cpa, b["start"], b["kv"], 64, N, b["first"], b["plen"], 64))
    assert not set(t[:, 2].tolist()) & skipped
    good = set(range(3 + P)) - skipped
    starts_ok = all(0 <= x <= N for x in b["start"]) and b["start"] == sorted(b["start"])
    if starts_ok:
        assert set(t[:, 2].tolist()) == good
    assert (t[:, 4] >= 0).all() and (t[:, 4] + t[:, 5] <= N).all()
    assert (t[:, 6] >= 0).all() and (t[:, 7] <= 64 * 16).all()


def test_shares_refusals(cpa):
    plan = make_plan(cpa)
    b = host_batch(cpa, [0, 1], [5], 100, 1)
    n = ctypes.c_int64()
    L = cpa._L()
    assert L.cp_paged_shares(plan.handle, b.ref, 1, None, 0, ctypes.byref(n)) == -1
    assert L.cp_paged_shares(plan.handle, b.ref, 153, None, 0, ctypes.byref(n)) == -1
    assert L.cp_paged_shares(plan.handle, b.ref, 152, None, 5, ctypes.byref(n)) == -1
    assert L.cp_paged_shares(plan.handle, b.ref, 152, None, 0, None) == -1
    assert L.cp_paged_shares(None, b.ref, 152, None, 0, ctypes.byref(n)) == -1
    one = (ctypes.c_int32 * 14)()
    assert L.cp_paged_shares(plan.handle, host_batch(cpa, [0, 1], [5000], 100, 1).ref, 152, one, 1, ctypes.byref(n)) == 0
    long = host_batch(cpa, [0, 1], [1500], 100, 1)
    assert L.cp_paged_shares(plan.handle, long.ref, 152, one, 1, ctypes.byref(n)) == cpa.CP_ERR_WORKSPACE and n.value > 1


def test_empty_batches(cpa):
    """No sequences or no rows: nothing to do, whatever the pointers."""
    plan = make_plan(cpa)
    b = cpa.PagedBatch(ints([0]), ints([]), torch.zeros(0, 100, dtype=torch.int32), n_tokens=0)
    assert len(cpa.cp_paged_shares(plan, b)) == 0


def test_binding_refusals(cpa):
    plan = make_plan(cpa)
    k = torch.zeros(10, 16, 2, 128, dtype=torch.bfloat16)
    cache = cpa.PagedCache(k, k.clone())
    for bad in (dict(q_start=ints([0, 1]).long()), dict(kv_len=ints([1, 2])), dict(page_table=torch.zeros(1, 99, 2, dtype=torch.int32)),
                dict(positions=ints([1, 2])), dict(prefix_first=ints([0, 1]))):
        a = dict(q_start=ints([0, 1]), kv_len=ints([1]), page_table=torch.zeros(1, 100, dtype=torch.int32), n_tokens=1)
        a.update(bad)
        with pytest.raises(cpa.CPError):
            cpa.PagedBatch(**a)
    with pytest.raises(cpa.CPError):
        cpa.PagedCache(k, k[:, :, :, ::2])
    with pytest.raises(cpa.CPError):
        cpa.PagedCache(k, k.float())
    b = cpa.PagedBatch(ints([0, 1]), ints([1]), torch.zeros(1, 100, dtype=torch.int32), n_tokens=1)
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(cpa.CPError, match="not the current device|cpu"):   # host tensors
        cpa.cp_attn_paged(plan, cache, b, q, q.clone(), torch.zeros(8, 1))
    other = cpa.PagedBatch(ints([0, 1]), ints([1]), torch.zeros(1, 101, dtype=torch.int32), n_tokens=1)
    with pytest.raises(cpa.CPError, match="columns"):
        cpa.cp_attn_paged(plan, cache, other, q, q.clone(), torch.zeros(8, 1))
