"""The pages of a cache (cp_pages_resize, cp_pages_fork, cp_pages_compact,
cp_pages_copy) against a page-by-page implementation."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

from serving_ref import Pool, Table  # noqa: E402
from test_gpu_paged_use import ints  # noqa: E402

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import context_long_sequence_gb300 as m
    return m


def plan_of(cpa, ps, Hkv=2, d=64, dtype=BF):
    return cpa.PagedPlan(2 * Hkv, Hkv, d, page_size=ps, dtype=dtype, max_seqs=8, max_tokens=8, max_new=1, max_pages=4)


class Both:
    """A pool and its tables on the GPU, and the same on the CPU."""

    def __init__(self, cpa, pages, ps, *shapes, seed=0, taken=0.0):
        self.cpa, self.rng = cpa, np.random.default_rng(seed)
        self.pool, self.ref = Pool(pages, ps), [Table(*s) for s in shapes]
        if taken:  # pages that others hold
            self.pool.refs[self.rng.random(pages) < taken] = 2
        self.plan, self.refs = plan_of(cpa, ps), ints(self.pool.refs)
        self.tables = [cpa.PageTable(ints(t.pages), ints(t.held)) for t in self.ref]
        self.moves = cpa.PageMoves(max(pages // 2, *[s[0] for s in shapes]))
        self.ws = cpa.alloc_pages_workspace(pages)

    def served(self, k):
        return torch.full((len(self.ref[k].held),), -7, dtype=torch.int32, device="cuda")

    def check(self, what=""):
        assert np.array_equal(self.refs.cpu().numpy(), self.pool.refs), what
        for t, r in zip(self.tables, self.ref):
            assert np.array_equal(t.held.cpu().numpy(), r.held), what
            got, mine = t.pages.cpu().numpy(), np.arange(r.pages.shape[1])[None] < r.held[:, None]
            assert np.array_equal(got[mine], r.pages[mine]), what

    def check_moves(self, moves, what=""):
        n = self.moves.count.item()
        assert n == len(moves), what
        got = torch.stack([self.moves.src, self.moves.dst, self.moves.tokens])[:, :n].cpu().numpy().T
        assert np.array_equal(got, np.array(moves, dtype=np.int64).reshape(-1, 3)), what

    def resize(self, tokens, k=0):
        out = self.served(k)
        self.cpa.cp_pages_resize(self.plan, self.refs, self.tables[k], ints(tokens), out)
        want = self.pool.resize(self.ref[k], tokens)
        assert out.tolist() == want
        self.check("resize")
        return want

    def fork(self, parent, tokens, src=0, dst=0):
        out = self.served(dst)
        self.cpa.cp_pages_fork(self.plan, self.refs, self.tables[src], self.tables[dst], ints(parent), ints(tokens), self.moves, out)
        want, moves = self.pool.fork(self.ref[src], self.ref[dst], parent, tokens)
        assert out.tolist() == want
        self.check("fork")
        self.check_moves(moves, "fork")
        return want

    def compact(self):
        used = torch.full((1,), -7, dtype=torch.int32, device="cuda")
        # Beside: out of place, which leaves the state as it was.
        refs_out, outs = torch.full_like(self.refs, -7), [self.cpa.PageTable(t.pages.clone(), t.held.clone()) for t in self.tables]
        before = [self.refs.clone()] + [t.pages.clone() for t in self.tables]
        self.cpa.cp_pages_compact(self.plan, self.refs, self.tables, self.moves, self.ws, refs_out=refs_out, tables_out=outs)
        assert all(torch.equal(a, b) for a, b in zip(before, [self.refs] + [t.pages for t in self.tables]))
        first = [self.moves.count.item(), self.moves.src.clone(), self.moves.dst.clone()]
        self.cpa.cp_pages_compact(self.plan, self.refs, self.tables, self.moves, self.ws, used=used)
        want, moves = self.pool.compact(*self.ref)
        assert used.item() == want
        self.check("compact")
        self.check_moves(moves, "compact")
        assert torch.equal(refs_out, self.refs) and all(torch.equal(a.pages, b.pages) for a, b in zip(outs, self.tables))
        n = first[0]
        assert n == len(moves) and torch.equal(first[1][:n], self.moves.src[:n]) and torch.equal(first[2][:n], self.moves.dst[:n])


SHAPES = {
    "one_page": (1, 16, (1, 1)),
    "few": (5, 16, (3, 4)),
    "odd": (131, 16, (7, 33), (3, 9)),
    "page_65536": (40, 65536, (5, 8)),
    "many_rows": (3001, 16, (1500, 3), (100, 20)),
    "most_rows": (20000, 32, (8192, 5)),
    "wide": (70001, 16, (9, 20000), (1, 5)),
    "large": (1 << 20, 16, (300, 4000), (40, 1000), (1, 1), (8192, 2)),
}


@pytest.mark.parametrize("name", list(SHAPES))
def test_pages_in_turn(cpa, name):
    """Resizes, forks and compactions one after another, at random, pages running
    out among them."""
    pages, ps, *shapes = SHAPES[name]
    b = Both(cpa, pages, ps, *shapes, seed=len(name), taken=0.2 if pages > 1 else 0)
    rng, used = b.rng, []
    for step in range(10 if pages < 100000 else 5):
        for k, (rows, columns) in enumerate(shapes):
            most = min(columns, 2 * pages // rows + 2) * ps
            tokens = np.where(rng.random(rows) < 0.3, -1, rng.integers(0, most + 1, rows) * (rng.random(rows) < 0.8))
            b.resize(tokens, k)
        for src, dst in ((0, 0), (0, len(shapes) - 1)):
            t, into = b.ref[src], b.ref[dst]
            parent = np.where((into.held == 0) & (rng.random(len(into.held)) < 0.7), rng.integers(0, len(t.held), len(into.held)), -1)
            room = np.minimum(t.held[parent], into.pages.shape[1]) * ps
            tokens = np.where(parent >= 0, (rng.random(len(parent)) * (room + 1)).astype(np.int64), 0)
            if ps > 1000:  # part pages and whole ones
                tokens -= (tokens % ps) * (rng.random(len(parent)) < 0.3).astype(np.int64)
            b.fork(parent, tokens, src, dst)
        used.append(int((b.pool.refs > 0).sum()))
        b.compact()
    for k in range(len(shapes)):
        b.resize(np.zeros(shapes[k][0]), k)
    assert set(np.unique(b.pool.refs)) <= {0, 2} and max(used) > 0


def test_a_pool_that_is_looked_at_in_parts(cpa):
    """More than a million pages, most of them taken in one call (a CTA lists 16K at a
    time and looks at refs again), then again among those that are held."""
    b = Both(cpa, (1 << 21) + 77, 16, (300, 6000), seed=5, taken=0.3)
    rng = b.rng
    b.resize(rng.integers(60000, 70000, 300))
    b.resize(np.where(rng.random(300) < 0.5, 0, -1))
    assert 0 in b.resize(rng.integers(90000, 96000, 300))
    b.compact()


def test_tables_beyond_32_bits(cpa):
    """8192 rows of 300000 pages: requests for more than 2^31 pages in all are not
    served, and the last rows' entries lie behind entry 2^31."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    rows, columns, pages = 8192, 300000, 1000
    plan = plan_of(cpa, 16)
    table = cpa.PageTable(torch.full((rows, columns), -1, dtype=torch.int32, device="cuda"), ints(np.zeros(rows)))
    refs, served = ints(np.zeros(pages)), ints(np.full(rows, -7))
    cpa.cp_pages_resize(plan, refs, table, ints(np.full(rows, columns * 16)), served)
    assert not served.any() and not table.held.any() and not refs.any()
    tokens = np.full(rows, -1)
    tokens[[0, 8000, 8191]] = 20, 100, 33
    cpa.cp_pages_resize(plan, refs, table, ints(tokens), served)
    assert served.all() and table.pages[0, :3].tolist() == [0, 1, -1] and table.pages[8000, :8].tolist() == [2, 3, 4, 5, 6, 7, 8, -1]
    parent, moves = np.full(rows, -1), cpa.PageMoves(rows)
    parent[8190] = 8191
    cpa.cp_pages_fork(plan, refs, table, table, ints(parent), ints(np.where(parent >= 0, 33, 0)), moves, served)
    assert served.all() and table.pages[8190, :4].tolist() == [9, 10, 12, -1] and moves.src[0].item() == 11
    cpa.cp_pages_resize(plan, refs, table, ints(np.where(np.arange(rows) == 8000, 0, -1)), served)
    used = ints([0])
    cpa.cp_pages_compact(plan, refs, [table], moves, cpa.alloc_pages_workspace(pages), used=used)
    assert used.item() == 6 and table.pages[8191, :3].tolist() == [2, 3, 4] and table.pages[8190, :3].tolist() == [2, 3, 5]


def test_no_moves(cpa):
    """A pool of one page, lists without room: nothing moves."""
    b = Both(cpa, 1, 16, (1, 1))
    b.moves = cpa.PageMoves(0)
    b.resize([16])
    b.compact()
    k = torch.zeros(1, 16, 2, 64, dtype=BF, device="cuda")
    cache = cpa.PagedCache(k, k.clone())
    cpa.cp_pages_copy(b.plan, [cache], [cache], b.moves)


def test_lengths_of_a_row(cpa):
    b = Both(cpa, 50, 16, (2, 10))
    for t in (0, 1, 15, 16, 17, 160, 159, 145, 144, 16, 1, 0, 160, 0):
        b.resize([t, -1])
    assert b.resize([160, 160]) == [1, 1]


def test_pages_run_out_in_order(cpa):
    """Rows are served in order; one that does not fit ends it, though a later one would."""
    b = Both(cpa, 10, 16, (5, 20))
    assert b.resize([16 * 4, 16 * 5, 16 * 2, 16 * 1, 0]) == [1, 1, 0, 0, 1]
    assert b.resize([16 * 4, 16 * 4, 16 * 2, 16 * 1, 0]) == [1, 1, 1, 0, 1]  # one let go in the call serves
    assert b.fork([-1, -1, -1, 0, 0], [0, 0, 0, 32, 33]) == [1, 1, 1, 1, 0]
    b.resize([-1, 0, -1, -1, -1])
    assert b.fork([-1, 2, -1, -1, 0], [0, 31, 0, 0, 33]) == [1, 1, 1, 1, 1]


def test_free_after_a_fork_keeps_shared_pages(cpa):
    b = Both(cpa, 40, 16, (6, 8))
    b.resize([100, 0, 0, 0, 0, 0])
    b.fork([-1, 0, 0, 0, -1, -1], [0, 100, 96, 0, 0, 0])     # a part page, whole pages, nothing
    b.fork([-1, -1, -1, 1, 1, 2], [0, 0, 0, 50, 100, 96])    # of children, in several rows
    b.resize([0, -1, -1, -1, -1, -1])
    b.compact()
    b.resize([64, 0, 33, 0, 100, -1])
    b.compact()
    b.resize([0] * 6)
    assert not b.refs.any()


def test_prefixes_and_rows(cpa):
    """A prompt becomes a prefix, and a prefix a sequence, between two tables."""
    b = Both(cpa, 64, 16, (4, 12), (2, 5))
    b.resize([70, 100, 0, 0])
    b.fork([0, 1], [64, 33], src=0, dst=1)
    b.resize([0, 0, 0, 0])
    b.fork([-1, 0, 1, 1], [0, 64, 20, 33], src=1, dst=0)
    b.compact()
    b.resize([0, 0], 1)
    b.compact()


def test_refused_rows_are_recorded(cpa):
    """Data out of bounds: the row is left as it was, the others are served."""
    b = Both(cpa, 64, 16, (6, 4), (2, 9))
    b.resize([64, 64, 10, 0, 0, 0])
    b.resize([0, 140], 1)

    def recorded():
        rec = cpa.cp_get_status_detail()
        return rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 10
    assert b.resize([65, -1, 2 ** 31 - 1, 3, 1000, 64]) == [0, 1, 0, 1, 0, 1] and recorded()
    #       occupied, no such row, more than it holds, fits not, of an empty row, good
    assert b.fork([1, -5, 6, 1, 3, 1], [5, 7, 1, 65, 17, 0]) == [0, 1, 0, 0, 0, 0] and recorded()
    b.resize([-1, -1, -1, 0, -1, 0])
    assert b.fork([-1, -1, -1, 1, 2 ** 31 - 1, 2], [0, 0, 0, 100, 1, -1], src=1, dst=0) == [1, 1, 1, 0, 0, 0] and recorded()
    for held in (-1, 5, 2 ** 31 - 1, -2 ** 31):
        b.tables[0].held[3] = held
        out, refs, pages = b.served(0), b.refs.clone(), b.tables[0].pages.clone()
        cpa.cp_pages_resize(b.plan, b.refs, b.tables[0], ints([-1, -1, -1, 5, -1, -1]), out)
        assert out.tolist() == [1, 1, 1, 0, 1, 1] and recorded()
        cpa.cp_pages_fork(b.plan, b.refs, b.tables[0], b.tables[1], ints([3, -1]), ints([5, 0]), b.moves, b.served(1))
        assert recorded()
        cpa.cp_pages_compact(b.plan, b.refs, [b.tables[0]], b.moves, b.ws, refs_out=torch.empty_like(b.refs),
                             tables_out=[cpa.PageTable(torch.empty_like(b.tables[0].pages), b.tables[0].held)])
        assert recorded()
        assert torch.equal(refs, b.refs) and torch.equal(pages, b.tables[0].pages) and b.tables[0].held[3].item() == held


@pytest.mark.parametrize("page", [-1, 64, 2 ** 31 - 1, -2 ** 31])
def test_bad_pages_are_recorded(cpa, page):
    """A page number outside the pool is neither counted nor followed."""
    b = Both(cpa, 64, 16, (4, 6))
    b.resize([96, 50, 0, 0])
    b.tables[0].pages[0, 2] = page
    b.tables[0].pages[1, 3] = page
    refs = b.refs.clone()
    out = b.served(0)

    def recorded():
        rec = cpa.cp_get_status_detail()
        return rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 10
    cpa.cp_pages_fork(b.plan, b.refs, b.tables[0], b.tables[0], ints([-1, -1, 0, 1]), ints([0, 0, 96, 50]), b.moves, out)
    assert recorded() and out.tolist() == [1] * 4 and b.tables[0].pages[2, 2].item() == -1
    # Row 3's part page has no source: the copy is left out and recorded.
    cache = [torch.randn(64, 16, 2, 64, device="cuda").to(BF) for _ in range(2)]
    before = [c.clone() for c in cache]
    cpa.cp_pages_copy(b.plan, [cpa.PagedCache(*cache)], [cpa.PagedCache(*cache)], b.moves)
    assert recorded() and all(torch.equal(x, y) for x, y in zip(cache, before))
    cpa.cp_pages_compact(b.plan, b.refs, b.tables, b.moves, b.ws)
    assert recorded() and b.tables[0].pages[0, 2].item() == page
    cpa.cp_pages_resize(b.plan, b.refs, b.tables[0], ints([0] * 4), out)
    assert recorded() and refs.sum() == 10 and b.refs.sum() == 2  # the two that the table has lost


def test_pages_held_by_no_one_are_not_let_go(cpa):
    """A table that holds a free page (its refs are 0): letting go does not take the count below 0."""
    b = Both(cpa, 20, 16, (2, 4))
    b.resize([64, 20])
    b.refs[1] = 0
    cpa.cp_pages_resize(b.plan, b.refs, b.tables[0], ints([0, -1]), b.served(0))
    assert cpa.cp_get_status_detail()[0] == cpa.CP_ERR_DEVICE_BOUNDS
    assert b.refs[:4].tolist() == [0] * 4 and b.refs[4:6].tolist() == [1, 1]


def test_compact_renames_pages_above_that_no_one_holds(cpa):
    """A table entry above `used` whose page is free goes nowhere, and is recorded."""
    b = Both(cpa, 30, 16, (2, 4))
    b.resize([64, 20])
    b.tables[0].pages[1, 0] = 29
    cpa.cp_pages_compact(b.plan, b.refs, b.tables, b.moves, b.ws)
    assert cpa.cp_get_status_detail()[0] == cpa.CP_ERR_DEVICE_BOUNDS and b.tables[0].pages[1, 0].item() == 29


# ---------------------------------------------------------------- copies

def strided(shape, layout, dtype, seed):
    """A cache [pages][ps][Hkv][d] on the GPU and the storage it lies in."""
    P, ps, H, d = shape
    gen = torch.Generator().manual_seed(seed)
    if layout == "heads_first":
        base = torch.randn(P, H, ps, d, generator=gen).to(dtype).cuda()
        return base.transpose(1, 2), base
    if layout == "gaps":  # between heads, tokens and pages
        base = torch.randn(P, ps + 1, H + 1, d + 8, generator=gen).to(dtype).cuda()
        return base[:, :ps, :H, :d], base
    if layout == "heads_first_gaps":
        base = torch.randn(P, H, ps + 2, d, generator=gen).to(dtype).cuda()
        return base[:, :, :ps].transpose(1, 2), base
    if layout == "heads_outside":  # heads further apart than pages
        base = torch.randn(H, P, ps, d, generator=gen).to(dtype).cuda()
        return base.permute(1, 2, 0, 3), base
    base = torch.randn(P, ps, H, d, generator=gen).to(dtype).cuda()
    return base, base


LAYOUTS = ["tokens", "heads_first", "gaps", "heads_first_gaps", "heads_outside"]


@pytest.mark.parametrize("shape", [(12, 16, 2, 64), (9, 16, 3, 128), (7, 64, 1, 128), (6, 256, 5, 64)])
@pytest.mark.parametrize("dst", LAYOUTS)
@pytest.mark.parametrize("src", LAYOUTS)
def test_copies_between_layouts(cpa, src, dst, shape):
    P, ps, H, d = shape
    dtype = BF if d == 64 else FP
    plan = plan_of(cpa, ps, H, d, dtype)
    layers = 3
    a = [[strided(shape, src, dtype, 10 * i + k) for k in range(2)] for i in range(layers)]
    b = [[strided((P + 3, *shape[1:]), dst, dtype, 100 + 10 * i + k) for k in range(2)] for i in range(layers)]
    want = [[base.clone() for _, base in c] for c in b]
    s, t, n = [3, 0, 3, 5, 1, 2], [P + 2, 1, 0, 5, 4, 2], [ps, 1, ps - 1, ps // 2, 0, 3]
    for i in range(layers):
        for k in range(2):
            view = torch.as_strided(want[i][k], b[i][k][0].shape, b[i][k][0].stride())
            for x, y, m in zip(s, t, n):
                view[y, :m] = a[i][k][0][x, :m]
    cpa.cp_pages_copy(plan, [cpa.PagedCache(*[x for x, _ in c]) for c in a], [cpa.PagedCache(*[x for x, _ in c]) for c in b],
                      cpa.PageMoves(src=ints(s), dst=ints(t), tokens=ints(n)))
    for i in range(layers):
        for k in range(2):
            assert torch.equal(b[i][k][1], want[i][k])  # what lies between is left as it was


def test_copies_within_a_cache(cpa):
    for layout in LAYOUTS:
        (k, kb), (v, vb) = (strided((20, 32, 2, 128), layout, BF, i) for i in range(2))
        want = [x.clone() for x in (kb, vb)]
        s, t, n = [1, 3, 1], [4, 5, 19], [32, 7, 32]
        for w, x in zip(want, (k, v)):
            view = torch.as_strided(w, x.shape, x.stride())
            for i, j, m in zip(s, t, n):
                view[j, :m] = x[i, :m]
        cache = cpa.PagedCache(k, v)
        cpa.cp_pages_copy(plan_of(cpa, 32, 2, 128), [cache], [cache], cpa.PageMoves(src=ints(s), dst=ints(t), tokens=ints(n)))
        assert torch.equal(kb, want[0]) and torch.equal(vb, want[1])


def test_copies_of_every_number_of_layers(cpa):
    plan = plan_of(cpa, 16, 1, 64)
    caches = [torch.full((4, 2, 16, 1, 64), float(i), device="cuda").to(BF) for i in range(128)]
    for n in (1, 2, 127, 128):
        for i, c in enumerate(caches):
            c[:] = i
            c[3] = -1
        views = [cpa.PagedCache(c[:, 0], c[:, 1]) for c in caches[:n]]
        cpa.cp_pages_copy(plan, views, views, cpa.PageMoves(src=ints([1]), dst=ints([3]), tokens=ints([16])))
        for i, c in enumerate(caches):
            assert (c[3] == (i if i < n else -1)).all()


def test_copies_with_other_counts(cpa):
    """The count is on the device: fewer than the capacity, none, or out of bounds (then nothing is copied, and it is recorded)."""
    plan = plan_of(cpa, 16, 1, 64)
    for count, copied in ((2, 2), (0, 0), (3, 3), (4, 0), (-1, 0), (2 ** 31 - 1, 0)):
        c = torch.arange(8, device="cuda").to(BF)[:, None, None, None].repeat(1, 16, 1, 64)
        cache = cpa.PagedCache(c, c.clone())
        cpa.cp_pages_copy(plan, [cache], [cache], cpa.PageMoves(src=ints([0, 1, 2]), dst=ints([5, 6, 7]), tokens=ints([16] * 3), count=ints([count])))
        assert c[5:, 0, 0, 0].tolist() == [0, 1, 2][:copied] + [5, 6, 7][copied:]
        assert (cpa.cp_get_status_detail()[0] != 0) == (not 0 <= count <= 3)


@pytest.mark.parametrize("move", [(-1, 2, 16), (8, 2, 16), (1, -1, 16), (1, 10, 16), (1, 2, 17), (1, 2, -1), (2 ** 31 - 1, 2, 16)])
def test_copies_out_of_bounds(cpa, move):
    plan = plan_of(cpa, 16, 1, 64)
    a, b = (torch.randn(n, 16, 1, 64, device="cuda").to(BF) for n in (8, 10))
    want = b.clone()
    want[9], want[0] = a[7], a[3]
    s, t, n = zip((7, 9, 16), move, (3, 0, 16))
    cpa.cp_pages_copy(plan, [cpa.PagedCache(a, a.clone())], [cpa.PagedCache(b, b.clone())], cpa.PageMoves(src=ints(s), dst=ints(t), tokens=ints(n)))
    rec = cpa.cp_get_status_detail()
    assert torch.equal(b, want) and rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 10


def test_copies_beyond_32_bits(cpa):
    """Pages 2^27 elements apart: the last lies 2^32 elements behind the first."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    P, stride = 33, 1 << 27
    buf = torch.empty(P * stride, dtype=BF, device="cuda")
    k, v = (buf[o:].as_strided((P, 16, 2, 64), (stride, 128, 64, 1)) for o in (0, 65536))
    x = torch.randn(2, 16, 2, 64, device="cuda").to(BF)
    k[32], v[32], k[0], v[0] = x[0], x[1], 0, 0
    k[31], v[31] = 0, 0
    cache = cpa.PagedCache(k, v)
    cpa.cp_pages_copy(plan_of(cpa, 16), [cache], [cache], cpa.PageMoves(src=ints([32, 32]), dst=ints([0, 31]), tokens=ints([16, 16])))
    for p in (0, 31):
        assert torch.equal(k[p], x[0]) and torch.equal(v[p], x[1])


def test_pages_captured(cpa):
    """A captured step (drop, take, fork, copy, compact, copy) follows its
    arrays; two graphs over two pools share nothing."""
    graphs = []
    for seed in range(2):
        b = Both(cpa, 400, 16, (20, 12), seed=seed, taken=0.3)
        b.resize(b.rng.integers(1, 150, 20))
        tokens, parent, lens, out = ints(np.full(20, -1)), ints(np.full(20, -1)), ints(np.zeros(20)), b.served(0)
        cache = [torch.randn(400, 16, 2, 64, device="cuda").to(BF) for _ in range(2)]
        caches = [cpa.PagedCache(*cache)]
        used = torch.zeros(1, dtype=torch.int32, device="cuda")

        def step(b=b, tokens=tokens, parent=parent, lens=lens, out=out, caches=caches, used=used):
            cpa.cp_pages_resize(b.plan, b.refs, b.tables[0], tokens, out)
            cpa.cp_pages_fork(b.plan, b.refs, b.tables[0], b.tables[0], parent, lens, b.moves, out)
            cpa.cp_pages_copy(b.plan, caches, caches, b.moves)
            cpa.cp_pages_compact(b.plan, b.refs, b.tables, b.moves, b.ws, used=used)
            cpa.cp_pages_copy(b.plan, caches, caches, b.moves)
        step()
        b.pool.compact(*b.ref)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        graphs.append((b, tokens, parent, lens, cache, graph))
    for turn in range(4):
        for b, tokens, parent, lens, cache, graph in graphs:
            mirror = [c.clone() for c in cache]
            ask = np.where(b.rng.random(20) < 0.4, 0, b.rng.integers(-1, 150, 20))
            b.pool.resize(b.ref[0], ask)
            p = np.where((b.ref[0].held == 0) & (b.rng.random(20) < 0.7), b.rng.integers(0, 20, 20), -1)
            n = np.where(p >= 0, (b.rng.random(20) * (b.ref[0].held[p] * 16 + 1)).astype(int), 0)
            for moves in (b.pool.fork(b.ref[0], b.ref[0], p, n)[1], b.pool.compact(*b.ref)[1]):
                for x, y, m in moves:
                    for c in mirror:
                        c[y, :m] = c[x, :m]
            tokens.copy_(ints(ask))
            parent.copy_(ints(p))
            lens.copy_(ints(n))
            graph.replay()
            b.check(f"turn {turn}")
            assert all(torch.equal(x, y) for x, y in zip(cache, mirror))


def test_pages_on_two_streams(cpa):
    both = [Both(cpa, 5000, 16, (300, 30), seed=s) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    asks = [[b.rng.integers(-1, 480, 300) for _ in range(6)] for b in both]
    given = [[ints(x) for x in a] for a in asks]
    outs = [[b.served(0) for _ in range(6)] for b in both]
    torch.cuda.synchronize()
    for i in range(6):
        for b, st, g, o in zip(both, streams, given, outs):
            with torch.cuda.stream(st):
                cpa.cp_pages_resize(b.plan, b.refs, b.tables[0], g[i], o[i])
    torch.cuda.synchronize()
    for b, a, o in zip(both, asks, outs):
        assert [b.pool.resize(b.ref[0], x) for x in a] == [x.tolist() for x in o]
        b.check()
