"""Verification of drafts (cp_verify_drafts) against its definition in 64 bits:
shapes and alignments, borders, rows without weight, numbers that are none,
bad data, streams and graphs."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

from serving_ref import verify  # noqa: E402
from test_gpu_paged_use import ints  # noqa: E402

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def cpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import context_long_sequence_gb300 as m
    return m


class Drafts:
    """A batch of drafts on the CPU."""

    def __init__(self, new, V, dtype=F32, q=True, pad=0, seed=0, spread=2.0, near=0.5, cut=0.3):
        gen = torch.Generator().manual_seed(seed)
        self.new, self.V, self.B = list(new), V, len(new)
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.n, self.N = int(self.start[-1]), int(self.start[-1]) + pad
        logit = torch.randn(self.N, V, generator=gen) * spread
        p = torch.softmax(logit, -1)
        if cut:  # part of the vocabulary is cut off, the best never
            p = torch.where((torch.rand(self.N, V, generator=gen) < cut) & (p < p.amax(-1, keepdim=True)), torch.zeros(()), p)
        self.p = (p / p.sum(-1, keepdim=True)).to(dtype)
        self.q = torch.softmax(logit + near * torch.randn(self.N, V, generator=gen), -1).to(dtype) if q else None
        drawn = torch.multinomial((self.q if q else self.p).float() + 1e-12, 1, generator=gen)[:, 0] if self.N else torch.zeros(0)
        self.tokens = torch.cat([torch.zeros(1), drawn])[:self.N].long()
        self.u, self.r = torch.rand(self.N, generator=gen), torch.rand(self.B, generator=gen)
        self.kv = np.arange(self.B) * 10 + 100 + np.array(new)

    def ref(self):
        q = None if self.q is None else self.q.double().numpy()
        return verify(self.start, self.kv, self.tokens.numpy(), self.p.double().numpy(), q, self.u.numpy(), self.r.numpy())

    def gpu(self, cpa, p=None, q=None, max_new=None):
        """plan, batch and arguments on the GPU; p, q: row strides, or tensors there."""
        def rows(x, how):
            if x is None or isinstance(how, torch.Tensor):
                return how if x is not None else None
            buf = torch.full((self.N, how or self.V), float("nan"), dtype=x.dtype, device="cuda")
            buf[:, :self.V] = x.cuda()
            return buf[:, :self.V]
        plan = cpa.PagedPlan(8, 2, 128, page_size=16, dtype=BF, max_seqs=max(1, self.B), max_tokens=max(1, self.N),
                             max_new=max_new or max(1, *self.new), max_pages=4)
        batch = cpa.PagedBatch(ints(self.start), ints(self.kv), ints(np.zeros((self.B, 4))), n_tokens=self.N)
        out = [torch.full((k,), -7, dtype=torch.int32, device="cuda") for k in (self.B, self.N, self.B)]
        return plan, batch, [ints(self.tokens.numpy()), rows(self.p, p), rows(self.q, q), self.u.cuda(), self.r.cuda(), *out]

    def run(self, cpa, **kw):
        plan, batch, args = self.gpu(cpa, **kw)
        cpa.cp_verify_drafts(plan, batch, *args)
        return args[5:]

    def check(self, cpa, **kw):
        got, ref = self.run(cpa, **kw), self.ref()
        for name, x, y in zip(("accepted", "out_tokens", "kv_len_out"), got, ref):
            assert np.array_equal(x.cpu().numpy(), y), (name, np.flatnonzero(x.cpu().numpy() != y)[:5], x.cpu().numpy()[:12], y[:12])
        return got


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("q", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 300, 1000, 5003, 33000, 131077])
def test_verify_vocabularies(cpa, V, q, dtype):
    Drafts([1, 4, 0, 2, 6], V, dtype, q, pad=3, seed=V, spread=2.0 if V < 5000 else 5.0).check(cpa)


@pytest.mark.parametrize("new", [[1], [5], [1] * 40, [2, 3] * 200, [0, 0], [0, 1, 0], [70, 1, 33, 34, 65]])
def test_verify_batches(cpa, new):
    Drafts(new, 777, seed=sum(new), near=0.1).check(cpa)
    Drafts(new, 777, seed=sum(new) + 1, q=False, spread=6.0, pad=2).check(cpa)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("p,q", [(1000, 1000), (1000, 1003), (1009, 1001), (1001, 1024), (1024, 1024)])
def test_verify_strides(cpa, p, q, dtype):
    """Rows of every alignment, p's and q's alike or not."""
    Drafts([4, 5, 3, 1, 6, 2, 4], 999, dtype, seed=p + q).check(cpa, p=p, q=q)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_verify_rows_of_a_larger_tensor(cpa, dtype):
    """p and q begin anywhere: an element's alignment is enough."""
    d = Drafts([4, 5, 3], 517, dtype, seed=19)
    for skip, (i, j) in ((1, (3, 0)), (2, (5, 7)), (0, (1, 1))):
        views = []
        for x, k in ((d.p, i), (d.q, j)):
            buf = torch.full((d.N + skip, 541), float("nan"), dtype=dtype, device="cuda")
            views.append(buf[skip:, k:k + 517])
            views[-1].copy_(x)
        d.check(cpa, p=views[0], q=views[1])


def test_verify_does_not_hang_on_the_batch(cpa):
    """A sequence alone (16 CTAs) gives what it gives among 300 (one)."""
    d = Drafts([3] * 300, 20011, seed=3)
    accepted, out, _ = d.check(cpa)
    for s in (0, 17, 299):
        one = Drafts([3], 20011, seed=0)
        t = slice(3 * s, 3 * s + 3)
        one.p, one.q, one.tokens, one.u, one.r = d.p[t], d.q[t], d.tokens[t], d.u[t], d.r[s:s + 1]
        a, o, _ = one.run(cpa)
        assert a.item() == accepted[s].item() and torch.equal(o, out[t])


@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("V", [8, 512, 4096])
def test_verify_borders_are_exact(cpa, V, dtype):
    """Equal dyadic weights, random numbers on their borders: r = k / V gives
    token k, the number just below it k - 1."""
    ks = sorted({0, 1, V // 3, V // 2, V - 1})
    d = Drafts([1] * (2 * len(ks)), V, dtype, seed=1)
    d.p = torch.full((d.N, V), 1.0 / V).to(dtype)
    d.r = torch.tensor([x for k in ks for x in (k / V, np.nextafter(np.float32(k / V), np.float32(-1)))], dtype=F32)
    _, out, _ = d.check(cpa)
    assert out.tolist() == [x for k in ks for x in (k, max(0, k - 1))]


def test_verify_acceptance_is_exact(cpa):
    """u q(x) = p(x) exactly is a rejection, one step below an acceptance."""
    d = Drafts([2] * 4, 64, seed=2, cut=0)
    p, q = 3 * 2.0 ** -10, 3 * 2.0 ** -6
    d.tokens[:] = 5
    d.p[:, 5], d.q[:, 5] = p, q
    u = np.float32(2.0 ** -4)
    for s, x in enumerate((u, np.nextafter(u, np.float32(0)), np.nextafter(u, np.float32(1)), 0.0)):
        d.u[2 * s] = float(x)
    accepted, _, _ = d.check(cpa)
    assert accepted.tolist() == [0, 1, 0, 1]


def test_verify_fine_sums(cpa):
    """131072 weights of 2^-17 and one of 2^-40 more: sums that fp32 does not hold."""
    V = 131072
    d = Drafts([1] * 8, V, seed=3)
    d.p = torch.full((8, V), 2.0 ** -17)
    d.p[:, 100] += 2.0 ** -40
    total = 1.0 + 2.0 ** -40
    ks = [99, 100, 101, 65536, 131000]
    d.r = torch.tensor([k / V for k in ks] + [0.0, 1 - 2.0 ** -24, 0.3])
    _, out, _ = d.check(cpa)
    # Behind weight 100 the borders lie 2^-40 higher, r total only r 2^-40: r = k / V falls just below border k.
    want = [k if k * 2.0 ** -17 * total >= k * 2.0 ** -17 + (2.0 ** -40 if k > 100 else 0) else k - 1 for k in ks]
    assert out.tolist()[:5] == want and out.tolist()[5:7] == [0, V - 1]


def test_verify_tiny_residual(cpa):
    """p and q alike but for the last places of a few numbers: the residual is theirs alone."""
    d = Drafts([2] * 30, 5000, seed=4, cut=0)
    d.q = d.p.clone()
    rows = torch.arange(0, 60, 2)
    spots = torch.randint(0, 5000, (30, 5), generator=torch.Generator().manual_seed(4))
    d.tokens[rows + 1] = 4999
    d.q[rows, 4999] = 0.5
    d.u[:] = 0.9999
    for i in range(5):
        x = d.p[rows, spots[:, i]]
        d.p[rows, spots[:, i]] = torch.nextafter(x, torch.ones(()))
    _, out, _ = d.check(cpa)
    assert all(out[2 * s].item() in spots[s].tolist() for s in range(30))


def test_verify_rows_without_weight(cpa):
    d = Drafts([1, 2, 2, 3, 1], 3001, seed=5)
    t = d.start
    d.p[t[0]] = 0                                  # nothing to draw from
    d.tokens[t[1] + 1] = 7                         # rejected, and the residual is empty: from p
    d.p[t[1], 7], d.u[t[1]] = 0, 0.5
    d.q[t[1]] = d.p[t[1]] + 0.25
    d.tokens[t[2] + 1], d.p[t[2]], d.u[t[2]] = 9, 0, 0.0  # rejected, and p is empty as well
    got = d.check(cpa)
    assert got[1][t[0]].item() == -1 and got[1][t[1]].item() >= 0 and got[1][t[2]].item() == -1


@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_verify_numbers_that_are_none(cpa, dtype):
    """NaN, negative numbers and infinities count as nothing (an infinite q
    leaves nothing), at drafts and elsewhere."""
    nan, inf = float("nan"), float("inf")
    d = Drafts([3] * 40, 1001, dtype, seed=6)
    gen = torch.Generator().manual_seed(6)
    for x, bad in ((d.p, (nan, -1.0, inf, -inf, -0.0)), (d.q, (nan, -0.5, inf, -inf))):
        for i, value in enumerate(bad):
            x[torch.rand(x.shape, generator=gen) < 0.05] = value
    hit = torch.rand(d.N, generator=gen) < 0.3  # some drafts among them
    for t in range(d.N - 1):
        if hit[t]:
            d.p[t, d.tokens[t + 1]] = (nan, -1.0, inf)[t % 3]
        elif t % 7 == 0:
            d.q[t, d.tokens[t + 1]] = (nan, inf, -1.0)[t % 3]
    d.check(cpa)


def test_verify_random_numbers_out_of_range(cpa):
    d = Drafts([1] * 7 + [2] * 5, 500, seed=7)
    d.r = torch.tensor([0.0, -0.0, 1.0, 2.0, -1.0, float("nan"), float("inf")] + [0.5] * 5)
    for s, u in enumerate((1.0, float("nan"), -1.0, float("inf"), 0.0)):
        d.u[7 + 2 * s] = u
    _, out, _ = d.check(cpa)
    first, last = (int(torch.nonzero(d.p[0])[i]) for i in (0, -1))
    assert out[0].item() == first and out[2].item() == int(torch.nonzero(d.p[2])[-1]) and last >= first


def test_verify_unnormalised_weights(cpa):
    d = Drafts([2] * 20, 3000, seed=8)
    d.p, d.q = d.p * 1e30, d.q * 1e30
    d.check(cpa)
    d = Drafts([2] * 20, 3000, seed=8)
    d.p, d.q = d.p * 1e-30, d.q * 1e-30  # down to fp32's smallest numbers
    d.check(cpa)


def test_verify_lengths_in_place(cpa):
    d = Drafts([1, 5, 0, 3], 900, seed=9)
    plan, batch, args = d.gpu(cpa)
    cpa.cp_verify_drafts(plan, batch, *args[:7], batch._keep[1])
    assert np.array_equal(batch._keep[1].cpu().numpy(), d.ref()[2])
    plan, batch, args = d.gpu(cpa)
    cpa.cp_verify_drafts(plan, batch, *args[:7])  # without
    assert np.array_equal(args[6].cpu().numpy(), d.ref()[1]) and (args[7] == -7).all()


@pytest.mark.parametrize("x", [-1, 900, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("q", [True, False])
def test_verify_drafts_outside_the_vocabulary(cpa, x, q):
    d = Drafts([4, 3], 900, seed=10, q=q)
    d.p[:, 3] = 1.0
    d.tokens[:], d.u[:] = 3, 0.0
    d.tokens[2] = x
    d.check(cpa)
    rec = cpa.cp_get_status_detail()
    assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 9


@pytest.mark.parametrize("start", [[0, -1, 3, 6], [0, 2, 1, 6], [0, 2, 3, 9999], [0, 2, 3, 60], [5, 2, 3, 6], [0, 2, 3, 2 ** 31 - 1]])
def test_verify_bad_starts(cpa, start):
    """Sequences whose rows leave the batch or the plan are left out and
    recorded, the others are served."""
    d = Drafts([2, 1, 3], 700, seed=11, pad=70)
    plan, batch, args = d.gpu(cpa, max_new=4)
    batch._keep[0].copy_(ints(start))
    cpa.cp_verify_drafts(plan, batch, *args)
    rec = cpa.cp_get_status_detail()
    assert rec[0] == cpa.CP_ERR_DEVICE_BOUNDS and rec[3] == 9
    ref, touched = d.ref(), np.zeros(d.N, bool)
    for s in range(3):
        good = 0 <= start[s] <= start[s + 1] <= d.N and start[s + 1] - start[s] <= 4
        if good and (start[s], start[s + 1]) == (d.start[s], d.start[s + 1]):
            assert args[5][s].item() == ref[0][s] and args[7][s].item() == ref[2][s]
            assert np.array_equal(args[6][start[s]:start[s + 1]].cpu().numpy(), ref[1][start[s]:start[s + 1]])
        if good:
            touched[start[s]:start[s + 1]] = True
        else:
            assert args[5][s].item() == -7 and args[7][s].item() == -7
    assert (args[6].cpu().numpy()[~touched] == -7).all()


def test_verify_empty_batches(cpa):
    d = Drafts([1, 2], 50, seed=12)
    plan, batch, args = d.gpu(cpa)
    empty = cpa.PagedBatch(ints([0]), ints([]), ints(np.zeros((0, 4))), n_tokens=0)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    cpa.cp_verify_drafts(plan, empty, none, args[1][:0], args[2][:0], args[3][:0], args[4][:0], none, none, none)


def test_verify_offsets_beyond_32_bits(cpa):
    d = Drafts([2] * 20, 1000, BF, seed=13)
    stride = 1 << 27
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    buf = torch.empty(d.N * stride, dtype=BF, device="cuda")
    p, q = buf.as_strided((d.N, 1000), (stride, 1)), buf[4096:].as_strided((d.N, 1000), (stride, 1))
    p.copy_(d.p)
    q.copy_(d.q)
    d.check(cpa, p=p, q=q)


def test_verify_captured_streams_and_repeats(cpa):
    d = Drafts([3, 1, 6, 2], 30011, seed=14)
    plan, batch, args = d.gpu(cpa)
    cpa.cp_verify_drafts(plan, batch, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.cp_verify_drafts(plan, batch, *args)
    for seed in (15, 16, 17):
        e = Drafts([3, 1, 6, 2], 30011, seed=seed)
        for x, y in zip(args[:5], (ints(e.tokens.numpy()), e.p, e.q, e.u, e.r)):
            x.copy_(y)
        graph.replay()
        for x, y in zip(args[5:], e.ref()):
            assert np.array_equal(x.cpu().numpy(), y)
    # Two calls at once, on two streams, over different batches.
    other = Drafts([2] * 100, 20000, seed=18)
    plan2, batch2, args2 = other.gpu(cpa)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            cpa.cp_verify_drafts(plan, batch, *args)
        with torch.cuda.stream(streams[1]):
            cpa.cp_verify_drafts(plan2, batch2, *args2)
    torch.cuda.synchronize()
    for x, y in zip(args[5:], e.ref()):
        assert np.array_equal(x.cpu().numpy(), y)
    for x, y in zip(args2[5:], other.ref()):
        assert np.array_equal(x.cpu().numpy(), y)
