"""Rotary positions with several axes: cp_rope over whole sequences, its
gradient, and cp_cache_append under plans of several axes, against fp64."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

import paged_ref  # noqa: E402
from paged_ref import Batch  # noqa: E402
from serving_ref import rotate  # noqa: E402
from test_gpu_paged_use import ints  # noqa: E402

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def cpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import context_long_sequence_gb300 as m
    return m


def frequencies(rope_dim, base=10000.0):
    return base ** (-2.0 * np.arange(rope_dim // 2) / rope_dim)


def check(got, ref, size, what=""):
    """Half a step of the output's type, and the fp32 work before it, below
    2^-21 (|a| + |b|): the half-turns are off by 2^-25 (one fp32 rounding below
    1, and 2^-32 of the fraction's cut), so the angle by pi 2^-25; sine and
    cosine by two fp32 steps more; two products and a sum by three half-steps."""
    got = got.double().cpu().numpy()
    tiny = 2.0 ** -25 if what == FP else 0.0
    err = np.abs(got - ref)
    bound = paged_ref.HALF_STEP[what] * np.abs(ref) + 2.0 ** -21 * size + tiny
    assert np.all(err <= bound), (err.max(), np.argwhere(~(err <= bound))[:3].tolist())


def axes_of(rope_dim, axes, cycled):
    half = rope_dim // 2
    return [j % axes for j in range(half)] if cycled else [min(axes - 1, j * axes // half) for j in range(half)]


CASES = {
    "one_token": dict(n=1, heads=(8, 2)),
    "no_tokens": dict(n=0, heads=(8, 2)),
    "train": dict(n=1531, heads=(8, 2), axes=3),
    "many": dict(n=6000, heads=(5, 1), d=64, rope_dim=64, axes=3, cycled=True),
    "interleaved": dict(n=77, heads=(3, 3), axes=3, interleaved=True),
    "partial": dict(n=77, heads=(4, 1), d=96, rope_dim=48, axes=2),
    "partial_interleaved": dict(n=77, heads=(4, 1), d=128, rope_dim=32, axes=4, cycled=True, interleaved=True),
    "d16": dict(n=33, heads=(7,), d=16, rope_dim=16),
    "d80": dict(n=501, heads=(16, 16), d=80, rope_dim=80, axes=2),
    "d112": dict(n=130, heads=(5, 3, 2), d=112, rope_dim=112, axes=3, cycled=True),
    "d256": dict(n=130, heads=(2, 1), d=256, rope_dim=256, axes=4),
    "eight_tensors": dict(n=19, heads=(1, 2, 3, 4, 5, 6, 7, 8), d=64, rope_dim=64, axes=2),
    "fp16": dict(n=200, heads=(8, 2), ti=FP, to=FP, axes=3),
    "fp32": dict(n=200, heads=(8, 2), ti=F32, to=F32, axes=3),
    "fp32_interleaved_d80": dict(n=201, heads=(8, 2), d=80, rope_dim=48, ti=F32, to=F32, axes=3, interleaved=True),
    "grad_to_bf16": dict(n=333, heads=(8, 2), ti=F32, to=BF, axes=3, inverse=True),
    "grad_to_fp16": dict(n=333, heads=(8, 2), d=64, rope_dim=64, ti=F32, to=FP, axes=2, inverse=True),
    "bf16_to_fp32": dict(n=333, heads=(8, 2), ti=BF, to=F32, axes=2),
    "fp16_to_fp32": dict(n=333, heads=(8, 2), ti=FP, to=F32, axes=2, inverse=True),
    "many_heads": dict(n=3, heads=(130, 128), axes=3),
}


def run(cpa, n, heads, d=128, rope_dim=128, axes=1, cycled=False, interleaved=False, ti=BF, to=BF, inverse=False, seed=0, packed=True,
        positions=None, freqs=None):
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    if positions is None:
        positions = rng.integers(0, 100000, (axes, n))
    axis = axes_of(rope_dim, axes, cycled)
    freqs = frequencies(rope_dim) if freqs is None else freqs
    plan = cpa.RopePlan(d, rope_dim, axes, axis if axes > 1 else None, rope_interleaved=interleaved, rope_freqs=[float(f) for f in freqs])
    if packed:  # side by side, as one projection writes them, with something behind
        all_ = torch.randn(n, sum(heads) + 1, d, generator=gen).to(ti)
        at = np.cumsum([0, *heads])
        xs = [all_.cuda()[:, a:b] for a, b in zip(at, at[1:])]
    else:
        xs = [torch.randn(n, h, d, generator=gen).to(ti).cuda() for h in heads]
    outs = [torch.full((n, h, d), float("nan"), dtype=to, device="cuda") for h in heads]
    cpa.cp_rope(plan, ints(positions), xs, outs, inverse=inverse)
    for x, o in zip(xs, outs):
        ref, size = rotate(x.double().cpu().numpy(), positions, axis, freqs, interleaved, inverse)
        check(o, ref, size, to)
    return xs, outs


@pytest.mark.parametrize("name", list(CASES))
def test_rope_matches_fp64(cpa, name):
    run(cpa, seed=len(name), **CASES[name])
    run(cpa, seed=len(name), **(CASES[name] | dict(packed=False, inverse=not CASES[name].get("inverse", False))))


@pytest.mark.parametrize("at", [0, 1048575, 2 ** 31 - 60, -2 ** 31])
def test_rope_far_positions(cpa, at):
    positions = np.stack([at + np.arange(50), np.arange(50), np.full(50, 7)])
    # Angles of the reference in fp64 are good to 2^31 * 2^-53 here.
    run(cpa, 50, (2, 1), axes=3, ti=F32, to=F32, positions=positions, freqs=np.linspace(1.0, 1e-6, 64))


def test_rope_in_place(cpa):
    x = torch.randn(300, 6, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    plan = cpa.RopePlan(128, 64, 3, axes_of(64, 3, True))
    pos = ints(np.random.default_rng(1).integers(0, 5000, (3, 300)))
    out = torch.empty_like(x)
    cpa.cp_rope(plan, pos, [x], [out])
    y = x.clone()
    cpa.cp_rope(plan, pos, [y[:, :4], y[:, 4:]], [y[:, :4], y[:, 4:]])
    assert torch.equal(y, out)
    assert torch.equal(out[..., 64:], x[..., 64:])


def test_one_axis_equals_alike_axes(cpa):
    """Text: all axes alike give what one axis gives, bit for bit."""
    x = torch.randn(200, 6, 128, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    pos, outs = ints(np.arange(200) * 37), []
    for axes in (1, 2, 3, 4):
        plan = cpa.RopePlan(128, 128, axes, axes_of(128, axes, True))
        outs.append(torch.empty_like(x))
        cpa.cp_rope(plan, pos if axes == 1 else pos.repeat(axes, 1), [x], [outs[-1]])
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_gradient_is_the_inverse_turn(cpa):
    """<rope(x), g> = <x, inverse(g)> for every x and g (the transpose), and
    a central difference of the loss in one direction, in fp32: the terms of
    the sums are products of size 1 off by 2^-20 each."""
    n, h, d = 64, 3, 128
    gen = torch.Generator().manual_seed(3)
    x, g, v = (torch.randn(n, h, d, generator=gen).cuda() for _ in range(3))
    plan = cpa.RopePlan(d, 96, 3, axes_of(96, 3, False))
    pos = ints(np.random.default_rng(3).integers(0, 9000, (3, n)))

    def turn(t, inverse=False):
        out = torch.empty_like(t)
        cpa.cp_rope(plan, pos, [t], [out], inverse=inverse)
        return out
    grad = turn(g, True)
    a, b = (turn(x).double() * g.double()).sum(), (x.double() * grad.double()).sum()
    size = (x.abs() * g.abs()).sum().item() + (turn(x).abs() * g.abs()).sum().item()
    assert abs(a - b) <= 2.0 ** -20 * size
    up, down = ((turn(x + s * v).double() * g.double()).sum() for s in (0.5, -0.5))  # linear: the difference is exact but for rounding
    assert abs((up - down) - (v.double() * grad.double()).sum()) <= 4 * 2.0 ** -20 * (size + (v.abs() * g.abs()).sum().item())
    back = turn(turn(x), True)
    assert (back - x).abs().max() <= 2.0 ** -19 * x.abs().max()


def test_rope_sequence_sharded(cpa):
    """Around cp_attn_fwd and cp_attn_bwd: queries and keys of a zigzag ring
    turned by their slots' positions; dQ and dK turned back equal the gradients
    of the whole, against fp64 of the formula on unrotated inputs."""
    L, Hq, Hkv, d = 512, 4, 2, 64
    plan = cpa.Plan(L, Hq, Hkv, d, ring_degree=4, layout=cpa.CP_LAYOUT_ZIGZAG)
    idx = plan.index_map()
    gen = torch.Generator().manual_seed(4)
    q, k, v, do = (torch.randn(L, h, d, generator=gen).to(BF) for h in (Hq, Hkv, Hkv, Hq))
    axis = axes_of(d, 2, True)
    rope = cpa.RopePlan(d, d, 2, axis)
    pos = np.stack([idx, idx % 17])
    sharded = [x[torch.from_numpy(idx.astype(np.int64))].contiguous().cuda() for x in (q, k, v, do)]
    turned = [torch.empty_like(x) for x in sharded[:2]]
    cpa.cp_rope(rope, ints(pos), sharded[:2], turned)
    o, lse = torch.empty_like(sharded[0]), torch.empty(plan.P, Hq, plan.n, device="cuda")
    cpa.cp_attn_fwd(plan, *turned, sharded[2], o, lse, cpa.alloc_workspace(plan))
    grads = [torch.empty(x.shape, device="cuda") for x in sharded[:3]]
    cpa.cp_attn_bwd(plan, *turned, sharded[2], o, lse, sharded[3], *grads, cpa.alloc_workspace(plan, cpa.CP_OP_BWD))
    dq, dk = (torch.empty_like(x) for x in grads[:2])
    cpa.cp_rope(rope, ints(pos), grads[:2], [dq, dk], inverse=True)

    def turn(x):
        c, s = (torch.from_numpy(f(pos[axis].T * frequencies(d)))[:, None] for f in (np.cos, np.sin))
        inv = torch.argsort(torch.from_numpy(idx.astype(np.int64)))
        c, s, a, b = c[inv], s[inv], x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)
    leaves = [x.double().requires_grad_() for x in (q, k, v)]
    qq, kk = turn(leaves[0]), turn(leaves[1])
    sc = torch.einsum("ihd,jhd->hij", qq, kk.repeat_interleave(Hq // Hkv, 1)) * d ** -0.5
    sc = sc.masked_fill(torch.ones(L, L, dtype=torch.bool).triu(1), float("-inf"))
    torch.einsum("hij,jhd->ihd", sc.softmax(-1), leaves[2].repeat_interleave(Hq // Hkv, 1)).backward(do.double())
    for got, leaf in zip((dq, dk, grads[2]), leaves):
        ref = leaf.grad[torch.from_numpy(idx.astype(np.int64))]
        err = (got.double().cpu() - ref).abs()
        # The backward's bounds (1e-2 and 1e-3 of the gradient's size), twice for queries and keys that the rotation has rounded.
        assert err.max() <= 2e-2 * max(1.0, ref.abs().max()) and err.mean() <= 2e-3 * max(1.0, ref.square().mean().sqrt())


def test_rope_offsets_beyond_32_bits(cpa):
    """Rows 2^27 elements apart: the last lies 2^32 elements behind the first."""
    n, stride = 33, 1 << 27
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("not enough memory")
    buf = torch.empty(n * stride, dtype=BF, device="cuda")
    x = buf.as_strided((n, 2, 128), (stride, 128, 1))
    out = buf[512:].as_strided((n, 2, 128), (stride, 128, 1))
    x.copy_(torch.randn(n, 2, 128, generator=torch.Generator().manual_seed(5)))
    plan = cpa.RopePlan(128, 128)
    pos = np.arange(n)[None] * 999
    cpa.cp_rope(plan, ints(pos), [x], [out])
    ref, size = rotate(x.double().cpu().numpy(), pos, [0] * 64, frequencies(128))
    check(out, ref, size, BF)


def test_rope_infinite_and_nan_elements(cpa):
    """What is not finite stays within its pair."""
    x = torch.randn(5, 2, 64, generator=torch.Generator().manual_seed(6))
    x[1, 0, 3], x[2, 1, 40] = float("inf"), float("nan")
    plan = cpa.RopePlan(64, 64)
    out = torch.empty(5, 2, 64, device="cuda")
    cpa.cp_rope(plan, ints(np.arange(5) * 11 + 1), [x.cuda()], [out])
    bad = ~torch.isfinite(out.cpu())
    want = torch.zeros_like(bad)
    want[1, 0, [3, 35]] = want[2, 1, [8, 40]] = True
    assert torch.equal(bad, want)


def test_rope_captured_and_on_another_stream(cpa):
    plan = cpa.RopePlan(128, 128, 2, axes_of(128, 2, True))
    x, pos, out = torch.randn(40, 4, 128, device="cuda").to(BF), ints(np.zeros((2, 40))), torch.empty(40, 4, 128, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cpa.cp_rope(plan, pos, [x], [out])
    side.synchronize()
    assert torch.equal(out, x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cpa.cp_rope(plan, pos, [x], [out])
    for seed in range(3):
        x.copy_(torch.randn(40, 4, 128, generator=torch.Generator().manual_seed(seed)))
        p = np.random.default_rng(seed).integers(0, 1000, (2, 40))
        pos.copy_(ints(p))
        graph.replay()
        ref, size = rotate(x.double().cpu().numpy(), p, axes_of(128, 2, True), frequencies(128))
        check(out, ref, size, BF)


# ---------------------------------------------------------------- into a cache

APPEND = {
    "decode": (dict(past=[0, 15, 16, 31, 500], new=[1] * 5, d=64, Hq=4, Hkv=4), dict(rope_dim=64, rope_axes=3)),
    "prompts_fp16": (dict(past=[0, 7, 0], new=[50, 1, 33], d=128, Hq=4, Hkv=2, dtype=FP, heads_first=True, page_size=32), dict(rope_dim=128, rope_axes=3)),
    "interleaved_partial": (dict(past=[3, 60], new=[4, 2], d=64, Hq=6, Hkv=3), dict(rope_dim=32, rope_interleaved=True, rope_axes=2)),
    "halves_partial": (dict(past=[3, 60], new=[4, 2], d=128, Hq=7, Hkv=1), dict(rope_dim=48, rope_axes=4)),
    "padded": (dict(past=[2, 0, 9], new=[1, 0, 3], pad=5, d=128, Hq=4, Hkv=2), dict(rope_dim=128, rope_axes=2)),
}


@pytest.mark.parametrize("cycled", [False, True])
@pytest.mark.parametrize("name", list(APPEND))
def test_append_of_several_axes(cpa, name, cycled):
    kw, plan_kw = APPEND[name]
    b = Batch(seed=len(name), appended=False, **kw)
    rd, axes = plan_kw["rope_dim"], plan_kw["rope_axes"]
    axis, positions = axes_of(rd, axes, cycled), np.random.default_rng(7).integers(0, 2 ** 20, (axes, b.N))
    plan = b.plan(cpa, rope_axis=axis, **plan_kw)
    cache, batch, q, k, v = b.to_gpu(cpa, positions)
    q_out = torch.full((b.N, b.Hq, b.d), float("nan"), dtype=b.dtype, device="cuda")
    cpa.cp_cache_append(plan, cache, batch, q, k, v, q_out)
    n, il = b.N - b.pad, plan_kw.get("rope_interleaved", False)
    for got, x in ((q_out[:n], b.q[:n]), (torch.stack([cache.k[int(b.page_table[s][at // b.ps]), at % b.ps] for s, at in b_rows(b)]), b.k[:n])):
        ref, size = rotate(x.double().numpy(), positions[:, :n], axis, frequencies(rd), il)
        check(got, ref, size, b.dtype)
    assert torch.isnan(q_out[n:]).all()
    for (s, at), row in zip(b_rows(b), b.v):
        assert torch.equal(cache.v[int(b.page_table[s][at // b.ps]), at % b.ps].cpu(), row)


def b_rows(b):
    return [(s, b.past[s] + i) for s in range(b.B) for i in range(b.new[s])]


def test_append_of_several_axes_without_positions(cpa):
    """Text behind a prefix: every axis has the token's place, bit for bit what one axis gives."""
    b = Batch(past=[2, 0, 9, 4], new=[1, 2, 1, 1], prefixes=[(2, 77), (1, 500)], d=128, Hq=4, Hkv=2, seed=9, appended=False)
    got = []
    for kw in (dict(), dict(rope_axes=3, rope_axis=axes_of(128, 3, True))):
        cache, batch, q, k, v = b.to_gpu(cpa)
        q_out = torch.empty(b.N, 4, 128, dtype=BF, device="cuda")
        cpa.cp_cache_append(b.plan(cpa, rope_dim=128, **kw), cache, batch, q, k, v, q_out)
        got.append((q_out, cache.k.view(torch.int16)))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


def test_append_refuses_other_axes(cpa):
    b = Batch(past=[2], new=[1], d=64, Hq=4, Hkv=2, seed=9, appended=False)
    for plan_kw, positions in ((dict(), np.zeros((2, 1))), (dict(rope_axes=2, rope_axis=[0] * 32), np.zeros(1)),
                               (dict(rope_axes=2, rope_axis=[0] * 32), np.zeros((3, 1)))):
        cache, batch, q, k, v = b.to_gpu(cpa, positions)
        with pytest.raises(cpa.CPError, match="axes"):
            cpa.cp_cache_append(b.plan(cpa, rope_dim=64, **plan_kw), cache, batch, None, k, v)
