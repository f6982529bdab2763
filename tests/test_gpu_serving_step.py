"""The operators of a serving step together: prompts of text and images into
two layers' caches, forked into samples, decoded with drafts, verified, their
pages trimmed and taken, the cache compacted; the attention of every step
against fp64 over the sequences' own tokens."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

pytestmark = pytest.mark.gpu

from paged_ref import check_attention  # noqa: E402
from serving_ref import rotate, verify  # noqa: E402
from test_gpu_paged_use import ints  # noqa: E402

BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cpa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import context_long_sequence_gb300 as m
    return m


def attention(q, keys, values, start, G, d):
    """Reference tuple of paged_ref.check_attention over rows that end their sequences."""
    N, Hq = q.shape[:2]
    O, A, LSE, W = np.zeros((N, Hq, d)), np.zeros((N, Hq, d)), np.zeros((Hq, N)), np.zeros((N, Hq))
    for s in range(len(start) - 1):
        n = start[s + 1] - start[s]
        for i in range(n):
            t, seen = start[s] + i, len(keys[s]) - n + i + 1
            for h in range(Hq):
                k, v = keys[s][:seen, h // G], values[s][:seen, h // G]
                x = k @ q[t, h] * d ** -0.5
                p = np.exp(x - x.max())
                LSE[h, t] = x.max() + np.log(p.sum())
                p /= p.sum()
                O[t, h], A[t, h] = p @ v, p @ np.abs(v)
                W[t, h] = d ** -0.5 * np.linalg.norm(q[t, h]) * np.linalg.norm(k, axis=1).max()
    return O, LSE, A, W


@pytest.mark.parametrize("dtype,d,ps", [(BF, 128, 16), (FP, 64, 32)])
def test_a_serving_loop(cpa, dtype, d, ps):
    Hq, Hkv, V, rows, columns, pages, layers = 8, 2, 500, 6, 16, 80, 2
    G, axes = Hq // Hkv, 3
    rng, gen = np.random.default_rng(d), torch.Generator().manual_seed(d)
    axis, freqs = [j % axes for j in range(d // 2)], 10000.0 ** (-2.0 * np.arange(d // 2) / d)
    make = lambda max_new: cpa.PagedPlan(Hq, Hkv, d, page_size=ps, dtype=dtype, max_seqs=rows, max_tokens=rows * 100, max_new=max_new,  # noqa: E731
                                         max_pages=columns, rope_dim=d, rope_axes=axes, rope_axis=axis)
    prompts, steps = make(100), make(4)
    caches = [cpa.PagedCache(*(torch.full((pages, ps, Hkv, d), float("nan"), dtype=dtype, device="cuda") for _ in range(2))) for _ in range(layers)]
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = cpa.PageTable(torch.full((rows, columns), -1, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda"))
    moves, served, ws = cpa.PageMoves(40), torch.zeros(rows, dtype=torch.int32, device="cuda"), cpa.alloc_paged_workspace(prompts)
    pages_ws = cpa.alloc_pages_workspace(pages)
    # The sequences as they should be: per layer, the rotated keys and the values as the cache's type holds them.
    held = [[(np.zeros((0, Hkv, d)), np.zeros((0, Hkv, d))) for _ in range(rows)] for _ in range(layers)]
    length = np.zeros(rows, int)

    def step(plan, new):
        """The new tokens of every row through the layers: append, attend."""
        nonlocal length
        start = np.concatenate([[0], np.cumsum(new)])
        N = int(start[-1])
        length = length + new
        cpa.cp_pages_resize(plan, refs, table, ints(length), served)
        assert served.all()
        positions = rng.integers(0, 3000, (axes, N))
        batch = cpa.PagedBatch(ints(start), ints(length), table.pages, n_tokens=N, positions=ints(positions))
        for layer, cache in enumerate(caches):
            qkv = torch.randn(N, Hq + 2 * Hkv, d, generator=gen).to(dtype)
            x = qkv.cuda()
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            q_out, o, lse = torch.empty(N, Hq, d, dtype=dtype, device="cuda"), torch.empty(N, Hq, d, dtype=dtype, device="cuda"), torch.empty(Hq, N, device="cuda")
            cpa.cp_cache_append(plan, cache, batch, q, k, v, q_out)
            cpa.cp_attn_paged(plan, cache, batch, q_out, o, lse, ws)
            turned, size = rotate(qkv[:, Hq:Hq + Hkv].double().numpy(), positions, axis, freqs)
            pages_now, got_k = table.pages.cpu().numpy(), cache.k.cpu().double().numpy()
            for s in range(rows):
                t = np.arange(length[s] - new[s], length[s])
                mine = got_k[pages_now[s, t // ps], t % ps]
                err = np.abs(mine - turned[start[s]:start[s + 1]])
                half = 2.0 ** -8 if dtype == BF else 2.0 ** -11
                assert np.all(err <= half * np.abs(turned[start[s]:start[s + 1]]) + 2.0 ** -21 * size[start[s]:start[s + 1]] + 2.0 ** -25)
                hk, hv = held[layer][s]
                held[layer][s] = (np.concatenate([hk, mine]), np.concatenate([hv, qkv[start[s]:start[s + 1], Hq + Hkv:].double().numpy()]))
            ref = attention(q_out.double().cpu().numpy(), [h[0] for h in held[layer]], [h[1] for h in held[layer]], start, G, d)
            check_attention(o, lse, ref, dtype, d, N, f"layer {layer}")
        return batch, start, N

    def settle(lengths):
        nonlocal length
        length = np.array(lengths)
        for layer in held:
            for s in range(rows):
                layer[s] = tuple(x[:length[s]] for x in layer[s])

    step(prompts, np.array([70, 33, 0, 0, 0, 0]))
    for turn in range(5):
        if turn in (0, 3):  # samples of the first rows
            parent = np.array([-1, -1, 0, 0, 1, -1]) if turn == 0 else np.array([-1, -1, -1, -1, 2, 2])
            asked = np.where(parent >= 0, length[parent], 0)
            cpa.cp_pages_fork(steps, refs, table, table, ints(parent), ints(asked), moves, served)
            cpa.cp_pages_copy(steps, caches, caches, moves)
            assert served.all()
            for s, p in enumerate(parent):
                if p >= 0:
                    length[s] = length[p]
                    for layer in held:
                        layer[s] = layer[p]
        new = np.where(length > 0, rng.integers(1, 5, rows), 0)
        batch, start, N = step(steps, new)
        p = torch.softmax(2 * torch.randn(N, V, generator=gen), -1)
        q = torch.softmax(torch.log(p) + 0.3 * torch.randn(N, V, generator=gen), -1)
        tokens = torch.cat([torch.zeros(1, dtype=torch.int64), torch.multinomial(q, 1, generator=gen)[:-1, 0]])
        u, r = torch.rand(N, generator=gen), torch.rand(rows, generator=gen)
        out = [torch.zeros(k, dtype=torch.int32, device="cuda") for k in (rows, N, rows)]
        cpa.cp_verify_drafts(steps, batch, ints(tokens.numpy()), p.cuda(), q.cuda(), u.cuda(), r.cuda(), *out)
        want = verify(start, length, tokens.numpy(), p.double().numpy(), q.double().numpy(), u.numpy(), r.numpy())
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(out, want))
        # What was not accepted leaves, straight from the verification's lengths; once a user too.
        keep = out[2]
        if turn == 2:
            keep[4:] = 0
        cpa.cp_pages_resize(steps, refs, table, keep, served)
        settle(keep.cpu().numpy())
        assert table.held.tolist() == [-(-int(n) // ps) for n in length]
        if turn % 2:
            used = torch.zeros(1, dtype=torch.int32, device="cuda")
            cpa.cp_pages_compact(steps, refs, [table], moves, pages_ws, used=used)
            cpa.cp_pages_copy(steps, caches, caches, moves)
            assert (refs[:used.item()] > 0).all() and not refs[used.item():].any()
    cpa.cp_pages_resize(steps, refs, table, ints(np.zeros(rows)), served)
    assert not refs.any() and (table.pages == -1).all()
