"""Plain fp64 implementations of the paged-cache operators and the batches
they are tested on (numpy; no code shared with the CUDA path)."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


class Batch:
    """A ragged batch on a paged cache, on the CPU.

    past, new: tokens held and new of each sequence; prefixes: list of
    (sequences, length), consecutive from sequence `first` on.  Rows of the
    cache that belong to nothing, and padding rows, hold NaN."""

    def __init__(self, past, new, page_size=16, Hq=4, Hkv=2, d=64, dtype=torch.bfloat16, prefixes=(), first=0, pad=0,
                 heads_first=False, seed=0, spare=3, appended=True):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        self.past, self.new = list(past), list(new)
        self.kv = [a + b for a, b in zip(past, new)]
        self.ps, self.Hq, self.Hkv, self.d, self.dtype = page_size, Hq, Hkv, d, dtype
        self.B, self.pad = len(past), pad
        self.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.N = int(self.start[-1]) + pad
        self.plen = [n for _, n in prefixes]
        self.first = (first + np.concatenate([[0], np.cumsum([c for c, _ in prefixes])])).astype(np.int32)
        self.of = [next((p for p in range(len(prefixes)) if self.first[p] <= b < self.first[p + 1]), -1) for b in range(self.B)]
        counts = [-(-k // page_size) for k in self.kv] + [-(-k // page_size) for k in self.plen]
        self.pages = sum(counts) + spare
        ids = rng.permutation(self.pages).astype(np.int32)

        def table(counts, at):
            out = np.full((len(counts), max(list(counts) + [1]) + 1), -1, np.int32)  # -1 behind the last page
            for i, c in enumerate(counts):
                out[i, :c] = ids[at:at + c]
                at += c
            return out, at
        self.page_table, at = table(counts[:self.B], 0)
        self.prefix_table, _ = table(counts[self.B:], at)

        def normal(*shape):
            return torch.randn(*shape, generator=gen).to(dtype)
        cache = [torch.full((self.pages, page_size, Hkv, d), float("nan"), dtype=dtype) for _ in range(2)]
        for b in range(self.B + len(self.plen)):
            n = self.kv[b] if b < self.B else self.plen[b - self.B]
            if b < self.B and not appended:
                n = self.past[b]
            rows = self.page_table[b] if b < self.B else self.prefix_table[b - self.B]
            j = np.arange(n)
            for c in cache:
                c[torch.from_numpy(rows[j // page_size].astype(np.int64)), torch.from_numpy(j % page_size)] = normal(n, Hkv, d)
        if heads_first:
            cache = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in cache]
        self.k_cache, self.v_cache = cache
        self.qkv = normal(self.N, Hq + 2 * Hkv, d)
        if pad:
            self.qkv[self.N - pad:] = float("nan")
        self.q, self.k, self.v = self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]

    # ---- on the GPU
    def plan(self, cpa, **kw):
        o = dict(page_size=self.ps, dtype=self.dtype, max_seqs=self.B, max_tokens=max(1, self.N), max_new=max(1, max(self.new)),
                 max_pages=self.page_table.shape[1], max_prefixes=len(self.plen),
                 max_prefix_pages=self.prefix_table.shape[1] if self.plen else 0)
        o.update(kw)
        return cpa.PagedPlan(self.Hq, self.Hkv, self.d, **o)

    def to_gpu(self, cpa, positions=None):
        """cache, batch and the q, k, v views of one fused projection, on the GPU."""
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.int32).cuda()  # noqa: E731
        pre = dict(prefix_first=t(self.first), prefix_len=t(np.array(self.plen)), prefix_table=t(self.prefix_table)) if self.plen else {}
        cuda = lambda x: torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda").copy_(x)  # noqa: E731
        cache = cpa.PagedCache(cuda(self.k_cache), cuda(self.v_cache))
        batch = cpa.PagedBatch(t(self.start), t(np.array(self.kv)), t(self.page_table), n_tokens=self.N,
                               positions=None if positions is None else t(positions), **pre)
        qkv = self.qkv.cuda()
        Hq, Hkv = self.Hq, self.Hkv
        return cache, batch, qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]

    # ---- fp64
    def keys_of(self, b, k_cache=None, v_cache=None):
        """Own keys and values of sequence b, in order."""
        j = np.arange(self.kv[b])
        return [c.double().numpy()[self.page_table[b][j // self.ps], j % self.ps]
                for c in (self.k_cache if k_cache is None else k_cache, self.v_cache if v_cache is None else v_cache)]

    def prefix_keys(self, p):
        j = np.arange(self.plen[p])
        return [c.double().numpy()[self.prefix_table[p][j // self.ps], j % self.ps] for c in (self.k_cache, self.v_cache)]

    def attention(self, causal=True, scale=0.0, q=None, k_cache=None, v_cache=None):
        """(O [N][Hq][d], LSE [Hq][N], weight of the rounding of P: sum p |v|,
        largest |scale| |q| |k| of the row) in fp64; NaN in padding rows."""
        scale = scale or 1.0 / math.sqrt(self.d)
        q = (self.q if q is None else q).double().numpy()
        O = np.full((self.N, self.Hq, self.d), np.nan)
        A = np.full((self.N, self.Hq, self.d), np.nan)
        LSE = np.full((self.Hq, self.N), np.nan)
        W = np.full((self.N, self.Hq), np.nan)
        G = self.Hq // self.Hkv
        for b in range(self.B):
            kv = self.keys_of(b, k_cache, v_cache)
            pre = self.prefix_keys(self.of[b]) if self.of[b] >= 0 else [np.zeros((0, self.Hkv, self.d))] * 2
            k, v = (np.concatenate([x, y]) for x, y in zip(pre, kv))
            for i in range(self.new[b]):
                t = int(self.start[b]) + i
                seen = len(pre[0]) + (max(0, self.kv[b] - self.new[b] + i + 1) if causal else self.kv[b])
                for h in range(self.Hq):
                    kk, vv = k[:seen, h // G], v[:seen, h // G]
                    if seen == 0:
                        O[t, h], A[t, h], LSE[h, t], W[t, h] = 0.0, 0.0, -np.inf, 0.0
                        continue
                    s = kk @ q[t, h] * scale
                    m = s.max()
                    p = np.exp(s - m)
                    LSE[h, t] = m + math.log(p.sum())
                    p /= p.sum()
                    O[t, h], A[t, h] = p @ vv, p @ np.abs(vv)
                    W[t, h] = scale * np.linalg.norm(q[t, h]) * np.linalg.norm(kk, axis=1).max()
        return O, LSE, A, W

    def append(self, rope_dim, freqs, interleaved=False, positions=None):
        """(q_out, k_cache, v_cache, size of the rounded terms of q_out and k_cache) in fp64."""
        out = self.q.double().numpy().copy()
        kc, vc = self.k_cache.double().numpy().copy(), self.v_cache.double().numpy().copy()
        q_size, k_size = np.zeros_like(out), np.zeros_like(kc)
        half = rope_dim // 2
        ia, ib = (np.arange(0, rope_dim, 2), np.arange(1, rope_dim, 2)) if interleaved else (np.arange(half), half + np.arange(half))
        for b in range(self.B):
            for i in range(self.new[b]):
                t, at = int(self.start[b]) + i, self.past[b] + i
                pos = positions[t] if positions is not None else at + (self.plen[self.of[b]] if self.of[b] >= 0 else 0)
                c, s = np.cos(pos * np.asarray(freqs)), np.sin(pos * np.asarray(freqs))
                row = (self.page_table[b][at // self.ps], at % self.ps)
                for x, y, size in ((self.q[t].double().numpy(), out[t], q_size[t]), (self.k[t].double().numpy(), None, None)):
                    z, w = x.copy(), np.zeros_like(x)
                    z[:, ia], z[:, ib] = x[:, ia] * c - x[:, ib] * s, x[:, ib] * c + x[:, ia] * s
                    w[:, ia] = w[:, ib] = np.abs(x[:, ia]) + np.abs(x[:, ib])
                    if y is None:
                        kc[row], k_size[row] = z, w
                    else:
                        y[:], size[:] = z, w
                vc[row] = self.v[t].double().numpy()
        return out, kc, vc, q_size, k_size


def check_attention(got_o, got_lse, ref, dtype, d, n_valid, what=""):
    """O and LSE against the fp64 reference.

    A score is an fp32 sum of d products: off by at most
    ds = d 2^-24 scale |q| |k|, plus the rounding of its scaling and of the
    exponent, 4 2^-24 of its size, itself at most scale |q| |k|.  A weight p is
    then off by ds + 2^-21 (the exponential's approximation) relatively, the
    sum l as much, and p is rounded to the cache's type for the product with V
    (half a step).  O is rounded once more at the end."""
    O, LSE, A, W = ref
    o, lse = got_o.double().cpu().numpy(), got_lse.double().cpu().numpy()
    ds = (d + 4) * 2.0 ** -24 * W + 2.0 ** -21
    p_step = HALF_STEP[dtype]
    bound = HALF_STEP[got_o.dtype] * np.abs(O) + 1.02 * (p_step + 2 * ds[:, :, None]) * A + 1e-30
    if got_o.dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a step of the smallest fp16 numbers
    err = np.abs(o[:n_valid] - O[:n_valid])
    assert np.all(err <= bound[:n_valid]), (
        f"{what}: O off by {np.nanmax(err)}, {np.nanmax(err / bound[:n_valid])} of its bound, at "
        f"{np.argwhere(~(err <= bound[:n_valid]))[:4].tolist()}")
    L, G = LSE[:, :n_valid], lse[:, :n_valid]
    assert np.array_equal(np.isneginf(L), np.isneginf(G)), f"{what}: rows without keys differ"
    fin = np.isfinite(L)
    le = np.abs(np.where(fin, G, 0) - np.where(fin, L, 0))
    lb = ds.T[:, :n_valid] + 4 * 2.0 ** -24 * np.where(fin, np.abs(L), 0) + 2.0 ** -20
    assert np.all(le <= lb), f"{what}: LSE off by {le.max()}, {(le / lb).max()} of its bound"
