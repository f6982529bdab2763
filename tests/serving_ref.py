"""Plain 64-bit implementations of the operators around a serving step's
attention (numpy; no code shared with the CUDA path): rotation by several
axes, verification of drafts, the pages of a cache."""
from __future__ import annotations

import numpy as np


def rotate(x, positions, axis_of, freqs, interleaved=False, inverse=False):
    """x [n][heads][d] turned to positions [axes][n]; (result, size of the rounded terms)."""
    x = np.asarray(x, dtype=np.float64)
    half = len(freqs)
    a = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    theta = np.asarray(positions)[np.asarray(axis_of)].T.astype(np.float64) * np.asarray(freqs)
    if inverse:
        theta = -theta
    c, s = np.cos(theta)[:, None], np.sin(theta)[:, None]
    out, size = x.copy(), np.zeros_like(x)
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return out, size


def verify(start, kv_len, tokens, p, q, accept_u, sample_u, fill=-7):
    """(accepted, out_tokens, kv_len_out) as cp_verify_drafts defines them; rows
    and sequences that it does not write hold `fill`."""
    p = np.asarray(p, dtype=np.float64)
    q = None if q is None else np.asarray(q, dtype=np.float64)
    weight = lambda x: np.where((x > 0) & (x < np.inf), x, 0.0)  # noqa: E731
    N, V = p.shape
    B = len(start) - 1
    accepted, kv, out = np.full(B, fill), np.full(B, fill), np.full(N, fill)
    for s in range(B):
        t0, n = int(start[s]), int(start[s + 1]) - int(start[s])
        a = 0
        if n == 0:
            accepted[s], kv[s] = 0, kv_len[s]
            continue
        while a < n - 1:
            x = int(tokens[t0 + a + 1])
            if not 0 <= x < V:
                break
            qx = 1.0 if q is None else (q[t0 + a, x] if q[t0 + a, x] > 0 else 0.0)
            with np.errstate(invalid="ignore"):
                if not float(accept_u[t0 + a]) * qx < weight(p[t0 + a, x]):
                    break
            a += 1
        w = weight(p[t0 + a])
        if a < n - 1:
            if q is None:
                less = np.zeros(V)
                if 0 <= tokens[t0 + a + 1] < V:
                    less[int(tokens[t0 + a + 1])] = 1.0
            else:
                less = np.where(q[t0 + a] > 0, q[t0 + a], 0.0)
            rest = np.where(w > less, w - np.minimum(less, w), 0.0)
            if rest.sum() > 0:
                w = rest
        r = np.float32(sample_u[s])
        r = 0.0 if not r >= 0 else float(min(r, np.float32(1 - 2.0 ** -24)))
        sums = np.cumsum(w)
        k = int(np.searchsorted(sums, r * sums[-1], side="right")) if sums[-1] > 0 else -1
        for i in range(n):
            out[t0 + i] = tokens[t0 + i + 1] if i < a else k if i == a else -1
        accepted[s], kv[s] = a, kv_len[s] - (n - 1 - a)
    return accepted, out, kv


class Pool:
    """refs and tables, one page after another."""

    def __init__(self, pages, page_size):
        self.refs, self.ps = np.zeros(pages, np.int64), page_size

    def _free(self):
        """Free pages, the lowest first (nothing is let go while it runs)."""
        return iter(np.flatnonzero(self.refs == 0).tolist())

    def _take(self, table, r, want, free):
        while table.held[r] < want:
            page = next(free)
            self.refs[page] = 1
            table.pages[r, table.held[r]] = page
            table.held[r] += 1

    def resize(self, table, tokens):
        wants = [table.held[r] if t < 0 else -(-int(t) // self.ps) for r, t in enumerate(tokens)]
        bad = [w > table.pages.shape[1] for w in wants]
        for r, w in enumerate(wants):
            while not bad[r] and table.held[r] > w:
                table.held[r] -= 1
                self.refs[table.pages[r, table.held[r]]] -= 1
                table.pages[r, table.held[r]] = -1
        left, served, free = int((self.refs == 0).sum()), [], self._free()
        for r, w in enumerate(wants):
            need = 0 if bad[r] else max(0, w - table.held[r])
            left -= need
            served.append(int(not bad[r] and (need == 0 or left >= 0)))
            if served[-1]:
                self._take(table, r, w, free)
        return served

    def fork(self, src, dst, parent, tokens):
        """(served, moves): moves are (src, dst, tokens)."""
        left, served, moves, free = int((self.refs == 0).sum()), [], [], self._free()
        src_held, dst_held, src_pages = src.held.copy(), dst.held.copy(), src.pages.copy()
        for r, (p, t) in enumerate(zip(parent, tokens)):
            if p < 0:
                served.append(1)
                continue
            full, part = divmod(int(t), self.ps)
            want = full + (part > 0)
            if t < 0 or p >= len(src_held) or dst_held[r] or not want <= src_held[p] or want > dst.pages.shape[1]:
                served.append(0)
                continue
            left -= part > 0
            served.append(int(part == 0 or left >= 0))
            if not served[-1]:
                continue
            dst.pages[r, :full] = src_pages[p, :full]
            for page in src_pages[p, :full]:
                self.refs[page] += 1
            dst.held[r] = full
            if part:
                self._take(dst, r, want, free)
                moves.append((int(src_pages[p, full]), int(dst.pages[r, full]), part))
        return served, moves

    def compact(self, *tables):
        """(used, moves)."""
        used = int((self.refs > 0).sum())
        holes = [p for p in range(used) if self.refs[p] == 0]
        high = [p for p in range(used, len(self.refs)) if self.refs[p] > 0]
        to = np.arange(len(self.refs))
        to[high] = holes
        for t in tables:
            for r in range(len(t.held)):
                t.pages[r, :t.held[r]] = to[t.pages[r, :t.held[r]]]
        self.refs[holes], self.refs[high] = self.refs[high], 0
        return used, [(a, b, self.ps) for a, b in zip(high, holes)]


class Table:
    def __init__(self, rows, columns):
        self.pages, self.held = np.full((rows, columns), -1, np.int64), np.zeros(rows, np.int64)
