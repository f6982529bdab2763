"""Host-side refusals of cp_rope, cp_verify_drafts, the cp_pages_ calls and plans
of several axes (no GPU: the checks come before any use of the addresses)."""
import ctypes
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(__file__))

from test_paged_host import FAKE, c_args, cpa, make_plan  # noqa: E402, F401

A = ctypes.addressof


# ---------------------------------------------------------------- rotation

def rope_plan(cpa, **kw):  # noqa: F811
    o = dict(d=128, rope_dim=128)
    o.update(kw)
    return cpa.RopePlan(**o)


@pytest.mark.parametrize("kw,code", [
    (dict(d=72, rope_dim=64), -2), (dict(d=272, rope_dim=16), -2), (dict(d=0), -1), (dict(rope_dim=0), -1), (dict(rope_dim=144), -1),
    (dict(rope_dim=24), -2), (dict(rope_axes=0), -1), (dict(rope_axes=5, rope_axis=[0] * 64), -1),
    (dict(rope_axes=3), -1), (dict(rope_axes=3, rope_axis=[0] * 63), -1), (dict(rope_axes=3, rope_axis=[0] * 63 + [3]), -1),
    (dict(rope_axes=2, rope_axis=[-1] + [0] * 63), -1), (dict(rope_base=0.0), -1), (dict(rope_base=float("inf")), -1),
    (dict(rope_freqs=[1.0] * 63), -1), (dict(rope_freqs=[float("nan")] * 64), -1),
])
def test_rope_plan_validation(cpa, kw, code):  # noqa: F811
    with pytest.raises(cpa.CPError) as e:
        rope_plan(cpa, **kw)
    assert e.value.code == code


def test_rope_plan_versions(cpa):  # noqa: F811
    h, L = ctypes.c_void_p(), cpa._L()
    assert L.cp_rope_create(None, ctypes.byref(h)) == -1
    assert L.cp_rope_create(ctypes.byref(cpa.cp_rope_desc_t()), ctypes.byref(h)) == -1
    L.cp_rope_destroy(None)


def test_rope_refusals(cpa):  # noqa: F811
    plan, L = rope_plan(cpa), cpa._L()

    def call(n=4, pos=FAKE, jobs=1, ti=0, to=0, inverse=0, **kw):
        j = cpa.cp_rope_job_t(FAKE, FAKE + 4096, 2, 256, 256)
        for k, v in kw.items():
            setattr(j, k, v)
        return L.cp_rope(plan.handle, n, pos, jobs, A(j), ti, to, inverse, None)
    assert call(n=-1) == -1 and call(n=0) == 0 and call(pos=None) == -1 and call(pos=FAKE + 2) == -3
    assert call(jobs=0) == -1 and call(jobs=9) == -1 and call(inverse=2) == -1
    assert call(ti=3, to=3) == -1 and call(ti=-1, to=-1) == -1 and call(ti=0, to=1) == -2 and call(ti=1, to=0) == -2
    assert call(inp=None) == -1 and call(out=None) == -1 and call(inp=FAKE + 8) == -3 and call(out=FAKE + 8) == -3
    assert call(heads=0) == -1 and call(heads=65537) == -1
    assert call(in_stride=248) == -1 and call(out_stride=248) == -1 and call(in_stride=260) == -1 and call(in_stride=1 << 36) == -1
    assert call(out_stride=258, to=2) == -1
    assert call(out=FAKE, out_stride=512) == -1      # in place with another stride
    assert call(out=FAKE, to=2) == -1                # or another type
    assert L.cp_rope(None, 4, FAKE, 1, A(cpa.cp_rope_job_t()), 0, 0, 0, None) == -1


def test_rope_binding_refusals(cpa):  # noqa: F811
    plan = rope_plan(cpa, rope_axes=2, rope_axis=[0, 1] * 32)
    x, pos = torch.zeros(3, 2, 128), torch.zeros(2, 3, dtype=torch.int32)

    def call(positions=pos, xs=(x,), outs=(x,)):
        cpa.cp_rope(plan, positions, list(xs), list(outs))
    for kw, why in [(dict(xs=(), outs=()), "1 to 8"), (dict(xs=(x, x)), "1 to 8"), (dict(positions=pos[0]), "positions"),
                    (dict(positions=pos.long()), "positions"), (dict(positions=torch.zeros(3, 2, dtype=torch.int32).T), "positions"),
                    (dict(outs=(x[:, :1],)), "contiguous heads"), (dict(xs=(x[..., :64],)), "contiguous heads"),
                    (dict(xs=(x[:2],), outs=(x[:2],)), "contiguous heads"),
                    (dict(xs=(torch.zeros(2, 3, 128).transpose(0, 1),)), "contiguous heads"),
                    (dict(xs=(x, x.half()), outs=(x, x)), "one type"), (dict(xs=(x.double(),)), "served"),
                    (dict(), "not the current")]:
        with pytest.raises(cpa.CPError, match=why):
            call(**kw)


@pytest.mark.parametrize("kw,ok", [
    (dict(rope_axes=3, rope_axis=[0, 1, 2] * 21 + [0]), True), (dict(rope_axes=4, rope_axis=[3] * 64), True),
    (dict(rope_axes=5, rope_axis=[0] * 64), False), (dict(rope_axes=-1), False), (dict(rope_axes=2), False),
    (dict(rope_axes=2, rope_axis=[0] * 63 + [2]), False), (dict(rope_axes=2, rope_axis=[0] * 10), False),
    (dict(rope_axes=2, rope_dim=0), True),           # nothing is turned
])
def test_paged_plan_axes(cpa, kw, ok):  # noqa: F811
    kw = dict(rope_dim=128) | kw
    if ok:
        make_plan(cpa, **kw)
        return
    with pytest.raises(cpa.CPError) as e:
        make_plan(cpa, **kw)
    assert e.value.code == -1


def test_paged_description_of_version_1(cpa):  # noqa: F811
    """A program compiled against version 1 passes a shorter description, one axis: what lies behind it is not read."""
    d = cpa.cp_paged_desc_t(1, 0, 8, 2, 128, 16, 4, 64, 16, 100, 0, 0, 1, 0, 0.0, 128, 0, 10000.0, None, 99, None)
    h = ctypes.c_void_p()
    assert cpa._L().cp_paged_create(ctypes.byref(d), ctypes.byref(h)) == 0
    cpa._L().cp_paged_destroy(h)
    for version, axes, code in ((2, 99, -1), (2, 0, 0), (3, 1, -1)):
        d.version, d.rope_axes = version, axes
        assert cpa._L().cp_paged_create(ctypes.byref(d), ctypes.byref(h)) == code
        if code == 0:
            cpa._L().cp_paged_destroy(h)


def test_positions_of_a_batch(cpa):  # noqa: F811
    i32 = dict(dtype=torch.int32)
    arrays = (torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 100, **i32))
    batch = lambda pos: cpa.PagedBatch(*arrays, n_tokens=5, positions=pos)  # noqa: E731
    assert batch(None).axes == 0 and batch(torch.zeros(5, **i32)).axes == 1 and batch(torch.zeros(3, 5, **i32)).axes == 3
    for bad in (torch.zeros(5, 3, **i32), torch.zeros(3, 5), torch.zeros(5, 3, **i32).T, torch.zeros(1, 3, 5, **i32)):
        with pytest.raises(cpa.CPError):
            batch(bad)


# ---------------------------------------------------------------- verification

def test_verify_refusals(cpa):  # noqa: F811
    plan, L = make_plan(cpa), cpa._L()

    def call(batch=None, **kw):
        _, b = c_args(cpa, plan, None, batch)
        v = cpa.cp_verify_t(1000, 2, FAKE, 1000, FAKE, 1000, *[FAKE + 4096 * i for i in range(1, 7)])
        for k, x in kw.items():
            setattr(v, k, x)
        return L.cp_verify_drafts(plan.handle, A(b), A(v), None)
    for name in ("p", "tokens", "accept_u", "sample_u", "accepted", "out_tokens"):
        assert call(**{name: None}) == -1, name
    for name in ("tokens", "accept_u", "sample_u", "accepted", "out_tokens", "kv_len_out"):
        assert call(**{name: FAKE + 2}) == -3, name
    assert call(p=FAKE + 2) == -3 and call(q=FAKE + 6) == -3 and call(dtype=0, p=FAKE + 1) == -3 and call(dtype=1, q=FAKE + 3) == -3
    assert call(vocab=0) == -1 and call(vocab=(1 << 30) + 1) == -1 and call(dtype=3) == -1 and call(dtype=-1) == -1
    assert call(p_stride=999) == -1 and call(q_stride=999) == -1 and call(p_stride=1 << 36) == -1
    assert call(batch=dict(n_seqs=5)) == -1 and call(batch=dict(n_tokens=65)) == -1 and call(batch=dict(q_start=None)) == -1
    assert call(out_tokens=FAKE + 4096) == -1 and call(kv_len_out=FAKE + 4096 * 4) == -1 and call(accepted=FAKE + 64) == -1
    assert call(batch=dict(n_seqs=0), p=None) == 0
    assert call(batch=dict(n_tokens=0), accepted=None) == -1 and call(batch=dict(n_tokens=0, q_start=None)) == -1
    assert L.cp_verify_drafts(None, None, None, None) == -1


def test_verify_binding_refusals(cpa):  # noqa: F811
    plan, i32 = make_plan(cpa), dict(dtype=torch.int32)
    batch = cpa.PagedBatch(torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, 100, **i32), n_tokens=5)
    good = dict(tokens=torch.zeros(5, **i32), p=torch.zeros(5, 10), q=torch.zeros(5, 10), accept_u=torch.zeros(5), sample_u=torch.zeros(2),
                accepted=torch.zeros(2, **i32), out_tokens=torch.zeros(5, **i32), kv_len_out=torch.zeros(2, **i32))
    for kw, why in [(dict(tokens=torch.zeros(4, **i32)), "tokens"), (dict(tokens=torch.zeros(5)), "tokens"),
                    (dict(accept_u=torch.zeros(5, dtype=torch.float64)), "accept_u"), (dict(sample_u=torch.zeros(5)), "sample_u"),
                    (dict(accepted=torch.zeros(4, **i32)[::2]), "accepted"), (dict(out_tokens=torch.zeros(2, **i32)), "out_tokens"),
                    (dict(kv_len_out=torch.zeros(3, **i32)), "kv_len_out"), (dict(p=torch.zeros(4, 10)), "vocab"),
                    (dict(p=torch.zeros(5, 9)), "vocab"), (dict(q=torch.zeros(5, 10).half()), "vocab"), (dict(p=torch.zeros(10, 5).T), "vocab"),
                    (dict(p=torch.zeros(5, 10).double(), q=None), "vocab"), (dict(), "not the current")]:
        with pytest.raises(cpa.CPError, match=why):
            cpa.cp_verify_drafts(plan, batch, **{**good, **kw})


# ---------------------------------------------------------------- pages

def structs(cpa, table=None, moves=None):  # noqa: F811
    t = cpa.cp_page_table_t(4, 100, FAKE, FAKE + 4096)
    m = cpa.cp_page_moves_t(50, FAKE, FAKE + 4, FAKE + 1024, FAKE + 2048)
    for s, kw in ((t, table), (m, moves)):
        for k, v in (kw or {}).items():
            setattr(s, k, v)
    return t, m


BAD_TABLES = [(dict(rows=0), -1), (dict(rows=8193), -1), (dict(columns=0), -1), (dict(columns=1 << 26), -1), (dict(pages=None), -1),
              (dict(held=None), -1), (dict(pages=FAKE + 2), -3), (dict(held=FAKE + 1), -3)]
BAD_MOVES = [(dict(capacity=3), -1), (dict(count=None), -1), (dict(src=None), -1), (dict(dst=None), -1), (dict(tokens=None), -1),
             (dict(count=FAKE + 2), -3), (dict(dst=FAKE + 1), -3)]
BAD_REFS = [(0, FAKE, -1), (-5, FAKE, -1), ((1 << 30) + 1, FAKE, -1), (100, None, -1), (100, FAKE + 4, -3)]


def test_resize_refusals(cpa):  # noqa: F811
    plan, L = make_plan(cpa), cpa._L()
    call = lambda t, n=100, refs=FAKE, tokens=FAKE + 64, served=FAKE + 128: L.cp_pages_resize(plan.handle, n, refs, A(t), tokens, served, None)  # noqa: E731
    for kw, code in BAD_TABLES:
        assert call(structs(cpa, kw)[0]) == code, kw
    t, _ = structs(cpa)
    for n, refs, code in BAD_REFS:
        assert call(t, n, refs) == code
    assert call(t, tokens=None) == -1 and call(t, served=None) == -1 and call(t, tokens=FAKE + 2) == -3
    assert call(t, served=FAKE + 64) == -1 and call(t, tokens=FAKE + 4096) == -1 and call(t, served=FAKE + 4096) == -1
    assert L.cp_pages_resize(None, 100, FAKE, A(t), FAKE, FAKE, None) == -1
    assert L.cp_pages_resize(plan.handle, 100, FAKE, None, FAKE, FAKE, None) == -1


def test_fork_refusals(cpa):  # noqa: F811
    plan, L = make_plan(cpa), cpa._L()

    def call(src=None, dst=None, moves=None, n=100, refs=FAKE, parent=FAKE + 64, tokens=FAKE + 128, served=FAKE + 192):
        (s, m), (d, _) = structs(cpa, src, moves), structs(cpa, dst)
        return L.cp_pages_fork(plan.handle, n, refs, A(s), A(d), parent, tokens, A(m), served, None)
    for kw, code in BAD_TABLES:
        assert call(src=kw) == code and call(dst=kw) == code, kw
    for kw, code in BAD_MOVES:
        assert call(moves=kw) == code, kw
    for n, refs, code in BAD_REFS:
        assert call(n=n, refs=refs) == code
    assert call(parent=None) == -1 and call(tokens=None) == -1 and call(served=None) == -1 and call(parent=FAKE + 1) == -3
    assert call(served=FAKE + 64) == -1 and call(served=FAKE + 128) == -1 and call(served=FAKE + 4096) == -1 and call(parent=FAKE + 4096) == -1


def test_compact_refusals(cpa):  # noqa: F811
    plan, L = make_plan(cpa), cpa._L()
    ws = cpa.cp_pages_workspace_size(100)
    assert ws == 16 + 400

    def call(table=None, out=None, moves=None, n=100, refs=FAKE, refs_out=FAKE, tables=1, used=FAKE, w=FAKE, wn=ws):
        (t, m), (o, _) = structs(cpa, table, moves), structs(cpa, out)
        return L.cp_pages_compact(plan.handle, n, refs, refs_out, tables, A(t), A(o), A(m), used, w, wn, None)
    for kw, code in BAD_TABLES:
        assert call(table=kw) == code, kw
    for kw, code in BAD_MOVES:
        assert call(moves=kw) == code, kw
    assert call(moves=dict(capacity=49)) == -1
    for n, refs, code in BAD_REFS:
        assert call(n=n, refs=refs) == code and call(n=n, refs_out=refs) == code
    assert call(tables=0) == -1 and call(tables=5) == -1 and call(used=FAKE + 2) == -3
    assert call(out=dict(rows=3)) == -1 and call(out=dict(columns=99)) == -1 and call(out=dict(pages=None)) == -1
    assert call(w=None) == cpa.CP_ERR_WORKSPACE and call(wn=ws - 1) == cpa.CP_ERR_WORKSPACE and call(w=FAKE + 8) == -3
    for n in (0, -1, (1 << 30) + 1):
        with pytest.raises(cpa.CPError):
            cpa.cp_pages_workspace_size(n)


def test_copy_refusals(cpa):  # noqa: F811
    plan, L = make_plan(cpa), cpa._L()

    def call(src=None, dst=None, moves=None, n=2, second=None):
        _, m = structs(cpa, None, moves)
        arrays = []
        for kw in (src, dst):
            c, _ = c_args(cpa, plan, kw)
            e, _ = c_args(cpa, plan, (kw or {}) | (second or {}))
            arrays.append((cpa.cp_paged_cache_t * 2)(c, e))
        return L.cp_pages_copy(plan.handle, n, arrays[0], arrays[1], A(m), None)
    for kw, code in [(dict(k=None), -1), (dict(v=FAKE + 8), -3), (dict(num_pages=0), -1), (dict(token_stride=252), -1),
                     (dict(page_stride=4088), -1)]:
        assert call(src=kw) == code and call(dst=kw) == code, kw
    for kw in (dict(num_pages=51), dict(page_stride=8192)):  # layers that are not alike
        assert call(second=kw) == -1
    for kw, code in BAD_MOVES[1:]:
        assert call(moves=kw) == code, kw
    assert call(moves=dict(capacity=-1)) == -1 and call(n=0) == -1 and call(n=129) == -1


def test_pages_binding_refusals(cpa):  # noqa: F811
    i32 = dict(dtype=torch.int32)
    z = lambda *s: torch.zeros(*s, **i32)  # noqa: E731
    for bad in ((z(4), z(4)), (z(4, 5), z(5)), (z(4, 5).long(), z(4)), (z(5, 4).T, z(4)), (z(4, 5), z(8)[::2])):
        with pytest.raises(cpa.CPError):
            cpa.PageTable(*bad)
    for kw in (dict(), dict(capacity=-1), dict(src=z(3)), dict(src=z(3), dst=z(3), tokens=z(4)), dict(capacity=4, src=z(3), dst=z(3), tokens=z(3)),
               dict(src=z(3), dst=z(3), tokens=z(3), count=z(2)), dict(capacity=3, count=z(1))):
        with pytest.raises(cpa.CPError):
            cpa.PageMoves(device="cpu", **kw)
    m = cpa.PageMoves(src=z(3), dst=z(3), tokens=z(3))
    assert m.capacity == 3 and m.count.tolist() == [3]
    plan, t, moves, refs = make_plan(cpa), cpa.PageTable(z(4, 5), z(4)), cpa.PageMoves(50, device="cpu"), z(100)
    ws = torch.zeros(416, dtype=torch.uint8)
    k = torch.zeros(10, 16, 2, 128, dtype=torch.bfloat16)
    c, other = cpa.PagedCache(k, k.clone()), cpa.PagedCache(k.half(), k.half())
    for f, args, why in [
            (cpa.cp_pages_resize, (plan, refs, t, z(3), z(4)), "tokens"), (cpa.cp_pages_resize, (plan, refs.long(), t, z(4), z(4)), "refs"),
            (cpa.cp_pages_resize, (plan, z(5, 20), t, z(4), z(4)), "refs"), (cpa.cp_pages_resize, (plan, refs, t, z(4), z(4)), "not the current"),
            (cpa.cp_pages_fork, (plan, refs, t, t, z(5), z(4), moves, z(4)), "parent"),
            (cpa.cp_pages_fork, (plan, refs, t, t, z(4), z(4), moves, z(4)), "not the current"),
            (cpa.cp_pages_compact, (plan, refs, [], moves, ws), "1 to 4"), (cpa.cp_pages_compact, (plan, refs, [t] * 5, moves, ws), "1 to 4"),
            (cpa.cp_pages_compact, (plan, refs, [t], moves, ws, z(99)), "refs_out"),
            (cpa.cp_pages_compact, (plan, refs, [t], moves, ws, None, [cpa.PageTable(z(4, 6), z(4))]), "alike"),
            (cpa.cp_pages_compact, (plan, refs, [t], moves, ws, None, None, z(2)), "used"),
            (cpa.cp_pages_compact, (plan, refs, [t], moves, ws), "not the current"),
            (cpa.cp_pages_copy, (plan, [], [], moves), "1 to 128"), (cpa.cp_pages_copy, (plan, [c], [c, c], moves), "1 to 128"),
            (cpa.cp_pages_copy, (plan, [c], [other], moves), "pages are"), (cpa.cp_pages_copy, (plan, [c], [c], moves), "not the current")]:
        with pytest.raises(cpa.CPError, match=why):
            f(*args)
