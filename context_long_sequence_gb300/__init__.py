"""Python binding of libcpattn (include/cp_attn.h): argument marshalling only.

Every function here forwards to the C ABI of the same name; all computation
runs in the library's CUDA kernels.  PyTorch is used only to own device
memory and to name the current stream.  Using this module fails loudly if
the library has not been built (``python -m context_long_sequence_gb300.build``):
the first call raises; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
# CPATTN_DEBUG=1 in the environment selects the bounds-checked debug build
# (libcpattn_debug.so, compiled with -DCP_DEBUG) for this process.
DEBUG = os.environ.get("CPATTN_DEBUG", "") not in ("", "0")
LIB_PATH = os.path.join(_HERE, "libcpattn_debug.so" if DEBUG else "libcpattn.so")

# Constants (mirrors include/cp_attn.h).
CP_ATTN_PLAN_VERSION = 1
CP_OK = 0
CP_ERR_INVALID_ARG = -1
CP_ERR_UNSUPPORTED = -2
CP_ERR_ALIGNMENT = -3
CP_ERR_CUDA = -4
CP_ERR_DEVICE_TIMEOUT = -5
CP_ERR_DEVICE_BOUNDS = -6
CP_ERR_WORKSPACE = -7
CP_ERR_ARCH = -8
CP_NOALLOC_SCRATCH_BYTES = 8 << 20
CP_LAYOUT_CONTIGUOUS = 0
CP_LAYOUT_ZIGZAG = 1
CP_LAYOUT_BALANCED = 2
CP_KV_RING = 0
CP_KV_ALLGATHER = 1
CP_SEQ_TO_HEAD = 0
CP_HEAD_TO_SEQ = 1
CP_TOKEN_MAJOR = 0
CP_HEAD_MAJOR = 1
CP_OP_FWD = 0
CP_OP_BWD = 1
CP_OP_BWD_RANK_STATS = 2


CP_RESHARD_MAX_JOBS = 8
CP_PAGED_VERSION = 1
CP_DTYPE_BF16 = 0
CP_DTYPE_FP16 = 1


class cp_reshard_job_t(ctypes.Structure):
    _fields_ = [
        ("direction", ctypes.c_int32),
        ("tensor_kind", ctypes.c_int32),
        ("H", ctypes.c_int32),
        ("row_elems", ctypes.c_int32),
        ("elem_bytes", ctypes.c_int32),
        ("inp", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
    ]


class cp_plan_desc_t(ctypes.Structure):
    _fields_ = [
        ("version", ctypes.c_int32),
        ("L", ctypes.c_int32),
        ("Hq", ctypes.c_int32),
        ("Hkv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("ulysses_degree", ctypes.c_int32),
        ("ring_degree", ctypes.c_int32),
        ("layout", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("num_docs", ctypes.c_int32),
        ("doc_offsets", ctypes.POINTER(ctypes.c_int32)),
        ("softmax_scale", ctypes.c_float),
        ("emit_partials", ctypes.c_int32),
        ("out_fp32", ctypes.c_int32),
        ("chunks_per_rank", ctypes.c_int32),
        ("kv_exchange", ctypes.c_int32),
    ]


class cp_paged_desc_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "version", "dtype", "Hq", "Hkv", "d", "page_size", "max_seqs", "max_tokens", "max_new", "max_pages",
        "max_prefixes", "max_prefix_pages", "causal", "out_fp32")] + [
        ("softmax_scale", ctypes.c_float),
        ("rope_dim", ctypes.c_int32),
        ("rope_interleaved", ctypes.c_int32),
        ("rope_base", ctypes.c_double),
        ("rope_freqs", ctypes.POINTER(ctypes.c_double)),
    ]


class cp_paged_cache_t(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("num_pages", ctypes.c_int32),
        ("page_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
    ]


class cp_paged_batch_t(ctypes.Structure):
    _fields_ = [
        ("n_seqs", ctypes.c_int32),
        ("n_tokens", ctypes.c_int32),
        ("q_start", ctypes.c_void_p),
        ("kv_len", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
        ("n_prefixes", ctypes.c_int32),
        ("prefix_first", ctypes.c_void_p),
        ("prefix_len", ctypes.c_void_p),
        ("prefix_table", ctypes.c_void_p),
        ("positions", ctypes.c_void_p),
    ]


_vp = ctypes.c_void_p
_i = ctypes.c_int
_lib = None


def _L():
    """The loaded library; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{os.path.basename(LIB_PATH)} is not built ({LIB_PATH}); run "
                           "`python -m context_long_sequence_gb300.build` first")
    lib = ctypes.CDLL(LIB_PATH)
    lib.cp_plan_create.argtypes = [ctypes.POINTER(cp_plan_desc_t), ctypes.POINTER(_vp)]
    lib.cp_plan_destroy.argtypes = [_vp]
    lib.cp_plan_destroy.restype = None
    lib.cp_index_map.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32)]
    lib.cp_workspace_size.argtypes = [_vp, _i, ctypes.POINTER(ctypes.c_size_t)]
    lib.ulysses_reshard.argtypes = [_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp]
    lib.ulysses_reshard_batch.argtypes = [_vp, _i, ctypes.POINTER(cp_reshard_job_t), _vp]
    lib.cp_attn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.cp_attn_fwd_local.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.cp_attn_fwd_rank.argtypes = [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.cp_attn_fwd_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.cp_attn_bwd.argtypes = [_vp] + [_vp] * 9 + [_vp, ctypes.c_size_t, _vp]
    lib.cp_attn_fwd_step.argtypes = [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.cp_attn_bwd_delta.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp]
    lib.cp_attn_bwd_step.argtypes = [_vp, _i, _i] + [_vp] * 8 + [_vp]
    lib.cp_merge_lse.argtypes = [_i, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]
    lib.cp_get_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32)]
    lib.cp_selftest_wait_timeout.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), _vp]
    lib.cp_selftest_bounds.argtypes = [ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), _vp]
    lib.cp_get_status_detail.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32)]
    lib.cp_tile_classes.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32), ctypes.c_int64,
                                    ctypes.POINTER(ctypes.c_int64), _vp]
    lib.cp_paged_create.argtypes = [ctypes.POINTER(cp_paged_desc_t), ctypes.POINTER(_vp)]
    lib.cp_paged_destroy.argtypes = [_vp]
    lib.cp_paged_destroy.restype = None
    lib.cp_paged_workspace_size.argtypes = [_vp, ctypes.POINTER(ctypes.c_size_t)]
    lib.cp_paged_shares.argtypes = [_vp, _vp, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32), ctypes.c_int64,
                                    ctypes.POINTER(ctypes.c_int64)]
    lib.cp_cache_append.argtypes = [_vp, _vp, _vp] + [_vp, ctypes.c_int64] * 4 + [_vp]
    lib.cp_attn_paged.argtypes = [_vp, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp, _vp, ctypes.c_size_t, _vp]
    lib.cp_debug_build.argtypes = []
    lib.cp_measure_rates.argtypes = [ctypes.POINTER(ctypes.c_double), _vp]
    lib.cp_measure_barrier_check.argtypes = [ctypes.POINTER(ctypes.c_double), _vp]
    lib.cp_strerror.argtypes = [_i]
    lib.cp_strerror.restype = ctypes.c_char_p
    _lib = lib
    return lib


EXPORTED = ["cp_plan_create", "cp_plan_destroy", "cp_index_map", "cp_workspace_size", "ulysses_reshard",
            "ulysses_reshard_batch",
            "cp_attn_fwd", "cp_attn_fwd_local", "cp_attn_fwd_rank", "cp_attn_fwd_noalloc", "cp_attn_bwd",
            "cp_attn_fwd_step", "cp_attn_bwd_delta", "cp_attn_bwd_step",
            "cp_paged_create", "cp_paged_destroy", "cp_paged_workspace_size", "cp_paged_shares", "cp_cache_append", "cp_attn_paged",
            "cp_merge_lse", "cp_get_status", "cp_get_status_detail", "cp_debug_build", "cp_strerror",
            "cp_selftest_wait_timeout", "cp_selftest_bounds", "cp_tile_classes", "cp_measure_rates", "cp_measure_barrier_check"]


class CPError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {cp_strerror(code)} ({code})")


def cp_strerror(code: int) -> str:
    return _L().cp_strerror(int(code)).decode()


def _check(rc: int, where: str):
    if rc != CP_OK:
        raise CPError(rc, where)


def _ptr(x):
    """Device address of a tensor (or an int address); None -> NULL."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        # The address alone: a torch.cuda.Stream object takes 3 us to make.
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class Plan:
    """Owns a cp_plan_t (cp_plan_create / cp_plan_destroy)."""

    def __init__(self, L, Hq, Hkv, d, ulysses_degree=1, ring_degree=1, layout=CP_LAYOUT_CONTIGUOUS,
                 doc_offsets=None, softmax_scale=0.0, emit_partials=False, causal=True, out_fp32=False,
                 chunks_per_rank=8, kv_exchange=CP_KV_RING):
        self._h = None
        desc = cp_plan_desc_t()
        desc.version = CP_ATTN_PLAN_VERSION
        desc.L, desc.Hq, desc.Hkv, desc.d = int(L), int(Hq), int(Hkv), int(d)
        desc.ulysses_degree, desc.ring_degree = int(ulysses_degree), int(ring_degree)
        desc.layout = int(layout)
        desc.causal = 1 if causal else 0
        self._offsets = None
        if doc_offsets is not None and len(doc_offsets) > 2:
            self._offsets = (ctypes.c_int32 * len(doc_offsets))(*[int(x) for x in doc_offsets])
            desc.num_docs = len(doc_offsets) - 1
            desc.doc_offsets = ctypes.cast(self._offsets, ctypes.POINTER(ctypes.c_int32))
        else:
            desc.num_docs = 0
            desc.doc_offsets = None
        desc.softmax_scale = float(softmax_scale)
        desc.emit_partials = 1 if emit_partials else 0
        desc.out_fp32 = 1 if out_fp32 else 0
        desc.chunks_per_rank = int(chunks_per_rank)
        desc.kv_exchange = int(kv_exchange)
        h = _vp()
        _check(_L().cp_plan_create(ctypes.byref(desc), ctypes.byref(h)), "cp_plan_create")
        self._h = h
        self.L, self.Hq, self.Hkv, self.d = desc.L, desc.Hq, desc.Hkv, desc.d
        self.U, self.R = desc.ulysses_degree, desc.ring_degree
        self.P = self.U * self.R
        self.n = self.L // self.P
        self.layout = desc.layout
        self.chunks_per_rank = desc.chunks_per_rank
        self.kv_exchange = desc.kv_exchange
        self.emit_partials = bool(emit_partials)
        self.out_fp32 = bool(out_fp32)

    @property
    def o_dtype(self):
        import torch
        return torch.float32 if self.out_fp32 else torch.bfloat16

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h is not None:
            _L().cp_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def index_map(self) -> np.ndarray:
        out = np.empty(self.L, dtype=np.int32)
        _check(_L().cp_index_map(self._h, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))), "cp_index_map")
        return out

    def workspace_size(self, op=CP_OP_FWD) -> int:
        n = ctypes.c_size_t()
        _check(_L().cp_workspace_size(self._h, int(op), ctypes.byref(n)), "cp_workspace_size")
        return n.value


def ulysses_reshard(plan: Plan, direction, tensor_kind, H, row_elems, elem_bytes, inp, out, stream=None):
    _check(_L().ulysses_reshard(plan.handle, int(direction), int(tensor_kind), int(H), int(row_elems),
                                int(elem_bytes), _ptr(inp), _ptr(out), _stream(stream)), "ulysses_reshard")


def ulysses_reshard_batch(plan: Plan, jobs, stream=None):
    """jobs: sequence of (direction, tensor_kind, H, row_elems, elem_bytes, inp, out)."""
    arr = (cp_reshard_job_t * max(1, len(jobs)))()
    for i, (direction, kind, H, row_elems, elem_bytes, inp, out) in enumerate(jobs):
        arr[i] = cp_reshard_job_t(int(direction), int(kind), int(H), int(row_elems), int(elem_bytes),
                                  _ptr(inp), _ptr(out))
    _check(_L().ulysses_reshard_batch(plan.handle, len(jobs), arr, _stream(stream)), "ulysses_reshard_batch")


def cp_attn_fwd(plan: Plan, q, k, v, o, lse, workspace=None, workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_L().cp_attn_fwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(workspace),
                            int(workspace_bytes), _stream(stream)), "cp_attn_fwd")


def cp_attn_fwd_rank(plan: Plan, rank, q, k, v, o, lse, stream=None):
    _check(_L().cp_attn_fwd_rank(plan.handle, int(rank), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                 _stream(stream)), "cp_attn_fwd_rank")


def cp_attn_fwd_local(plan: Plan, q, k, v, o, lse, stream=None):
    _check(_L().cp_attn_fwd_local(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _stream(stream)),
           "cp_attn_fwd_local")


def cp_attn_fwd_noalloc(plan: Plan, q, k, v, o, lse, stream=None):
    """cp_attn_fwd for an emit-partials plan, with the partials kept in the
    library's static device scratch instead of an allocated workspace."""
    _check(_L().cp_attn_fwd_noalloc(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _stream(stream)),
           "cp_attn_fwd_noalloc")


def cp_attn_bwd(plan: Plan, q, k, v, o, lse, dO, dq, dk, dv, workspace=None, workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_L().cp_attn_bwd(plan.handle, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(dO), _ptr(dq),
                            _ptr(dk), _ptr(dv), _ptr(workspace), int(workspace_bytes), _stream(stream)),
           "cp_attn_bwd")


def cp_attn_fwd_step(plan: Plan, rank, step, q_rank, k_chunk, v_chunk, o_part, lse_part, stream=None):
    _check(_L().cp_attn_fwd_step(plan.handle, int(rank), int(step), _ptr(q_rank), _ptr(k_chunk), _ptr(v_chunk),
                                 _ptr(o_part), _ptr(lse_part), _stream(stream)), "cp_attn_fwd_step")


def cp_attn_bwd_delta(plan: Plan, o_rank, do_rank, lse_rank, stats_rank, stream=None):
    _check(_L().cp_attn_bwd_delta(plan.handle, _ptr(o_rank), _ptr(do_rank), _ptr(lse_rank), _ptr(stats_rank),
                                  _stream(stream)), "cp_attn_bwd_delta")


def cp_attn_bwd_step(plan: Plan, rank, step, q_rank, do_rank, stats_rank, k_chunk, v_chunk, dq_rank, dk_chunk,
                     dv_chunk, stream=None):
    _check(_L().cp_attn_bwd_step(plan.handle, int(rank), int(step), _ptr(q_rank), _ptr(do_rank), _ptr(stats_rank),
                                 _ptr(k_chunk), _ptr(v_chunk), _ptr(dq_rank), _ptr(dk_chunk), _ptr(dv_chunk),
                                 _stream(stream)), "cp_attn_bwd_step")


def cp_merge_lse(n_parts, rows, H, d, o_parts, lse_parts, o_out, lse_out, stream=None):
    _check(_L().cp_merge_lse(int(n_parts), int(rows), int(H), int(d), _ptr(o_parts), _ptr(lse_parts),
                             _ptr(o_out), _ptr(lse_out), _stream(stream)), "cp_merge_lse")


def cp_selftest_wait_timeout(limit_us, stream=None):
    """Run the bounded-wait self-test; returns (timed_out, left_on_abort, wait_us)."""
    out = (ctypes.c_int32 * 3)()
    _check(_L().cp_selftest_wait_timeout(int(limit_us), out, _stream(stream)), "cp_selftest_wait_timeout")
    return int(out[0]), int(out[1]), int(out[2])


def cp_tile_classes(plan, stream=None) -> np.ndarray:
    """The forward's tile-class table of `plan`: int32 [n][8] rows
    {a, q0, len, step, kpos0, klen, class0, class1} (see include/cp_attn.h)."""
    n = ctypes.c_int64()
    _check(_L().cp_tile_classes(plan.handle, None, 0, ctypes.byref(n), _stream(stream)), "cp_tile_classes")
    out = np.zeros((max(n.value, 1), 8), dtype=np.int32)
    _check(_L().cp_tile_classes(plan.handle, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)), n.value,
                                ctypes.byref(n), _stream(stream)), "cp_tile_classes")
    return out[:n.value]


def cp_selftest_bounds(block, stream=None) -> int:
    """Run the bounds-record self-test in block `block`; returns the source
    line the kernel recorded (read the record with cp_get_status_detail)."""
    line = ctypes.c_int32()
    _check(_L().cp_selftest_bounds(int(block), ctypes.byref(line), _stream(stream)), "cp_selftest_bounds")
    return line.value


def cp_get_status_detail(stream=None):
    """Read and clear the device status record: (code, block, line, file id)."""
    out = (ctypes.c_int32 * 4)()
    _check(_L().cp_get_status_detail(_stream(stream), out), "cp_get_status_detail")
    return tuple(int(x) for x in out)


def cp_measure_rates(stream=None):
    """(ex2 results per SM clock, SM clocks per M128 N128 K16 bf16 MMA)."""
    out = (ctypes.c_double * 2)()
    _check(_L().cp_measure_rates(out, _stream(stream)), "cp_measure_rates")
    return float(out[0]), float(out[1])


def cp_measure_barrier_check(stream=None) -> float:
    """SM clocks per warp-wide check of a completed mbarrier phase."""
    out = ctypes.c_double(0.0)
    _check(_L().cp_measure_barrier_check(ctypes.byref(out), _stream(stream)), "cp_measure_barrier_check")
    return float(out.value)


def cp_debug_build() -> bool:
    """True when the loaded library is the -DCP_DEBUG build."""
    return bool(_L().cp_debug_build())


def cp_get_status(stream=None) -> int:
    code = ctypes.c_int32()
    _check(_L().cp_get_status(_stream(stream), ctypes.byref(code)), "cp_get_status")
    return code.value


def alloc_workspace(plan: Plan, op=CP_OP_FWD, device="cuda"):
    """A device byte buffer of cp_workspace_size() bytes (None when zero)."""
    import torch
    n = plan.workspace_size(op)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _refuse(where: str, why: str):
    e = CPError(CP_ERR_INVALID_ARG, where)
    e.args = (f"{e.args[0]}: {why}",)
    raise e


class PagedPlan:
    """Owns a cp_paged_t (cp_paged_create / cp_paged_destroy): the shapes and
    bounds of serving steps over a paged cache.  The kernels go by the bounds:
    a plan for decode steps beside one for prompts is faster than one for
    both.  ``dtype`` is torch.bfloat16 or torch.float16; ``rope_freqs`` (rope_dim/2 numbers) replaces
    ``rope_base``."""

    def __init__(self, Hq, Hkv, d, page_size, dtype, max_seqs, max_tokens, max_new, max_pages, max_prefixes=0,
                 max_prefix_pages=0, causal=True, out_fp32=False, softmax_scale=0.0, rope_dim=0, rope_interleaved=False,
                 rope_base=10000.0, rope_freqs=None):
        import torch
        self._h = None
        codes = {torch.bfloat16: CP_DTYPE_BF16, torch.float16: CP_DTYPE_FP16}
        if dtype not in codes:
            _refuse("cp_paged_create", f"dtype {dtype} is neither bfloat16 nor float16")
        desc = cp_paged_desc_t(CP_PAGED_VERSION, codes[dtype], int(Hq), int(Hkv), int(d), int(page_size), int(max_seqs),
                               int(max_tokens), int(max_new), int(max_pages), int(max_prefixes), int(max_prefix_pages),
                               1 if causal else 0, 1 if out_fp32 else 0, float(softmax_scale), int(rope_dim),
                               1 if rope_interleaved else 0, float(rope_base), None)
        if rope_freqs is not None:
            if len(rope_freqs) != int(rope_dim) // 2:
                _refuse("cp_paged_create", f"{len(rope_freqs)} rope_freqs for rope_dim {rope_dim}")
            freqs = (ctypes.c_double * max(1, len(rope_freqs)))(*[float(x) for x in rope_freqs])
            desc.rope_freqs = ctypes.cast(freqs, ctypes.POINTER(ctypes.c_double))
        h = _vp()
        _check(_L().cp_paged_create(ctypes.byref(desc), ctypes.byref(h)), "cp_paged_create")
        self._h = h
        self.Hq, self.Hkv, self.d, self.page_size, self.dtype = desc.Hq, desc.Hkv, desc.d, desc.page_size, dtype
        self.max_seqs, self.max_tokens, self.max_new = desc.max_seqs, desc.max_tokens, desc.max_new
        self.max_pages, self.max_prefixes, self.max_prefix_pages = desc.max_pages, desc.max_prefixes, desc.max_prefix_pages
        self.out_fp32 = bool(out_fp32)
        self.lse_dtype = torch.float32
        self.o_dtype = torch.float32 if out_fp32 else dtype
        self.page = (desc.page_size, desc.Hkv, desc.d, dtype)
        # A decode step's calls take the host about as long as the GPU: torch's
        # functions that they need are looked up once (a torch without CUDA has
        # none; its tensors are refused before they would be called).
        self._current = tuple(getattr(torch._C, name, None) for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h is not None:
            _L().cp_paged_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def workspace_size(self) -> int:
        n = ctypes.c_size_t()
        _check(_L().cp_paged_workspace_size(self._h, ctypes.byref(n)), "cp_paged_workspace_size")
        return n.value


class PagedCache:
    """The cache's tensors, as cp_paged_cache_t: ``k`` and ``v`` are
    [pages][page_size][Hkv][d] views of equal strides (a cache stored
    [pages][Hkv][page_size][d] is passed transposed)."""

    def __init__(self, k, v):
        strides = []
        for x in (k, v):  # the stride of a dimension of one element says nothing
            strides.append([st if n > 1 else x.shape[-1] for n, st in zip(x.shape, x.stride())] if x.dim() == 4 else None)
        if k.dim() != 4 or k.shape != v.shape or strides[0] != strides[1] or k.dtype != v.dtype or k.device != v.device \
                or k.stride(3) != 1:
            _refuse("PagedCache", "k and v are [pages][page_size][Hkv][d] tensors alike, the last dimension contiguous")
        self.k, self.v, self.device, self._dev = k, v, k.device, k.get_device()
        self.page = (k.shape[1], k.shape[2], k.shape[3], k.dtype)
        self.c = cp_paged_cache_t(k.data_ptr(), v.data_ptr(), k.shape[0], *strides[0][:3])
        self.ref = ctypes.addressof(self.c)


class PagedBatch:
    """A step's batch, as cp_paged_batch_t: int32 tensors on the cache's
    device, kept alive here and read by the kernels when they run."""

    def __init__(self, q_start, kv_len, page_table, n_tokens, prefix_first=None, prefix_len=None, prefix_table=None,
                 positions=None):
        import torch
        self.n_seqs, self.n_tokens = kv_len.shape[0], int(n_tokens)
        self.n_prefixes = 0 if prefix_len is None else prefix_len.shape[0]
        self.device, self._dev = q_start.device, q_start.get_device()
        self.max_pages = page_table.shape[1] if page_table.dim() == 2 else -1
        self.max_prefix_pages = prefix_table.shape[1] if prefix_table is not None and prefix_table.dim() == 2 else 0
        want = [(q_start, (self.n_seqs + 1,)), (kv_len, (self.n_seqs,)), (page_table, (self.n_seqs, self.max_pages)),
                (positions, (self.n_tokens,))]
        given = [x is not None for x in (prefix_first, prefix_len, prefix_table)]
        if any(given) and not all(given):
            _refuse("PagedBatch", "prefix_first, prefix_len and prefix_table come together")
        want += [(prefix_first, (self.n_prefixes + 1,)), (prefix_len, (self.n_prefixes,)),
                 (prefix_table, (self.n_prefixes, self.max_prefix_pages))]
        for x, shape in want:
            if x is not None and (x.dtype != torch.int32 or tuple(x.shape) != shape or not x.is_contiguous()
                                  or x.device != self.device):
                _refuse("PagedBatch", f"a contiguous int32 tensor of shape {shape} on {self.device} is wanted, got "
                                      f"{x.dtype} {tuple(x.shape)} on {x.device}")
        self._keep = (q_start, kv_len, page_table, prefix_first, prefix_len, prefix_table, positions)
        self.c = cp_paged_batch_t(self.n_seqs, self.n_tokens, _ptr(q_start), _ptr(kv_len), _ptr(page_table),
                                  self.n_prefixes, _ptr(prefix_first), _ptr(prefix_len), _ptr(prefix_table),
                                  _ptr(positions))
        self.ref = ctypes.addressof(self.c)


def _paged_stream(where, plan, cache, batch, stream):
    """The checks that need the tensors' shapes, types and devices (the
    library sees addresses); the stream the call goes to."""
    dev, (current, raw_stream) = cache._dev, plan._current
    if cache.page == plan.page and batch.max_pages == plan.max_pages and batch._dev == dev and dev >= 0 and current() == dev \
            and (not batch.n_prefixes or batch.max_prefix_pages == plan.max_prefix_pages):
        return raw_stream(dev) if stream is None else _stream(stream)
    if cache.page != plan.page:
        _refuse(where, f"the cache's pages are {cache.page}, the plan's {plan.page}")
    if batch.max_pages != plan.max_pages or (batch.n_prefixes and batch.max_prefix_pages != plan.max_prefix_pages):
        _refuse(where, "the page tables' columns differ from the plan's")
    if batch._dev != dev:
        _refuse(where, f"the batch is on {batch.device}, the cache on {cache.device}")
    _refuse(where, f"the tensors are on {cache.device}, which is not the current device")


def _tokens(where, name, x, n, heads, plan, dev):
    """Address and token stride of a [n_tokens][heads][d] tensor on device
    number `dev`."""
    s, d = x.stride(), plan.d
    if x.shape == (n, heads, d) and x.dtype is plan.dtype and s[2] == 1 and (s[1] == d or heads == 1) and x.get_device() == dev:
        return x.data_ptr(), s[0] if n > 1 else heads * d
    _refuse(where, f"{name} is [{n}][{heads}][{d}] {plan.dtype} with contiguous heads on cuda:{dev}, got "
                   f"{x.dtype} {tuple(x.shape)} with strides {s} on {x.device}")


def cp_cache_append(plan: PagedPlan, cache: PagedCache, batch: PagedBatch, q, k, v, q_out=None, stream=None):
    where = "cp_cache_append"
    st = _paged_stream(where, plan, cache, batch, stream)
    n, dev = batch.n_tokens, cache._dev
    qa = oa = (None, 0)
    if q is not None:
        if q_out is None:
            _refuse(where, "q needs q_out")
        qa = _tokens(where, "q", q, n, plan.Hq, plan, dev)
        oa = _tokens(where, "q_out", q_out, n, plan.Hq, plan, dev)
    ka = _tokens(where, "k", k, n, plan.Hkv, plan, dev)
    va = _tokens(where, "v", v, n, plan.Hkv, plan, dev)
    rc = _L().cp_cache_append(plan._h, cache.ref, batch.ref, *qa, *ka, *va, *oa, st)
    if rc != CP_OK:
        _check(rc, where)


def cp_attn_paged(plan: PagedPlan, cache: PagedCache, batch: PagedBatch, q, o, lse, workspace=None, stream=None):
    where = "cp_attn_paged"
    st = _paged_stream(where, plan, cache, batch, stream)
    n, dev = batch.n_tokens, cache._dev
    qa = _tokens(where, "q", q, n, plan.Hq, plan, dev)
    if o.shape != (n, plan.Hq, plan.d) or o.dtype != plan.o_dtype or not o.is_contiguous() or o.get_device() != dev:
        _refuse(where, f"o is a contiguous [{n}][{plan.Hq}][{plan.d}] {plan.o_dtype} on cuda:{dev}")
    if lse.shape != (plan.Hq, n) or lse.dtype is not plan.lse_dtype or not lse.is_contiguous() or lse.get_device() != dev:
        _refuse(where, f"lse is a contiguous [{plan.Hq}][{n}] float32 on cuda:{dev}")
    wa = wn = 0
    if workspace is not None:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            _refuse(where, f"the workspace is a contiguous tensor on cuda:{dev}")
        wa, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    rc = _L().cp_attn_paged(plan._h, cache.ref, batch.ref, *qa, o.data_ptr(), lse.data_ptr(), wa, wn, st)
    if rc != CP_OK:
        _check(rc, where)


def cp_paged_shares(plan: PagedPlan, batch: PagedBatch, ctas=152) -> np.ndarray:
    """How cp_attn_paged shares out `batch` (whose tensors are on the CPU here):
    int32 [n][14] rows {large, worker, entry, KV head, first token, tokens,
    first key, end key, mode, row, parts, first part row, second part row, row
    stride} (see include/cp_attn.h)."""
    if batch.device.type != "cpu" or batch.max_pages != plan.max_pages \
            or (batch.n_prefixes and batch.max_prefix_pages != plan.max_prefix_pages):
        _refuse("cp_paged_shares", "a batch on the CPU with the plan's page tables is wanted")
    n = ctypes.c_int64()
    _check(_L().cp_paged_shares(plan._h, batch.ref, int(ctas), None, 0, ctypes.byref(n)), "cp_paged_shares")
    out = np.zeros((max(n.value, 1), 14), dtype=np.int32)
    _check(_L().cp_paged_shares(plan._h, batch.ref, int(ctas), out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                n.value, ctypes.byref(n)), "cp_paged_shares")
    return out[:n.value]


def alloc_paged_workspace(plan: PagedPlan, device="cuda"):
    """A device byte buffer of cp_paged_workspace_size() bytes (None when zero)."""
    import torch
    n = plan.workspace_size()
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None
