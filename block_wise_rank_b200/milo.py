"""Thin ctypes binding of libmilo (include/milo.h), same names as the C ABI.

Argument marshalling only: every step of the path runs in libmilo's CUDA
kernels.  Tensors are passed as raw device (or host) pointers; PyTorch is
used for device memory and streams.  There is no fallback: if libmilo.so is
missing or fails to load, every call raises.

A call with `stream` runs as if it were made under torch.cuda.stream(stream): what it
makes itself (outputs, workspaces) is that stream's memory.  Its inputs have to be
ready on that stream, and another stream that reads its outputs waits for it first.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmilo.so")

MILO_OK = 0
MILO_WARN_NOT_CONVERGED = 1
MILO_ERR_INVALID_ARG = -1
MILO_ERR_UNSUPPORTED = -2
MILO_ERR_CUDA = -3
MILO_ERR_WORKSPACE = -4
MILO_ERR_NONFINITE = -5
MILO_ERR_BOUNDS = -6
MILO_ERR_TIMEOUT = -7

MILO_F32, MILO_BF16, MILO_INT8, MILO_INT2, MILO_INT4, MILO_FP8 = 0, 1, 2, 3, 4, 5
DTYPES = {"f32": MILO_F32, "bf16": MILO_BF16, "int8": MILO_INT8, "int2": MILO_INT2}
KV_DTYPES = {"int8": MILO_INT8, "fp8": MILO_FP8, "int4": MILO_INT4}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


class milo_cache_shape(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int32), ("H", ctypes.c_int32), ("T", ctypes.c_int32), ("d", ctypes.c_int32),
                ("block_len", ctypes.c_int32), ("in_dtype", ctypes.c_int), ("n_blocks", ctypes.c_int32),
                ("block_starts", ctypes.c_void_p)]


class milo_compress_params(ctypes.Structure):
    _fields_ = [("budget_frac", ctypes.c_double), ("budget_abs", ctypes.c_int64), ("eps_rel", ctypes.c_double),
                ("eps_scope", ctypes.c_int32), ("r_min", ctypes.c_int32), ("r_max", ctypes.c_int32),
                ("factor_dtype", ctypes.c_int), ("max_sweeps", ctypes.c_int32), ("jacobi_tol", ctypes.c_float)]


class milo_rope_params(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int32), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_ctx", ctypes.c_double), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double),
                ("low_freq", ctypes.c_double), ("high_freq", ctypes.c_double), ("attn_factor", ctypes.c_double)]


class milo_kv_shape(ctypes.Structure):
    _fields_ = [("L", ctypes.c_int32), ("S", ctypes.c_int32), ("H", ctypes.c_int32), ("cap", ctypes.c_int32),
                ("d", ctypes.c_int32), ("block_len", ctypes.c_int32), ("dtype", ctypes.c_int)]


class MiloError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None
EXPORTS = [
    "milo_factor_arena_size", "milo_compress_workspace_size", "milo_rank_budget", "milo_default_params",
    "milo_compress", "milo_allocate_workspace_size", "milo_allocate", "milo_decode_workspace_size",
    "milo_decode_attn", "milo_factors_get", "milo_factors_wrap", "milo_factors_export",
    "milo_factors_import", "milo_factors_destroy", "milo_get_status", "milo_status_string", "milo_version",
    "milo_allocate_noalloc", "milo_test_decode_inject", "milo_timing_enable", "milo_timing_read",
    "milo_jacobi_rounds", "milo_decode_tail_workspace_size", "milo_decode_attn_tail",
    "milo_decode_offload_workspace_size", "milo_decode_attn_offload", "milo_bm25_workspace_size",
    "milo_bm25_select", "milo_factors_shape", "milo_decode_attn_offload_tail",
    "milo_rope_default_params", "milo_rope_freqs", "milo_rope", "milo_kv_cache_size", "milo_kv_layout",
    "milo_kv_append", "milo_kv_read", "milo_kv_select_workspace_size", "milo_kv_select",
    "milo_kv_attn_workspace_size", "milo_kv_attn", "milo_decode_kv_workspace_size", "milo_decode_attn_kv",
]

# stages of milo_timing_read, in order (milo_timed_stage)
TIMED_STAGES = ["gram", "jacobi", "refine", "select", "project", "decode_prep", "decode", "combine", "tail",
                "stage", "retrieve", "rope", "kv_write", "kv_read", "kv_select", "kv_attn"]

MILO_NOALLOC_MAX_BLOCKS = 65536
MILO_ROPE_MAX_D = 512


def lib():
    """Load libmilo.so (raises if it is absent: there is no other path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmilo.so not built at {LIB_PATH}; run block_wise_rank_b200/build.py")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        SP, PP = ctypes.POINTER(milo_cache_shape), ctypes.POINTER(milo_compress_params)
        L.milo_factor_arena_size.argtypes = [SP, PP]; L.milo_factor_arena_size.restype = SZ
        L.milo_compress_workspace_size.argtypes = [SP, PP]; L.milo_compress_workspace_size.restype = SZ
        L.milo_rank_budget.argtypes = [SP, PP]; L.milo_rank_budget.restype = I64
        L.milo_default_params.argtypes = [PP]; L.milo_default_params.restype = None
        L.milo_compress.argtypes = [SP, P, P, PP, P, SZ, P, SZ, ctypes.POINTER(P), P]
        L.milo_compress.restype = ctypes.c_int
        L.milo_allocate_workspace_size.argtypes = [I32, I32, I32]; L.milo_allocate_workspace_size.restype = SZ
        L.milo_allocate.argtypes = [P, P, I32, I32, I32, I32, I32, I64, I32, I32, P, P, SZ, P]
        L.milo_allocate.restype = ctypes.c_int
        L.milo_allocate_noalloc.argtypes = [P, P, I32, I32, I32, I32, I32, I64, I32, I32, P, P]
        L.milo_allocate_noalloc.restype = ctypes.c_int
        L.milo_decode_workspace_size.argtypes = [P, I32, I32, I32]; L.milo_decode_workspace_size.restype = SZ
        L.milo_decode_attn.argtypes = [P, P, I32, I32, P, P, I32, ctypes.c_double, P, P, SZ, P]
        L.milo_decode_tail_workspace_size.argtypes = [P, I32, I32, I32]
        L.milo_decode_tail_workspace_size.restype = SZ
        L.milo_decode_attn_tail.argtypes = [P, P, I32, I32, P, P, I32, ctypes.c_double, P, P, I32, I32, P, P, P,
                                            SZ, P]
        L.milo_decode_attn_tail.restype = ctypes.c_int
        L.milo_decode_offload_workspace_size.argtypes = [P, I32, I32, I32]
        L.milo_decode_offload_workspace_size.restype = SZ
        L.milo_decode_attn_offload.argtypes = [P, P, I32, I32, P, P, I32, ctypes.c_double, P, P, SZ, P]
        L.milo_decode_attn_offload.restype = ctypes.c_int
        L.milo_decode_attn_offload_tail.argtypes = [P, P, I32, I32, P, P, I32, ctypes.c_double, P, P, I32, I32, P,
                                                    P, P, SZ, P]
        L.milo_decode_attn_offload_tail.restype = ctypes.c_int
        L.milo_bm25_workspace_size.argtypes = [I32, I32, I32]
        L.milo_bm25_workspace_size.restype = SZ
        L.milo_bm25_select.argtypes = [P, P, P, P, I32, I32, I32, P, P, P, I32, I32, ctypes.c_double,
                                       ctypes.c_double, I32, P, P, P, SZ, P]
        L.milo_bm25_select.restype = ctypes.c_int
        L.milo_decode_attn.restype = ctypes.c_int
        L.milo_factors_get.argtypes = [P, I32, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.POINTER(P),
                                       ctypes.POINTER(P), ctypes.POINTER(P), ctypes.POINTER(P),
                                       ctypes.POINTER(P), ctypes.POINTER(I64)]
        L.milo_factors_get.restype = ctypes.c_int
        L.milo_factors_wrap.argtypes = [SP, PP, P, SZ, ctypes.POINTER(P)]; L.milo_factors_wrap.restype = ctypes.c_int
        L.milo_factors_export.argtypes = [P, P, ctypes.POINTER(SZ), P]; L.milo_factors_export.restype = ctypes.c_int
        L.milo_factors_import.argtypes = [P, SZ, P, SZ, ctypes.POINTER(P), P]
        L.milo_factors_import.restype = ctypes.c_int
        L.milo_factors_destroy.argtypes = [P]; L.milo_factors_destroy.restype = None
        L.milo_factors_shape.argtypes = [P, ctypes.POINTER(milo_cache_shape), ctypes.POINTER(milo_compress_params)]
        L.milo_factors_shape.restype = ctypes.c_int
        L.milo_get_status.argtypes = [P]; L.milo_get_status.restype = ctypes.c_int
        L.milo_status_string.argtypes = [ctypes.c_int]; L.milo_status_string.restype = ctypes.c_char_p
        L.milo_version.argtypes = []; L.milo_version.restype = ctypes.c_char_p
        L.milo_test_decode_inject.argtypes = [I32, ctypes.c_uint64]
        L.milo_test_decode_inject.restype = ctypes.c_int
        L.milo_timing_enable.argtypes = [I32]; L.milo_timing_enable.restype = ctypes.c_int
        L.milo_timing_read.argtypes = [P, P, I32]; L.milo_timing_read.restype = ctypes.c_int
        L.milo_jacobi_rounds.argtypes = [P, P, P]; L.milo_jacobi_rounds.restype = ctypes.c_int
        RP, KP, F64 = ctypes.POINTER(milo_rope_params), ctypes.POINTER(milo_kv_shape), ctypes.c_double
        L.milo_rope_default_params.argtypes = [RP, I32, F64]; L.milo_rope_default_params.restype = None
        L.milo_rope_freqs.argtypes = [RP, P, P]; L.milo_rope_freqs.restype = ctypes.c_int
        L.milo_rope.argtypes = [RP, P, I32, I64, I64, P, I32, I64, I64, P, I64, I64, I32, I32, P]
        L.milo_rope.restype = ctypes.c_int
        L.milo_kv_cache_size.argtypes = [KP]; L.milo_kv_cache_size.restype = SZ
        L.milo_kv_layout.argtypes = [KP, P]; L.milo_kv_layout.restype = ctypes.c_int
        L.milo_kv_append.argtypes = [KP, P, SZ, P, P, I32, P, I32, P, P, P]
        L.milo_kv_append.restype = ctypes.c_int
        L.milo_kv_read.argtypes = [KP, P, SZ, I32, P, P, P, P, I32, P]
        L.milo_kv_read.restype = ctypes.c_int
        L.milo_kv_select_workspace_size.argtypes = [KP, I32]; L.milo_kv_select_workspace_size.restype = SZ
        L.milo_kv_select.argtypes = [KP, P, SZ, P, I32, I32, I32, P, I32, I32, I32, P, P, P, SZ, P]
        L.milo_kv_select.restype = ctypes.c_int
        L.milo_kv_attn_workspace_size.argtypes = [KP, I32, I32, I32]; L.milo_kv_attn_workspace_size.restype = SZ
        L.milo_kv_attn.argtypes = [KP, P, SZ, P, I32, I32, I32, P, P, I32, F64, P, P, P, SZ, P]
        L.milo_kv_attn.restype = ctypes.c_int
        L.milo_decode_kv_workspace_size.argtypes = [P, I32, I32, I32, KP, I32]
        L.milo_decode_kv_workspace_size.restype = SZ
        L.milo_decode_attn_kv.argtypes = [P, P, I32, I32, P, P, I32, F64, KP, P, SZ, P, P, I32, P, P, SZ, P]
        L.milo_decode_attn_kv.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().milo_status_string(int(s)).decode()


def _check(s: int, what: str, allow_warn: bool = False):
    if s == MILO_OK or (allow_warn and s == MILO_WARN_NOT_CONVERGED):
        return s
    raise MiloError(s, what)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _tensors(x):
    """The CUDA tensors of a call's arguments or results."""
    if isinstance(x, torch.Tensor):
        return [x] if x.is_cuda else []
    if isinstance(x, (tuple, list)):
        return [t for y in x for t in _tensors(y)]
    x = getattr(x, "buf", getattr(x, "arena", None))                # KvCache, Factors
    return [x] if isinstance(x, torch.Tensor) and x.is_cuda else []


def _under(stream, call, *args):
    """call(*args) on `stream`, in that stream's memory: taken from the current stream's, an output or workspace
    would be used beside earlier work that may still be under way there.  The allocator is told that the arguments
    are used on `stream`, and the results by the current stream's program."""
    now = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        r = call(*args)
    for t in _tensors(args):
        t.record_stream(stream)
    for t in _tensors(r):
        t.record_stream(now)
    return r


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return MILO_F32
    if t == torch.bfloat16:
        return MILO_BF16
    raise ValueError(f"unsupported cache dtype {t}")


def default_params(**kw) -> milo_compress_params:
    p = milo_compress_params()
    lib().milo_default_params(ctypes.byref(p))
    for k, v in kw.items():
        if k == "factor_dtype" and isinstance(v, str):
            v = DTYPES[v]
        setattr(p, k, v)
    return p


def cache_shape(L, H, T, d, block_len, in_dtype, starts=None) -> milo_cache_shape:
    """The C shape; `starts` (token offsets of variable-length blocks, n_b + 1
    values from 0 to T) is kept alive on the returned object."""
    if isinstance(in_dtype, torch.dtype):
        in_dtype = _dtype_code(in_dtype)
    if starts is None:
        return milo_cache_shape(L, H, T, d, block_len, in_dtype, 0, None)
    arr = (ctypes.c_int32 * len(starts))(*[int(x) for x in starts])
    s = milo_cache_shape(L, H, T, d, block_len, in_dtype, len(starts) - 1, ctypes.cast(arr, ctypes.c_void_p))
    s._starts = arr
    return s


def block_starts(shape: milo_cache_shape):
    """The variable blocks' starts of a shape (a list), or None."""
    if not shape.n_blocks or not shape.block_starts:
        return None
    return list((ctypes.c_int32 * (shape.n_blocks + 1)).from_address(shape.block_starts))


def milo_factor_arena_size(shape, params) -> int:
    return lib().milo_factor_arena_size(ctypes.byref(shape), ctypes.byref(params))


def milo_compress_workspace_size(shape, params) -> int:
    return lib().milo_compress_workspace_size(ctypes.byref(shape), ctypes.byref(params))


def milo_rank_budget(shape, params) -> int:
    return lib().milo_rank_budget(ctypes.byref(shape), ctypes.byref(params))


def _bytes(n: int, device) -> torch.Tensor:
    # 256-byte aligned device buffer (the caching allocator aligns to 512 B)
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


@dataclass
class Factors:
    """A libmilo factor handle plus the device arena it views."""
    handle: ctypes.c_void_p
    arena: torch.Tensor
    shape: milo_cache_shape
    params: milo_compress_params

    def view(self, kind: int):
        """Device views of one kind as torch tensors (ranks, offsets, sigma, eps, data, scaleA, scaleB, R)."""
        P = ctypes.c_void_p
        ptrs = [P() for _ in range(7)]
        R = ctypes.c_int64()
        _check(lib().milo_factors_get(self.handle, kind, *[ctypes.byref(p) for p in ptrs], ctypes.byref(R)),
               "milo_factors_get")
        return [p.value for p in ptrs], R.value

    def close(self):
        if self.handle is not None and self.handle.value:
            lib().milo_factors_destroy(self.handle)
            self.handle = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def milo_compress(K: torch.Tensor, V: torch.Tensor, block_len: int, params=None, workspace=None,
                  arena=None, stream=None, starts=None) -> Factors:
    """Compress caches K (pre-RoPE) and V, [L][H][T][d] device tensors.  With
    `starts` (n_b + 1 token offsets) the blocks have variable lengths and
    block_len is the longest."""
    if stream is not None:
        return _under(stream, milo_compress, K, V, block_len, params, workspace, arena, None, starts)
    assert K.shape == V.shape and K.dtype == V.dtype and K.is_cuda and V.is_cuda
    assert K.is_contiguous() and V.is_contiguous()
    L, H, T, d = K.shape
    shape = cache_shape(L, H, T, d, block_len, K.dtype, starts)
    params = params or default_params()
    ws_n = milo_compress_workspace_size(shape, params)
    ar_n = milo_factor_arena_size(shape, params)
    if ws_n == 0 or ar_n == 0:
        raise MiloError(MILO_ERR_INVALID_ARG, "milo_compress sizes")
    if workspace is None:
        workspace = _bytes(ws_n, K.device)
    if arena is None:
        arena = _bytes(ar_n, K.device)
    h = ctypes.c_void_p()
    s = lib().milo_compress(ctypes.byref(shape), _ptr(K), _ptr(V), ctypes.byref(params), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _ptr(arena),
                            arena.numel() * arena.element_size(), ctypes.byref(h), _stream())
    _check(s, "milo_compress")
    return Factors(h, arena, shape, params)


def milo_allocate_workspace_size(n_groups: int, n_b: int, d: int = 128) -> int:
    return lib().milo_allocate_workspace_size(n_groups, n_b, d)


def milo_allocate(sigma: torch.Tensor, eps: torch.Tensor, n_groups: int, n_b: int, T: int, block_len: int,
                  R: int, r_min: int = 0, r_max: int = 0, ranks_out=None, workspace=None, stream=None):
    """Ranks int32 [n_groups * n_b] for sigma float32 [n_groups*n_b][128], eps float64 [n_groups]."""
    if stream is not None:
        return _under(stream, milo_allocate, sigma, eps, n_groups, n_b, T, block_len, R, r_min, r_max,
                      ranks_out, workspace)
    assert sigma.dtype == torch.float32 and eps.dtype == torch.float64 and sigma.is_contiguous()
    d = sigma.shape[-1]
    if ranks_out is None:
        ranks_out = torch.empty(n_groups * n_b, dtype=torch.int32, device=sigma.device)
    if workspace is None:
        workspace = _bytes(milo_allocate_workspace_size(n_groups, n_b, d), sigma.device)
    s = lib().milo_allocate(_ptr(sigma), _ptr(eps), n_groups, n_b, d, T, block_len, int(R), r_min, r_max,
                            _ptr(ranks_out), _ptr(workspace), workspace.numel(), _stream())
    _check(s, "milo_allocate")
    return ranks_out


def milo_allocate_noalloc(sigma: torch.Tensor, eps: torch.Tensor, n_groups: int, n_b: int, T: int, block_len: int,
                          R: int, r_min: int = 0, r_max: int = 0, ranks_out=None, stream=None):
    """milo_allocate without a workspace: the library's built-in device scratch
    (at most MILO_NOALLOC_MAX_BLOCKS blocks) stands in for it."""
    if stream is not None:
        return _under(stream, milo_allocate_noalloc, sigma, eps, n_groups, n_b, T, block_len, R, r_min, r_max,
                      ranks_out)
    assert sigma.dtype == torch.float32 and eps.dtype == torch.float64 and sigma.is_contiguous()
    d = sigma.shape[-1]
    if ranks_out is None:
        ranks_out = torch.empty(n_groups * n_b, dtype=torch.int32, device=sigma.device)
    s = lib().milo_allocate_noalloc(_ptr(sigma), _ptr(eps), n_groups, n_b, d, T, block_len, int(R), r_min, r_max,
                                    _ptr(ranks_out), _stream())
    _check(s, "milo_allocate_noalloc")
    return ranks_out


def milo_decode_workspace_size(f: Factors, S: int, Hq: int, n_sel: int) -> int:
    return lib().milo_decode_workspace_size(f.handle, S, Hq, n_sel)


def milo_decode_attn(f: Factors, q: torch.Tensor, selected: torch.Tensor, positions=None, rope_base=1e6,
                     out=None, workspace=None, stream=None):
    """GQA decode attention over the selected compressed blocks; q [L][S][Hq][d] fp32."""
    if stream is not None:
        return _under(stream, milo_decode_attn, f, q, selected, positions, rope_base, out, workspace)
    assert q.dtype == torch.float32 and q.is_contiguous() and q.is_cuda
    L, S, Hq, d = q.shape
    n_sel = selected.shape[1]
    assert selected.dtype == torch.int32 and selected.shape[0] == S and selected.is_contiguous()
    if positions is not None:
        assert positions.dtype == torch.int32 and positions.shape == selected.shape and positions.is_contiguous()
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = _bytes(milo_decode_workspace_size(f, S, Hq, n_sel), q.device)
    s = lib().milo_decode_attn(f.handle, _ptr(q), S, Hq, _ptr(selected), _ptr(positions), n_sel, float(rope_base),
                               _ptr(out), _ptr(workspace), workspace.numel(), _stream())
    _check(s, "milo_decode_attn")
    return out


def milo_decode_tail_workspace_size(f: Factors, S: int, Hq: int, n_sel: int) -> int:
    return lib().milo_decode_tail_workspace_size(f.handle, S, Hq, n_sel)


def milo_decode_attn_tail(f: Factors, q: torch.Tensor, selected: torch.Tensor, k_tail: torch.Tensor,
                          v_tail: torch.Tensor, tail_len: torch.Tensor, positions=None, rope_base=1e6, out=None,
                          workspace=None, stream=None):
    """Decode attention over the selected compressed blocks and each session's
    recent uncompressed tokens: k_tail / v_tail [L][S][H][tail_cap][d] (fp32 or
    bf16, keys already rotated), tail_len int32 [S]."""
    if stream is not None:
        return _under(stream, milo_decode_attn_tail, f, q, selected, k_tail, v_tail, tail_len, positions,
                      rope_base, out, workspace)
    assert q.dtype == torch.float32 and q.is_contiguous() and q.is_cuda
    L, S, Hq, d = q.shape
    n_sel = selected.shape[1]
    assert selected.dtype == torch.int32 and selected.shape[0] == S and selected.is_contiguous()
    if positions is not None:
        assert positions.dtype == torch.int32 and positions.shape == selected.shape and positions.is_contiguous()
    assert k_tail.dtype == v_tail.dtype and k_tail.dtype in (torch.float32, torch.bfloat16)
    assert k_tail.shape == v_tail.shape and k_tail.dim() == 5 and k_tail.shape[:2] == (L, S) and k_tail.shape[4] == d
    assert k_tail.shape[2] == f.shape.H
    assert k_tail.is_contiguous() and v_tail.is_contiguous()
    assert tail_len.dtype == torch.int32 and tail_len.shape == (S,) and tail_len.is_contiguous()
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = _bytes(milo_decode_tail_workspace_size(f, S, Hq, n_sel), q.device)
    dt = MILO_BF16 if k_tail.dtype == torch.bfloat16 else MILO_F32
    s = lib().milo_decode_attn_tail(f.handle, _ptr(q), S, Hq, _ptr(selected), _ptr(positions), n_sel,
                                    float(rope_base), _ptr(k_tail), _ptr(v_tail), dt, k_tail.shape[3],
                                    _ptr(tail_len), _ptr(out), _ptr(workspace), workspace.numel(), _stream())
    _check(s, "milo_decode_attn_tail")
    return out


def factors_to_host(f: Factors) -> Factors:
    """A handle over a pinned host copy of f's arena (for milo_decode_attn_offload)."""
    n = f.arena.numel()
    raw = torch.empty(n + 256, dtype=torch.uint8, pin_memory=True)
    host = raw[(-raw.data_ptr()) % 256:][:n]   # the arena's 256-byte alignment
    host.copy_(f.arena)
    return milo_factors_wrap(f.shape, f.params, host)


def milo_decode_offload_workspace_size(f: Factors, S: int, Hq: int, n_sel: int) -> int:
    return lib().milo_decode_offload_workspace_size(f.handle, S, Hq, n_sel)


def milo_decode_attn_offload(f: Factors, q: torch.Tensor, selected: torch.Tensor, positions=None, rope_base=1e6,
                             out=None, workspace=None, stream=None):
    """milo_decode_attn for a handle whose arena is in pinned host memory: the
    selected blocks' factors are staged on the device each call."""
    if stream is not None:
        return _under(stream, milo_decode_attn_offload, f, q, selected, positions, rope_base, out, workspace)
    assert q.dtype == torch.float32 and q.is_contiguous() and q.is_cuda
    L, S, Hq, d = q.shape
    n_sel = selected.shape[1]
    assert selected.dtype == torch.int32 and selected.shape[0] == S and selected.is_contiguous()
    if positions is not None:
        assert positions.dtype == torch.int32 and positions.shape == selected.shape and positions.is_contiguous()
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = _bytes(milo_decode_offload_workspace_size(f, S, Hq, n_sel), q.device)
    s = lib().milo_decode_attn_offload(f.handle, _ptr(q), S, Hq, _ptr(selected), _ptr(positions), n_sel,
                                       float(rope_base), _ptr(out), _ptr(workspace), workspace.numel(),
                                       _stream())
    _check(s, "milo_decode_attn_offload")
    return out


def milo_bm25_select(tables, vocab: int, n_sel: int, k1: float = 1.2, beta: float = 0.75, device="cuda",
                     workspace=None, stream=None):
    """BM25 block retrieval on the GPU.  tables = (blk_ptr, blk_term, blk_tf,
    blk_len, q_ptr, q_term, q_tf), int32 (any device).  Returns (selected
    int32 [S][n_sel], scores fp64 [S][n_b]) on `device`."""
    if stream is not None:
        return _under(stream, milo_bm25_select, tables, vocab, n_sel, k1, beta, device, workspace)
    t = [x.to(device=device, dtype=torch.int32).contiguous() for x in tables]
    blk_ptr, blk_term, blk_tf, blk_len, q_ptr, q_term, q_tf = t
    n_b, S = blk_len.numel(), q_ptr.numel() - 1
    selected = torch.empty(S, n_sel, dtype=torch.int32, device=device)
    scores = torch.empty(S, n_b, dtype=torch.float64, device=device)
    if workspace is None:
        workspace = _bytes(lib().milo_bm25_workspace_size(n_b, vocab, S), device)
    s = lib().milo_bm25_select(_ptr(blk_ptr), _ptr(blk_term), _ptr(blk_tf), _ptr(blk_len), n_b, blk_term.numel(),
                               vocab, _ptr(q_ptr), _ptr(q_term), _ptr(q_tf), S, q_term.numel(), float(k1),
                               float(beta), n_sel, _ptr(selected), _ptr(scores), _ptr(workspace), workspace.numel(),
                               _stream())
    _check(s, "milo_bm25_select")
    return selected, scores


def milo_decode_attn_offload_tail(f: Factors, q: torch.Tensor, selected: torch.Tensor, k_tail: torch.Tensor,
                                  v_tail: torch.Tensor, tail_len: torch.Tensor, positions=None, rope_base=1e6,
                                  out=None, workspace=None, stream=None):
    """milo_decode_attn_offload with each session's recent uncompressed tokens
    (device tensors, as milo_decode_attn_tail) in the same softmax."""
    if stream is not None:
        return _under(stream, milo_decode_attn_offload_tail, f, q, selected, k_tail, v_tail, tail_len,
                      positions, rope_base, out, workspace)
    assert q.dtype == torch.float32 and q.is_contiguous() and q.is_cuda
    L, S, Hq, d = q.shape
    n_sel = selected.shape[1]
    assert selected.dtype == torch.int32 and selected.shape[0] == S and selected.is_contiguous()
    assert k_tail.dtype == v_tail.dtype and k_tail.dtype in (torch.float32, torch.bfloat16)
    assert k_tail.shape == v_tail.shape and k_tail.is_contiguous() and v_tail.is_contiguous()
    assert tail_len.dtype == torch.int32 and tail_len.shape == (S,)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = _bytes(milo_decode_offload_workspace_size(f, S, Hq, n_sel), q.device)
    dt = MILO_BF16 if k_tail.dtype == torch.bfloat16 else MILO_F32
    s = lib().milo_decode_attn_offload_tail(f.handle, _ptr(q), S, Hq, _ptr(selected), _ptr(positions), n_sel,
                                            float(rope_base), _ptr(k_tail), _ptr(v_tail), dt, k_tail.shape[3],
                                            _ptr(tail_len), _ptr(out), _ptr(workspace), workspace.numel(),
                                            _stream())
    _check(s, "milo_decode_attn_offload_tail")
    return out


# ------------------------------------------------- rotary positions
def rope_params(d: int, base: float = 1e6, rotary_dim: int = 0, interleaved: bool = False, scaling: str = "none",
                **kw) -> milo_rope_params:
    """The C parameters of milo_rope; further fields of milo_rope_params by name."""
    p = milo_rope_params()
    lib().milo_rope_default_params(ctypes.byref(p), d, base)
    p.rotary_dim, p.interleaved, p.scaling = rotary_dim, int(interleaved), ROPE_SCALINGS[scaling]
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def milo_rope_freqs(params: milo_rope_params):
    """(angles per position of every pair as a list, factor on the turned channels)."""
    w = (ctypes.c_double * (MILO_ROPE_MAX_D // 2))()
    m = ctypes.c_double()
    _check(lib().milo_rope_freqs(ctypes.byref(params), ctypes.cast(w, ctypes.c_void_p),
                                 ctypes.cast(ctypes.byref(m), ctypes.c_void_p)), "milo_rope_freqs")
    return list(w)[:(params.rotary_dim or params.d) // 2], m.value


def _on(t: torch.Tensor) -> int:
    """The raw current stream of a call on t, which lives on the current CUDA device."""
    if not t.is_cuda:
        raise ValueError(f"tensor on {t.device}, a CUDA tensor expected")
    dev = t.get_device()
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensor on {t.device}, and the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(dev)


def _same_device(first, *tensors):
    dev = first.get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on {first.device} and {t.device}")


def _int32(t: torch.Tensor, shape, what: str):
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous int32 {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")


def milo_rope(x: torch.Tensor, positions: torch.Tensor, params: milo_rope_params, out=None, out_dtype=None,
              transpose: bool = False, stream=None) -> torch.Tensor:
    """Rows x [n_tokens][n_heads][d] (fp32 or bf16, any strides, d contiguous)
    turned to positions int32 [n_pos] (token t takes positions[t % n_pos]);
    transpose=True gives the gradient with respect to x of a gradient x.
    out=x turns in place."""
    if stream is not None:
        return _under(stream, milo_rope, x, positions, params, out, out_dtype, transpose)
    if x.dim() != 3 or x.shape[2] != params.d or (x.numel() and x.stride(2) != 1):
        raise ValueError(f"x: [n_tokens][n_heads][{params.d}] with contiguous rows expected, got {tuple(x.shape)}")
    s = _on(x)
    if out is None:
        out = torch.empty_like(x, dtype=out_dtype, memory_format=torch.contiguous_format)
    elif out.shape != x.shape or (out.numel() and out.stride(2) != 1):
        raise ValueError(f"out: {tuple(x.shape)} with contiguous rows expected, got {tuple(out.shape)}")
    n_pos = positions.numel()
    _int32(positions, (n_pos,), "positions")
    _same_device(x, out, positions)
    n, h, _ = x.shape
    xs, ys = x.stride(), out.stride()
    rc = lib().milo_rope(params, x.data_ptr(), _dtype_code(x.dtype), xs[0], xs[1], out.data_ptr(),
                         _dtype_code(out.dtype), ys[0], ys[1], positions.data_ptr(), n_pos, n, h, transpose, s)
    _check(rc, "milo_rope")
    return out


# ------------------------------------- quantised cache of recent tokens
def kv_shape(L: int, S: int, H: int, cap: int, block_len: int = 64, dtype="int8", d: int = 128) -> milo_kv_shape:
    return milo_kv_shape(L, S, H, cap, d, block_len, KV_DTYPES[dtype] if isinstance(dtype, str) else dtype)


def milo_kv_cache_size(shape: milo_kv_shape) -> int:
    return lib().milo_kv_cache_size(ctypes.byref(shape))


def milo_kv_layout(shape: milo_kv_shape):
    """Byte offsets of a layer's sections (k, v, k params, v params, bounds, bound codes, bound scales)."""
    o = (ctypes.c_size_t * 7)()
    _check(lib().milo_kv_layout(ctypes.byref(shape), ctypes.cast(o, ctypes.c_void_p)), "milo_kv_layout")
    return list(o)


class KvCache:
    """A quantised cache of recent tokens: its shape and its buffer (uint8,
    at least milo_kv_cache_size bytes; made on `device` when not given)."""

    def __init__(self, shape: milo_kv_shape, buf=None, device="cuda"):
        n = milo_kv_cache_size(shape)
        if n == 0:
            raise MiloError(MILO_ERR_INVALID_ARG, "milo_kv_cache_size")
        self.shape = shape
        self.buf = _bytes(n, device) if buf is None else buf
        if self.buf.dtype != torch.uint8 or not self.buf.is_contiguous():
            raise ValueError("a cache's buffer is a contiguous uint8 tensor")
        self._sizes = {}   # workspace bytes by call shape

    def _ws(self, name: str, *args) -> int:
        n = self._sizes.get((name, args))
        if n is None:
            n = self._sizes[name, args] = getattr(lib(), name)(ctypes.byref(self.shape), *args)
        return n

    @property
    def n_b(self) -> int:
        return -(-self.shape.cap // self.shape.block_len)

    def layer(self, l: int) -> "KvCache":
        """The part of layer l as a cache of its own (the same memory)."""
        s = self.shape
        if not 0 <= l < s.L:
            raise IndexError(l)
        n = milo_kv_cache_size(s) // s.L
        one = milo_kv_shape(1, s.S, s.H, s.cap, s.d, s.block_len, s.dtype)
        return KvCache(one, self.buf[l * n:(l + 1) * n])


def _strides(t: torch.Tensor):
    """t's strides; 0 where a dimension has one index (any stride is as good)."""
    return tuple(0 if n == 1 else s for n, s in zip(t.shape, t.stride()))


def milo_kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, start: torch.Tensor, count=None,
                   stream=None) -> None:
    """Quantise k, v [L][S][H][n][d] (fp32 or bf16; any strides that k and v
    share, d contiguous) into rows start[s] .. of every session; count int32
    [S]: only the first count[s] tokens."""
    if stream is not None:
        return _under(stream, milo_kv_append, cache, k, v, start, count)
    c = cache.shape
    if k.shape != v.shape or k.dtype != v.dtype or k.dim() != 5 or \
            tuple(k.shape[:3]) != (c.L, c.S, c.H) or k.shape[4] != c.d:
        raise ValueError(f"k, v: [{c.L}][{c.S}][{c.H}][n][{c.d}] expected, got {tuple(k.shape)} and {tuple(v.shape)}")
    st = _strides(k)
    if k.numel() and (st != _strides(v) or st[4] != 1):
        raise ValueError("k and v: equal strides and contiguous rows expected")
    s = _on(k)
    _int32(start, (c.S,), "start")
    if count is not None:
        _int32(count, (c.S,), "count")
    _same_device(k, v, start, count, cache.buf)
    strides = None if k.is_contiguous() else (ctypes.c_int64 * 4)(*st[:4])
    rc = lib().milo_kv_append(c, cache.buf.data_ptr(), cache.buf.numel(), k.data_ptr(), v.data_ptr(),
                              _dtype_code(k.dtype), strides, k.shape[3], start.data_ptr(),
                              None if count is None else count.data_ptr(), s)
    _check(rc, "milo_kv_append")


def milo_kv_read(cache: KvCache, start: torch.Tensor, n: int, count=None, k_out=None, v_out=None,
                 out_dtype=torch.float32, stream=None):
    """(k, v) [L][S][H][n][d]: rows start[s] .. start[s] + n - 1 as values.
    With count, rows behind count[s] are left as they were in k_out / v_out."""
    if stream is not None:
        return _under(stream, milo_kv_read, cache, start, n, count, k_out, v_out, out_dtype)
    c = cache.shape
    shape = (c.L, c.S, c.H, n, c.d)
    if k_out is None:
        k_out = cache.buf.new_empty(shape, dtype=out_dtype)
    if v_out is None:
        v_out = torch.empty_like(k_out)
    for t in (k_out, v_out):
        if tuple(t.shape) != shape or not t.is_contiguous() or t.dtype != k_out.dtype:
            raise ValueError(f"k_out, v_out: contiguous {shape} of one type expected, got {t.dtype} {tuple(t.shape)}")
    s = _on(k_out)
    _int32(start, (c.S,), "start")
    if count is not None:
        _int32(count, (c.S,), "count")
    _same_device(k_out, v_out, start, count, cache.buf)
    rc = lib().milo_kv_read(c, cache.buf.data_ptr(), cache.buf.numel(), n, start.data_ptr(),
                            None if count is None else count.data_ptr(), k_out.data_ptr(), v_out.data_ptr(),
                            _dtype_code(k_out.dtype), s)
    _check(rc, "milo_kv_read")
    return k_out, v_out


def _kv_listed(selected: torch.Tensor) -> int:
    """Blocks of a selection; an empty one would be taken for none, which stands for every token."""
    if selected.dim() == 0 or selected.shape[-1] == 0:
        raise ValueError("a selection of at least one block id expected (-1 for none)")
    return selected.shape[-1]


def _kv_queries(cache: KvCache, q: torch.Tensor, length: torch.Tensor):
    """(n_q, Hq) of q [L][S][n_q][Hq][d] or [L][S][Hq][d]."""
    c = cache.shape
    shape = q.shape
    if len(shape) not in (4, 5) or shape[0] != c.L or shape[1] != c.S or shape[-1] != c.d or not q.is_contiguous():
        raise ValueError(f"q: contiguous [{c.L}][{c.S}]([n_q])[Hq][{c.d}] expected, got {tuple(shape)}")
    _int32(length, (c.S,), "length")
    return (shape[2] if len(shape) == 5 else 1), shape[-2]


def milo_kv_select(cache: KvCache, q: torch.Tensor, length: torch.Tensor, n_sel: int, n_first: int = 0,
                   n_last: int = 1, selected=None, scores=None, return_scores: bool = False, workspace=None,
                   stream=None):
    """Blocks of the cache picked by each query: int32 [L][S](n_q)[H][n_sel] ids,
    ascending, -1 behind the last; with return_scores also the fp32 scores
    [L][S](n_q)[H][n_b] (-inf: not a candidate)."""
    if stream is not None:
        return _under(stream, milo_kv_select, cache, q, length, n_sel, n_first, n_last, selected, scores,
                      return_scores, workspace)
    c = cache.shape
    n_q, Hq = _kv_queries(cache, q, length)
    lead = (c.L, c.S, n_q, c.H) if q.dim() == 5 else (c.L, c.S, c.H)
    s = _on(q)
    if selected is None:
        selected = length.new_empty(lead + (n_sel,))
    _int32(selected, lead + (n_sel,), "selected")
    if scores is None and return_scores:
        scores = q.new_empty(lead + (cache.n_b,), dtype=torch.float32)
    if scores is not None and (scores.dtype != torch.float32 or tuple(scores.shape) != lead + (cache.n_b,) or
                               not scores.is_contiguous()):
        raise ValueError(f"scores: contiguous float32 {lead + (cache.n_b,)} expected")
    if workspace is None:
        workspace = cache.buf.new_empty(cache._ws("milo_kv_select_workspace_size", n_q))
    _same_device(q, length, selected, scores, workspace, cache.buf)
    rc = lib().milo_kv_select(c, cache.buf.data_ptr(), cache.buf.numel(), q.data_ptr(), _dtype_code(q.dtype), n_q, Hq,
                              length.data_ptr(), n_sel, n_first, n_last, selected.data_ptr(),
                              None if scores is None else scores.data_ptr(), workspace.data_ptr(), workspace.numel(),
                              s)
    _check(rc, "milo_kv_select")
    return (selected, scores) if return_scores else selected


def milo_kv_attn_workspace_size(shape: milo_kv_shape, n_q: int, Hq: int, n_sel: int = 0) -> int:
    return lib().milo_kv_attn_workspace_size(ctypes.byref(shape), n_q, Hq, n_sel)


def milo_kv_attn(cache: KvCache, q: torch.Tensor, length: torch.Tensor, selected=None, scale: float = 0.0, out=None,
                 return_lse: bool = False, workspace=None, stream=None):
    """GQA attention of q [L][S](n_q)[Hq][d] (fp32 or bf16) over the cached
    tokens that each query sees, or those of the blocks in `selected`
    [L][S](n_q)[H][n_sel]; with return_lse also the fp32 log-sum-exp."""
    if stream is not None:
        return _under(stream, milo_kv_attn, cache, q, length, selected, scale, out, return_lse, workspace)
    c = cache.shape
    n_q, Hq = _kv_queries(cache, q, length)
    n_sel = 0 if selected is None else _kv_listed(selected)
    s = _on(q)
    if selected is not None:
        _int32(selected, tuple(q.shape[:-2]) + (c.H, n_sel), "selected")
    if out is None:
        out = torch.empty_like(q)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out: like q expected")
    lse = q.new_empty(q.shape[:-1], dtype=torch.float32) if return_lse else None
    if workspace is None:
        workspace = cache.buf.new_empty(cache._ws("milo_kv_attn_workspace_size", n_q, Hq, n_sel))
    _same_device(q, length, selected, out, workspace, cache.buf)
    rc = lib().milo_kv_attn(c, cache.buf.data_ptr(), cache.buf.numel(), q.data_ptr(), _dtype_code(q.dtype), n_q, Hq,
                            length.data_ptr(), None if selected is None else selected.data_ptr(), n_sel, scale,
                            out.data_ptr(), None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                            workspace.numel(), s)
    _check(rc, "milo_kv_attn")
    return (out, lse) if return_lse else out


def milo_decode_attn_kv(f: Factors, q: torch.Tensor, selected: torch.Tensor, cache: KvCache, length: torch.Tensor,
                        kv_selected=None, positions=None, rope_base=1e6, out=None, workspace=None, stream=None):
    """milo_decode_attn_tail with the recent tokens in a quantised cache: q
    [L][S][Hq][d] fp32, length int32 [S] tokens held, kv_selected int32
    [L][S][H][kv_n_sel] blocks of the cache (None: all its tokens)."""
    if stream is not None:
        return _under(stream, milo_decode_attn_kv, f, q, selected, cache, length, kv_selected, positions,
                      rope_base, out, workspace)
    c = cache.shape
    if q.dtype != torch.float32 or q.dim() != 4:
        raise ValueError("q: float32 [L][S][Hq][d] expected")
    _, Hq = _kv_queries(cache, q, length)
    kv_n_sel = 0 if kv_selected is None else _kv_listed(kv_selected)
    s = _on(q)
    _int32(selected, (c.S, selected.shape[-1]), "selected")
    if positions is not None:
        _int32(positions, selected.shape, "positions")
    if kv_selected is not None:
        _int32(kv_selected, (c.L, c.S, c.H, kv_n_sel), "kv_selected")
    if out is None:
        out = torch.empty_like(q)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous():
        raise ValueError("out: like q expected")
    n_sel = selected.shape[-1]
    if workspace is None:
        workspace = _bytes(lib().milo_decode_kv_workspace_size(f.handle, c.S, Hq, n_sel, c, kv_n_sel), q.device)
    _same_device(q, length, selected, positions, kv_selected, out, workspace, cache.buf)
    rc = lib().milo_decode_attn_kv(f.handle, q.data_ptr(), c.S, Hq, selected.data_ptr(),
                                   None if positions is None else positions.data_ptr(), n_sel, float(rope_base), c,
                                   cache.buf.data_ptr(), cache.buf.numel(), length.data_ptr(),
                                   None if kv_selected is None else kv_selected.data_ptr(), kv_n_sel, out.data_ptr(),
                                   workspace.data_ptr(), workspace.numel(), s)
    _check(rc, "milo_decode_attn_kv")
    return out


def milo_factors_wrap(shape, params, arena: torch.Tensor) -> Factors:
    h = ctypes.c_void_p()
    _check(lib().milo_factors_wrap(ctypes.byref(shape), ctypes.byref(params), _ptr(arena),
                                   arena.numel() * arena.element_size(), ctypes.byref(h)), "milo_factors_wrap")
    return Factors(h, arena, shape, params)


def milo_factors_export(f: Factors, stream=None) -> bytes:
    n = ctypes.c_size_t(0)
    _check(lib().milo_factors_export(f.handle, None, ctypes.byref(n), _stream(stream)), "milo_factors_export")
    buf = ctypes.create_string_buffer(n.value)
    _check(lib().milo_factors_export(f.handle, buf, ctypes.byref(n), _stream(stream)), "milo_factors_export")
    return buf.raw


def milo_factors_import(blob: bytes, arena: torch.Tensor, stream=None) -> Factors:
    h = ctypes.c_void_p()
    _check(lib().milo_factors_import(blob, len(blob), _ptr(arena), arena.numel() * arena.element_size(),
                                     ctypes.byref(h), _stream(stream)), "milo_factors_import")
    # shape and params from the new handle (its block starts stay valid while it lives)
    shape, params = milo_cache_shape(), milo_compress_params()
    _check(lib().milo_factors_shape(h, ctypes.byref(shape), ctypes.byref(params)), "milo_factors_shape")
    return Factors(h, arena, shape, params)


def milo_get_status(stream=None) -> int:
    return lib().milo_get_status(_stream(stream))


def milo_test_decode_inject(mode: int, wait_ns: int = 0) -> int:
    """Test hook: arm (mode 1) a withheld copy and a wait limit of wait_ns for
    the next tensor-core decode call, or disarm (mode 0).  Returns the status."""
    return lib().milo_test_decode_inject(int(mode), int(wait_ns))


def milo_timing_enable(on: bool = True) -> None:
    """Start (dropping earlier records) or stop bracketing each stage's kernels
    with CUDA events on their launch stream."""
    _check(lib().milo_timing_enable(1 if on else 0), "milo_timing_enable")


def milo_timing_read() -> dict:
    """{stage: (summed ms, launches)} of the records since milo_timing_enable;
    waits for the events and drops them."""
    n = len(TIMED_STAGES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    _check(lib().milo_timing_read(ctypes.cast(ms, ctypes.c_void_p), ctypes.cast(cnt, ctypes.c_void_p), n),
           "milo_timing_read")
    return {name: (float(ms[i]), int(cnt[i])) for i, name in enumerate(TIMED_STAGES)}


def milo_jacobi_rounds(stream=None) -> tuple:
    """(rounds that applied rotations, rotations applied) of the Jacobi
    eigensolves since the last read (synchronises)."""
    v = ctypes.c_int64(0)
    w = ctypes.c_int64(0)
    _check(lib().milo_jacobi_rounds(ctypes.cast(ctypes.byref(v), ctypes.c_void_p),
                                    ctypes.cast(ctypes.byref(w), ctypes.c_void_p), _stream(stream)),
           "milo_jacobi_rounds")
    return int(v.value), int(w.value)


def milo_version() -> str:
    return lib().milo_version().decode()
