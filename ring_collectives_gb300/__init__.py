"""ring_collectives_gb300 -- ring collectives over P logical ranks in one GB300's HBM.

A thin ctypes binding over ``libringcoll.so`` (the C ABI of
``include/ringcoll.h``).  Every function here only marshals arguments: the
work runs in the library's CUDA kernels.  PyTorch supplies device memory and
the current stream.

Slots are rows: a 2-D CUDA tensor ``t`` of shape ``[P, L]`` whose rows are
contiguous (``t.stride(1) == 1``) holds slot r at row r, so the slot stride is
``t.stride(0) * t.element_size()`` bytes.  Supported dtypes: float32,
bfloat16, int32.  Each call is asynchronous on the current CUDA stream (or the
``stream`` given); device-side errors are read with :func:`ring_status`.

If the library has not been built (``__graft_entry__.build()`` or
``python -m ring_collectives_gb300._build``) every call raises: there is no
fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

__all__ = [
    "RingError", "ring_ppermute_right", "ring_all_gather", "ring_reduce_scatter", "ring_reduce_scatter_bidir",
    "ring_allreduce", "ring_allreduce_ex", "ring_allreduce_workspace_bytes", "ring_allreduce_host",
    "ring_allreduce_fused", "ring_psum", "ring_allreduce_noalloc", "ag_gemm", "gemm_rs", "ring_status",
    "ring_status_ex", "ring_all_gather_ex", "ring_all_gather_workspace_bytes", "ring_reduce_scatter_ex",
    "ring_reduce_scatter_workspace_bytes", "ring_reduce_scatter_bidir_ex", "ring_reduce_scatter_bidir_workspace_bytes",
    "ag_gemm_ex", "ag_gemm_kn", "ag_gemm_workspace_bytes", "RC_B_NK", "RC_B_KN", "gemm_rs_ex", "gemm_rs_workspace_bytes",
    "ring_last_error", "ring_set_timeout_ms", "ring_set_slices", "ring_debug_skip_notify", "ag_gemm_debug_skip_piece",
    "ring_debug_set_trace", "ring_debug_l2_rate", "ring_finalize", "library_path", "load",
    "attn_fwd", "attn_fwd_workspace_bytes", "attn_bwd", "attn_bwd_workspace_bytes",
    "qk_norm_rope", "qk_norm_rope_bwd", "qk_norm_rope_bwd_workspace_bytes", "RC_ROPE_HALF", "RC_ROPE_PAIRS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libringcoll.so")

RC_OK, RC_ERR_INVALID, RC_ERR_CUDA, RC_ERR_TIMEOUT, RC_ERR_UNSUPPORTED, RC_ERR_NOMEM = range(6)
RC_ROPE_HALF, RC_ROPE_PAIRS = 0, 1   # rotated pairs (i, i + D/2) or (2i, 2i + 1)
RC_B_NK, RC_B_KN = 0, 1   # ag_gemm weight layouts: [N][K] (nn.Linear) or [K][N] (x @ W)
_DTYPE = {torch.float32: 0, torch.bfloat16: 1, torch.int32: 2}

_vp, _sz, _i, _u = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint
# C signatures of include/ringcoll.h: name -> (argument types, result type)
_SIGNATURES = {
    "ring_ppermute_right": ([_vp, _sz, _vp, _sz, _i, _sz, _i, _vp], _i),
    "ring_all_gather": ([_vp, _sz, _vp, _sz, _i, _sz, _i, _vp], _i),
    "ring_all_gather_ex": ([_vp, _sz, _vp, _sz, _i, _sz, _i, _vp, _sz, _vp], _i),
    "ring_all_gather_workspace_bytes": ([_i, _sz, _i], _sz),
    "ring_reduce_scatter_ex": ([_vp, _sz, _vp, _sz, _i, _sz, _i, _vp, _sz, _vp], _i),
    "ring_reduce_scatter_workspace_bytes": ([_i, _sz, _i], _sz),
    "ring_reduce_scatter_bidir_ex": ([_vp, _sz, _vp, _sz, _i, _sz, _i, _vp, _sz, _vp], _i),
    "ring_reduce_scatter_bidir_workspace_bytes": ([_i, _sz, _i], _sz),
    "ag_gemm_ex": ([_vp, _sz, _vp, _vp, _i, _vp, _i, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "ag_gemm_kn": ([_vp, _sz, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp], _i),
    "ag_gemm_workspace_bytes": ([_i, _i], _sz),
    "gemm_rs_ex": ([_vp, _sz, _vp, _sz, _vp, _sz, _i, _i, _i, _i, _vp, _sz, _vp], _i),
    "gemm_rs_workspace_bytes": ([_i, _i, _i, _i], _sz),
    "ring_reduce_scatter": ([_vp, _sz, _vp, _sz, _i, _sz, _i, _vp], _i),
    "ring_reduce_scatter_bidir": ([_vp, _sz, _vp, _sz, _i, _sz, _i, _vp], _i),
    "ring_allreduce": ([_vp, _sz, _i, _sz, _i, _vp], _i),
    "ring_allreduce_ex": ([_vp, _sz, _i, _sz, _i, _vp, _sz, _vp], _i),
    "ring_allreduce_workspace_bytes": ([_i, _sz, _i], _sz),
    "ring_allreduce_host": ([_vp, _sz, _vp, _sz, _vp, _sz, _i, _sz, _i, _vp], _i),
    "ring_allreduce_fused": ([_vp, _sz, _i, _sz, _i, _vp], _i),
    "ring_psum": ([_vp, _sz, _i, _sz, _i, _vp], _i),
    "ring_allreduce_noalloc": ([_vp, _sz, _i, _sz, _i, _vp], _i),
    "ag_gemm": ([_vp, _sz, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp], _i),
    "gemm_rs": ([_vp, _sz, _vp, _sz, _vp, _sz, _i, _i, _i, _i, _vp], _i),
    "ring_status": ([_vp], _i),
    "ring_status_ex": ([_vp, _vp], _i),
    "ring_last_error": ([], ctypes.c_char_p),
    "ring_set_timeout_ms": ([_u], _i),
    "ring_set_slices": ([_i], _i),
    "ring_debug_skip_notify": ([_i, _i], _i),
    "ag_gemm_debug_skip_piece": ([_i], _i),
    "ring_debug_set_trace": ([_vp, _sz], _i),
    "ring_debug_l2_rate": ([_vp, _vp, _vp, _sz, _i, _i, _vp], _i),
    "ring_finalize": ([], _i),
    "attn_fwd": ([ctypes.c_char_p, _vp], _i),
    "attn_fwd_workspace_bytes": ([ctypes.c_char_p], _sz),
    "attn_bwd": ([ctypes.c_char_p, _vp], _i),
    "attn_bwd_workspace_bytes": ([ctypes.c_char_p], _sz),
    "qk_norm_rope": ([ctypes.c_char_p, _vp], _i),
    "qk_norm_rope_bwd": ([ctypes.c_char_p, _vp], _i),
    "qk_norm_rope_bwd_workspace_bytes": ([ctypes.c_char_p], _sz),
}

_lib = None


class RingError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[rc={code}] {msg}")
        self.code = code


def library_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libringcoll.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(L, name)   # AttributeError here: the library is older than this module
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def ring_last_error() -> str:
    return load().ring_last_error().decode(errors="replace")


def _check(rc: int) -> None:
    if rc != RC_OK:
        raise RingError(rc, ring_last_error())


def _stream(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _slots(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 2 or (t.size(1) > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D [P, L] with contiguous rows")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return t.data_ptr(), t.stride(0) * t.element_size(), _DTYPE[t.dtype]


def ring_ppermute_right(src: torch.Tensor, dst: torch.Tensor, n: int | None = None, stream=None) -> torch.Tensor:
    """dst[r, :n] = src[(r-1+P) % P, :n]."""
    sp, ss, dt = _slots(src, "src")
    dp, ds, dt2 = _slots(dst, "dst")
    if dt != dt2 or src.size(0) != dst.size(0):
        raise ValueError("src and dst differ in dtype or rank count")
    n = min(src.size(1), dst.size(1)) if n is None else n
    with torch.cuda.device(src.device):
        _check(load().ring_ppermute_right(sp, ss, dp, ds, src.size(0), n, dt, _stream(stream, src.device)))
    return dst


def ring_all_gather(inp: torch.Tensor, out: torch.Tensor, n: int | None = None, stream=None) -> torch.Tensor:
    """out[r, k*n:(k+1)*n] = inp[k, :n] for every r, k."""
    ip, is_, dt = _slots(inp, "inp")
    op, os_, dt2 = _slots(out, "out")
    if dt != dt2 or inp.size(0) != out.size(0):
        raise ValueError("inp and out differ in dtype or rank count")
    n = inp.size(1) if n is None else n
    if out.size(1) < inp.size(0) * n:
        raise ValueError("out rows are shorter than P*n")
    with torch.cuda.device(inp.device):
        _check(load().ring_all_gather(ip, is_, op, os_, inp.size(0), n, dt, _stream(stream, inp.device)))
    return out


def ring_reduce_scatter(bufs: torch.Tensor, out: torch.Tensor, N: int | None = None, stream=None) -> torch.Tensor:
    """out[r, :N/P] = ring sum of chunk r; ``bufs`` is clobbered."""
    bp, bs, dt = _slots(bufs, "bufs")
    op, os_, dt2 = _slots(out, "out")
    if dt != dt2 or bufs.size(0) != out.size(0):
        raise ValueError("bufs and out differ in dtype or rank count")
    N = bufs.size(1) if N is None else N
    with torch.cuda.device(bufs.device):
        _check(load().ring_reduce_scatter(bp, bs, op, os_, bufs.size(0), N, dt, _stream(stream, bufs.device)))
    return out


def ring_reduce_scatter_bidir(bufs: torch.Tensor, out: torch.Tensor, N: int | None = None,
                              stream=None) -> torch.Tensor:
    """Bidirectional reduce-scatter (top halves travel left, bottom halves right);
    out[r, :N/P] = block r summed over ranks; ``bufs`` is clobbered."""
    fn = load().ring_reduce_scatter_bidir
    bp, bs, dt = _slots(bufs, "bufs")
    op, os_, dt2 = _slots(out, "out")
    if dt != dt2 or bufs.size(0) != out.size(0):
        raise ValueError("bufs and out differ in dtype or rank count")
    N = bufs.size(1) if N is None else N
    with torch.cuda.device(bufs.device):
        _check(fn(bp, bs, op, os_, bufs.size(0), N, dt, _stream(stream, bufs.device)))
    return out


def ring_allreduce(bufs: torch.Tensor, N: int | None = None, stream=None) -> torch.Tensor:
    """In-place ring all-reduce over the first N elements of every row."""
    bp, bs, dt = _slots(bufs, "bufs")
    N = bufs.size(1) if N is None else N
    with torch.cuda.device(bufs.device):
        _check(load().ring_allreduce(bp, bs, bufs.size(0), N, dt, _stream(stream, bufs.device)))
    return bufs


def ring_allreduce_workspace_bytes(P: int, N: int, dtype=torch.float32) -> int:
    fn = load().ring_allreduce_workspace_bytes
    return int(fn(P, N, _DTYPE[dtype]))


def ring_allreduce_ex(bufs: torch.Tensor, workspace: torch.Tensor, N: int | None = None, stream=None) -> torch.Tensor:
    """ring_allreduce with a caller-owned workspace (a zeroed CUDA byte tensor of
    at least ring_allreduce_workspace_bytes bytes); calls with distinct
    workspaces may run concurrently on different streams."""
    fn = load().ring_allreduce_ex
    bp, bs, dt = _slots(bufs, "bufs")
    if not workspace.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    N = bufs.size(1) if N is None else N
    with torch.cuda.device(bufs.device):
        _check(fn(bp, bs, bufs.size(0), N, dt, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                  _stream(stream, bufs.device)))
    return bufs


def _ws(workspace):
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def ring_all_gather_workspace_bytes(P: int, n: int, dtype=torch.float32) -> int:
    return int(load().ring_all_gather_workspace_bytes(P, n, _DTYPE[dtype]))


def ring_all_gather_ex(inp: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, n: int | None = None,
                       stream=None) -> torch.Tensor:
    """ring_all_gather with a caller-owned workspace (zeroed CUDA tensor of at
    least ring_all_gather_workspace_bytes bytes)."""
    ip, is_, dt = _slots(inp, "inp")
    op, os_, dt2 = _slots(out, "out")
    if dt != dt2 or inp.size(0) != out.size(0):
        raise ValueError("inp and out differ in dtype or rank count")
    n = inp.size(1) if n is None else n
    if out.size(1) < inp.size(0) * n:
        raise ValueError("out rows are shorter than P*n")
    wp, wb = _ws(workspace)
    with torch.cuda.device(inp.device):
        _check(load().ring_all_gather_ex(ip, is_, op, os_, inp.size(0), n, dt, wp, wb, _stream(stream, inp.device)))
    return out


def ring_reduce_scatter_workspace_bytes(P: int, N: int, dtype=torch.float32) -> int:
    return int(load().ring_reduce_scatter_workspace_bytes(P, N, _DTYPE[dtype]))


def ring_reduce_scatter_bidir_workspace_bytes(P: int, N: int, dtype=torch.float32) -> int:
    return int(load().ring_reduce_scatter_bidir_workspace_bytes(P, N, _DTYPE[dtype]))


def _rs_ex(fn, bufs, out, workspace, N, stream):
    bp, bs, dt = _slots(bufs, "bufs")
    op, os_, dt2 = _slots(out, "out")
    if dt != dt2 or bufs.size(0) != out.size(0):
        raise ValueError("bufs and out differ in dtype or rank count")
    N = bufs.size(1) if N is None else N
    wp, wb = _ws(workspace)
    with torch.cuda.device(bufs.device):
        _check(fn(bp, bs, op, os_, bufs.size(0), N, dt, wp, wb, _stream(stream, bufs.device)))
    return out


def ring_reduce_scatter_ex(bufs: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, N: int | None = None,
                           stream=None) -> torch.Tensor:
    """ring_reduce_scatter with a caller-owned workspace; ``bufs`` is clobbered."""
    return _rs_ex(load().ring_reduce_scatter_ex, bufs, out, workspace, N, stream)


def ring_reduce_scatter_bidir_ex(bufs: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
                                 N: int | None = None, stream=None) -> torch.Tensor:
    """ring_reduce_scatter_bidir with a caller-owned workspace; ``bufs`` is clobbered."""
    return _rs_ex(load().ring_reduce_scatter_bidir_ex, bufs, out, workspace, N, stream)


def ring_allreduce_fused(bufs: torch.Tensor, N: int | None = None, stream=None) -> torch.Tensor:
    """Single-pass all-reduce with the ring's result (bit-identical to ring_allreduce)."""
    fn = load().ring_allreduce_fused
    bp, bs, dt = _slots(bufs, "bufs")
    N = bufs.size(1) if N is None else N
    with torch.cuda.device(bufs.device):
        _check(fn(bp, bs, bufs.size(0), N, dt, _stream(stream, bufs.device)))
    return bufs


def ring_psum(bufs: torch.Tensor, n: int | None = None, stream=None) -> torch.Tensor:
    """Rotate-and-accumulate all-reduce (each rank folds in its own rotated order), in place."""
    fn = load().ring_psum
    bp, bs, dt = _slots(bufs, "bufs")
    n = bufs.size(1) if n is None else n
    with torch.cuda.device(bufs.device):
        _check(fn(bp, bs, bufs.size(0), n, dt, _stream(stream, bufs.device)))
    return bufs


def ring_allreduce_host(h_in: torch.Tensor, h_out: torch.Tensor, d_bufs: torch.Tensor, N: int | None = None,
                        stream=None) -> torch.Tensor:
    """All-reduce of host slots ``h_in`` (pinned CPU [P, L]) through device slots
    ``d_bufs``; the result lands in ``h_out`` once the stream completes."""
    if h_in.is_cuda or h_out.is_cuda:
        raise TypeError("h_in and h_out must be CPU tensors")
    if h_in.dim() != 2 or h_out.dim() != 2 or h_in.stride(1) != 1 or h_out.stride(1) != 1:
        raise ValueError("host slots must be 2-D [P, L] with contiguous rows")
    dp, ds, dt = _slots(d_bufs, "d_bufs")
    if _DTYPE.get(h_in.dtype) != dt or _DTYPE.get(h_out.dtype) != dt:
        raise TypeError("host and device slots differ in dtype")
    P = h_in.size(0)
    N = h_in.size(1) if N is None else N
    es = h_in.element_size()
    with torch.cuda.device(d_bufs.device):
        _check(load().ring_allreduce_host(h_in.data_ptr(), h_in.stride(0) * es, h_out.data_ptr(),
                                          h_out.stride(0) * es, dp, ds, P, N, dt, _stream(stream, d_bufs.device)))
    return h_out


def _ag_gemm_args(a_shards, a_gathered, B, C, b_layout):
    for name, t in (("a_shards", a_shards), ("a_gathered", a_gathered), ("B", B), ("C", C)):
        if not t.is_cuda or t.dtype != torch.bfloat16:
            raise TypeError(f"{name} must be a bf16 CUDA tensor")
    if a_shards.dim() != 3 or a_shards.stride(2) != 1 or a_shards.stride(1) != a_shards.size(2):
        raise ValueError("a_shards must be [P, M_r, K] with row-major shards")
    P, M_r, K = a_shards.shape
    N = B.size(0) if b_layout == RC_B_NK else B.size(1)
    if tuple(a_gathered.shape) != (P * M_r, K) or not a_gathered.is_contiguous():
        raise ValueError("a_gathered must be contiguous [P*M_r, K]")
    want_b = (N, K) if b_layout == RC_B_NK else (K, N)
    if tuple(B.shape) != want_b or not B.is_contiguous():
        raise ValueError(f"B must be contiguous {list(want_b)}")
    if tuple(C.shape) != (P * M_r, N) or not C.is_contiguous():
        raise ValueError("C must be contiguous [P*M_r, N]")
    return P, M_r, N, K


def ag_gemm(a_shards: torch.Tensor, a_gathered: torch.Tensor, B: torch.Tensor, C: torch.Tensor, rank: int,
            stream=None) -> torch.Tensor:
    """a_shards [P, M_r, K], a_gathered [P*M_r, K], B [N, K], C [P*M_r, N], all bf16:
    gathers the shards and computes C = A_g . B^T (fp32 accumulate, bf16 out)."""
    P, M_r, N, K = _ag_gemm_args(a_shards, a_gathered, B, C, RC_B_NK)
    with torch.cuda.device(a_shards.device):
        _check(load().ag_gemm(a_shards.data_ptr(), a_shards.stride(0) * 2, a_gathered.data_ptr(), B.data_ptr(),
                              C.data_ptr(), P, rank, M_r, N, K, _stream(stream, a_shards.device)))
    return C


def ag_gemm_kn(a_shards: torch.Tensor, a_gathered: torch.Tensor, B: torch.Tensor, C: torch.Tensor, rank: int,
               stream=None) -> torch.Tensor:
    """As ag_gemm with the weight stored [K, N] (the x @ W layout): C = A_g . B."""
    P, M_r, N, K = _ag_gemm_args(a_shards, a_gathered, B, C, RC_B_KN)
    with torch.cuda.device(a_shards.device):
        _check(load().ag_gemm_kn(a_shards.data_ptr(), a_shards.stride(0) * 2, a_gathered.data_ptr(), B.data_ptr(),
                                 C.data_ptr(), P, rank, M_r, N, K, _stream(stream, a_shards.device)))
    return C


def ag_gemm_workspace_bytes(P: int, M_r: int) -> int:
    return int(load().ag_gemm_workspace_bytes(P, M_r))


def ag_gemm_ex(a_shards: torch.Tensor, a_gathered: torch.Tensor, B: torch.Tensor, C: torch.Tensor, rank: int,
               workspace: torch.Tensor, b_layout: int = RC_B_NK, stream=None) -> torch.Tensor:
    """ag_gemm (b_layout RC_B_NK, B [N, K]) or ag_gemm_kn (RC_B_KN, B [K, N])
    with a caller-owned workspace (zeroed CUDA tensor of at least
    ag_gemm_workspace_bytes(P, M_r) bytes)."""
    P, M_r, N, K = _ag_gemm_args(a_shards, a_gathered, B, C, b_layout)
    wp, wb = _ws(workspace)
    with torch.cuda.device(a_shards.device):
        _check(load().ag_gemm_ex(a_shards.data_ptr(), a_shards.stride(0) * 2, a_gathered.data_ptr(), B.data_ptr(),
                                 b_layout, C.data_ptr(), P, rank, M_r, N, K, wp, wb, _stream(stream, a_shards.device)))
    return C


def gemm_rs_workspace_bytes(P: int, M: int, N: int, K: int) -> int:
    return int(load().gemm_rs_workspace_bytes(P, M, N, K))


def gemm_rs_ex(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor,
               stream=None) -> torch.Tensor:
    """gemm_rs with a caller-owned workspace (zeroed CUDA tensor of at least
    gemm_rs_workspace_bytes bytes)."""
    for name, t in (("A", A), ("B", B), ("out", out)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 3 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous 3-D bf16 CUDA tensor")
    P, M, K = A.shape
    N = B.size(1)
    if B.size(0) != P or B.size(2) != K or tuple(out.shape) != (P, M, N // P):
        raise ValueError("shapes must be A [P,M,K], B [P,N,K], out [P,M,N/P]")
    wp, wb = _ws(workspace)
    with torch.cuda.device(A.device):
        _check(load().gemm_rs_ex(A.data_ptr(), A.stride(0) * 2, B.data_ptr(), B.stride(0) * 2, out.data_ptr(),
                                 out.stride(0) * 2, P, M, N, K, wp, wb, _stream(stream, A.device)))
    return out


def gemm_rs(A: torch.Tensor, B: torch.Tensor, out: torch.Tensor, stream=None) -> torch.Tensor:
    """A [P, M, K], B [P, N, K], out [P, M, N/P], all bf16: out[r] = column chunk r
    of the ring reduce-scatter of the bf16 partial products A[q] . B[q]^T."""
    fn = load().gemm_rs
    for name, t in (("A", A), ("B", B), ("out", out)):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 3 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous 3-D bf16 CUDA tensor")
    P, M, K = A.shape
    N = B.size(1)
    if B.size(0) != P or B.size(2) != K or tuple(out.shape) != (P, M, N // P):
        raise ValueError("shapes must be A [P,M,K], B [P,N,K], out [P,M,N/P]")
    with torch.cuda.device(A.device):
        _check(fn(A.data_ptr(), A.stride(0) * 2, B.data_ptr(), B.stride(0) * 2, out.data_ptr(), out.stride(0) * 2,
                  P, M, N, K, _stream(stream, A.device)))
    return out


def ring_status(stream=None, device=None) -> int:
    """Waits for the stream and returns (and clears) the device status code."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        return load().ring_status(_stream(stream, dev))


def ring_status_ex(workspace: torch.Tensor, stream=None) -> int:
    """Waits for the stream and returns (and clears) the status recorded in a
    caller-owned workspace (the one given to :func:`ring_allreduce_ex`)."""
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    with torch.cuda.device(workspace.device):
        return load().ring_status_ex(workspace.data_ptr(), _stream(stream, workspace.device))


def ring_set_timeout_ms(ms: int) -> None:
    _check(load().ring_set_timeout_ms(ms))


def ring_set_slices(slices: int) -> None:
    _check(load().ring_set_slices(slices))


def ring_debug_skip_notify(rank: int, step: int) -> None:
    _check(load().ring_debug_skip_notify(rank, step))


def ag_gemm_debug_skip_piece(row: int) -> None:
    """The next ag_gemm launch never publishes the ready flag of the gather
    piece starting at A_g row `row`; -1 cancels (see include/ringcoll.h)."""
    _check(load().ag_gemm_debug_skip_piece(row))


def ring_finalize() -> None:
    _check(load().ring_finalize())


def ring_debug_set_trace(buf) -> None:
    """Step stamps of later ring launches go to ``buf`` (a CUDA uint64/int64
    tensor) -- see ring_debug_set_trace in include/ringcoll.h; None: off."""
    fn = load().ring_debug_set_trace
    if buf is None:
        _check(fn(None, 0))
    else:
        _check(fn(buf.data_ptr(), buf.numel() * buf.element_size()))


def ring_debug_l2_rate(dst: torch.Tensor, a: torch.Tensor, b: torch.Tensor | None = None, reps: int = 1,
                       stream=None) -> None:
    """The ring kernel's copy (b None) or f32 add (dst = a + b) loop, ``reps``
    times over the bytes of ``dst`` in one launch (see include/ringcoll.h)."""
    fn = load().ring_debug_l2_rate
    for name, t in (("dst", dst), ("a", a)) + ((("b", b),) if b is not None else ()):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous CUDA tensor")
    nb = dst.numel() * dst.element_size()
    if a.numel() * a.element_size() < nb or (b is not None and b.numel() * b.element_size() < nb):
        raise ValueError("inputs are shorter than dst")
    with torch.cuda.device(dst.device):
        _check(fn(dst.data_ptr(), a.data_ptr(), None if b is None else b.data_ptr(), nb, reps,
                  0 if b is None else 1, _stream(stream, dst.device)))


def ring_allreduce_noalloc(bufs: torch.Tensor, N: int | None = None, stream=None) -> torch.Tensor:
    """ring_allreduce without any device allocation by the library: the signal
    rows live in a fixed 256 KiB array compiled into the library (P <= 32).
    For callers that cannot let a library allocate device memory; see the
    declaration in include/ringcoll.h for set-up and ordering rules.  Device
    timeouts of these calls are read with :func:`ring_status`."""
    L = load()
    fn = L.ring_allreduce_noalloc
    bp, bs, dt = _slots(bufs, "bufs")
    N = bufs.size(1) if N is None else N
    with torch.cuda.device(bufs.device):
        _check(fn(bp, bs, bufs.size(0), N, dt, _stream(stream, bufs.device)))
    return bufs


# rc_attn_args of include/ringcoll.h: eight rc_heads, six pointers and sizes, eight ints, scale, reserved
_ATTN_ARGS = struct.Struct("@32Q6Q8ifi")
_NO_HEADS = (0, 0, 0, 0)
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _launch(fn, args: bytes, device, stream) -> None:
    """One call of a struct-argument entry point on `stream` (default: the current one)."""
    index = device.index
    if stream is None and index == torch._C._cuda_getDevice():
        rc = fn(args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            rc = fn(args, _stream(stream, device))
    if rc != RC_OK:
        _check(rc)


def _elsewhere(t, name: str, what: str) -> Exception:
    """Why `t` is not on the device of a call's queries."""
    if not t.is_cuda:
        return TypeError(f"{name} must be {what}")
    return ValueError(f"{name} must be on the device of q, not on GPU {t.get_device()}")


def _heads(t: torch.Tensor, name: str, gpu: int, shape=None):
    """gpu: the index of the queries' device (negative: not a GPU)."""
    if t.dtype is not _BF16 or gpu < 0:
        raise TypeError(f"{name} must be a bf16 CUDA tensor")
    if t.get_device() != gpu:
        raise _elsewhere(t, name, "a bf16 CUDA tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    st = t.stride()
    if len(st) != 4 or (st[3] != 1 and t.size(3) > 1):
        raise ValueError(f"{name} must be [P, T, H, D] with contiguous heads")
    return t.data_ptr(), 2 * st[0], 2 * st[1], 2 * st[2]


def _index(t, name: str, gpu: int, n: int) -> int:
    if t.dtype is not _I32 or t.shape != (n,) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 CUDA tensor of {n} elements")
    if t.get_device() != gpu:
        raise _elsewhere(t, name, "a CUDA tensor")
    return t.data_ptr()


def _space(workspace, gpu: int):
    ws = _ws(workspace)
    if workspace.get_device() != gpu:
        raise _elsewhere(workspace, "workspace", "a CUDA tensor")
    return ws


def _attn_sizes(P, B, Tq, Tk, Hq, Hkv, D, causal, scale):
    return P, B, Tq, Tk, Hq, Hkv, D, int(bool(causal)), D ** -0.5 if scale is None else scale, 0


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor | None,
             cu_q: torch.Tensor, cu_k: torch.Tensor, used_k: torch.Tensor | None = None, causal: bool = True,
             scale: float | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention of P ranks' heads over packed sequences, bf16.

    q, out [P, Tq, Hq, D]; k, v [P, Tk, Hkv, D]; lse float32 [P, Tq, Hq] or None.  Any
    strides with contiguous heads and 16-byte multiples, so q, k, v may be views of the
    fused activations that ag_gemm writes.  Sequence b holds queries cu_q[b]:cu_q[b+1]
    and keys cu_k[b]:cu_k[b+1], or the first used_k[b] of them (a cache); int32 on the
    device.  causal: the last query of a sequence sees all its keys, each earlier one a
    key less.  scale defaults to D ** -0.5.  workspace: as for the ``_ex`` calls."""
    P, Tq, Hq, D = qshape = q.shape
    _, Tk, Hkv, _ = k.shape
    kshape = (P, Tk, Hkv, D)
    B = cu_q.numel() - 1
    gpu = q.get_device()
    args = _ATTN_ARGS.pack(
        *_heads(q, "q", gpu), *_heads(k, "k", gpu, kshape), *_heads(v, "v", gpu, kshape), *_heads(out, "out", gpu, qshape),
        *_NO_HEADS * 4, 0 if lse is None else _lse(lse, gpu, P, Tq, Hq), _index(cu_q, "cu_q", gpu, B + 1),
        _index(cu_k, "cu_k", gpu, B + 1), 0 if used_k is None else _index(used_k, "used_k", gpu, B),
        *((0, 0) if workspace is None else _space(workspace, gpu)),
        *_attn_sizes(P, B, Tq, Tk, Hq, Hkv, D, causal, scale))
    _launch(load().attn_fwd, args, q.device, stream)
    return out


def _lse(lse, gpu, P, Tq, Hq):
    if lse.dtype is not _F32 or lse.shape != (P, Tq, Hq) or not lse.is_contiguous():
        raise TypeError(f"lse must be a contiguous float32 CUDA tensor of shape {[P, Tq, Hq]}")
    if lse.get_device() != gpu:
        raise _elsewhere(lse, "lse", "a CUDA tensor")
    return lse.data_ptr()


def attn_fwd_workspace_bytes(P: int, B: int, Tq: int, Tk: int, Hq: int, Hkv: int, D: int) -> int:
    args = _ATTN_ARGS.pack(*(0,) * 38, *_attn_sizes(P, B, Tq, Tk, Hq, Hkv, D, True, None))
    return int(load().attn_fwd_workspace_bytes(args))


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor, lse: torch.Tensor,
             dout: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, cu_q: torch.Tensor,
             cu_k: torch.Tensor, used_k: torch.Tensor | None = None, causal: bool = True, scale: float | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Gradients of :func:`attn_fwd` (``out`` and ``lse`` are its results): writes dq
    [P, Tq, Hq, D] and dk, dv [P, Tk, Hkv, D], which may be views of one fused gradient
    buffer.  The other arguments are those of the forward call."""
    P, Tq, Hq, D = qshape = q.shape
    _, Tk, Hkv, _ = k.shape
    kshape = (P, Tk, Hkv, D)
    B = cu_q.numel() - 1
    gpu = q.get_device()
    args = _ATTN_ARGS.pack(
        *_heads(q, "q", gpu), *_heads(k, "k", gpu, kshape), *_heads(v, "v", gpu, kshape), *_heads(out, "out", gpu, qshape),
        *_heads(dout, "dout", gpu, qshape), *_heads(dq, "dq", gpu, qshape), *_heads(dk, "dk", gpu, kshape),
        *_heads(dv, "dv", gpu, kshape), _lse(lse, gpu, P, Tq, Hq), _index(cu_q, "cu_q", gpu, B + 1),
        _index(cu_k, "cu_k", gpu, B + 1), 0 if used_k is None else _index(used_k, "used_k", gpu, B),
        *((0, 0) if workspace is None else _space(workspace, gpu)),
        *_attn_sizes(P, B, Tq, Tk, Hq, Hkv, D, causal, scale))
    _launch(load().attn_bwd, args, q.device, stream)
    return dq, dk, dv


def attn_bwd_workspace_bytes(P: int, B: int, Tq: int, Tk: int, Hq: int, Hkv: int, D: int) -> int:
    args = _ATTN_ARGS.pack(*(0,) * 38, *_attn_sizes(P, B, Tq, Tk, Hq, Hkv, D, True, None))
    return int(load().attn_bwd_workspace_bytes(args))


# rc_qk_norm_args of include/ringcoll.h: six rc_heads, nine pointers and sizes, seven ints, eps
_QK_NORM_ARGS = struct.Struct("@24Q9Q7if")


def _f32(t, name: str, gpu: int, shape) -> int:
    if t.dtype is not _F32 or t.shape != shape or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 CUDA tensor of shape {list(shape)}")
    if t.get_device() != gpu:
        raise _elsewhere(t, name, "a CUDA tensor")
    return t.data_ptr()


def _qk_norm(q, k, gamma_q, gamma_k, cos, sin, pos, layout, eps, q_out, k_out, grads, workspace):
    P, T, Hq, D = qshape = q.shape
    kshape = (P, T, k.shape[2], D)
    table = (cos.shape[0], D // 2)
    gpu = q.get_device()
    heads = _NO_HEADS * 2 if grads is None else _heads(grads[0], "dq", gpu, qshape) + _heads(grads[1], "dk", gpu, kshape)
    dg = (0, 0) if grads is None else (_f32(grads[2], "dgamma_q", gpu, (P, D)), _f32(grads[3], "dgamma_k", gpu, (P, D)))
    names = ("q_out", "k_out") if grads is None else ("dq_out", "dk_out")
    return _QK_NORM_ARGS.pack(
        *_heads(q, "q", gpu), *_heads(k, "k", gpu, kshape), *_heads(q_out, names[0], gpu, qshape),
        *_heads(k_out, names[1], gpu, kshape), *heads, _f32(gamma_q, "gamma_q", gpu, (D,)),
        _f32(gamma_k, "gamma_k", gpu, (D,)), _f32(cos, "cos", gpu, table), _f32(sin, "sin", gpu, table),
        _index(pos, "pos", gpu, T), *dg, *((0, 0) if workspace is None else _space(workspace, gpu)),
        P, T, Hq, kshape[2], D, table[0], layout, eps)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, gamma_q: torch.Tensor, gamma_k: torch.Tensor, cos: torch.Tensor,
                 sin: torch.Tensor, pos: torch.Tensor, q_out: torch.Tensor, k_out: torch.Tensor,
                 layout: int = RC_ROPE_HALF, eps: float = 1e-6, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """RMS norm of every query and key head with weights gamma [D], then the rotation by
    the angles whose cosines and sines are rows pos[t] of cos, sin (float32 [npos, D/2]).
    q, q_out [P, T, Hq, D], k, k_out [P, T, Hkv, D] bf16, any strides as for attn_fwd; in
    place when q_out is q and k_out is k."""
    args = _qk_norm(q, k, gamma_q, gamma_k, cos, sin, pos, layout, eps, q_out, k_out, None, None)
    _launch(load().qk_norm_rope, args, q.device, stream)
    return q_out, k_out


def qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, gamma_q: torch.Tensor, gamma_k: torch.Tensor,
                     cos: torch.Tensor, sin: torch.Tensor, pos: torch.Tensor, dq_out: torch.Tensor,
                     dk_out: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dgamma_q: torch.Tensor,
                     dgamma_k: torch.Tensor, layout: int = RC_ROPE_HALF, eps: float = 1e-6,
                     workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of :func:`qk_norm_rope` from its inputs and the gradients dq_out, dk_out of
    its outputs: writes dq, dk (bf16; may be dq_out, dk_out) and each rank's own sums of
    the weight gradients, dgamma_q and dgamma_k (float32 [P, D]).  workspace: a CUDA tensor
    of at least qk_norm_rope_bwd_workspace_bytes bytes, which other calls may use too in
    stream order; None takes the library's own."""
    args = _qk_norm(q, k, gamma_q, gamma_k, cos, sin, pos, layout, eps, dq_out, dk_out, (dq, dk, dgamma_q, dgamma_k),
                    workspace)
    _launch(load().qk_norm_rope_bwd, args, q.device, stream)
    return dq, dk


def qk_norm_rope_bwd_workspace_bytes(P: int, T: int, Hq: int, Hkv: int, D: int) -> int:
    args = _QK_NORM_ARGS.pack(*(0,) * 33, P, T, Hq, Hkv, D, 1, RC_ROPE_HALF, 0.0)
    return int(load().qk_norm_rope_bwd_workspace_bytes(args))
