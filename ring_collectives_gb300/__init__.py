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
    "act8_empty", "act8_pack", "act8_unpack", "block_norm", "block_norm_bwd", "block_norm_bwd_workspace_bytes",
    "glu", "glu_bwd", "RC_GLU_SILU", "RC_GLU_GELU", "gemm_wgrad", "gemm_wgrad_workspace_bytes",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libringcoll.so")

RC_OK, RC_ERR_INVALID, RC_ERR_CUDA, RC_ERR_TIMEOUT, RC_ERR_UNSUPPORTED, RC_ERR_NOMEM = range(6)
RC_ROPE_HALF, RC_ROPE_PAIRS = 0, 1   # rotated pairs (i, i + D/2) or (2i, 2i + 1)
RC_GLU_SILU, RC_GLU_GELU = 0, 1      # glu activations: x s(x), or the tanh form of gelu
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
    "act8_pack": ([ctypes.c_char_p, _vp], _i),
    "act8_unpack": ([ctypes.c_char_p, _vp], _i),
    "block_norm": ([ctypes.c_char_p, _vp], _i),
    "block_norm_bwd": ([ctypes.c_char_p, _vp], _i),
    "block_norm_bwd_workspace_bytes": ([ctypes.c_char_p], _sz),
    "glu": ([ctypes.c_char_p, _vp], _i),
    "glu_bwd": ([ctypes.c_char_p, _vp], _i),
    "gemm_wgrad": ([ctypes.c_char_p, _vp], _i),
    "gemm_wgrad_workspace_bytes": ([ctypes.c_char_p], _sz),
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


# rc_act8_args of include/ringcoll.h: three rc_rows, four ints; rc_block_norm_args: fourteen rc_rows, eight pointers and
# sizes, five ints, alpha, eps, an int; rc_glu_args: twelve rc_rows, six ints; rc_wgrad_args: four rc_rows, workspace
# and its size, eight ints
_ACT8_ARGS = struct.Struct("@9Q4i")
_BLOCK_NORM_ARGS = struct.Struct("@42Q8Q5iffi")
_GLU_ARGS = struct.Struct("@36Q6i")
_WGRAD_ARGS = struct.Struct("@14Q8i")
_NO_ROWS, _NO_ACT8 = (0,) * 3, (0,) * 6
_I8, _U8 = torch.int8, torch.uint8


def _here(t, name: str, kind: str, gpu: int) -> None:
    """`t` has to be a CUDA tensor on the device of the call's rows; gpu: its index (negative: not a GPU)."""
    if gpu < 0 or not t.is_cuda:
        raise TypeError(f"{name} must be a {kind} CUDA tensor")
    if t.get_device() != gpu:
        raise ValueError(f"{name} must be on GPU {gpu} with the other tensors of the call, not on GPU {t.get_device()}")


def _rows(t, name: str, gpu: int, shape, dtype=_BF16, kind="bf16", size=2):
    """Address and strides in bytes of rows [P, T, N] of elements of `size` bytes."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be a {kind} CUDA tensor")
    if gpu < 0 or t.get_device() != gpu:
        _here(t, name, kind, gpu)
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    slot, row, channel = t.stride()
    if channel != 1 and shape[2] > 1:
        raise ValueError(f"{name} must be [P, T, N] with contiguous rows")
    return t.data_ptr(), size * slot, size * row


def _act8(x8, name: str, gpu: int, shape):
    q, e = x8
    P, T, N = shape
    return (*_rows(q, name + "[0]", gpu, shape, _I8, "int8", 1), *_rows(e, name + "[1]", gpu, (P, T, -(-N // 32)), _U8, "uint8", 1))


def act8_empty(shape, device=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Room for the 8-bit form of an activation [P, T, N]: int8 [P, T, N] and uint8 [P, T, ceil(N / 32)]."""
    P, T, N = shape
    device = torch.device("cuda") if device is None else device
    return torch.empty((P, T, N), dtype=_I8, device=device), torch.empty((P, T, -(-N // 32)), dtype=_U8, device=device)


def _act8_call(fn, x, x8, stream):
    P, T, N = shape = x.shape
    gpu = x.get_device()
    if x8 is None:
        raise TypeError("x8 must be a pair of CUDA tensors")
    _launch(fn, _ACT8_ARGS.pack(*_rows(x, "x", gpu, shape), *(_NO_ACT8 if x8 is None else _act8(x8, "x8", gpu, shape)), P, T, N, 0), x.device, stream)


def act8_pack(x: torch.Tensor, x8, stream=None):
    """The 8-bit form of a bf16 activation x [P, T, N] (any strides of 16-byte multiples with
    contiguous rows), a pair x8 as act8_empty makes: signed bytes q and, for every 32 channels
    of a row, the biased exponent e of the least power of two that keeps them within 127:
    x is close to q * 2 ** (e - 127).  e = 255 marks a group that holds an infinity or a NaN."""
    _act8_call(load().act8_pack, x, x8, stream)
    return x8


def act8_unpack(x8, x: torch.Tensor, stream=None) -> torch.Tensor:
    """The bf16 values [P, T, N] that the pair x8 stands for, exactly."""
    _act8_call(load().act8_unpack, x, x8, stream)
    return x


def _weights(t, name: str, gpu: int, shape) -> int:
    if t.get_device() != gpu:
        _here(t, name, "float32", gpu)
    return _f32(t, name, gpu, shape)


def _room(workspace, gpu: int):
    if workspace is None:
        return 0, 0
    ws = _ws(workspace)
    _here(workspace, "workspace", "contiguous", gpu)
    return ws


def _cols(t, shape) -> bool:
    """Whether a block's output or its gradient lies in column chunks [P, P * T, N / P]."""
    P, T, N = shape
    return P > 1 and N % P == 0 and t.shape == (P, P * T, N // P)


def _side(t, name: str, gpu: int, shape):
    P, T, N = shape
    cols = _cols(t, shape)
    return _rows(t, name, gpu, (P, P * T, N // P) if cols else shape), int(cols)


def block_norm(y: torch.Tensor, res: torch.Tensor, h: torch.Tensor, z: torch.Tensor | None = None,
               gamma_post: torch.Tensor | None = None, gate: torch.Tensor | None = None,
               gamma_pre: torch.Tensor | None = None, alpha: float = 1.0, eps: float = 1e-6, y8=None, res8=None, z8=None,
               stream=None) -> tuple[torch.Tensor, torch.Tensor | None]:
    """What lies between a block's last matmul and the next one's first, in one pass over rows:

        u = rms_norm(y) * gamma_post   (u = y without gamma_post)
        h = res + alpha * gate * u
        z = rms_norm(h) * gamma_pre    (z and gamma_pre: both or neither)

    res, h, z [P, T, N] bf16, the row shards that ag_gemm gathers; y alike or as gemm_rs leaves
    it, [P, P * T, N / P].  Weights float32 [N].  h may be res.  y8, res8, z8: pairs as from
    act8_empty that receive the 8-bit forms of y, res and z."""
    P, T, N = shape = res.shape
    gpu = res.get_device()
    rows, cols = _side(y, "y", gpu, shape)
    args = _BLOCK_NORM_ARGS.pack(
        *rows, *_rows(res, "res", gpu, shape), *_rows(h, "h", gpu, shape), *(_NO_ROWS if z is None else _rows(z, "z", gpu, shape)),
        *_NO_ROWS * 4, *(_NO_ACT8 if y8 is None else _act8(y8, "y8", gpu, shape)),
        *(_NO_ACT8 if res8 is None else _act8(res8, "res8", gpu, shape)), *(_NO_ACT8 if z8 is None else _act8(z8, "z8", gpu, shape)),
        0 if gamma_post is None else _weights(gamma_post, "gamma_post", gpu, (N,)),
        0 if gate is None else _weights(gate, "gate", gpu, (N,)), 0 if gamma_pre is None else _weights(gamma_pre, "gamma_pre", gpu, (N,)),
        0, 0, 0, 0, 0, P, T, N, cols, 0, alpha, eps, 0)
    _launch(load().block_norm, args, res.device, stream)
    return h, z


def block_norm_bwd(y, res, dh: torch.Tensor | None, dz: torch.Tensor | None, dy: torch.Tensor, dres: torch.Tensor,
                   dgamma_post: torch.Tensor | None = None, dgate: torch.Tensor | None = None,
                   dgamma_pre: torch.Tensor | None = None, gamma_post: torch.Tensor | None = None,
                   gate: torch.Tensor | None = None, gamma_pre: torch.Tensor | None = None, alpha: float = 1.0,
                   eps: float = 1e-6, workspace: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of :func:`block_norm`.  y and res are its inputs, or both are the pairs y8 and
    res8 that it left (the gradient is then that at their values).  dh (or None) and dz are the
    gradients of h and z (dz in either layout of y: gemm_rs may have left it); writes dy (likewise) and dres, and where the weight is
    given each rank's own sums dgamma_post, dgate, dgamma_pre (float32 [P, N]).  dres and dy
    may each be dh or dz.  workspace: a CUDA tensor of at least block_norm_bwd_workspace_bytes bytes, which
    other calls may use too in stream order; None takes the library's own.  Above 8192 channels a wait that
    runs out is reported by ring_status(), with a workspace too."""
    P, T, N = shape = dres.shape
    gpu = dres.get_device()
    held = isinstance(y, (tuple, list))
    if held != isinstance(res, (tuple, list)):
        raise TypeError("y and res are both tensors or both 8-bit pairs")
    rows, cols = (_NO_ROWS, 0) if held else _side(y, "y", gpu, shape)
    drows, dcols = _side(dy, "dy", gpu, shape)
    zrows, zcols = (_NO_ROWS, 0) if dz is None else _side(dz, "dz", gpu, shape)
    args = _BLOCK_NORM_ARGS.pack(
        *rows, *(_NO_ROWS if held else _rows(res, "res", gpu, shape)), *_NO_ROWS * 2,
        *(_NO_ROWS if dh is None else _rows(dh, "dh", gpu, shape)), *zrows,
        *drows, *_rows(dres, "dres", gpu, shape), *(_act8(y, "y", gpu, shape) if held else _NO_ACT8),
        *(_act8(res, "res", gpu, shape) if held else _NO_ACT8), *_NO_ACT8,
        0 if gamma_post is None else _weights(gamma_post, "gamma_post", gpu, (N,)),
        0 if gate is None else _weights(gate, "gate", gpu, (N,)), 0 if gamma_pre is None else _weights(gamma_pre, "gamma_pre", gpu, (N,)),
        0 if dgamma_post is None else _weights(dgamma_post, "dgamma_post", gpu, (P, N)),
        0 if dgate is None else _weights(dgate, "dgate", gpu, (P, N)),
        0 if dgamma_pre is None else _weights(dgamma_pre, "dgamma_pre", gpu, (P, N)),
        *_room(workspace, gpu), P, T, N, cols, dcols, alpha, eps, zcols)
    _launch(load().block_norm_bwd, args, dres.device, stream)
    return dy, dres


def block_norm_bwd_workspace_bytes(P: int, T: int, N: int, post: bool = True, gate: bool = True, pre: bool = True,
                                   held: bool = False) -> int:
    """Bytes of workspace that block_norm_bwd needs with these weights given (held: from 8-bit pairs)."""
    args = _BLOCK_NORM_ARGS.pack(*(0,) * 24, int(held), *(0,) * 17, int(post), int(gate), int(pre), *(0,) * 5, P, T, N, 0, 0, 1.0, 0.0, 0)
    return int(load().block_norm_bwd_workspace_bytes(args))


def glu(a: torch.Tensor, b: torch.Tensor, h: torch.Tensor, act: int = RC_GLU_SILU, a8=None, b8=None, h8=None,
        stream=None) -> torch.Tensor:
    """h = act(a) * b, the gated activation between an MLP's matmuls; bf16 [P, T, N], a and b
    commonly the halves of one fused ag_gemm result.  act: RC_GLU_SILU or RC_GLU_GELU (tanh
    form).  a8, b8, h8: pairs as from act8_empty that receive the 8-bit forms.  h may be a or b."""
    P, T, N = shape = a.shape
    gpu = a.get_device()
    args = _GLU_ARGS.pack(*_rows(a, "a", gpu, shape), *_rows(b, "b", gpu, shape), *_rows(h, "h", gpu, shape), *_NO_ROWS * 3,
                          *(_NO_ACT8 if a8 is None else _act8(a8, "a8", gpu, shape)), *(_NO_ACT8 if b8 is None else _act8(b8, "b8", gpu, shape)),
                          *(_NO_ACT8 if h8 is None else _act8(h8, "h8", gpu, shape)),
                          P, T, N, act, 0, 0)
    _launch(load().glu, args, a.device, stream)
    return h


def glu_bwd(a, b, dh: torch.Tensor, da: torch.Tensor, db: torch.Tensor, h: torch.Tensor | None = None,
            act: int = RC_GLU_SILU, h8=None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of :func:`glu`, from a and b or from the pairs a8 and b8 that it left: writes
    da = dh b act'(a) and db = dh act(a), and where given h = act(a) b again and its 8-bit form
    h8.  da and db may each be a, b or dh."""
    P, T, N = shape = dh.shape
    gpu = dh.get_device()
    held = isinstance(a, (tuple, list))
    if held != isinstance(b, (tuple, list)):
        raise TypeError("a and b are both tensors or both 8-bit pairs")
    args = _GLU_ARGS.pack(
        *(_NO_ROWS * 2 if held else _rows(a, "a", gpu, shape) + _rows(b, "b", gpu, shape)),
        *(_NO_ROWS if h is None else _rows(h, "h", gpu, shape)), *_rows(dh, "dh", gpu, shape), *_rows(da, "da", gpu, shape),
        *_rows(db, "db", gpu, shape), *(_act8(a, "a", gpu, shape) + _act8(b, "b", gpu, shape) if held else _NO_ACT8 * 2),
        *(_NO_ACT8 if h8 is None else _act8(h8, "h8", gpu, shape)), P, T, N, act, 0, 0)
    _launch(load().glu_bwd, args, dh.device, stream)
    return da, db


def gemm_wgrad(dy: torch.Tensor, x8, dw: torch.Tensor, accumulate: bool = False, workspace: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """The weight gradient of either collective matmul from an activation held in 8 bits:
    dw[r] = dy[r].T @ x[r] for every rank, summed in binary32 (accumulate: added to dw).
    dy [P, T, N] bf16, x8 the pair of an activation [P, T, K], dw [P, N, K] bf16 or float32.
    What all ranks share (the gathered activation of ag_gemm, the gradient of gemm_rs's
    result) is given with slot stride 0, as from ``expand``.  workspace: a zeroed CUDA tensor of
    at least gemm_wgrad_workspace_bytes bytes, as for the ``_ex`` calls; None: the library's own."""
    P, T, N = dy.shape
    K = x8[0].shape[2]
    gpu = dw.get_device()
    f32 = dw.dtype is _F32
    args = _WGRAD_ARGS.pack(*_rows(dy, "dy", gpu, (P, T, N)), *_act8(x8, "x8", gpu, (P, T, K)),
                            *_rows(dw, "dw", gpu, (P, N, K), _F32 if f32 else _BF16, "bf16 or float32", 4 if f32 else 2), *_room(workspace, gpu),
                            P, T, N, K, _DTYPE[dw.dtype], int(bool(accumulate)), 0, 0)
    _launch(load().gemm_wgrad, args, dw.device, stream)
    return dw


def gemm_wgrad_workspace_bytes(P: int, T: int, N: int, K: int) -> int:
    return int(load().gemm_wgrad_workspace_bytes(_WGRAD_ARGS.pack(*(0,) * 14, P, T, N, K, 1, 0, 0, 0)))
