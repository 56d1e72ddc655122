"""Python binding of the block operators' C ABI (include/dyt_block.h): layer
norm and attention, argument marshalling only.

Every computation runs in the HIP library ``libdyt_block.so``; like the DyT
binding this module checks tensors, allocates outputs and workspace with
PyTorch and passes device pointers and torch's current HIP stream. There is
no CPU fallback: importing this module fails if the library is missing.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import _lib
from ._lib import DYT_OK, DytError, _keep_alive_on
from .build import BLOCK_DEPENDS, BLOCK_LIB_PATH, source_hash

BLOCK_ABI_VERSION = 1
DYT_ATTN_MAX_D = 128
DYT_ATTN_MAX_BUCKETS = 128
DYT_ATTN_MAX_DISTANCE = 1024

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float
_size = ctypes.c_size_t

SIGNATURES = {
    "dyt_block_abi_version": (_int, []),
    "dyt_block_build_id": (ctypes.c_char_p, []),
    "dyt_ln_forward": (_int, [_vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _i64, _f32, _int, _int, _vp]),
    "dyt_ln_forward_residual": (_int, [_vp] * 8 + [_i64, _i64, _f32, _int, _int, _vp]),
    "dyt_ln_backward_workspace_size": (_size, [_i64, _i64, _int, _int]),
    "dyt_ln_backward": (_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _size, _i64, _i64,
                               _int, _int, _vp]),
    "dyt_ln_backward_residual": (_int, [_vp] * 10 + [_size, _i64, _i64, _int, _int, _vp]),
    "dyt_attn_forward_workspace_size": (_size, [_vp]),
    "dyt_attn_backward_workspace_size": (_size, [_vp]),
    "dyt_attn_forward": (_int, [_vp] * 7 + [_size, _vp]),
    "dyt_attn_backward": (_int, [_vp] * 12 + [_size, _vp]),
    "dyt_attn_bucket_borders": (_int, [_int, _int, _int, _vp]),
}


def _load(path: str = BLOCK_LIB_PATH, any_sources: bool = False) -> ctypes.CDLL:
    """Load the block operators' library, built from the current sources."""
    if not os.path.exists(path):
        raise ImportError(
            f"block operators' HIP library not found at {path}; build it first "
            "(python bwd_dyt_forward_amd/build.py, or __graft_entry__.build())")
    lib = ctypes.CDLL(path, mode=ctypes.RTLD_LOCAL)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    found = lib.dyt_block_abi_version()
    if found != BLOCK_ABI_VERSION:
        raise ImportError(f"{path} has ABI version {found}, this binding expects {BLOCK_ABI_VERSION}; "
                          "rebuild the library")
    built, want = lib.dyt_block_build_id().decode(), source_hash((), BLOCK_DEPENDS)
    if built != want and not any_sources:
        raise ImportError(f"{path} was built from other sources (build id {built}, sources "
                          f"{want}); rebuild it (python bwd_dyt_forward_amd/build.py)")
    return lib


block_lib = _load()
BLOCK_LIB_FILE = BLOCK_LIB_PATH
_CODES = _lib._TORCH_TO_CODE


def _check(fn: str, status: int) -> None:
    if status != DYT_OK:
        raise DytError(fn, status, _lib.lib.dyt_status_string(status).decode())


def _code(name: str, t: torch.Tensor) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {t.dtype} of {name}")
    return code


def _stream_for(t: torch.Tensor, stream) -> int:
    """The raw HIP stream to launch on: the given one, or torch's current one.
    Kernels launch on the current device, so the tensors have to be there."""
    index = t.device.index
    if index != torch._C._cuda_getDevice():
        raise ValueError("the tensors must be on the current device (torch.cuda.device)")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return _lib._stream(stream)


def _empty(like: torch.Tensor, shape) -> torch.Tensor:
    """A contiguous tensor of like's type (empty_like is the cheapest call)."""
    if like.is_contiguous():
        return torch.empty_like(like)
    return torch.empty(shape, dtype=like.dtype, device=like.device)


def _on_device(name: str, t, like: torch.Tensor) -> None:
    if not isinstance(t, torch.Tensor) or t.device != like.device:
        raise ValueError(f"{name} must be a tensor on {like.device}")


# --------------------------------------------------------------- layer norm
def _check_rows(name: str, t: torch.Tensor, like: torch.Tensor | None = None, dense: bool = False) -> int:
    """A 2-D [M, N] device tensor with unit column stride (like `like`);
    returns its row pitch in elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D [M, N] tensor")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must match {tuple(like.shape)} {like.dtype} on {like.device}")
    M, N = t.shape
    sm, sn = t.stride()
    pitch = sm if M > 1 else N
    if (N > 1 and sn != 1) or pitch < N or (dense and pitch != N):
        raise ValueError(f"{name} must " + ("be contiguous" if dense else
                                            "have unit column stride and row stride >= N"))
    return pitch


def _check_vectors(like: torch.Tensor, N: int, **vecs) -> int:
    """Parameter vectors: contiguous, N elements, one dtype, on like's device."""
    dt = None
    for name, t in vecs.items():
        _on_device(name, t, like)
        if t.numel() != N or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with {N} elements")
        if dt is None:
            dt = t.dtype
        elif t.dtype != dt:
            raise ValueError(f"{' and '.join(vecs)} must share one dtype")
    return _code(name, t)


def _check_stats(like: torch.Tensor, M: int, **vecs) -> None:
    for name, t in vecs.items():
        _on_device(name, t, like)
        if t.dtype != torch.float32 or t.numel() != M or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous float32 with {M} elements")


def dyt_ln_forward(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float = 1e-5,
                   y: torch.Tensor | None = None, mean: torch.Tensor | None = None,
                   rstd: torch.Tensor | None = None, stream=None):
    """Layer norm of the rows of x [M, N]: returns (y, mean, rstd), the
    statistics float32 [M]. x and y may be row-strided (unit column stride)."""
    ldx = _check_rows("x", x)
    M, N = x.shape
    pc = _check_vectors(x, N, gamma=gamma, beta=beta)
    xc = _code("x", x)
    s = _stream_for(x, stream)
    made = (y is None, mean is None, rstd is None)
    if y is None:
        y = _empty(x, (M, N))
    ldy = N if made[0] else _check_rows("y", y, x)
    if mean is None:
        mean = torch.empty(M, dtype=torch.float32, device=x.device)
    if rstd is None:
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    if not (made[1] and made[2]):
        _check_stats(x, M, mean=mean, rstd=rstd)
    _check("dyt_ln_forward", block_lib.dyt_ln_forward(
        x.data_ptr(), ldx, gamma.data_ptr(), beta.data_ptr(), y.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr(),
        M, N, eps, xc, pc, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((y, mean, rstd), made) if m))
    return y, mean, rstd


def dyt_ln_forward_residual(x: torch.Tensor, r: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor,
                            eps: float = 1e-5, h: torch.Tensor | None = None, y: torch.Tensor | None = None,
                            mean: torch.Tensor | None = None, rstd: torch.Tensor | None = None, stream=None):
    """h = x + r (rounded to x's dtype) and its layer norm: (h, y, mean, rstd)."""
    _check_rows("x", x, dense=True)
    _check_rows("r", r, x, dense=True)
    M, N = x.shape
    pc = _check_vectors(x, N, gamma=gamma, beta=beta)
    xc = _code("x", x)
    s = _stream_for(x, stream)
    made = (h is None, y is None, mean is None, rstd is None)
    if h is None:
        h = _empty(x, (M, N))
    else:
        _check_rows("h", h, x, dense=True)
    if y is None:
        y = _empty(x, (M, N))
    else:
        _check_rows("y", y, x, dense=True)
    if mean is None:
        mean = torch.empty(M, dtype=torch.float32, device=x.device)
    if rstd is None:
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    if not (made[2] and made[3]):
        _check_stats(x, M, mean=mean, rstd=rstd)
    _check("dyt_ln_forward_residual", block_lib.dyt_ln_forward_residual(
        x.data_ptr(), r.data_ptr(), gamma.data_ptr(), beta.data_ptr(), h.data_ptr(), y.data_ptr(), mean.data_ptr(),
        rstd.data_ptr(), M, N, eps, xc, pc, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((h, y, mean, rstd), made) if m))
    return h, y, mean, rstd


def dyt_ln_backward_workspace_size(M: int, N: int, x_dtype, param_dtype) -> int:
    return int(block_lib.dyt_ln_backward_workspace_size(int(M), int(N), _lib._code(x_dtype), _lib._code(param_dtype)))


def _ln_backward(x, dy, dres, mean, rstd, gamma, dx, dgamma, dbeta, workspace, stream):
    res = dres is not None
    xname = "h" if res else "x"
    ldx = _check_rows(xname, x, dense=res)
    lddy = _check_rows("dy", dy, x, dense=res)
    if res:
        _check_rows("dres", dres, x, dense=True)
    M, N = x.shape
    pc = _check_vectors(x, N, gamma=gamma)
    _check_stats(x, M, mean=mean, rstd=rstd)
    xc = _code(xname, x)
    s = _stream_for(x, stream)
    dev = x.device
    made = (dx is None, dgamma is None, dbeta is None, workspace is None)
    if dx is None:
        dx = _empty(x, (M, N))
        lddx = N
    else:
        lddx = _check_rows("dx", dx, x, dense=res)
    if dgamma is None:
        dgamma = torch.empty(N, dtype=gamma.dtype, device=dev)
    if dbeta is None:
        dbeta = torch.empty(N, dtype=gamma.dtype, device=dev)
    if not (made[1] and made[2]):
        _check_vectors(x, N, gamma=gamma, dgamma=dgamma, dbeta=dbeta)
    if workspace is None:
        need = block_lib.dyt_ln_backward_workspace_size(M, N, xc, pc)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _on_device("workspace", workspace, x)
        need = workspace.numel() * workspace.element_size()
    if res:
        _check("dyt_ln_backward_residual", block_lib.dyt_ln_backward_residual(
            x.data_ptr(), dy.data_ptr(), dres.data_ptr(), mean.data_ptr(), rstd.data_ptr(), gamma.data_ptr(),
            dx.data_ptr(), dgamma.data_ptr(), dbeta.data_ptr(), workspace.data_ptr(), need, M, N, xc, pc, s))
    else:
        _check("dyt_ln_backward", block_lib.dyt_ln_backward(
            x.data_ptr(), ldx, dy.data_ptr(), lddy, mean.data_ptr(), rstd.data_ptr(), gamma.data_ptr(),
            dx.data_ptr(), lddx, dgamma.data_ptr(), dbeta.data_ptr(), workspace.data_ptr(), need, M, N, xc, pc, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((dx, dgamma, dbeta, workspace), made) if m))
    return dx, dgamma, dbeta


def dyt_ln_backward(x: torch.Tensor, dy: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                    gamma: torch.Tensor, dx: torch.Tensor | None = None, dgamma: torch.Tensor | None = None,
                    dbeta: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Layer norm's backward at x with the forward's statistics: (dx, dgamma,
    dbeta). x, dy and dx may be row-strided (unit column stride)."""
    return _ln_backward(x, dy, None, mean, rstd, gamma, dx, dgamma, dbeta, workspace, stream)


def dyt_ln_backward_residual(h: torch.Tensor, dy: torch.Tensor, dres: torch.Tensor, mean: torch.Tensor,
                             rstd: torch.Tensor, gamma: torch.Tensor, dx: torch.Tensor | None = None,
                             dgamma: torch.Tensor | None = None, dbeta: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None):
    """dx = dres + (layer norm's backward of dy at h): (dx, dgamma, dbeta);
    dx is the gradient of both x and r."""
    if not isinstance(dres, torch.Tensor):
        raise ValueError("dres must be a device tensor")
    return _ln_backward(h, dy, dres, mean, rstd, gamma, dx, dgamma, dbeta, workspace, stream)


# ---------------------------------------------------------------- attention
# struct dyt_attn_desc: 6 sizes, 8 x 3 strides, 3 pointers, 6 int32, scale, reserved
_DESC = struct.Struct("=30q3Q6ifi")


def _check_heads(name: str, t: torch.Tensor, like: torch.Tensor | None, shape=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1):
        raise ValueError(f"{name} must be [B, S, H, D] with unit stride along D")
    if like is not None and (t.dtype != like.dtype or t.device != like.device):
        raise ValueError(f"{name} must have {like.dtype} on {like.device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")


def _check_list(name: str, t: torch.Tensor | None, like: torch.Tensor, B: int) -> int:
    if t is None:
        return 0
    _on_device(name, t, like)
    if t.dtype != torch.int32 or t.shape != (B,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of {B} elements")
    return t.data_ptr()


def _attn_problem(q, k, v, causal, scale, seqlens_k, q_start, table, max_distance, bidirectional):
    """Checks q, k, v and the options; returns the descriptor's parts around
    the strides and B, Sq, Hq, D."""
    _check_heads("q", q, None)
    code = _code("q", q)
    _check_heads("k", k, q)
    B, Sq, Hq, D = q.shape
    Bk, Sk, Hkv, Dk = k.shape
    _check_heads("v", v, q, k.shape)
    if Bk != B or Dk != D:
        raise ValueError("k and v must have q's batch and head dimension")
    if Hkv < 1 or Hq % Hkv:
        raise ValueError("q's heads must be a multiple of k's")
    if not 1 <= D <= DYT_ATTN_MAX_D:
        raise ValueError(f"the head dimension must be 1 to {DYT_ATTN_MAX_D}, got {D}")
    if scale is None:
        scale = D ** -0.5
    elif not 0.0 < scale < float("inf"):
        raise ValueError("scale must be positive and finite")
    tp, tc, buckets = 0, 0, 0
    if table is not None:
        _on_device("table", table, q)
        if table.dim() != 2 or table.shape[1] != Hq or not table.is_contiguous():
            raise ValueError(f"table must be a contiguous [num_buckets, {Hq}] tensor")
        tc = _code("table", table)
        tp, buckets = table.data_ptr(), table.shape[0]
        _check_buckets(buckets, max_distance, bidirectional)
    tail = (_check_list("seqlens_k", seqlens_k, q, B), _check_list("q_start", q_start, q, B), tp, code, tc,
            1 if causal else 0, 1 if table is not None and bidirectional else 0, buckets,
            int(max_distance) if table is not None else 0, scale, 0)
    return (B, Sq, Sk, Hq, Hkv, D), tail


def _check_buckets(buckets: int, max_distance: int, bidirectional: bool) -> None:
    n = buckets // 2 if bidirectional else buckets
    if buckets > DYT_ATTN_MAX_BUCKETS or n < 2 or (bidirectional and buckets % 2):
        raise ValueError(f"table must have 2 to {DYT_ATTN_MAX_BUCKETS} buckets (bidirectional: an even number "
                         f"of at least 4), got {buckets}")
    if not n // 2 < max_distance <= DYT_ATTN_MAX_DISTANCE:
        raise ValueError(f"max_distance must be over {n // 2} and at most {DYT_ATTN_MAX_DISTANCE}")


_NO_STRIDES = (0, 0, 0)


def dyt_attn_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, causal: bool = False,
                     scale: float | None = None, seqlens_k: torch.Tensor | None = None,
                     q_start: torch.Tensor | None = None, table: torch.Tensor | None = None,
                     max_distance: int = 128, bidirectional: bool = True, o: torch.Tensor | None = None,
                     stats: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Attention of q [B, Sq, Hq, D] over k, v [B, Sk, Hkv, D]; returns (o,
    stats), stats [B, Hq, Sq] float32 the log sums the backward needs.

    Query row i of batch entry b stands at position q_start[b] + i (default:
    Sk - Sq, so that the last query meets the last key) and sees the keys
    j < seqlens_k[b] and, with ``causal``, j <= its position; a row that sees
    none gives zeros. ``table`` [num_buckets, Hq] adds a learned bias by
    relative position (``max_distance``, ``bidirectional``: see
    include/dyt_block.h); ``scale`` defaults to D ** -0.5. Any strides of B, S
    and H are taken (a cache's layout, slices of a fused projection, expanded
    heads)."""
    sizes, tail = _attn_problem(q, k, v, causal, scale, seqlens_k, q_start, table, max_distance, bidirectional)
    B, Sq, Sk, Hq, Hkv, D = sizes
    s = _stream_for(q, stream)
    made = (o is None, stats is None, workspace is None)
    if o is None:
        o = _empty(q, (B, Sq, Hq, D))
    else:
        _check_heads("o", o, q, q.shape)
    if stats is None:
        stats = torch.empty((B, Hq, Sq), dtype=torch.float32, device=q.device)
    else:
        _check_stats_tensor(stats, q, B, Hq, Sq)
    desc = _DESC.pack(*sizes, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *o.stride()[:3],
                      *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *_NO_STRIDES, *tail)
    if workspace is None:
        need = block_lib.dyt_attn_forward_workspace_size(desc)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    else:
        _on_device("workspace", workspace, q)
        need = workspace.numel() * workspace.element_size()
    _check("dyt_attn_forward", block_lib.dyt_attn_forward(
        desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), stats.data_ptr(),
        workspace.data_ptr() if workspace is not None else None, need, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((o, stats, workspace), made) if m))
    return o, stats


def _check_stats_tensor(stats, q, B, Hq, Sq) -> None:
    _on_device("stats", stats, q)
    if stats.dtype != torch.float32 or stats.shape != (B, Hq, Sq) or not stats.is_contiguous():
        raise ValueError(f"stats must be a contiguous float32 [{B}, {Hq}, {Sq}] tensor")


def dyt_attn_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, do: torch.Tensor,
                      stats: torch.Tensor, *, causal: bool = False, scale: float | None = None,
                      seqlens_k: torch.Tensor | None = None, q_start: torch.Tensor | None = None,
                      table: torch.Tensor | None = None, max_distance: int = 128, bidirectional: bool = True,
                      dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                      dv: torch.Tensor | None = None, dtable: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """Gradients of dyt_attn_forward's o (with its options, o and stats) for
    the upstream gradient do: (dq, dk, dv), and dtable with a table."""
    sizes, tail = _attn_problem(q, k, v, causal, scale, seqlens_k, q_start, table, max_distance, bidirectional)
    B, Sq, Sk, Hq, Hkv, D = sizes
    s = _stream_for(q, stream)
    dev = q.device
    _check_heads("o", o, q, q.shape)
    _check_heads("do", do, q, q.shape)
    _check_stats_tensor(stats, q, B, Hq, Sq)
    made = (dq is None, dk is None, dv is None, dtable is None, workspace is None)
    if dq is None:
        dq = _empty(q, (B, Sq, Hq, D))
    else:
        _check_heads("dq", dq, q, q.shape)
    if dk is None:
        dk = _empty(k, (B, Sk, Hkv, D))
    else:
        _check_heads("dk", dk, q, k.shape)
    if dv is None:
        dv = _empty(v, (B, Sk, Hkv, D))
    else:
        _check_heads("dv", dv, q, k.shape)
    if table is None:
        dtable = None
    elif dtable is None:
        dtable = torch.empty(table.shape, dtype=table.dtype, device=dev)
    else:
        _on_device("dtable", dtable, q)
        if dtable.shape != table.shape or dtable.dtype != table.dtype or not dtable.is_contiguous():
            raise ValueError("dtable must match table and be contiguous")
    desc = _DESC.pack(*sizes, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3], *o.stride()[:3], *do.stride()[:3],
                      *dq.stride()[:3], *dk.stride()[:3], *dv.stride()[:3], *tail)
    if workspace is None:
        need = block_lib.dyt_attn_backward_workspace_size(desc)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _on_device("workspace", workspace, q)
        need = workspace.numel() * workspace.element_size()
    _check("dyt_attn_backward", block_lib.dyt_attn_backward(
        desc, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), stats.data_ptr(), dq.data_ptr(),
        dk.data_ptr(), dv.data_ptr(), dtable.data_ptr() if dtable is not None else None, workspace.data_ptr(), need,
        s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((dq, dk, dv, dtable, workspace), made) if m and t is not None))
    return (dq, dk, dv) if dtable is None else (dq, dk, dv, dtable)


def dyt_attn_bucket_borders(num_buckets: int, max_distance: int, bidirectional: bool = True) -> list[int]:
    """The smallest distance of every bucket of one direction (host only)."""
    _check_buckets(num_buckets, max_distance, bidirectional)
    out = (ctypes.c_int32 * num_buckets)()
    n = block_lib.dyt_attn_bucket_borders(num_buckets, int(max_distance), 1 if bidirectional else 0, out)
    return list(out[:n])
