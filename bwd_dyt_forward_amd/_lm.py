"""Python binding of the C ABI of the operators around a decoder's blocks
(include/dyt_lm.h): root-mean-square norm, embedding, log probabilities and
AdamW, argument marshalling only.

Every computation runs in the HIP library ``libdyt_lm.so``; like the other
bindings this module checks tensors, allocates outputs and workspace with
PyTorch and passes device pointers and torch's current HIP stream. There is no
CPU fallback: importing this module fails if the library is missing.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._block import _check, _check_rows, _check_stats, _check_vectors, _code, _empty, _on_device, _stream_for
from ._lib import _keep_alive_on
from .build import LM_DEPENDS, LM_LIB_PATH, source_hash

LM_ABI_VERSION = 1
DYT_Q8_GROUPS = (0, 32, 64, 128)

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
_f32 = ctypes.c_float
_size = ctypes.c_size_t

SIGNATURES = {
    "dyt_lm_abi_version": (_int, []),
    "dyt_lm_build_id": (ctypes.c_char_p, []),
    "dyt_rms_forward": (_int, [_vp, _i64, _vp, _vp, _i64, _vp, _i64, _i64, _f32, _int, _int, _vp]),
    "dyt_rms_forward_residual": (_int, [_vp] * 6 + [_i64, _i64, _f32, _int, _int, _vp]),
    "dyt_rms_forward_q8": (_int, [_vp, _i64] + [_vp] * 5 + [_i64, _i64, _int, _f32, _int, _int, _vp]),
    "dyt_rms_backward_workspace_size": (_size, [_i64, _i64, _int, _int]),
    "dyt_rms_backward": (_int, [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _size, _i64, _i64, _int, _int,
                                _vp]),
    "dyt_rms_backward_residual": (_int, [_vp] * 8 + [_size, _i64, _i64, _int, _int, _vp]),
    "dyt_embed_forward": (_int, [_vp, _i64, _vp, _vp, _i64, _i64, _i64, _i64, _f32, _int, _int, _int, _vp]),
    "dyt_embed_backward_workspace_size": (_size, [_i64, _i64, _i64]),
    "dyt_embed_backward": (_int, [_vp, _i64, _vp, _vp, _i64, _vp, _size, _i64, _i64, _i64, _f32, _int, _int, _int, _int,
                                  _vp]),
    "dyt_logprob_forward_workspace_size": (_size, [_i64, _i64, _int, _int]),
    "dyt_logprob_forward": (_int, [_vp, _i64] + [_vp] * 7 + [_size, _i64, _i64, _f32, _int, _int, _int, _vp]),
    "dyt_logprob_forward_norm": (_int, [_vp, _i64] + [_vp] * 8 + [_size, _i64, _i64, _f32, _int, _int, _int, _vp]),
    "dyt_logprob_backward_norm": (_int, [_vp, _i64] + [_vp] * 5 + [_i64, _i64, _i64, _f32, _int, _int, _vp]),
    "dyt_logprob_backward": (_int, [_vp, _i64] + [_vp] * 6 + [_i64, _i64, _i64, _f32, _int, _int, _vp]),
    "dyt_adamw_step": (_int, [_vp, _i64, _vp, _vp]),
    "dyt_adamw_check": (_int, [_vp, _i64, _vp]),
    "dyt_adamw_values": (_int, [_vp, _i64, _int, _vp]),
}


def _load(path: str = LM_LIB_PATH, any_sources: bool = False) -> ctypes.CDLL:
    """Load the decoder operators' library, built from the current sources."""
    if not os.path.exists(path):
        raise ImportError(
            f"decoder operators' HIP library not found at {path}; build it first "
            "(python bwd_dyt_forward_amd/build.py, or __graft_entry__.build())")
    lib = ctypes.CDLL(path, mode=ctypes.RTLD_LOCAL)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name, None)
        if fn is None:
            raise ImportError(f"{path} has no {name}: it was built from other sources; rebuild it "
                              "(python bwd_dyt_forward_amd/build.py)")
        fn.restype = res
        fn.argtypes = args
    found = lib.dyt_lm_abi_version()
    if found != LM_ABI_VERSION:
        raise ImportError(f"{path} has ABI version {found}, this binding expects {LM_ABI_VERSION}; "
                          "rebuild the library")
    built, want = lib.dyt_lm_build_id().decode(), source_hash((), LM_DEPENDS)
    if built != want and not any_sources:
        raise ImportError(f"{path} was built from other sources (build id {built}, sources "
                          f"{want}); rebuild it (python bwd_dyt_forward_amd/build.py)")
    return lib


lm_lib = _load()
LM_LIB_FILE = LM_LIB_PATH


# ---------------------------------------------------- root-mean-square norm
def dyt_rms_forward(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5, y: torch.Tensor | None = None,
                    rstd: torch.Tensor | None = None, stream=None):
    """Root-mean-square norm of the rows of x [M, N]: returns (y, rstd), rstd
    float32 [M]. x and y may be row-strided (unit column stride)."""
    ldx = _check_rows("x", x)
    M, N = x.shape
    pc = _check_vectors(x, N, gamma=gamma)
    xc = _code("x", x)
    s = _stream_for(x, stream)
    made = (y is None, rstd is None)
    if y is None:
        y = _empty(x, (M, N))
    ldy = N if made[0] else _check_rows("y", y, x)
    if rstd is None:
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    else:
        _check_stats(x, M, rstd=rstd)
    _check("dyt_rms_forward", lm_lib.dyt_rms_forward(
        x.data_ptr(), ldx, gamma.data_ptr(), y.data_ptr(), ldy, rstd.data_ptr(), M, N, eps, xc, pc, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((y, rstd), made) if m))
    return y, rstd


def dyt_rms_forward_residual(x: torch.Tensor, r: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5,
                             h: torch.Tensor | None = None, y: torch.Tensor | None = None,
                             rstd: torch.Tensor | None = None, stream=None):
    """h = x + r (rounded to x's dtype) and its norm: (h, y, rstd)."""
    _check_rows("x", x, dense=True)
    _check_rows("r", r, x, dense=True)
    M, N = x.shape
    pc = _check_vectors(x, N, gamma=gamma)
    xc = _code("x", x)
    s = _stream_for(x, stream)
    made = (h is None, y is None, rstd is None)
    if h is None:
        h = _empty(x, (M, N))
    else:
        _check_rows("h", h, x, dense=True)
    if y is None:
        y = _empty(x, (M, N))
    else:
        _check_rows("y", y, x, dense=True)
    if rstd is None:
        rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    else:
        _check_stats(x, M, rstd=rstd)
    _check("dyt_rms_forward_residual", lm_lib.dyt_rms_forward_residual(
        x.data_ptr(), r.data_ptr(), gamma.data_ptr(), h.data_ptr(), y.data_ptr(), rstd.data_ptr(), M, N, eps, xc, pc,
        s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((h, y, rstd), made) if m))
    return h, y, rstd


def _rms_q8(x, r, gamma, eps, group, h, q, scales, stream):
    ldx = _check_rows("x", x, dense=r is not None)
    M, N = x.shape
    pc = _check_vectors(x, N, gamma=gamma)
    xc = _code("x", x)
    if group not in DYT_Q8_GROUPS:
        raise ValueError(f"group must be one of {DYT_Q8_GROUPS} (0: one scale for each row)")
    groups = -(-N // group) if group else 1
    s = _stream_for(x, stream)
    made = (h is None and r is not None, q is None, scales is None)
    if r is not None:
        _check_rows("r", r, x, dense=True)
        if h is None:
            h = _empty(x, (M, N))
        else:
            _check_rows("h", h, x, dense=True)
    if q is None:
        q = torch.empty((M, N), dtype=torch.float8_e4m3fn, device=x.device)
    else:
        _on_device("q", q, x)
        if q.dtype != torch.float8_e4m3fn or q.shape != x.shape or not q.is_contiguous():
            raise ValueError(f"q must be a contiguous float8_e4m3fn [{M}, {N}] tensor")
    if scales is None:
        scales = torch.empty((M, groups), dtype=torch.float32, device=x.device)
    else:
        _on_device("scales", scales, x)
        if scales.dtype != torch.float32 or scales.shape != (M, groups) or not scales.is_contiguous():
            raise ValueError(f"scales must be a contiguous float32 [{M}, {groups}] tensor")
    _check("dyt_rms_forward_q8", lm_lib.dyt_rms_forward_q8(
        x.data_ptr(), ldx, r.data_ptr() if r is not None else None, gamma.data_ptr(),
        h.data_ptr() if r is not None else None, q.data_ptr(), scales.data_ptr(), M, N, group, eps, xc, pc, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((h, q, scales), made) if m))
    return h, q, scales


def dyt_rms_forward_q8(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5, group: int = 0,
                       q: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """The norm in 8 bits: (q, scales), q float8_e4m3fn [M, N], y about q *
    scales; one float32 scale for each row (group 0, scales [M, 1]) or for
    each ``group`` = 32, 64 or 128 columns (scales [M, ceil(N / group)])."""
    return _rms_q8(x, None, gamma, eps, group, None, q, scales, stream)[1:]


def dyt_rms_forward_residual_q8(x: torch.Tensor, r: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5,
                                group: int = 0, h: torch.Tensor | None = None, q: torch.Tensor | None = None,
                                scales: torch.Tensor | None = None, stream=None):
    """h = x + r and its norm in 8 bits: (h, q, scales)."""
    if not isinstance(r, torch.Tensor):
        raise ValueError("r must be a device tensor")
    return _rms_q8(x, r, gamma, eps, group, h, q, scales, stream)


def dyt_rms_backward_workspace_size(M: int, N: int, x_dtype, param_dtype) -> int:
    return int(lm_lib.dyt_rms_backward_workspace_size(int(M), int(N), _lib._code(x_dtype), _lib._code(param_dtype)))


def _rms_backward(x, dy, dres, rstd, gamma, dx, dgamma, workspace, stream):
    res = dres is not None
    xname = "h" if res else "x"
    ldx = _check_rows(xname, x, dense=res)
    lddy = _check_rows("dy", dy, x, dense=res)
    if res:
        _check_rows("dres", dres, x, dense=True)
    M, N = x.shape
    pc = _check_vectors(x, N, gamma=gamma)
    _check_stats(x, M, rstd=rstd)
    xc = _code(xname, x)
    s = _stream_for(x, stream)
    made = (dx is None, dgamma is None, workspace is None)
    if dx is None:
        dx = _empty(x, (M, N))
        lddx = N
    else:
        lddx = _check_rows("dx", dx, x, dense=res)
    if dgamma is None:
        dgamma = torch.empty(N, dtype=gamma.dtype, device=x.device)
    else:
        _check_vectors(x, N, gamma=gamma, dgamma=dgamma)
    if workspace is None:
        need = lm_lib.dyt_rms_backward_workspace_size(M, N, xc, pc)
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    else:
        _on_device("workspace", workspace, x)
        need = workspace.numel() * workspace.element_size()
    if res:
        _check("dyt_rms_backward_residual", lm_lib.dyt_rms_backward_residual(
            x.data_ptr(), dy.data_ptr(), dres.data_ptr(), rstd.data_ptr(), gamma.data_ptr(), dx.data_ptr(),
            dgamma.data_ptr(), workspace.data_ptr(), need, M, N, xc, pc, s))
    else:
        _check("dyt_rms_backward", lm_lib.dyt_rms_backward(
            x.data_ptr(), ldx, dy.data_ptr(), lddy, rstd.data_ptr(), gamma.data_ptr(), dx.data_ptr(), lddx,
            dgamma.data_ptr(), workspace.data_ptr(), need, M, N, xc, pc, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((dx, dgamma, workspace), made) if m))
    return dx, dgamma


def dyt_rms_backward(x: torch.Tensor, dy: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor,
                     dx: torch.Tensor | None = None, dgamma: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """The norm's backward at x with the forward's rstd: (dx, dgamma). x, dy
    and dx may be row-strided (unit column stride)."""
    return _rms_backward(x, dy, None, rstd, gamma, dx, dgamma, workspace, stream)


def dyt_rms_backward_residual(h: torch.Tensor, dy: torch.Tensor, dres: torch.Tensor, rstd: torch.Tensor,
                              gamma: torch.Tensor, dx: torch.Tensor | None = None, dgamma: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, stream=None):
    """dx = dres + (the norm's backward of dy at h): (dx, dgamma); dx is the
    gradient of both x and r."""
    if not isinstance(dres, torch.Tensor):
        raise ValueError("dres must be a device tensor")
    return _rms_backward(h, dy, dres, rstd, gamma, dx, dgamma, workspace, stream)


# ------------------------------------------------------------------ tokens
_TOKEN_BITS = {torch.int32: 32, torch.int64: 64}


def _check_tokens(tokens, like: torch.Tensor) -> int:
    """A contiguous int32 or int64 tensor on like's device; returns its bits."""
    _on_device("tokens", tokens, like)
    bits = _TOKEN_BITS.get(tokens.dtype)
    if bits is None or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous int32 or int64 tensor")
    return bits


def _workspace(workspace, need: int, like: torch.Tensor):
    """(tensor or None, its bytes): the given one or a new one of `need`."""
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=like.device) if need else None), need
    _on_device("workspace", workspace, like)
    return workspace, workspace.numel() * workspace.element_size()


def _ptr(t: torch.Tensor | None):
    return t.data_ptr() if t is not None else None


# --------------------------------------------------------------- embedding
def dyt_embed_forward(weight: torch.Tensor, tokens: torch.Tensor, scale: float = 1.0, dtype=None,
                      y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows of weight [V, D] for tokens [T] (int32 or int64), times scale: y
    [T, D] of ``dtype`` (weight's). A token outside [0, V) gives zeros. weight
    and y may be row-strided (unit column stride)."""
    ldw = _check_rows("weight", weight)
    V, D = weight.shape
    wc = _code("weight", weight)
    bits = _check_tokens(tokens, weight)
    if tokens.dim() != 1:
        raise ValueError("tokens must have one dimension")
    T = tokens.shape[0]
    s = _stream_for(weight, stream)
    made = y is None
    if made:
        y = torch.empty((T, D), dtype=dtype or weight.dtype, device=weight.device)
        ldy = D
    else:
        ldy = _check_rows("y", y)
        if y.shape != (T, D) or y.device != weight.device or dtype not in (None, y.dtype):
            raise ValueError(f"y must be [{T}, {D}] on {weight.device}, of the dtype asked for")
    _check("dyt_embed_forward", lm_lib.dyt_embed_forward(
        weight.data_ptr(), ldw, tokens.data_ptr(), y.data_ptr(), ldy, T, V, D, scale, wc, _code("y", y), bits, s))
    if stream is not None and made:
        _keep_alive_on(stream, y)
    return y


def dyt_embed_backward_workspace_size(T: int, V: int, D: int) -> int:
    return int(lm_lib.dyt_embed_backward_workspace_size(int(T), int(V), int(D)))


def dyt_embed_backward(dy: torch.Tensor, tokens: torch.Tensor, num_rows: int, scale: float = 1.0, dtype=None,
                       dweight: torch.Tensor | None = None, accumulate: bool = False,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The lookup's gradient for dy [T, D]: dweight [num_rows, D] of ``dtype``
    (dy's), zeros in the rows of tokens that do not occur. With
    ``accumulate`` it is added to the given dweight, whose other rows stay."""
    lddy = _check_rows("dy", dy)
    T, D = dy.shape
    V = int(num_rows)
    yc = _code("dy", dy)
    bits = _check_tokens(tokens, dy)
    if tokens.shape != (T,):
        raise ValueError(f"tokens must have shape ({T},)")
    s = _stream_for(dy, stream)
    made = (dweight is None, workspace is None)
    if dweight is None:
        if accumulate:
            raise ValueError("accumulate adds to a given dweight")
        dweight = torch.empty((V, D), dtype=dtype or dy.dtype, device=dy.device)
        lddw = D
    else:
        lddw = _check_rows("dweight", dweight)
        if dweight.shape != (V, D) or dweight.device != dy.device or dtype not in (None, dweight.dtype):
            raise ValueError(f"dweight must be [{V}, {D}] on {dy.device}, of the dtype asked for")
    workspace, need = _workspace(workspace, lm_lib.dyt_embed_backward_workspace_size(T, V, D), dy)
    _check("dyt_embed_backward", lm_lib.dyt_embed_backward(
        dy.data_ptr(), lddy, tokens.data_ptr(), dweight.data_ptr(), lddw, _ptr(workspace), need, T, V, D, scale, yc,
        _code("dweight", dweight), bits, 1 if accumulate else 0, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((dweight, workspace), made) if m and t is not None))
    return dweight


# ------------------------------------------------- token log probabilities
DYT_LOGPROB_MAX_TOP = 64


def _check_scale(scale: float) -> None:
    if not 0.0 < scale < float("inf"):
        raise ValueError("scale must be positive and finite")


def _check_norm(norm, logits: torch.Tensor, T: int) -> None:
    _on_device("norm", norm, logits)
    if norm.dtype != torch.float32 or norm.shape != (T, 3) or not norm.is_contiguous():
        raise ValueError(f"norm must be a contiguous float32 [{T}, 3] tensor")


def dyt_logprob_forward_workspace_size(T: int, V: int, top: int, dtype) -> int:
    return int(lm_lib.dyt_logprob_forward_workspace_size(int(T), int(V), int(top), _lib._code(dtype)))


def dyt_logprob_forward(logits: torch.Tensor, tokens: torch.Tensor, *, scale: float = 1.0, top: int = 0,
                        logp: torch.Tensor | None = None, entropy: torch.Tensor | None = None,
                        lse: torch.Tensor | None = None, top_logp: torch.Tensor | None = None,
                        top_tokens: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        norm: torch.Tensor | None = None, stream=None):
    """Log probabilities of tokens [T] (int32 or int64) under the rows of
    logits [T, V] (row-strided; times ``scale``, an inverse temperature):
    (logp, entropy, lse), each [T] float32; with ``top`` also (top_logp,
    top_tokens) [T, top], the largest logits' in falling order, equal ones from
    the lowest place on. A token outside [0, V) has logp 0. ``norm`` (float32 [T, 3]),
    where given, is filled for the backward."""
    ld = _check_rows("logits", logits)
    T, V = logits.shape
    code = _code("logits", logits)
    bits = _check_tokens(tokens, logits)
    if tokens.shape != (T,):
        raise ValueError(f"tokens must have shape ({T},)")
    _check_scale(scale)
    if not 0 <= top <= min(V, DYT_LOGPROB_MAX_TOP):
        raise ValueError(f"top must be 0 to {DYT_LOGPROB_MAX_TOP} and at most {V}")
    s = _stream_for(logits, stream)
    dev = logits.device
    made = (logp is None, entropy is None, lse is None, top_logp is None, top_tokens is None, workspace is None)
    if logp is None:
        logp = torch.empty(T, dtype=torch.float32, device=dev)
    if entropy is None:
        entropy = torch.empty(T, dtype=torch.float32, device=dev)
    if lse is None:
        lse = torch.empty(T, dtype=torch.float32, device=dev)
    if not (made[0] and made[1] and made[2]):
        _check_stats(logits, T, logp=logp, entropy=entropy, lse=lse)
    if top:
        if top_logp is None:
            top_logp = torch.empty((T, top), dtype=torch.float32, device=dev)
        if top_tokens is None:
            top_tokens = torch.empty((T, top), dtype=torch.int64, device=dev)
        for name, t, dt in (("top_logp", top_logp, torch.float32), ("top_tokens", top_tokens, torch.int64)):
            _on_device(name, t, logits)
            if t.dtype != dt or t.shape != (T, top) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dt} [{T}, {top}] tensor")
    else:
        top_logp = top_tokens = None
    workspace, need = _workspace(workspace, lm_lib.dyt_logprob_forward_workspace_size(T, V, top, code), logits)
    if norm is None:
        _check("dyt_logprob_forward", lm_lib.dyt_logprob_forward(
            logits.data_ptr(), ld, tokens.data_ptr(), logp.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
            _ptr(top_logp), _ptr(top_tokens), _ptr(workspace), need, T, V, scale, top, code, bits, s))
    else:
        _check_norm(norm, logits, T)
        _check("dyt_logprob_forward_norm", lm_lib.dyt_logprob_forward_norm(
            logits.data_ptr(), ld, tokens.data_ptr(), logp.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
            norm.data_ptr(), _ptr(top_logp), _ptr(top_tokens), _ptr(workspace), need, T, V, scale, top, code, bits, s))
    if stream is not None:
        _keep_alive_on(stream, *(t for t, m in zip((logp, entropy, lse, top_logp, top_tokens, workspace), made)
                                 if m and t is not None))
    return (logp, entropy, lse, top_logp, top_tokens) if top else (logp, entropy, lse)


def dyt_logprob_backward(logits: torch.Tensor, tokens: torch.Tensor, entropy: torch.Tensor | None = None,
                         lse: torch.Tensor | None = None,
                         dlogp: torch.Tensor | None = None, dentropy: torch.Tensor | None = None, *,
                         scale: float = 1.0, dlogits: torch.Tensor | None = None, norm: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Gradient of the logits for those of logp and entropy ([T] float32, each
    may be None) with the forward's entropy and lse, or with its ``norm`` in their
    place: lse is one float32 number, and the relative error of a gradient from it
    grows with |lse| 2^-23. ``dlogits`` may be the logits themselves."""
    ld = _check_rows("logits", logits)
    T, V = logits.shape
    code = _code("logits", logits)
    bits = _check_tokens(tokens, logits)
    if tokens.shape != (T,):
        raise ValueError(f"tokens must have shape ({T},)")
    _check_scale(scale)
    stats = {"entropy": entropy, "lse": lse} if norm is None else {}
    if dlogp is not None:
        stats["dlogp"] = dlogp
    if dentropy is not None:
        stats["dentropy"] = dentropy
    _check_stats(logits, T, **stats)
    s = _stream_for(logits, stream)
    made = dlogits is None
    if made:
        dlogits = _empty(logits, (T, V))
        ldd = V
    else:
        ldd = _check_rows("dlogits", dlogits, logits)
    if norm is None:
        _check("dyt_logprob_backward", lm_lib.dyt_logprob_backward(
            logits.data_ptr(), ld, tokens.data_ptr(), entropy.data_ptr(), lse.data_ptr(), _ptr(dlogp), _ptr(dentropy),
            dlogits.data_ptr(), ldd, T, V, scale, code, bits, s))
    else:
        _check_norm(norm, logits, T)
        _check("dyt_logprob_backward_norm", lm_lib.dyt_logprob_backward_norm(
            logits.data_ptr(), ld, tokens.data_ptr(), norm.data_ptr(), _ptr(dlogp), _ptr(dentropy), dlogits.data_ptr(),
            ldd, T, V, scale, code, bits, s))
    if stream is not None and made:
        _keep_alive_on(stream, dlogits)
    return dlogits


# ------------------------------------------------------------------- AdamW
DYT_ADAMW_BLOCK = 128
# struct dyt_adamw_tensor: 7 pointers, n, 2 dtypes; dyt_adamw_options: 5 doubles,
# step, 3 pointers, seed, seeded, state_bits, reserved; dyt_adamw_codes: 3
# pointers, n, second, reserved
_ADAMW_TENSOR = struct.Struct("=7Qq2i")
_ADAMW_OPTIONS = struct.Struct("=5dq3QI3i")
_ADAMW_CODES = struct.Struct("=3Qq2i")


def _blocks(n: int) -> int:
    return -(-n // DYT_ADAMW_BLOCK)


def _one(name: str, t, dtype, device: int) -> int:
    if not isinstance(t, torch.Tensor) or t.get_device() != device or t.dtype != dtype or t.numel() != 1:
        raise ValueError(f"{name} must be a number or a {dtype} tensor of one element on the parameters' device")
    return t.data_ptr()


def dyt_adamw_step(params, grads, exp_avgs, exp_avg_sqs, *, lr, betas=(0.9, 0.999), eps: float = 1e-8,
                   weight_decay: float = 0.01, step, masters=None, avg_scales=None, sq_scales=None,
                   grad_scale: torch.Tensor | None = None, seed: int | None = None, stream=None) -> None:
    """One AdamW step, in place, over lists of tensors on the current device.

    Parameters are float32, bfloat16 or float16, gradients of the parameter's
    dtype or float32, all contiguous. ``masters`` (float32, None for single
    parameters): the step is theirs and the parameter is written from them.
    States are float32; with ``avg_scales`` and ``sq_scales`` (float32
    [ceil(n / 128)]) they are 8-bit codes, int8 and uint8 (see
    include/dyt_lm.h), rounded at random with a ``seed`` and to the nearest
    code without.

    ``step`` counts from 1. ``lr``, ``step`` (int64) and ``grad_scale`` may be
    device tensors of one element, which a captured step then follows."""
    table = _adamw_table(params, grads, exp_avgs, exp_avg_sqs, lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                         step=step, masters=masters, avg_scales=avg_scales, sq_scales=sq_scales, grad_scale=grad_scale,
                         seed=seed, stream=stream)
    if table is not None:
        _adamw_run(params, table)


def _adamw_check(table) -> None:
    """Raises what _adamw_run would be refused with."""
    _check("dyt_adamw_step", lm_lib.dyt_adamw_check(*table[:3]))


def _adamw_run(params, table) -> None:
    _check("dyt_adamw_step", lm_lib.dyt_adamw_step(*table))
    increment_version(params)


def _adamw_table(params, grads, exp_avgs, exp_avg_sqs, *, lr, betas, eps, weight_decay, step, masters=None, avg_scales=None,
                 sq_scales=None, grad_scale=None, seed=None, stream=None):
    """dyt_adamw_step's checks; the arguments of the library's call (None of no tensors)."""
    n = len(params)
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == n):
        raise ValueError("params, grads, exp_avgs and exp_avg_sqs must have equal lengths")
    bits8 = avg_scales is not None
    if bits8 != (sq_scales is not None):
        raise ValueError("8-bit states have both avg_scales and sq_scales")
    for name, x in (("masters", masters), ("avg_scales", avg_scales), ("sq_scales", sq_scales)):
        if x is not None and len(x) != n:
            raise ValueError(f"{name} must have one entry for each parameter")
    if n == 0:
        return None
    dev = params[0].get_device()
    if dev < 0:
        raise ValueError("params must be device tensors")
    s = _stream_for(params[0], stream)
    m_dt, v_dt = (torch.int8, torch.uint8) if bits8 else (torch.float32, torch.float32)
    f32 = torch.float32
    pack = _ADAMW_TENSOR.pack
    rows = []
    for i, (p, g, m, v) in enumerate(zip(params, grads, exp_avgs, exp_avg_sqs)):
        k, pd, gd = p.numel(), p.dtype, g.dtype
        master = masters[i] if masters is not None else None
        if not (p.get_device() == g.get_device() == m.get_device() == v.get_device() == dev):
            raise ValueError(f"tensors {i} must all be on device {dev}")
        if not (p.is_contiguous() and g.is_contiguous() and m.is_contiguous() and v.is_contiguous()):
            raise ValueError(f"tensors {i} must be contiguous")
        if not k == g.numel() == m.numel() == v.numel():
            raise ValueError(f"tensors {i} must have equal numbers of elements")
        if m.dtype != m_dt or v.dtype != v_dt:
            raise ValueError(f"states {i} must be {m_dt} and {v_dt}")
        if gd != pd and gd != f32:
            raise ValueError(f"gradient {i} must have its parameter's dtype or float32")
        a = b = c = 0
        if bits8:
            sa, sv = avg_scales[i], sq_scales[i]
            for t in (sa, sv):
                if t.get_device() != dev or t.dtype != f32 or t.numel() != _blocks(k) or not t.is_contiguous():
                    raise ValueError(f"scales {i} must be contiguous float32 with {_blocks(k)} elements on device {dev}")
            a, b = sa.data_ptr(), sv.data_ptr()
        if master is not None:
            if (master.get_device() != dev or master.dtype != f32 or master.numel() != k or not master.is_contiguous()
                    or pd == f32):
                raise ValueError(f"master {i} must be contiguous float32 like its 16-bit parameter")
            c = master.data_ptr()
        rows.append(pack(p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), a, b, c, k, _code("params", p),
                         _CODE[gd]))
    lr_dev = step_dev = gs = 0
    if isinstance(lr, torch.Tensor):
        lr, lr_dev = 0.0, _one("lr", lr, f32, dev)
    if isinstance(step, torch.Tensor):
        step, step_dev = 0, _one("step", step, torch.int64, dev)
    elif step < 1:
        raise ValueError("step counts from 1")
    if grad_scale is not None:
        gs = _one("grad_scale", grad_scale, f32, dev)
    for name, x in (("lr", lr), ("beta1", betas[0]), ("beta2", betas[1]), ("eps", eps), ("weight_decay", weight_decay)):
        if not 0.0 <= x < (1.0 if name.startswith("beta") else math.inf):
            raise ValueError(f"{name} is out of range: {x}")
    options = _ADAMW_OPTIONS.pack(lr, betas[0], betas[1], eps, weight_decay, int(step), lr_dev, step_dev, gs,
                                  (seed or 0) & 0xFFFFFFFF, 0 if seed is None else 1, 8 if bits8 else 32, 0)
    return b"".join(rows), n, options, s


_CODE = _lib._TORCH_TO_CODE


def dyt_adamw_values(codes, scales, dtype=torch.float32, values=None, stream=None):
    """The values that lists of 8-bit codes (int8: first moments, uint8: second
    moments) with their scales stand for, as tensors of ``dtype``."""
    if len(codes) != len(scales) or (values is not None and len(values) != len(codes)):
        raise ValueError("codes, scales and values must have equal lengths")
    if not codes:
        return []
    s = _stream_for(codes[0], stream)
    made = values is None
    out, rows = [], []
    for i, (c, a) in enumerate(zip(codes, scales)):
        n = c.numel()
        if c.device != codes[0].device or c.dtype not in (torch.int8, torch.uint8) or not c.is_contiguous():
            raise ValueError(f"codes {i} must be contiguous int8 or uint8 on {codes[0].device}")
        if a.device != c.device or a.dtype != torch.float32 or a.numel() != _blocks(n) or not a.is_contiguous():
            raise ValueError(f"scales {i} must be contiguous float32 with {_blocks(n)} elements on {c.device}")
        v = torch.empty(c.shape, dtype=dtype, device=c.device) if made else values[i]
        if v.device != c.device or v.dtype != dtype or v.numel() != n or not v.is_contiguous():
            raise ValueError(f"values {i} must be contiguous {dtype} with {n} elements on {c.device}")
        out.append(v)
        rows.append(_ADAMW_CODES.pack(c.data_ptr(), a.data_ptr(), v.data_ptr(), n, 1 if c.dtype == torch.uint8 else 0, 0))
    _check("dyt_adamw_values", lm_lib.dyt_adamw_values(b"".join(rows), len(rows), _code("values", out[0]), s))
    if stream is not None and made:
        _keep_alive_on(stream, *out)
    return out
