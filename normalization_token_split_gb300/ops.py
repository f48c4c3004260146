"""Torch-facing binding of libnts: argument marshalling only.  Every step of
the computation runs in the library's CUDA kernels; these functions check
tensor placement, allocate missing outputs with torch, and pass raw pointers
and the current CUDA stream through the C ABI.  Names follow the C ABI
(include/nts.h), without the ``nts_`` prefix."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from ._lib import check, lib, marshal

FMT_E4M3 = 0
FMT_E2M1 = 1
FMT_NVFP4 = 2   # E2M1 elements, B = 16, E4M3 block scales
_FMT_NAMES = {"e4m3": FMT_E4M3, "e2m1": FMT_E2M1, "nvfp4": FMT_NVFP4,
              FMT_E4M3: FMT_E4M3, FMT_E2M1: FMT_E2M1, FMT_NVFP4: FMT_NVFP4}


class MxOut(NamedTuple):
    codes: torch.Tensor     # uint8 [T, D] (E4M3) or [T, D/2] (E2M1)
    scales: torch.Tensor    # uint8 [T, D/B] E8M0
    rinv: Optional[torch.Tensor]   # fp32 [T]
    amax: Optional[torch.Tensor]   # fp32 [T, D/B]


def _fmt(fmt) -> int:
    try:
        return _FMT_NAMES[fmt.lower() if isinstance(fmt, str) else fmt]
    except KeyError:
        raise ValueError(f"unknown element format {fmt!r}") from None


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need_cuda(name: str, t: torch.Tensor, dtype) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def codes_row_bytes(D: int, fmt) -> int:
    return D if _fmt(fmt) == FMT_E4M3 else D // 2


def qknorm_rms(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, N: int = 1,
               out: Optional[torch.Tensor] = None, rinv: Optional[torch.Tensor] = None,
               want_rinv: bool = False, stream=None):
    """Layerwise QK-RMSNorm of x [T, H] (bf16) with gain gamma [H] (fp32),
    split into N cluster shards.  Returns (y, rinv or None).  out may be x."""
    _need_cuda("x", x, torch.bfloat16)
    _need_cuda("gamma", gamma, torch.float32)
    T, H = x.shape
    if out is None:
        out = torch.empty_like(x)
    _need_cuda("out", out, torch.bfloat16)
    if rinv is None and want_rinv:
        rinv = torch.empty(T, device=x.device, dtype=torch.float32)
    if rinv is not None:
        _need_cuda("rinv", rinv, torch.float32)
    check(lib().nts_qknorm_rms(_ptr(x), _ptr(gamma), _ptr(out), _ptr(rinv), T, H,
                               float(eps), int(N), _stream(stream)))
    return out, rinv


def qknorm_rms_fp8(x_codes: torch.Tensor, x_scale: float, gamma: torch.Tensor,
                   eps: float = 1e-6, N: int = 1, out: Optional[torch.Tensor] = None,
                   rinv: Optional[torch.Tensor] = None, want_rinv: bool = False, stream=None):
    """QK-RMSNorm of FP8-E4M3 activations: x_codes uint8 (or float8_e4m3fn)
    [T, H], value = code * x_scale.  Returns (y bf16 [T, H], rinv or None)."""
    if x_codes.dtype == torch.float8_e4m3fn:
        x_codes = x_codes.view(torch.uint8)
    _need_cuda("x_codes", x_codes, torch.uint8)
    _need_cuda("gamma", gamma, torch.float32)
    T, H = x_codes.shape
    if out is None:
        out = torch.empty(T, H, device=x_codes.device, dtype=torch.bfloat16)
    _need_cuda("out", out, torch.bfloat16)
    if rinv is None and want_rinv:
        rinv = torch.empty(T, device=x_codes.device, dtype=torch.float32)
    if rinv is not None:
        _need_cuda("rinv", rinv, torch.float32)
    check(lib().nts_qknorm_rms_fp8(_ptr(x_codes), float(x_scale), _ptr(gamma), _ptr(out),
                                   _ptr(rinv), T, H, float(eps), int(N), _stream(stream)))
    return out, rinv


def qknorm_rms_heads(x: torch.Tensor, gamma: torch.Tensor, head_dim: int, eps: float = 1e-6,
                     N: int = 1, out: Optional[torch.Tensor] = None,
                     rinv: Optional[torch.Tensor] = None, want_rinv: bool = False, stream=None):
    """Headwise QK-Norm of x [T, H] (H = nheads * head_dim) with gamma
    [head_dim] shared by the heads.  Returns (y, rinv [T, nheads] or None)."""
    _need_cuda("x", x, torch.bfloat16)
    _need_cuda("gamma", gamma, torch.float32)
    T, H = x.shape
    if out is None:
        out = torch.empty_like(x)
    _need_cuda("out", out, torch.bfloat16)
    if rinv is None and want_rinv:
        rinv = torch.empty(T, H // head_dim, device=x.device, dtype=torch.float32)
    if rinv is not None:
        _need_cuda("rinv", rinv, torch.float32)
    check(lib().nts_qknorm_rms_heads(_ptr(x), _ptr(gamma), _ptr(out), _ptr(rinv), T, H,
                                     int(head_dim), float(eps), int(N), _stream(stream)))
    return out, rinv


def layernorm_split(x: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor] = None,
                    eps: float = 1e-5, N: int = 1, out: Optional[torch.Tensor] = None,
                    mean: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                    want_stats: bool = False, stream=None):
    """LayerNorm of x [T, H] (bf16) with gain gamma and optional shift beta
    (fp32 [H]), the statistics exchanged as per-shard (sum, sum of squares)
    between N cluster shards.  Returns (y, mean or None, rstd or None)."""
    _need_cuda("x", x, torch.bfloat16)
    _need_cuda("gamma", gamma, torch.float32)
    if beta is not None:
        _need_cuda("beta", beta, torch.float32)
    T, H = x.shape
    if out is None:
        out = torch.empty_like(x)
    _need_cuda("out", out, torch.bfloat16)
    if want_stats:
        mean = torch.empty(T, device=x.device, dtype=torch.float32) if mean is None else mean
        rstd = torch.empty(T, device=x.device, dtype=torch.float32) if rstd is None else rstd
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t is not None:
            _need_cuda(name, t, torch.float32)
    check(lib().nts_layernorm_split(_ptr(x), _ptr(gamma), _ptr(beta), _ptr(out), _ptr(mean),
                                    _ptr(rstd), T, H, float(eps), int(N), _stream(stream)))
    return out, mean, rstd


def qknorm_rms_mxcast(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6, N: int = 1,
                      B: int = 32, fmt="e4m3", codes=None, scales=None, rinv=None,
                      want_rinv: bool = False, stream=None) -> "MxOut":
    """Layerwise QK-RMSNorm of x [T, H] split into N cluster shards, written
    as an MX / NVFP4 block cast (codes, scales) instead of bf16 rows.
    Returns MxOut(codes, scales, rinv or None, None)."""
    _need_cuda("x", x, torch.bfloat16)
    _need_cuda("gamma", gamma, torch.float32)
    T, H = x.shape
    f = _fmt(fmt)
    codes, scales, rinv, _ = _mx_outputs(x, H, B, f, codes, scales, rinv, None, want_rinv,
                                         False)
    check(lib().nts_qknorm_rms_mxcast(_ptr(x), _ptr(gamma), _ptr(codes), _ptr(scales),
                                      _ptr(rinv), T, H, float(eps), int(N), int(B), f,
                                      _stream(stream)))
    return MxOut(codes, scales, rinv, None)


def qknorm_rms_qk_mxcast(q: torch.Tensor, gamma_q: torch.Tensor, k: torch.Tensor,
                         gamma_k: torch.Tensor, eps: float = 1e-6, N: int = 1, B: int = 32,
                         fmt="e4m3", out_q: Optional["MxOut"] = None,
                         out_k: Optional["MxOut"] = None, want_rinv: bool = False,
                         stream=None):
    """qknorm_rms_mxcast of Q [T, Hq] and K [T, Hk] in one launch.  out_q /
    out_k may carry preallocated (codes, scales, rinv or None) buffers.
    Returns (MxOut for Q, MxOut for K)."""
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16),
                        ("gamma_q", gamma_q, torch.float32), ("gamma_k", gamma_k, torch.float32)):
        _need_cuda(name, t, dt)
    T, Hq = q.shape
    Tk, Hk = k.shape
    if Tk != T:
        raise ValueError("q and k must have the same number of tokens")
    f = _fmt(fmt)
    bufs = []
    for x, H, o in ((q, Hq, out_q), (k, Hk, out_k)):
        c, s_, r = (o.codes, o.scales, o.rinv) if o is not None else (None, None, None)
        c, s_, r, _ = _mx_outputs(x, H, B, f, c, s_, r, None, want_rinv, False)
        bufs.append((c, s_, r))
    (cq, sq, rq), (ck, sk, rk) = bufs
    check(lib().nts_qknorm_rms_qk_mxcast(_ptr(q), _ptr(gamma_q), _ptr(cq), _ptr(sq), _ptr(rq),
                                         _ptr(k), _ptr(gamma_k), _ptr(ck), _ptr(sk), _ptr(rk),
                                         T, Hq, Hk, float(eps), int(N), int(B), f,
                                         _stream(stream)))
    return MxOut(cq, sq, rq, None), MxOut(ck, sk, rk, None)


def qknorm_rms_qk(q: torch.Tensor, gamma_q: torch.Tensor, k: torch.Tensor,
                  gamma_k: torch.Tensor, eps: float = 1e-6, N: int = 1,
                  out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None,
                  rinv_q: Optional[torch.Tensor] = None, rinv_k: Optional[torch.Tensor] = None,
                  want_rinv: bool = False, stream=None):
    """Layerwise QK-RMSNorm of Q [T, Hq] and K [T, Hk] in one launch.
    Returns (yq, yk, rinv_q or None, rinv_k or None)."""
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16),
                        ("gamma_q", gamma_q, torch.float32), ("gamma_k", gamma_k, torch.float32)):
        _need_cuda(name, t, dt)
    T, Hq = q.shape
    Tk, Hk = k.shape
    if Tk != T:
        raise ValueError("q and k must have the same number of tokens")
    out_q = torch.empty_like(q) if out_q is None else out_q
    out_k = torch.empty_like(k) if out_k is None else out_k
    if want_rinv:
        rinv_q = torch.empty(T, device=q.device, dtype=torch.float32) if rinv_q is None else rinv_q
        rinv_k = torch.empty(T, device=q.device, dtype=torch.float32) if rinv_k is None else rinv_k
    check(lib().nts_qknorm_rms_qk(_ptr(q), _ptr(gamma_q), _ptr(out_q), _ptr(rinv_q), _ptr(k),
                                  _ptr(gamma_k), _ptr(out_k), _ptr(rinv_k), T, Hq, Hk,
                                  float(eps), int(N), _stream(stream)))
    return out_q, out_k, rinv_q, rinv_k


def _mx_outputs(x, D, B, fmt, codes, scales, rinv, amax, want_rinv, want_amax):
    T = x.shape[0]
    if codes is None:
        codes = torch.empty(T, codes_row_bytes(D, fmt), device=x.device, dtype=torch.uint8)
    if scales is None:
        scales = torch.empty(T, D // B, device=x.device, dtype=torch.uint8)
    if rinv is None and want_rinv:
        rinv = torch.empty(T, device=x.device, dtype=torch.float32)
    if amax is None and want_amax:
        amax = torch.empty(T, D // B, device=x.device, dtype=torch.float32)
    _need_cuda("codes", codes, torch.uint8)
    _need_cuda("scales", scales, torch.uint8)
    if rinv is not None:
        _need_cuda("rinv", rinv, torch.float32)
    if amax is not None:
        _need_cuda("amax", amax, torch.float32)
    return codes, scales, rinv, amax


def rmsnorm_mxcast(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                   B: int = 32, fmt="e4m3", codes=None, scales=None, rinv=None, amax=None,
                   want_rinv: bool = False, want_amax: bool = False, stream=None) -> MxOut:
    """RMSNorm of x [T, D] fused with the MX cast to E4M3/E2M1 + E8M0 scales."""
    _need_cuda("x", x, torch.bfloat16)
    if gamma is not None:
        _need_cuda("gamma", gamma, torch.float32)
    T, D = x.shape
    f = _fmt(fmt)
    codes, scales, rinv, amax = _mx_outputs(x, D, B, f, codes, scales, rinv, amax,
                                            want_rinv, want_amax)
    check(lib().nts_rmsnorm_mxcast(_ptr(x), _ptr(gamma), _ptr(codes), _ptr(scales), _ptr(rinv),
                                   _ptr(amax), T, D, float(eps), int(B), f, _stream(stream)))
    return MxOut(codes, scales, rinv, amax)


def mxnorm_cast(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                B: int = 32, fmt="e4m3", p: int = 2, codes=None, scales=None, rinv=None,
                amax=None, want_rinv: bool = False, want_amax: bool = False,
                stream=None) -> MxOut:
    """MXNorm of x [T, D]: RMS estimated from the MX block absmaxes, then the
    MX cast."""
    _need_cuda("x", x, torch.bfloat16)
    if gamma is not None:
        _need_cuda("gamma", gamma, torch.float32)
    T, D = x.shape
    f = _fmt(fmt)
    codes, scales, rinv, amax = _mx_outputs(x, D, B, f, codes, scales, rinv, amax,
                                            want_rinv, want_amax)
    check(lib().nts_mxnorm_cast(_ptr(x), _ptr(gamma), _ptr(codes), _ptr(scales), _ptr(rinv),
                                _ptr(amax), T, D, float(eps), int(B), f, int(p),
                                _stream(stream)))
    return MxOut(codes, scales, rinv, amax)


def mxnorm_postround_cast(x: torch.Tensor, gamma: Optional[torch.Tensor] = None,
                          eps: float = 1e-6, B: int = 32, fmt="e4m3", p: int = 2, codes=None,
                          scales=None, rinv=None, amax=None, want_rinv: bool = False,
                          want_amax: bool = False, stream=None) -> MxOut:
    """Post-round MXNorm: the RMS estimate from E8M0-rounded block absmaxes."""
    _need_cuda("x", x, torch.bfloat16)
    if gamma is not None:
        _need_cuda("gamma", gamma, torch.float32)
    T, D = x.shape
    f = _fmt(fmt)
    codes, scales, rinv, amax = _mx_outputs(x, D, B, f, codes, scales, rinv, amax,
                                            want_rinv, want_amax)
    check(lib().nts_mxnorm_postround_cast(_ptr(x), _ptr(gamma), _ptr(codes), _ptr(scales),
                                          _ptr(rinv), _ptr(amax), T, D, float(eps), int(B), f,
                                          int(p), _stream(stream)))
    return MxOut(codes, scales, rinv, amax)


# ------------------------------------------ the operators around a projection


class BlockOut(NamedTuple):
    codes: torch.Tensor     # uint8 [T, D], or [D, Tp] transposed
    scales: torch.Tensor    # fp32, one per block of 128 values
    rinv: Optional[torch.Tensor]   # fp32 [T]


class GroupOut(NamedTuple):
    codes: torch.Tensor     # uint8 [N, K/2], the even value's code in bits 0 to 3
    scales: torch.Tensor    # bf16 [N, ceil(K/group)]


class AddNormOut(NamedTuple):
    h: torch.Tensor         # [T, D], the residual's type
    codes: torch.Tensor     # uint8 [T, D]
    scales: torch.Tensor    # fp32 [T, ceil(D/128)]
    rinv: Optional[torch.Tensor]   # fp32 [T]


# The checks, missing outputs and the call itself are in binding/marshal.cpp:
# these operators serve single tokens, where Python's share of a call would be
# the larger part of it.
#
# stream: the current one when None.  What a call makes belongs to its stream.
# On CUDA's per-thread stream, which torch has no pool for, the workspace is the
# caller's, and the outputs too unless the default stream is current.

def rope_table(P: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """The rotation table of qknorm_rope: fp32 [P, rot_dim], row pos the
    cosines of pos * base^(-2i/rot_dim), then the sines (formed on the host
    in double precision)."""
    t = torch.empty(int(P), int(rot_dim), dtype=torch.float32)
    check(lib().nts_rope_table_host(int(P), int(rot_dim), float(base), _ptr(t)))
    return t.to(device)


def qknorm_rope(q: torch.Tensor, gamma_q: torch.Tensor, k: torch.Tensor, gamma_k: torch.Tensor,
                positions: torch.Tensor, table: torch.Tensor, head_dim: int, eps: float = 1e-6,
                interleaved: bool = False, out_q: Optional[torch.Tensor] = None,
                out_k: Optional[torch.Tensor] = None, rinv_q: Optional[torch.Tensor] = None,
                rinv_k: Optional[torch.Tensor] = None, want_rinv: bool = False, stream=None):
    """Headwise QK-RMSNorm of q [T, nheads_q * head_dim] and k [T, nheads_k *
    head_dim] (bf16, rows contiguous, any row stride: columns of a packed QKV
    buffer) with the rotary position embedding of positions (int64 [T],
    negative: padding row, zeros out) by table (rope_table).  out_q may be q,
    out_k may be k.  Returns (yq, yk, rinv_q or None, rinv_k or None)."""
    return marshal().qknorm_rope(q, gamma_q, k, gamma_k, positions, table, head_dim, eps,
                                 interleaved, out_q, out_k, rinv_q, rinv_k, want_rinv, stream)


def qknorm_rope_backward(dyq: torch.Tensor, dyk: torch.Tensor, q: torch.Tensor,
                         gamma_q: torch.Tensor, k: torch.Tensor, gamma_k: torch.Tensor,
                         positions: torch.Tensor, table: torch.Tensor, head_dim: int,
                         eps: float = 1e-6, interleaved: bool = False,
                         out_dq: Optional[torch.Tensor] = None,
                         out_dk: Optional[torch.Tensor] = None,
                         dgamma_q: Optional[torch.Tensor] = None,
                         dgamma_k: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of qknorm_rope: dyq and dyk are the gradients of its outputs, q
    and k its inputs.  out_dq and out_dk may be columns of one packed buffer.
    Returns (dq, dk, dgamma_q, dgamma_k), the gains' gradients in fp32
    [head_dim].  Without a workspace (uint8, rope_backward_workspace bytes)
    one is taken from torch's allocator for the call."""
    return marshal().qknorm_rope_backward(dyq, dyk, q, gamma_q, k, gamma_k, positions, table,
                                          head_dim, eps, interleaved, out_dq, out_dk, dgamma_q,
                                          dgamma_k, workspace, stream)


def rope_backward_workspace(head_dim: int) -> int:
    """Workspace bytes of qknorm_rope_backward."""
    n = ctypes.c_int64()
    check(lib().nts_qknorm_rope_backward_workspace(int(head_dim), ctypes.byref(n)))
    return n.value


def rope_axes(sections, cyclic: bool = False) -> bytes:
    """The axis of each pair for qknorm_rope_axes: sections[a] pairs turn by axis
    a, in runs one axis after another, or (cyclic) the axes taking the pairs in
    turn, for as long as the shorter ones last."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= 4 or min(left) < 0:
        raise ValueError("sections must be 1 to 4 counts of pairs")
    if not cyclic:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    order = []
    while any(left):
        for a, n in enumerate(left):
            if n > 0:
                order.append(a)
                left[a] -= 1
    return bytes(order)


def qknorm_rope_axes(q: torch.Tensor, gamma_q: torch.Tensor, k: torch.Tensor,
                     gamma_k: torch.Tensor, positions: torch.Tensor, table: torch.Tensor,
                     axes: bytes, head_dim: int, eps: float = 1e-6, interleaved: bool = False,
                     out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None,
                     rinv_q: Optional[torch.Tensor] = None, rinv_k: Optional[torch.Tensor] = None,
                     want_rinv: bool = False, stream=None):
    """qknorm_rope for tokens with a position on each of 1 to 4 axes: positions
    is int64 [T, A] with any strides (a transposed [A, T] too), axes the axis of
    each of the rot_dim / 2 pairs (rope_axes).  A token with a negative position on
    any axis is a padding row.  Pair i's angle is column i of the table, so a
    table's columns may hold any frequencies: rope_table's, or those of one
    rope_table per axis side by side (their cosines, then their sines)."""
    return marshal().qknorm_rope_axes(q, gamma_q, k, gamma_k, positions, table, head_dim, eps,
                                      interleaved, out_q, out_k, rinv_q, rinv_k, want_rinv, stream,
                                      axes)


def qknorm_rope_axes_backward(dyq: torch.Tensor, dyk: torch.Tensor, q: torch.Tensor,
                              gamma_q: torch.Tensor, k: torch.Tensor, gamma_k: torch.Tensor,
                              positions: torch.Tensor, table: torch.Tensor, axes: bytes,
                              head_dim: int, eps: float = 1e-6, interleaved: bool = False,
                              out_dq: Optional[torch.Tensor] = None,
                              out_dk: Optional[torch.Tensor] = None,
                              dgamma_q: Optional[torch.Tensor] = None,
                              dgamma_k: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of qknorm_rope_axes; everything else as qknorm_rope_backward
    (its workspace too)."""
    return marshal().qknorm_rope_axes_backward(dyq, dyk, q, gamma_q, k, gamma_k, positions, table,
                                               head_dim, eps, interleaved, out_dq, out_dk, dgamma_q,
                                               dgamma_k, workspace, stream, axes)


def rmsnorm_blockcast(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                      codes=None, scales=None, rinv=None, want_rinv: bool = False,
                      stream=None) -> BlockOut:
    """RMSNorm of x [T, D] (bf16) fused with the cast to E4M3 codes with an
    fp32 scale per 128 values: BlockOut(codes [T, D], scales [T, ceil(D/128)],
    rinv or None)."""
    return BlockOut(*marshal().rmsnorm_blockcast(x, gamma, eps, codes, scales, rinv, want_rinv,
                                                 stream))


def add_rmsnorm_blockcast(x: torch.Tensor, residual: torch.Tensor,
                          gamma: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          out: Optional[torch.Tensor] = None, codes=None, scales=None, rinv=None,
                          want_rinv: bool = False, stream=None) -> AddNormOut:
    """rmsnorm_blockcast of h = x + residual, both [T, D], x in bf16 and the
    residual in bf16 or fp32, h in the residual's type and written too:
    AddNormOut(h, codes [T, D], scales [T, ceil(D/128)], rinv or None).  out (h)
    may be the residual, or x when that has its type."""
    return AddNormOut(*marshal().add_rmsnorm_blockcast(x, residual, gamma, eps, out, codes, scales,
                                                       rinv, want_rinv, stream))


def add_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, rinv: torch.Tensor,
                         gamma: Optional[torch.Tensor] = None,
                         dres: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                         out_x: Optional[torch.Tensor] = None,
                         dgamma: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of add_rmsnorm_blockcast, the cast taken as exact: dy (bf16) is
    the gradient of the normalized rows, h and rinv the forward pass's, dres the
    gradient of h from the layers behind (h's type).  Returns (the gradient of
    the residual and of x in h's type, the same in bf16 when h is fp32 or None,
    gamma's gradient in fp32 [D] or None).  out may be dres or h, or dy when that
    has its type; out_x may be dy.  Without a workspace (uint8,
    add_rmsnorm_backward_workspace bytes) one is taken from torch's allocator for
    the call."""
    return marshal().add_rmsnorm_backward(dy, h, rinv, gamma, dres, out, out_x, dgamma, workspace,
                                          stream)


def add_rmsnorm_backward_workspace(D: int) -> int:
    """Workspace bytes of add_rmsnorm_backward."""
    n = ctypes.c_int64()
    check(lib().nts_add_rmsnorm_backward_workspace(int(D), ctypes.byref(n)))
    return n.value


def blockcast(x: torch.Tensor, block_rows: int = 1, codes=None, scales=None,
              stream=None) -> BlockOut:
    """Cast of x [T, D] (bf16) to E4M3 codes with an fp32 scale per block of
    block_rows x 128 values (1: activations, 128: weights):
    BlockOut(codes [T, D], scales [ceil(T/block_rows), ceil(D/128)], None)."""
    return BlockOut(*marshal().blockcast(x, block_rows, codes, scales, stream))


def blockcast_t(x: torch.Tensor, codes=None, scales=None, stream=None) -> BlockOut:
    """The transpose of x [T, D] (bf16) as E4M3 codes with an fp32 scale per
    128 tokens of a column: BlockOut(codes [D, Tp], scales [D, ceil(T/128)],
    None), Tp = T rounded up to a multiple of 16 (zero codes beyond T)."""
    return BlockOut(*marshal().blockcast_t(x, codes, scales, stream))


def gemm_blockscaled(a_codes: torch.Tensor, a_scales: torch.Tensor, w_codes: torch.Tensor,
                     w_scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                     out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """Y = A W^T of E4M3 operands (uint8 or float8_e4m3fn) with an fp32 scale
    per 128 values along K: a_codes [M, K] with a_scales [M, ceil(K/128)],
    w_codes [N, K] with w_scales [ceil(N/128), ceil(K/128)] (128 x 128 blocks)
    or [N, ceil(K/128)].  Returns Y [M, N], bf16 or fp32 (out_dtype, or out's)."""
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise ValueError(f"the output must be bfloat16 or float32, got {out_dtype}")
    return marshal().gemm_blockscaled(a_codes, a_scales, w_codes, w_scales, out,
                                      out_dtype is torch.float32, stream)


_W4_NAMES = {"e2m1": 0, "int4": 1}


def _w4(fmt) -> int:
    try:
        return _W4_NAMES[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"4-bit weights are 'e2m1' or 'int4', got {fmt!r}") from None


def groupcast(w: torch.Tensor, group: int = 32, fmt="e2m1", device="cuda") -> GroupOut:
    """Weights w [N, K] (bf16, finite) as 4-bit codes with a bf16 scale per group
    of 32, 64 or 128 values along K, formed on the host:
    GroupOut(codes uint8 [N, K/2], scales [N, ceil(K/group)])."""
    if w.dtype != torch.bfloat16 or w.dim() != 2:
        raise ValueError("w must be a matrix of torch.bfloat16")
    N, K = w.shape
    w = w.detach().to("cpu").contiguous()
    f, g = _w4(fmt), int(group)
    codes = torch.empty(N, K // 2, dtype=torch.uint8)
    scales = torch.empty(N, -(-K // g) if g > 0 else 0, dtype=torch.bfloat16)
    check(lib().nts_groupcast_host(_ptr(w), _ptr(codes), _ptr(scales), N, K, g, f))
    return GroupOut(codes.to(device), scales.to(device))


def gemv_groupscaled(a: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor,
                     a_scales: Optional[torch.Tensor] = None, group: int = 32, fmt="e2m1",
                     out: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                     stream=None) -> torch.Tensor:
    """Y = A W^T of few rows with 4-bit weights (groupcast): w_codes uint8
    [N, K/2] with w_scales bf16 [N, ceil(K/group)], fmt "e2m1" or "int4".  a [M, K]
    is bf16 (contiguous rows, any row stride), or E4M3 codes (uint8 or
    float8_e4m3fn) with a_scales fp32 [M, ceil(K/128)] (a BlockOut's).  Returns
    Y [M, N], bf16 or fp32 (out_dtype, or out's).  Scales of w are at most 2^102
    in magnitude; from 9 rows on gemm_blockscaled's weights of 8 bits take less
    time."""
    if out_dtype is not torch.bfloat16 and out_dtype is not torch.float32:
        raise ValueError(f"the output must be bfloat16 or float32, got {out_dtype}")
    return marshal().gemv_groupscaled(a, w_codes, w_scales, a_scales, group, _w4(fmt), out,
                                      out_dtype is torch.float32, stream)


def mxnorm_correction(B: int, p: int) -> float:
    c = ctypes.c_double()
    check(lib().nts_mxnorm_correction(int(B), int(p), ctypes.byref(c)))
    return c.value


def check_status(stream=None) -> None:
    """Synchronize the stream and raise if a kernel timed out or failed."""
    check(lib().nts_check_status(_stream(stream)))


# ----------------------------------------------------------- host-buffer forms

def _need_host(name: str, t: torch.Tensor) -> None:
    if t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous host tensor")


def qknorm_rms_host(x_host, gamma_dev, y_host, x_dev, y_dev, eps=1e-6, N=1, rinv_host=None,
                    rinv_dev=None, stream=None) -> None:
    """Enqueue H2D copy of x, the kernel, and D2H copies of y (and rinv)."""
    _need_host("x_host", x_host)
    _need_host("y_host", y_host)
    T, H = x_host.shape
    check(lib().nts_qknorm_rms_host(_ptr(x_host), _ptr(gamma_dev), _ptr(y_host), _ptr(rinv_host),
                                    _ptr(x_dev), _ptr(y_dev), _ptr(rinv_dev), T, H, float(eps),
                                    int(N), _stream(stream)))


def qknorm_rms_qk_host(q_host, gamma_q_dev, yq_host, k_host, gamma_k_dev, yk_host, q_dev,
                       yq_dev, k_dev, yk_dev, eps=1e-6, N=1, stream=None) -> None:
    """Enqueue the H2D copies of q and k, the one launch normalizing both,
    and the D2H copies of yq and yk."""
    for name, t in (("q_host", q_host), ("yq_host", yq_host), ("k_host", k_host),
                    ("yk_host", yk_host)):
        _need_host(name, t)
    T, Hq = q_host.shape
    Tk, Hk = k_host.shape
    if Tk != T:
        raise ValueError("q and k must have the same number of tokens")
    check(lib().nts_qknorm_rms_qk_host(
        _ptr(q_host), _ptr(gamma_q_dev), _ptr(yq_host), _ptr(k_host), _ptr(gamma_k_dev),
        _ptr(yk_host), _ptr(q_dev), _ptr(yq_dev), _ptr(k_dev), _ptr(yk_dev), T, Hq, Hk,
        float(eps), int(N), _stream(stream)))


def rmsnorm_mxcast_host(x_host, gamma_dev, codes_host, scales_host, x_dev, codes_dev,
                        scales_dev, eps=1e-6, B=32, fmt="e4m3", stream=None) -> None:
    _need_host("x_host", x_host)
    T, D = x_host.shape
    check(lib().nts_rmsnorm_mxcast_host(_ptr(x_host), _ptr(gamma_dev), _ptr(codes_host),
                                        _ptr(scales_host), _ptr(x_dev), _ptr(codes_dev),
                                        _ptr(scales_dev), T, D, float(eps), int(B), _fmt(fmt),
                                        _stream(stream)))


def mxnorm_cast_host(x_host, gamma_dev, codes_host, scales_host, x_dev, codes_dev, scales_dev,
                     eps=1e-6, B=32, fmt="e4m3", p=2, stream=None) -> None:
    _need_host("x_host", x_host)
    T, D = x_host.shape
    check(lib().nts_mxnorm_cast_host(_ptr(x_host), _ptr(gamma_dev), _ptr(codes_host),
                                     _ptr(scales_host), _ptr(x_dev), _ptr(codes_dev),
                                     _ptr(scales_dev), T, D, float(eps), int(B), _fmt(fmt),
                                     int(p), _stream(stream)))


# ------------------------------------------------------------------ tuning

def mxnorm_cast_host_noalloc(x_host, gamma_host, codes_host, scales_host, eps=1e-6, B=32,
                             fmt="e4m3", p=2, stream=None) -> None:
    """MXNorm of host rows with the library's fixed device staging (no
    caller-owned device buffers; calls that overlap in time race)."""
    _need_host("x_host", x_host)
    T, D = x_host.shape
    if gamma_host is not None:
        _need_host("gamma_host", gamma_host)
    check(lib().nts_mxnorm_cast_host_noalloc(_ptr(x_host), _ptr(gamma_host), _ptr(codes_host),
                                             _ptr(scales_host), T, D, float(eps), int(B),
                                             _fmt(fmt), int(p), _stream(stream)))


def set_tuning(vpt=0, rows=0, stages=0, grid=0, smem_budget=0) -> None:
    check(lib().nts_debug_set_tuning(int(vpt), int(rows), int(stages), int(grid),
                                     int(smem_budget)))


def set_wait_limit_ns(ns: int) -> None:
    check(lib().nts_debug_set_wait_limit_ns(int(ns)))


def set_schedule(dynamic: bool) -> None:
    check(lib().nts_debug_set_schedule(1 if dynamic else 0))


def set_direct(on: bool) -> None:
    check(lib().nts_debug_set_direct(1 if on else 0))


def check_nvfp4_scale() -> tuple:
    """(code mismatches, quotient mismatches) of the kernels' NVFP4 block
    scale against the IEEE-division route over every non-negative fp32
    absmax (nts_debug_check_nvfp4_scale); runs on the current device."""
    a, b = ctypes.c_uint64(0), ctypes.c_uint64(0)
    check(lib().nts_debug_check_nvfp4_scale(ctypes.byref(a), ctypes.byref(b)))
    return int(a.value), int(b.value)


def set_host_chunks(max_chunks: int = 0, min_chunk_bytes: int = 0) -> None:
    """Chunking of the host-buffer forms (0, 0 = defaults); results do not
    depend on it (nts_debug_set_host_chunks)."""
    check(lib().nts_debug_set_host_chunks(int(max_chunks), int(min_chunk_bytes)))


def inject_failure(status: str = "CUDA", count: int = 1) -> None:
    """The next `count` launches fail with NTS_ERR_<status> (CUDA,
    UNSUPPORTED or TIMEOUT) without touching the device; count=0 turns the
    hook off (nts_debug_inject_failure)."""
    codes = {"CUDA": 3, "UNSUPPORTED": 2, "TIMEOUT": 4}
    check(lib().nts_debug_inject_failure(codes[status], int(count)))


def set_pdl(on: bool) -> None:
    """Launch with programmatic stream serialization (default on); results
    do not depend on it (nts_debug_set_pdl)."""
    check(lib().nts_debug_set_pdl(1 if on else 0))


def check_e8m0() -> int:
    """Absmaxes whose E8M0 exponent, as the kernels form it, differs from
    the field-by-field definition (nts_debug_check_e8m0); 0 when right."""
    a = ctypes.c_uint64(0)
    check(lib().nts_debug_check_e8m0(ctypes.byref(a)))
    return int(a.value)


def set_missing_tx(nbytes: int) -> None:
    check(lib().nts_debug_set_missing_tx(int(nbytes)))
