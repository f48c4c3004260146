"""Plain fp64 forms of the operators around a QKV projection, and the bounds
their fp32 kernels have to keep.

Roundings count half a step each: U32 = 2^-24, bf16 2^-8, E4M3 2^-4 (2^-10
absolute below its normal range).  A sum of n fp32 terms is off by at most
n U32 times the sum of the terms' magnitudes, in any order.
"""
from __future__ import annotations

import torch

U32 = 2.0 ** -24
UBF16 = 2.0 ** -8
BLOCK = 128


def rope_pairs(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(v, c, s, rot, interleaved, back=False):
    a, b = rope_pairs(rot, interleaved)
    c, s = c[:, None, :], (-s if back else s)[:, None, :]
    y = v.clone()
    y[..., a], y[..., b] = v[..., a] * c - v[..., b] * s, v[..., b] * c + v[..., a] * s
    return y


def rotate_abs(v, c, s, rot, interleaved):
    """Sum of the magnitudes of each rotated value's two products."""
    a, b = rope_pairs(rot, interleaved)
    v, c, s = v.abs(), c.abs()[:, None, :], s.abs()[:, None, :]
    y = v.clone()
    y[..., a], y[..., b] = v[..., a] * c + v[..., b] * s, v[..., b] * c + v[..., a] * s
    return y


def table_rows(pos, table):
    rot = table.shape[1]
    keep = (pos >= 0) & (pos < table.shape[0])
    rows = table.double()[torch.where(keep, pos, torch.zeros_like(pos))]
    return rows[:, :rot // 2], rows[:, rot // 2:], keep


def rope_forward(x, gamma, pos, table, d, eps, interleaved):
    """(y, rinv, bound on |kernel - y|), fp64 on the CPU."""
    T, rot = x.shape[0], table.shape[1]
    c, s, keep = table_rows(pos, table)
    v = torch.where(keep[:, None], x.double(), 0.0).reshape(T, -1, d)
    rinv = (v.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = v * gamma.double() * rinv
    y = rotate(n, c, s, rot, interleaved) * keep[:, None, None]
    # rinv: a sum of d squares, halved by the root, and a few roundings (the
    # hardware's reciprocal root is within 2 of them); then two products and
    # a rotation of two products and a sum
    c32 = (d / 2 + 12) * U32
    room = c32 * rotate_abs(n, c, s, rot, interleaved) * keep[:, None, None]
    bound = UBF16 * y.abs() + (1 + UBF16) * room + 2.0 ** -133
    return y.reshape(T, -1), (rinv[..., 0] * keep[:, None]), bound.reshape(T, -1)


def rope_backward(dy, x, gamma, pos, table, d, eps, interleaved):
    """(dx, dgamma, bound on dx, bound on dgamma), fp64 on the CPU."""
    T, rot = x.shape[0], table.shape[1]
    c, s, keep = table_rows(pos, table)
    v = torch.where(keep[:, None], x.double(), 0.0).reshape(T, -1, d)
    dyv = torch.where(keep[:, None], dy.double(), 0.0).reshape(T, -1, d)
    gm = gamma.double()
    rinv = (v.square().mean(-1, keepdim=True) + eps).rsqrt()
    g = rotate(dyv, c, s, rot, interleaved, back=True)
    ga = rotate_abs(dyv, c, s, rot, interleaved)
    u, ua = g * gm, ga * gm.abs()
    dx = (u - v * rinv.square() * (u * v).mean(-1, keepdim=True)) * rinv
    dxa = (ua + v.abs() * rinv.square() * (ua * v.abs()).mean(-1, keepdim=True)) * rinv
    # three factors rinv (d/2 + 6 roundings each), a sum of d products, and
    # ten more roundings
    bx = UBF16 * dx.abs() + (1 + UBF16) * (2.5 * d + 28) * U32 * dxa + 2.0 ** -133
    terms = T * v.shape[1]
    bg = (terms + d / 2 + 16) * U32 * (ga * v.abs() * rinv).sum((0, 1)) + 2.0 ** -126
    return dx.reshape(T, -1), (g * v * rinv).sum((0, 1)), bx.reshape(T, -1), bg


def block_scales(w, rows):
    """fp32 scales of w's rows x 128 blocks, by the definition's fp32 steps."""
    T, D = w.shape
    nt, nd = -(-T // rows), -(-D // BLOCK)
    p = torch.zeros(nt * rows, nd * BLOCK, dtype=torch.float32)
    p[:T, :D] = w
    a = p.reshape(nt, rows, nd, BLOCK).abs().amax((1, 3))
    return a.clamp_min(2.0 ** -100) / torch.tensor(448.0)


def spread(scales, rows, T, D):
    return scales.repeat_interleave(rows, 0)[:T].repeat_interleave(BLOCK, 1)[:, :D]


def block_codes(w, scales, rows):
    """E4M3 codes (uint8) of fp32 w by its fp32 scales; fp32 steps."""
    inv = torch.tensor(1.0) / scales
    q = w * spread(inv, rows, *w.shape)
    return q.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def e4m3(codes):
    return codes.view(torch.float8_e4m3fn).double()


def gemm(a, sa, w, sw, rows):
    """(Y, sum of the products' magnitudes), fp64 on the operands' device."""
    A = e4m3(a) * spread(sa.double(), 1, *a.shape)
    W = e4m3(w) * spread(sw.double(), rows, *w.shape)
    return A @ W.t(), A.abs() @ W.abs().t()


def gemm_bound(y, mag, K, fp32_out):
    # products of two E4M3 values are exact in fp32; 128 of them are added in
    # fp32 (counted as truncations: a whole step each), then scaled by the
    # rounded product of two scales and added over the blocks
    blocks = -(-K // BLOCK)
    room = (128 * 2 + blocks + 4) * U32 * mag
    return room + 2.0 ** -126 if fp32_out else UBF16 * y.abs() + (1 + UBF16) * room + 2.0 ** -133
