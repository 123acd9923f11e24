"""MXFP4: E2M1 codes with one E8M0 scale byte per 32 values, and products of them.

Test infrastructure (see the package docstring).

[CMP] holds routed experts at 4 bits without fixing a format; the reading is
the OCP microscaling format MXFP4 v1.0, which gfx950's matrix cores take as
it is: element levels 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign bit, scale 2^(b-127)
for byte b, 255 = NaN.  The conversion's scale exponent is floor(log2(amax)) - 2
(2 is the exponent of the largest power of two among the levels), clamped to
E8M0's -127.  Readings taken where the format leaves it open: a block of zeros
gets the scale 1; a block with an infinity or a NaN gets the NaN scale and
codes 0; a value half way between two levels takes the even code.
"""
from __future__ import annotations

import math

import numpy as np

MX_BLOCK = 32
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx_scale(byte) -> np.ndarray:
    """2^(b - 127) in float64, NaN for 255."""
    b = np.asarray(byte, dtype=np.int64)
    return np.where(b == 255, np.nan, np.exp2((b - 127).astype(np.float64)))


def mx_quant(values):
    """fp32 (or bf16 held in fp32) rows [R, K] -> (packed codes uint8 [R, K/2], scale bytes uint8 [R, K/32])."""
    v = np.asarray(values, dtype=np.float64)
    R, K = v.shape
    g = v.reshape(R, K // MX_BLOCK, MX_BLOCK)
    codes = np.zeros(g.shape, dtype=np.uint8)
    byte = np.zeros(g.shape[:2], dtype=np.uint8)
    with np.errstate(invalid="ignore"):
        top = np.abs(g).max(-1)
    finite = np.isfinite(g).all(-1)
    _, e = np.frexp(np.where(finite, top, 1.0))                   # top = m 2^e, 0.5 <= m < 1
    byte[:] = np.maximum(e - 1 - 2 + 127, 0)
    byte[finite & (top == 0)] = 127
    byte[~finite] = 255
    # distance to each level; argmin takes the lowest code, so odd codes are looked at after the even ones
    look = np.array([0, 2, 4, 6, 1, 3, 5, 7])
    a = np.abs(np.where(finite[..., None], g, 0.0)) / mx_scale(np.where(finite, byte, 127))[..., None]
    for r in range(R):                                            # row by row to bound memory
        d = np.abs(np.minimum(a[r], 6.0)[..., None] - E2M1[look])
        codes[r] = look[np.argmin(d, -1)]
    codes |= np.where(np.signbit(g) & finite[..., None], 8, 0).astype(np.uint8)
    c = codes.reshape(R, K // 2, 2)
    return c[..., 0] | (c[..., 1] << 4), byte


def mx_values(packed, scales) -> np.ndarray:
    """float64 values [..., K] of packed codes [..., K/2] and scale bytes [..., K/32]."""
    p = np.asarray(packed, dtype=np.uint8)
    nib = np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], p.shape[-1] * 2)
    mag = E2M1[nib & 7]
    s = np.repeat(mx_scale(scales), MX_BLOCK, axis=-1)
    return np.where(nib & 8, -mag, mag) * s


def mx_product(x, w):
    """(x @ w^T, |x| @ |w|^T) in float64: the sums and what rounding errors are measured against."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def route_sort(ids, E):
    """(order [P], inverse [M, k], offsets [E+1]) of pairs by expert, stable, -1 for none."""
    ids = np.asarray(ids)
    M, k = ids.shape
    flat = ids.reshape(-1)
    order = [p for e in range(E) for p in np.nonzero(flat == e)[0].tolist()]
    inverse = np.full(M * k, -1, dtype=np.int32)
    inverse[order] = np.arange(len(order), dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]).astype(np.int32)
    full = np.full(M * k, -1, dtype=np.int32)
    full[:len(order)] = order
    return full, inverse.reshape(M, k), offsets


def route_dispatch(x, order, k):
    """xs[r] = x[order[r] // k], zeros where order is -1."""
    o = np.asarray(order)
    return np.where((o >= 0)[:, None], np.asarray(x)[np.maximum(o, 0) // k], 0.0)


def route_combine(ys, inverse, w):
    """(sum_s w ys[inverse], sum_s |w ys[inverse]|) in float64."""
    ys, inv = np.asarray(ys, dtype=np.float64), np.asarray(inverse)
    t = np.where((inv >= 0)[..., None], ys[np.maximum(inv, 0)] * np.asarray(w, dtype=np.float64)[..., None], 0.0)
    return t.sum(1), np.abs(t).sum(1)


def route_combine_grad(dy, ys, order, inverse, w):
    """dys [P, H], dw [M, k] and the sum of |dy ys| behind each dw, in float64."""
    dy, ys = np.asarray(dy, dtype=np.float64), np.asarray(ys, dtype=np.float64)
    M, k = np.asarray(inverse).shape
    wf = np.asarray(w, dtype=np.float64).reshape(-1)
    dys = np.zeros_like(ys)
    dw, mag = np.zeros(M * k), np.zeros(M * k)
    for r, p in enumerate(np.asarray(order).tolist()):
        if p >= 0:
            dys[r] = wf[p] * dy[p // k]
            dw[p] = math.fsum(dy[p // k] * ys[r])
            mag[p] = np.abs(dy[p // k] * ys[r]).sum()
    return dys, dw.reshape(M, k), mag.reshape(M, k)
