"""E2M1 codes with an E4M3 scale per 16 dims: the codec, the quantization rule
and the physical pages of a 4-bit cache (include/kvq.h), in float64 numpy.

Test infrastructure.  A code's low three bits count the magnitudes 0, 0.5, 1,
1.5, 2, 3, 4, 6 (exponent bias 1, one mantissa bit, no infinity, no NaN), bit 3
is the sign.
"""
from __future__ import annotations

import numpy as np

from . import e4m3

BLOCK = 16
P = 16


def decode_code(code: int) -> float:
    """Value of one code from its sign / exponent / mantissa fields."""
    e, m = (code >> 1) & 3, code & 1
    size = m / 2 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)
    return -size if code & 8 else size


VALUES = np.array([decode_code(c) for c in range(16)])


def decode(codes) -> np.ndarray:
    return VALUES[np.asarray(codes)]


def encode(values) -> np.ndarray:
    """Nearest code of each float32 value, ties to the even code, beyond 6 to
    6, the sign kept: |v| is compared with the midpoints of neighbours."""
    v = np.asarray(values, np.float32).astype(np.float64)
    a = np.abs(v)
    code = np.zeros(v.shape, np.uint8)
    for i in range(7):
        mid = (VALUES[i] + VALUES[i + 1]) / 2
        code = np.where((a > mid) | ((a == mid) & (i % 2 == 1)), i + 1, code).astype(np.uint8)
    return code | (np.signbit(v).astype(np.uint8) << 3)


def quantize(x, scale):
    """x float32 [..., D], scale float32 broadcastable to [...]: (codes [..., D],
    E4M3 block scales [..., D / 16])."""
    x = np.asarray(x, np.float32)
    blocks = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    s = np.broadcast_to(np.asarray(scale, np.float32), x.shape[:-1])[..., None]
    amax = np.abs(blocks).max(-1)
    sb = e4m3.encode(amax / (np.float32(6) * s))
    step = (e4m3.decode(sb).astype(np.float32) * s)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        codes = np.where(step > 0, encode(blocks / step), 0).astype(np.uint8)
    return codes.reshape(x.shape), sb


def dequantize(codes, sb) -> np.ndarray:
    """Values [..., D] without the head's scale (exact)."""
    v = decode(codes)
    return (v.reshape(*v.shape[:-1], v.shape[-1] // BLOCK, BLOCK) * e4m3.decode(sb)[..., None]).reshape(v.shape)


def v_byte(t: int, j: int) -> int:
    """Place of dims 2j, 2j + 1 of token t among a V page's code bytes."""
    hi, c, lo = t // 8, (t % 8) // 2, t % 2
    h, b, r = j // 32, (j // 8) % 4, j % 8
    return h * 512 + r * 64 + c * 16 + b * 4 + hi * 2 + lo


def v_scale_byte(t: int, i: int) -> int:
    """Place of the scale of block i of token t among a V page's scale bytes."""
    hi, c, lo = t // 8, (t % 8) // 2, t % 2
    return (i // 4) * 64 + c * 16 + (i % 4) * 4 + hi * 2 + lo


def pages(k, ks, v, vs):
    """Logical codes [nb, H, 16, D] and scales [nb, H, 16, D / 16] of K and V
    -> (K pages, V pages) [nb, H, page bytes]."""
    nb, H, _, D = k.shape

    def pairs(c):
        return c[..., 0::2] | (c[..., 1::2] << 4)

    kd = np.concatenate([pairs(k).reshape(nb, H, -1), ks.reshape(nb, H, -1)], -1)
    vd = np.zeros_like(kd)
    vp = pairs(v)
    for t in range(P):
        for j in range(D // 2):
            vd[..., v_byte(t, j)] = vp[..., t, j]
        for i in range(D // BLOCK):
            vd[..., P * D // 2 + v_scale_byte(t, i)] = vs[..., t, i]
    return kd, vd


def from_pages(kd, vd, D):
    """The reverse of pages()."""
    nb, H = kd.shape[:2]
    n = P * D // 2

    def split(b):
        return np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)

    k, ks = split(kd[..., :n].reshape(nb, H, P, D // 2)), kd[..., n:].reshape(nb, H, P, D // BLOCK)
    at = np.array([[v_byte(t, j) for j in range(D // 2)] for t in range(P)])
    sat = np.array([[n + v_scale_byte(t, i) for i in range(D // BLOCK)] for t in range(P)])
    return k, ks, split(vd[..., at]), vd[..., sat]


def attend(q, k, v, sm_scale):
    """softmax(q k^T sm_scale) v of one KV head in float64: q [g, D], k, v [n,
    D] values; returns (out [g, D], sum_j p_j |v_j|), zeros where n is 0."""
    if len(k) == 0:
        return np.zeros_like(q), np.zeros_like(q)
    s = q @ k.T * sm_scale
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return p @ v, p @ np.abs(v)
