"""4-bit weights with group scales, written from the format definition.

TEST INFRASTRUCTURE ONLY (see the package docstring).

``W[n,k] = (c[n,k] - z[n,k//G]) * d[n,k//G]`` with codes ``c`` and zero points
``z`` in 0..15 and f16 scales ``d``; two codes to a byte, the even k in the low
half.  Without zero points z = 8.
"""
import numpy as np

from . import f16


def unpack(codes):
    """Codes uint8 [..., K/2] -> [..., K]."""
    out = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=np.uint8)
    out[..., 0::2] = codes & 15
    out[..., 1::2] = codes >> 4
    return out


def pack(c):
    """Codes [..., K] (0..15) -> uint8 [..., K/2]."""
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def dequant(codes, scale_bits, zeros, group):
    """W in float64."""
    c = unpack(codes).astype(np.float64)
    z = np.full(scale_bits.shape, 8.0) if zeros is None else (zeros & 15).astype(np.float64)
    return (c - np.repeat(z, group, -1)) * np.repeat(f16.bits_to_float(scale_bits), group, -1)


def quantize(w, group, with_zeros):
    """The producer's formula in float32, step by step: (codes, scale bits, zeros or None)."""
    w = np.asarray(w, dtype=np.float32)
    g = w.reshape(w.shape[:-1] + (w.shape[-1] // group, group))
    lo = np.minimum(g.min(-1), np.float32(0))
    hi = np.maximum(g.max(-1), np.float32(0))
    want = (hi - lo) / np.float32(15) if with_zeros else np.maximum(hi, -lo) / np.float32(7)
    d = np.minimum(want, np.float32(65504)).astype(np.float16)
    df = d.astype(np.float32)
    safe = np.where(df > 0, df, np.float32(1))
    if with_zeros:
        z = np.where(df > 0, np.clip(np.rint(-lo / safe), 0, 15), 0).astype(np.float32)
    else:
        z = np.full(df.shape, 8, dtype=np.float32)
    q = np.clip(np.rint(g / safe[..., None]) + z[..., None], 0, 15)
    q = np.where(df[..., None] > 0, q, z[..., None]).astype(np.uint8).reshape(w.shape)
    return pack(q), d.view(np.uint16), z.astype(np.uint8) if with_zeros else None


def gemm(x, W):
    return np.asarray(x, np.float64) @ W.T


def gemm_abs(x, W):
    """sum_k |x[m,k] W[n,k]|: the scale of the error bounds."""
    return np.abs(np.asarray(x, np.float64)) @ np.abs(W).T
