"""Oracle: head norms and rotation, the 4-bit key/value cache and attention over it, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Written row by row from the definitions in
the public header; the block format (levels, nearest level, ties, absmax below 2^-126) is the
weight quantizer's, taken from the weight oracle.  bf16 values travel as uint16 bit patterns.
"""
from __future__ import annotations

import functools

import numpy as np

from . import nf4

NAN16 = 0x7FC0


def f64(u16) -> np.ndarray:
    return (np.asarray(u16, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


# ---- norm of each head and rotation by position ----------------------------------------------------------
def _angles(pos, freq):
    return np.asarray(pos, np.float64)[:, None] * np.asarray(freq, np.float32).astype(np.float64)


def rotate(x, pos, freq, interleaved=False, sign=1.0):
    """x [rows][heads][D] float64; pairs (i, i + R/2), or (2i, 2i + 1), turned by sign * pos * freq[i]."""
    y = x.copy()
    half = len(freq)
    t = sign * _angles(pos, freq)
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = np.cos(t[:, i])[:, None], np.sin(t[:, i])[:, None]
        y[..., ia] = x[..., ia] * c - x[..., ib] * s
        y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def norm_rope(x, w, pos, freq, eps, interleaved=False):
    """x [rows][heads][D] float64, w [D] float64 or None."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(x, pos, freq, interleaved)


def norm_rope_bwd(dy, x, w, pos, freq, eps, interleaved=False):
    """(dx, dw or None) of <norm_rope(x), dy>."""
    g = rotate(dy, pos, freq, interleaved, -1.0)
    if w is None:
        return g, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dw = (g * x * r).sum((0, 1))
    u = g * w
    return r * (u - x * r * r * (u * x).mean(-1, keepdims=True)), dw


# ---- the cache ---------------------------------------------------------------------------------------------
def key_dword(e: int, dim: int) -> int:
    """Where dword e (elements 8e .. 8e + 7) of a key row lies."""
    n = 2 if dim == 64 else 4
    section, r = divmod(e, 4 * n)
    k, g = divmod(r, 4)
    return section * 4 * n + n * g + k


def quantize_row(x16, block: int, book: str):
    """One head's row (bf16 bits [D]) -> (codes [D], scales as bf16 bits [D / block])."""
    lv = nf4.codebook_levels(book)
    zero = int(np.nonzero(lv == 0)[0][0])
    x16 = np.asarray(x16, np.uint16)
    codes = np.empty(x16.size, np.int64)
    scales = []
    for b in range(0, x16.size, block):
        u = x16[b:b + block]
        mag = int((u & 0x7FFF).max())
        if mag >= 0x7F80:
            codes[b:b + block] = zero
            scales.append(NAN16)
        elif mag < 0x0080:
            codes[b:b + block] = zero
            scales.append(0)
        else:
            a = nf4.bf16_to_f32(np.array([mag], np.uint16))[0]
            share = nf4.bf16_to_f32(u) * (np.float32(1.0) / a)     # fl32 of fl32
            codes[b:b + block] = nf4.nearest_level(share, lv)
            scales.append(mag)
    return codes, np.array(scales, np.uint16)


@functools.lru_cache(None)
def _places(dim: int, key: bool):
    """(byte, shift) of every element of a row."""
    byte, shift = [], []
    for d in range(dim):
        e, j = divmod(d, 8)
        byte.append(4 * (key_dword(e, dim) if key else e) + j % 4)
        shift.append(4 * (j // 4))
    return np.array(byte), np.array(shift)


def pack_row(codes, key: bool) -> np.ndarray:
    """Codes [D] -> bytes [D / 2]."""
    byte, shift = _places(len(codes), key)
    out = np.zeros(len(codes) // 2, np.uint8)
    np.bitwise_or.at(out, byte, (np.asarray(codes) << shift).astype(np.uint8))
    return out


def unpack_row(data, key: bool) -> np.ndarray:
    byte, shift = _places(2 * len(data), key)
    return (np.asarray(data).astype(np.int64)[byte] >> shift) & 15


def row_values(codes, scales16, book: str) -> np.ndarray:
    """What a stored row stands for, float64, no rounding."""
    lv = nf4.codebook_levels(book).astype(np.float64)
    return lv[codes] * np.repeat(f64(scales16), len(codes) // len(scales16))


def row_bf16(codes, scales16, book: str) -> np.ndarray:
    """What a stored row reads back as: bf16 bits of fl32(level * scale)."""
    lv = nf4.codebook_levels(book)
    with np.errstate(invalid="ignore", over="ignore"):
        v = (lv[codes] * nf4.bf16_to_f32(np.repeat(scales16, len(codes) // len(scales16)))).astype(np.float32)
    out = nf4.f32_to_bf16(np.where(np.isnan(v), np.float32(0), v))
    return np.where(np.isnan(v), np.uint16(NAN16), out)


# ---- attention -----------------------------------------------------------------------------------------------
def attention(q, k, v, length: int, scale: float, causal=True, window=0):
    """q [n][Hq][D] float64, the last n tokens of a sequence whose cache is k, v [length][H][D] float64.
    Returns (o [n][Hq][D], lse [n][Hq], bound [n][Hq][D]): the output, the logarithm of the sum, and
    sum_j p_j |v_j|, which errors of p and v are relative to."""
    n, hq, dim = q.shape
    heads = k.shape[1] if length else 1
    group = hq // heads
    o, lse = np.zeros_like(q), np.full((n, hq), -np.inf)
    bound = np.zeros_like(q)
    for i in range(n):
        p = length - n + i
        hi = min(p + 1, length) if causal else length
        lo = max(0, p + 1 - window) if window else 0
        if hi <= lo:
            continue
        for h in range(hq):
            s = scale * (k[lo:hi, h // group] @ q[i, h])
            m = s.max()
            e = np.exp(s - m)
            w = e / e.sum()
            o[i, h] = w @ v[lo:hi, h // group]
            bound[i, h] = w @ np.abs(v[lo:hi, h // group])
            lse[i, h] = m + np.log(e.sum())
    return o, lse, bound
