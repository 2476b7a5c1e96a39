"""Paged key/value cache: the 4-bit rows, where a token lies, and attention over what a cache holds; CPU.

TEST INFRASTRUCTURE ONLY, like the rest of the oracle: the library never imports it, and it shares no code
with the CUDA kernels.

4-bit rows: groups of 64 values with least value lo and greatest hi;
  zero = bf16 not above lo,  scale = bf16 not below max((hi - zero) / 15, 2^-20 max|.|, 2^-100),
  code = rint((x - zero) / scale), a value is zero + scale * code.
The library states these steps in fp32, each rounded; ``quantise`` follows them so that codes can
be compared bit for bit. ``attention_paged`` is fp64.

Readings: keys of sequence b are positions 0 .. n_b - 1; the last Nq of them belong to the queries, so with
the causal mask query i sees keys j <= i + n_b - Nq; rows that see none give O = 0, LSE = -inf.
"""
from __future__ import annotations

import numpy as np

from .attention import attention_head, kv_head

GROUP = 64


def bf16_toward(x, up: bool) -> np.ndarray:
    """float32 values cut to bf16 (as float32), upward or downward."""
    x = np.asarray(x, dtype=np.float32)
    bits = x.view(np.uint32)
    cut = bits & np.uint32(0xFFFF0000)
    low = cut.view(np.float32)
    wrong = (low < x) if up else (low > x)
    return np.where(wrong, (cut + np.uint32(0x10000)).view(np.float32), low)


def bf16_nearest(x) -> np.ndarray:
    """float32 values rounded to bf16 (as float32), ties to even."""
    bits = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7FFF + ((bits >> 16) & 1)) & 0xFFFF0000
    return bits.astype(np.uint32).view(np.float32)


def turn_f32(x, cos, sin, interleaved: bool) -> np.ndarray:
    """float32 rows x [T, heads, d] turned by the angles cos, sin [T, half]; every product, sum and difference rounded."""
    x = np.asarray(x, dtype=np.float32)
    c, s = np.float32(cos)[:, None], np.float32(sin)[:, None]
    half = c.shape[-1]
    a = np.arange(half) * 2 if interleaved else np.arange(half)
    b = a + 1 if interleaved else a + half
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def quantise(x):
    """float32 rows x [..., d] -> (codes uint8 [..., d], scale and zero float32 [..., d / 64])."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(-1), g.max(-1)
    zero = bf16_toward(lo, False)
    least = np.maximum(np.maximum(np.abs(lo), np.abs(hi)) * np.float32(2.0 ** -20), np.float32(2.0 ** -100))
    scale = bf16_toward(np.maximum((hi - zero) / np.float32(15), least), True)
    codes = np.clip(np.rint((g - zero[..., None]) / scale[..., None]), 0, 15).astype(np.uint8)
    return codes.reshape(x.shape), scale, zero


def values(codes, scale, zero) -> np.ndarray:
    """fp64 values that codes [..., d] stand for."""
    g = np.asarray(codes, dtype=np.float64).reshape(*codes.shape[:-1], -1, GROUP)
    return (np.float64(zero)[..., None] + np.float64(scale)[..., None] * g).reshape(codes.shape)


def pack(codes) -> np.ndarray:
    """Codes [..., d] as bytes [..., d / 2], even dims in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def place(table_row, position: int, page_size: int):
    """(page, row in page) of a position."""
    return int(table_row[position // page_size]), position % page_size


def attention_paged(q, keys, vals, scale: float, causal: bool):
    """q [B, Nq, H, d]; keys and vals: per sequence [n_b, Hkv, d]. O [B, Nq, H, d], LSE [B, H, Nq]."""
    q = np.asarray(q, dtype=np.float64)
    B, Nq, H, d = q.shape
    o, lse = np.zeros(q.shape), np.full((B, H, Nq), -np.inf)
    for b in range(B):
        n, Hkv = keys[b].shape[:2]
        if n == 0:
            continue
        for h in range(H):
            j = kv_head(h, H, Hkv)
            o[b, :, h], lse[b, h] = attention_head(q[b, :, h], np.float64(keys[b][:, j]), np.float64(vals[b][:, j]), scale,
                                                   causal, causal_offset=n - Nq)
    return o, lse
