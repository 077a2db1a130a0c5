"""Paged key-value cache: the row formats, the pages and attention over them, in float64.

TEST INFRASTRUCTURE (see oracle/__init__.py): never imported by the product path.

A row (one token's K or V in one KV head) is stored with a power of two 2^(b - 127):
  fp8    e4m3 codes of x * 2^(127-b), b the least byte with max|x| <= 448 * 2^(b-127)
  nvfp4  per 16 elements an e4m3 scale s of max16|x| * 2^(127-b) / 6, and e2m1 codes of
         x * 2^(127-b) / s (0 where s is 0), b the least byte with max|x| <= 2688 * 2^(b-127)
to nearest, ties to even. A row with an infinity or a NaN: b = 255, everything else 0.
"""
from __future__ import annotations

import numpy as np

from .codecs import bf16_round, e2m1_decode, e4m3_decode, e4m3_encode, nvfp4_unpack

LARGEST = {"fp8": 448.0, "nvfp4": 448.0 * 6.0}
_E2M1_POS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_encode(x) -> np.ndarray:
    """Codes of x rounded to nearest-even on the e2m1 grid, saturated to +-6."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    code = np.zeros(a.shape, dtype=np.uint8)
    for i in range(7):
        mid = (_E2M1_POS[i] + _E2M1_POS[i + 1]) / 2
        # the code above the midpoint i | i+1: a tie goes to the even one of the two
        code += ((a > mid) | ((a == mid) & (i % 2 == 1))).astype(np.uint8)
    return np.where(np.signbit(x), code | np.uint8(8), code).astype(np.uint8)


def row_byte(x, fmt) -> np.ndarray:
    """Scale byte of each row of x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    b = np.zeros(x.shape[:-1], dtype=np.int64)
    amax = np.max(np.abs(np.where(np.isfinite(x), x, 0.0)), axis=-1)
    while np.any(amax > LARGEST[fmt] * 2.0 ** (b - 127)):
        b += amax > LARGEST[fmt] * 2.0 ** (b - 127)
    return np.where(np.all(np.isfinite(x), axis=-1), b, 255).astype(np.uint8)


def quantise(x, fmt):
    """(codes, row bytes, block scales or None) of rows x [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    b = row_byte(x, fmt)
    y = np.where((b == 255)[..., None], 0.0, x) * 2.0 ** (127.0 - np.where(b == 255, 127, b))[..., None]
    if fmt == "fp8":
        return e4m3_encode(y), b, None
    y = y.reshape(y.shape[:-1] + (-1, 16))
    s = e4m3_encode(np.max(np.abs(y), axis=-1) / 6.0)
    sv = e4m3_decode(s)[..., None]
    code = np.where(sv > 0, e2m1_encode(y / np.where(sv > 0, sv, 1.0)), 0).astype(np.uint8)
    code = code.reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), b, s


def dequantise(codes, b, s, fmt) -> np.ndarray:
    """Values [..., D] (float64); a row of byte 255 is NaN."""
    scale = np.where(b == 255, np.nan, 2.0 ** (np.asarray(b, np.float64) - 127.0))[..., None]
    if fmt == "fp8":
        return e4m3_decode(codes) * scale
    v = e2m1_decode(nvfp4_unpack(codes))
    v = v.reshape(v.shape[:-1] + (-1, 16)) * e4m3_decode(s)[..., None]
    return v.reshape(v.shape[:-2] + (-1,)) * scale


class PagedKV:
    """Pages [num_pages][n_kv][page_size][...] and a page table, as NumPy arrays.
    fmt "bf16": k, v hold the values; "fp8", "nvfp4": codes, with row and block scales."""

    def __init__(self, fmt, k, v, table, row=None, block=None, window=0):
        self.fmt, self.k, self.v, self.table = fmt, np.array(k), np.array(v), np.array(table)
        self.row = None if row is None else np.array(row)
        self.block = None if block is None else np.array(block)
        self.window, self.page_size = window, self.k.shape[2]

    def place(self, s, p):
        p = np.asarray(p)
        return self.table[s, (p - 1) // self.page_size], (p - 1) % self.page_size

    def store(self, s, p, k, v):
        """One token's K and V [n_kv][D] at position p of sequence s; p = 0 stores nothing."""
        if p == 0:
            return
        pg, off = self.place(s, p)
        for i, (arr, x) in enumerate(((self.k, k), (self.v, v))):
            if self.fmt == "bf16":
                arr[pg, :, off] = x
                continue
            codes, b, sc = quantise(x, self.fmt)
            arr[pg, :, off] = codes
            self.row[pg, :, i, off] = b
            if sc is not None:
                self.block[pg, :, i, off] = sc

    def load(self, s, positions):
        """K, V values [n_kv][n][D] (float64)."""
        pg, off = self.place(s, positions)
        out = []
        for i, arr in enumerate((self.k, self.v)):
            x = np.moveaxis(arr[pg, :, off], 0, 1)
            if self.fmt == "bf16":
                out.append(x.astype(np.float64))
                continue
            b = np.moveaxis(self.row[pg, :, i, off], 0, 1)
            sc = None if self.block is None else np.moveaxis(self.block[pg, :, i, off], 0, 1)
            out.append(dequantise(x, b, sc, self.fmt))
        return out


def paged_attention(n_q, q, cache: PagedKV, seq_id, pos, g=None, gate_bias=None):
    """out [T][n_q * D] (float64, not rounded): each row's attention over keys max(1, p-W+1)..p,
    gated by sigmoid(g + bias) where g is given; a row at position 0 is zero. Also returns the
    weighted magnitudes sum p|v| of the same shape (before the gate), for error bounds."""
    T, _, D = q.shape
    o, mag = np.zeros((T, n_q, D)), np.zeros((T, n_q, D))
    n_kv = cache.k.shape[1]
    grp = n_q // n_kv
    for t in range(T):
        p = int(pos[t])
        if p == 0:
            continue
        lo = max(1, p - cache.window + 1) if cache.window else 1
        K, V = cache.load(int(seq_id[t]), np.arange(lo, p + 1))
        for h in range(n_q):
            x = K[h // grp] @ q[t, h] / np.sqrt(D)
            w = np.exp(x - x.max())
            w /= w.sum()
            o[t, h] = w @ V[h // grp]
            mag[t, h] = w @ np.abs(V[h // grp])
    o, mag = o.reshape(T, -1), mag.reshape(T, -1)
    if g is not None:
        o = o / (1.0 + np.exp(-(np.asarray(g, np.float64) + np.repeat(np.asarray(gate_bias, np.float64), D))))
    return o, mag


__all__ = ["PagedKV", "bf16_round", "dequantise", "e2m1_encode", "paged_attention", "quantise",
           "row_byte"]
