"""Microscaled formats and the norms around the layer, in fp64 numpy, from their definitions.

Formats: blocks of 32 values with one power-of-two scale byte s (2^(s - 127)); "mxfp4" holds
E2M1 codes, "mxfp6" E2M3 codes. Values are looked up in the table of all code values.
"""
from __future__ import annotations

import numpy as np

BITS = {"mxfp4": 4, "mxfp6": 6}


def code_values(fmt: str) -> np.ndarray:
    """Value of every code: a sign bit, two exponent bits (bias 1) and the mantissa."""
    bits = BITS[fmt]
    mb = bits - 3
    c = np.arange(1 << bits)
    f, m = (c >> mb) & 3, (c & ((1 << mb) - 1)) / (1 << mb)
    v = np.where(f == 0, m, (1 + m) * 2.0 ** (f - 1))
    return np.where(c >> (bits - 1), -v, v)


def quantize(x: np.ndarray, fmt: str):
    """x [..., K] -> (codes [..., K] uint8, one a value; scales [..., K/32] uint8)."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(b).max(axis=-1)
    finite = np.isfinite(amax)
    a = np.where(finite & (amax > 0), amax, 1.0)
    e = np.frexp(a)[1] - 1                                     # floor(log2 a)
    s = np.where(finite, np.where(amax > 0, np.maximum(1, e - 2 + 127), 1), 255)
    with np.errstate(invalid="ignore"):
        t = np.abs(b) * np.exp2(127.0 - np.where(finite, s, 127))[..., None]
    vals = code_values(fmt)[:1 << (BITS[fmt] - 1)]
    mid = (vals[1:] + vals[:-1]) / 2
    lo, hi = np.searchsorted(mid, t, "left"), np.searchsorted(mid, t, "right")
    code = np.where(lo == hi, lo, lo + (lo & 1))               # a tie: the even code
    code = code + (np.signbit(b) << (BITS[fmt] - 1))
    code = np.where(finite[..., None], code, 0)
    return code.reshape(x.shape).astype(np.uint8), s.astype(np.uint8)


def pack(codes: np.ndarray, fmt: str) -> np.ndarray:
    """One code a value -> the packed code plane: code i of a row in bits i*bits and up."""
    bits = BITS[fmt]
    bit = (codes[..., None] >> np.arange(bits)) & 1
    return np.packbits(bit.reshape(*codes.shape[:-1], -1).astype(np.uint8), axis=-1,
                       bitorder="little")


def unpack(q: np.ndarray, fmt: str) -> np.ndarray:
    bits = BITS[fmt]
    bit = np.unpackbits(q, axis=-1, bitorder="little")
    bit = bit.reshape(*q.shape[:-1], -1, bits).astype(np.uint8)
    return (bit << np.arange(bits, dtype=np.uint8)).sum(-1).astype(np.uint8)


def dequantize(q: np.ndarray, s: np.ndarray, fmt: str) -> np.ndarray:
    """Packed codes and scales -> fp64 values."""
    v = code_values(fmt)[unpack(q, fmt)]
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return (v.reshape(*s.shape, 32) * scale[..., None]).reshape(v.shape)


def rms_norm(v: np.ndarray, weight: np.ndarray, eps: float) -> np.ndarray:
    return v / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps) * weight


def add_norm(resid, weight, eps, delta=None, scale=1.0):
    """-> (x, s) before any rounding."""
    s = resid if delta is None else resid + scale * delta
    return rms_norm(s, weight, eps), s


def combine_norm(y, inv_perm, w, resid, eps, post=None, gate=None, scale=1.0, nxt=None):
    """-> (s, x or None) before any rounding."""
    T, k = w.shape
    p = inv_perm.reshape(T, k).astype(np.int64)
    c = np.zeros_like(resid)
    for j in range(k):
        ok = (p[:, j] >= 0) & (p[:, j] < T * k)
        c += np.where(ok[:, None], w[:, j:j + 1] * y[np.where(ok, p[:, j], 0)], 0.0)
    n = c if post is None else rms_norm(c, post, eps)
    s = resid + scale * (n if gate is None else gate * n)
    return s, None if nxt is None else rms_norm(s, nxt, eps)
