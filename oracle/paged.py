"""Paged K/V cache, chunk attention over it and cross attention: the definitions in fp64 (CPU).

A cached row x of d values (one token of one head) is s = fl32(amax / 127) and codes
rint_half_even(fl32(x / s)), 0 where s = 0; it stands for code * s. New token i of n in a
sequence of kv tokens is at position p = kv - n + i and sees key t iff t < kv, t <= p (causal)
and t > p - window (window > 0).
"""
from __future__ import annotations

import math

import numpy as np


def quantize_rows(x: np.ndarray):
    """Codes (int8) and scales (fp32) of the rows of x [..., d] (fp32 values)."""
    x = np.asarray(x, np.float32)
    s = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
    safe = np.where(s > 0, s, np.float32(1))[..., None]
    q = np.rint((x / safe).astype(np.float32))
    return np.where(s[..., None] > 0, np.clip(q, -127, 127), 0).astype(np.int8), s


def dequantize_rows(codes: np.ndarray, s: np.ndarray) -> np.ndarray:
    return codes.astype(np.float64) * s.astype(np.float64)[..., None]


def visible(n: int, kv: int, causal: bool = True, window: int = 0) -> np.ndarray:
    """Which of kv keys each of n new tokens sees: bool [n, kv]."""
    p = (kv - n + np.arange(n))[:, None]
    t = np.arange(kv)[None]
    ok = np.ones((n, kv), bool)
    if causal:
        ok &= t <= p
    if window:
        ok &= t > p - window
    return ok


def attention_rows(q: np.ndarray, k: np.ndarray, v: np.ndarray, ok: np.ndarray, scale: float | None = None):
    """One head: (out [n, d], lse [n], weighted mean of |v| [n, d]); rows without a key: 0, -inf, 0.
    The third is what rounding errors of the weights are relative to."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    scale = 1 / math.sqrt(q.shape[1]) if scale is None else scale
    n = q.shape[0]
    if k.shape[0] == 0:
        return np.zeros((n, v.shape[1])), np.full(n, -np.inf), np.zeros((n, v.shape[1]))
    x = np.where(ok, scale * (q @ k.T), -np.inf)
    m = x.max(1)
    m0 = np.where(np.isfinite(m), m, 0)
    p = np.exp(x - m0[:, None])
    l = p.sum(1)
    safe = np.where(l > 0, l, 1)[:, None]
    v = np.where(ok.any(0)[:, None], v, 0)
    with np.errstate(divide="ignore"):
        return p @ v / safe, m0 + np.log(l), p @ np.abs(v) / safe
