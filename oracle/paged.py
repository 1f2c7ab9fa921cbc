"""Oracle of the paged key/value cache and its attention (numpy).

Sources: paged KV blocks and the block manager, TensorRT-LLM 深度工程实践, §3.2; the
FMHA call between the QKV projection and o_proj, same page, §2.2.

Readings:
  R14 rotation: (a, b) -> (a cos - b sin, b cos + a sin) for the pairs
      (i, i + rot / 2), or (2i, 2i + 1) interleaved; the tables are inputs. The
      products and sums are rounded to fp32 one by one and the result once to bf16,
      because the 4-bit codes are decided on it.
  R15 4-bit rows: lo = min, s = (max - lo) / 15 in fp32, rounded up to bf16;
      code = round((x - lo) / s) to nearest even in fp32, 0 where s = 0; a code
      stands for lo + code s.
  R16 attention: causal by position, position of new token i of n in a sequence of
      len tokens = len - n + i; with a window, keys j > pos - window or j < sinks.
      A token that sees nothing gives 0 and log-sum-exp -inf. All in fp64.
"""
from __future__ import annotations

import numpy as np

from .core import bf16_round


def rotate(x, cos, sin, interleaved=False):
    """x [H, M, D] (bf16 values), cos and sin [M, rot / 2] fp32 -> bf16 values, fp64."""
    x = np.asarray(x, np.float32)
    cos, sin = np.asarray(cos, np.float32), np.asarray(sin, np.float32)
    half = cos.shape[-1]
    i = np.arange(half)
    one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., one], x[..., two]
    y = x.copy()
    y[..., one] = a * cos - b * sin
    y[..., two] = b * cos + a * sin
    return bf16_round(y.astype(np.float64))


def int4_rows(x):
    """Rows [..., D] of bf16 values -> (codes int [..., D], scale [...], minimum [...])."""
    x = np.asarray(x, np.float32)
    lo, hi = x.min(-1), x.max(-1)
    t = ((hi - lo) / np.float32(15)).astype(np.float32)
    s = bf16_round(t.astype(np.float64))
    up = ((s.astype(np.float32).view(np.uint32) + np.uint32(0x10000)) & np.uint32(0xFFFF0000)).view(np.float32)
    s = np.where(s < t, up, s).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        c = np.rint((x - lo[..., None]) / s[..., None])
    c = np.where(s[..., None] > 0, np.clip(c, 0, 15), 0)
    return c.astype(np.int64), s.astype(np.float64), lo.astype(np.float64)


def int4_values(codes, s, lo):
    """What 4-bit rows stand for, fp64."""
    return lo[..., None] + codes * s[..., None]


def pack_codes(codes):
    """Codes [..., D] -> bytes [..., D / 2], the even d in the low nibble."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def sees(pos, key, window=0, sinks=0):
    """Whether the token at position pos sees the key at position key."""
    pos, key = np.asarray(pos)[:, None], np.asarray(key)[None, :]
    ok = key <= pos
    if window:
        ok = ok & ((key > pos - window) | (key < sinks))
    return ok


def attention(q, k, v, pos, scale, window=0, sinks=0):
    """q [n, D] at positions pos [n], k and v [L, D] -> (out [n, D], lse [n], p [n, L])."""
    z = (np.asarray(q, np.float64) @ np.asarray(k, np.float64).T) * scale
    z = np.where(sees(pos, np.arange(len(k)), window, sinks), z, -np.inf)
    top = z.max(-1, keepdims=True) if len(k) else np.full((len(z), 1), -np.inf)
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(z - top)
    den = e.sum(-1, keepdims=True)
    p = e / np.where(den > 0, den, 1.0)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(den))[:, 0]
    return p @ np.asarray(v, np.float64), lse, p
