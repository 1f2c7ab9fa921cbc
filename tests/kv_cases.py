"""Paged-cache cases shared by the CPU and GPU tests: lengths, pages, and the
elementwise bound of the attention kernels' error."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged

HALF_STEP = 2.0 ** -8     # bf16: torch.finfo(torch.bfloat16).eps / 2


class Cache:
    """Sequences of the given lengths in pages (CPU tensors): `dense[b]` is (k, v) of
    bf16 values [Hkv, len, D]. Slots without a token hold NaN (or garbage codes with
    NaN scales); table entries without a token hold `unused`."""

    def __init__(self, fmt, lens, Hkv, D, page, seed=0, unused=-1, spare=3, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.lens, self.Hkv, self.D, self.page = fmt, list(lens), Hkv, D, page
        counts = [-(-n // page) for n in lens]
        pool = sum(counts) + spare
        order = torch.randperm(pool, generator=g).tolist()
        self.table = torch.full((len(lens), max(counts + [1])), unused, dtype=torch.int32)
        if fmt == "bf16":
            self.pages = [torch.full((pool, Hkv, page, D), float("nan"), dtype=torch.bfloat16) for _ in range(2)]
            self.scales = [None, None]
        else:
            self.pages = [torch.randint(0, 256, (pool, Hkv, page, D // 2), generator=g, dtype=torch.uint8)
                          for _ in range(2)]
            self.scales = [torch.full((pool, Hkv, page, 2), float("nan"), dtype=torch.bfloat16) for _ in range(2)]
        self.dense = []
        for b, n in enumerate(lens):
            ids = order[:counts[b]]
            order = order[counts[b]:]
            self.table[b, :counts[b]] = torch.tensor(ids, dtype=torch.int32)
            kv = []
            for i in range(2):
                x = (spread * torch.randn(Hkv, n, D, generator=g)).to(torch.bfloat16)
                self.store(i, ids, 0, x)
                kv.append(x)
            self.dense.append(kv)

    def store(self, i, ids, first, x):
        pos = np.arange(first, first + x.shape[1])
        page = torch.tensor([ids[p // self.page] for p in pos], dtype=torch.long)
        off = torch.tensor(pos % self.page)
        if self.fmt == "bf16":
            self.pages[i][page, :, off] = x.transpose(0, 1)
        else:
            c, s, lo = paged.int4_rows(x.double().numpy())
            self.pages[i][page, :, off] = torch.from_numpy(paged.pack_codes(c)).transpose(0, 1)
            sl = torch.from_numpy(np.stack([s, lo], -1)).to(torch.bfloat16)
            self.scales[i][page, :, off] = sl.transpose(0, 1)

    def parts(self, b, i, h):
        """Head h of sequence b as (values, centred part, offset): values = part + offset
        in fp64 (offset 0 for bf16 pages), [len, D], [len, D], [len]."""
        x = self.dense[b][i][h].double().numpy()
        if self.fmt == "bf16":
            return x, x, np.zeros(len(x))
        c, s, lo = paged.int4_rows(x)
        return paged.int4_values(c, s, lo), (c - 8) * s[:, None], lo + 8 * s


def attention_reference(cache, new, q, scale, window=0, sinks=0):
    """Oracle outputs of a packed batch, q bf16 [Hq, M, D] with new[b] tokens of each
    sequence at the end of its keys: (out, its bound, lse, its bound), [M, Hq, D] and
    [Hq, M], for the rows of the batch.

    Bound of one output: 2^-8 |ref| for its own rounding; 2^-8 of the sum of p |v| for
    the rounding of each probability (4-bit pages: of p s |c - 8|, the rounded
    operand); and what fp32 costs: a score is a sum of D products, each partial sum off
    by at most 2^-23 of the terms' magnitudes, so it is off by e = (D + 4) 2^-23 of
    their sum (4-bit pages: the terms are s (128 + c) |q| and (|m| + 128 s) |sum q|);
    p then by a factor 1 + 2 e + 2^-21 (exponential, its argument's own rounding in
    base 2, with |argument| at most z below), and the sums over n keys by n 2^-23 of
    their terms. lse: e + 2^-21 (|lse| + z) + n 2^-23."""
    Hq, M, D = q.shape
    group = Hq // cache.Hkv
    out, tol = np.zeros((M, Hq, D)), np.zeros((M, Hq, D))
    lse, ltol = np.zeros((Hq, M)), np.zeros((Hq, M))
    at = 0
    for b, n in enumerate(new):
        L = cache.lens[b]
        pos = np.arange(L - n, L)
        for h in range(cache.Hkv):
            k, _, _ = cache.parts(b, 0, h)
            v, part, off = cache.parts(b, 1, h)
            if cache.fmt == "int4":
                c, s, lo = paged.int4_rows(cache.dense[b][0][h].double().numpy())
                kmag = (128 + c) * s[:, None]
                koff = np.abs(lo - 128 * s)
            for hq in range(h * group, (h + 1) * group):
                x = q[hq, at:at + n].double().numpy()
                o, l, p = paged.attention(x, k, v, pos, scale, window, sinks)
                if cache.fmt == "int4":
                    terms = np.abs(x) @ kmag.T + np.abs(x).sum(-1, keepdims=True) * koff
                else:
                    terms = np.abs(x) @ np.abs(k).T
                seen = p > 0
                e = (D + 4) * 2.0 ** -23 * scale * np.max(np.where(seen, terms, 0.0), axis=-1, initial=0.0)
                z = scale * np.max(np.where(seen, np.abs(x @ k.T), 0.0), axis=-1, initial=0.0)
                f = 2 * e + 2.0 ** -21 * (1 + 2 * z) + L * 2.0 ** -23
                mag = p @ np.abs(part) + (p @ np.abs(off))[:, None]
                out[at:at + n, hq], lse[hq, at:at + n] = o, l
                tol[at:at + n, hq] = HALF_STEP * (np.abs(o) + p @ np.abs(part)) + f[:, None] * mag * (1 + HALF_STEP)
                ltol[hq, at:at + n] = e + 2.0 ** -21 * (np.where(np.isfinite(l), np.abs(l), 0) + z + 1) + L * 2.0 ** -23
        at += n
    return out, tol, lse, ltol
