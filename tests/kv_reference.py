"""The operators of the 4-bit cache from their definitions, on the CPU in 64 bits: blocks and their places in a page,
attention sequence by sequence, eviction entry by entry.  Shares nothing with the library."""
import numpy as np
import torch

import bit_quantized_mat_quantize_amd as qmm

DIMS = [64, 96, 128, 192, 256]
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def encode(x):
    """(d as fp16, codes) of blocks of 32 along the last axis, by the rule of the header."""
    x = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 32)
    first = np.abs(x).argmax(-1)[..., None]
    top = np.take_along_axis(x, first, -1)
    with np.errstate(all="ignore"):
        d = (np.float32(0) - top / np.float32(8)).astype(np.float32)
        h = d.astype(np.float16)
        inv = np.float32(1) / d
        q = np.clip(np.rint((x * inv).astype(np.float32)) + np.float32(8), 0, 15)
    bad = ~np.isfinite(x).all(-1, keepdims=True) | ~np.isfinite(h)
    h = np.where(bad, np.float16(np.nan), h)
    q = np.where(bad | (h == 0), 8, q)
    return h[..., 0], q.astype(np.uint8).reshape(*x.shape[:-2], -1)


def decode(h, q):
    return (q.reshape(*h.shape, 32).astype(np.float64) - 8) * h.astype(np.float64)[..., None]


class Cache:
    """A cache on the host as scales and codes per (page, keys or values, head, entry), and its bytes."""

    def __init__(self, pages, heads, D, page, fill=0xFF):
        self.pages, self.heads, self.D, self.page = pages, heads, D, page
        self.h = np.full((pages, 2, heads, page, D // 32), np.nan, np.float16)
        self.q = np.full((pages, 2, heads, page, D), 15, np.uint8)
        self.fill = fill

    def put(self, page, t, part, x):
        """Entry t of a page from numbers [heads, D]."""
        self.h[page, part, :, t], self.q[page, part, :, t] = encode(x)

    def get(self, page, t, part):
        return decode(self.h[page, part, :, t], self.q[page, part, :, t]).reshape(self.heads, self.D)

    def bytes(self):
        D, page = self.D, self.page
        out = np.zeros((self.pages, 2, self.heads, page * D * 9 // 16), np.uint8)
        words = np.zeros((self.pages, 2, self.heads, page, D // 8), np.uint64)
        for i in range(8):
            words |= self.q[..., i::8].astype(np.uint64) << np.uint64(4 * i)
        w = words.astype(np.uint32)
        t, e = np.meshgrid(np.arange(page), np.arange(D // 8), indexing="ij")
        for part, at in ((0, t * (D // 8) + (e % 4) * (D // 32) + e // 4), (1, (t // 4 * (D // 8) + e) * 4 + t % 4)):
            flat = np.zeros((self.pages, self.heads, page * D // 8), np.uint32)
            flat[..., at.ravel()] = w[:, part].reshape(self.pages, self.heads, -1)
            out[:, part, :, : page * D // 2] = flat.view(np.uint8)
        scales = np.ascontiguousarray(self.h.swapaxes(-1, -2)).reshape(self.pages, 2, self.heads, -1)
        out[..., page * D // 2:] = scales.view(np.uint8)
        return out

    def to_dev(self):
        b = torch.from_numpy(self.bytes()).cuda()
        return b.view(self.pages, 2, self.heads, self.page, self.D * 9 // 16)


class Batch:
    """Sequences of given lengths and new rows over pages in no order, some pages nobody's."""

    def __init__(self, rng, lens, rows, heads, D, page, width=None, spare=2, scale=1.0):
        self.lens, self.rows, self.heads, self.D, self.page = list(lens), list(rows), heads, D, page
        need = [-(-n // page) for n in lens]
        self.width = width or max(1, max(need, default=1))
        order = rng.permutation(sum(need) + spare)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = Cache(max(1, sum(need) + spare), heads, D, page)
        for b, n in enumerate(lens):
            for p in range(n):
                for part in (0, 1):
                    x = rng.standard_normal((heads, D)) * scale
                    self.cache.put(self.table[b, p // page], p % page, part, x.astype(np.float32))

    @property
    def T(self):
        return sum(self.rows)

    def starts(self):
        return np.concatenate(([0], np.cumsum(self.rows))).astype(np.int32)

    def entries(self, b, part):
        """[len, heads, D] in 64 bits."""
        return np.stack([self.cache.get(self.table[b, p // self.page], p % self.page, part) if self.table[b, p // self.page] >= 0
                         and self.table[b, p // self.page] < self.cache.pages
                         else np.full((self.heads, self.D), np.nan) for p in range(self.lens[b])]) \
            if self.lens[b] else np.zeros((0, self.heads, self.D))

    def dev(self):
        """(cache, table, lens, starts) on the GPU."""
        return (self.cache.to_dev(), torch.from_numpy(self.table).cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                torch.from_numpy(self.starts()).cuda())


def seen(n, L, causal, window):
    """bool [n, L]: what row i of n sees of L entries."""
    pos, j = np.arange(L - n, L)[:, None], np.arange(L)
    see = j <= pos if causal else np.ones((n, L), bool)
    return see & (j > pos - window) if window else see


def attention(batch, q, scale, causal=True, window=0):
    """(out, lse, mass, slack) of q [T, q_heads, D]; slack: what the tolerances are made of, per row and head: the largest
    sum of |q k| * |scale| of a seen entry, and per element the sums of p |v| and of |v|."""
    T, HQ, D = q.shape
    G = HQ // batch.heads
    out, lse = np.zeros((T, HQ, D)), np.full((T, HQ), -np.inf)
    terms, weight, total = np.zeros((T, HQ)), np.zeros((T, HQ, D)), np.zeros((T, HQ, D))
    mass = np.zeros((len(batch.lens), batch.heads, batch.width * batch.page))
    at = 0
    for b, n in enumerate(batch.rows):
        L = batch.lens[b]
        k, v = batch.entries(b, 0), batch.entries(b, 1)
        see = seen(n, L, causal, window)
        for hq in range(HQ):
            h = hq // G
            for i in range(n):
                w = see[i]
                if not w.any():
                    continue
                kk, vv = k[w, h], v[w, h]
                s = kk @ q[at + i, hq].astype(np.float64) * scale
                m = s.max()
                e = np.exp(s - m)
                out[at + i, hq] = e @ vv / e.sum()
                lse[at + i, hq] = m + np.log(e.sum())
                terms[at + i, hq] = (np.abs(kk) @ np.abs(q[at + i, hq].astype(np.float64))).max() * abs(scale)
                weight[at + i, hq] = e @ np.abs(vv) / e.sum()
                total[at + i, hq] = np.abs(vv).sum(0)
                mass[b, h, :L][w] += e / e.sum()
        at += n
    return out, lse, mass, (terms, weight, total)


def tolerance(kind, D, L, slack, out, rounded_keys=False):
    """|out error| <= this, by rounding steps (eps / 2 each: fp16 2^-11, bf16 2^-8, fp32 2^-24).

    A score is a sum of D products in fp32 and D/32 scalings (each half a step of the sum of magnitudes at most), of
    queries held to 2^-22 of their row's largest (fp32; 16-bit ones are exact) against keys that are exact, or rounded to
    fp16 once (`rounded_keys`), then multiplied twice.  The log2 scale and 2^x add 3 steps of the score's size and 2^-22.
    Weights change by that much, in the numerator and in the sum: twice.  16-bit queries round p and v to fp16 once each;
    fp32 ones hold both to 2^-22.  Sums over L entries are fp32, and the result is rounded to its type.

    A weight's last piece is fp16, whose half step is at least 2^-25.  Weights are 2^(x - r + 8) with a reference r that
    is at most the row's largest score so far, so the largest weight, and with it their sum, is at least 2^8: each weight
    is off by at most 2^-33 of the sum on top of the above, and the result by 2^-33 times the sum of |v|."""
    terms, weight, total = slack
    D32 = D + D // 32 + 8
    ds = terms * (D32 * 2.0 ** -24 + (2.0 ** -22 if kind == "f32" else 0.0) + (2.0 ** -11 if rounded_keys and kind != "f32" else 0.0))
    ds = ds + 2.0 ** -22
    per = 2 * ds + (2 * 2.0 ** -21 if kind == "f32" else 2 * 2.0 ** -11) + (L + 8) * 2.0 ** -24
    step = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[kind]
    return per[..., None] * weight * 1.01 + 2.0 ** -33 * total + step * np.abs(out) + (2.0 ** -25 if kind == "f16" else 0.0), ds


def evict(lens, mass, budget, recent):
    """(ids, mass, lens) by sorting every entry by (weight, position)."""
    B, H, _ = mass.shape
    ids = np.full((B, H, budget), -1, np.int32)
    kept = np.zeros((B, H, budget), np.float32)
    for b in range(B):
        for h in range(H):
            L, m = lens[b], mass[b, h]
            old = range(max(0, L - recent)) if L > budget else range(0)
            best = sorted(old, key=lambda p: (-(np.inf if np.isnan(m[p]) else m[p]), not np.isnan(m[p]), p))[: budget - recent]
            keep = sorted(best) + list(range(max(0, L - recent), L)) if L > budget else list(range(L))
            ids[b, h, : len(keep)] = keep
            kept[b, h, : len(keep)] = m[keep]
    return ids, kept, np.minimum(lens, budget).astype(np.int32)


def to_host(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy() if t.dtype in (torch.float16, torch.bfloat16) else t.detach().cpu().numpy()


__all__ = ["DIMS", "TYPES", "Batch", "Cache", "attention", "decode", "encode", "evict", "qmm", "seen", "to_host", "tolerance"]
