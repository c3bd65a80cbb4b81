"""The 4-bit key/value cache in 64 bits, written from the definitions in
include/bq.h with plain loops over sequences: the yardstick of its tests."""
import math

import numpy as np
import torch


def page_bytes(page, D, G):
    return page * (D + 8 * (D // G))


def quantize(x, G):
    """x [..., D] -> (codes uint8 [..., D], steps, minima float16 [..., D/G])."""
    x = np.asarray(x, dtype=np.float32).reshape(x.shape[:-1] + (-1, G))
    with np.errstate(all="ignore"):
        low, high = x.min(-1), x.max(-1)  # (NaN if there is one)
        bad = ~np.isfinite(high - low)
        m = np.clip(low, -65504, 65504).astype(np.float16)
        rng = np.maximum(high - m.astype(np.float32), np.float32(0))
        s = np.minimum(rng / np.float32(15), np.float32(65504)).astype(np.float16)
        q = (x.astype(np.float64) - m.astype(np.float64)[..., None]) / s.astype(np.float64)[..., None]
        c = np.where((s > 0)[..., None], np.clip(np.rint(q), 0, 15), 0)
        c = np.where(bad[..., None], 0, c).astype(np.uint8)
    s = np.where(bad, np.float16(np.nan), s)
    m = np.where(bad, np.float16(np.nan), m)
    return c.reshape(c.shape[:-2] + (-1,)), s, m


class Cache:
    """A pool on the host, with what it holds."""

    def __init__(self, pages, H, D, G, page, fill=None):
        self.pages, self.H, self.D, self.G, self.page = pages, H, D, G, page
        self.pool = np.zeros((pages, H, page_bytes(page, D, G)), dtype=np.uint8) if fill is None else fill.copy()

    def _part(self, which):
        """Views (codes [pages, H, page, D/2], params [pages, H, page, D/G, 2]) of K (0) or V (1)."""
        a, b = self.page * self.D // 2, self.page * (self.D // 2 + 4 * (self.D // self.G))
        o = which * b
        codes = self.pool[:, :, o:o + a].reshape(self.pages, self.H, self.page, self.D // 2)
        par = self.pool[:, :, o + a:o + b].view(np.float16).reshape(self.pages, self.H, self.page, -1, 2)
        assert codes.base is not None and par.base is not None
        return codes, par

    def put(self, page, slot, k, v):
        """k, v [H, D] at one place."""
        for which, x in ((0, k), (1, v)):
            c, s, m = quantize(x, self.G)
            o = which * page_bytes(self.page, self.D, self.G) // 2
            packed = (c[:, 0::2] | (c[:, 1::2] << 4)).astype(np.uint8)
            self.pool[page, :, o + slot * self.D // 2: o + (slot + 1) * self.D // 2] = packed
            par = np.stack((s, m), -1).astype(np.float16).reshape(self.H, -1)
            at = o + self.page * self.D // 2 + slot * 4 * (self.D // self.G)
            self.pool[page, :, at: at + 4 * (self.D // self.G)] = par.view(np.uint8)

    def values(self, which, pages, n, dtype=np.float64):
        """[n, H, D] of the first n positions of a sequence held in `pages`, s * code + m computed in `dtype`."""
        codes, par = self._part(which)
        pages = np.asarray(pages[: -(-n // self.page)], dtype=np.int64)
        c, p = codes[pages], par[pages].astype(dtype)
        x = np.stack((c & 15, c >> 4), -1).reshape(c.shape[:-1] + (-1, self.G)).astype(dtype)
        with np.errstate(all="ignore"):
            x = x * p[..., :1] + p[..., 1:]
        x = x.reshape(len(pages), self.H, self.page, self.D).transpose(0, 2, 1, 3)
        return x.reshape(-1, self.H, self.D)[:n]


def attention(q, cache, table, lens, cu, scale, window=0, softcap=0.0, slopes=None):
    """(out, lse, tol) of q [T, Hq, D] (float64): tol bounds a kernel's distance from out before the last rounding.

    How the bound comes about (u = 2^-23, one fp32 step with truncation; z the score, p the softmax, v the values):
      scores     a dot product of D terms and the minimum's term in fp32: |dz| <= (D + 16) u |scale| sum|q| (15 s + |m|);
                 the cap adds 8 u cap, the distance bias 4 u |slope| (p - t), the exponential's argument 4 u |z| more;
      weights    p changes by a factor 1 + e, |e| <= 2^-11 (p * step rounded once to fp16, the sum that divides taken
                 of the rounded weights) + 2 max|dz| + 2^-20 (exponential, reciprocal), which moves the output by at
                 most sum p |e| |v - out|;
      sums       n terms in fp32, 16 at a time and over splits: (n / 16 + 64) u sum p (15 s + |m|);
      underflow  a weight below 2^-38 of the largest may become 0: n 2^-38 max (15 s + |m|).
    """
    T, Hq, D = q.shape
    out, lse, tol = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf), np.zeros((T, Hq, D))
    u = 2.0 ** -23
    share = Hq // cache.H
    for b in range(len(lens)):
        n, rows = int(lens[b]), range(int(cu[b]), int(cu[b + 1]))
        if n <= 0 or not len(rows):
            continue
        k, v = cache.values(0, table[b], n), cache.values(1, table[b], n)
        mag = []
        for which in (0, 1):
            par = cache._part(which)[1][np.asarray(table[b][: -(-n // cache.page)], dtype=np.int64)].astype(np.float64)
            par = 15 * par[..., 0] + np.abs(par[..., 1])
            par = par.transpose(0, 2, 1, 3).reshape(-1, cache.H, par.shape[-1])[:n]
            mag.append(np.repeat(par, cache.G, axis=2))
        key = np.arange(n)
        for j, t in enumerate(rows):
            pos = n - len(rows) + j
            if pos < 0:
                continue
            sees = key[(key <= pos) & (key > pos - window if window else True)]
            for h in range(Hq):
                g = h // share
                with np.errstate(all="ignore"):
                    z = scale * (k[sees, g] @ q[t, h])
                    dz = (D + 16) * u * abs(scale) * (mag[0][sees, g] @ np.abs(q[t, h]))
                    if softcap:
                        z = softcap * np.tanh(z / softcap)
                        dz = dz + 8 * u * softcap
                    if slopes is not None:
                        z = z + slopes[h] * (sees - pos)
                        dz = dz + 4 * u * abs(slopes[h]) * (pos - sees)
                    dz = dz + 4 * u * np.abs(z)
                    top = z.max()
                    p = np.exp(z - top)
                    lse[t, h] = top + math.log(p.sum()) if np.isfinite(top) else np.nan
                    p = p / p.sum()
                    o = p @ v[sees, g]
                    out[t, h] = o
                    e = 2.0 ** -11 + 2 * dz.max() + 2.0 ** -20
                    tol[t, h] = 1.02 * e * (p @ np.abs(v[sees, g] - o)) + (n / 16 + 64) * u * (p @ mag[1][sees, g]) + \
                        n * 2.0 ** -38 * mag[1][sees, g].max()
    return out, lse, tol


def to_torch(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
