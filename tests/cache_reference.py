"""The paged 8-bit latent cache in float64 numpy, from the definitions in
include/dsa.h: rows and scales, append, and attention row by row. Test
infrastructure only; it shares no code with the library."""
from __future__ import annotations

import numpy as np


def _values():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


VALUES = _values()
_POSITIVE = VALUES[:127]  # codes 0 .. 126 ascend from 0 to 448


def encode(x):
    """e4m3 codes of float64 values, |x| <= 448: nearest, ties to the even code."""
    x = np.asarray(x, dtype=np.float64)
    mag = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_POSITIVE, mag)
    lo = np.maximum(hi - 1, 0)
    hi = np.minimum(hi, 126)
    dl, dh = mag - _POSITIVE[lo], _POSITIVE[hi] - mag
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def need_scale(amax):
    s = 2.0 ** -32
    while amax > 448 * s:
        s *= 2
    return s


def rotate(x, t, inv_freq, halves):
    """x [..., Dr] at position t."""
    d = x.shape[-1]
    ang = float(t) * inv_freq.astype(np.float64)
    c, s = np.cos(ang), np.sin(ang)
    a, b = (x[..., :d // 2], x[..., d // 2:]) if halves else (x[..., 0::2], x[..., 1::2])
    u, v = a * c - b * s, b * c + a * s
    out = np.empty(x.shape)
    if halves:
        out[..., :d // 2], out[..., d // 2:] = u, v
    else:
        out[..., 0::2], out[..., 1::2] = u, v
    return out


class Cache:
    """latent / rope codes [n_pages, page, width] and scale [n_pages]."""

    def __init__(self, latent, rope, scale, table, cu, lens):
        self.latent, self.rope, self.scale = latent.copy(), rope.copy(), scale.astype(np.float64)
        self.table, self.cu, self.lens = table, cu, lens
        self.n_pages, self.ps = latent.shape[:2]

    def sound(self, b, n_tok):
        c0, c1, n = int(self.cu[b]), int(self.cu[b + 1]), int(self.lens[b])
        return 0 <= c0 <= c1 <= n_tok and c1 - c0 <= n <= self.table.shape[1] * self.ps

    def append(self, latent, rope, inv_freq, halves, q_rope=None):
        """Returns the rotated q_rope (float64), rows of no sequence NaN."""
        n_tok = latent.shape[0]
        q = None if q_rope is None else np.full(q_rope.shape, np.nan)
        for b in range(len(self.lens)):
            if not self.sound(b, n_tok):
                continue
            c0, c1, n = int(self.cu[b]), int(self.cu[b + 1]), int(self.lens[b])
            first = n - (c1 - c0)
            pages = {}
            for i in range(c0, c1):
                t = first + i - c0
                if q is not None:
                    q[i] = rotate(q_rope[i].astype(np.float64), t, inv_freq, halves)
                row = np.concatenate([latent[i].astype(np.float64),
                                      rotate(rope[i].astype(np.float64), t, inv_freq, halves)])
                pages.setdefault(t // self.ps, []).append((t % self.ps, row))
            for j, rows in pages.items():
                p = int(self.table[b, j])
                if not 0 <= p < self.n_pages:
                    continue
                s = need_scale(max(np.abs(r).max() for _, r in rows))
                r0 = rows[0][0]
                if r0 > 0 and s < self.scale[p]:
                    s = self.scale[p]
                elif r0 > 0 and s > self.scale[p]:
                    f = self.scale[p] / s
                    self.latent[p, :r0] = encode(VALUES[self.latent[p, :r0]] * f)
                    self.rope[p, :r0] = encode(VALUES[self.rope[p, :r0]] * f)
                self.scale[p] = s
                dc = self.latent.shape[2]
                for r, row in rows:
                    self.latent[p, r] = encode(row[:dc] / s)
                    self.rope[p, r] = encode(row[dc:] / s)
        return q

    def rows(self, b, pos):
        """Values [len(pos), Dc + Dr] and which of them are in the pool."""
        pg = self.table[b, pos // self.ps]
        ok = (pg >= 0) & (pg < self.n_pages)
        p = np.where(ok, pg, 0)
        codes = np.concatenate([self.latent[p, pos % self.ps], self.rope[p, pos % self.ps]], 1)
        return VALUES[codes] * self.scale[p][:, None], ok

    def attend(self, q, scale, window, n_sink):
        """out, lse, sum p|v| / sum p, and max_s scale * sum|q_c k_c| for each row;
        rows of no (sound) sequence NaN."""
        n_tok, h, _ = q.shape
        dc = self.latent.shape[2]
        out, mag = np.full((n_tok, h, dc), np.nan), np.full((n_tok, h, dc), np.nan)
        lse, zabs = np.full((n_tok, h), np.nan), np.full((n_tok, h), np.nan)
        for b in range(len(self.lens)):
            if not self.sound(b, n_tok):
                continue
            c0, c1, n = int(self.cu[b]), int(self.cu[b + 1]), int(self.lens[b])
            for i in range(c0, c1):
                t = n - (c1 - c0) + i - c0
                pos = np.arange(t + 1)
                if window:
                    pos = pos[(pos > t - window) | (pos < n_sink)]
                kv, ok = self.rows(b, pos)
                kv = kv[ok]
                if not len(kv):
                    out[i], mag[i], lse[i], zabs[i] = 0.0, 0.0, -np.inf, 0.0
                    continue
                z = scale * (q[i] @ kv.T)
                top = z.max(1, keepdims=True)
                p = np.exp(z - top)
                l = p.sum(1, keepdims=True)
                out[i] = p @ kv[:, :dc] / l
                mag[i] = p @ np.abs(kv[:, :dc]) / l
                lse[i] = (np.log(l) + top)[:, 0]
                zabs[i] = (scale * (np.abs(q[i]) @ np.abs(kv).T)).max(1)
        return out, lse, mag, zabs
