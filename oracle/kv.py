"""Plain fp64 restatement of the 8-bit KV cache calls and of the rotary positions, slow and
literal: one block, token, query and head at a time.  Shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np

from . import lsa_oracle as O

SCALE_MIN = 2.0 ** -24


def e4m3_round(y):
    """fp64 values rounded to the nearest e4m3 value (ties to even mantissa, saturating)."""
    y = np.asarray(y, dtype=np.float64)
    m, e = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
    ulp = np.ldexp(1.0, e - 4)
    return np.clip(np.rint(y / ulp) * ulp, -448.0, 448.0)


def e4m3_code(v):
    """Codes of values that are e4m3 values (inverse of lsa_oracle's decoding)."""
    table = O.decode_e4m3(np.arange(256, dtype=np.uint8))
    order = {float(x): c for c, x in reversed(list(enumerate(table))) if math.isfinite(x)}
    flat = [order[float(x)] if x != 0 or not np.signbit(x) else 0x80 for x in np.ravel(v)]
    return np.array(flat, dtype=np.uint8).reshape(np.shape(v))


def block_scale(amax):
    """Smallest power of two s >= 2^-24 with amax / s <= 448; NaN for a non-finite amax."""
    if not math.isfinite(amax):
        return math.nan
    s = SCALE_MIN
    while amax / s > 448.0:
        s *= 2.0
    return s


class Cache:
    """rows [pages][page][G][W] codes, scale [B][blocks][G] fp64, table [B][pages of N] or None."""

    def __init__(self, rows, scale, table, N, block, page, seq_pages):
        self.rows, self.scale, self.table = rows, scale, table
        self.N, self.block, self.page, self.seq_pages = N, block, page, seq_pages

    def place(self, b, t):
        """(page, place) of token t of sequence b, or None when it is not resident."""
        p = t // self.page if self.table is None else int(self.table[b][t // self.page])
        if p < 0 or (self.seq_pages > 0 and p >= self.seq_pages) or b * self.seq_pages + p >= self.rows.shape[0]:
            return None
        return b * self.seq_pages + p, t % self.page

    def values(self, b, t):
        """fp64 values [G][W] of token t."""
        return O.decode_e4m3(self.rows[self.place(b, t)]) * self.scale[b, t // self.block][:, None]


def write(c: Cache, x, start, count):
    """x [B][T][G][W] fp64; updates c.rows and c.scale.  True when a token was skipped: outside the
    cache, of a sequence that starts below 0, not resident, or in a block whose scale would change while
    an earlier token of it is not resident."""
    skipped = False
    B, T, G, W = x.shape
    for b in range(B):
        new = {int(start[b]) + i: x[b, i] for i in range(min(int(count[b]), T))}
        skipped |= any(t < 0 or t >= c.N for t in new)
        if new and int(start[b]) < 0:
            continue
        new = {t: v for t, v in new.items() if 0 <= t < c.N}
        here = {t: v for t, v in new.items() if c.place(b, t) is not None}
        skipped |= len(here) < len(new)
        for j in sorted({t // c.block for t in here}):
            mine = [t for t in here if t // c.block == j]
            old = list(range(j * c.block, int(start[b])))
            away = any(c.place(b, t) is None for t in old)
            for g in range(G):
                amax = max((math.inf if not np.isfinite(new[t][g]).all() else float(np.abs(new[t][g]).max()))
                           for t in mine)
                s, before = block_scale(amax), float(c.scale[b, j, g])
                if old:
                    s = math.nan if math.isnan(s) or not math.isfinite(before) else max(s, before)
                    if away and not (s == before or math.isnan(s) and math.isnan(before)):
                        skipped = True
                        continue
                c.scale[b, j, g] = s
                ok = not math.isnan(s)
                for t in mine:
                    c.rows[c.place(b, t)][g] = e4m3_code(e4m3_round(new[t][g] / s)) if ok else 0
                for t in old:
                    at = c.place(b, t)
                    if at is None or s == before:
                        continue
                    c.rows[at][g] = e4m3_code(e4m3_round(O.decode_e4m3(c.rows[at][g]) * before / s)) if ok else 0
    return skipped


def read(c: Cache, idx, count, out):
    """out[b][j] = values of token idx[b][j], j < count[b]; other rows untouched."""
    skipped = False
    for b in range(idx.shape[0]):
        for j in range(min(int(count[b]), idx.shape[1])):
            t = int(idx[b, j])
            if t < 0:
                continue
            if t >= c.N or c.place(b, t) is None:
                skipped = True
                continue
            out[b, j] = c.values(b, t)
    return skipped


def attend(c: Cache, q, sm, length, sinks, window, idx, count, d, dv, voff):
    """q [B][Tq][H][d] fp64.  Returns a dict: out [B][Tq][H][dv] and lse [B][Tq][H], and what
    tolerances need: mean = sum softmax |V| [B][Tq][H][dv]; per (b, i, h) mag = the largest
    |sm| sum |q||K| of a visible token, top = |sm| max|q| times the largest sum |K|, wide = the
    number of visible tokens; lost = sum (min(W, 2^-17 max W) + min(W / 8, 2^-13 max W)) |V| / scale, W = softmax * |scale|."""
    B, Tq, H, _ = q.shape
    G = c.rows.shape[2]
    r = dict(out=np.zeros((B, Tq, H, dv)), mean=np.zeros((B, Tq, H, dv)), lse=np.full((B, Tq, H), -np.inf),
             mag=np.zeros((B, Tq, H)), top=np.zeros((B, Tq, H)), wide=np.zeros((B, Tq, H)),
             lost=np.zeros((B, Tq, H, dv)))
    for b in range(B):
        n = min(max(int(length[b]), 0), c.N)
        cached = {}
        for i in range(Tq):
            p = n - Tq + i
            seen = [t for t in range(max(p + 1, 0)) if window < 0 or t < sinks or t > p - window]
            if idx is not None:
                own = set(seen)
                seen += [int(e) for e in idx[b, : max(0, min(int(count[b]), idx.shape[1]))]
                         if 0 <= e < n and int(e) not in own]
            seen = [t for t in seen if c.place(b, t) is not None]
            if not seen:
                continue
            for t in seen:
                if t not in cached:
                    cached[t] = c.values(b, t)
            v = np.stack([cached[t] for t in seen])
            for h in range(H):
                g = h // (H // G)
                a = sm * (v[:, g, :d] @ q[b, i, h])
                m = a.max()
                w = np.exp(a - m)
                r["lse"][b, i, h] = m + math.log(w.sum())
                w = w / w.sum()
                r["out"][b, i, h] = w @ v[:, g, voff: voff + dv]
                r["mean"][b, i, h] = w @ np.abs(v[:, g, voff: voff + dv])
                s = np.abs(np.array([c.scale[b, t // c.block, g] for t in seen]))
                top = (w * s).max()
                low = np.minimum(w * s, 2.0 ** -17 * top) + np.minimum(w * s / 8, 2.0 ** -13 * top)
                r["lost"][b, i, h] = low / np.where(s == 0, 1.0, s) @ np.abs(v[:, g, voff: voff + dv])
                size = np.abs(v[:, g, :d])
                r["mag"][b, i, h] = abs(sm) * (size @ np.abs(q[b, i, h])).max()
                r["top"][b, i, h] = abs(sm) * np.abs(q[b, i, h]).max() * size.sum(1).max()
                r["wide"][b, i, h] = len(seen)
    return r


def rope(x, pos, freq, half, mscale, inverse):
    """x [R][H][rot] fp64 rotated pair by pair."""
    out = np.empty_like(x)
    n = x.shape[2] // 2
    for r in range(x.shape[0]):
        for i in range(n):
            a = float(pos[r]) * float(freq[i]) * (-1.0 if inverse else 1.0)
            iu, iv = (i, i + n) if half else (2 * i, 2 * i + 1)
            u, v = x[r, :, iu], x[r, :, iv]
            out[r, :, iu] = mscale * (u * math.cos(a) - v * math.sin(a))
            out[r, :, iv] = mscale * (u * math.sin(a) + v * math.cos(a))
    return out
