"""Shared helpers of the 8-bit KV cache tests: seeded caches in the three layouts (dense,
paged pool, per-sequence slots) on the device and as the oracle sees them."""
from __future__ import annotations

import numpy as np
import torch

import lookahead_sparse_kv_score_b200 as lsa
from oracle import kv as OK

U32 = 2.0 ** -24


class Cache:
    """A cache of random finite codes; .dev() pieces go to the calls, .oracle() to the oracle."""

    def __init__(self, seed, B, N, G, W, block=1, page=1, store="dense", spread=3, device="cuda"):
        g = np.random.default_rng(seed)
        per = -(-N // page)
        self.B, self.N, self.G, self.W, self.block, self.page = B, N, G, W, block, page
        self.table, self.seq_pages, self.pages = None, per, B * per
        if store == "paged":
            self.pages = B * per + 3
            self.table = g.permutation(self.pages)[: B * per].reshape(B, per).astype(np.int32)
            self.seq_pages = 0
        elif store == "slots":
            self.seq_pages, self.pages = per + 5, B * (per + 5)
            self.table = np.stack([g.permutation(per + 5)[:per] for _ in range(B)]).astype(np.int32)
        codes = g.integers(0, 256, size=(self.pages, page, G, W), dtype=np.uint8)
        codes[(codes & 0x7F) == 0x7F] = 0x11                    # no NaN codes
        codes = np.where((codes & 0x7F) > 0x60, codes & 0x9F, codes).astype(np.uint8)   # at most 32: scores stay ordinary
        self.codes = codes
        self.scale = np.exp2(g.integers(-5 - spread, -4, size=(B, -(-N // block), G))).astype(np.float32)
        self.device = device
        self.push()

    def push(self):
        d = self.device
        self.rows_d = torch.from_numpy(self.codes.copy()).to(d)
        self.scale_d = torch.from_numpy(self.scale.copy()).to(d)
        self.table_d = None if self.table is None else torch.from_numpy(np.ascontiguousarray(self.table)).to(d)

    def args(self):
        return (self.block, self.page, self.seq_pages, self.pages, self.table_d, self.rows_d, self.scale_d)

    def oracle(self):
        return OK.Cache(self.codes.copy(), self.scale.astype(np.float64).copy(), self.table, self.N, self.block,
                        self.page, self.seq_pages)


def attend(c, q, sm, length, sinks, window, idx, count, d, dv, voff, lse=True, stream=None):
    """lsa_kv_attend with fresh outputs; q a device tensor [B][Tq][H][d].  (out, lse, status)."""
    B, Tq, H, _ = q.shape
    dev = q.device
    cap = 0 if idx is None else idx.shape[1]
    out = torch.full((B, Tq, H, dv), float("nan"), dtype=q.dtype, device=dev)
    le = torch.full((B, Tq, H), float("nan"), device=dev) if lse else None
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    dt = lsa.dtype_code(q)
    size = (B, Tq, c.N, H, c.G, d, dv, voff, c.W)
    ws = lsa.workspace(lsa.lsa_kv_attend_workspace_bytes(*size, dt, sinks, window, cap), dev)
    ws.fill_(0xFF)                                             # stale contents must not matter
    lsa.lsa_kv_attend(*size, dt, q, sm, length, sinks, window, idx, cap, count, *c.args(), out, le, ws, st,
                      stream=stream)
    return out, le, st


def i32(x, device="cuda"):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(device)


def tolerances(dtype, d, r, vmax):
    """Bounds on |out - r.out| and |lse - r.lse| from the roundings each path makes; vmax is
    the largest |code| times the largest scale of the cache.

    Scores (dx): fp32 products and sums of d terms and the scalings, (d + 8) 2^-24 of the largest
    sum |q||K| |sm|.  A bf16 query is held as two e4m3 terms of q / s, s the power of two that
    brings its row's largest element to (224, 448]: exact but for at most 2^-10 / 224 of that
    element where the second term is subnormal.
    Weights: e^(2 dx) - 1 (the token's own score and the sum's), the exponential (2^-21) and
    the fp32 sums, (wide + 16) 2^-24.  The bf16 path multiplies the codes by a weight W = softmax *
    scale held as an e4m3 plus an e5m2 term, in units where the largest of its part is at least
    1: off by at most half a step of each, 2^-4 * 2^-3 of itself.  Below 2^-6 the first term's steps
    are 2^-9, so what is left for the second is at most 2^-10 (and at most W) and its half step
    2^-3 of that; and half the smallest e5m2 value is 2^-17 (below that all of W): r.lost.
    A weight below the smallest normal fp32 number may become 0: it is below 2^-126 of the
    largest weight, so the sum of values moves by at most wide 2^-126 vmax.
    The result is rounded once, by half a step (bf16 2^-8, fp32 2^-24)."""
    bf16 = dtype == torch.bfloat16
    dx = (d + 8) * U32 * r["mag"] + (2.0 ** -10 / 224 * r["top"] if bf16 else 0.0)
    rel = np.expm1(2 * dx) + (r["wide"] + 16) * U32 + 2.0 ** -21
    lse = dx + (r["wide"] + 16) * U32 + 2.0 ** -21 + 2.0 ** -22 * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0))
    if bf16:
        rel = rel + 2.0 ** -7
    out = rel[..., None] * r["mean"] + (2.0 ** -8 if bf16 else U32) * np.abs(r["out"])
    out = out + (2.0 ** -126 * vmax * r["wide"])[..., None]
    if bf16:
        out = out + r["lost"]
    return out, lse


def check_attend(c, q, sm, length, sinks, window, idx, count, d, dv, voff, status=0, stream=None):
    """One call against the oracle, element by element."""
    dev = q.device
    to = lambda x: None if x is None else i32(x, dev)  # noqa: E731
    out, lse, st = attend(c, q, sm, to(length), sinks, window, to(idx), to(count), d, dv, voff, stream=stream)
    torch.cuda.synchronize()
    r = OK.attend(c.oracle(), q.double().cpu().numpy(), sm, length, sinks, window, idx, count, d, dv, voff)
    vmax = float(np.nanmax(np.abs(OK.O.decode_e4m3(c.codes)))) * float(np.nanmax(c.scale))
    to_, tl = tolerances(q.dtype, d, r, vmax)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isinf(r["lse"])
    assert np.array_equal(gl[empty], r["lse"][empty]) and not got[empty].any(), "a query that sees nothing"
    assert np.isfinite(got).all()
    off = np.abs(gl[~empty] - r["lse"][~empty])
    assert np.all(off <= tl[~empty]), float(np.max(off / tl[~empty]))
    bad = np.abs(got - r["out"]) > to_
    assert not bad.any(), (int(bad.sum()), bad.size, float(np.max(np.abs(got - r["out"]) / np.maximum(to_, 1e-30))))
    assert int(st.item()) == status
    return out, lse
