"""The 8-bit KV cache operators, each as one pass over prepared inputs: writing rows into the
cache, reading rows back, attention over the cache, and the rotary positions of the rows and
queries.

``listed()`` names the measured cases and ``draw`` makes more of the same ranges.  A case is
prepared on the GPU from a seed and run either in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, where ``own`` is true, through the package's calls.

The cache.  B sequences of up to N tokens; a token has G heads' rows of W bytes (e4m3 codes),
and each head of each block of ``block`` tokens has one fp32 scale, a power of two.  The
rows lie dense ("dense"), in pages drawn from one pool ("paged"), or, as the fetched
compressed entries do, in the slots of a per-sequence hot pool ("hot").  Keys are the first d
columns of a row and values the dv columns from voff on (the latent rows of the workloads,
512 latent + 64 rotary, have both in the same columns).
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SMIN = 2.0 ** -24          # smallest scale of a block (a block of zeros has it)


def _latent(**kw):
    """A case on the workloads' compressed rows: one KV head of 512 latent + 64 rotary columns."""
    return dict(dict(op="attend", Tq=1, H=64, G=1, d=576, dv=512, voff=0, W=576, dtype="bf16", sinks=0, window=0,
                     cap=0, block=1, page=1, store="dense", slots=0), **kw)


def _heads(**kw):
    """A case on rows with a key and a value part of 128 columns for each of several KV heads."""
    return dict(dict(op="attend", Tq=1, H=32, G=8, d=128, dv=128, voff=128, W=256, dtype="bf16", sinks=0, window=-1,
                     cap=0, block=64, page=64, store="paged", slots=0), **kw)


def listed():
    return [
        # one decoded token over the 512 entries selected in a 128K-token context: latency
        _latent(name="attend_b1_top512", B=1, N=32768, cap=512, store="hot", slots=1024),
        # the 1M-token decode batch over its 2048 selected entries a sequence, in the hot pool
        _latent(name="attend_b32_top2048", B=32, N=262144, cap=2048, store="hot", slots=4096),
        # one long context read whole, latent rows in blocks of 64 tokens (512K tokens at 4:1)
        _latent(name="attend_b1_all_131072", B=1, N=131072, window=-1, block=64, page=64, store="paged"),
        # a large decode batch with grouped heads, every token visible: bandwidth
        _heads(name="attend_b32_gqa_16384", B=32, N=16384, H=64),
        # four drafted tokens a sequence over a window of 4096 and four first tokens, with odd
        # lengths and head groups
        _heads(name="attend_b8_window4096_draft4", B=8, N=20011, Tq=4, H=35, G=7, window=4096, sinks=4, block=16,
               page=16),
        # the 16K-token fp32 step: one token over its 64 selected entries
        _latent(name="attend_f32_top64", B=1, N=4096, H=8, cap=64, dtype="f32"),
        # one decoded token appended to every sequence of the batch: latency
        dict(name="write_b32_token", op="write", B=32, T=1, G=1, W=576, N=4096, dtype="bf16", block=1, page=1,
             store="dense"),
        # a long prompt's rows written in blocks of 64 tokens, starting inside a block
        dict(name="write_b4_prompt", op="write", B=4, T=8191, G=8, W=256, N=8448, dtype="bf16", block=64, page=64,
             store="paged"),
        # selected entries read back at full width
        dict(name="read_b32_top2048", op="read", B=32, G=1, W=576, N=16384, cap=2048, dtype="bf16", block=1, page=1,
             store="dense"),
        # a short odd list read back in 32 bits
        dict(name="read_b3_f32_odd", op="read", B=3, G=5, W=144, N=3001, cap=777, dtype="f32", block=16, page=16,
             store="paged"),
        # the rotary part of one decoded token's 64 query heads, far positions, scaled for long contexts
        dict(name="rope_b32_h64", op="rope", R=32, H=64, D=576, rot=64, layout="interleaved", dtype="bf16",
             inverse=False, far=1048576, factor=16.0),
        # a long prompt's queries, half layout; the inverse rotation is the backward pass
        dict(name="rope_grad_16384", op="rope", R=16384, H=32, D=128, rot=128, layout="half", dtype="bf16",
             inverse=True, far=16384, factor=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        c = _draw(rng)
        if all(work(c)[k] <= most[k] for k in most):
            return c


def _draw(rng):
    kind = rng.choice(["latent", "latent", "heads", "heads", "write", "read", "rope"])
    if kind == "latent":
        store = rng.choice(["hot", "paged", "dense"])
        H = rng.choice([8, 16, 33, 64, 64, 128])
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        if store == "hot":
            cap = _log(rng, 1, 4096)
            c = _latent(B=_log(rng, 1, 32), N=_log(rng, 8192, 262144), H=H, cap=cap, store="hot",
                        slots=cap + rng.randrange(1, 512), Tq=rng.choice([1, 1, 2]), dtype=dtype)
        else:
            N = _log(rng, 100, 131072)
            full = rng.random() < 0.5
            c = _latent(B=min(_log(rng, 1, 32), max(1, 262144 // N)), N=N, H=H, store=store, dtype=dtype,
                        window=-1 if full else _log(rng, 1, 4096), sinks=0 if full else rng.choice([0, 4, 17]),
                        cap=0 if full else rng.choice([0, min(N, _log(rng, 1, 1024))]),
                        block=rng.choice([1, 16, 64, 128]), page=rng.choice([16, 64]))
        if dtype == "f32":
            c["B"], c["H"] = min(c["B"], 4), min(c["H"], 16)
            c["N"] = min(c["N"], 16384) if store != "hot" else c["N"]
        return c
    if kind == "heads":
        G = rng.choice([1, 2, 4, 7, 8])
        hg = rng.choice([1, 4, 5, 8, 16])
        d = rng.choice([64, 128, 128, 192])
        N = _log(rng, 50, 65536)
        full = rng.random() < 0.5
        voff = {64: 64, 128: 128, 192: 256}[d]
        dv = {64: 64, 128: 128, 192: 128}[d]
        return _heads(B=max(1, min(_log(rng, 1, 32), 4000000 // (N * G))), N=N, G=G, H=G * hg, d=d, dv=dv, voff=voff,
                      W=voff + dv, Tq=rng.choice([1, 1, 1, 3, 8]), window=-1 if full else _log(rng, 1, 8192),
                      sinks=0 if full else rng.choice([0, 1, 4]), block=rng.choice([1, 16, 64]),
                      page=rng.choice([16, 64]), store=rng.choice(["paged", "dense"]))
    if kind == "write":
        G, W = rng.choice([(1, 576), (1, 128), (8, 256), (3, 160), (4, 192)])
        T = _log(rng, 1, 8192)
        return dict(op="write", B=max(1, min(_log(rng, 1, 32), 60000000 // (T * G * W))), T=T, G=G, W=W, N=T + rng.randrange(64, 999),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), block=rng.choice([1, 16, 64, 128]),
                    page=rng.choice([1, 16, 64]), store=rng.choice(["paged", "dense"]))
    if kind == "read":
        G, W = rng.choice([(1, 576), (1, 128), (8, 256), (3, 160)])
        cap = _log(rng, 1, 8192)
        return dict(op="read", B=max(1, min(_log(rng, 1, 32), 60000000 // (cap * G * W))), G=G, W=W, N=cap + rng.randrange(10, 9999), cap=cap,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), block=rng.choice([1, 16, 64]),
                    page=rng.choice([1, 16, 64]), store=rng.choice(["paged", "dense"]))
    D, rot = rng.choice([(576, 64), (128, 128), (128, 64), (96, 40), (192, 64)])
    H = rng.choice([1, 5, 8, 64])
    return dict(op="rope", R=_log(rng, 1, max(2, 60000000 // (H * D))), H=H, D=D, rot=rot,
                layout=rng.choice(["interleaved", "half"]), dtype=rng.choice(["bf16", "f32"]),
                inverse=rng.random() < 0.4, far=rng.choice([8192, 131072, 1048576]),
                factor=rng.choice([1.0, 8.0, 40.0]))


# ------------------------------------------------------------------------------ inputs

def _lengths(c):
    """Tokens in each sequence: N for the first, down to about half of N for the last."""
    B, N = c["B"], c["N"]
    return [max(1, N - b * (N // (2 * B))) for b in range(B)]


def _counts(c, key="cap"):
    """Entries in each sequence's list: the capacity for the first, down to three quarters."""
    B, cap = c["B"], c[key]
    return [cap - b * (cap // (4 * B)) for b in range(B)]


def _lists(g, B, N, cap, counts, lengths, dev):
    """Distinct ascending random entries below each sequence's length, padded with -1."""
    idx = torch.full((B, cap), -1, dtype=torch.int32, device=dev)
    got = []
    for b in range(B):
        n = min(counts[b], lengths[b])
        idx[b, :n] = torch.randperm(lengths[b], generator=g, device=dev)[:n].sort().values.to(torch.int32)
        got.append(n)
    return idx, torch.tensor(got, dtype=torch.int32, device=dev)


def _codes(g, n, dev):
    """n e4m3 codes of normal draws (standard deviation 80, within the type's range)."""
    out = torch.empty(n, dtype=torch.uint8, device=dev)
    step = 1 << 28
    for a in range(0, n, step):
        x = torch.randn(min(step, n - a), generator=g, device=dev).mul_(80.0).clamp_(-448.0, 448.0)
        out[a:a + step] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _scales(g, shape, dev):
    return 2.0 ** -8 * (1 << torch.randint(0, 3, shape, generator=g, device=dev)).float()


def _store(c, g, dev, resident=None):
    """Rows, page table (or None), pages in all and pages a sequence of the case's cache."""
    B, N, G, W, page = c["B"], c["N"], c["G"], c["W"], c["page"]
    per = -(-N // page)
    if c["store"] == "hot":
        slots = c["slots"]
        table = torch.full((B, N), -1, dtype=torch.int32, device=dev)
        for b in range(B):
            e = resident[b]
            table[b, e] = torch.randperm(slots, generator=g, device=dev)[: e.numel()].to(torch.int32)
        return dict(rows=_codes(g, B * slots * G * W, dev).view(B * slots, 1, G, W), table=table, pages=B * slots,
                    seq_pages=slots)
    table = None
    if c["store"] == "paged":
        table = torch.randperm(B * per, generator=g, device=dev).to(torch.int32).view(B, per)
    return dict(rows=_codes(g, B * per * page * G * W, dev).view(B * per, page, G, W), table=table, pages=B * per,
                seq_pages=per if table is None else 0)


def _frequencies(rot, factor, base=10000.0, original=65536, fast=32.0, slow=1.0):
    """Radians a position for each pair, the long-context scaling blended in over the pairs
    that turn between `slow` and `fast` times within the original length."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / rot)
    if factor > 1.0:
        at = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot // 2 - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = f * (1 - ramp) + f / factor * ramp
    return f


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(c=c)
    if c["op"] == "rope":
        R, H, D, rot = c["R"], c["H"], c["D"], c["rot"]
        s["x"] = torch.randn(R, H, D, generator=g, device=dev).to(_DT[c["dtype"]])
        s["out"] = torch.zeros(R, H, rot, dtype=_DT[c["dtype"]], device=dev)
        s["pos"] = torch.randint(0, c["far"], (R,), generator=g, device=dev).to(torch.int32)
        s["freq"] = _frequencies(rot, c["factor"]).to(dev)
        s["mscale"] = 1.0 if c["factor"] <= 1.0 else 0.1 * math.log(c["factor"]) + 1.0
        return s
    lens = _lengths(c)
    B, N, G, W, block = c["B"], c["N"], c["G"], c["W"], c["block"]
    if c["op"] == "write":
        s.update(_store(c, g, dev))
        s["scale"] = _scales(g, (B, -(-N // block), G), dev)
        # the rows of one token share a magnitude that varies from token to token
        mag = torch.exp(torch.randn(B, c["T"], 1, 1, generator=g, device=dev))
        s["x"] = (torch.randn(B, c["T"], G, W, generator=g, device=dev) * mag).to(_DT[c["dtype"]])
        s["start"] = torch.tensor([(5 + 7 * b) % (N - c["T"] + 1) for b in range(B)], dtype=torch.int32, device=dev)
        s["count"] = torch.tensor(_counts(c, "T"), dtype=torch.int32, device=dev)
        return s
    if c["cap"]:
        s["idx"], s["count"] = _lists(g, B, N, c["cap"], _counts(c), lens, dev)
        have = s["count"].tolist()
        resident = [s["idx"][b, : have[b]].long() for b in range(B)]
    else:
        s["idx"], s["count"], resident = None, None, None
    s.update(_store(c, g, dev, resident))
    s["scale"] = _scales(g, (B, -(-N // block), G), dev)
    if c["op"] == "read":
        s["out"] = torch.zeros(B, c["cap"], G, W, dtype=_DT[c["dtype"]], device=dev)
        return s
    s["q"] = torch.randn(B, c["Tq"], c["H"], c["d"], generator=g, device=dev).to(_DT[c["dtype"]])
    s["len"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["sm"] = c["d"] ** -0.5
    s["out"] = torch.empty(B, c["Tq"], c["H"], c["dv"], dtype=_DT[c["dtype"]], device=dev)
    s["lse"] = torch.empty(B, c["Tq"], c["H"], device=dev)
    return s


# ------------------------------------------------------------------------------ plain forms

def _rows_of(s, t):
    """Row numbers of tokens t [B][M] (valid ones) in the flat [pages * page][G][W] view."""
    c = s["c"]
    page, b = c["page"], torch.arange(c["B"], device=t.device)[:, None]
    p = t // page
    if s["table"] is not None:
        p = s["table"].long().gather(1, p)
    return (b * s["seq_pages"] + p) * page + t % page


def _values(s, t):
    """fp32 values of tokens t [B][M]: [B][M][G][W]."""
    c = s["c"]
    codes = s["rows"].view(-1, c["G"], c["W"])[_rows_of(s, t)]
    sc = s["scale"].gather(1, (t // c["block"])[:, :, None].expand(-1, -1, c["G"]))
    return codes.view(torch.float8_e4m3fn).float() * sc[..., None]


def _plain_attend(s):
    c = s["c"]
    B, Tq, H, G, N, w, sinks = c["B"], c["Tq"], c["H"], c["G"], c["N"], c["window"], c["sinks"]
    dev = s["q"].device
    n = s["len"].long()[:, None]                                     # [B][1]
    p = n - Tq + torch.arange(Tq, device=dev)                        # [B][Tq]
    main = lambda t: (t >= 0) & (t <= p[:, :, None]) & ((w < 0) | (t < sinks) | (t > p[:, :, None] - w))  # noqa: E731
    parts, seen = [], []
    if w < 0:
        t = torch.arange(N, device=dev).expand(B, N)
        parts.append(t)
        seen.append(main(t[:, None, :]))
    elif w or sinks:
        t = torch.arange(min(sinks, N), device=dev).expand(B, -1)
        parts.append(t)
        seen.append(main(t[:, None, :]))
        t = (p[:, :1] - w + 1).clamp(min=0) + torch.arange(min(w + Tq - 1, N), device=dev)
        parts.append(t)
        seen.append(main(t[:, None, :]) & (t[:, None, :] >= sinks))
    if s["idx"] is not None:
        t = s["idx"].long()
        listed_ = (torch.arange(c["cap"], device=dev) < s["count"].long()[:, None]) & (t >= 0) & (t < n)
        parts.append(t)
        seen.append(listed_[:, None, :] & ~main(t[:, None, :]))
    t, seen = torch.cat(parts, 1), torch.cat(seen, 2)                # [B][M], [B][Tq][M]
    any_ = seen.any(1)
    if s["table"] is not None and c["store"] == "hot":
        t0 = s["idx"][:, :1].long().clamp(min=0)                     # an entry that is resident
        val = _values(s, torch.where(any_, t, t0))
    else:
        val = _values(s, torch.where(any_, t, torch.zeros_like(t)))
    val = val.permute(0, 2, 1, 3)                                    # [B][G][M][W]
    q = s["q"].float().view(B, Tq, G, H // G, c["d"]).permute(0, 2, 1, 3, 4).reshape(B, G, -1, c["d"])
    x = (q @ val[..., : c["d"]].transpose(2, 3)) * s["sm"]
    x = x.view(B, G, Tq, H // G, -1).masked_fill(~seen[:, None, :, None, :], float("-inf"))
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(m.isinf(), torch.zeros_like(m), m))
    l = e.sum(-1, keepdim=True)
    o = (e / torch.where(l > 0, l, torch.ones_like(l))).view(B, G, Tq * (H // G), -1)
    o = o @ val[..., c["voff"]: c["voff"] + c["dv"]]
    o = o.view(B, G, Tq, H // G, -1).permute(0, 2, 1, 3, 4).reshape(B, Tq, H, -1)
    lse = (m + torch.log(l)).squeeze(-1).permute(0, 2, 1, 3).reshape(B, Tq, H)
    return o.to(_DT[c["dtype"]]), lse


def _plain_write(s):
    c = s["c"]
    B, T, G, W, N, block = c["B"], c["T"], c["G"], c["W"], c["N"], c["block"]
    dev = s["x"].device
    start, count = s["start"].long()[:, None], s["count"].long()[:, None]
    nb = (T + 2 * block - 2) // block                                # blocks a sequence can touch
    first = start // block
    t = (first * block + torch.arange(nb * block, device=dev))       # [B][nb * block]
    new = (t >= start) & (t < start + count)
    old = (t < start) & (start + 0 * t < start + count)
    x = s["x"].float().gather(1, (t - start).clamp(0, T - 1)[:, :, None, None].expand(-1, -1, G, W))
    a = torch.where(new[:, :, None], x.abs().amax(-1), x.new_zeros(()))
    a = a.view(B, nb, block, G).amax(2)                              # largest new magnitude of each block and head
    mant, e = torch.frexp(a)
    e = torch.where(mant <= 0.875, e - 9, e - 8)                     # smallest power of two with a / s <= 448
    sc = torch.where(a > 0, ((e + 127) << 23).view(torch.float32), torch.zeros_like(a)).clamp(min=_SMIN)
    tb = (first + torch.arange(nb, device=dev)).clamp(max=s["scale"].shape[1] - 1)
    at = tb[:, :, None].expand(-1, -1, G)
    before = s["scale"].gather(1, at)
    has_old, has_new = old.view(B, nb, block).any(2), new.view(B, nb, block).any(2)
    sc = torch.where(has_old[:, :, None], torch.maximum(sc, before), sc)
    per = lambda v: v[:, :, None, :].expand(B, nb, block, G).reshape(B, nb * block, G, 1)  # noqa: E731
    rows = s["rows"].view(-1, G, W)
    r = _rows_of(s, t.clamp(max=N - 1))
    was = rows[r].view(torch.float8_e4m3fn).float() * (per(before) / per(sc))
    code = torch.where(new[:, :, None, None], x / per(sc), was).to(torch.float8_e4m3fn).view(torch.uint8)
    touched = new | (old & has_new[:, :, None].expand(B, nb, block).reshape(B, -1))
    rows[r[touched]] = code[touched]
    b = torch.arange(B, device=dev)[:, None].expand(B, nb)
    s["scale"][b[has_new], tb[has_new]] = sc[has_new]
    return s["rows"].view(torch.float8_e4m3fn), s["scale"]


def _plain_read(s):
    c = s["c"]
    t = s["idx"].long()
    ok = (torch.arange(c["cap"], device=t.device) < s["count"].long()[:, None]) & (t >= 0)
    v = _values(s, torch.where(ok, t, torch.zeros_like(t))).to(s["out"].dtype)
    return torch.where(ok[:, :, None, None], v, s["out"])


def _plain_rope(s):
    c = s["c"]
    a = s["pos"].double()[:, None] * s["freq"]
    if c["inverse"]:
        a = -a
    co, si = (torch.cos(a) * s["mscale"]).float()[:, None, :], (torch.sin(a) * s["mscale"]).float()[:, None, :]
    x = s["x"][..., c["D"] - c["rot"]:].float()
    if c["layout"] == "half":
        u, v = x[..., : c["rot"] // 2], x[..., c["rot"] // 2:]
        y = torch.cat([u * co - v * si, u * si + v * co], -1)
    else:
        u, v = x[..., 0::2], x[..., 1::2]
        y = torch.stack([u * co - v * si, u * si + v * co], -1).flatten(-2)
    return y.to(s["out"].dtype)


# ------------------------------------------------------------------------------ one pass

def run(s):
    c = s["c"]
    if not own:
        return {"attend": _plain_attend, "write": _plain_write, "read": _plain_read, "rope": _plain_rope}[c["op"]](s)
    import lookahead_sparse_kv_score_b200 as lsa
    if c["op"] == "rope":
        H, D, rot = c["H"], c["D"], c["rot"]
        x = s["x"][..., D - rot:]
        lsa.lsa_rope(c["R"], H, rot, c["layout"] == "half", lsa.dtype_code(x), x, H * D, D, s["pos"], s["freq"],
                     s["mscale"], c["inverse"], s["out"], H * rot, rot)
        return s["out"]
    B, G, W, N = c["B"], c["G"], c["W"], c["N"]
    cache = (c["block"], c["page"], s["seq_pages"], s["pages"], s["table"], s["rows"], s["scale"])
    if c["op"] == "write":
        lsa.lsa_kv_write(B, c["T"], N, G, W, lsa.dtype_code(s["x"]), s["x"], G * W, s["start"], s["count"], *cache)
        return s["rows"].view(torch.float8_e4m3fn), s["scale"]
    if c["op"] == "read":
        lsa.lsa_kv_read(B, N, G, W, s["idx"], c["cap"], s["count"], *cache, lsa.dtype_code(s["out"]), s["out"])
        return s["out"]
    size = (B, c["Tq"], N, c["H"], G, c["d"], c["dv"], c["voff"], W)
    dt = lsa.dtype_code(s["q"])
    if "ws" not in s:
        s["ws"] = lsa.workspace(lsa.lsa_kv_attend_workspace_bytes(*size, dt, c["sinks"], c["window"], c["cap"]))
    lsa.lsa_kv_attend(*size, dt, s["q"], s["sm"], s["len"], c["sinks"], c["window"], s["idx"], c["cap"], s["count"],
                      *cache, s["out"], s["lse"], s["ws"])
    return s["out"], s["lse"]


# ------------------------------------------------------------------------------ work

def _visible(c):
    """Per sequence: tokens that any query sees, and (query, token) pairs."""
    tokens, pairs = 0, 0
    for b, n in enumerate(_lengths(c)):
        k = min(_counts(c)[b], n) if c["cap"] else 0
        span = n if c["window"] < 0 else min(n, c["sinks"] + c["window"] + c["Tq"] - 1)
        one = n if c["window"] < 0 else min(n, c["sinks"] + c["window"])
        share = 1 - span / n                                         # of a random list, outside the window
        tokens += span + k * share
        pairs += c["Tq"] * (one + k * share)
    return tokens, pairs


def work(case):
    c = case
    e = 2 if c.get("dtype") == "bf16" else 4
    if c["op"] == "rope":
        n = c["R"] * c["H"] * c["rot"]
        return {"bytes": 2 * n * e + c["R"] * 4 + c["rot"] * 4, "flops": 3 * n}
    G, W = c["G"], c["W"]
    if c["op"] == "write":
        n = sum(_counts(c, "T"))
        return {"bytes": n * G * (W * (e + 1) + 4 / c["block"]) + 8 * c["B"], "flops": 2 * n * G * W}
    if c["op"] == "read":
        n = sum(min(k, m) for k, m in zip(_counts(c), _lengths(c)))
        return {"bytes": n * (4 + G * (W * (e + 1) + 4 / c["block"])), "flops": n * G * W}
    tokens, pairs = _visible(c)
    used = max(c["d"], c["voff"] + c["dv"]) if c["voff"] <= c["d"] else c["d"] + c["dv"]
    qo = c["B"] * c["Tq"] * c["H"] * ((c["d"] + c["dv"]) * e + 4)
    idx = sum(_counts(c)) * 4 if c["cap"] else 0
    table = 0 if c["store"] == "dense" else tokens * 4 / c["page"]
    return {"bytes": tokens * G * (used + 4 / c["block"]) + qo + idx + table,
            "flops": 2 * pairs * c["H"] * (c["d"] + c["dv"])}


# ------------------------------------------------------------------------------ in 64 bits

def _pow2(e):
    """2 to the power of whole numbers, exactly (the device's exp2 and log2 need not be)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _decode64(codes):
    """fp64 values of e4m3 codes from their fields."""
    v = codes.to(torch.int32)
    ex, ma = (v >> 3) & 15, (v & 7).double()
    mag = torch.where(ex == 0, ma * 2.0 ** -9, (8 + ma) * _pow2(ex - 10))
    return torch.where(v >= 128, -mag, mag)


def _e4m3_64(y):
    """fp64 values rounded to the nearest e4m3 value, ties to even."""
    ulp = _pow2(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(y / ulp) * ulp


def _where(s, b, t):
    """Flat row numbers of tokens t of sequence b."""
    c = s["c"]
    p = t // c["page"]
    if s["table"] is not None:
        p = s["table"][b].long()[p]
    return (p + b * s["seq_pages"]) * c["page"] + t % c["page"]


def _tokens64(s, b, t):
    c = s["c"]
    sc = s["scale"][b][t // c["block"]].double()
    return _decode64(s["rows"].view(-1, c["G"], c["W"])[_where(s, b, t)]) * sc[:, :, None]


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "rope":
        x = s["x"][..., c["D"] - c["rot"]:].double()
        half = c["rot"] // 2
        z = torch.complex(x[..., :half], x[..., half:]) if c["layout"] == "half" else torch.view_as_complex(
            x.reshape(*x.shape[:-1], half, 2).contiguous())
        turn = torch.polar(torch.full_like(s["freq"], s["mscale"]).expand(c["R"], -1).contiguous(),
                           s["pos"].double()[:, None] * s["freq"] * (-1.0 if c["inverse"] else 1.0))
        z = z * turn[:, None, :]
        return torch.cat([z.real, z.imag], -1) if c["layout"] == "half" else torch.view_as_real(z).flatten(-2)
    B, G, W = c["B"], c["G"], c["W"]
    if c["op"] == "read":
        out = s["out"].double()
        for b, n in enumerate(s["count"].tolist()):
            out[b, :n] = _tokens64(s, b, s["idx"][b, :n].long())
        return out
    if c["op"] == "write":
        # the stored codes are returned as the values of the e4m3 type, apart from their scale
        code = _decode64(s["rows"].view(-1, G, W))
        scale = s["scale"].double()
        k = c["block"]
        for b, (a, n) in enumerate(zip(s["start"].tolist(), s["count"].tolist())):
            lo, hi = a // k * k, -(-(a + n) // k) * k
            t = torch.arange(lo, min(a + n, c["N"]), device=code.device)
            at = _where(s, b, t)
            x = torch.cat([code[at[: a - lo]] * scale[b, lo // k, :, None], s["x"][b, :n].double()])
            pad = torch.zeros(hi - lo, G, W, dtype=torch.float64, device=x.device)
            pad[a - lo: a - lo + n] = x[a - lo:]
            big = pad.view(-1, k, G, W).abs().amax((1, 3))
            m, e = torch.frexp((big / 448.0).clamp(min=2.0 ** -24))
            sc = _pow2(torch.where(m == 0.5, e - 1, e))
            if a > lo:
                sc[0] = torch.maximum(sc[0], scale[b, lo // k])
            code[at] = _e4m3_64(x / sc.repeat_interleave(k, 0)[: x.shape[0], :, None])
            scale[b, lo // k: hi // k] = sc
        return code.view(s["rows"].shape), scale
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=out.device)
    hg = c["H"] // G
    for b, n in enumerate(s["len"].tolist()):
        for i in range(c["Tq"]):
            p = n - c["Tq"] + i
            t = torch.arange(max(p + 1, 0), device=out.device)
            if c["window"] >= 0:
                t = t[(t < c["sinks"]) | (t > p - c["window"])]
            if s["idx"] is not None:
                e = s["idx"][b, : int(s["count"][b])].long()
                t = torch.cat([t, e[(e >= 0) & (e < n) & ~torch.isin(e, t)]])
            if not t.numel():
                continue
            v = _tokens64(s, b, t)
            q = s["q"][b, i].double().view(G, hg, c["d"])
            x = torch.einsum("ghd,tgd->ght", q, v[..., : c["d"]]) * s["sm"]
            lse[b, i] = torch.logsumexp(x, -1).reshape(-1)
            w = torch.softmax(x, -1)
            out[b, i] = torch.einsum("ght,tgd->ghd", w, v[..., c["voff"]: c["voff"] + c["dv"]]).reshape(c["H"], -1)
    return out, lse
