"""The 8-bit KV cache calls at sizes where a block walks many tiles: parity with fp64 torch on the
device (vectorised; the same tolerances as the element-wise tests), caches past 4 GB, two calls
at once, and outputs between canaries."""
import numpy as np
import pytest
import torch

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import build

import kv_cases as K
from test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    lsa.lib()


def _decode(codes):
    v = codes.to(torch.int64)
    e, m = (v >> 3) & 15, (v & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(v >= 128, -mag, mag)


def _values(c, b, t):
    """fp64 values [T][G][W] of tokens t of sequence b (all resident)."""
    p = t // c.page
    if c.table_d is not None:
        p = c.table_d[b].long()[p]
    rows = c.rows_d.view(-1, c.G, c.W)[(p + b * c.seq_pages) * c.page + t % c.page]
    return _decode(rows) * c.scale_d[b][t // c.block].double()[:, :, None]


def _reference(c, q, sm, length, sinks, window, idx, count, d, dv, voff):
    """What oracle.kv.attend returns, as numpy arrays."""
    B, Tq, H, _ = q.shape
    hg = H // c.G
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    r = dict(out=z(B, Tq, H, dv), mean=z(B, Tq, H, dv), lse=torch.full((B, Tq, H), -np.inf, dtype=torch.float64, device="cuda"),
             mag=z(B, Tq, H), top=z(B, Tq, H), wide=z(B, Tq, H), lost=z(B, Tq, H, dv))
    for b in range(B):
        n = int(length[b])
        for i in range(Tq):
            p = n - Tq + i
            t = torch.arange(max(p + 1, 0), device="cuda")
            if window >= 0:
                t = t[(t < sinks) | (t > p - window)]
            if idx is not None:
                e = idx[b, : int(count[b])].long()
                e = e[(e >= 0) & (e < n)]
                t = torch.cat([t, e[~torch.isin(e, t)]])
            if not t.numel():
                continue
            v = _values(c, b, t).permute(1, 0, 2)                       # [G][T][W]
            k, vv = v[..., :d], v[..., voff: voff + dv]
            qq = q[b, i].double().view(c.G, hg, d)
            a = sm * qq @ k.transpose(1, 2)
            w = torch.softmax(a, -1)
            r["lse"][b, i] = torch.logsumexp(a, -1).reshape(-1)
            r["out"][b, i] = (w @ vv).reshape(H, dv)
            r["mean"][b, i] = (w @ vv.abs()).reshape(H, dv)
            s = c.scale_d[b][t // c.block].double().T[:, None, :]       # [G][1][T]
            top = (w * s).amax(-1, keepdim=True)
            low = (torch.minimum(w * s, 2.0 ** -17 * top) + torch.minimum(w * s / 8, 2.0 ** -13 * top)) / s
            r["lost"][b, i] = (low @ vv.abs()).reshape(H, dv)
            r["mag"][b, i] = (abs(sm) * qq.abs() @ k.abs().transpose(1, 2)).amax(-1).reshape(-1)
            r["top"][b, i] = (abs(sm) * qq.abs().amax(-1) * k.abs().sum(-1).amax(-1)[:, None]).reshape(-1)
            r["wide"][b, i] = t.numel()
    return {k: x.cpu().numpy() for k, x in r.items()}


def _check(c, q, sm, length, sinks, window, idx, count, d, dv, voff, vmax):
    out, lse, st = K.attend(c, q, sm, K.i32(length), sinks, window, idx, None if count is None else K.i32(count), d, dv, voff)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    r = _reference(c, q, sm, length, sinks, window, idx, count, d, dv, voff)
    tol, tl = K.tolerances(q.dtype, d, r, vmax)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isinf(r["lse"])
    assert not got[empty].any() and np.isneginf(gl[empty]).all()
    assert np.all(np.abs(gl - r["lse"])[~empty] <= tl[~empty])
    bad = np.abs(got - r["out"]) > tol
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - r["out"]) / tol).max()))


def _q(seed, B, Tq, H, d, dtype=BF):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((B, Tq, H, d))).to(dtype).cuda()


def _vmax(c):
    return float(_decode(torch.arange(127, device="cuda"))[torch.from_numpy(np.unique(c.codes & 0x7F)).cuda().long()].max()) * float(c.scale.max())


CASES = [  # G, hg, d, dv, voff, W, B, N, block, page, store, Tq, window, sinks
    (1, 64, 576, 512, 0, 576, 40, 2100, 64, 64, "paged", 1, -1, 0),      # latent rows: chunks divided among warps
    (1, 64, 576, 512, 0, 576, 40, 2100, 1, 1, "slots", 1, -1, 0),        # latent rows, scattered
    (1, 64, 576, 512, 0, 576, 33, 1777, 16, 16, "paged", 2, 1000, 5),    # boxes of 16 rows, a window
    (1, 16, 576, 512, 0, 576, 1, 40000, 128, 32, "paged", 1, -1, 0),     # more than one cluster, long parts
    (4, 8, 128, 128, 128, 256, 40, 3001, 64, 64, "paged", 1, -1, 0),     # grouped heads, two blocks an SM
    (4, 8, 128, 128, 128, 256, 24, 3001, 16, 1, "dense", 3, 2500, 4),    # 24 columns, a dense cache
    (8, 8, 128, 128, 128, 256, 3, 20000, 1, 16, "slots", 1, -1, 0),
    (2, 20, 320, 256, 64, 320, 40, 1500, 16, 32, "paged", 1, -1, 0),     # three chunks
    (2, 16, 256, 256, 256, 512, 30, 1500, 64, 128, "paged", 4, -1, 0),   # four chunks, 64 columns
    (3, 5, 64, 64, 64, 128, 60, 2000, 1, 1, "dense", 1, 1999, 1),        # one chunk
    (5, 1, 192, 128, 256, 384, 40, 1300, 32, 64, "slots", 1, -1, 0),     # a tail and a gap
    (1, 12, 72, 40, 200, 240, 50, 900, 4, 8, "slots", 1, -1, 0),         # odd columns
]


@pytest.mark.parametrize("case", CASES)
def test_attend_many_tiles(case):
    G, hg, d, dv, voff, W, B, N, block, page, store, Tq, window, sinks = case
    c = K.Cache(N + W, B, N, G, W, block, page, store)
    length = [N - (b * 7) % (N // 2) for b in range(B)]
    _check(c, _q(d, B, Tq, G * hg, d), d ** -0.5, length, sinks, window, None, None, d, dv, voff, _vmax(c))


@pytest.mark.parametrize("window,sinks,Tq", [(0, 0, 1), (300, 4, 1), (300, 4, 3)])
@pytest.mark.parametrize("G,hg,d,dv,voff,W", [(1, 64, 576, 512, 0, 576), (2, 8, 128, 128, 128, 256)])
def test_attend_long_lists(G, hg, d, dv, voff, W, window, sinks, Tq):
    B, N, cap = 30, 5000, 2000
    c = K.Cache(3, B, N, G, W, 16, 16, "paged")
    g = torch.Generator(device="cuda").manual_seed(1)
    idx = torch.stack([torch.randperm(4000, generator=g, device="cuda")[:cap].sort().values for _ in range(B)]).to(torch.int32)
    idx[3, 500:900] = -1
    idx[4, 64:1024] = torch.arange(128, 1088, device="cuda", dtype=torch.int32)   # entries that follow one another
    count = [cap - 31 * b for b in range(B)]
    _check(c, _q(7, B, Tq, G * hg, d), d ** -0.5, [N - b for b in range(B)], sinks, window, idx, count, d, dv, voff, _vmax(c))


def test_attend_weights_rise_with_every_tile():
    """References move in many tiles of one block, by few columns and by all of them."""
    G, hg, d, dv, voff, W, B, N = 1, 64, 576, 512, 0, 576, 40, 1900
    c = K.Cache(9, B, N, G, W, 1, 64, "dense")
    c.codes[..., 600 % W] = 0x38                                        # column 24: 1.0
    c.scale[:, :, 0] = 2.0 ** -6
    c.push()
    lift = torch.linspace(0, 60, N, device="cuda")
    c.scale_d[:, :, 0] *= torch.exp2((lift / 6).floor())               # scales rise 2^10 over the sequence
    q = _q(2, B, 1, hg, d)
    q[:, :, 5, 24] = 8.0
    q[:, :, 6, 24] = -8.0
    c.scale = c.scale_d.cpu().numpy()
    _check(c, q, 0.02, [N] * B, 0, -1, None, None, d, dv, voff, _vmax(c))


def test_cache_past_four_gigabytes():
    """Rows, list entries and windows beyond 2^32 bytes: write, read and both ways of bringing
    rows into the attention."""
    W, N, B = 576, 4_000_000, 2
    rows = torch.zeros(B * N, 1, 1, W, dtype=torch.uint8, device="cuda")
    scale = torch.full((B, N, 1), 2.0 ** -6, device="cuda")
    T = 700
    x = _q(1, B, T, 1, W)
    start = K.i32([N - T, N - T])
    cache = (1, 1, N, B * N, None, rows, scale)
    lsa.lsa_kv_write(B, T, N, 1, W, 1, x, W, start, None, *cache)
    back = torch.zeros(B, T, 1, W, dtype=F32, device="cuda")
    idx = torch.arange(N - T, N, device="cuda", dtype=torch.int32).expand(B, T).contiguous()
    lsa.lsa_kv_read(B, N, 1, W, idx, T, K.i32([T, T]), *cache, lsa.LSA_F32, back)
    torch.cuda.synchronize()
    s = scale[:, N - T:, 0].double()[:, :, None, None]
    err = (back.double() - x.double()).abs()
    assert bool((err <= back.double().abs() * 2.0 ** -4 + s * 2.0 ** -10).all())
    c = type("C", (), dict(N=N, G=1, W=W, block=1, page=1, seq_pages=N, pages=B * N, table_d=None, rows_d=rows, scale_d=scale,
                           args=lambda self: cache))()
    vmax = 448.0 * float(scale.max())
    q = _q(3, B, 1, 64, W)
    _check(c, q, W ** -0.5, [N, N - 5], 0, 650, None, None, W, 512, 0, vmax)
    _check(c, q, W ** -0.5, [N, N], 0, 0, idx, [T, T - 100], W, 512, 0, vmax)


def test_two_calls_at_once():
    """Calls on two streams with workspaces of their own, many times over, are each the same bits
    as alone."""
    G, hg, d, dv, voff, W, N = 1, 64, 576, 512, 0, 576, 40000
    c1, c2 = K.Cache(1, 1, N, G, W, 64, 64, "paged"), K.Cache(2, 4, 3000, 4, 256, 16, 16, "paged")
    q1, q2 = _q(1, 1, 1, hg, d), _q(2, 4, 2, 32, 128)
    a1 = K.attend(c1, q1, 0.05, K.i32([N]), 0, -1, None, None, d, dv, voff)
    a2 = K.attend(c2, q2, 0.1, K.i32([3000, 100, 2000, 1]), 4, 500, None, None, 128, 128, 128)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(6):
        with torch.cuda.stream(s1):
            b1 = K.attend(c1, q1, 0.05, K.i32([N]), 0, -1, None, None, d, dv, voff)
        with torch.cuda.stream(s2):
            b2 = K.attend(c2, q2, 0.1, K.i32([3000, 100, 2000, 1]), 4, 500, None, None, 128, 128, 128)
        got.append((b1, b2))
    torch.cuda.synchronize()
    for b1, b2 in got:
        assert torch.equal(b1[0], a1[0]) and torch.equal(b1[1], a1[1])
        assert torch.equal(b2[0], a2[0]) and torch.equal(b2[1], a2[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_empty_calls(dtype):
    q = torch.zeros(2, 1, 4, 64, dtype=dtype, device="cuda")
    c = K.Cache(1, 2, 16, 2, 128, 1, 1, "dense")
    out, lse, _ = K.attend(c, q, 1.0, K.i32([0, 0]), 4, 8, None, None, 64, 64, 64)
    torch.cuda.synchronize()
    assert not out.any() and torch.isneginf(lse).all()
    dt = lsa.dtype_code(q)
    size = (2, 1, 0, 4, 2, 64, 64, 64, 128)
    ws = lsa.workspace(lsa.lsa_kv_attend_workspace_bytes(*size, dt, 0, -1, 0))
    out.fill_(1.0)
    empty = (1, 1, 0, 0, None, c.rows_d, c.scale_d)
    lsa.lsa_kv_attend(*size, dt, q, 1.0, K.i32([0, 0]), 0, -1, None, 0, None, *empty, out, lse, ws)      # a cache of no tokens
    torch.cuda.synchronize()
    assert not out.any() and torch.isneginf(lse).all()


@pytest.mark.parametrize("d,dv,voff,W,hg", [(576, 512, 0, 576, 33), (128, 128, 128, 256, 5), (72, 37, 101, 144, 3)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_guards_kv(dtype, d, dv, voff, W, hg):
    """Ragged sizes between canaries: nothing outside the outputs is written."""
    B, N, G, cap = 3, 777, 2, 131
    c = K.Cache(5, B, N, G, W, 16, 1, "dense")
    rows = Guarded(tuple(c.codes.shape), torch.uint8)
    rows.t.copy_(c.rows_d)
    scale = Guarded(tuple(c.scale.shape), torch.float32)
    scale.t.copy_(c.scale_d)
    c.rows_d, c.scale_d = rows.t, scale.t
    H = G * hg
    q = _q(1, B, 2, H, d, dtype)
    out, lse, st = Guarded((B, 2, H, dv), dtype), Guarded((B, 2, H), torch.float32), Guarded((1,), torch.int32)
    dt = lsa.dtype_code(q)
    size = (B, 2, N, H, G, d, dv, voff, W)
    ws = Guarded((lsa.lsa_kv_attend_workspace_bytes(*size, dt, 3, 100, cap),), torch.uint8)
    idx = torch.randint(0, 600, (B, cap), device="cuda", dtype=torch.int32)
    lsa.lsa_kv_attend(*size, dt, q, 0.1, K.i32([N, 1, 300]), 3, 100, idx, cap, K.i32([cap, 2, 0]), *c.args(), out.t, lse.t, ws.t, st.t)
    back = Guarded((B, cap, G, W), dtype)
    lsa.lsa_kv_read(B, N, G, W, idx, cap, K.i32([cap, 1, 50]), *c.args(), dt, back.t, st.t)
    x = _q(4, B, 45, G, W, dtype)
    lsa.lsa_kv_write(B, 45, N, G, W, dt, x, G * W, K.i32([3, 700, N - 45]), None, *c.args(), st.t)
    ro = Guarded((B, 45, G, 10), dtype)
    f = lsa.lsa_rope_frequencies(10).cuda()
    lsa.lsa_rope(B * 45, G, 10, 1, dt, x, G * W, W, K.i32(np.arange(B * 45)), f, 1.0, 0, ro.t, G * 10, 10)
    torch.cuda.synchronize()
    for t in (rows, scale, out, lse, st, ws, back, ro):
        assert t.intact()


@pytest.mark.parametrize("B,G,hg,d,dv,voff,W,N,cap", [
    (1, 1, 8, 576, 512, 0, 576, 500, 0),       # few columns: every warp of a block on one
    (1, 1, 1, 576, 512, 512, 1024, 200, 0),    # rows wider than what is read ahead
    (2, 2, 3, 36, 60, 100, 176, 333, 0),       # a short score, shared out among two warps
    (2, 1, 11, 33, 31, 34, 80, 150, 20),       # columns that take no vectors, with a list
    (75, 2, 8, 64, 64, 64, 128, 70, 40),       # blocks for every SM: a warp a column
    (30, 1, 16, 96, 80, 96, 176, 130, 9)])
def test_attend_f32_teams(B, G, hg, d, dv, voff, W, N, cap):
    """fp32 queries over every division of a block's warps among columns."""
    c = K.Cache(d, B, N, G, W, 4, 8, "slots")
    g = np.random.default_rng(B)
    q = torch.from_numpy(g.standard_normal((B, 2, G * hg, d))).float().cuda()
    length = [max(2, N - 13 * b) for b in range(B)]
    idx = count = None
    if cap:
        idx = np.stack([g.integers(-1, n, size=cap) for n in length]).astype(np.int32)
        count = g.integers(0, cap + 1, size=B)
    K.check_attend(c, q, d ** -0.5, length, 3 if cap else 0, 50 if cap else -1, idx, count, d, dv, voff)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_to_any_aligned_output(dtype):
    """Outputs on 16 bytes that are not on 32 get the same rows as others."""
    B, N, G, W, cap = 3, 90, 2, 48, 37
    c = K.Cache(8, B, N, G, W, 4, 8, "paged")
    idx = K.i32(np.random.default_rng(1).integers(-1, N, size=(B, cap)))
    count = K.i32([cap, 11, 0])
    n, step = B * cap * G * W, 128 // torch.finfo(dtype).bits
    outs = []
    for off in (0, step):
        buf = torch.full((n + 2 * step,), 5.0, dtype=dtype, device="cuda")
        lsa.lsa_kv_read(B, N, G, W, idx, cap, count, *c.args(), lsa.dtype_code(dtype), buf[off: off + n])
        torch.cuda.synchronize()
        assert (buf[:off] == 5).all() and (buf[off + n:] == 5).all()
        outs.append(buf[off: off + n])
    assert (outs[0].data_ptr() % 32, outs[1].data_ptr() % 32) == (0, 16)
    assert torch.equal(outs[0], outs[1]) and (outs[0] != 5).any()


@pytest.mark.parametrize("G,hg,d,dv,voff,W,B,N", [(1, 8, 576, 512, 0, 576, 150, 1900), (8, 5, 128, 128, 128, 256, 40, 2000),
                                                  (2, 3, 64, 64, 64, 128, 150, 1500), (1, 9, 128, 128, 128, 256, 300, 1300)])
def test_attend_few_columns_with_rising_weights(G, hg, d, dv, voff, W, B, N):
    """Blocks with at most eight columns (and with one more): references that move in many tiles, for
    some columns and for all of them, and one column that falls."""
    c = K.Cache(13, B, N, G, W, 1, 64, "dense")
    c.codes[..., 24] = 0x38                                            # column 24: 1.0
    c.scale[:] = np.exp2(np.floor(np.linspace(0, 10, N)) - 6)[None, :, None]
    c.push()
    q = _q(3, B, 1, G * hg, d)
    q[::2, :, :, 24] = 8.0                                             # all columns of every second sequence rise
    q[:, :, 1, 24] = -8.0
    q[1::4, :, 2, 24] = 12.0
    _check(c, q, 0.02, [N - b for b in range(B)], 0, -1, None, None, d, dv, voff, _vmax(c))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_two_host_threads(dtype):
    """Calls of two sizes from two host threads, each on its own stream: the larger one's shared memory
    must not depend on what the other thread launches in between."""
    import threading

    work = []
    for G, hg, d, dv, voff, W, N in [(1, 12, 576, 512, 0, 576, 400), (2, 4, 64, 64, 64, 128, 90)]:
        c = K.Cache(d, 2, N, G, W, 16, 16, "paged")
        q = _q(W, 2, 1, G * hg, d, dtype)
        args = (c, q, d ** -0.5, K.i32([N, N - 7]), 0, -1, None, None, d, dv, voff)
        want, _, _ = K.attend(*args)
        work.append((args, want))
    torch.cuda.synchronize()
    failed = []

    def run(args, want):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(150):
                    out, _, st = K.attend(*args)
                    s.synchronize()
                    assert torch.equal(out, want) and int(st.item()) == 0
        except Exception as e:                                         # noqa: BLE001 (shown below)
            failed.append(e)

    threads = [threading.Thread(target=run, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
