"""Parity of the 8-bit KV cache calls and of the rotary positions with the fp64 oracle: every
element, at the sizes, layouts and masks where each can go wrong."""
import math

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import build
from oracle import kv as OK

import kv_cases as K
import lsa_cases as C

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    lsa.lib()


def _x(seed, shape, dtype, spread=1.0):
    g = np.random.default_rng(seed)
    m = np.exp(spread * g.standard_normal(shape[:2] + (1,) * (len(shape) - 2)))
    return torch.from_numpy(g.standard_normal(shape) * m).to(dtype).cuda()


# ----------------------------------------------------------------------------- write

def _write(c, x, start, count, x_stride=None, T=None, stream=None):
    B = c.B
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lsa.lsa_kv_write(B, T or x.shape[1], c.N, c.G, c.W, lsa.dtype_code(x), x, x_stride or c.G * c.W, K.i32(start),
                     None if count is None else K.i32(count), *c.args(), st, stream=stream)
    return st


def _same_cache(c, want):
    """Codes and scales equal the oracle's, bit for bit (NaN scales in the same places)."""
    torch.cuda.synchronize()
    got = c.scale_d.cpu().double().numpy()
    assert np.array_equal(np.nan_to_num(got, nan=-1.0), np.nan_to_num(want.scale, nan=-1.0))
    a, b = c.rows_d.cpu().numpy(), want.rows
    zero = ((a | b) & 0x7F) == 0                              # +0 and -0 are one value
    assert np.array_equal(np.where(zero, 0, a), np.where(zero, 0, b))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("store", ["dense", "paged", "slots"])
@pytest.mark.parametrize("block,page,G,W,T", [(1, 1, 1, 576, 1), (1, 1, 3, 16, 5), (16, 4, 2, 144, 37), (64, 64, 2, 256, 130),
                                             (128, 16, 1, 576, 200), (4, 32, 5, 48, 1)])
def test_write_matches_oracle(dtype, store, block, page, G, W, T):
    B, N = 3, T + 150
    c = K.Cache(T + W, B, N, G, W, block, page, store)
    x = _x(W + block, (B, T, G, W), dtype)
    start, count = [0, 5, 149], [T, max(T - 1, 0), T]
    want = c.oracle()
    assert not OK.write(want, x.double().cpu().numpy(), start, count)
    st = _write(c, x, start, count)
    _same_cache(c, want)
    assert int(st.item()) == 0
    # tokens appended one at a time behind them, larger and smaller than what is there
    at = np.array(start) + np.array(count)
    for k, mag in enumerate((1e-3, 30.0, 1.0)):
        y = _x(900 + k, (B, 1, G, W), dtype) * mag
        go = np.minimum(at, N - 1)
        OK.write(want, y.double().cpu().numpy(), go, [1, 1, 0])
        _write(c, y, go, [1, 1, 0])
        at = at + 1
    _same_cache(c, want)


def test_write_ranges_padding_and_strides():
    """Tokens past N, a negative start and missing pages are skipped and reported; a strided
    source; sequences with nothing to write; bytes behind the last token stay."""
    B, N, G, W, block, page = 4, 40, 2, 32, 8, 4
    c = K.Cache(3, B, N, G, W, block, page, "slots")
    c.table[2, 3] = -1                                         # tokens 12..15 of sequence 2
    c.table[3, 0] = 99                                         # outside the sequence's pool
    c.push()
    want = c.oracle()
    wide = _x(5, (B, 6, 3 * G * W), BF)
    x = wide[:, :, G * W: 2 * G * W]                           # a slice of a wider activation
    start, count = [38, 7, 10, 0], [6, 0, 6, 5]
    assert OK.write(want, x.reshape(B, 6, G, W).double().cpu().numpy(), start, count)
    st = _write(c, x, start, count, x_stride=3 * G * W, T=6)
    _same_cache(c, want)
    assert int(st.item()) == lsa.LSA_ERR_RANGE
    before = c.rows_d.clone()
    st = _write(c, x, [-1, 0, 0, 0], [6, 0, 0, 0], x_stride=3 * G * W, T=6)
    torch.cuda.synchronize()
    assert int(st.item()) == lsa.LSA_ERR_RANGE and torch.equal(before, c.rows_d)


def test_write_special_values():
    """Zeros, subnormals, the largest finite value, NaN and infinities, exact halves."""
    B, T, G, W = 1, 8, 1, 32
    c = K.Cache(1, B, 16, G, W, 1, 1, "dense")
    x = torch.zeros(B, T, G, W)
    x[0, 1, 0, 0] = math.nan
    x[0, 2, 0, 3] = -math.inf
    x[0, 3, 0] = 3.0e38
    x[0, 4, 0] = 1e-40
    x[0, 5, 0, :4] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10])     # ties: 17 -> 16, 19 -> 20, 2^-10 -> 0
    x[0, 6, 0, :2] = torch.tensor([448.01, -448.01])
    x[0, 7, 0, :3] = torch.tensor([2.0 ** -24 * 100, 2.0 ** -33, -2.0 ** -34])
    x = x.cuda()
    want = c.oracle()
    OK.write(want, x.double().cpu().numpy(), [0], [T])
    _write(c, x, [0], None)
    _same_cache(c, want)
    assert math.isnan(c.scale_d[0, 1, 0]) and math.isnan(c.scale_d[0, 2, 0]) and c.scale_d[0, 0, 0] == 2.0 ** -24


def test_write_makes_indexer_keys():
    """Rows written with one head and no table are a K_IComp array: the score reads them."""
    w = C.W.scaled(C.W.WORKLOADS["lsa_step_128k_b1_bf16"], N=2048, L=1)
    g = np.random.default_rng(8)
    keys = torch.from_numpy(g.standard_normal((1, w.N, 1, w.dI))).to(BF).cuda()
    K8 = torch.zeros(1, 1, w.N, w.dI, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(1, 1, w.N, device="cuda")
    lsa.lsa_kv_write(1, w.N, w.N, 1, w.dI, lsa.LSA_BF16, keys, w.dI, K.i32([0]), None, 1, 1, w.N, w.N, None, K8, ks)
    q = torch.from_numpy(g.standard_normal((1, 1, w.H, w.dI))).to(BF).cuda()
    wv = torch.from_numpy(g.standard_normal((1, 1, w.H))).float().cuda()
    bias = torch.zeros(4, device="cuda")
    mask = torch.zeros(1, 1, (w.N + 31) // 32, dtype=torch.int32, device="cuda")
    z = torch.zeros(1, 1, w.N, device="cuda")
    ws = lsa.workspace(lsa.lsa_index_score_workspace_bytes(1, 1, w.N, w.D, w.r, w.H, w.dI, 1, 2))
    lsa.lsa_index_score(1, 1, w.N, w.D, w.r, w.H, w.dI, 1, None, None, None, None, bias, 2, K8, ks, -1, q, wv, None,
                        None, mask, z, None, ws)
    torch.cuda.synchronize()
    kd = OK.O.decode_e4m3(K8[0, 0].cpu().numpy()) * ks[0, 0].double().cpu().numpy()[:, None]
    want = np.maximum(kd @ q[0, 0].double().cpu().numpy().T, 0) @ wv[0, 0].double().cpu().numpy()
    assert np.all(np.abs(z[0, 0].double().cpu().numpy() - want) <= C.tol_z("e4m3"))
    err = np.abs(kd - keys[0, :, 0].double().cpu().numpy())
    assert np.all(err <= np.abs(kd) * 2.0 ** -4 + ks[0, 0].double().cpu().numpy()[:, None] * 2.0 ** -10)


# ----------------------------------------------------------------------------- read

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,page,G,W,store", [(1, 1, 1, 576, "slots"), (16, 4, 3, 16, "paged"), (64, 64, 2, 144, "dense")])
def test_read_matches_oracle(dtype, block, page, G, W, store):
    B, N, cap = 3, 301, 77
    c = K.Cache(W, B, N, G, W, block, page, store, spread=12)
    g = np.random.default_rng(2)
    idx = g.integers(0, N, size=(B, cap)).astype(np.int32)     # repeats among them
    idx[0, 5:9] = -1
    count = [cap, 0, 40]
    out = torch.full((B, cap, G, W), 7.0, dtype=dtype, device="cuda")
    want = np.full((B, cap, G, W), 7.0)
    assert not OK.read(c.oracle(), idx, count, want)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lsa.lsa_kv_read(B, N, G, W, K.i32(idx), cap, K.i32(count), *c.args(), lsa.dtype_code(dtype), out, st)
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want) and int(st.item()) == 0   # code * 2^k is exact in bf16 too


def test_read_whole_prefix_and_bad_entries():
    B, N, G, W = 2, 50, 2, 32
    c = K.Cache(4, B, N, G, W, 8, 4, "slots")
    c.table[1, 2] = -1
    c.push()
    out = torch.full((B, 20, G, W), 7.0, device="cuda")
    want = np.full((B, 20, G, W), 7.0)
    OK.read(c.oracle(), np.tile(np.arange(20), (B, 1)), [20, 20], want)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lsa.lsa_kv_read(B, N, G, W, None, 20, None, *c.args(), lsa.LSA_F32, out, st)
    torch.cuda.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want) and int(st.item()) == lsa.LSA_ERR_RANGE
    st.zero_()
    out.fill_(3.0)
    lsa.lsa_kv_read(B, N, G, W, K.i32([[50], [0]]), 1, K.i32([1, 9]), *c.args(), lsa.LSA_F32, out, st)
    torch.cuda.synchronize()
    assert int(st.item()) == lsa.LSA_ERR_RANGE and (out.view(-1)[: G * W] == 3.0).all()


# ----------------------------------------------------------------------------- rope

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("R,H,D,rot", [(1, 1, 64, 64), (5, 3, 96, 40), (33, 64, 576, 64), (7, 5, 10, 2), (3, 2, 130, 128)])
def test_rope_matches_oracle(dtype, half, R, H, D, rot):
    g = np.random.default_rng(R + rot)
    x = torch.from_numpy(g.standard_normal((R, H, D))).to(dtype).cuda()
    pos = g.integers(0, 1 << 20, size=R)
    pos[0] = (1 << 31) - 1 if R > 1 else 0
    f = lsa.lsa_rope_frequencies(rot, factor=8.0, original=4096)
    for inverse in (0, 1):
        out = torch.full((R, H, rot), float("nan"), dtype=dtype, device="cuda")
        xr = x[:, :, D - rot:]
        lsa.lsa_rope(R, H, rot, half, lsa.dtype_code(x), xr, H * D, D, K.i32(pos), f.cuda(), 1.25, inverse, out,
                     H * rot, rot)
        torch.cuda.synchronize()
        want = OK.rope(xr.double().cpu().numpy(), pos, f.numpy(), half, 1.25, inverse)
        # sine and cosine: 2^-25 of a turn in the angle (2 pi 2^-25), 2 ulp each; products and sum
        # 3 * 2^-24, of at most mscale (|u| + |v|); the result rounded by half a step
        u = np.abs(xr.double().cpu().numpy())
        n = rot // 2
        pair = np.concatenate([u[..., :n] + u[..., n:]] * 2, -1) if half else np.repeat(u[..., 0::2] + u[..., 1::2], 2, -1)
        tol = 1.25 * pair * (2 * math.pi * 2.0 ** -25 + 2.0 ** -22 + 3 * 2.0 ** -24)
        tol = tol + np.abs(want) * torch.finfo(dtype).eps / 2
        assert np.all(np.abs(out.double().cpu().numpy() - want) <= tol)


def test_rope_in_place_leaves_other_columns():
    R, H, D, rot = 9, 3, 576, 64
    x = _x(1, (R, H, D), BF)
    keep = x.clone()
    f = lsa.lsa_rope_frequencies(rot).cuda()
    pos = K.i32(np.arange(R))
    out = torch.empty(R, H, rot, dtype=BF, device="cuda")
    lsa.lsa_rope(R, H, rot, 0, 1, x[:, :, 512:], H * D, D, pos, f, 1.0, 0, out, H * rot, rot)
    lsa.lsa_rope(R, H, rot, 0, 1, x[:, :, 512:], H * D, D, pos, f, 1.0, 0, x[:, :, 512:], H * D, D)
    torch.cuda.synchronize()
    assert torch.equal(x[:, :, 512:], out) and torch.equal(x[:, :, :512], keep[:, :, :512])
    assert torch.equal(x[0], keep[0])                          # position 0 does not turn
    # heads-major storage [H][R][rot]: the head stride is the larger one
    y = keep[:, :, 512:].permute(1, 0, 2).contiguous()
    lsa.lsa_rope(R, H, rot, 0, 1, y, rot, R * rot, pos, f, 1.0, 0, y, rot, R * rot)
    torch.cuda.synchronize()
    assert torch.equal(y.permute(1, 0, 2), out)


# ----------------------------------------------------------------------------- attend

SHAPES = [  # G, heads a KV head, d, dv, voff, W
    (1, 64, 576, 512, 0, 576), (1, 8, 576, 512, 0, 576), (1, 128, 576, 512, 0, 576), (1, 33, 576, 512, 0, 576),
    (4, 8, 128, 128, 128, 256), (2, 5, 64, 64, 64, 128), (3, 1, 192, 128, 256, 384), (2, 16, 96, 80, 96, 176),
    (1, 3, 40, 24, 8, 48), (2, 4, 256, 256, 256, 512), (1, 20, 320, 256, 64, 320)]


def _q(seed, B, Tq, H, d, dtype):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((B, Tq, H, d))).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G,hg,d,dv,voff,W", SHAPES)
def test_attend_shapes(dtype, G, hg, d, dv, voff, W):
    """Every visible token, ragged lengths (one token, a tile's edges, none)."""
    N = 300
    length = [300, 1, 0, 129, 128]
    c = K.Cache(W + d, 5, N, G, W, 16, 16, "paged")
    q = _q(d + hg, 5, 1, G * hg, d, dtype)
    K.check_attend(c, q, d ** -0.5, length, 0, -1, None, None, d, dv, voff)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sinks,window,Tq", [(0, -1, 3), (4, 37, 1), (4, 37, 5), (0, 1, 2), (7, 0, 2), (0, 0, 1), (200, 200, 4),
                                             (3, 129, 9), (0, 2 ** 31 - 1, 3), (2 ** 31 - 1, 5, 2)])
@pytest.mark.parametrize("shape", [0, 4])
def test_attend_windows_and_first_tokens(dtype, sinks, window, Tq, shape):
    G, hg, d, dv, voff, W = SHAPES[shape]
    hg = min(hg, 12)
    N = 333
    length = [333, 2, 131, 40]
    c = K.Cache(Tq + sinks % 100, 4, N, G, W, 64, 16, "slots")
    q = _q(Tq, 4, Tq, G * hg, d, dtype)
    K.check_attend(c, q, d ** -0.5, length, sinks, window, None, None, d, dv, voff)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sinks,window,Tq", [(0, 0, 1), (0, 0, 3), (2, 20, 1), (2, 20, 4)])
@pytest.mark.parametrize("shape", [0, 4])
def test_attend_lists(dtype, sinks, window, Tq, shape):
    """Listed entries with padding, repeats, an empty list and entries the window holds too."""
    G, hg, d, dv, voff, W = SHAPES[shape]
    hg = min(hg, 16)
    B, N, cap = 5, 400, 150
    g = np.random.default_rng(7)
    length = [400, 300, 350, 12, 0]
    idx = np.full((B, cap), -1, dtype=np.int32)
    count = [150, 0, 131, 60, 150]
    for b in range(B):
        if length[b]:
            idx[b] = g.integers(0, length[b], size=cap)
    idx[0, 3:140:5] = -1
    idx[2, :129] = -1                                          # a whole tile of padding
    c = K.Cache(11, B, N, G, W, 1, 1, "slots")
    q = _q(Tq + 1, B, Tq, G * hg, d, dtype)
    K.check_attend(c, q, d ** -0.5, length, sinks, window, idx, count, d, dv, voff)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_missing_pages_and_bad_entries(dtype):
    """Tokens that are not resident and entries past the length are skipped and reported."""
    G, hg, d, dv, voff, W = SHAPES[4]
    c = K.Cache(3, 2, 200, G, W, 4, 8, "slots")
    c.table[0, 3:9] = -1
    c.table[1, 2] = 1000
    c.push()
    q = _q(9, 2, 1, G * hg, d, dtype)
    K.check_attend(c, q, 0.1, [200, 90], 0, -1, None, None, d, dv, voff, status=lsa.LSA_ERR_RANGE)
    idx = np.array([[5, 199, 60, -1], [89, 90, 2 ** 30, 3]], dtype=np.int32)
    K.check_attend(c, q, 0.1, [200, 90], 0, 0, idx, [4, 4], d, dv, voff, status=lsa.LSA_ERR_RANGE)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_steep_scores_and_uneven_scales(dtype):
    """Scores that rise along the sequence (every tile raises the maximum), that fall, that all
    sit in one token, that are equal, and neighbouring scales 2^18 apart."""
    G, hg, d, dv, voff, W = 1, 16, 128, 128, 128, 256
    N = 700
    c = K.Cache(5, 3, N, G, W, 1, 1, "dense")
    g = np.random.default_rng(1)
    c.codes[..., 0] = 0x30                                     # 0.5: column 0 carries the trend
    c.scale[0, :, 0] = np.exp2(np.linspace(-12, 0, N).round())
    c.scale[1, :, 0] = np.exp2(np.linspace(0, -12, N).round())
    c.scale[2, :, 0] = np.exp2(g.choice([-12, 6], size=N))
    c.push()
    q = _q(4, 3, 1, G * hg, d, dtype)
    q[:, :, 1:, 0] = 40.0
    q[:, :, 2, :] = 0.0                                        # equal scores
    q[:, :, 3, 0] = -40.0
    K.check_attend(c, q, 0.3, [N, N, N], 0, -1, None, None, d, dv, voff)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_large_and_small_queries(dtype):
    """Query rows of zeros, tiny and huge elements, and one huge element among tiny ones."""
    G, hg, d, dv, voff, W = 1, 8, 576, 512, 0, 576
    c = K.Cache(6, 1, 260, G, W, 1, 1, "dense")
    q = _q(4, 1, 1, hg, d, torch.float32)
    q[0, 0, 0] = 0
    q[0, 0, 1] *= 1e-30
    q[0, 0, 2] *= 1e-3
    q[0, 0, 3, 7] = 3000.0
    q[0, 0, 4] *= 50
    K.check_attend(c, q.to(dtype), 0.05, [260], 0, -1, None, None, d, dv, voff)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_non_finite_tokens(dtype):
    """A token marked non-finite makes the queries that see it NaN and no other; codes of rows
    that nobody sees may be anything."""
    G, hg, d, dv, voff, W = SHAPES[4]
    N, Tq, L = 260, 3, 250
    c = K.Cache(8, 1, N, G, W, 1, 1, "dense")
    c.scale[0, 249] = math.nan                                 # seen by the last query alone
    c.codes[249] = 0
    c.scale[0, 100] = math.nan                                 # outside every window
    c.codes[100] = 0
    c.codes[L:] = 0x7F                                         # stale rows behind the sequence
    c.scale[0, L:] = math.nan
    c.codes[30] = 0x7F                                         # an unseen row with NaN codes
    c.push()
    q = _q(3, 1, Tq, G * hg, d, dtype)
    out, lse, st = K.attend(c, q, 0.1, K.i32([L]), 5, 100, None, None, d, dv, voff)
    torch.cuda.synchronize()
    assert torch.isfinite(out[0, :2]).all() and torch.isfinite(lse[0, :2]).all()
    assert torch.isnan(out[0, 2]).all() and torch.isnan(lse[0, 2]).all() and int(st.item()) == 0
    clean = K.Cache(8, 1, N, G, W, 1, 1, "dense")
    ref, rl, _ = K.attend(clean, q, 0.1, K.i32([L]), 5, 100, None, None, d, dv, voff)
    torch.cuda.synchronize()
    assert torch.equal(out[0, :2], ref[0, :2]) and torch.equal(lse[0, :2], rl[0, :2])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_repeats_and_shared_pool(dtype):
    """The same call twice is the same bits; all sequences may read one shared prefix."""
    G, hg, d, dv, voff, W = SHAPES[0]
    c = K.Cache(2, 1, 1500, G, W, 64, 16, "paged")
    q = _q(5, 3, 1, 64, d, dtype)
    share = lambda x: x.expand(3, *x.shape[1:]).contiguous()  # noqa: E731
    c.B, c.table_d, c.scale_d = 3, share(c.table_d), share(c.scale_d)
    a = K.attend(c, q, 0.05, K.i32([1500, 700, 1500]), 4, 1000, None, None, d, dv, voff)
    b = K.attend(c, q, 0.05, K.i32([1500, 700, 1500]), 4, 1000, None, None, d, dv, voff)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.table, c.scale, c.B = np.tile(c.table, (3, 1)), np.tile(c.scale, (3, 1, 1)), 3
    r = OK.attend(c.oracle(), q.double().cpu().numpy(), 0.05, [1500, 700, 1500], 4, 1000, None, None, d, dv, voff)
    tol, _ = K.tolerances(dtype, d, r, 64.0 * float(c.scale.max()))
    assert np.all(np.abs(a[0].double().cpu().numpy() - r["out"]) <= tol)


# ----------------------------------------------------------------------------- together

def test_decode_step_through_the_pool():
    """One trigger and decode step as they are used: latent rows rotated and written, fetched
    in 8 bits from the cold pool through the residency update, the top-k inside the fetched set,
    attention over it, and the read-back of the same entries; on a side stream, then captured
    and replayed on new inputs."""
    B, N, H, k, W = 2, 1024, 64, 96, 576
    g = np.random.default_rng(0)
    dev = torch.device("cuda")
    x = torch.from_numpy(g.standard_normal((B, N, 1, W))).to(BF).to(dev)
    pos = K.i32(np.tile(np.arange(N), B))
    f = lsa.lsa_rope_frequencies(64, factor=16.0, original=65536).to(dev)
    xr = x.view(B * N, 1, W)[:, :, 512:]
    lsa.lsa_rope(B * N, 1, 64, 0, 1, xr, W, W, pos, f, 1.0, 0, xr, W, W)
    full = torch.zeros(B * N, 1, 1, W, dtype=torch.uint8, device=dev)
    scale = torch.zeros(B, N, 1, device=dev)
    start = K.i32([0] * B)
    lsa.lsa_kv_write(B, N, N, 1, W, 1, x, W, start, None, 1, 1, N, B * N, None, full, scale)
    torch.cuda.synchronize()
    cold = full.view(B, N, W).cpu().pin_memory()               # the cold pool: 576 bytes an entry
    marks = g.random((B, N)) < 0.2
    U = torch.from_numpy(OK.O.pack_bits(marks).view(np.int32)).to(dev)
    slots = 300
    state = torch.zeros(lsa.lsa_hot_pool_state_bytes(B, N, slots), dtype=torch.uint8, device=dev)
    hws = lsa.workspace(lsa.lsa_hot_pool_workspace_bytes(B, N, slots))
    hot = torch.zeros(B * slots, 1, 1, W, dtype=torch.uint8, device=dev)
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    off = lsa.lsa_hot_pool_layout(B, N, slots)
    table = state[off[0]: off[0] + 4 * B * N].view(torch.int32).view(B, N)
    idx = torch.zeros(B, N, dtype=torch.int32, device=dev)
    cnt = torch.zeros(B, dtype=torch.int32, device=dev)
    logit = torch.from_numpy(g.standard_normal((1, B, N))).float().to(dev)
    topk = torch.zeros(B, k, dtype=torch.int32, device=dev)
    tcnt = torch.zeros(B, dtype=torch.int32, device=dev)
    tws = lsa.workspace(lsa.lsa_topk_workspace_bytes(B, N))
    q = _q(1, B, 1, H, W, BF)
    out, lse = torch.zeros(B, 1, H, 512, dtype=BF, device=dev), torch.zeros(B, 1, H, device=dev)
    back = torch.zeros(B, k, 1, W, dtype=BF, device=dev)
    length = K.i32([N] * B)
    size = (B, 1, N, H, 1, W, 512, 0, W)
    ws = lsa.workspace(lsa.lsa_kv_attend_workspace_bytes(*size, 1, 0, 0, k))

    def step():
        lsa.lsa_compact(B, N, U, N, idx, cnt)
        lsa.lsa_topk(B, 1, N, k, idx, N, cnt, logit, topk, tcnt, tws)
        lsa.lsa_kv_attend(*size, 1, q, W ** -0.5, length, 0, 0, topk, k, tcnt, 1, 1, slots, B * slots, table, hot,
                          scale, out, lse, ws, st)
        lsa.lsa_kv_read(B, N, 1, W, topk, k, tcnt, 1, 1, slots, B * slots, table, hot, scale, 1, back, st)

    def check():
        tk, tc = topk.cpu().numpy(), tcnt.cpu().numpy()
        c = OK.Cache(cold.numpy().reshape(B * N, 1, 1, W), scale.double().cpu().numpy(), None, N, 1, 1, N)
        r = OK.attend(c, q.double().cpu().numpy(), W ** -0.5, [N] * B, 0, 0, tk, tc, W, 512, 0)
        tol, tl = K.tolerances(BF, W, r, 448.0 * float(scale.max()))
        assert np.all(np.abs(out.double().cpu().numpy() - r["out"]) <= tol)
        assert np.all(np.abs(lse.double().cpu().numpy() - r["lse"]) <= tl)
        want = np.zeros((B, k, 1, W))
        OK.read(c, tk, tc, want)
        assert np.array_equal(back.double().cpu().numpy(), want) and int(st.item()) == 0

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lsa.lsa_hot_pool_reset(B, N, slots, state)
        lsa.lsa_hot_pool_update(B, N, slots, W, 1, U, cold, hot, state, None, st, hws)
        step()
    side.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    q.copy_(_q(2, B, 1, H, W, BF))
    logit.copy_(torch.from_numpy(g.standard_normal((1, B, N))).float())
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    check()
