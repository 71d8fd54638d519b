"""Precision of the bf16 attention's softmax weights where one token takes almost all of the weight and
carries little or no value (a first token that every query looks at): what the other tokens add must
come out as with bf16 weights."""
import math

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import build

import kv_cases as K
from test_gpu_kv_large import _reference, _values

pytestmark = pytest.mark.gpu

SHAPES = [  # G, hg, d, dv, voff, W; column of the heavy key, outside the values
    (2, 8, 128, 128, 128, 256, 0), (2, 24, 64, 64, 64, 128, 0), (1, 64, 576, 512, 0, 576, 575)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    lsa.lib()


def _case(seed, shape, B, N, heavy, margin, value, Tq=1):
    """Normal keys and values, scores of deviation 1; the tokens `heavy` have one key column of their own,
    which lifts their scores `margin` above every other token's, and `value` times a normal value."""
    G, hg, d, dv, voff, W, col = shape
    g = np.random.default_rng(seed)
    c = K.Cache(seed, B, N, G, W, 1, 16, "paged")
    x = torch.from_numpy(g.standard_normal((c.pages, 16, G, W)) * 32)
    c.codes = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    c.codes[..., col] = 0
    for b, t in ((b, t) for b in range(B) for t in heavy):
        at = c.codes[c.table[b, t // 16], t % 16]
        kept = torch.from_numpy(at[:, voff: voff + dv].copy()).view(torch.float8_e4m3fn).double() * value
        at[:] = 0
        at[:, voff: voff + dv] = kept.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        at[:, col] = 0x7E                                          # 448
    c.scale[:] = 2.0 ** -5
    c.push()
    q = torch.from_numpy(g.standard_normal((B, Tq, G * hg, d)))
    sm = d ** -0.5
    q[..., col] = 0
    if margin:
        t = torch.arange(N, device="cuda")
        for b in range(B):
            k = _values(c, b, t)[..., :d].permute(1, 0, 2)
            for i in range(Tq):
                a = sm * q[b, i].cuda().bfloat16().double().view(G, hg, d) @ k.transpose(1, 2)
                a[:, :, list(heavy)] -= 1e9
                q[b, i, :, col] = ((a.amax(-1).reshape(-1) + margin) / (sm * 14)).cpu()
        q[:, :, 1::4, col] = 0                                     # every fourth head has no heavy token
    return c, q.bfloat16().cuda(), sm


@pytest.mark.parametrize("value", [0.0, 1e-3])
@pytest.mark.parametrize("margin", [0, 6, 8, 10])
@pytest.mark.parametrize("B,N,heavy", [(1, 512, (0,)), (24, 512, (0,)), (24, 2048, (0, 1, 70)), (24, 2048, (1030,)), (2, 16384, (0,)),
                                       (70, 900, (0, 500))])
@pytest.mark.parametrize("shape", SHAPES)
def test_heavy_token_of_little_value(shape, B, N, heavy, margin, value):
    c, q, sm = _case(N + margin, shape, B, N, heavy, margin, value)
    _hold(c, q, sm, shape, B, N, heavy, 0, -1)


@pytest.mark.parametrize("margin", [0, 6, 10])
@pytest.mark.parametrize("B,N,sinks,window,Tq", [(24, 3000, 4, 1000, 1), (8, 3000, 4, 1900, 4), (2, 700, 1, 300, 3)])
@pytest.mark.parametrize("shape", SHAPES)
def test_heavy_first_token_and_a_window(shape, B, N, sinks, window, Tq, margin):
    c, q, sm = _case(N + margin, shape, B, N, (0,), margin, 0.0, Tq)
    _hold(c, q, sm, shape, B, N, (0,), sinks, window)


def _hold(c, q, sm, shape, B, N, heavy, sinks, window):
    """One call within the bounds of bf16 weights, element by element and on the whole."""
    G, hg, d, dv, voff, W, _ = shape
    out, lse, st = K.attend(c, q, sm, K.i32([N] * B), sinks, window, None, None, d, dv, voff)
    torch.cuda.synchronize()
    r = _reference(c, q, sm, [N] * B, sinks, window, None, None, d, dv, voff)
    err = np.abs(out.double().cpu().numpy() - r["out"])
    # A bf16 weight is off by 2^-8 of itself and the fp16 value that is split by 2^-11; tokens of a
    # heavy one's tile by half a step of the format's smallest, 2^-14 of a unit, a unit being 2^-12 of
    # the largest weight (at most 1); scores and sums as in K.tolerances; the result is rounded once.
    dx = (d + 8) * K.U32 * r["mag"] + 2.0 ** -10 / 224 * r["top"]
    rel = np.expm1(2 * dx) + (N + 16) * K.U32 + 2.0 ** -21 + 2.0 ** -8 + 2.0 ** -11
    if window < 0:
        near = torch.cat([torch.arange(t, min(t + 128, N)) for t in sorted({t // 128 * 128 for t in heavy})])
    else:                                                          # its tile goes on with the window's first tokens
        lo = max(N - q.shape[1] - window - 15, 0)
        near = torch.cat([torch.arange(sinks), torch.arange(lo, lo + 144)])
    near = np.stack([_values(c, b, near.cuda())[..., voff: voff + dv].abs().sum(0).repeat_interleave(hg, 0).cpu().numpy()
                     for b in range(B)])[:, None]
    tol = rel[..., None] * r["mean"] + 2.0 ** -8 * np.abs(r["out"]) + 2.0 ** -26 * near
    assert np.all(err <= tol), float((err / tol).max())
    # Taken together the weights' errors do not add up: with a bf16 weight's rms (2^-7 / sqrt(12) of the
    # binade's foot at most) and the result's of the same size the root of their sum is below 2^-8.
    got = math.sqrt((err ** 2).sum() / (r["out"] ** 2).sum())
    assert got <= 2.0 ** -8, got
    heads = np.sqrt((err ** 2).sum((0, 1, 3)) / (r["out"] ** 2).sum((0, 1, 3)))
    assert heads.max() <= 2.0 ** -8, heads
    assert int(st.item()) == 0
