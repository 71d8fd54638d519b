"""Attention over caches whose stored scales are zero, negative or far apart: a value is its code times its
scale, so a token of scale 0 has score 0 and value 0 and still counts among the weights."""
import math

import numpy as np
import pytest
import torch

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import build

import kv_cases as K

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

SHAPES = [  # G, hg, d, dv, voff, W
    (1, 20, 576, 512, 0, 576), (2, 8, 128, 128, 128, 256), (1, 33, 256, 256, 256, 512), (3, 3, 64, 64, 64, 128)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    lsa.lib()


def _q(seed, B, Tq, H, d, dtype):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((B, Tq, H, d))).to(dtype).cuda()


def _spoil(c, kind, seed):
    """Scales of the given kind; sequence 1 has zeros alone where zeros are meant."""
    g = np.random.default_rng(seed)
    if kind in ("zero", "both"):
        c.scale[g.random(c.scale.shape) < 0.4] = 0.0
        c.scale[1] = 0.0
        c.scale[2, :2] = -0.0
    if kind in ("negative", "both"):
        c.scale *= np.where(g.random(c.scale.shape) < 0.5, -1, 1).astype(np.float32)
    if kind == "small":
        c.scale[:] = 2.0 ** -50 * np.exp2(g.integers(0, 3, size=c.scale.shape))
    c.push()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["zero", "negative", "both", "small"])
@pytest.mark.parametrize("store,page,block", [("dense", 1, 16), ("slots", 1, 1), ("paged", 64, 64)])
@pytest.mark.parametrize("G,hg,d,dv,voff,W", SHAPES)
def test_scales(G, hg, d, dv, voff, W, store, page, block, kind, dtype):
    B, N = 4, 420
    c = K.Cache(W + block, B, N, G, W, block, page, store)
    _spoil(c, kind, page + d)
    q = _q(hg, B, 1, G * hg, d, dtype)
    out, lse = K.check_attend(c, q, d ** -0.5, [N, 300, 131, 1], 0, -1, None, None, d, dv, voff)
    if kind in ("zero", "both"):
        assert not out[1].any() and np.allclose(lse[1].cpu().numpy(), math.log(300), rtol=0, atol=1e-5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["zero", "both"])
@pytest.mark.parametrize("G,hg,d,dv,voff,W", SHAPES[:2])
def test_scales_with_windows_lists_and_drafts(G, hg, d, dv, voff, W, kind, dtype):
    B, N, cap = 3, 500, 150
    c = K.Cache(3, B, N, G, W, 1, 16, "paged")
    _spoil(c, kind, 5)
    idx = np.random.default_rng(1).integers(-1, 300, size=(B, cap)).astype(np.int32)
    q = _q(hg, B, 4, G * min(hg, 8), d, dtype)
    K.check_attend(c, q, d ** -0.5, [N, 333, 301], 3, 40, idx, [cap, 20, 140], d, dv, voff)
    q1 = _q(hg, B, 1, G * hg, d, dtype)
    K.check_attend(c, q1, d ** -0.5, [N, 333, 301], 0, 0, idx, [cap, 20, 140], d, dv, voff)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G,hg,d,dv,voff,W", SHAPES[:2])
def test_zero_tokens_that_weigh_most(G, hg, d, dv, voff, W, dtype):
    """Every other score is far below 0, then far above."""
    B, N = 2, 700
    c = K.Cache(8, B, N, G, W, 1, 1, "dense")
    c.codes[..., 0] = 0x38                                         # 1.0
    c.scale[:] = 2.0 ** -5
    c.scale[:, ::9] = 0.0
    c.push()
    q = _q(3, B, 1, G * hg, d, dtype)
    q[0, ..., 0] = -800.0
    q[1, ..., 0] = 800.0
    K.check_attend(c, q, 0.3, [N, N - 5], 0, -1, None, None, d, dv, voff)


def test_bf16_takes_the_smallest_scales_for_zero():
    """Scales below 2^-60 in magnitude, subnormal ones among them, count as 0 with bf16 queries."""
    G, hg, d, dv, voff, W = SHAPES[1]
    outs = []
    for tiny in (0.0, 2.0 ** -61, -1e-38, 1e-45):
        c = K.Cache(8, 2, 300, G, W, 4, 16, "paged")
        c.scale[:, ::3] = tiny
        c.push()
        q = _q(3, 2, 1, G * hg, d, BF)
        out, lse, st = K.attend(c, q, 0.1, K.i32([300, 200]), 0, -1, None, None, d, dv, voff)
        torch.cuda.synchronize()
        assert torch.isfinite(out).all() and torch.isfinite(lse).all() and int(st.item()) == 0
        outs.append((out, lse))
    for o, l in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])
