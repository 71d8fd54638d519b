"""Attention over the 8-bit KV cache where rows have chunks that only the values use, and tiles of
scattered rows stand beside tiles whose rows follow one another: many tiles a block, against fp64."""
import numpy as np
import pytest
import torch

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import build

import kv_cases as K
from test_gpu_kv_large import _check, _q, _vmax

pytestmark = pytest.mark.gpu

SHAPES = [  # G, hg, d, dv, voff, W: one or two chunks of keys, and behind them two of values alone
    (2, 16, 128, 256, 128, 384), (1, 33, 128, 256, 64, 320), (2, 8, 256, 256, 256, 512), (1, 20, 192, 384, 256, 640)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    lsa.lib()


@pytest.mark.parametrize("store,page", [("paged", 64), ("slots", 16), ("dense", 1)])
@pytest.mark.parametrize("G,hg,d,dv,voff,W", SHAPES)
def test_value_chunks_over_many_tiles(G, hg, d, dv, voff, W, store, page):
    B, N = 80, 1700
    c = K.Cache(W + page, B, N, G, W, 16, page, store)
    length = [N - (b * 13) % (N // 2) for b in range(B)]
    _check(c, _q(d, B, 1, G * hg, d), d ** -0.5, length, 0, -1, None, None, d, dv, voff, _vmax(c))


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("G,hg,d,dv,voff,W", SHAPES)
def test_scattered_tiles_before_runs(G, hg, d, dv, voff, W, page):
    """Lists whose tiles are random rows, runs of rows, or both, in changing order: a stage takes a
    tile of copies after one of boxes and a tile of boxes after one of copies."""
    B, N, cap = 80, 6000, 1664
    c = K.Cache(dv + page, B, N, G, W, 16, page, "paged")
    g = np.random.default_rng(page)
    idx = np.empty((B, cap // 128, 128), dtype=np.int32)
    for b in range(B):
        for t in range(cap // 128):
            kind = (t >> (b % 3)) % 2 if b % 4 else int(g.integers(0, 2))
            first = int(g.integers(0, (N - 128) // 64)) * 64
            idx[b, t] = first + np.arange(128) if kind else g.integers(0, N, size=128)
            if b % 5 == 4:                                     # half a tile of each
                idx[b, t, 64:] = g.integers(0, N, size=64)
    idx = torch.from_numpy(idx.reshape(B, cap)).cuda()
    _check(c, _q(W, B, 1, G * hg, d), d ** -0.5, [N] * B, 0, 0, idx, [cap - 5 * b for b in range(B)], d, dv, voff, _vmax(c))
