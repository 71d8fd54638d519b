"""Writes into blocks of which some tokens are not resident (their codes lie in the cold pool): a scale
that those codes depend on does not change."""
import numpy as np
import pytest
import torch

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import build
from oracle import kv as OK

import kv_cases as K
from test_gpu_kv import _same_cache, _write, _x

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    lsa.lib()


# block, page, G, W: one warp a block of tokens and eight of them; rows of one vector a lane and of more
SIZES = [(4, 1, 2, 32), (8, 2, 1, 576), (16, 4, 3, 144), (64, 16, 2, 256), (128, 4, 1, 576)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,page,G,W", SIZES)
def test_growing_blocks(block, page, G, W, dtype):
    """Appends that grow the scale, that do not, and that are not finite, to blocks whose earlier tokens are
    all there, partly away (among them the one just before) and all away."""
    B, N = 5, 3 * block
    c = K.Cache(W + block, B, N, G, W, block, page, "slots")
    at = block + block // 2                                        # the second block's middle, a page's start
    first = block // page
    c.table[1, first] = -1
    c.table[2, at // page - 1] = -1
    c.table[3, first: at // page] = -1
    c.table[4, 0] = -1                                             # another block's
    c.push()
    want = c.oracle()
    T = max(block // 4, 1)
    for k, mag in enumerate((1e-4, 1.0, 1e5, 1e-2)):
        x = _x(40 + k, (B, T, G, W), dtype) * mag
        if k == 3:
            x[:, 0, G - 1, 5] = float("inf")                       # one head alone
        skipped = OK.write(want, x.double().cpu().numpy(), [at] * B, [T] * B)
        st = _write(c, x, [at] * B, None)
        _same_cache(c, want)
        assert int(st.item()) == (lsa.LSA_ERR_RANGE if skipped else 0), k


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block,page,G,W", SIZES + [(4, 16, 2, 32), (64, 64, 2, 256)])
def test_new_tokens_away(block, page, G, W, dtype):
    """New tokens that are not resident are far larger than the others: they have no part in the scales."""
    B, N, T = 4, 4 * max(block, page), 3 * max(block, page)
    c = K.Cache(W + block, B, N, G, W, block, page, "slots")
    g = np.random.default_rng(block)
    c.table[1, g.random(c.table.shape[1]) < 0.3] = -1
    c.table[2, ::2] = 10 ** 6
    c.table[3] = -1
    c.push()
    want = c.oracle()
    start = [0, 3, max(block, page), 1]
    x = _x(7, (B, T, G, W), dtype)
    for b in range(B):
        for i in range(T):
            if want.place(b, start[b] + i) is None:
                x[b, i] *= 1e6
    assert OK.write(want, x.double().cpu().numpy(), start, [T] * B)
    scale = c.scale_d.clone()
    st = _write(c, x, start, None)
    _same_cache(c, want)
    assert int(st.item()) == lsa.LSA_ERR_RANGE and torch.equal(c.scale_d[3], scale[3])


def test_a_cold_block_keeps_its_values():
    """Codes fetched back after a refused append decode to what was written."""
    B, N, G, W, block, page = 1, 32, 1, 64, 16, 4
    c = K.Cache(1, B, N, G, W, block, page, "slots")
    x = _x(1, (B, 8, G, W), BF)
    _write(c, x, [0], None)
    out = torch.zeros(B, 8, G, W, device="cuda")
    read = lambda: lsa.lsa_kv_read(B, N, G, W, None, 8, None, *c.args(), lsa.LSA_F32, out)  # noqa: E731
    read()
    torch.cuda.synchronize()
    was, table = out.clone(), c.table_d.clone()
    c.table_d[0, 0] = -1                                           # tokens 0 to 3 leave
    st = _write(c, x[:, :4] * 1e4, [8], None)
    torch.cuda.synchronize()
    assert int(st.item()) == lsa.LSA_ERR_RANGE
    c.table_d.copy_(table)                                         # and come back
    read()
    torch.cuda.synchronize()
    assert torch.equal(out, was)
