"""Attention of many query tokens at once (a prompt or a long draft), whole and windowed: column groups
whose queries stand at different places, against fp64."""
import pytest
import torch

from lookahead_sparse_kv_score_b200 import build
import lookahead_sparse_kv_score_b200 as lsa

import kv_cases as K
from test_gpu_kv_large import _check, _q, _vmax

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    build.build()
    lsa.lib()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window,sinks", [(-1, 0), (100, 0), (37, 5), (1, 0), (0, 3)])
@pytest.mark.parametrize("G,hg,d,dv,voff,W,Tq,N", [
    (2, 4, 128, 128, 128, 256, 300, 300), (1, 64, 576, 512, 0, 576, 65, 700), (3, 5, 64, 64, 64, 128, 129, 1000),
    (1, 1, 128, 128, 128, 256, 513, 900)])
def test_prompts(G, hg, d, dv, voff, W, Tq, N, window, sinks, dtype):
    """Lengths above, at and below the number of query tokens."""
    c = K.Cache(Tq, 3, N, G, W, 16, 16, "paged")
    _check(c, _q(N, 3, Tq, G * hg, d, dtype), d ** -0.5, [N, Tq, Tq // 3], sinks, window, None, None, d, dv, voff, _vmax(c))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_with_a_list(dtype):
    B, N, Tq, cap, G, hg, d = 2, 800, 96, 200, 2, 8, 128
    c = K.Cache(1, B, N, G, 256, 1, 1, "slots")
    idx = torch.randint(-1, 600, (B, cap), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
    _check(c, _q(2, B, Tq, G * hg, d, dtype), d ** -0.5, [N, 650], 4, 64, idx, [cap, 77], d, 128, 128, _vmax(c))
