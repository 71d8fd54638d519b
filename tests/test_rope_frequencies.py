"""The scaled rotary frequencies against values worked out by hand from the rule: the blend runs
from the pair that turns `fast` times within the original length (rounded down) to the one that
turns `slow` times (rounded up), wherever that lies."""
import math

import numpy as np
import pytest

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lsa.lib()


# Pair i of rot columns turns n = original / (2 pi) * 10000^(-2 i / rot) times, so n turns are at
# i = rot * ln(original / (2 pi n)) / (2 ln 10000).  `first`, `last`: ends by that, rounded outwards.
@pytest.mark.parametrize("rot,factor,original,first,last", [
    (64, 16.0, 65536, 20, 33),        # 20.11 and 32.15: the end lies past the last pair, 31
    (128, 8.0, 131072, 45, 70),       # 45.03 and 69.11
    (64, 16.0, 4096, 10, 23),         # 10.47 and 22.51
    (128, 40.0, 8192, 25, 50),        # 25.76 and 49.85
    (64, 4.0, 500, 3, 16)])           # 3.17 and 15.21
def test_blend_ends(rot, factor, original, first, last):
    f = lsa.lsa_rope_frequencies(rot).numpy()
    s = lsa.lsa_rope_frequencies(rot, factor=factor, original=original).numpy()
    i = np.arange(rot // 2)
    turns = original / (2 * math.pi) * 10000.0 ** (-2.0 * i / rot)
    assert (turns[i <= first] >= 32).all() and first < last
    if last < rot // 2:
        assert (turns[i >= last] <= 1).all() and (turns[i >= last] < 1).any()
    want = np.array([1.0 if k <= first else 1 / factor if k >= last else
                     1 - (1 - 1 / factor) * (k - first) / (last - first) for k in range(rot // 2)])
    assert np.allclose(s / f, want, rtol=1e-12)
    assert ((turns > 1) & (want > 1 / factor) == (turns > 1)).all()      # only pairs that turn less than once lose it all


def test_pairs_by_hand():
    share = (lsa.lsa_rope_frequencies(64, factor=16.0, original=65536) / lsa.lsa_rope_frequencies(64)).numpy()
    # 1 - 15/16 * (i - 20) / 13
    for i, want in ((20, 1.0), (24, 0.7115384615384616), (28, 0.4230769230769231), (30, 0.27884615384615385),
                    (31, 0.20673076923076927)):
        assert share[i] == pytest.approx(want, rel=1e-12), i
    last = (lsa.lsa_rope_frequencies(128, factor=8.0, original=131072) / lsa.lsa_rope_frequencies(128)).numpy()[63]
    assert last == pytest.approx(1 - 7 / 8 * 18 / 25, rel=1e-12)         # it turns 2.4 times


def test_ends_are_cut_to_the_columns():
    """Ends before the first pair and past `rot - 1` are moved there."""
    f = lsa.lsa_rope_frequencies(16).numpy()
    s = lsa.lsa_rope_frequencies(16, factor=4.0, original=1e6, fast=1e12, slow=1e-6).numpy()    # -13.6 and 22.4 -> 0 and 15
    assert np.allclose(s / f, 1 - 3 / 4 * np.arange(8) / 15, rtol=1e-12)
