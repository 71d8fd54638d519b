"""Pins of the oracle's 8-bit KV cache and rotary positions: closed forms, brute force and
hand-made cases, on the CPU."""
import math

import numpy as np
import pytest
import torch

from oracle import kv as OK
from oracle import lsa_oracle as O


def test_e4m3_rounding_matches_torch_on_every_midpoint():
    v = np.sort(np.unique(O.decode_e4m3(np.array([c for c in range(128) if c != 127], dtype=np.uint8))))
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), [448.0, 460.0, 1e-9]])
    x = np.concatenate([x, -x])
    want = torch.from_numpy(x.clip(-448, 448)).float().to(torch.float8_e4m3fn).double().numpy()
    x32 = torch.from_numpy(x.clip(-448, 448)).float().double().numpy()
    assert np.array_equal(OK.e4m3_round(x32), want)
    assert np.array_equal(O.decode_e4m3(OK.e4m3_code(v)), v)


@pytest.mark.parametrize("amax,s", [(448.0, 1.0), (448.1, 2.0), (0.0, 2.0 ** -24), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                    (1.76, 2.0 ** -7), (math.inf, math.nan), (math.nan, math.nan)])
def test_block_scale(amax, s):
    got = OK.block_scale(amax)
    assert got == s or (math.isnan(got) and math.isnan(s))


def _empty(B, N, G, W, block, page=1):
    return OK.Cache(np.zeros((B * (-(-N // page)), page, G, W), np.uint8), np.ones((B, -(-N // block), G)), None, N, block,
                    page, -(-N // page))


def test_write_read_round_trip_and_growing_block():
    c = _empty(1, 8, 1, 16, 4)
    x = np.zeros((1, 2, 1, 16))
    x[0, 0, 0, :3] = [1.0, -3.0, 0.5]
    assert not OK.write(c, x, [0], [2])
    assert c.scale[0, 0, 0] == 2.0 ** -7 and np.array_equal(c.values(0, 0)[0, :3], [1.0, -3.0, 0.5])
    big = np.full((1, 1, 1, 16), 1000.0)                  # raises the block's scale to 4
    OK.write(c, big, [2], [1])
    assert c.scale[0, 0, 0] == 4.0
    assert np.array_equal(c.values(0, 0)[0, :3], [1.0, -3.0, 0.5])      # exact: powers of two
    assert c.values(0, 2)[0, 0] == OK.e4m3_round(250.0) * 4.0
    OK.write(c, np.full((1, 1, 1, 16), 0.01), [3], [1])   # a smaller token does not lower it
    assert c.scale[0, 0, 0] == 4.0
    out = np.full((1, 3, 1, 16), 7.0)
    assert OK.read(c, np.array([[2, -1, 9]]), [3], out)   # 9 is out of range
    assert out[0, 0, 0, 0] == c.values(0, 2)[0, 0] and (out[0, 1:] == 7.0).all()


def test_write_marks_non_finite_blocks():
    c = _empty(1, 4, 1, 16, 2)
    x = np.ones((1, 3, 1, 16))
    x[0, 1, 0, 5] = math.inf
    OK.write(c, x, [0], [3])
    assert math.isnan(c.scale[0, 0, 0]) and not c.rows[:2].any() and c.scale[0, 1, 0] == 2.0 ** -8


def test_attend_against_closed_forms():
    c = _empty(1, 6, 1, 16, 1)
    x = np.zeros((1, 6, 1, 16))
    x[0, :, 0, 1] = np.arange(6)
    OK.write(c, x, [0], [6])
    q = np.zeros((1, 2, 1, 4))                            # zero query: the mean of the visible values
    r = OK.attend(c, q, 1.0, [6], 1, 2, None, None, 4, 16, 0)
    assert r["out"][0, 0, 0, 1] == pytest.approx((0 + 3 + 4) / 3) and r["out"][0, 1, 0, 1] == pytest.approx((0 + 4 + 5) / 3)
    assert r["lse"][0, 0, 0] == pytest.approx(math.log(3))
    r = OK.attend(c, q, 1.0, [6], 1, 2, np.array([[0, 1, 1, -1, 5, 99]]), [6], 4, 16, 0)
    assert r["wide"][0, 0, 0] == 6 and r["wide"][0, 1, 0] == 5   # {0,3,4} + 1, 1, 5; {0,4,5} + 1, 1
    assert r["out"][0, 1, 0, 1] == pytest.approx((0 + 4 + 5 + 1 + 1) / 5)
    q[0, :, 0, 1] = 100.0                                 # a steep query picks the largest key
    r = OK.attend(c, q, 1.0, [6], 0, -1, None, None, 4, 16, 0)
    assert r["out"][0, 0, 0, 1] == pytest.approx(4.0) and r["out"][0, 1, 0, 1] == pytest.approx(5.0)
    r = OK.attend(c, q, 1.0, [1], 0, -1, None, None, 4, 16, 0)
    assert np.isinf(r["lse"][0, 0, 0]) and not r["out"][0, 0].any()


def test_rope_is_a_rotation_and_its_inverse_the_gradient():
    g = np.random.default_rng(0)
    x, dy = g.standard_normal((3, 2, 8)), g.standard_normal((3, 2, 8))
    pos, f = np.array([0, 5, 1000003]), 10000.0 ** (-np.arange(4) / 4)
    for half in (0, 1):
        y = OK.rope(x, pos, f, half, 1.5, 0)
        assert np.allclose(np.linalg.norm(y, axis=2), 1.5 * np.linalg.norm(x, axis=2))
        assert np.allclose(y[0], 1.5 * x[0])
        back = OK.rope(dy, pos, f, half, 1.5, 1)
        assert np.isclose((back * x).sum(), (dy * y).sum())             # the adjoint
        e = 1e-6                                                        # against differences
        i = (1, 1, 3)
        xp, xm = x.copy(), x.copy()
        xp[i] += e
        xm[i] -= e
        d = ((OK.rope(xp, pos, f, half, 1.5, 0) - OK.rope(xm, pos, f, half, 1.5, 0)) * dy).sum() / (2 * e)
        assert d == pytest.approx(back[i], abs=1e-8)
