"""What the binding passes on: views whose own strides are not the ones that the call walks are refused,
and numbers past 32 bits are not cut (host tensors that pass for device ones; nothing is launched)."""
import sys

import pytest
import torch

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import build


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    lsa.lib()


class Fake(torch.Tensor):
    def get_device(self):
        return 0


def _view(*shape):
    return torch.arange(float(torch.Size(shape).numel())).view(shape).as_subclass(Fake)


def _ok(t, counts, strides):
    span = 1 + sum((n - 1) * s for n, s in zip(counts, strides))
    return lsa._dev_strided(t, "x", lsa._QTYPES, span, 0, counts, strides) == t.data_ptr()


def test_time_slices():
    buf = _view(3, 7, 32)
    for T in (1, 4):
        with pytest.raises(ValueError, match="walks"):
            _ok(buf[:, :T], (3 * T, 32), (32, 1))                  # sequence 1 lies 7 tokens on, not T
    assert _ok(buf, (21, 32), (32, 1)) and _ok(buf[:1, :4], (4, 32), (32, 1)) and _ok(buf[1:, :], (14, 32), (32, 1))
    assert _ok(buf[:, :, 8:24], (21, 16), (32, 1))                 # a slice of the columns of every token
    assert _ok(buf[:, :, 8:24].unflatten(2, (2, 8)), (21, 16), (32, 1))
    assert _ok(buf[:, :1, 8:24], (3, 16), (224, 1)) and _ok(buf[0, :, 8:24], (5, 16), (32, 1))
    with pytest.raises(ValueError, match="walks"):
        _ok(buf[:, :, 8:24], (21, 16), (16, 1))
    with pytest.raises(ValueError, match="walks"):
        _ok(buf[:2, :3, 8:24], (6, 16), (32, 1))
    with pytest.raises(ValueError, match="walks"):
        _ok(buf[:, :, 8:24], (5, 32), (32, 1))                     # wider than the view's rows


def test_heads():
    x = _view(5, 3, 96)
    part = x[:, :, 64:]
    assert _ok(part, (5, 3, 32), (288, 96, 1)) and _ok(part[:, :1], (5, 1, 32), (288, 32, 1))
    assert _ok(part[:1], (1, 3, 32), (32, 96, 1)) and _ok(part, (15, 1, 32), (96, 32, 1))
    for strides in ((96, 288, 1), (288, 32, 1), (192, 96, 1)):
        with pytest.raises(ValueError, match="walks"):
            _ok(part, (5, 3, 32), strides)
    heads_first = x.permute(1, 0, 2)                               # a view [3][5][96] of tokens first
    with pytest.raises(ValueError, match="walks"):
        _ok(heads_first, (5, 3, 96), (288, 96, 1))
    assert _ok(heads_first, (3, 5, 96), (96, 288, 1))


def test_calls_pass_their_walks(monkeypatch):
    seen = []
    monkeypatch.setattr(lsa, "_call", lambda fn, where, device, stream, *args: seen.append(where))
    i, rows, scale = (torch.zeros(n, dtype=d).as_subclass(Fake) for n, d in
                      ((64, torch.int32), (32 * 4 * 64, torch.uint8), (64, torch.float32)))
    buf = _view(2, 9, 64)
    with pytest.raises(ValueError, match="walks"):
        lsa.lsa_kv_write(2, 4, 64, 2, 32, 0, buf[:, :4], 64, i, None, 4, 4, 16, 32, None, rows, scale)
    lsa.lsa_kv_write(2, 9, 64, 2, 32, 0, buf, 64, i, None, 4, 4, 16, 32, None, rows, scale)
    freq = torch.zeros(8, dtype=torch.float64).as_subclass(Fake)
    part, out = _view(4, 2, 32)[:, :, 16:], _view(4, 2, 16)
    lsa.lsa_rope(4, 2, 16, 0, 0, part, 64, 32, i, freq, 1.0, 0, out, 32, 16)
    for x_s, o in (((32, 64), out), ((64, 32), part.permute(1, 0, 2))):
        with pytest.raises(ValueError, match="walks"):
            lsa.lsa_rope(4, 2, 16, 0, 0, part, *x_s, i, freq, 1.0, 0, o, *((32, 16) if o is out else (64, 32)))
    assert seen == ["lsa_kv_write", "lsa_rope"]


@pytest.mark.parametrize("given,passed", [(2 ** 32, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (sys.maxsize, 2 ** 31 - 1),
                                          (2 ** 31 - 1, 2 ** 31 - 1), (7, 7), (0, 0), (-1, -1), (-2 ** 40, -2 ** 31)])
def test_windows_past_32_bits(monkeypatch, given, passed):
    seen = []
    monkeypatch.setattr(lsa, "_call", lambda fn, where, device, stream, *args: seen.append(args))
    size = (1, 1, 64, 2, 1, 32, 32, 0, 32)
    q, out, i = _view(1, 1, 2, 32), _view(1, 1, 2, 32), torch.zeros(64, dtype=torch.int32).as_subclass(Fake)
    rows, scale = torch.zeros(2048, dtype=torch.uint8).as_subclass(Fake), torch.zeros(64).as_subclass(Fake)
    lsa.lsa_kv_attend(*size, 0, q, 1.0, i, max(given, 0), given, None, 0, None, 1, 1, 64, 64, None, rows, scale, out, None, rows)
    at = len(size) + 4
    assert seen[0][at: at + 2] == (max(passed, 0), passed)
    assert lsa.lsa_kv_attend_workspace_bytes(*size, 0, max(given, 0), given, 0) == \
        lsa.lsa_kv_attend_workspace_bytes(*size, 0, max(passed, 0), passed, 0)
