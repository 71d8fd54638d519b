"""The 8-bit KV cache calls and the rotary positions refuse bad arguments on the host, before
anything is launched (fake, aligned device addresses; no GPU)."""
import ctypes
import math

import pytest
import torch

import lookahead_sparse_kv_score_b200 as lsa
from lookahead_sparse_kv_score_b200 import _abi, build

A = 256                                   # an aligned non-null address, never dereferenced
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _abi.load()


def _named(defaults, order, kw):
    unknown = set(kw) - set(defaults)
    assert not unknown, unknown
    return [{**defaults, **kw}[k] for k in order]


WRITE = dict(B=2, T=4, N=64, G=2, W=32, xdt=1, x=A, x_stride=64, start=A, count=A, block=4, page=4, seq_pages=16,
             pages=32, table=None, rows=A, scale=A, status=None, stream=None)
READ = dict(B=2, N=64, G=2, W=32, idx=A, cap=8, count=A, block=4, page=4, seq_pages=16, pages=32, table=None, rows=A,
            scale=A, odt=1, out=A, status=None, stream=None)
ATTEND = dict(B=2, Tq=1, N=64, H=4, G=2, d=32, dv=32, voff=0, W=32, qdt=1, q=A, sm=F(0.1), length=A, sinks=0,
              window=-1, idx=None, cap=0, count=None, block=4, page=4, seq_pages=16, pages=32, table=None, rows=A,
              scale=A, out=A, lse=None, status=None, ws=A, wsb=1 << 30, stream=None)
ROPE = dict(R=4, H=2, rot=8, half=0, dt=1, x=A, x_token=16, x_head=8, pos=A, freq=A, mscale=F(1.0), inverse=0, out=A,
            o_token=16, o_head=8, stream=None)
CACHE_BAD = [dict(W=24), dict(W=0), dict(G=0), dict(B=-1), dict(N=-1), dict(block=3), dict(block=256), dict(block=0),
             dict(page=6), dict(seq_pages=-1), dict(seq_pages=15), dict(pages=31), dict(rows=None), dict(scale=None),
             dict(rows=A + 8), dict(scale=A + 2), dict(table=A + 2)]


@pytest.mark.parametrize("kw", CACHE_BAD)
def test_cache_arguments(lib, kw):
    for fn, d in ((lib.lsa_kv_write, WRITE), (lib.lsa_kv_read, READ), (lib.lsa_kv_attend, ATTEND)):
        assert fn(*_named(d, d, kw)) == lsa.LSA_ERR_INVALID_ARG, kw
        assert lib.lsa_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(x=None), 1), (dict(start=None), 1), (dict(x=A + 8), 1), (dict(x_stride=60), 1),
    (dict(x_stride=56), 1), (dict(xdt=2), 2), (dict(seq_pages=0), 1), (dict(count=A + 1), 1),
    (dict(T=1 << 28, B=4, pages=64), 2), (dict(pages=1 << 30, table=A), 2), (dict(T=0), 0), (dict(B=0, rows=None), 0)])
def test_write_arguments(lib, kw, code):
    assert lib.lsa_kv_write(*_named(WRITE, WRITE, kw)) == code


@pytest.mark.parametrize("kw,code", [(dict(cap=-1), 1), (dict(odt=2), 2), (dict(out=None), 1), (dict(out=A + 8), 1),
                                     (dict(idx=None, cap=65), 1), (dict(cap=0), 0), (dict(N=0), 0)])
def test_read_arguments(lib, kw, code):
    assert lib.lsa_kv_read(*_named(READ, READ, kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(H=5), 1), (dict(d=33), 1), (dict(voff=16), 1), (dict(voff=-1), 1), (dict(d=0), 1), (dict(dv=0), 1),
    (dict(Tq=-1), 1), (dict(sinks=-1), 1), (dict(idx=A, cap=-1), 1), (dict(idx=A, cap=4, count=None), 1),
    (dict(q=None), 1), (dict(length=None), 1), (dict(out=None), 1), (dict(out=A + 8), 1), (dict(qdt=2), 2),
    (dict(d=577, W=592), 2), (dict(dv=513, W=528), 2), (dict(voff=1000, W=1040), 2), (dict(Tq=1 << 16), 2),
    (dict(Tq=1 << 24, H=2), 2), (dict(sm=F(math.inf)), 1), (dict(sm=F(math.nan)), 1), (dict(ws=None), 4),
    (dict(ws=A + 16), 4), (dict(N=4096, seq_pages=1024, pages=2048, wsb=0), 4), (dict(Tq=0), 0), (dict(B=0), 0)])
def test_attend_arguments(lib, kw, code):
    assert lib.lsa_kv_attend(*_named(ATTEND, ATTEND, kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rot=7), 1), (dict(rot=-2), 1), (dict(rot=1026), 1), (dict(R=-1), 1), (dict(dt=2), 2), (dict(x=None), 1),
    (dict(pos=None), 1), (dict(freq=None), 1), (dict(out=None), 1), (dict(x=A + 1), 1), (dict(freq=A + 4), 1),
    (dict(x_head=6), 1), (dict(o_token=4), 1), (dict(o_token=8), 1), (dict(o_token=8, o_head=24), 1),
    (dict(H=1 << 22), 2), (dict(R=0), 0), (dict(H=0), 0), (dict(rot=0), 0)])
def test_rope_arguments(lib, kw, code):
    assert lib.lsa_rope(*_named(ROPE, ROPE, kw)) == code


def test_rope_frequencies(lib):
    import numpy as np
    f = lsa.lsa_rope_frequencies(64).numpy()
    assert np.allclose(f, 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    s = lsa.lsa_rope_frequencies(64, factor=16.0, original=65536).numpy()
    turns = 65536 * f / (2 * math.pi)
    assert np.array_equal(s[turns > 33], f[turns > 33]) and (turns > 33).any()
    slow = turns < 0.7
    assert np.allclose(s[slow], f[slow] / 16) and np.all((s <= f) & (s >= f / 16 * (1 - 1e-15)))
    assert lsa.lsa_rope_frequencies(0).numel() == 0
    for bad in (dict(rot=3), dict(rot=8, base=1.0), dict(rot=8, factor=0.5), dict(rot=8, factor=2.0),
                dict(rot=8, factor=2.0, original=100.0, fast=1.0, slow=1.0), dict(rot=8, factor=math.nan)):
        with pytest.raises(lsa.LsaError):
            lsa.lsa_rope_frequencies(**bad)


def test_binding_refuses_host_tensors_types_and_short_arrays(lib):
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    rows, scale = torch.zeros(32, 4, 2, 32, dtype=torch.uint8), torch.zeros(2, 16, 2)
    with pytest.raises(ValueError, match="one CUDA device"):
        lsa.lsa_kv_write(2, 4, 64, 2, 32, 1, x, 64, i, None, 4, 4, 16, 32, None, rows, scale, stream=0)
    with pytest.raises(ValueError, match="xdt"):
        lsa.lsa_kv_write(2, 4, 64, 2, 32, 0, x, 64, i, None, 4, 4, 16, 32, None, rows, scale, stream=0)
    with pytest.raises(ValueError, match="expected"):
        lsa._dev(torch.zeros(4, dtype=torch.int64), "idx", (torch.int32,), 4, 0)
    with pytest.raises(ValueError, match="one CUDA device"):
        lsa.lsa_rope(2, 1, 8, 0, 1, x, 64, 8, i, torch.zeros(4, dtype=torch.float64), 1.0, 0, x, 64, 8, stream=0)


def test_binding_refuses_views_it_cannot_walk():
    """Strided sources are walked with the call's strides: the last dimension must be dense and the
    span must lie in the storage (checked on the host's own tensors; nothing is launched)."""
    x = torch.zeros(4, 6, 64)
    d = x.get_device()
    ok = lambda t, span: lsa._bad(t, "x", lsa._QTYPES, span, d)  # noqa: E731
    assert "one CUDA device" in ok(x, 0)
    class Fake(torch.Tensor):
        def get_device(self):
            return 0
    f = x.as_subclass(Fake)
    assert lsa._dev_strided(f, "x", lsa._QTYPES, x.numel(), 0) == x.data_ptr()
    assert lsa._dev_strided(f[:, :, 32:], "x", lsa._QTYPES, x.numel() - 32, 0) == x.data_ptr() + 128
    for t, span in ((f, x.numel() + 1), (f[1:], x.numel()), (f, -1), (f.transpose(1, 2), 8)):
        with pytest.raises(ValueError):
            lsa._dev_strided(t, "x", lsa._QTYPES, span, 0)
