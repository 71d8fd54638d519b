"""Python binding of liblsa, the B200 (sm_100a) library for the Lookahead Sparse
Attention indexer step: scoring, OR-union, compaction, cold->hot gather, top-k in the
fetched set and cross-layer vote labels.

The functions keep the C names and only marshal arguments: tensors become raw
pointers, dtypes become lsa_dtype codes, and the current torch CUDA stream is passed
unless one is given.  Every computation runs in liblsa's kernels; a nonzero status
raises LsaError.  Shapes and layouts are documented in include/lsa.h.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi

LSA_OK, LSA_ERR_INVALID_ARG, LSA_ERR_UNSUPPORTED, LSA_ERR_CAPACITY = 0, 1, 2, 3
LSA_ERR_NOMEM, LSA_ERR_CUDA, LSA_ERR_TIMEOUT, LSA_ERR_RANGE = 4, 5, 6, 7
LSA_F32, LSA_BF16, LSA_E4M3 = 0, 1, 2


class LsaError(RuntimeError):
    def __init__(self, code: int, where: str, detail: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({detail})")


def lib():
    return _abi.load()


def status_string(code: int) -> str:
    return lib().lsa_status_string(code).decode()


def dtype_code(t) -> int:
    dt = t.dtype if isinstance(t, torch.Tensor) else t
    if dt == torch.float32:
        return LSA_F32
    if dt == torch.bfloat16:
        return LSA_BF16
    if dt in (torch.uint8, torch.float8_e4m3fn):
        return LSA_E4M3
    raise TypeError(f"no lsa_dtype for {dt}")


def _p(t):
    """Raw pointer of a tensor (None -> NULL); plain ints pass through.  The library reads
    and writes every array densely in the layout the header gives, so a strided view is
    refused here rather than read as if it were dense."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError(f"tensor of shape {tuple(t.shape)} with strides {t.stride()} is not contiguous")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != LSA_OK:
        raise LsaError(rc, where, lib().lsa_last_error().decode())


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A 256-byte aligned device workspace (torch allocations are 512-byte aligned)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def kernel_launches() -> int:
    """Kernels liblsa has launched in this process so far."""
    return int(lib().lsa_kernel_launches())


# ----------------------------------------------------------------------------- scoring

def lsa_index_project_workspace_bytes(B, L, D, r, H, dI, wdt) -> int:
    return int(lib().lsa_index_project_workspace_bytes(B, L, D, r, H, dI, wdt))


def lsa_index_project(B, L, D, r, H, dI, wdt, h, W_down, W_up, W_w, layer, q_out, w_out,
                      workspace, stream=None):
    _check(lib().lsa_index_project(B, L, D, r, H, dI, wdt, _p(h), _p(W_down), _p(W_up), _p(W_w),
                                   layer, _p(q_out), _p(w_out), _p(workspace),
                                   0 if workspace is None else workspace.numel(), _stream(stream)),
           "lsa_index_project")


def lsa_index_score_workspace_bytes(B, L, N, D, r, H, dI, wdt, kdt) -> int:
    return int(lib().lsa_index_score_workspace_bytes(B, L, N, D, r, H, dI, wdt, kdt))


def lsa_index_score(B, L, N, D, r, H, dI, wdt, h, W_down, W_up, W_w, bias, kdt, K, kscale,
                    layer, q_in, w_in, q_out, w_out, mask, logit, score, workspace, status=None,
                    stream=None):
    rc = lib().lsa_index_score(B, L, N, D, r, H, dI, wdt, _p(h), _p(W_down), _p(W_up), _p(W_w),
                               _p(bias), kdt, _p(K), _p(kscale), layer, _p(q_in), _p(w_in),
                               _p(q_out), _p(w_out), _p(mask), _p(logit), _p(score), _p(status),
                               _p(workspace), 0 if workspace is None else workspace.numel(),
                               _stream(stream))
    _check(rc, "lsa_index_score")


# ----------------------------------------------------------------------------- selection

def lsa_select_union(B, Nw, mask_l, U, new_l, stream=None):
    _check(lib().lsa_select_union(B, Nw, _p(mask_l), _p(U), _p(new_l), _stream(stream)),
           "lsa_select_union")


def lsa_compact(B, N, bits, cap, idx, count, status=None, stream=None):
    _check(lib().lsa_compact(B, N, _p(bits), cap, _p(idx), _p(count), _p(status), _stream(stream)),
           "lsa_compact")


def lsa_select_fetch_workspace_bytes(B, N) -> int:
    return int(lib().lsa_select_fetch_workspace_bytes(B, N))


def lsa_select_fetch(B, L, N, mask, U, new_l, cap, idx_new, cnt_new, idx_U, cnt_U, workspace, logit=None,
                     key_U=None, status=None, stream=None):
    _check(lib().lsa_select_fetch(B, L, N, _p(mask), _p(U), _p(new_l), cap, _p(idx_new), _p(cnt_new), _p(idx_U),
                                  _p(cnt_U), _p(logit), _p(key_U), _p(status), _p(workspace),
                                  0 if workspace is None else workspace.numel(), _stream(stream)), "lsa_select_fetch")


def lsa_topk_keyed(B, k, idx, cap, count, key, topk, topk_count, stream=None):
    _check(lib().lsa_topk_keyed(B, k, _p(idx), cap, _p(count), _p(key), _p(topk), _p(topk_count), _stream(stream)),
           "lsa_topk_keyed")


def lsa_topk_workspace_bytes(B, cap) -> int:
    return int(lib().lsa_topk_workspace_bytes(B, cap))


def lsa_topk(B, L, N, k, idx, cap, count, logit, topk, topk_count, workspace, stream=None):
    _check(lib().lsa_topk(B, L, N, k, _p(idx), cap, _p(count), _p(logit), _p(topk), _p(topk_count),
                          _p(workspace), 0 if workspace is None else workspace.numel(),
                          _stream(stream)), "lsa_topk")


def lsa_fine_score_workspace_bytes(B, H, dI, kdt) -> int:
    return int(lib().lsa_fine_score_workspace_bytes(B, H, dI, kdt))


def lsa_fine_score(B, N, H, dI, qdt, q, w, kdt, K, kscale, idx, cap, count, score, workspace, status=None,
                   stream=None):
    _check(lib().lsa_fine_score(B, N, H, dI, qdt, _p(q), _p(w), kdt, _p(K), _p(kscale), _p(idx), cap, _p(count),
                                _p(score), _p(status), _p(workspace), 0 if workspace is None else workspace.numel(),
                                _stream(stream)), "lsa_fine_score")


def lsa_topk_noalloc(B, L, N, k, idx, cap, count, logit, topk, topk_count, stream=None):
    """lsa_topk with its scratch in the library's built-in device array (no workspace)."""
    _check(lib().lsa_topk_noalloc(B, L, N, k, _p(idx), cap, _p(count), _p(logit), _p(topk), _p(topk_count),
                                  _stream(stream)), "lsa_topk_noalloc")


def lsa_gather_cold(B, N, row_bytes, cold_host, idx, count, cap, hot, status=None, stream=None):
    _check(lib().lsa_gather_cold(B, N, row_bytes, _p(cold_host), _p(idx), _p(count), cap, _p(hot),
                                 _p(status), _stream(stream)), "lsa_gather_cold")


# ----------------------------------------------------------------------------- hot pool

def lsa_hot_pool_state_bytes(B, N, slots) -> int:
    return int(lib().lsa_hot_pool_state_bytes(B, N, slots))


def lsa_hot_pool_workspace_bytes(B, N, slots) -> int:
    return int(lib().lsa_hot_pool_workspace_bytes(B, N, slots))


def lsa_hot_pool_layout(B, N, slots):
    """Byte offsets of (slot_of, entry_of, stamp, resident) inside the state."""
    off = (ctypes.c_size_t * 4)()
    _check(lib().lsa_hot_pool_layout(B, N, slots, off), "lsa_hot_pool_layout")
    return tuple(int(x) for x in off)


def lsa_hot_pool_reset(B, N, slots, state, stream=None):
    _check(lib().lsa_hot_pool_reset(B, N, slots, _p(state), _stream(stream)), "lsa_hot_pool_reset")


def lsa_hot_pool_update(B, N, slots, row_bytes, trigger, U, cold_host, hot, state, moved, status,
                        workspace, stream=None):
    _check(lib().lsa_hot_pool_update(B, N, slots, row_bytes, trigger, _p(U), _p(cold_host), _p(hot), _p(state),
                                     _p(moved), _p(status), _p(workspace),
                                     0 if workspace is None else workspace.numel(), _stream(stream)),
           "lsa_hot_pool_update")


# ----------------------------------------------------------------------------- 8-bit KV cache

_CODES = (torch.uint8, torch.float8_e4m3fn)
_QTYPES = (torch.float32, torch.bfloat16)
_I32, _F32, _F64, _U8 = (torch.int32,), (torch.float32,), (torch.float64,), (torch.uint8,)
_QTYPE = {LSA_F32: torch.float32, LSA_BF16: torch.bfloat16}


def _bad(t, name, dtypes, n, device):
    """Why a tensor cannot be passed on (the library would read it as it is)."""
    if t.dtype not in dtypes:
        return f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}"
    if t.get_device() != device or device < 0:
        return f"{name} is on {t.device}; every tensor of the call must be on one CUDA device"
    if not t.is_contiguous():
        return f"{name} of shape {tuple(t.shape)} with strides {t.stride()} is not contiguous"
    return f"{name} has {t.numel()} elements, the call uses {n}"


def _dev(t, name, dtypes, n, device):
    """Raw pointer of a dense device tensor of one of `dtypes` with at least n elements (None
    -> NULL); device: the CUDA device's index."""
    if t is None:
        return None
    if t.dtype in dtypes and t.get_device() == device >= 0 and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    raise ValueError(_bad(t, name, dtypes, n, device))


def _runs(counts, strides):
    """(count, stride) of a nest of dimensions, the innermost first, those that continue one another as one."""
    runs = []
    for n, s in zip(reversed(counts), reversed(strides)):
        if n == 1:
            continue
        if runs and runs[-1][0] * runs[-1][1] == s:
            runs[-1] = (runs[-1][0] * n, runs[-1][1])
        else:
            runs.append((n, s))
    return runs


def _same_walk(t, counts, strides):
    """Whether the view's first elements, in its own order, are those that `counts` steps of
    `strides` meet (outermost first)."""
    view, call = _runs(t.shape, t.stride()), _runs(counts, strides)
    for k, (n, s) in enumerate(call):
        if k >= len(view) or view[k][1] != s or view[k][0] < n or (view[k][0] > n and k + 1 < len(call)):
            return False
    return True


def _dev_strided(t, name, dtypes, span, device, counts=None, strides=None):
    """As _dev for a view that the call walks with strides of its own: `span` elements from the
    view's first one must lie in its storage, and a view that is not dense must have the elements that
    the call meets (counts and strides of its dimensions, outermost first)."""
    if t.dtype not in dtypes or t.get_device() != device or device < 0:
        raise ValueError(_bad(t, name, dtypes, 0, device))
    if 0 <= span <= t.numel() and t.is_contiguous() or t.shape == counts and t.stride() == strides and span >= 0:
        return t.data_ptr()
    if t.dim() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension has stride {t.stride(-1)}; it must be dense")
    if span < 0 or (t.storage_offset() + span) * t.element_size() > t.untyped_storage().nbytes():
        raise ValueError(f"{name}: {span} elements from its first one lie outside its storage")
    if counts is not None and span and not t.is_contiguous() and not _same_walk(t, counts, strides):
        raise ValueError(f"{name} of shape {tuple(t.shape)} has strides {t.stride()}, the call walks {counts} by {strides}")
    return t.data_ptr()


def _call(fn, where, device, stream, *args):
    """fn(*args, stream) with `device` current, on that device's current stream unless one is
    given."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if device == torch._C._cuda_getDevice():
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream)
    if rc != LSA_OK:
        _check(rc, where)


def _kv_cache(B, N, G, W, block, page, seq_pages, pages, table, rows, scale, device):
    """The cache arguments common to the three calls, checked against the tensors' sizes."""
    if block < 1 or page < 1:
        raise ValueError(f"block = {block}, page = {page}: powers of two")
    return (block, page, seq_pages, pages, _dev(table, "table", _I32, B * -(-N // page), device),
            _dev(rows, "rows", _CODES, pages * page * G * W, device),
            _dev(scale, "scale", _F32, B * -(-N // block) * G, device))


def lsa_kv_write(B, T, N, G, W, xdt, x, x_stride, start, count, block, page, seq_pages, pages, table, rows, scale,
                 status=None, stream=None):
    d = x.get_device()
    if x.dtype != _QTYPE.get(xdt):
        raise ValueError(f"x is {x.dtype}, xdt {xdt}")
    _call(lib().lsa_kv_write, "lsa_kv_write", d, stream, B, T, N, G, W, xdt,
          _dev_strided(x, "x", _QTYPES, (B * T - 1) * x_stride + G * W if B * T > 0 else 0, d, (B * T, G * W), (x_stride, 1)),
          x_stride,
          _dev(start, "start", _I32, B, d), _dev(count, "count", _I32, B, d),
          *_kv_cache(B, N, G, W, block, page, seq_pages, pages, table, rows, scale, d),
          _dev(status, "status", _I32, 1, d))


def lsa_kv_read(B, N, G, W, idx, cap, count, block, page, seq_pages, pages, table, rows, scale, odt, out,
                status=None, stream=None):
    d = out.get_device()
    if out.dtype != _QTYPE.get(odt):
        raise ValueError(f"out is {out.dtype}, odt {odt}")
    _call(lib().lsa_kv_read, "lsa_kv_read", d, stream, B, N, G, W, _dev(idx, "idx", _I32, B * cap, d), cap,
          _dev(count, "count", _I32, B, d),
          *_kv_cache(B, N, G, W, block, page, seq_pages, pages, table, rows, scale, d), odt,
          _dev(out, "out", _QTYPES, B * cap * G * W, d), _dev(status, "status", _I32, 1, d))


def _clip32(n):
    """n, or the nearest 32-bit number (a C int would take the low bits): for counts of tokens that may
    be larger than any sequence."""
    return n if -0x80000000 <= n <= 0x7FFFFFFF else 0x7FFFFFFF if n > 0 else -0x80000000


def lsa_kv_attend_workspace_bytes(B, Tq, N, H, G, d, dv, voff, W, qdt, sinks, window, cap) -> int:
    return int(lib().lsa_kv_attend_workspace_bytes(B, Tq, N, H, G, d, dv, voff, W, qdt, _clip32(sinks), _clip32(window), cap))


def lsa_kv_attend(B, Tq, N, H, G, d, dv, voff, W, qdt, q, sm_scale, length, sinks, window, idx, cap, count, block,
                  page, seq_pages, pages, table, rows, scale, out, lse, workspace, status=None, stream=None):
    dev = q.get_device()
    if q.dtype != _QTYPE.get(qdt) or out.dtype != q.dtype:
        raise ValueError(f"q is {q.dtype}, out {out.dtype}, qdt {qdt}")
    i32 = _I32
    _call(lib().lsa_kv_attend, "lsa_kv_attend", dev, stream, B, Tq, N, H, G, d, dv, voff, W, qdt,
          _dev(q, "q", _QTYPES, B * Tq * H * d, dev), float(sm_scale), _dev(length, "length", i32, B, dev), _clip32(sinks),
          _clip32(window), _dev(idx, "idx", i32, B * cap, dev), cap, _dev(count, "count", i32, B, dev),
          *_kv_cache(B, N, G, W, block, page, seq_pages, pages, table, rows, scale, dev),
          _dev(out, "out", _QTYPES, B * Tq * H * dv, dev), _dev(lse, "lse", _F32, B * Tq * H, dev),
          _dev(status, "status", i32, 1, dev), _dev(workspace, "workspace", _U8, 0, dev),
          0 if workspace is None else workspace.numel())


def lsa_rope(R, H, rot, half, dt, x, x_token, x_head, pos, freq, mscale, inverse, out, o_token, o_head, stream=None):
    d = x.get_device()
    if x.dtype != _QTYPE.get(dt) or out.dtype != x.dtype:
        raise ValueError(f"x is {x.dtype}, out {out.dtype}, dt {dt}")
    some, r, h = R > 0 and H > 0, R - 1, H - 1
    _call(lib().lsa_rope, "lsa_rope", d, stream, R, H, rot, int(half), dt,
          _dev_strided(x, "x", _QTYPES, r * x_token + h * x_head + rot if some else 0, d, (R, H, rot), (x_token, x_head, 1)),
          x_token, x_head,
          _dev(pos, "pos", _I32, R, d), _dev(freq, "freq", _F64, rot // 2, d), float(mscale),
          int(inverse), _dev_strided(out, "out", _QTYPES, r * o_token + h * o_head + rot if some else 0, d, (R, H, rot),
                                   (o_token, o_head, 1)), o_token, o_head)


def lsa_rope_frequencies(rot, base=10000.0, factor=1.0, original=0.0, fast=32.0, slow=1.0) -> torch.Tensor:
    """Host fp64 tensor [rot/2] of the pairs' frequencies; copy it to the device for lsa_rope."""
    f = torch.empty(max(rot, 0) // 2, dtype=torch.float64)
    _check(lib().lsa_rope_frequencies(rot, base, factor, original, fast, slow, f.data_ptr()), "lsa_rope_frequencies")
    return f


# ----------------------------------------------------------------------------- training step

def lsa_index_train_step_workspace_bytes(P, N, D, r, H, dI) -> int:
    return int(lib().lsa_index_train_step_workspace_bytes(P, N, D, r, H, dI))


def lsa_index_train_step(P, N, D, r, H, dI, wdt, h, W_down, W_up, W_w, bias, kdt, K, kscale, labels, gamma,
                         c_in, q_in, w_in, loss, dW_down, dW_up, dW_w, dbias, workspace, status=None, stream=None):
    _check(lib().lsa_index_train_step(P, N, D, r, H, dI, wdt, _p(h), _p(W_down), _p(W_up), _p(W_w), float(bias), kdt,
                                      _p(K), _p(kscale), _p(labels), float(gamma), _p(c_in), _p(q_in), _p(w_in),
                                      _p(loss), _p(dW_down), _p(dW_up), _p(dW_w), _p(dbias), _p(status),
                                      _p(workspace), 0 if workspace is None else workspace.numel(),
                                      _stream(stream)), "lsa_index_train_step")


# ----------------------------------------------------------------------------- self-check

def lsa_check_bounded_wait(limit_us, status, stream=None):
    _check(lib().lsa_check_bounded_wait(limit_us, _p(status), _stream(stream)), "lsa_check_bounded_wait")


# ----------------------------------------------------------------------------- labels

def lsa_vote_labels_workspace_bytes(L, P, N) -> int:
    return int(lib().lsa_vote_labels_workspace_bytes(L, P, N))


def lsa_vote_labels(L, P, N, logits, top_p, theta, golden, counts, scores, gamma, loss,
                    workspace, stream=None):
    _check(lib().lsa_vote_labels(L, P, N, _p(logits), float(top_p), theta, _p(golden), _p(counts),
                                 _p(scores), float(gamma), _p(loss), _p(workspace),
                                 0 if workspace is None else workspace.numel(), _stream(stream)),
           "lsa_vote_labels")
