"""Thin ctypes binding of libtoktier.so (include/toktier.h).

Functions carry the C names and only marshal arguments: torch CUDA tensors
and numpy arrays are passed as raw pointers, streams as cudaStream_t.  Every
step of the tokenization runs in the library's CUDA kernels; there is no
Python or CPU fallback, and loading fails loudly if the library is missing.
"""
import ctypes
import os
import re
import threading

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libtoktier.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "toktier.h")

TT_OK, TT_ERR_INVALID_ARG, TT_ERR_BAD_VOCAB, TT_ERR_BAD_FAMILY, TT_ERR_INVALID_UTF8, \
    TT_ERR_CAPACITY, TT_ERR_OOM, TT_ERR_CUDA, TT_ERR_TIMEOUT = range(9)
TT_FAMILY_CL100K_STYLE, TT_FAMILY_O200K_STYLE, TT_FAMILY_DEEPSEEK_STYLE = 1, 2, 3
TT_NOALLOC_MAX_BYTES, TT_NOALLOC_MAX_REQUESTS = 256 * 1024, 1024
TT_F32, TT_F16, TT_BF16 = range(3)
TT_MAX_IDS = 1 << 29

_lib = None
_lock = threading.Lock()


class TokTierError(RuntimeError):
    def __init__(self, status, what=""):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, status_string(status) if _lib else "", status))


def lib():
    """The loaded library with declared signatures (raises if not built)."""
    global _lib
    if _lib is not None:          # loaded once; no lock on the hot path
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libtoktier.so is not built (run __graft_entry__.build() or "
                                   "python -m exact_bpe_tokenization_gb300.build)")
            L = ctypes.CDLL(LIB_PATH)
            p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
            L.tt_create.argtypes = [p, i64, p, p, i64, i32, ctypes.POINTER(p)]
            L.tt_destroy.argtypes = [p]
            L.tt_encode_batch.argtypes = [p, p, p, i64, p, p, p]
            L.tt_encode_batch_bounded.argtypes = [p, p, p, i64, i64, p, p, p]
            L.tt_encode_batch_spans.argtypes = [p, p, p, i64, i64, p, p, p, p]
            L.tt_set_added_tokens.argtypes = [p, p, p, p, i64]
            L.tt_encode_batch_noalloc.argtypes = [p, p, p, i64, i64, p, p, p]
            L.tt_encode_host.argtypes = [p, p, p, i64, p, i64, p, p]
            L.tt_get_status.argtypes = [p, p, ctypes.POINTER(i64)]
            L.tt_pretokenize_batch.argtypes = [p, p, p, i64, p, p, p]
            L.tt_status_string.argtypes = [ctypes.c_int]
            L.tt_status_string.restype = ctypes.c_char_p
            L.tt_profile.argtypes = [p, ctypes.c_int]
            L.tt_profile_read.argtypes = [p, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                                          ctypes.POINTER(i64), ctypes.c_int]
            L.tt_launch_count.argtypes = [p]
            L.tt_launch_count.restype = i64
            L.tt_table_digest.restype = ctypes.c_char_p
            L.tt_debug_lookback.argtypes = [p, i32, i32]
            f32 = ctypes.c_float
            L.tt_embed.argtypes = [p, i64, p, p, i32, i64, i64, i64, f32, p, i32, i64, p, p]
            L.tt_embed_grad.argtypes = [p, i64, p, p, i32, i64, i64, f32, p, i32, i64, i64, i32, p, i64, p, p]
            L.tt_embed_grad_workspace.argtypes = [i64, i64, i64]
            L.tt_embed_grad_workspace.restype = i64
            L.tt_token_loss.argtypes = [p, i32, i64, i64, i64, p, p, p, p, p, i64, p, p]
            L.tt_token_loss_grad.argtypes = [p, i32, i64, i64, i64, p, p, p, p, i64, p, p]
            L.tt_sample.argtypes = [p, i32, i64, i64, i64, p, p, p, p, p, p, p, p, p]
            for name in ("tt_create", "tt_encode_batch", "tt_encode_batch_bounded", "tt_encode_batch_spans",
                         "tt_set_added_tokens",
                         "tt_encode_batch_noalloc",
                         "tt_encode_host",
                         "tt_get_status", "tt_pretokenize_batch", "tt_profile_read", "tt_debug_lookback",
                         "tt_embed", "tt_embed_grad", "tt_token_loss", "tt_token_loss_grad", "tt_sample"):
                getattr(L, name).restype = ctypes.c_int
            _lib = L
    return _lib


def declared_symbols():
    """Names of the functions include/toktier.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[\w\s\*]*?\b(tt_\w+)\s*\(", text, flags=re.M)))


def _ptr(x):
    """Raw address of a torch tensor, numpy array or None."""
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if isinstance(x, np.ndarray):
        return _np_addr(x)
    return int(x)


def _np_addr(a):
    """Address of a numpy array's data (a writable buffer through ctypes,
    a third of the cost of ndarray.ctypes; read-only or empty ones the slow way)."""
    try:
        return ctypes.addressof(ctypes.c_char.from_buffer(a))
    except (TypeError, ValueError):
        return a.ctypes.data


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _check(rc, what):
    if rc != TT_OK:
        raise TokTierError(rc, what)


def status_string(s):
    return lib().tt_status_string(int(s)).decode()


def tt_table_digest():
    return lib().tt_table_digest().decode()


def tt_create(merges, vocab_bytes, vocab_offsets, family):
    """Handle for (merges [k,2] int32, vocab bytes, vocab offsets [n+1] int64, family)."""
    m = np.ascontiguousarray(merges, dtype=np.int32).reshape(-1, 2)
    vb = np.ascontiguousarray(vocab_bytes, dtype=np.uint8)
    vo = np.ascontiguousarray(vocab_offsets, dtype=np.int64)
    h = ctypes.c_void_p()
    rc = lib().tt_create(m.ctypes.data if len(m) else None, len(m), vb.ctypes.data if len(vb) else None,
                         vo.ctypes.data, len(vo) - 1, int(family), ctypes.byref(h))
    _check(rc, "tt_create")
    return h


def tt_destroy(h):
    lib().tt_destroy(h)


def tt_encode_batch(h, d_utf8, d_byte_offsets, n_requests, d_out_ids, d_out_id_offsets, stream=None):
    _check(lib().tt_encode_batch(h, _ptr(d_utf8), _ptr(d_byte_offsets), int(n_requests), _ptr(d_out_ids),
                                 _ptr(d_out_id_offsets), _stream(stream)), "tt_encode_batch")


def tt_encode_batch_bounded(h, d_utf8, d_byte_offsets, n_requests, max_total_bytes, d_out_ids, d_out_id_offsets,
                            stream=None):
    _check(lib().tt_encode_batch_bounded(h, _ptr(d_utf8), _ptr(d_byte_offsets), int(n_requests),
                                         int(max_total_bytes), _ptr(d_out_ids), _ptr(d_out_id_offsets),
                                         _stream(stream)), "tt_encode_batch_bounded")


def tt_set_added_tokens(h, literals):
    """literals: {bytes: id} (host); an empty dict removes the set."""
    items = list(literals.items())
    data = np.frombuffer(b"".join(k for k, _ in items), dtype=np.uint8).copy()
    offs = np.zeros(len(items) + 1, dtype=np.int64)
    np.cumsum([len(k) for k, _ in items], out=offs[1:])
    ids = np.array([v for _, v in items], dtype=np.int32)
    _check(lib().tt_set_added_tokens(h, _ptr(data) if len(data) else None, _ptr(offs),
                                     _ptr(ids) if len(ids) else None, len(items)), "tt_set_added_tokens")


def tt_encode_batch_spans(h, d_utf8, d_byte_offsets, n_requests, max_total_bytes, d_out_ids, d_out_id_offsets,
                          d_out_spans, stream=None):
    _check(lib().tt_encode_batch_spans(h, _ptr(d_utf8), _ptr(d_byte_offsets), int(n_requests), int(max_total_bytes),
                                       _ptr(d_out_ids), _ptr(d_out_id_offsets), _ptr(d_out_spans),
                                       _stream(stream)), "tt_encode_batch_spans")


def tt_encode_batch_noalloc(h, d_utf8, d_byte_offsets, n_requests, max_total_bytes, d_out_ids, d_out_id_offsets,
                            stream=None):
    """As tt_encode_batch_bounded, with the library's fixed scratch: no device
    allocation, batches up to TT_NOALLOC_MAX_BYTES / TT_NOALLOC_MAX_REQUESTS."""
    _check(lib().tt_encode_batch_noalloc(h, _ptr(d_utf8), _ptr(d_byte_offsets), int(n_requests),
                                         int(max_total_bytes), _ptr(d_out_ids), _ptr(d_out_id_offsets),
                                         _stream(stream)), "tt_encode_batch_noalloc")


def tt_encode_host(h, utf8, byte_offsets, out_ids, out_id_offsets, stream=None):
    """Host buffers in and out (numpy).  Returns the batch's status code."""
    u = np.ascontiguousarray(utf8, dtype=np.uint8)
    o = np.ascontiguousarray(byte_offsets, dtype=np.int64)
    return lib().tt_encode_host(h, _np_addr(u) if len(u) else None, _np_addr(o), len(o) - 1,
                                _np_addr(out_ids), len(out_ids), _np_addr(out_id_offsets), _stream(stream))


def tt_get_status(h, stream=None):
    """(status code, lowest rejected request or -1); waits for the stream."""
    bad = ctypes.c_int64(-1)
    rc = lib().tt_get_status(h, _stream(stream), ctypes.byref(bad))
    return rc, bad.value


def tt_pretokenize_batch(h, d_utf8, d_byte_offsets, n_requests, d_piece_starts, d_piece_offsets, stream=None):
    _check(lib().tt_pretokenize_batch(h, _ptr(d_utf8), _ptr(d_byte_offsets), int(n_requests), _ptr(d_piece_starts),
                                      _ptr(d_piece_offsets), _stream(stream)), "tt_pretokenize_batch")


def tt_profile(h, enable):
    lib().tt_profile(h, int(bool(enable)))


def tt_profile_read(h, cap=16):
    names = (ctypes.c_char_p * cap)()
    ms = (ctypes.c_double * cap)()
    n = (ctypes.c_int64 * cap)()
    k = lib().tt_profile_read(h, names, ms, n, cap)
    return {names[i].decode(): (ms[i], n[i]) for i in range(k)}


def tt_launch_count(h):
    return lib().tt_launch_count(h)


def tt_debug_lookback(h, spin_limit, withhold_tile=-1):
    """Test setting: poll limit of the pre-tokenizer's look-back waits (0: the
    default) and a tile that publishes nothing (-1: none)."""
    _check(lib().tt_debug_lookback(h, int(spin_limit), int(withhold_tile)), "tt_debug_lookback")


# ---- operators around token IDs: the C calls

def tt_embed(d_ids, max_ids, d_n_ids, d_table, table_type, n_vocab, dim, table_stride, scale, d_out, out_type,
             out_stride, d_status=None, stream=None):
    _check(lib().tt_embed(_ptr(d_ids), max_ids, _ptr(d_n_ids), _ptr(d_table), table_type, n_vocab, dim, table_stride,
                          scale, _ptr(d_out), out_type, out_stride, _ptr(d_status), _stream(stream)), "tt_embed")


def tt_embed_grad(d_ids, max_ids, d_n_ids, d_dout, dout_type, dim, dout_stride, scale, d_dtable, dtable_type, n_vocab,
                  dtable_stride, accumulate, d_workspace, workspace_bytes, d_status=None, stream=None):
    _check(lib().tt_embed_grad(_ptr(d_ids), max_ids, _ptr(d_n_ids), _ptr(d_dout), dout_type, dim, dout_stride, scale,
                               _ptr(d_dtable), dtable_type, n_vocab, dtable_stride, int(accumulate),
                               _ptr(d_workspace), workspace_bytes, _ptr(d_status), _stream(stream)), "tt_embed_grad")


def tt_embed_grad_workspace(max_ids, n_vocab, dim):
    """Bytes of scratch, or -1 for sizes that tt_embed_grad rejects."""
    return lib().tt_embed_grad_workspace(int(max_ids), int(n_vocab), int(dim))


def tt_token_loss(d_logits, dtype, n_rows, n_vocab, logits_stride, d_targets, d_loss, d_lse, d_row_grads, d_dlogits,
                  dlogits_stride, d_status=None, stream=None):
    _check(lib().tt_token_loss(_ptr(d_logits), dtype, n_rows, n_vocab, logits_stride, _ptr(d_targets), _ptr(d_loss),
                               _ptr(d_lse), _ptr(d_row_grads), _ptr(d_dlogits), dlogits_stride, _ptr(d_status),
                               _stream(stream)), "tt_token_loss")


def tt_token_loss_grad(d_logits, dtype, n_rows, n_vocab, logits_stride, d_targets, d_lse, d_row_grads, d_dlogits,
                       dlogits_stride, d_status=None, stream=None):
    _check(lib().tt_token_loss_grad(_ptr(d_logits), dtype, n_rows, n_vocab, logits_stride, _ptr(d_targets),
                                    _ptr(d_lse), _ptr(d_row_grads), _ptr(d_dlogits), dlogits_stride, _ptr(d_status),
                                    _stream(stream)), "tt_token_loss_grad")


def tt_sample(d_logits, dtype, n_rows, n_vocab, logits_stride, d_uniform, d_temperature, d_top_k, d_top_p, d_min_p,
              d_out_ids, d_out_logprobs, d_status=None, stream=None):
    _check(lib().tt_sample(_ptr(d_logits), dtype, n_rows, n_vocab, logits_stride, _ptr(d_uniform),
                           _ptr(d_temperature), _ptr(d_top_k), _ptr(d_top_p), _ptr(d_min_p), _ptr(d_out_ids),
                           _ptr(d_out_logprobs), _ptr(d_status), _stream(stream)), "tt_sample")


# ---- the same on torch CUDA tensors: outputs and scratch allocated where they
# are not given, shapes, types and devices checked.  The kernels run on `stream` (the
# current one if None); what is allocated here is handed to that stream, and
# tensors that come from another one are the caller's to order and to keep
# (record_stream).  Small calls cost a few microseconds of device time, so these
# call the library without a layer in between.
#
# They are forward and backward calls, not autograd functions: tensors that require
# gradients are taken by their values, and no output has a graph behind it.

_codes = {}          # torch dtype -> tt_dtype; filled with the first use of torch
_torch = None        # the module, which this one does not need for anything else


def _load_torch():
    global _torch
    import torch
    _codes.update({torch.float32: TT_F32, torch.float16: TT_F16, torch.bfloat16: TT_BF16})
    _torch = torch
    return torch


def _cuda(on):
    return "CUDA" if on is None else "cuda:%d" % on


def _matrix(x, what, rows=None, cols=None, on=None):
    """(dtype code, rows, columns, row stride) of a 2-D CUDA tensor with unit
    column stride, on the device of index `on` if that is given."""
    code = _codes.get(x.dtype)
    if code is None:
        raise ValueError("%s: float32, float16 or bfloat16 wanted, got %s" % (what, x.dtype))
    shape, at = x.shape, x.get_device()
    if len(shape) != 2 or at < 0 or (on is not None and at != on) or (rows is not None and shape[0] != rows) or \
            (cols is not None and shape[1] != cols):
        raise ValueError("%s: a tensor [%s, %s] on %s wanted, got %s on %s" % (
            what, "n" if rows is None else rows, "n" if cols is None else cols, _cuda(on), list(shape), x.device))
    n, d = shape
    s0, s1 = x.stride()
    if s1 != 1 and d > 1:
        raise ValueError("%s: columns must be contiguous" % what)
    return code, n, d, (s0 if n > 1 else d)


def _vector(x, what, on, dtype, n=None, optional=False):
    """The address of a contiguous 1-D tensor on the device of index `on` (or
    None where it is optional)."""
    if x is None:
        if optional:
            return None
        raise ValueError("%s: a tensor wanted" % what)
    if x.dtype != dtype or x.get_device() != on or x.dim() != 1 or (n is not None and x.shape[0] != n) or \
            not x.is_contiguous():
        raise ValueError("%s: a contiguous tensor %s [%s] on %s wanted, got %s %s on %s" % (
            what, dtype, "n" if n is None else n, _cuda(on), x.dtype, list(x.shape), x.device))
    return x.data_ptr()


def _new(torch, rows, cols, dtype, device, what):
    """An output of its own: the tensor and its dtype code."""
    code = _codes.get(dtype)
    if code is None:
        raise ValueError("%s: float32, float16 or bfloat16 wanted, got %s" % (what, dtype))
    return torch.empty((rows, cols), dtype=dtype, device=device), code


def _on(torch, stream, on, *tensors):
    """The stream's address.  Tensors allocated here come from the current
    stream's pool: another stream waits for it and keeps them."""
    if torch._C._cuda_getDevice() != on:
        raise ValueError("the tensors are on cuda:%d, which is not the current device" % on)
    current = torch._C._cuda_getCurrentRawStream(on)
    if stream is None:
        return current
    raw = _stream(stream)
    mine = [t for t in tensors if t is not None]
    if raw != current and mine:
        s = torch.cuda.ExternalStream(raw, on)
        s.wait_stream(torch.cuda.current_stream(on))
        for t in mine:
            t.record_stream(s)
    return raw


def embed(ids, table, scale=1.0, n_ids=None, dtype=None, out=None, status=None, stream=None):
    """scale * table[ids] (zero rows for padding): out [len(ids), dim] of
    `dtype` (the table's if None).  n_ids: a device int64 count."""
    torch = _torch or _load_torch()
    t, vocab, dim, ts = _matrix(table, "table")
    on = table.get_device()
    pi = _vector(ids, "ids", on, torch.int32)
    n = ids.shape[0]
    mine = None
    if out is None:
        out, o = _new(torch, n, dim, dtype or table.dtype, table.device, "dtype")
        mine, os_ = out, dim
    else:
        o, _, _, os_ = _matrix(out, "out", n, dim, on)
    _check(lib().tt_embed(pi, n, _vector(n_ids, "n_ids", on, torch.int64, 1, True), table.data_ptr(), t, vocab, dim, ts,
                          scale, out.data_ptr(), o, os_, _vector(status, "status", on, torch.int32, 1, True),
                          _on(torch, stream, on, mine)), "tt_embed")
    return out


def embed_grad(ids, dout, n_vocab, scale=1.0, n_ids=None, dtype=None, out=None, accumulate=False, workspace=None,
               status=None, stream=None):
    """The gradient of embed: [n_vocab, dim] of `dtype` (float32 if None), the
    scaled sums of dout's rows by ID; with accumulate, added to `out`.
    workspace: a contiguous tensor of any type, of tt_embed_grad_workspace()
    bytes (allocated if None)."""
    torch = _torch or _load_torch()
    d, n, dim, ds = _matrix(dout, "dout")
    on = dout.get_device()
    pi = _vector(ids, "ids", on, torch.int32, n)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if workspace is not None and (workspace.get_device() != on or not workspace.is_contiguous()):
        raise ValueError("workspace: a contiguous tensor on cuda:%d wanted, got %s with strides %s on %s" % (
            on, list(workspace.shape), list(workspace.stride()), workspace.device))
    mine = scratch = None
    if out is None:
        out, o = _new(torch, n_vocab, dim, dtype or torch.float32, dout.device, "dtype")
        mine, os_ = out, dim
    else:
        o, _, _, os_ = _matrix(out, "out", n_vocab, dim, on)
    if workspace is None:
        workspace = scratch = torch.empty(max(lib().tt_embed_grad_workspace(n, n_vocab, dim), 16), dtype=torch.uint8,
                                          device=dout.device)
    _check(lib().tt_embed_grad(pi, n, _vector(n_ids, "n_ids", on, torch.int64, 1, True),
                               dout.data_ptr(), d, dim, ds, scale, out.data_ptr(), o, n_vocab, os_, bool(accumulate),
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               _vector(status, "status", on, torch.int32, 1, True),
                               _on(torch, stream, on, mine, scratch)), "tt_embed_grad")
    return out


def token_loss(logits, targets, row_grads=None, want_grad=False, dlogits=None, status=None, stream=None):
    """Next-token loss of each row: (loss, lse), and with want_grad or dlogits
    (which may be logits itself) the logits' gradient as a third."""
    torch = _torch or _load_torch()
    t, n, vocab, ls = _matrix(logits, "logits")
    on = logits.get_device()
    pt, pg = _vector(targets, "targets", on, torch.int32, n), _vector(row_grads, "row_grads", on, torch.float32, n, True)
    loss = torch.empty(n, dtype=torch.float32, device=logits.device)
    lse = torch.empty(n, dtype=torch.float32, device=logits.device)
    mine = None
    if dlogits is None and want_grad:
        dlogits = mine = torch.empty((n, vocab), dtype=logits.dtype, device=logits.device)
    d, ds, pd = t, vocab, None
    if dlogits is not None:
        if mine is None:
            d, _, _, ds = _matrix(dlogits, "dlogits", n, vocab, on)
        pd = dlogits.data_ptr()
    if d != t:
        raise ValueError("dlogits: the type of logits wanted")
    _check(lib().tt_token_loss(logits.data_ptr(), t, n, vocab, ls, pt, loss.data_ptr(), lse.data_ptr(), pg, pd, ds,
                               _vector(status, "status", on, torch.int32, 1, True),
                               _on(torch, stream, on, loss, lse, mine)), "tt_token_loss")
    return (loss, lse) if dlogits is None else (loss, lse, dlogits)


def token_loss_grad(logits, targets, lse, row_grads=None, dlogits=None, status=None, stream=None):
    """The gradient of token_loss from the lse that it returned."""
    torch = _torch or _load_torch()
    t, n, vocab, ls = _matrix(logits, "logits")
    on = logits.get_device()
    pt, pl = _vector(targets, "targets", on, torch.int32, n), _vector(lse, "lse", on, torch.float32, n)
    pg = _vector(row_grads, "row_grads", on, torch.float32, n, True)
    mine = None
    if dlogits is None:
        dlogits = mine = torch.empty((n, vocab), dtype=logits.dtype, device=logits.device)
    d, _, _, ds = _matrix(dlogits, "dlogits", n, vocab, on)
    if d != t:
        raise ValueError("dlogits: the type of logits wanted")
    _check(lib().tt_token_loss_grad(logits.data_ptr(), t, n, vocab, ls, pt, pl, pg, dlogits.data_ptr(), ds,
                                    _vector(status, "status", on, torch.int32, 1, True),
                                    _on(torch, stream, on, mine)), "tt_token_loss_grad")
    return dlogits


def sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, status=None, stream=None):
    """One token ID drawn from each row: (ids int32, logprobs float32).  The
    parameters are device tensors with an entry a row, or None (off)."""
    torch = _torch or _load_torch()
    t, n, vocab, ls = _matrix(logits, "logits")
    on, f = logits.get_device(), torch.float32
    pu = _vector(uniform, "uniform", on, f, n)
    ids = torch.empty(n, dtype=torch.int32, device=logits.device)
    logprobs = torch.empty(n, dtype=f, device=logits.device)
    _check(lib().tt_sample(logits.data_ptr(), t, n, vocab, ls, pu, _vector(temperature, "temperature", on, f, n, True),
                           _vector(top_k, "top_k", on, torch.int32, n, True), _vector(top_p, "top_p", on, f, n, True),
                           _vector(min_p, "min_p", on, f, n, True), ids.data_ptr(), logprobs.data_ptr(),
                           _vector(status, "status", on, torch.int32, 1, True), _on(torch, stream, on, ids, logprobs)),
           "tt_sample")
    return ids, logprobs


class Tokenizer:
    """Convenience owner of a handle; device arrays are torch CUDA tensors."""

    def __init__(self, merges, vocab_bytes, vocab_offsets, family):
        self.h = tt_create(merges, vocab_bytes, vocab_offsets, family)
        self.family = family

    def close(self):
        if self.h is not None:
            tt_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def encode(self, d_utf8, d_offsets, max_total_bytes=None, stream=None, out_ids=None, out_offsets=None):
        """Encode a device batch; returns (ids, id_offsets) device tensors."""
        import torch
        n = d_offsets.numel() - 1
        if max_total_bytes is None:
            max_total_bytes = d_utf8.numel()
        if out_ids is None:
            out_ids = torch.empty(max(int(max_total_bytes), 1), dtype=torch.int32, device=d_utf8.device)
        if out_offsets is None:
            out_offsets = torch.empty(n + 1, dtype=torch.int64, device=d_utf8.device)
        tt_encode_batch_bounded(self.h, d_utf8, d_offsets, n, max_total_bytes, out_ids, out_offsets, stream)
        return out_ids, out_offsets

    def set_added_tokens(self, literals):
        """Reserve literal byte strings as single IDs ({bytes: id})."""
        tt_set_added_tokens(self.h, literals)

    def encode_spans(self, d_utf8, d_offsets, max_total_bytes=None, stream=None):
        """Encode a device batch with byte spans; returns (ids, id_offsets,
        spans) device tensors, spans int32 [capacity, 2] (start, end) from the
        batch start."""
        import torch
        n = d_offsets.numel() - 1
        if max_total_bytes is None:
            max_total_bytes = d_utf8.numel()
        cap = max(int(max_total_bytes), 1)
        out_ids = torch.empty(cap, dtype=torch.int32, device=d_utf8.device)
        out_offsets = torch.empty(n + 1, dtype=torch.int64, device=d_utf8.device)
        spans = torch.empty((cap, 2), dtype=torch.int32, device=d_utf8.device)
        tt_encode_batch_spans(self.h, d_utf8, d_offsets, n, max_total_bytes, out_ids, out_offsets, spans, stream)
        return out_ids, out_offsets, spans

    def pretokenize(self, d_utf8, d_offsets, stream=None):
        import torch
        n = d_offsets.numel() - 1
        starts = torch.empty(max(d_utf8.numel(), 1), dtype=torch.int64, device=d_utf8.device)
        offs = torch.empty(n + 1, dtype=torch.int64, device=d_utf8.device)
        tt_pretokenize_batch(self.h, d_utf8, d_offsets, n, starts, offs, stream)
        return starts, offs

    def encode_host(self, utf8, offsets, stream=None):
        """Host in, host out: (ids, id_offsets, status)."""
        offsets = np.asarray(offsets, dtype=np.int64)
        total = int(offsets[-1] - offsets[0]) if len(offsets) > 1 else 0
        ids = np.empty(max(total, 1), dtype=np.int32)
        io = np.empty(len(offsets), dtype=np.int64)
        st = tt_encode_host(self.h, np.frombuffer(utf8, dtype=np.uint8) if isinstance(utf8, (bytes, bytearray))
                            else utf8, offsets, ids, io, stream)
        return ids[:int(io[-1])], io, st

    def status(self, stream=None):
        return tt_get_status(self.h, stream)
