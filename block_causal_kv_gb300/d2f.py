"""Python binding of libd2f (ctypes): argument marshalling only.

Every function takes torch CUDA tensors, passes their device pointers, sizes
and the current CUDA stream to the C entry point of the same name, and raises
D2FError on a non-OK status. No computation happens here; there is no CPU
fallback: if libd2f.so is missing the import fails.

With `stream` a call runs there instead. What it makes itself (results, a workspace) belongs to
that stream; the caller orders its inputs before the call and its use of the results after it.

    from block_causal_kv_gb300 import d2f
    out, lse = d2f.block_attn(q, k_win, v_win, k_pool, v_pool, page_table, ctx_len,
                              q_start, block_size=16, max_q_per_seq=48, max_ctx=1024)
    res = d2f.commit(logits, tokens, masked, q_start, block_phase, tau,
                     block_size=16, mask_id=126464)
    d2f.kv_append(k_win, v_win, src_row, dst_page, k_pool, v_pool, block_size=16)
    pool = d2f.kv4_pool("cuda", num_pages=4096, num_heads_kv=32, head_dim=128, block_size=16)
    d2f.kv4_append(k_win, v_win, src_row, dst_page, pool, block_size=16)
    out, lse = d2f.block_attn_kv4(q, k_win, v_win, pool, page_table, ctx_len, q_start,
                                  block_size=16, max_q_per_seq=48, max_ctx=1024)
    lp = d2f.token_logprobs(logits, res["argmax"], top_k=5)
"""
import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libd2f.so")

BF16 = 0
F32 = 1
PHASE_CONSERVATIVE = 0
PHASE_AGGRESSIVE = 1

STATUS = {0: "D2F_OK", 1: "D2F_ERR_INVALID_ARG", 2: "D2F_ERR_UNSUPPORTED", 3: "D2F_ERR_CUDA",
          4: "D2F_ERR_BAD_INDEX", 5: "D2F_ERR_TIMEOUT", 6: "D2F_ERR_WORKSPACE",
          7: "D2F_ERR_NO_PAGE"}

# Every symbol include/d2f.h declares.
EXPORTS = ("d2f_version", "d2f_status_string", "d2f_last_error_string",
           "d2f_block_attn_workspace_size", "d2f_block_attn", "d2f_block_attn_flags",
           "d2f_block_attn_append", "d2f_block_attn_part",
           "d2f_commit_workspace_size",
           "d2f_commit", "d2f_commit_metric", "d2f_commit_noalloc", "d2f_kv_append",
           "d2f_kv_append_dev", "d2f_block_attn_append_dev", "d2f_window_step",
           "d2f_kv4_page_bytes", "d2f_kv4_append", "d2f_kv4_read",
           "d2f_block_attn_kv4_workspace_size", "d2f_block_attn_kv4", "d2f_page_map",
           "d2f_page_map_flags",
           "d2f_token_logprobs_workspace_size", "d2f_token_logprobs")

# attention parts of block_attn(part=...) (include/d2f.h D2F_ATTN_*)
ATTN_ALL, ATTN_CACHED, ATTN_WINDOW = 0, 1, 2
# d2f_block_attn_flags: the cache and window layout are final before the preceding kernel
CACHE_READY = 1
# d2f_page_map_flags: ctx_len_out / free_count_out hold nothing yet
PAGE_MAP_FRESH = 1
# confidence metrics of commit(metric=...) (include/d2f.h D2F_CONF_*)
CONF_PMAX, CONF_NEG_ENTROPY, CONF_MARGIN, CONF_LOGIT_GAP = 0, 1, 2, 3


class D2FError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s: %s" % (STATUS.get(status, status), message))
        self.status = status


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t


def load(path=LIB_PATH):
    """Load libd2f.so (built in-tree by __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError("libd2f.so is not built (%s); run __graft_entry__.build()" % path)
    lib = ctypes.CDLL(path)
    lib.d2f_version.restype = _I
    lib.d2f_status_string.restype = ctypes.c_char_p
    lib.d2f_status_string.argtypes = [_I]
    lib.d2f_last_error_string.restype = ctypes.c_char_p
    lib.d2f_block_attn_workspace_size.restype = _I
    lib.d2f_block_attn_workspace_size.argtypes = [_I] * 10 + [ctypes.POINTER(_SZ)]
    lib.d2f_block_attn.restype = _I
    lib.d2f_block_attn.argtypes = ([_P] * 6 + [_I] + [_P] * 2 + [_P, _P] + [_I] * 10 +
                                   [ctypes.c_float, _I, _P, _SZ, _P, _P])
    lib.d2f_block_attn_flags.restype = _I
    lib.d2f_block_attn_flags.argtypes = ([_P] * 6 + [_I] + [_P] * 2 + [_P, _P] + [_I] * 10 +
                                         [ctypes.c_float, _I, _P, _SZ, ctypes.c_uint, _P, _P])
    lib.d2f_block_attn_append.restype = _I
    lib.d2f_block_attn_append.argtypes = ([_P] * 6 + [_I] + [_P] * 2 + [_P, _P] + [_I] * 10 +
                                          [ctypes.c_float, _I, _P, _SZ, _P, _P, _I, _P, _P])
    lib.d2f_block_attn_part.restype = _I
    lib.d2f_block_attn_part.argtypes = ([_P] * 6 + [_I] + [_P] * 2 + [_P, _P] + [_I] * 10 +
                                        [ctypes.c_float, _I, _P, _SZ, _I, _P, _P, _P, _P])
    lib.d2f_commit_workspace_size.restype = _I
    lib.d2f_commit_workspace_size.argtypes = [_I] * 5 + [ctypes.POINTER(_SZ)]
    lib.d2f_commit.restype = _I
    lib.d2f_commit.argtypes = ([_P, ctypes.c_int64, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I,
                                ctypes.c_int32, _P, _P, _P, _I, _P, _SZ, _P, _P])
    lib.d2f_commit_metric.restype = _I
    lib.d2f_commit_metric.argtypes = ([_P, ctypes.c_int64, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I,
                                       _I, _I, ctypes.c_int32, _I, _P, _P, _P, _P, _P, _I, _P, _SZ,
                                       _P, _P])
    lib.d2f_commit_noalloc.restype = _I
    lib.d2f_commit_noalloc.argtypes = ([_P, ctypes.c_int64, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I,
                                        _I, _I, ctypes.c_int32, _P, _P, _P, _I, _P, _P])
    lib.d2f_kv_append.restype = _I
    lib.d2f_kv_append.argtypes = [_P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P]
    lib.d2f_kv_append_dev.restype = _I
    lib.d2f_kv_append_dev.argtypes = [_P, _P, _P, _P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _I,
                                      _P, _P]
    lib.d2f_block_attn_append_dev.restype = _I
    lib.d2f_block_attn_append_dev.argtypes = ([_P] * 6 + [_I] + [_P] * 2 + [_P, _P] + [_I] * 10 +
                                              [ctypes.c_float, _I, _P, _SZ, _P, _P, _P, _I, _P,
                                               _P])
    lib.d2f_window_step.restype = _I
    lib.d2f_window_step.argtypes = ([_I] * 5 + [ctypes.c_int32, ctypes.c_float, ctypes.c_float] +
                                    [_P] * 18)
    lib.d2f_kv4_page_bytes.restype = _I
    lib.d2f_kv4_page_bytes.argtypes = [_I, _I, ctypes.POINTER(_SZ)]
    lib.d2f_kv4_append.restype = _I
    lib.d2f_kv4_append.argtypes = [_P] * 6 + [_I, _I, _P] + [_I] * 7 + [_P, _P]
    lib.d2f_kv4_read.restype = _I
    lib.d2f_kv4_read.argtypes = [_P, _P, _I, _P, _P] + [_I] * 7 + [_P, _P]
    lib.d2f_block_attn_kv4_workspace_size.restype = _I
    lib.d2f_block_attn_kv4_workspace_size.argtypes = [_I] * 9 + [ctypes.POINTER(_SZ)]
    lib.d2f_block_attn_kv4.restype = _I
    lib.d2f_block_attn_kv4.argtypes = ([_P] * 5 + [_I] + [_P] * 4 + [_I] * 12 +
                                       [ctypes.c_float, _P, _SZ, _P, _P])
    lib.d2f_page_map.restype = _I
    lib.d2f_page_map.argtypes = [_I] * 5 + [_P] * 16
    lib.d2f_page_map_flags.restype = _I
    lib.d2f_page_map_flags.argtypes = [_I] * 5 + [_P] * 14 + [ctypes.c_uint, _P, _P]
    lib.d2f_token_logprobs_workspace_size.restype = _I
    lib.d2f_token_logprobs_workspace_size.argtypes = [_I] * 4 + [ctypes.POINTER(_SZ)]
    lib.d2f_token_logprobs.restype = _I
    lib.d2f_token_logprobs.argtypes = ([_P, ctypes.c_int64, _I, _I, _I, _P, _P, _I, _I] +
                                       [_P] * 4 + [_P, _SZ, _P, _P])
    _lib = lib
    return lib


def _check(status):
    if status != 0:
        raise D2FError(status, _lib.d2f_last_error_string().decode())


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("libd2f takes bfloat16 or float32 tensors, got %s" % t.dtype)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _on(stream, make):
    """make, for a tensor that a call on `stream` writes (None: the current one). It is made on that
    stream (its fill, or what used its memory before, is ordered with the call there), and its
    memory is kept for what the caller's current stream does with it."""
    return make if stream is None else functools.partial(_make_on, stream, make)


def _make_on(stream, make, *args, **kw):
    current = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    t.record_stream(current)
    return t


def _dev(t, name, dtype=None):
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _refuse(name, t, dtype, shape, dev):
    """Raise for the tensor that `_device` found wrong, with the reason."""
    _dev(t, name, dtype)
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s is on cuda:%d, the others on cuda:%d" % (name, t.get_device(), dev))


def _device(*tensors):
    """The device of the given tensors, which must be contiguous CUDA tensors of that device.
    Entries are (name, tensor or None, dtype, shape or None). (One loop with the cheapest checks: it
    is a third of what a small call costs.)"""
    dev = tensors[0][1].get_device()
    for name, t, dtype, shape in tensors:
        if t is not None and (t.dtype is not dtype or (shape is not None and t.shape != shape) or
                              t.get_device() != dev or not t.is_contiguous()):
            _refuse(name, t, dtype, shape, dev)
    if dev < 0:
        _dev(tensors[0][1], tensors[0][0])
    return dev


def _launch(fn, dev, stream, *args):
    """fn(*args, stream) with `dev` current; its current stream unless one is given."""
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == dev:
        status = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, s)
    if status != 0:
        _check(status)


def status_string(status):
    return load().d2f_status_string(status).decode()


def version():
    return load().d2f_version()


# ---------------------------------------------------------------------------
# block attention
# ---------------------------------------------------------------------------
def attn_workspace_size(batch, total_q, max_q_per_seq, max_ctx, num_heads_q, num_heads_kv,
                        head_dim, block_size, dtype=BF16, num_splits=0):
    lib = load()
    n = _SZ(0)
    _check(lib.d2f_block_attn_workspace_size(batch, total_q, max_q_per_seq, max_ctx, num_heads_q,
                                             num_heads_kv, head_dim, block_size, dtype,
                                             num_splits, ctypes.byref(n)))
    return n.value


def attn_workspace(device, **kw):
    """A zero-filled workspace of the size attn_workspace_size(**kw) returns."""
    return torch.zeros(max(attn_workspace_size(**kw), 1), dtype=torch.uint8, device=device)


def block_attn(q, k_win, v_win, k_pool, v_pool, page_table, ctx_len, q_start, *, block_size,
               max_q_per_seq, max_ctx, softmax_scale=None, num_splits=0, out=None, lse=None,
               want_lse=True, workspace=None, err=None, stream=None, append_src_row=None,
               append_dst_page=None, part=ATTN_ALL, prev_out=None, prev_lse=None,
               append_n_dev=None, cache_ready=False):
    """Block-causal attention of the window over [paged cache ; window] (one layer).
    With append_src_row / append_dst_page (int32 [n_append]) the finished blocks
    are appended to their pages in the same launch (d2f_block_attn_append).
    With append_n_dev (int32 [1] on the device, d2f_block_attn_append_dev) the list's
    length is read there, at most len(append_src_row).
    part ATTN_CACHED / ATTN_WINDOW (d2f_block_attn_part): one part of the keys; the
    window part composes a kept cached part given as prev_out / prev_lse.
    cache_ready=True (d2f_block_attn_flags with D2F_ATTN_CACHE_READY, the whole
    attention only): page_table, ctx_len, q_start and the cached pages are not
    written by the kernel that precedes this call in the stream.

    Returns (out [total_q, Hq, D] like q, lse [total_q, Hq] float32 or None)."""
    lib = load()
    for name, t in (("q", q), ("k_win", k_win), ("v_win", v_win), ("k_pool", k_pool),
                    ("v_pool", v_pool)):
        _dev(t, name, q.dtype)
    _dev(page_table, "page_table", torch.int32)
    _dev(ctx_len, "ctx_len", torch.int32)
    _dev(q_start, "q_start", torch.int32)
    total_q, hq, d = q.shape
    hkv = k_win.shape[1]
    batch = ctx_len.shape[0]
    dt = _dtype_code(q)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    empty = _on(stream, torch.empty)
    if out is None:
        out = _on(stream, torch.empty_like)(q)
    _dev(out, "out", q.dtype)
    if lse is None and want_lse:
        lse = empty((total_q, hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _on(stream, attn_workspace)(
            q.device, batch=batch, total_q=total_q, max_q_per_seq=max_q_per_seq, max_ctx=max_ctx,
            num_heads_q=hq, num_heads_kv=hkv, head_dim=d, block_size=block_size, dtype=dt,
            num_splits=num_splits)
    args = (_ptr(q), _ptr(k_win), _ptr(v_win), _ptr(k_pool), _ptr(v_pool), _ptr(page_table),
            page_table.shape[1] if page_table is not None else 0, _ptr(ctx_len), _ptr(q_start),
            _ptr(out), _ptr(lse), batch, total_q, max_q_per_seq, max_ctx, hq, hkv, d, block_size,
            k_pool.shape[0] if k_pool is not None else 0, dt, float(softmax_scale), num_splits,
            _ptr(workspace), workspace.numel() * workspace.element_size())
    if cache_ready and (part != ATTN_ALL or append_src_row is not None):
        raise ValueError("cache_ready goes with the whole attention, without an append")
    if part != ATTN_ALL:
        if append_src_row is not None:
            raise ValueError("an append goes with the whole attention (part ATTN_ALL)")
        _dev(prev_out, "prev_out", q.dtype)
        _dev(prev_lse, "prev_lse", torch.float32)
        _check(lib.d2f_block_attn_part(*args, int(part), _ptr(prev_out), _ptr(prev_lse), _ptr(err),
                                       _stream(stream)))
    elif append_src_row is None and cache_ready:
        _check(lib.d2f_block_attn_flags(*args, CACHE_READY, _ptr(err), _stream(stream)))
    elif append_src_row is None:
        _check(lib.d2f_block_attn(*args, _ptr(err), _stream(stream)))
    elif append_n_dev is not None:
        _dev(append_src_row, "append_src_row", torch.int32)
        _dev(append_dst_page, "append_dst_page", torch.int32)
        _dev(append_n_dev, "append_n_dev", torch.int32)
        _check(lib.d2f_block_attn_append_dev(*args, _ptr(append_src_row), _ptr(append_dst_page),
                                             _ptr(append_n_dev), append_src_row.shape[0],
                                             _ptr(err), _stream(stream)))
    else:
        _dev(append_src_row, "append_src_row", torch.int32)
        _dev(append_dst_page, "append_dst_page", torch.int32)
        _check(lib.d2f_block_attn_append(*args, _ptr(append_src_row), _ptr(append_dst_page),
                                         append_src_row.shape[0], _ptr(err), _stream(stream)))
    return out, lse


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
def commit_workspace_size(total_q, vocab, block_size, dtype=BF16, num_splits=0):
    lib = load()
    n = _SZ(0)
    _check(lib.d2f_commit_workspace_size(total_q, vocab, dtype, block_size, num_splits,
                                         ctypes.byref(n)))
    return n.value


def commit_workspace(device, **kw):
    return torch.zeros(max(commit_workspace_size(**kw), 1), dtype=torch.uint8, device=device)


def commit(logits, tokens, masked, q_start, block_phase, tau, *, block_size, mask_id,
           logit_row=None, num_splits=0, conf=None, argmax=None, block_remaining=None,
           want_outputs=True, workspace=None, err=None, stream=None, metric=CONF_PMAX,
           early_gap=None, stopped=None):
    """Confidence commit + remask, in place on tokens / masked.

    logits may be a row-strided view ([rows, vocab] with stride(1) == 1).
    metric: CONF_PMAX (d2f_commit) or another CONF_* (d2f_commit_metric; tau in
    the metric's units). early_gap (float32 [batch]) turns on the early commit
    of whole sequences; stopped (uint8 [batch]) receives its flags. Returns
    dict(conf, argmax, block_remaining, stopped) (device tensors, or None)."""
    lib = load()
    if not logits.is_cuda or logits.stride(-1) != 1:
        raise ValueError("logits must be a CUDA tensor with unit stride along the vocabulary")
    _dev(tokens, "tokens", torch.int32)
    _dev(masked, "masked", torch.uint8)
    _dev(q_start, "q_start", torch.int32)
    _dev(block_phase, "block_phase", torch.uint8)
    _dev(tau, "tau", torch.float32)
    _dev(logit_row, "logit_row", torch.int32)
    total_q = tokens.shape[0]
    rows, vocab = logits.shape
    dt = _dtype_code(logits)
    dev = tokens.device
    empty = _on(stream, torch.empty)
    if want_outputs:
        if conf is None:
            conf = empty(total_q, dtype=torch.float32, device=dev)
        if argmax is None:
            argmax = empty(total_q, dtype=torch.int32, device=dev)
        if block_remaining is None:
            block_remaining = empty(max(total_q // block_size, 1), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _on(stream, commit_workspace)(dev, total_q=total_q, vocab=vocab,
                                                  block_size=block_size, dtype=dt,
                                                  num_splits=num_splits)
    _dev(early_gap, "early_gap", torch.float32)
    _dev(stopped, "stopped", torch.uint8)
    if metric == CONF_PMAX and early_gap is None:
        _check(lib.d2f_commit(
            _ptr(logits), logits.stride(0), dt, vocab, rows, _ptr(logit_row), _ptr(tokens),
            _ptr(masked), _ptr(q_start), _ptr(block_phase), _ptr(tau), q_start.shape[0] - 1,
            total_q, block_size, int(mask_id), _ptr(conf), _ptr(argmax), _ptr(block_remaining),
            num_splits, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err),
            _stream(stream)))
    else:
        _check(lib.d2f_commit_metric(
            _ptr(logits), logits.stride(0), dt, vocab, rows, _ptr(logit_row), _ptr(tokens),
            _ptr(masked), _ptr(q_start), _ptr(block_phase), _ptr(tau), q_start.shape[0] - 1,
            total_q, block_size, int(mask_id), int(metric), _ptr(early_gap), _ptr(stopped),
            _ptr(conf), _ptr(argmax), _ptr(block_remaining), num_splits, _ptr(workspace),
            workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream)))
    return {"conf": conf, "argmax": argmax, "block_remaining": block_remaining,
            "stopped": stopped}


def commit_noalloc(logits, tokens, masked, q_start, block_phase, tau, *, block_size, mask_id,
                   logit_row=None, num_splits=0, conf=None, argmax=None, block_remaining=None,
                   err=None, stream=None):
    """d2f_commit_noalloc: the commit without a workspace, for callers that cannot
    allocate device memory; its scratch is a fixed array inside the library (see
    include/d2f.h for the size limit and the rule that calls must not overlap)."""
    lib = load()
    if not logits.is_cuda or logits.stride(-1) != 1:
        raise ValueError("logits must be a CUDA tensor with unit stride along the vocabulary")
    total_q = tokens.shape[0]
    rows, vocab = logits.shape
    _check(lib.d2f_commit_noalloc(
        _ptr(logits), logits.stride(0), _dtype_code(logits), vocab, rows, _ptr(logit_row),
        _ptr(tokens), _ptr(masked), _ptr(q_start), _ptr(block_phase), _ptr(tau),
        q_start.shape[0] - 1, total_q, block_size, int(mask_id), _ptr(conf), _ptr(argmax),
        _ptr(block_remaining), num_splits, _ptr(err), _stream(stream)))
    return {"conf": conf, "argmax": argmax, "block_remaining": block_remaining}


# ---------------------------------------------------------------------------
# KV append
# ---------------------------------------------------------------------------
def kv_append(k_win, v_win, src_row, dst_page, k_pool, v_pool, *, block_size, err=None,
              stream=None, n_append_dev=None):
    """Copy finished blocks (rows src_row[a] .. +B of the window K/V) into pages dst_page[a].
    n_append_dev (int32 [1] on the device, d2f_kv_append_dev): the list's length is
    read there, at most len(src_row)."""
    lib = load()
    for name, t in (("k_win", k_win), ("v_win", v_win), ("k_pool", k_pool), ("v_pool", v_pool)):
        _dev(t, name, k_win.dtype)
    _dev(src_row, "src_row", torch.int32)
    _dev(dst_page, "dst_page", torch.int32)
    total_q, hkv, d = k_win.shape
    if n_append_dev is not None:
        _dev(n_append_dev, "n_append_dev", torch.int32)
        _check(lib.d2f_kv_append_dev(
            _ptr(k_win), _ptr(v_win), _ptr(src_row), _ptr(dst_page), _ptr(n_append_dev),
            src_row.shape[0], total_q, _ptr(k_pool), _ptr(v_pool), hkv, d, block_size,
            k_pool.shape[0], _dtype_code(k_win), _ptr(err), _stream(stream)))
        return
    _check(lib.d2f_kv_append(
        _ptr(k_win), _ptr(v_win), _ptr(src_row), _ptr(dst_page), src_row.shape[0], total_q,
        _ptr(k_pool), _ptr(v_pool), hkv, d, block_size, k_pool.shape[0], _dtype_code(k_win),
        _ptr(err), _stream(stream)))


# ---------------------------------------------------------------------------
# pipelined window scheduler
# ---------------------------------------------------------------------------
class WindowState:
    """Device buffers of the window scheduler (d2f_window_step), one attribute per
    argument of that name: q_start, tokens, masked, block_phase, row_pos,
    ctx_len, page_table, next_block, gen_blocks, n_leaving, stopped, free_pages,
    free_count, app_src, app_dst, n_append. Created empty (no window, nothing
    listed); the caller fills ctx_len / page_table (prompt pages), gen_blocks
    and the free list."""

    def __init__(self, device, *, batch, block_size, max_blocks, max_pages_per_seq, num_free,
                 mask_id, capacity=None):
        i32 = dict(dtype=torch.int32, device=device)
        u8 = dict(dtype=torch.uint8, device=device)
        cap = batch * max_blocks * block_size if capacity is None else capacity
        self.batch, self.block_size, self.max_blocks, self.capacity = (batch, block_size,
                                                                       max_blocks, cap)
        self.mask_id = mask_id
        self.q_start = torch.zeros(batch + 1, **i32)
        self.tokens = torch.full((cap,), mask_id, **i32)
        self.masked = torch.zeros(cap, **u8)
        self.block_phase = torch.zeros(max(cap // block_size, 1), **u8)
        self.row_pos = torch.full((cap,), -1, **i32)
        self.ctx_len = torch.zeros(batch, **i32)
        self.page_table = torch.full((batch, max_pages_per_seq), -1, **i32)
        self.next_block = torch.zeros(batch, **i32)
        self.gen_blocks = torch.zeros(batch, **i32)
        self.n_leaving = torch.zeros(batch, **i32)
        self.stopped = torch.zeros(batch, **u8)
        self.free_pages = torch.zeros(max(num_free, 1), **i32)
        self.free_count = torch.zeros(1, **i32)
        self.app_src = torch.zeros(max(cap // block_size, 1), **i32)
        self.app_dst = torch.zeros_like(self.app_src)
        self.n_append = torch.zeros(1, **i32)


def window_step(st, *, tau_add, tau_act, err=None, stream=None, use_stopped=True):
    """One call of the device window scheduler on WindowState `st` (in place)."""
    lib = load()
    _check(lib.d2f_window_step(
        st.batch, st.block_size, st.max_blocks, st.capacity, st.page_table.shape[1],
        int(st.mask_id), float(tau_add), float(tau_act), _ptr(st.q_start), _ptr(st.tokens),
        _ptr(st.masked), _ptr(st.block_phase), _ptr(st.row_pos), _ptr(st.ctx_len),
        _ptr(st.page_table), _ptr(st.next_block), _ptr(st.gen_blocks), _ptr(st.n_leaving),
        _ptr(st.stopped) if use_stopped else None, _ptr(st.free_pages), _ptr(st.free_count),
        _ptr(st.app_src), _ptr(st.app_dst), _ptr(st.n_append), _ptr(err), _stream(stream)))


# ---------------------------------------------------------------------------
# 4-bit paged cache
# ---------------------------------------------------------------------------
@functools.lru_cache(maxsize=32)  # (every call on a pool asks)
def kv4_page_bytes(head_dim, block_size):
    """Bytes of one page of one KV head in a 4-bit pool."""
    lib = load()
    n = _SZ(0)
    _check(lib.d2f_kv4_page_bytes(head_dim, block_size, ctypes.byref(n)))
    return n.value


def kv4_pool(device, *, num_pages, num_heads_kv, head_dim, block_size):
    """A zero-filled 4-bit pool: uint8 [num_pages, num_heads_kv, page bytes]."""
    return torch.zeros((num_pages, num_heads_kv, kv4_page_bytes(head_dim, block_size)),
                       dtype=torch.uint8, device=device)


def _kv4_pool_shape(pool, num_heads_kv, head_dim, block_size):
    if pool.dim() != 3:
        raise ValueError("the 4-bit pool is [num_pages, num_heads_kv, page bytes]")
    return (pool.shape[0], num_heads_kv, kv4_page_bytes(head_dim, block_size))


def kv4_append(k_win, v_win, src_row, dst_page, pool, *, block_size, n_rows=None, k_exp=0,
               v_exp=0, n_append_dev=None, err=None, stream=None):
    """Quantise blocks (rows src_row[a] .. + n_rows[a] of K/V [rows, Hkv, D]; n_rows None:
    block_size each) into pages dst_page[a] of a 4-bit pool. With n_append_dev (int32 [1]
    on the device) the list's length is read there, at most len(src_row)."""
    shape = k_win.shape
    total_q, hkv, d = shape
    n = src_row.shape[0]
    i32 = torch.int32
    dev = _device(("k_win", k_win, k_win.dtype, shape), ("v_win", v_win, k_win.dtype, shape),
                  ("src_row", src_row, i32, (n,)), ("dst_page", dst_page, i32, (n,)),
                  ("pool", pool, torch.uint8, _kv4_pool_shape(pool, hkv, d, block_size)),
                  ("n_rows", n_rows, i32, (n,)), ("n_append_dev", n_append_dev, i32, (1,)),
                  ("err", err, i32, None))
    _launch(load().d2f_kv4_append, dev, stream, k_win.data_ptr(), v_win.data_ptr(),
            src_row.data_ptr(), dst_page.data_ptr(), _ptr(n_rows), _ptr(n_append_dev), n, total_q,
            pool.data_ptr(), hkv, d, block_size, pool.shape[0], int(k_exp), int(v_exp),
            _dtype_code(k_win), _ptr(err))


def kv4_read(pool, slot, *, head_dim, block_size, dtype=torch.bfloat16, k_exp=0, v_exp=0,
             k=None, v=None, err=None, stream=None):
    """Tokens at int64 slots (page * block_size + offset; -1 gives zeros) of a 4-bit pool.

    Returns (k, v) [len(slot), Hkv, D] of `dtype`, exact."""
    pool_shape = _kv4_pool_shape(pool, pool.shape[1], head_dim, block_size)
    hkv = pool_shape[1]
    n = slot.shape[0]
    shape = (n, hkv, head_dim)
    empty = _on(stream, torch.empty)
    if k is None:
        k = empty(shape, dtype=dtype, device=pool.device)
    if v is None:
        v = empty(shape, dtype=dtype, device=pool.device)
    dev = _device(("pool", pool, torch.uint8, pool_shape), ("slot", slot, torch.int64, (n,)),
                  ("k", k, dtype, shape), ("v", v, dtype, shape),
                  ("err", err, torch.int32, None))
    _launch(load().d2f_kv4_read, dev, stream, pool.data_ptr(), slot.data_ptr(), n, k.data_ptr(),
            v.data_ptr(), hkv, head_dim, block_size, pool_shape[0], int(k_exp), int(v_exp),
            _dtype_code(k), _ptr(err))
    return k, v


def attn_kv4_workspace_size(batch, total_q, max_q_per_seq, max_ctx, num_heads_q, num_heads_kv,
                            head_dim, block_size, dtype=BF16):
    lib = load()
    n = _SZ(0)
    _check(lib.d2f_block_attn_kv4_workspace_size(batch, total_q, max_q_per_seq, max_ctx,
                                                 num_heads_q, num_heads_kv, head_dim, block_size,
                                                 dtype, ctypes.byref(n)))
    return n.value


def attn_kv4_workspace(device, **kw):
    """A zero-filled workspace of the size attn_kv4_workspace_size(**kw) returns."""
    with torch.cuda.device(device):
        return torch.zeros(max(attn_kv4_workspace_size(**kw), 1), dtype=torch.uint8, device=device)


def block_attn_kv4(q, k_win, v_win, pool, page_table, ctx_len, q_start, *, block_size,
                   max_q_per_seq, max_ctx, k_exp=0, v_exp=0, softmax_scale=None, out=None,
                   lse=None, want_lse=True, workspace=None, err=None, stream=None):
    """Block-causal attention of the window over [4-bit paged cache ; window] (one layer):
    block_attn with one 4-bit pool in place of k_pool and v_pool.

    Returns (out [total_q, Hq, D] like q, lse [total_q, Hq] float32 or None)."""
    total_q, hq, d = q.shape
    hkv = k_win.shape[1]
    batch = ctx_len.shape[0]
    max_pages = page_table.shape[-1]
    dt = _dtype_code(q)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(d)
    empty = _on(stream, torch.empty)
    if out is None:
        out = _on(stream, torch.empty_like)(q)
    if lse is None and want_lse:
        lse = empty((total_q, hq), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _on(stream, attn_kv4_workspace)(
            q.device, batch=batch, total_q=total_q, max_q_per_seq=max_q_per_seq, max_ctx=max_ctx,
            num_heads_q=hq, num_heads_kv=hkv, head_dim=d, block_size=block_size, dtype=dt)
    qd, i32 = q.dtype, torch.int32
    win = (total_q, hkv, d)
    dev = _device(("q", q, qd, q.shape), ("k_win", k_win, qd, win), ("v_win", v_win, qd, win),
                  ("pool", pool, torch.uint8, _kv4_pool_shape(pool, hkv, d, block_size)),
                  ("page_table", page_table, i32, (batch, max_pages)),
                  ("ctx_len", ctx_len, i32, (batch,)), ("q_start", q_start, i32, (batch + 1,)),
                  ("out", out, qd, q.shape), ("lse", lse, torch.float32, (total_q, hq)),
                  ("workspace", workspace, workspace.dtype, None),
                  ("err", err, i32, None))
    _launch(load().d2f_block_attn_kv4, dev, stream, q.data_ptr(), k_win.data_ptr(),
            v_win.data_ptr(), pool.data_ptr(), page_table.data_ptr(), max_pages,
            ctx_len.data_ptr(), q_start.data_ptr(), out.data_ptr(), _ptr(lse), batch, total_q,
            max_q_per_seq, max_ctx, hq, hkv, d, block_size, pool.shape[0], int(k_exp), int(v_exp),
            dt, float(softmax_scale), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _ptr(err))
    return out, lse


# ---------------------------------------------------------------------------
# page map of a batch of requests
# ---------------------------------------------------------------------------
def page_map(num_new, ctx_len, page_table, free_pages, free_count, *, block_size, capacity,
             max_append, ctx_len_out=None, free_count_out=None, err=None, stream=None):
    """Lay out num_new[b] new tokens of each request behind its ctx_len[b] cached ones, with
    pages off the free list (d2f_page_map). page_table is written in place; ctx_len_out and
    free_count_out are new tensors unless given (ctx_len and free_count themselves update
    in place). An inconsistent state lays out nothing (n_append -1, admitted 0, slot -1, an
    empty list) and leaves the contexts and the free count as they were.

    Returns a dict: page_table, ctx_len, row_start [batch + 1], admitted uint8 [batch], slot
    int64 [capacity], app_src / app_dst / app_rows [max_append] and n_append [1] (the list
    kv4_append takes), free_count [1]."""
    batch = num_new.shape[0]
    device = num_new.device
    max_pages = page_table.shape[-1]
    if capacity < 0 or max_append < 0:
        raise ValueError("capacity and max_append must not be negative")
    i32 = torch.int32
    empty = _on(stream, torch.empty)
    # the int32 results, one allocation (no gradients here, so the split without view
    # tracking does: 8 us for the seven against 13 with it and 10 for seven allocations)
    ctx_new, free_new, row_start, n_append, src, dst, rows = empty(
        2 * batch + 3 + 3 * max_append, dtype=i32, device=device).unsafe_split_with_sizes(
            [batch, 1, batch + 1, 1, max_append, max_append, max_append])
    # a refused state leaves tensors that were given as they are, and the inputs in new ones
    # (PAGE_MAP_FRESH writes both: one that was given beside a new one takes its input too)
    flags = 0 if ctx_len_out is not None and free_count_out is not None else PAGE_MAP_FRESH
    if ctx_len_out is None:
        ctx_len_out = ctx_new
    if free_count_out is None:
        free_count_out = free_new
    admitted = empty(batch, dtype=torch.uint8, device=device)
    slot = empty(capacity, dtype=torch.int64, device=device)
    dev = _device(("num_new", num_new, i32, (batch,)), ("ctx_len", ctx_len, i32, (batch,)),
                  ("page_table", page_table, i32, (batch, max_pages)),
                  ("free_pages", free_pages, i32, None),
                  ("free_count", free_count, i32, (1,)), ("ctx_len_out", ctx_len_out, i32, (batch,)),
                  ("free_count_out", free_count_out, i32, (1,)), ("err", err, i32, None))
    _launch(load().d2f_page_map_flags, dev, stream, batch, block_size, max_pages, capacity,
            max_append, num_new.data_ptr(), ctx_len.data_ptr(), free_pages.data_ptr(),
            free_count.data_ptr(), page_table.data_ptr(), ctx_len_out.data_ptr(), free_count_out.data_ptr(),
            row_start.data_ptr(), admitted.data_ptr(), slot.data_ptr(), src.data_ptr(),
            dst.data_ptr(), rows.data_ptr(), n_append.data_ptr(), flags, _ptr(err))
    return {"page_table": page_table, "ctx_len": ctx_len_out, "row_start": row_start,
            "admitted": admitted, "slot": slot, "app_src": src, "app_dst": dst,
            "app_rows": rows, "n_append": n_append, "free_count": free_count_out}


# ---------------------------------------------------------------------------
# log probabilities of given tokens
# ---------------------------------------------------------------------------
def logprobs_workspace_size(n, vocab, top_k, dtype=BF16):
    lib = load()
    b = _SZ(0)
    _check(lib.d2f_token_logprobs_workspace_size(n, vocab, top_k, dtype, ctypes.byref(b)))
    return b.value


def logprobs_workspace(device, **kw):
    """A zero-filled workspace of the size logprobs_workspace_size(**kw) returns."""
    with torch.cuda.device(device):
        return torch.zeros(max(logprobs_workspace_size(**kw), 1), dtype=torch.uint8, device=device)


def token_logprobs(logits, tokens, *, logit_row=None, top_k=0, want_entropy=True, logprob=None,
                   entropy=None, top_id=None, top_logprob=None, workspace=None, err=None,
                   stream=None):
    """Log probability of tokens[r] (int32; < 0: no token, the row is not read) in each row's
    distribution, its entropy and its top_k alternatives (d2f_token_logprobs).

    logits may be a row-strided view ([rows, vocab] with stride(1) == 1). Returns
    dict(logprob [n], entropy [n] or None, top_id [n, top_k], top_logprob [n, top_k])."""
    if not logits.is_cuda or logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA tensor with unit stride along the vocabulary")
    n = tokens.shape[0]
    rows, vocab = logits.shape
    if logit_row is None and rows < n:
        raise ValueError("%d tokens for %d logit rows" % (n, rows))
    dt = _dtype_code(logits)
    device, f32, i32 = logits.device, torch.float32, torch.int32
    if tokens.device != device:
        raise ValueError("tokens is on %s, logits on %s" % (tokens.device, device))
    empty = _on(stream, torch.empty)
    if logprob is None:
        logprob = empty(n, dtype=f32, device=device)
    if entropy is None and want_entropy:
        entropy = empty(n, dtype=f32, device=device)
    if top_id is None:
        top_id = empty((n, top_k), dtype=i32, device=device)
    if top_logprob is None:
        top_logprob = empty((n, top_k), dtype=f32, device=device)
    if workspace is None:
        workspace = _on(stream, logprobs_workspace)(device, n=n, vocab=vocab, top_k=top_k,
                                                    dtype=dt)
    stride = logits.stride(0) if rows > 1 else max(logits.stride(0), vocab)
    dev = _device(("tokens", tokens, i32, (n,)), ("logit_row", logit_row, i32, (n,)),
                  ("logprob", logprob, f32, (n,)), ("entropy", entropy, f32, (n,)),
                  ("top_id", top_id, i32, (n, top_k)), ("top_logprob", top_logprob, f32, (n, top_k)),
                  ("workspace", workspace, workspace.dtype, None),
                  ("err", err, i32, None))
    _launch(load().d2f_token_logprobs, dev, stream, logits.data_ptr(), stride, dt, vocab, rows,
            _ptr(logit_row), tokens.data_ptr(), n, top_k, logprob.data_ptr(), _ptr(entropy),
            top_id.data_ptr(), top_logprob.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _ptr(err))
    return {"logprob": logprob, "entropy": entropy, "top_id": top_id, "top_logprob": top_logprob}
