"""Binding of the operators beside the decode step (include/mk_ops.h):
argument marshalling only, on torch-owned device memory.

    cache = KvCache(k_pool, v_pool, rope_base)
    kv_append(cache, layer, k, v, cu_seqlens, cache_lens, block_tables, q=q, q_out=q_out, positions=pos)
    tree_attn(cache, layer, q_out, out, cu_seqlens, cache_lens, block_tables, workspace,
              tree_mask=mask, positions=pos, window=4096)
    kv_commit(cache, cache_lens, path, path_lens, block_tables, new_lens=new_lens)
    beam_select(logits, scores, out_scores, out_parents, out_tokens, workspace)
    beam_reorder(cache, lens, parents, tables_in, tables_out)

Every call is asynchronous on `stream` (a torch stream; the current one of the
tensors' device if None).  A tensor of the wrong type, shape, layout or device
raises MkError (MK_ERR_ARG) before anything is launched; `status` is an int32
[8] tensor, zeroed by the caller, read by check_status.
"""
from __future__ import annotations

import ctypes

from . import MK_ERR_ARG, MkError, _check, last_error, lib

MK_BF16, MK_F32 = 0, 1


class MkKvConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("n_layers", "n_kv", "page_size", "head_dim")] + \
               [("num_pages", ctypes.c_int64), ("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("rope_base", ctypes.c_double)]


class MkTokens(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "n_tokens", "max_pages")] + \
               [(n, ctypes.c_void_p) for n in ("cu_seqlens", "cache_lens", "block_tables", "positions")]


class MkAppendIo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "q_out")] + \
               [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride", "q_out_stride")] + \
               [("n_q", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class MkAttnIo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "out", "lse", "tree_mask")] + \
               [("q_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)] + \
               [(n, ctypes.c_int32) for n in ("n_q", "mask_words", "window")] + [("scale", ctypes.c_float)]


_L = torch = None  # loaded by the first call: the package is imported without torch


def _lib():
    global _L, torch
    if _L is None:
        import torch
        L = lib()
        vp, i32, i64, sz, p = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER
        sig = {
            "mk_kv_open": (ctypes.c_int, [p(MkKvConfig), p(vp)]),
            "mk_kv_free": (None, [vp]),
            "mk_kv_append": (ctypes.c_int, [vp, i32, p(MkTokens), p(MkAppendIo), vp, vp]),
            "mk_tree_attn_workspace_bytes": (sz, [vp]),
            "mk_tree_attn": (ctypes.c_int, [vp, i32, p(MkTokens), p(MkAttnIo), vp, sz, vp, vp]),
            "mk_kv_commit": (ctypes.c_int, [vp, i32, vp, vp, vp, i32, vp, i32, vp, vp, vp]),
            "mk_beam_select_workspace_bytes": (sz, [i32, i32, i32, i32]),
            "mk_beam_select": (ctypes.c_int, [vp, i64, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]),
            "mk_beam_reorder": (ctypes.c_int, [vp, i32, i32, vp, vp, vp, vp, i32, vp, vp]),
            "mk_check_status": (ctypes.c_int, [vp, vp]),
        }
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _L = L
    return _L


def _bad(msg: str):
    raise MkError(MK_ERR_ARG, msg)


def _int32(v, name: str) -> int:
    """v as the int32 that the call takes (ctypes would cut it off)."""
    if not -1 << 31 <= v < 1 << 31:
        _bad(f"{name}: {v} does not fit 32 bits")
    return v


def _dims(t, name: str, n: int) -> None:
    if t.dim() != n:
        _bad(f"{name}: {n} dimensions are wanted, got {tuple(t.shape)}")


def _take(t, name: str, dtype, shape, device):
    """The address of a contiguous tensor of this type, shape and device (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        _bad(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on {device} is wanted, got "
             f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _rows(t, name: str, dtype, shape, device):
    """(address, elements from row to row) of a [tokens][heads][dim] tensor whose heads lie side by side."""
    if t.dtype is not dtype or t.shape != shape or t.device != device:
        _bad(f"{name}: a {dtype} tensor of shape {tuple(shape)} on {device} is wanted, got {t.dtype} "
             f"{tuple(t.shape)} on {t.device}")
    s = t.stride()
    if s[2] != 1 or (shape[1] > 1 and s[1] != shape[2]):
        _bad(f"{name}: the heads of a token must lie side by side, got strides {s}")
    return t.data_ptr(), (s[0] if shape[0] > 1 else shape[1] * shape[2])


def _call(fn, device, stream, *args) -> None:
    """fn(*args, raw stream) with the tensors' device current."""
    if device.type != "cuda":
        _bad(f"tensors on {device}: a CUDA device is wanted")
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        _bad(f"a stream of {stream.device} for tensors on {device}")
    else:
        raw = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, raw)
    if rc:
        raise MkError(rc, last_error())


class KvCache:
    """mk_kv_open: the paged pools bf16 [layers][pages][n_kv][page][head_dim]
    and the rotation's base.  Keeps the tensors alive."""

    def __init__(self, k_pool, v_pool, rope_base: float = 500000.0):
        _lib()
        for t in (k_pool, v_pool):
            if t.dim() != 5 or t.shape != k_pool.shape or not t.is_contiguous() or t.device != k_pool.device or \
                    t.dtype not in (torch.bfloat16, torch.uint16):
                _bad("pools: two contiguous bf16 tensors [layers][pages][n_kv][page][head_dim] on one device are wanted")
        self.k_pool, self.v_pool, self.device = k_pool, v_pool, k_pool.device
        self.n_layers, self.num_pages, self.n_kv, self.page_size, self.head_dim = k_pool.shape
        self.rope_base = float(rope_base)
        cfg = MkKvConfig(self.n_layers, self.n_kv, self.page_size, self.head_dim, self.num_pages,
                         k_pool.data_ptr(), v_pool.data_ptr(), self.rope_base)
        h = ctypes.c_void_p()
        _check(_lib().mk_kv_open(ctypes.byref(cfg), ctypes.byref(h)))
        self.handle = h

    def __del__(self):
        if getattr(self, "handle", None) and _L is not None:
            _L.mk_kv_free(self.handle)
            self.handle = None


def _tokens(cache, n_tokens, cu_seqlens, cache_lens, block_tables, positions):
    i32, dev = torch.int32, cache.device
    _dims(cache_lens, "cache_lens", 1)
    _dims(block_tables, "block_tables", 2)
    batch, max_pages = cache_lens.shape[0], block_tables.shape[1]
    return MkTokens(_int32(batch, "batch"), _int32(n_tokens, "tokens"), _int32(max_pages, "page columns"),
                    _take(cu_seqlens, "cu_seqlens", i32, (batch + 1,), dev),
                    _take(cache_lens, "cache_lens", i32, (batch,), dev),
                    _take(block_tables, "block_tables", i32, (batch, max_pages), dev),
                    _take(positions, "positions", i32, (n_tokens,), dev))


def _status(status, device):
    return _take(status, "status", torch.int32, (8,), device)


def kv_append(cache: KvCache, layer: int, k, v, cu_seqlens, cache_lens, block_tables, q=None, q_out=None,
              positions=None, status=None, stream=None) -> None:
    """mk_kv_append: k and v [tokens][n_kv][head_dim] (bf16 or fp32) into
    `layer` of the pools, k rotated; q [tokens][n_q][head_dim] of the same type
    rotated into q_out (bf16)."""
    _dims(k, "k", 3)
    dev, T, d = cache.device, k.shape[0], cache.head_dim
    if k.dtype not in (torch.bfloat16, torch.float32):
        _bad(f"k: bf16 or fp32 is wanted, got {k.dtype}")
    kp, ks = _rows(k, "k", k.dtype, (T, cache.n_kv, d), dev)
    vp, vs = _rows(v, "v", k.dtype, (T, cache.n_kv, d), dev)
    if (q is None) != (q_out is None):
        _bad("q and q_out go together")
    qp = qs = op = os_ = n_q = 0
    if q is not None:
        _dims(q, "q", 3)
        if q.shape[1] < 1:
            _bad(f"q: [tokens][heads][head_dim] is wanted, got {tuple(q.shape)}")
        n_q = q.shape[1]
        qp, qs = _rows(q, "q", k.dtype, (T, n_q, d), dev)
        op, os_ = _rows(q_out, "q_out", torch.bfloat16, (T, n_q, d), dev)
    io = MkAppendIo(qp, kp, vp, op, qs, ks, vs, os_, n_q, MK_F32 if k.dtype is torch.float32 else MK_BF16)
    tok = _tokens(cache, T, cu_seqlens, cache_lens, block_tables, positions)
    st = _status(status, dev)
    _call(_lib().mk_kv_append, dev, stream, cache.handle, _int32(layer, "layer"), tok, io, st)


def tree_attn_workspace_bytes(cache: KvCache) -> int:
    """mk_tree_attn_workspace_bytes on the cache's device."""
    with torch.cuda.device(cache.device):
        return int(_lib().mk_tree_attn_workspace_bytes(cache.handle))


def tree_attn(cache: KvCache, layer: int, q, out, cu_seqlens, cache_lens, block_tables, workspace, tree_mask=None,
              positions=None, window: int = 0, scale: float | None = None, lse=None, status=None,
              stream=None) -> None:
    """mk_tree_attn: q and out bf16 [tokens][n_q][head_dim]; tree_mask int64
    [tokens][words] (the bits of uint64 words) or None for a run of tokens;
    lse fp32 [tokens][n_q] or None; workspace uint8."""
    dev, bf = cache.device, torch.bfloat16
    _dims(q, "q", 3)
    T, n_q, _ = q.shape
    if scale is not None and not ctypes.c_float(scale).value > 0:  # as fp32: 0 would stand for the default
        _bad(f"scale must be positive, got {scale}")
    qp, qs = _rows(q, "q", bf, (T, n_q, cache.head_dim), dev)
    op, os_ = _rows(out, "out", bf, (T, n_q, cache.head_dim), dev)
    words = 0
    if tree_mask is not None:  # without words it would have no address, as if there were none
        _dims(tree_mask, "tree_mask", 2)
        words = _int32(tree_mask.shape[1], "mask words")
        if words < 1:
            _bad("tree_mask: one word per token at least is wanted")
    io = MkAttnIo(qp, op, _take(lse, "lse", torch.float32, (T, n_q), dev),
                  _take(tree_mask, "tree_mask", torch.int64, (T, words), dev), qs, os_, n_q, words,
                  _int32(window, "window"),
                  0.0 if scale is None else scale)
    tok = _tokens(cache, T, cu_seqlens, cache_lens, block_tables, positions)
    ws = _take(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    st = _status(status, dev)
    _call(_lib().mk_tree_attn, dev, stream, cache.handle, _int32(layer, "layer"), tok, io, ws, workspace.numel(), st)


def kv_commit(cache: KvCache, cache_lens, path, path_lens, block_tables, new_lens=None, status=None,
              stream=None) -> None:
    """mk_kv_commit: path int32 [batch][max_path], path_lens int32 [batch]."""
    dev, i32 = cache.device, torch.int32
    _dims(cache_lens, "cache_lens", 1)
    _dims(path, "path", 2)
    _dims(block_tables, "block_tables", 2)
    B, width = _int32(cache_lens.shape[0], "batch"), _int32(path.shape[1], "path width")
    pages = _int32(block_tables.shape[1], "page columns")
    args = (_take(cache_lens, "cache_lens", i32, (B,), dev), _take(path, "path", i32, (B, width), dev),
            _take(path_lens, "path_lens", i32, (B,), dev), width,
            _take(block_tables, "block_tables", i32, (B, pages), dev), pages,
            _take(new_lens, "new_lens", i32, (B,), dev), _status(status, dev))
    _call(_lib().mk_kv_commit, dev, stream, cache.handle, B, *args)


def beam_select_workspace_bytes(requests: int, beams: int, vocab: int, n_out: int) -> int:
    """mk_beam_select_workspace_bytes (0: a shape that beam_select refuses)."""
    shape = (requests, beams, vocab, n_out)
    if any(not 0 <= x < 1 << 31 for x in shape):  # ctypes would cut them off
        return 0
    return int(_lib().mk_beam_select_workspace_bytes(*shape))


def beam_select(logits, scores, out_scores, out_parents, out_tokens, workspace, finished=None, eos: int = -1,
                stream=None) -> None:
    """mk_beam_select: logits fp32 [requests * beams][vocab] (rows may be
    strided), scores fp32 [requests][beams], finished uint8 [requests][beams];
    outputs [requests][n_out] fp32, int32, int32."""
    _lib()
    dev, f32, i32 = logits.device, torch.float32, torch.int32
    if scores.dim() != 2 or logits.dim() != 2 or out_scores.dim() != 2:
        _bad("logits, scores and outputs have two dimensions")
    R, W = _int32(scores.shape[0], "requests"), _int32(scores.shape[1], "beams")
    V, n = _int32(logits.shape[1], "vocab"), _int32(out_scores.shape[1], "outputs")
    if logits.dtype is not f32 or logits.shape[0] != R * W or (V > 1 and logits.stride(1) != 1):
        _bad(f"logits: fp32 [{R * W}][vocab] with the vocabulary side by side is wanted, got {logits.dtype} "
             f"{tuple(logits.shape)} strides {logits.stride()}")
    args = (logits.stride(0) if R * W > 1 else V, _take(scores, "scores", f32, (R, W), dev),
            _take(finished, "finished", torch.uint8, (R, W), dev), _int32(eos, "eos"), R, W, V, n,
            _take(out_scores, "out_scores", f32, (R, n), dev), _take(out_parents, "out_parents", i32, (R, n), dev),
            _take(out_tokens, "out_tokens", i32, (R, n), dev),
            _take(workspace, "workspace", torch.uint8, (workspace.numel(),), dev), workspace.numel())
    _call(_lib().mk_beam_select, dev, stream, logits.data_ptr(), *args)


def beam_reorder(cache: KvCache, lens, parents, tables_in, tables_out, status=None, stream=None) -> None:
    """mk_beam_reorder: lens int32 [requests], parents int32
    [requests][beams], tables int32 [requests * beams][max_pages]."""
    dev, i32 = cache.device, torch.int32
    _dims(parents, "parents", 2)
    _dims(tables_in, "tables_in", 2)
    R, W = _int32(parents.shape[0], "requests"), _int32(parents.shape[1], "beams")
    pages = _int32(tables_in.shape[1], "page columns")
    args = (R, W, _take(lens, "lens", i32, (R,), dev), _take(parents, "parents", i32, (R, W), dev),
            _take(tables_in, "tables_in", i32, (R * W, pages), dev),
            _take(tables_out, "tables_out", i32, (R * W, pages), dev), pages, _status(status, dev))
    _call(_lib().mk_beam_reorder, dev, stream, cache.handle, *args)


def check_status(status, stream=None) -> None:
    """mk_check_status: waits for the stream; raises MkError if a call that
    was given `status` found a value out of range or gave up a wait."""
    _lib()
    st = _status(status, status.device)
    _call(_lib().mk_check_status, status.device, stream, st)
