"""Refusals of the operators beside the decode step (include/mk_ops.h): every
bad argument comes back as an error code before anything is launched.  Made-up
addresses: nothing here reaches a device."""
import ctypes
import os

import pytest

import moe_decode_megakernel_gb300 as mk
from moe_decode_megakernel_gb300 import ops

A = 1 << 20  # addresses far apart


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(mk.LIB_PATH):
        from moe_decode_megakernel_gb300.build import build
        build()


def open_kv(**kw):
    cfg = dict(n_layers=2, n_kv=2, page_size=16, head_dim=64, num_pages=8, k_pool=1 << 40, v_pool=1 << 41,
               rope_base=500000.0)
    cfg.update(kw)
    h = ctypes.c_void_p()
    rc = ops._lib().mk_kv_open(ops.MkKvConfig(**cfg), ctypes.byref(h))
    return rc, h


@pytest.fixture(scope="module")
def kv():
    rc, h = open_kv()
    assert rc == mk.MK_OK
    yield h
    ops._lib().mk_kv_free(h)


@pytest.mark.parametrize("bad,code", [
    (dict(n_layers=0), mk.MK_ERR_ARG), (dict(n_kv=0), mk.MK_ERR_ARG), (dict(num_pages=0), mk.MK_ERR_ARG),
    (dict(head_dim=96), mk.MK_ERR_UNSUPPORTED), (dict(page_size=8), mk.MK_ERR_UNSUPPORTED),
    (dict(page_size=48), mk.MK_ERR_UNSUPPORTED), (dict(page_size=512), mk.MK_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 26), mk.MK_ERR_ARG), (dict(num_pages=1 << 62), mk.MK_ERR_ARG),
    (dict(k_pool=None), mk.MK_ERR_ARG), (dict(v_pool=(1 << 41) + 8), mk.MK_ERR_ARG),
    (dict(rope_base=1.0), mk.MK_ERR_ARG), (dict(rope_base=float("nan")), mk.MK_ERR_ARG),
    (dict(rope_base=float("inf")), mk.MK_ERR_ARG)])
def test_open_refuses(bad, code):
    rc, h = open_kv(**bad)
    assert rc == code and not h.value and mk.last_error()


def test_open_refuses_null():
    assert ops._lib().mk_kv_open(None, None) == mk.MK_ERR_ARG
    ops._lib().mk_kv_free(None)


def tokens(**kw):
    t = dict(batch=2, n_tokens=4, max_pages=4, cu_seqlens=A, cache_lens=2 * A, block_tables=3 * A, positions=None)
    t.update(kw)
    return ops.MkTokens(**t)


BAD_TOKENS = [dict(batch=-1), dict(n_tokens=-1), dict(max_pages=0), dict(max_pages=(1 << 26) + 1), dict(cu_seqlens=None),
              dict(cache_lens=None), dict(block_tables=None), dict(cu_seqlens=A + 2), dict(cache_lens=2 * A + 1),
              dict(block_tables=3 * A + 3), dict(positions=A + 1)]


def append_io(**kw):
    io = dict(q=4 * A, k=5 * A, v=6 * A, q_out=7 * A, q_stride=256, k_stride=128, v_stride=128, q_out_stride=256, n_q=4,
              dtype=ops.MK_BF16)
    io.update(kw)
    return ops.MkAppendIo(**io)


@pytest.mark.parametrize("bad", BAD_TOKENS)
def test_append_refuses_batches(kv, bad):
    assert ops._lib().mk_kv_append(kv, 0, tokens(**bad), append_io(), None, None) == mk.MK_ERR_ARG
    assert mk.last_error()


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(q_out=None), dict(n_q=0), dict(n_q=-1), dict(dtype=2), dict(k=5 * A + 2),
    dict(q=4 * A + 8), dict(q_out=7 * A + 4), dict(k_stride=120), dict(v_stride=132), dict(q_stride=252),
    dict(q_out_stride=128), dict(q_out=4 * A + 16), dict(q_out=5 * A), dict(q_out=6 * A - 64),
    # in place, with k among q's columns
    dict(q=4 * A, q_out=4 * A, q_stride=512, q_out_stride=512, k=4 * A + 256, k_stride=512),
    # in place, the types differ
    dict(q=4 * A, q_out=4 * A, dtype=ops.MK_F32)])
def test_append_refuses(kv, bad):
    assert ops._lib().mk_kv_append(kv, 0, tokens(), append_io(**bad), None, None) == mk.MK_ERR_ARG
    assert mk.last_error()


@pytest.mark.parametrize("layer", [-1, 2])
def test_layers_outside_the_pools(kv, layer):
    assert ops._lib().mk_kv_append(kv, layer, tokens(), append_io(), None, None) == mk.MK_ERR_ARG
    assert ops._lib().mk_tree_attn(kv, layer, tokens(), attn_io(), 16 * A, 1 << 40, None, None) == mk.MK_ERR_ARG


def test_null_handles():
    L = ops._lib()
    assert L.mk_kv_append(None, 0, tokens(), append_io(), None, None) == mk.MK_ERR_ARG
    assert L.mk_tree_attn(None, 0, tokens(), attn_io(), 16 * A, 1 << 40, None, None) == mk.MK_ERR_ARG
    assert L.mk_kv_commit(None, 1, A, A, A, 1, A, 1, None, None, None) == mk.MK_ERR_ARG
    assert L.mk_beam_reorder(None, 1, 2, A, A, A, 2 * A, 1, None, None) == mk.MK_ERR_ARG
    assert L.mk_tree_attn_workspace_bytes(None) == 0
    assert L.mk_check_status(None, None) == mk.MK_ERR_ARG


def test_nothing_to_do(kv):
    L = ops._lib()
    assert L.mk_kv_append(kv, 0, tokens(n_tokens=0), append_io(), None, None) == mk.MK_OK
    assert L.mk_kv_append(kv, 0, tokens(n_tokens=0), append_io(k=None, v=None, q=None), None, None) == mk.MK_OK
    assert L.mk_tree_attn(kv, 0, tokens(n_tokens=0), attn_io(q=None, out=None), None, 0, None, None) == mk.MK_OK
    assert L.mk_kv_append(kv, 0, tokens(batch=0, cu_seqlens=None), append_io(), None, None) == mk.MK_OK
    assert L.mk_tree_attn(kv, 0, tokens(n_tokens=0), attn_io(), 16 * A, 1 << 40, None, None) == mk.MK_OK
    assert L.mk_kv_commit(kv, 0, None, None, None, 0, None, 1, None, None, None) == mk.MK_OK
    assert L.mk_beam_reorder(kv, 0, 4, None, None, None, None, 1, None, None) == mk.MK_OK
    assert L.mk_beam_select(None, 10, None, None, -1, 0, 1, 10, 1, None, None, None, None, 0, None) == mk.MK_OK


def attn_io(**kw):
    io = dict(q=4 * A, out=5 * A, lse=None, tree_mask=6 * A, q_stride=256, out_stride=256, n_q=4, mask_words=1, window=0,
              scale=0.0)
    io.update(kw)
    return ops.MkAttnIo(**io)


@pytest.mark.parametrize("bad", BAD_TOKENS)
def test_attn_refuses_batches(kv, bad):
    assert ops._lib().mk_tree_attn(kv, 0, tokens(**bad), attn_io(), 16 * A, 1 << 40, None, None) == mk.MK_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(out=None), dict(n_q=0), dict(n_q=1), dict(n_q=3), dict(n_q=-2), dict(q=4 * A + 8),
    dict(out=5 * A + 2), dict(q_stride=248), dict(q_stride=260), dict(out_stride=192), dict(out=4 * A), dict(out=4 * A + 512),
    dict(mask_words=0), dict(mask_words=-1), dict(tree_mask=None), dict(window=-1), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(lse=5 * A + 64), dict(lse=4 * A),
    dict(lse=16 * A + 256), dict(out=16 * A + 256), dict(tree_mask=6 * A + 4), dict(lse=7 * A + 2)])
def test_attn_refuses(kv, bad):
    assert ops._lib().mk_tree_attn(kv, 0, tokens(), attn_io(**bad), 16 * A, 1 << 40, None, None) == mk.MK_ERR_ARG
    assert mk.last_error()


@pytest.mark.parametrize("ws", [None, 16 * A + 8])
def test_attn_refuses_workspaces(kv, ws):
    assert ops._lib().mk_tree_attn(kv, 0, tokens(), attn_io(), ws, 1 << 40, None, None) == mk.MK_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=65536), dict(max_pages=(1 << 26) + 1), dict(max_path=-1), dict(max_pages=0), dict(cache_lens=None), dict(path=None),
    dict(path_lens=None), dict(block_tables=None), dict(new_lens=2 * A), dict(new_lens=2 * A + 4), dict(new_lens=4 * A),
    dict(new_lens=3 * A + 28), dict(new_lens=5 * A + 16), dict(new_lens=6 * A + 2), dict(path=3 * A + 1)])
def test_commit_refuses(kv, bad):
    a = dict(batch=2, cache_lens=2 * A, path=3 * A, path_lens=4 * A, max_path=4, block_tables=5 * A, max_pages=4, new_lens=6 * A)
    a.update(bad)
    assert ops._lib().mk_kv_commit(kv, *a.values(), None, None) == mk.MK_ERR_ARG
    assert mk.last_error()


@pytest.mark.parametrize("bad", [
    dict(requests=-1), dict(max_pages=(1 << 26) + 1), dict(beams=0), dict(beams=65), dict(lens=None), dict(parents=None), dict(tables_in=None),
    dict(tables_out=None), dict(max_pages=0), dict(tables_out=4 * A), dict(tables_out=4 * A + 100), dict(tables_out=3 * A),
    dict(tables_out=5 * A + 2), dict(lens=2 * A + 3)])
def test_reorder_refuses(kv, bad):
    a = dict(requests=2, beams=4, lens=2 * A, parents=3 * A, tables_in=4 * A, tables_out=5 * A, max_pages=4)
    a.update(bad)
    assert ops._lib().mk_beam_reorder(kv, *a.values(), None, None) == mk.MK_ERR_ARG
    assert mk.last_error()


SELECT = dict(logits=A, stride=1000, scores=8 * A, finished=9 * A, eos=2, requests=2, beams=4, vocab=1000, n_out=8,
              out_scores=10 * A, out_parents=11 * A, out_tokens=12 * A, workspace=13 * A, bytes=1 << 30)


@pytest.mark.parametrize("bad", [
    dict(requests=-1), dict(beams=0), dict(beams=65), dict(vocab=0), dict(n_out=0), dict(n_out=129),
    dict(beams=1, vocab=4, n_out=5), dict(vocab=1 << 30), dict(logits=None), dict(scores=None), dict(out_scores=None),
    dict(out_parents=None), dict(out_tokens=None), dict(stride=999), dict(eos=-1), dict(eos=1000), dict(workspace=None),
    dict(workspace=13 * A + 4), dict(bytes=100), dict(out_scores=8 * A), dict(out_scores=11 * A + 8),
    dict(out_tokens=A + 64), dict(out_parents=9 * A), dict(out_scores=13 * A + 4), dict(requests=20000),
    dict(logits=A + 2), dict(scores=8 * A + 1), dict(out_tokens=12 * A + 2), dict(workspace=8 * A - 4096, bytes=8192),
    dict(workspace=9 * A - 4096, bytes=8192), dict(workspace=A + 1024, bytes=8192)])
def test_select_refuses(bad):
    a = dict(SELECT)
    a.update(bad)
    assert ops._lib().mk_beam_select(*a.values(), None) == mk.MK_ERR_ARG
    assert mk.last_error()


@pytest.mark.parametrize("beams,vocab", [(1, (1 << 31) - 1), (1, (1 << 30) + 1), (4, (1 << 28) + 1), (64, 1 << 25)])
def test_select_refuses_vocabularies_beyond_its_counters(beams, vocab):
    a = dict(SELECT, beams=beams, vocab=vocab, stride=vocab, logits=1 << 44, bytes=1 << 40, requests=1, workspace=1 << 42)
    assert ops._lib().mk_beam_select(*a.values(), None) == mk.MK_ERR_ARG
    assert mk.beam_select_workspace_bytes(1, beams, vocab, 8) == 0
    assert mk.beam_select_workspace_bytes(1, beams, (1 << 30) // beams, 8) > 0


def test_select_workspace_sizes():
    f = mk.beam_select_workspace_bytes
    assert f(0, 65, 10, 1) == 0 and f(1, 1, 0, 1) == 0 and f(1, 1, 4, 5) == 0
    assert 0 < f(1, 4, 32768, 4) <= f(2, 4, 32768, 4)


def test_binding_refuses_tensors():
    import torch
    bf = dict(dtype=torch.bfloat16)
    with pytest.raises(mk.MkError):
        mk.KvCache(torch.empty(2, 8, 2, 16, 64), torch.empty(2, 8, 2, 16, 64))
    with pytest.raises(mk.MkError):
        mk.KvCache(torch.empty(2, 8, 2, 16, 64, **bf), torch.empty(2, 7, 2, 16, 64, **bf))
    with pytest.raises(mk.MkError):
        mk.KvCache(torch.empty(2, 8, 2, 64, 16, **bf).transpose(3, 4), torch.empty(2, 8, 2, 16, 64, **bf))
    pool = torch.zeros(2, 8, 2, 16, 64, **bf)
    c = mk.KvCache(pool, pool.clone())
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k, q = torch.zeros(4, 2, 64, **bf), torch.zeros(4, 4, 64, **bf)
    good = dict(k=k, v=k.clone(), cu_seqlens=i(3), cache_lens=i(2), block_tables=i(2, 4), q=q, q_out=torch.empty_like(q))
    for bad in (dict(k=k.double()), dict(v=k.float()), dict(v=k[:, :, :32]), dict(cu_seqlens=i(2)), dict(cu_seqlens=i(3).long()),
                dict(block_tables=i(4, 2).t()), dict(q_out=None), dict(q=None), dict(q=q[..., 0]), dict(positions=i(3)),
                dict(status=i(7)), dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)), dict(q_out=q.float()),
                {}):  # the last one: CPU tensors
        with pytest.raises(mk.MkError) as e:
            mk.kv_append(c, 0, **{**good, **bad})
        assert e.value.code == mk.MK_ERR_ARG
    w = torch.zeros(64, dtype=torch.uint8)
    good = dict(q=q, out=torch.empty_like(q), cu_seqlens=i(3), cache_lens=i(2), block_tables=i(2, 4), workspace=w,
                tree_mask=torch.zeros(4, 1, dtype=torch.int64))
    for bad in (dict(q=q.float()), dict(out=q[:2]), dict(tree_mask=i(4, 1)), dict(tree_mask=torch.zeros(3, 1, dtype=torch.int64)),
                dict(lse=torch.zeros(4, 2)), dict(scale=0.0), dict(scale=-1.0), dict(workspace=w.float()), {}):
        with pytest.raises(mk.MkError) as e:
            mk.tree_attn(c, 0, **{**good, **bad})
        assert e.value.code == mk.MK_ERR_ARG


def test_status_addresses(kv):
    L = ops._lib()
    assert L.mk_kv_append(kv, 0, tokens(), append_io(), 15 * A + 2, None) == mk.MK_ERR_ARG
    assert L.mk_tree_attn(kv, 0, tokens(), attn_io(), 16 * A, 1 << 40, 15 * A + 2, None) == mk.MK_ERR_ARG
    assert L.mk_kv_commit(kv, 2, 2 * A, 3 * A, 4 * A, 4, 5 * A, 4, 6 * A, 15 * A + 2, None) == mk.MK_ERR_ARG
    assert L.mk_beam_reorder(kv, 2, 4, 2 * A, 3 * A, 4 * A, 5 * A, 4, 15 * A + 2, None) == mk.MK_ERR_ARG
    assert L.mk_check_status(15 * A + 2, None) == mk.MK_ERR_ARG


def test_binding_refuses_what_ctypes_would_take():
    """Integers of more than 32 bits, a scale that is 0 as fp32, a mask without words (no address: a run),
    tensors of other dimensions; by a stand-in for the device, so that only the binding refuses."""
    import torch

    class Fake:
        device, n_layers, n_kv, head_dim, handle = torch.device("cpu"), 2, 2, 64, None
    bf, c, w = torch.bfloat16, Fake(), torch.zeros(64, dtype=torch.uint8)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q, k = torch.zeros(4, 4, 64, dtype=bf), torch.zeros(4, 2, 64, dtype=bf)
    batch = dict(cu_seqlens=i(3), cache_lens=i(2), block_tables=i(2, 4))
    ops._lib()

    def refused(f, *args, **kw):
        with pytest.raises(mk.MkError) as e:
            f(*args, **kw)
        assert e.value.code == mk.MK_ERR_ARG
        return "a CUDA device is wanted" not in str(e.value)  # the check that every call here ends with
    attn = dict(q=q, out=torch.empty_like(q), workspace=w, **batch)
    assert not refused(mk.tree_attn, c, 0, **attn)
    for bad in (dict(window=(1 << 32) + 5), dict(window=1 << 31), dict(scale=1e-50), dict(scale=float("nan")),
                dict(tree_mask=torch.zeros(4, 0, dtype=torch.int64)), dict(tree_mask=torch.tensor(0)),
                dict(cache_lens=torch.tensor(0, dtype=torch.int32)), dict(block_tables=i(8))):
        assert refused(mk.tree_attn, c, 0, **{**attn, **bad}), bad
    assert refused(mk.tree_attn, c, 1 << 32, **attn)
    append = dict(k=k, v=k.clone(), **batch)
    assert not refused(mk.kv_append, c, 0, **append)
    assert refused(mk.kv_append, c, 1 << 32, **append) and refused(mk.kv_append, c, 0, **{**append, "k": torch.tensor(1.0)})
    wide = torch.zeros(1, dtype=torch.int32).expand(1 << 33).unflatten(0, (2, 1 << 32))  # no memory behind it
    assert refused(mk.kv_append, c, 0, **{**append, "block_tables": wide})
    commit = (i(2), i(2, 3), i(2), i(2, 4))
    assert not refused(mk.kv_commit, c, *commit)
    for at, bad in ((0, torch.tensor(0)), (1, i(6)), (3, i(8)), (1, wide), (3, wide)):
        assert refused(mk.kv_commit, c, *commit[:at], bad, *commit[at + 1:])
    assert not refused(mk.beam_reorder, c, i(2), i(2, 4), i(8, 3), i(8, 3))
    assert refused(mk.beam_reorder, c, i(2), i(2, 4), torch.tensor(0), i(8, 3))
    select = dict(logits=torch.zeros(2, 8), scores=torch.zeros(1, 2), out_scores=torch.zeros(1, 4), out_parents=i(1, 4),
                  out_tokens=i(1, 4), workspace=w)
    assert not refused(mk.beam_select, **select)
    assert refused(mk.beam_select, **select, eos=1 << 32)
    assert refused(mk.beam_select, **{**select, "logits": torch.zeros(1).expand(1 << 33).unflatten(0, (2, 1 << 32))})


@pytest.mark.parametrize("requests,beams", [(65536, 1), (1024, 64), (1 << 20, 2), (16384, 4)])
def test_select_sizes_no_workspace_for_rows_that_it_refuses(requests, beams):
    a = dict(SELECT, requests=requests, beams=beams, vocab=16, stride=16, logits=1 << 44, scores=1 << 43, finished=None,
             out_scores=1 << 42, out_parents=3 << 41, out_tokens=5 << 40, bytes=1 << 36)
    assert ops._lib().mk_beam_select(*a.values(), None) == mk.MK_ERR_ARG
    assert mk.beam_select_workspace_bytes(requests, beams, 16, 8) == 0
    assert mk.beam_select_workspace_bytes(65535 // beams, beams, 16, 8) > 0


def test_binding_counts_requests_in_32_bits():
    """More requests, beams or outputs than the call's integers hold: refused, not cut off (tensors without memory)."""
    import torch
    n, i32 = (1 << 32) + 1, dict(dtype=torch.int32, device="meta")

    class Fake:
        device, n_layers, n_kv, head_dim, handle = torch.device("meta"), 2, 2, 64, None

    def f32(*s):
        return torch.empty(*s, device="meta")

    def refused(f, *args):
        with pytest.raises(mk.MkError) as e:
            f(*args)
        return "32 bits" in str(e.value)
    w = torch.empty(64, dtype=torch.uint8, device="meta")
    for R, W, out in ((n, 1, 1), (0, n, 1), (0, 1, n)):
        o = [torch.empty(R, out, **i32) for _ in range(2)]
        assert refused(mk.beam_select, f32(R * W, 4), f32(R, W), f32(R, out), *o, w), (R, W, out)
    for R, W in ((n, 1), (0, n)):
        t = torch.empty(R * W, 4, **i32)
        assert refused(mk.beam_reorder, Fake(), torch.empty(R, **i32), torch.empty(R, W, **i32), t, torch.empty_like(t))
    for shape in ((n, 1, 16, 4), (1, n, 16, 4), (1, 1, n, 4), (1, 4, 16, n), (-1, 1, 16, 4), (1 - (1 << 32), 1, 16, 4)):
        assert mk.beam_select_workspace_bytes(*shape) == 0


POOL_K, POOL_V, POOL = 1 << 40, 1 << 41, 2 * 8 * 2 * 16 * 64 * 2  # the fixture's pools


@pytest.mark.parametrize("at", [A + 8, 2 * A, 3 * A + 16, 8 * A, POOL_K + POOL - 16, POOL_V, 15 * A], ids=hex)
def test_outputs_over_the_batch_the_pools_or_the_record(kv, at):
    L, t = ops._lib(), tokens(positions=8 * A)
    at16 = at // 16 * 16
    assert L.mk_kv_append(kv, 0, t, append_io(q_out=at16), 15 * A, None) == mk.MK_ERR_ARG
    for io, ws in ((attn_io(out=at16), 32 * A), (attn_io(lse=at), 32 * A), (attn_io(), at16)):
        assert L.mk_tree_attn(kv, 0, t, io, ws, 4096, 15 * A, None) == mk.MK_ERR_ARG
        assert "overlaps the batch" in mk.last_error()
    assert L.mk_tree_attn(kv, 0, t, attn_io(lse=6 * A + 16), 32 * A, 4096, 15 * A, None) == mk.MK_ERR_ARG  # the mask
    assert "overlaps the batch" in mk.last_error()


@pytest.mark.parametrize("at", [POOL_K + POOL - 4, POOL_V, 15 * A + 28], ids=hex)
def test_lengths_and_tables_over_the_pools_or_the_record(kv, at):
    L = ops._lib()
    assert L.mk_kv_commit(kv, 2, 2 * A, 3 * A, 4 * A, 4, 5 * A, 4, at, 15 * A, None) == mk.MK_ERR_ARG
    assert L.mk_beam_reorder(kv, 2, 4, 2 * A, 3 * A, 4 * A, at, 4, 15 * A, None) == mk.MK_ERR_ARG


@pytest.mark.parametrize("stride", [1 << 62, (1 << 62) + 256, (1 << 63) - 8, 1 << 48])
def test_strides_whose_offsets_pass_64_bits(kv, stride):
    """Arrays longer than addresses reach: offsets would wrap, and the overlaps with them."""
    L = ops._lib()
    for bad in (dict(q_stride=stride), dict(k_stride=stride), dict(v_stride=stride), dict(q_out_stride=stride)):
        assert L.mk_kv_append(kv, 0, tokens(), append_io(**bad), None, None) == mk.MK_ERR_ARG, bad
        assert "stride" in mk.last_error()
    for bad in (dict(q_stride=stride), dict(out_stride=stride)):
        assert L.mk_tree_attn(kv, 0, tokens(), attn_io(**bad), 32 * A, 4096, None, None) == mk.MK_ERR_ARG
        assert "stride" in mk.last_error()
    assert L.mk_beam_select(*dict(SELECT, stride=stride).values(), None) == mk.MK_ERR_ARG
    assert "stride" in mk.last_error()


def test_open_refuses_pools_beyond_addresses():
    rc, h = open_kv(n_layers=(1 << 31) - 1, num_pages=1 << 25)
    assert rc == mk.MK_ERR_ARG and not h.value
