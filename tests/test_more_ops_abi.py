"""Refusals of the further operators of include/mk_ops.h: every bad argument
comes back as an error code before anything is launched.  Made-up addresses:
nothing here reaches a device."""
import ctypes

import pytest

import moe_decode_megakernel_gb300 as mk
from moe_decode_megakernel_gb300 import ops
from test_ops_abi import A, BAD_TOKENS, append_io, attn_io, built, kv, open_kv, tokens  # noqa: F401

ARG, OK = mk.MK_ERR_ARG, mk.MK_OK


# ------------------------------------------------------------ append with norms

def axes_of(values, n=32):
    return (ctypes.c_uint8 * n)(*(values * n)[:n])


def head_norm(**kw):
    h = dict(q_gain=20 * A, k_gain=21 * A, axis_positions=22 * A, pair_axis=axes_of([0, 1, 2]), n_axes=3, eps=1e-6)
    h.update(kw)
    if h["pair_axis"] is not None:
        h["pair_axis"] = ctypes.cast(h["pair_axis"], ctypes.c_void_p)
    return ops.MkHeadNorm(**h)


@pytest.mark.parametrize("bad", BAD_TOKENS)
def test_append_norm_refuses_batches(kv, bad):
    assert ops._lib().mk_kv_append_norm(kv, 0, tokens(**bad), append_io(), head_norm(), None, None) == ARG


@pytest.mark.parametrize("bad", [
    dict(k=None), dict(v=None), dict(q_out=None), dict(n_q=0), dict(dtype=2), dict(k=5 * A + 2), dict(q=4 * A + 8),
    dict(k_stride=120), dict(q_out_stride=128), dict(q_out=5 * A), dict(q_out=20 * A - 64), dict(q_out=21 * A),
    dict(q_out=22 * A - 1536)])
def test_append_norm_refuses_tokens(kv, bad):
    assert ops._lib().mk_kv_append_norm(kv, 0, tokens(), append_io(**bad), head_norm(), None, None) == ARG
    assert mk.last_error()


@pytest.mark.parametrize("bad", [
    dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(eps=1e-39), dict(eps=0.0),
    dict(eps=0.0, q_gain=None), dict(q_gain=20 * A + 4), dict(k_gain=21 * A + 8), dict(axis_positions=22 * A + 2),
    dict(n_axes=-1), dict(n_axes=9), dict(n_axes=0), dict(n_axes=2), dict(axis_positions=None), dict(pair_axis=None),
    dict(n_axes=0, axis_positions=None), dict(pair_axis=axes_of([0, 3]))])
def test_append_norm_refuses(kv, bad):
    assert ops._lib().mk_kv_append_norm(kv, 0, tokens(), append_io(), head_norm(**bad), None, None) == ARG
    assert mk.last_error()


def test_append_norm_null_and_nothing_to_do(kv):
    L = ops._lib()
    assert L.mk_kv_append_norm(None, 0, tokens(), append_io(), head_norm(), None, None) == ARG
    assert L.mk_kv_append_norm(kv, 0, tokens(), append_io(), None, None, None) == ARG
    assert L.mk_kv_append_norm(kv, 2, tokens(), append_io(), head_norm(), None, None) == ARG
    assert L.mk_kv_append_norm(kv, 0, tokens(n_tokens=0), append_io(k=None), head_norm(), None, None) == OK
    assert L.mk_kv_append_norm(kv, 0, tokens(batch=0, cu_seqlens=None), append_io(), head_norm(), None, None) == OK


# ------------------------------------------------------------ accumulated attention weight

def mass_io(**kw):
    io = dict(q=4 * A, lse=5 * A, mass=7 * A, tree_mask=6 * A, q_stride=256, mass_stride=64, n_q=4, mask_words=1, window=0,
              scale=0.0, decay=1.0)
    io.update(kw)
    return ops.MkMassIo(**io)


@pytest.mark.parametrize("bad", BAD_TOKENS)
def test_mass_refuses_batches(kv, bad):
    assert ops._lib().mk_attn_mass(kv, 0, tokens(**bad), mass_io(), None, None) == ARG


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(lse=None), dict(mass=None), dict(n_q=0), dict(n_q=1), dict(n_q=3), dict(n_q=-2), dict(n_q=1 << 17),
    dict(q=4 * A + 8), dict(q_stride=248), dict(q_stride=260), dict(q_stride=1 << 39), dict(q_stride=1 << 62), dict(lse=5 * A + 2),
    dict(mass=7 * A + 1), dict(tree_mask=6 * A + 4), dict(mask_words=0), dict(tree_mask=None), dict(window=-1),
    dict(scale=-1.0), dict(scale=float("nan")), dict(scale=3e38), dict(decay=-0.5), dict(decay=1.5),
    dict(decay=float("nan")), dict(mass_stride=0), dict(mass_stride=1 << 60), dict(mass=4 * A + 64), dict(mass=5 * A),
    dict(mass=6 * A - 512), dict(mass=A), dict(mass=2 * A), dict(mass=3 * A), dict(mass=1 << 40), dict(mass=1 << 41)])
def test_mass_refuses(kv, bad):
    assert ops._lib().mk_attn_mass(kv, 0, tokens(), mass_io(**bad), None, None) == ARG
    assert mk.last_error()


def test_mass_null_and_nothing_to_do(kv):
    L = ops._lib()
    assert L.mk_attn_mass(None, 0, tokens(), mass_io(), None, None) == ARG
    assert L.mk_attn_mass(kv, 0, tokens(), None, None, None) == ARG
    assert L.mk_attn_mass(kv, -1, tokens(), mass_io(), None, None) == ARG
    assert L.mk_attn_mass(kv, 0, tokens(), mass_io(mass=8 * A), 8 * A, None) == ARG  # over the status record
    assert L.mk_attn_mass(kv, 0, tokens(n_tokens=0), mass_io(q=None), None, None) == OK
    assert L.mk_attn_mass(kv, 0, tokens(batch=0, cu_seqlens=None), mass_io(), None, None) == OK


# ------------------------------------------------------------ eviction

def evict(kv, batch=2, lens=A, tables=2 * A, out_tables=3 * A, max_pages=4, status=None, **kw):
    io = dict(keep=4 * A, mass=5 * A, mass_out=6 * A, kept=7 * A, new_lens=8 * A, mass_stride=64, max_keep=32, sinks=4,
              recent=8)
    io.update(kw)
    return ops._lib().mk_kv_evict(kv, batch, lens, tables, out_tables, max_pages, ops.MkEvictIo(**io), status, None)


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(max_pages=0), dict(max_pages=(1 << 26) + 1), dict(max_keep=-1), dict(sinks=-1), dict(recent=-1),
    dict(sinks=25), dict(sinks=2**31 - 1, recent=2**31 - 1), dict(lens=None), dict(tables=None), dict(keep=None),
    dict(mass=None), dict(kept=None), dict(lens=A + 2), dict(tables=2 * A + 1), dict(out_tables=3 * A + 2), dict(keep=4 * A + 1),
    dict(mass=5 * A + 2), dict(mass_out=6 * A + 2), dict(kept=7 * A + 2), dict(new_lens=8 * A + 2), dict(status=9 * A + 2),
    dict(mass_stride=0), dict(mass_stride=1 << 60), dict(batch=1 << 25), dict(mass_out=5 * A + 64), dict(mass_out=A),
    dict(kept=5 * A), dict(kept=6 * A + 256), dict(kept=3 * A), dict(kept=1 << 40), dict(mass_out=1 << 41), dict(new_lens=A),
    dict(new_lens=4 * A), dict(new_lens=7 * A + 4), dict(new_lens=5 * A), dict(new_lens=6 * A), dict(new_lens=9 * A, status=9 * A)])
def test_evict_refuses(kv, bad):
    assert evict(kv, **bad) == ARG
    assert mk.last_error()


def test_evict_null_and_nothing_to_do(kv):
    L = ops._lib()
    assert L.mk_kv_evict(None, 1, A, A, None, 1, ops.MkEvictIo(), None, None) == ARG
    assert L.mk_kv_evict(kv, 1, A, A, None, 1, None, None, None) == ARG
    assert evict(kv, batch=0, lens=None, tables=None) == OK


# ------------------------------------------------------------ shared prefixes

def prefix_of(**kw):
    p = dict(n_groups=1, group_seqs=20 * A, prefix_lens=21 * A)
    p.update(kw)
    return ops.MkPrefix(**p)


def prefix_attn(kv, tok=None, io=None, prefix=None, layer=0, ws=16 * A, size=1 << 40, status=None):
    return ops._lib().mk_prefix_attn(kv, layer, tok or tokens(), io or attn_io(), prefix or prefix_of(), ws, size, status, None)


@pytest.mark.parametrize("bad", BAD_TOKENS)
def test_prefix_refuses_batches(kv, bad):
    assert prefix_attn(kv, tokens(**bad)) == ARG


@pytest.mark.parametrize("bad", [
    dict(n_groups=-1), dict(n_groups=3), dict(group_seqs=None), dict(prefix_lens=None), dict(group_seqs=20 * A + 2),
    dict(prefix_lens=21 * A + 1), dict(group_seqs=5 * A + 16), dict(prefix_lens=5 * A), dict(group_seqs=16 * A + 64),
    dict(prefix_lens=17 * A)])
def test_prefix_refuses_groups(kv, bad):
    assert prefix_attn(kv, prefix=prefix_of(**bad)) == ARG
    assert mk.last_error()


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(out=None), dict(n_q=3), dict(q=4 * A + 8), dict(out=4 * A), dict(mask_words=0), dict(window=-1),
    dict(scale=-1.0), dict(lse=5 * A + 64), dict(lse=20 * A)])
def test_prefix_refuses(kv, bad):
    assert prefix_attn(kv, io=attn_io(**bad)) == ARG
    assert mk.last_error()


def test_prefix_null_and_nothing_to_do(kv):
    L = ops._lib()
    assert prefix_attn(None) == ARG and prefix_attn(kv, layer=2) == ARG
    assert prefix_attn(kv, ws=None) == ARG and prefix_attn(kv, ws=16 * A + 8) == ARG
    assert L.mk_prefix_attn(kv, 0, None, attn_io(), prefix_of(), 16 * A, 1 << 40, None, None) == ARG
    assert L.mk_prefix_attn(kv, 0, tokens(), None, prefix_of(), 16 * A, 1 << 40, None, None) == ARG
    assert L.mk_prefix_attn(kv, 0, tokens(), attn_io(), None, 16 * A, 1 << 40, None, None) == ARG
    assert prefix_attn(kv, tokens(n_tokens=0), attn_io(q=None)) == OK
    assert prefix_attn(kv, tokens(batch=0, cu_seqlens=None), prefix=prefix_of(n_groups=0, group_seqs=None, prefix_lens=None)) == OK
    assert L.mk_prefix_attn_workspace_bytes(None, 1, 1, 1) == 0
    for shape in ((-1, 4, 1), (1, 3, 1), (1, 0, 1), (1, 4, -1), (1, 1 << 17, 1)):
        assert L.mk_prefix_attn_workspace_bytes(kv, *shape) == 0


# ------------------------------------------------------------ the binding

def refused(f, *args, **kw):
    """Whether f refuses for another reason than that the tensors are on no CUDA device, which every call here ends with."""
    with pytest.raises(mk.MkError) as e:
        f(*args, **kw)
    assert e.value.code == ARG
    return "a CUDA device is wanted" not in str(e.value)


def test_binding_refuses():
    import torch

    class Fake:
        device, n_layers, n_kv, head_dim, handle = torch.device("cpu"), 2, 2, 64, None
    c, bf, w = Fake(), torch.bfloat16, torch.zeros(64, dtype=torch.uint8)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q, k = torch.zeros(4, 4, 64, dtype=bf), torch.zeros(4, 2, 64, dtype=bf)
    batch = dict(cu_seqlens=i(3), cache_lens=i(2), block_tables=i(2, 4))
    wide = torch.zeros(1, dtype=torch.int32).expand(1 << 33).unflatten(0, (2, 1 << 32))  # no memory behind it
    ops._lib()

    good = dict(k=k, v=k.clone(), q=q, q_out=torch.empty_like(q), eps=1e-6, q_gain=torch.ones(64), k_gain=torch.ones(64),
                axis_positions=i(3, 4), pair_axis=[0, 1, 2, 0] * 8, **batch)
    assert not refused(mk.kv_append_norm, c, 0, **good)
    assert not refused(mk.kv_append_norm, c, 0, **{**good, "pair_axis": bytes(32), "q_gain": None})
    for bad in (dict(k=k.double()), dict(v=k.float()), dict(q=None), dict(positions=i(3)), dict(block_tables=wide), dict(eps=-1.0),
                dict(eps=1e-50), dict(eps=float("nan")), dict(eps=float("inf")), dict(q_gain=torch.ones(32)),
                dict(k_gain=torch.ones(64, dtype=bf)), dict(axis_positions=None), dict(pair_axis=None), dict(axis_positions=i(4)),
                dict(axis_positions=i(3, 5)), dict(axis_positions=i(3, 4).long()), dict(axis_positions=i(2, 4)),
                dict(axis_positions=i(0, 4)), dict(pair_axis=[0] * 31), dict(pair_axis=[0] * 31 + [3]), dict(pair_axis=[-1] * 32),
                dict(pair_axis=[256] * 32), dict(pair_axis=[0.5] * 32), dict(status=i(7))):
        assert refused(mk.kv_append_norm, c, 0, **{**good, **bad}), bad
    assert refused(mk.kv_append_norm, c, 1 << 32, **good)

    good = dict(q=q, out=torch.empty_like(q), group_seqs=i(3), prefix_lens=i(2), workspace=w, **batch)
    assert not refused(mk.prefix_attn, c, 0, **good)
    for bad in (dict(q=q.float()), dict(out=q[:2]), dict(tree_mask=i(4, 1)), dict(lse=torch.zeros(4, 2)), dict(scale=0.0),
                dict(window=1 << 32), dict(workspace=w.float()), dict(group_seqs=i(2)), dict(group_seqs=i(3).long()),
                dict(prefix_lens=i(3)), dict(prefix_lens=i(2).long()), dict(prefix_lens=torch.tensor(0)), dict(block_tables=wide)):
        assert refused(mk.prefix_attn, c, 0, **{**good, **bad}), bad

    good = dict(q=q, lse=torch.zeros(4, 4), mass=torch.zeros(2, 2, 9), **batch)
    assert not refused(mk.attn_mass, c, 0, **good)
    for bad in (dict(q=q.float()), dict(q=q[..., 0]), dict(lse=torch.zeros(4, 2)), dict(lse=torch.zeros(4, 4, dtype=bf)),
                dict(mass=torch.zeros(2, 4, 9)), dict(mass=torch.zeros(3, 2, 9)), dict(mass=torch.zeros(2, 2, 9).double()),
                dict(mass=torch.zeros(2, 9, 2).transpose(1, 2)), dict(mass=torch.zeros(4, 9)), dict(tree_mask=i(4, 1)),
                dict(tree_mask=torch.zeros(4, 0, dtype=torch.int64)), dict(window=1 << 31), dict(scale=-1.0), dict(positions=i(5)),
                dict(cache_lens=torch.tensor(0, dtype=torch.int32))):
        assert refused(mk.attn_mass, c, 0, **{**good, **bad}), bad

    m = torch.zeros(2, 3, 2, 9)
    good = dict(lens=i(3), keep=i(3), mass=m, kept=i(2, 3, 2, 5), block_tables=i(3, 4), out_tables=i(3, 4), mass_out=m.clone(),
                new_lens=i(3))
    assert not refused(mk.kv_evict, c, **good)
    for bad in (dict(lens=i(2)), dict(lens=i(3, 1)), dict(keep=i(3).long()), dict(mass=m[0]), dict(mass=m[:1]), dict(mass=m.double()),
                dict(mass_out=torch.zeros(2, 3, 2, 8)), dict(kept=i(2, 3, 1, 5)), dict(kept=i(2, 3, 2, 5).long()), dict(kept=i(2, 3)),
                dict(block_tables=i(12)), dict(block_tables=wide), dict(out_tables=i(3, 5)), dict(new_lens=i(4)), dict(sinks=1 << 32),
                dict(recent=-(1 << 32)), dict(status=i(7))):
        assert refused(mk.kv_evict, c, **{**good, **bad}), bad

    for shape in (((1 << 32) + 1, 4, 1), (1, 1 << 32, 1), (1, 4, (1 << 32) + 1), (-1, 4, 1)):
        assert ops.prefix_attn_workspace_bytes(c, *shape) == 0


def pair_axes():
    import array

    import numpy as np
    import torch
    a = [0] * 12 + [1] * 10 + [2] * 10
    return {"list": a, "tuple": tuple(a), "bytes": bytes(a), "bytearray": bytearray(a), "array": array.array("i", a),
            "array of 64 bits": array.array("q", a), "int64": np.array(a), "int32": np.array(a, np.int32),
            "uint8": np.array(a, np.uint8), "strided": np.repeat(np.array(a, np.int16), 2)[::2], "tensor": torch.tensor(a),
            "tensor of bytes": torch.tensor(a, dtype=torch.uint8), "numbers": [np.int64(x) for x in a]}


@pytest.mark.parametrize("kind", pair_axes())
def test_binding_passes_axes_whatever_holds_them(kind, monkeypatch):
    """pair_axis are whole numbers, not the bytes that an array keeps them in."""
    import torch

    class Fake:
        device, n_layers, n_kv, head_dim, handle = torch.device("cpu"), 2, 2, 64, None
    got = []

    def call(fn, device, stream, *args):
        norm = next(x for x in args if isinstance(x, ops.MkHeadNorm))
        got.append((ctypes.string_at(norm.pair_axis, 32), norm.n_axes))

    ops._lib()
    monkeypatch.setattr(ops, "_call", call)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(4, 2, 64)
    mk.kv_append_norm(Fake(), 0, k, k.clone(), i(3), i(2), i(2, 4), axis_positions=i(3, 4), pair_axis=pair_axes()[kind])
    assert got == [(bytes([0] * 12 + [1] * 10 + [2] * 10), 3)]


def test_binding_refuses_axes_that_are_no_whole_numbers():
    import numpy as np
    import torch

    class Fake:
        device, n_layers, n_kv, head_dim, handle = torch.device("cpu"), 2, 2, 64, None
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(4, 2, 64)
    ops._lib()
    for bad in (np.zeros(32), np.zeros(32, np.float16), np.zeros((32, 2), np.int64), np.full(32, 3), np.full(32, -1),
                np.full(32, 256), torch.zeros(32), "0" * 32, 32):
        assert refused(mk.kv_append_norm, Fake(), 0, k, k.clone(), i(3), i(2), i(2, 4), axis_positions=i(3, 4), pair_axis=bad), bad
