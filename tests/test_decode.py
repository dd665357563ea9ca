"""The decoding operators' oracle and host side: pins of the oracle's
definitions, the scaled rotary frequencies, and the refusals of the C ABI and
of the binding. Nothing here reaches a kernel."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_context_sparse_segment_b200 as pbs
from long_context_sparse_segment_b200 import _lib
from long_context_sparse_segment_b200._lib import Cache, Rows
from oracle import decode_oracle as dec

FAKE = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 8)
TWO = ctypes.c_void_p((1 << 20) + 2)


def rows(**kw):
    return Rows(*(dict(dict(p=1 << 20, layer=0, batch=1024, head=128, row=512), **kw).values()))


def cache(**kw):
    f = dict(dict(layers=1, pages=64, hkv=2, page=16, d=64, seqs=4, width=8), **kw)
    return Cache(*f.values())


# --------------------------------------------------------------------- oracle
def test_oracle_rope_turns_by_relative_positions():
    """q(s) . k(t) depends on s - t only, and the transpose undoes the turn."""
    r = np.random.default_rng(0)
    f = pbs.rope_freqs(32)[0].numpy()
    for layout in ("half", "pairs"):
        q, k = r.normal(size=(1, 1, 1, 48)), r.normal(size=(1, 1, 1, 48))
        dot = lambda s, t: (dec.rope(q, np.array([[s]]), f, layout=layout)
                            * dec.rope(k, np.array([[t]]), f, layout=layout)).sum()
        assert abs(dot(7, 3) - dot(1004, 1000)) < 1e-10
        y = dec.rope(q, np.array([[9]]), f, 2.0, layout)
        assert np.allclose(dec.rope(y, np.array([[9]]), f, 0.5, layout, True), q)
        assert np.array_equal(y[..., 32:], q[..., 32:])


def test_oracle_tree_and_attention():
    see = dec.visible([-1, 0, 0, 2, -1], 5)
    assert [list(np.nonzero(x)[0]) for x in see] == [[0], [0, 1], [0, 2], [0, 2, 3], [4]]
    assert not dec.visible([-1, 0], 1)[:, 1].any()
    q, k, v = np.zeros((2, 4)), np.zeros((3, 4)), np.arange(12.0).reshape(3, 4)
    v[2] = np.nan
    o, lse, _ = dec.attend(q, k, v, 1, np.array([[True, False], [False, False]]), 1.0)
    assert np.allclose(o, [v[:2].mean(0), v[0]]) and np.allclose(lse, [math.log(2), 0])
    o, lse, _ = dec.attend(q[:1], k[:0], v[:0], 0, np.zeros((1, 0), bool), 1.0)
    assert (o == 0).all() and lse[0] == -np.inf


def test_oracle_books_share_and_copy_pages():
    b = dec.Books(3, 4, 8, 16)
    assert b.reserve([20, 0, 0]) == [(-1, -1)] * 3 and b.table[0][:3] == [0, 1, -1]
    b.lens[0] = 20
    b.fork([0, 0], [1, 2])
    assert b.refs[:3] == [3, 3, 0]
    # two of three holders write: both copy the open page; the first keeps it
    assert b.reserve([0, 33, 21]) == [(-1, -1), (1, 2), (1, 4)]
    assert b.table == [[0, 1, -1, -1], [0, 2, 3, -1], [0, 4, -1, -1]]
    assert b.refs == [3, 1, 1, 1, 1, 0, 0, 0]
    b.trim([0, -1, 16])
    assert b.refs == [2, 0, 1, 1, 0, 0, 0, 0] and b.lens == [0, 20, 16]
    assert b.compact() == [(3, 1)]
    assert b.table[1] == [0, 2, 1, -1]
    # all holders write: the last one keeps the page
    c = dec.Books(2, 2, 4, 16)
    c.reserve([5, 0])
    c.lens[0] = 5
    c.fork([0], [1])
    assert c.reserve([6, 6]) == [(0, 1), (-1, -1)] and c.refs == [1, 1, 0, 0]
    assert dec.Books(1, 9, 2, 16).reserve([48]) is None


# ---------------------------------------------------------------- frequencies
def test_rope_freqs_scalings():
    f, gain = pbs.rope_freqs(64, 10000.0)
    assert f.dtype == torch.float64 and gain == 1.0
    assert np.allclose(f.numpy(), [10000.0 ** (-i / 32) for i in range(32)], rtol=1e-14)
    lin, _ = pbs.rope_freqs(64, scaling=dict(type="linear", factor=4))
    assert torch.equal(lin, f / 4)
    ntk, _ = pbs.rope_freqs(64, scaling=dict(type="ntk", factor=8))
    assert ntk[0] == 1 and abs(float(ntk[-1] / f[-1]) - 1 / 8) < 1e-12
    ramp, _ = pbs.rope_freqs(64, scaling=dict(type="ramp", factor=8, original=8192))
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(ramp[turns >= 4], f[turns >= 4])
    assert torch.allclose(ramp[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and ((ramp < f) & (ramp > f / 8))[mid].all()
    yarn, gain = pbs.rope_freqs(64, scaling=dict(type="yarn", factor=16, original=4096))
    assert abs(gain - (0.1 * math.log(16) + 1)) < 1e-15
    assert yarn[0] == f[0] and abs(float(yarn[-1] / f[-1]) - 1 / 16) < 1e-12
    assert pbs.rope_freqs(0)[0].numel() == 0


@pytest.mark.parametrize("kw", [dict(rot=24), dict(rot=-16), dict(rot=64, base=0.0),
                                dict(rot=64, scaling=dict(type="linear", factor=0.5)),
                                dict(rot=64, scaling=dict(type="other", factor=2)),
                                dict(rot=64, base=1.0), dict(rot=64, scaling=dict(factor=2)),
                                dict(rot=64, scaling=dict(type="linear")),
                                dict(rot=64, scaling=dict(type="yarn", factor=2)),
                                dict(rot=64, scaling=dict(type="linear", factor=2, low=1)),
                                dict(rot=64, scaling=dict(type="ramp", factor=2, original=8,
                                                          low=4, high=4))])
def test_rope_freqs_refusals(kw):
    with pytest.raises(ValueError):
        pbs.rope_freqs(**kw)


# ------------------------------------------------------------------- refusals
def call_rope(q=None, qo=None, hq=4, k=None, ko=None, hkv=2, pos=FAKE, freq=FAKE, b=2, n=3, d=64,
              rot=64, layout=0, dtype=0):
    r = rows()
    return pbs.lib().pbs_rope(q or r, qo or r, hq, k or r, ko or r, hkv, pos, n, freq, 1.0, b, n, d,
                              rot, layout, 0, dtype, None)


@pytest.mark.parametrize("kw", [
    dict(d=72), dict(d=0), dict(d=2048), dict(rot=24), dict(rot=80), dict(rot=-16), dict(layout=2),
    dict(dtype=3), dict(b=-1), dict(n=-1), dict(hq=-1), dict(pos=None), dict(pos=TWO),
    dict(freq=None), dict(freq=ctypes.c_void_p((1 << 20) + 4)), dict(q=rows(p=(1 << 20) + 8)),
    dict(q=rows(p=0)), dict(qo=rows(row=516)), dict(k=rows(head=4)), dict(ko=rows(batch=12))])
def test_rope_refusals(kw):
    assert call_rope(**kw) == _lib.ERR_INVALID_ARG


def test_empty_calls_launch_nothing():
    lib, c, none = pbs.lib(), cache(), cache(seqs=0)
    assert call_rope(b=0) == 0 and call_rope(n=0) == 0 and call_rope(hq=0, hkv=0) == 0
    r = rows()
    assert lib.pbs_cache_reserve(*[None] * 6, none, None, 0, None) == 0
    assert lib.pbs_cache_append(r, r, 0, *[None] * 5, c, None) == 0
    assert lib.pbs_cache_copy(*[None] * 4, 0, c, None, 0, None) == 0
    assert lib.pbs_cache_fork(*[None] * 5, 0, c, None) == 0
    assert lib.pbs_cache_trim(*[None] * 4, none, None) == 0
    assert lib.pbs_cache_accept(*[None] * 7, 0, c, None) == 0
    assert lib.pbs_tree_mask(None, None, None, 0, 5, None) == 0
    assert lib.pbs_tree_attn(r, *[None] * 8, 4, 0, c, 0.0, 0, 0, None, 0, None) == 0
    assert lib.pbs_tree_attn(r, *[None] * 8, 4, 3, none, 0.0, 0, 0, None, 0, None) == 0


@pytest.mark.parametrize("kw", [dict(layers=0), dict(pages=0), dict(hkv=0), dict(page=0),
                                dict(d=0), dict(d=12), dict(seqs=-1), dict(width=0),
                                dict(seqs=1 << 16, width=1 << 16)])
def test_bad_caches_are_refused(kw):
    lib, c, r = pbs.lib(), cache(**kw), rows()
    bad = _lib.ERR_INVALID_ARG
    assert lib.pbs_cache_reserve(*[FAKE] * 6, c, FAKE, 1 << 30, None) == bad
    assert lib.pbs_cache_append(r, r, 1, *[FAKE] * 5, c, None) == bad
    assert lib.pbs_cache_copy(*[FAKE] * 4, 1, c, FAKE, 1 << 30, None) == bad
    assert lib.pbs_cache_fork(*[FAKE] * 5, 1, c, None) == bad
    assert lib.pbs_cache_trim(*[FAKE] * 4, c, None) == bad
    assert lib.pbs_cache_compact(*[FAKE] * 6, c, FAKE, 1 << 30, None) == bad
    assert lib.pbs_cache_accept(*[FAKE] * 7, 1, c, None) == bad
    assert lib.pbs_cache_workspace_bytes(c, _lib.CACHE_RESERVE, 0) == 0


def with_one(n, i, x):
    return [x if j == i else FAKE for j in range(n)]


def test_cache_pointers_and_workspaces():
    lib, c, r, bad = pbs.lib(), cache(), rows(), _lib.ERR_INVALID_ARG
    for i in range(6):
        for x in (None, TWO):
            assert lib.pbs_cache_reserve(*with_one(6, i, x), c, FAKE, 1 << 20, None) == bad
            assert lib.pbs_cache_compact(*with_one(6, i, x), c, FAKE, 1 << 20, None) == bad
            if i < 5:
                assert lib.pbs_cache_fork(*with_one(5, i, x), 1, c, None) == bad
            if i < 4:
                assert lib.pbs_cache_trim(*with_one(4, i, x), c, None) == bad
                assert lib.pbs_cache_copy(*with_one(4, i, x), 1, c, None, 0, None) == bad
                assert lib.pbs_cache_append(r, r, 1, *with_one(4, i, x), None, c, None) == bad
            if i < 4:
                assert lib.pbs_cache_accept(*with_one(4, i, x), FAKE, None, None, 1, c,
                                            None) == bad
    assert lib.pbs_cache_append(rows(row=4), r, 1, *[FAKE] * 4, None, c, None) == bad
    assert lib.pbs_cache_copy(ODD, *[FAKE] * 3, 1, c, None, 0, None) == bad
    need = lib.pbs_cache_workspace_bytes(c, _lib.CACHE_RESERVE, 0)
    assert need == 4 * (64 + 4)
    assert lib.pbs_cache_reserve(*[FAKE] * 6, c, FAKE, need - 1, None) == _lib.ERR_WORKSPACE
    need = lib.pbs_cache_workspace_bytes(c, _lib.CACHE_COMPACT, 0)
    assert lib.pbs_cache_compact(*[FAKE] * 6, c, FAKE, need - 1, None) == _lib.ERR_WORKSPACE
    assert lib.pbs_cache_workspace_bytes(c, _lib.CACHE_COPY, 512) == 0
    need = lib.pbs_cache_workspace_bytes(c, _lib.CACHE_COPY, 513)
    assert need == 4 * 64
    assert lib.pbs_cache_copy(*[FAKE] * 4, 513, c, None, need, None) == bad
    assert lib.pbs_cache_copy(*[FAKE] * 4, 513, c, FAKE, need - 1, None) == _lib.ERR_WORKSPACE


def call_tree(c, hq=4, tree=3, q=None, ptrs=None, dtype=0, ws=FAKE, ws_bytes=1 << 40):
    return pbs.lib().pbs_tree_attn(q or rows(), *(ptrs or [FAKE] * 8), hq, tree, c, 0.0, 0, dtype, ws,
                                   ws_bytes, None)


def test_tree_refusals():
    bad, no = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED
    for kw in (dict(hkv=0), dict(seqs=-1), dict(pages=0), dict(width=0), dict(page=0)):
        assert call_tree(cache(**kw)) == bad
    for kw in (dict(d=96), dict(page=8), dict(page=48), dict(page=512), dict(seqs=65536),
               dict(pages=1 << 27), dict(width=1 << 27)):
        assert call_tree(cache(**kw)) == no
        assert pbs.lib().pbs_tree_workspace_bytes(4, 3, cache(**kw)) == 0
    assert call_tree(cache(), hq=5) == bad and call_tree(cache(), tree=-1) == bad
    assert call_tree(cache(), tree=1025) == no
    assert call_tree(cache(), dtype=_lib.FP32) == bad
    assert call_tree(cache(), q=rows(head=4)) == bad
    for i in (0, 1, 2, 3, 6):  # k, v, table, start, out
        assert call_tree(cache(), ptrs=with_one(8, i, None)) == bad
    for i in range(8):
        assert call_tree(cache(), ptrs=with_one(8, i, TWO)) == bad
    assert call_tree(cache(), ws=None) == bad
    need = pbs.lib().pbs_tree_workspace_bytes(4, 3, cache())
    assert need > 0 and call_tree(cache(), ws_bytes=need - 1) == _lib.ERR_WORKSPACE
    lib = pbs.lib()
    assert lib.pbs_tree_mask(FAKE, FAKE, None, 1, 1025, None) == no
    assert lib.pbs_tree_mask(None, FAKE, None, 1, 5, None) == bad
    assert lib.pbs_tree_mask(FAKE, TWO, None, 1, 5, None) == bad


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    f = pbs.rope_freqs(64)[0]
    with pytest.raises(ValueError):
        pbs.rope(x, None, i[:3], f)
    with pytest.raises(ValueError):
        pbs.cache_copy(x, x, i, i)
    with pytest.raises(ValueError):
        pbs.cache_trim(torch.zeros(4, 2, dtype=torch.int32), i, i, i, 16)
    with pytest.raises(ValueError):
        pbs.tree_mask(torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        pbs.tree_attn(x, x, x, torch.zeros(1, 2, dtype=torch.int32), i[:1])
    with pytest.raises(TypeError):
        pbs.rope([1.0], None, i, f)
    for bad in ((x, [0], i), (x, i, i)):
        with pytest.raises((TypeError, ValueError)):
            pbs.cache_copy(x, *bad)
    with pytest.raises(ValueError):
        pbs.PagedCache(0, 16, 4, 2, 64, device="cpu")
    with pytest.raises(TypeError):
        pbs.PagedCache(1, 16, 4, 2, 64, dtype=torch.float32, device="cpu")


def test_rows_of_strided_tensors():
    from long_context_sparse_segment_b200.decode import _rows
    x = torch.zeros(2, 5, 6, 64, dtype=torch.bfloat16).transpose(1, 2)
    r = _rows(x, "x", written=True)
    assert (r.batch, r.head, r.row) == (5 * 6 * 64, 64, 6 * 64)
    # a stride that is never taken may be odd
    odd = torch.zeros(500, dtype=torch.bfloat16).as_strided((1, 1, 3, 64), (7, 3, 64, 1))
    assert (_rows(odd, "x").batch, _rows(odd, "x", True).head) == (0, 0)
    for bad in (x[..., ::2], x[..., 1:33], torch.zeros(1, 1, 3, 68, dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            _rows(bad, "x")
    with pytest.raises(ValueError):
        _rows(x[:, :1].expand(2, 6, 5, 64), "x", written=True)
