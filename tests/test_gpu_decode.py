"""The decoding operators on the GPU against the fp64 oracle: rotary
positions and their gradient, the paged cache's bookkeeping and moves, the
attention of drafted trees, and a run of them together behind a prefill."""
import itertools
import math
import random

import numpy as np
import pytest
import torch

import long_context_sparse_segment_b200 as pbs
from long_context_sparse_segment_b200 import _lib
from oracle import decode_oracle as dec
from pbs_testutil import f64

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def clean_status(dev):
    pbs.device_status()
    yield
    assert pbs.device_status() == 0


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def half_step(t):
    return torch.finfo(t).eps / 2


# ------------------------------------------------------------------------ rope
def rope_bound(x, y, gain, t, rot):
    """Half a step of the result, and of each product the angle's error: fp32
    keeps half a turn to 2^-25 of it (pi 2^-25 radians), sincospif is within
    2^-22, the two products and their sum round to 2^-24 each. 8 * 2^-23
    covers their sum; subnormal results are off by half the smallest step."""
    x = np.abs(x)
    pair = x.copy()
    if rot:
        pair[..., :rot] = x[..., :rot].max(-1, keepdims=True) * 2
    return half_step(t) * np.abs(y) + 8 * 2.0 ** -23 * gain * pair + float(
        torch.finfo(t).smallest_normal) * torch.finfo(t).eps


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 0, 64, 64), (2, 4, 2, 1, 128, 128),
                                   (3, 3, 1, 37, 128, 64), (1, 2, 2, 300, 80, 48),
                                   (2, 1, 1, 5, 64, 0), (1, 40, 8, 130, 16, 16)])
def test_rope(shape, layout, dtype, dev):
    b, hq, hkv, n, d, rot = shape
    n = n or 1
    g = torch.Generator().manual_seed(n)
    q = torch.randn(b, hq, n, d, generator=g).to(dtype)
    k = torch.randn(b, hkv, n, d, generator=g).to(dtype)
    pos = torch.randint(0, 1 << 20, (b, n), generator=g, dtype=torch.int32)
    f, _ = pbs.rope_freqs(rot, 500000.0)
    for transpose, gain in ((False, 1.0), (True, 1.25)):
        got = pbs.rope(q.to(dev), k.to(dev), pos.to(dev), f.to(dev), gain, layout, transpose)
        for x, y in zip((q, k), got):
            want = dec.rope(f64(x), pos.numpy(), f.numpy(), gain, layout, transpose)
            assert y.dtype == dtype and y.shape == x.shape
            assert (np.abs(f64(y) - want) <= rope_bound(f64(x), want, gain, dtype, rot)).all()
            assert torch.equal(y.cpu()[..., rot:], x[..., rot:])


def test_rope_strides_in_place_and_far_positions(dev):
    """Slices of one projection turned in place, at the ends of int32, with one
    row of positions for the batch; and without k."""
    b, n, hq, hkv, d = 2, 19, 6, 2, 64
    qkv = torch.randn(b, n, hq + 2 * hkv, d, device=dev).to(BF16)
    before = qkv.clone()
    q, k = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + hkv].transpose(1, 2)
    pos = torch.arange(n, dtype=torch.int32)
    pos[-1], pos[-2], pos[-3] = 2 ** 31 - 1, -2 ** 31, -1
    f = pbs.rope_freqs(d)[0]
    want = [dec.rope(f64(x), np.broadcast_to(pos.numpy(), (b, n)), f.numpy()) for x in (q, k)]
    x = [f64(q), f64(k)]
    only_q = pbs.rope(q, None, pos.to(dev), f.to(dev))
    out = pbs.rope(q, k, pos.to(dev), f.to(dev), q_out=q, k_out=k)
    assert out[0] is q and torch.equal(only_q, q)
    for a, y, w in zip(x, out, want):
        # the oracle's own angle, pos * f in fp64, is off by 2^-53 of itself
        slack = 2.0 ** 31 * 2.0 ** -52 * 2 * np.abs(a).max()
        assert (np.abs(f64(y) - w) <= rope_bound(a, w, 1.0, BF16, d) + slack).all()
    assert torch.equal(qkv[:, :, hq + hkv:], before[:, :, hq + hkv:])


def test_rope_gradient_against_differences(dev):
    """The map is linear: its differences along a direction, times a cotangent,
    equal the direction times the transposed map of the cotangent. In fp32
    each of the n products is off by 8 * 2^-23 of |v||g|."""
    shape = (2, 3, 11, 64)
    x, v, g = (torch.randn(shape, device=dev) for _ in range(3))
    pos, f = i32(np.arange(22).reshape(2, 11) * 991, dev), pbs.rope_freqs(32)[0].to(dev)
    for layout in ("half", "pairs"):
        up = lambda t: pbs.rope(t, None, pos, f, 1.5, layout)
        down = pbs.rope(g, None, pos, f, 1.5, layout, transpose=True)
        diff = (up(x + v).double() - up(x).double())
        a, c = (diff * g.double()).sum().item(), (v.double() * down.double()).sum().item()
        size = sum(float((t.abs() * g.abs()).sum()) for t in (x, v, x + v))
        assert abs(a - c) <= 8 * 2.0 ** -23 * 1.5 * 2 * 4 * size


def test_rope_refuses(dev):
    q = torch.zeros(2, 4, 3, 64, dtype=BF16, device=dev)
    f, pos = pbs.rope_freqs(64)[0].to(dev), torch.zeros(2, 3, dtype=torch.int32, device=dev)
    for bad in (lambda: pbs.rope(q, q.half(), pos, f), lambda: pbs.rope(q, q[:1], pos, f),
                lambda: pbs.rope(q, None, pos[:1], f), lambda: pbs.rope(q, None, pos.long(), f),
                lambda: pbs.rope(q, None, pos, f.float()), lambda: pbs.rope(q[..., :32], None, pos, f),
                lambda: pbs.rope(q, None, pos, f, layout="x"), lambda: pbs.rope(q[0], None, pos, f),
                lambda: pbs.rope(q.double(), None, pos, f), lambda: pbs.rope(q[..., ::2], None, pos, f[:16]),
                lambda: pbs.rope(q, None, pos, f, k_out=q), lambda: pbs.rope(q, None, pos, f.cpu()),
                lambda: pbs.rope(q, None, pos, f, q_out=q[:1].expand(2, 4, 3, 64)),
                lambda: pbs.rope(q[:1], None, pos[:1], f, q_out=q.view(-1)[64:64 + 768].view(1, 4, 3, 64))):
        with pytest.raises((ValueError, TypeError)):
            bad()
    assert pbs.rope(q[:0], None, pos[:0], f).shape == (0, 4, 3, 64)


# ----------------------------------------------------------------------- books
def same_books(b, table, refs, lens):
    assert table.tolist() == b.table and refs.tolist() == b.refs and lens.tolist() == b.lens


@pytest.mark.parametrize("seqs,width,pages,page", [(1, 1, 1, 1), (5, 4, 11, 16), (40, 9, 150, 7),
                                                   (70, 40, 3000, 16), (3, 70, 5000, 1)])
def test_books_follow_the_oracle(seqs, width, pages, page, dev):
    """Random reserves, forks, trims and compactions: every table, count and
    pair as the definition gives them, pools without room included."""
    r = random.Random(seqs * 1000 + pages)
    b = dec.Books(seqs, width, pages, page)
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=dev)
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    lens = torch.zeros(seqs, dtype=torch.int32, device=dev)
    k = torch.zeros(1, pages, 1, page, 8, dtype=BF16, device=dev)
    full = 0
    for _ in range(40):
        op = r.choice(["reserve", "reserve", "fork", "fork", "trim", "compact"])
        if op == "reserve":
            want = [min(width * page, n + r.choice([0, 0, 1, page, 2 * page])) if r.random() < 0.7
                    else 0 for n in b.lens]
            src, dst = pbs.cache_reserve(table, refs, lens, i32(want, dev), page)
            pairs = b.reserve(want)
            if pairs is None:
                full += 1
                assert pbs.device_status() == _lib.ERR_PAGES
                pairs = [(-1, -1)] * seqs
            else:
                b.lens = [max(n, w) for n, w in zip(b.lens, want)]
                lens.copy_(i32(b.lens, dev))
            assert list(zip(src.tolist(), dst.tolist())) == pairs
        elif op == "fork":
            empty = [s for s in range(seqs) if not b.held(s)]
            live = [s for s in range(seqs) if b.lens[s]]
            if not empty or not live:
                continue
            dst = r.sample(empty, r.randint(1, len(empty)))
            src = [r.choice(live) for _ in dst]
            b.fork(src, dst)
            pbs.cache_fork(table, refs, lens, i32(src + [-1], dev), i32(dst + [-1], dev), page)
        elif op == "trim":
            keep = [r.choice([-1, -1, 0, r.randint(0, n + 2)]) for n in b.lens]
            b.trim(keep)
            pbs.cache_trim(table, refs, lens, i32(keep, dev), page)
        else:
            moves = b.compact()
            src, dst = pbs.cache_compact(k, k.clone(), table, refs)
            moves += [(-1, -1)] * (pages - len(moves))
            assert list(zip(src.tolist(), dst.tolist())) == moves
        same_books(b, table, refs, lens)
        assert pbs.device_status() == 0


def test_reserve_in_a_large_pool(dev):
    """More pages than one pass of the plan ranks, sequences that need many."""
    pages, seqs, width = 70001, 300, 260
    refs = (torch.rand(pages, generator=torch.Generator().manual_seed(1)) < 0.5).to(torch.int32)
    free = torch.nonzero(refs == 0)[:, 0]
    want = torch.randint(0, width * 16, (seqs,), generator=torch.Generator().manual_seed(2))
    want[7], want[-1] = 0, width * 16
    need = -(-want // 16)
    short = int(need.sum()) > len(free)
    if short:
        want[:150], need[:150] = 0, 0
    table = torch.full((seqs, width), -1, dtype=torch.int32, device=dev)
    d_refs, lens = refs.to(dev), torch.zeros(seqs, dtype=torch.int32, device=dev)
    pbs.cache_reserve(table, d_refs, lens, want.to(dev, torch.int32), 16)
    at, exp = 0, torch.full((seqs, width), -1, dtype=torch.int32)
    for s, n in enumerate(need.tolist()):
        exp[s, :n] = free[at:at + n]
        at += n
    refs[free[:at]] = 1
    assert torch.equal(table.cpu(), exp) and torch.equal(d_refs.cpu(), refs)


def test_bad_books_are_reported_and_left(dev):
    """What points outside or contradicts itself changes nothing else."""
    page, c = 16, lambda *x: i32(list(x), dev)
    table = i32([[0, 1], [-1, -1], [-1, -1], [99, -1]], dev)
    refs, lens = c(1, 1, 0, 0), c(20, 0, 0, 16)
    t0, r0, l0 = table.clone(), refs.clone(), lens.clone()

    def refused(code=_lib.ERR_DEVICE_ASSERT):
        assert pbs.device_status() == code
        assert torch.equal(table, t0) and torch.equal(refs, r0) and torch.equal(lens, l0)

    for src, dst in (([0], [0]), ([0], [4]), ([-1], [1]), ([5], [1]), ([0], [3]), ([3], [1]),
                     ([1, 2], [2, 1])):
        pbs.cache_fork(table, refs, lens, c(*src), c(*dst), page)
        refused()
    # a second pair onto the same sequence: the first one counts
    pbs.cache_fork(table, refs, lens, c(0, 0), c(1, 1), page)
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
    assert table[1].tolist() == [0, 1] and refs.tolist() == [2, 2, 0, 0]
    pbs.cache_trim(table, refs, lens, c(-1, 0, -1, -1), page)
    refused(0)
    # want beyond the table; a negative length; too few pages
    src, dst = pbs.cache_reserve(table, refs, lens, c(33, 0, 0, 0), page)
    refused()
    assert src.tolist() == [-1] * 4
    pbs.cache_reserve(table, refs, c(-3, 0, 0, 16), c(4, 0, 0, 0), page)
    refused()
    pbs.cache_reserve(table, refs, lens, c(0, 32, 16, 0), page)
    refused(_lib.ERR_PAGES)
    pbs.cache_trim(table, refs, lens, c(-1, -1, -1, 0), page)  # page 99 does not exist
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
    assert refs.tolist() == [1, 1, 0, 0] and table[3].tolist() == [-1, -1]


# ----------------------------------------------------------------------- moves
def ids(shape, dev, dtype=BF16, seed=0):
    """Random 16-bit patterns, NaN and infinities among them: moves keep bits."""
    g = torch.Generator(dev).manual_seed(seed)
    x = torch.randint(-32768, 32768, shape, generator=g, device=dev, dtype=torch.int16)
    return x.view(dtype)


def bits(x):
    return x.view(torch.int16)


@pytest.mark.parametrize("layers,hkv,page,d,n", [(1, 1, 16, 8, 1), (2, 3, 5, 24, 7),
                                                 (3, 2, 64, 128, 40), (1, 1, 1, 64, 700),
                                                 (2, 8, 128, 128, 3)])
def test_copy(layers, hkv, page, d, n, dev):
    pages = 2 * n + 3
    k, v = (ids((layers, pages, hkv, page, d), dev, seed=s) for s in (1, 2))
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(n))
    src, dst = perm[:n].clone(), perm[n:2 * n].clone()
    src[1::5] = src[0]  # a source may be read twice
    want = [bits(x).clone() for x in (k, v)]
    for w in want:
        w[:, dst] = w[:, src]
    skip = torch.full((1,), -1)
    pbs.cache_copy(k, v, torch.cat([src, skip]).to(dev, torch.int32),
                   torch.cat([dst, skip]).to(dev, torch.int32))
    assert torch.equal(bits(k), want[0]) and torch.equal(bits(v), want[1])


@pytest.mark.parametrize("n", [6, 600])
def test_copy_refuses_pairs_that_meet(n, dev):
    """A repeated destination, a source that is written, a page outside, half a
    pair: reported, skipped, the sound pairs done. On one layer's 4-D pools."""
    pages = 2 * n
    k, v = (ids((pages, 2, 16, 64), dev, FP16, seed=s) for s in (3, 4))
    src, dst = torch.arange(n), torch.arange(n, 2 * n)
    dst[3] = dst[1]            # the second one onto page n + 1
    src[2], dst[4] = n + 5, -1  # page n + 5 is written by pair 5
    src[0] = pages
    want = bits(k).clone()
    sound = [i for i in range(n) if i not in (0, 2, 3, 4)]
    want[dst[sound]] = want[src[sound]]
    pbs.cache_copy(k, v, src.to(dev, torch.int32), dst.to(dev, torch.int32))
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
    assert torch.equal(bits(k), want)


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("hkv,page,d,n", [(1, 16, 64, 1), (3, 5, 24, 9), (2, 64, 128, 150)])
def test_append(layers, hkv, page, d, n, dev):
    """Rows of ragged batches at odd starts; every other row stays."""
    seqs, r = 4, random.Random(n)
    start = [0, page - 1, r.randint(0, 200), 3]
    count = [n, 0, r.randint(0, n), min(n, 2)]
    width = (max(start) + n) // page + 2
    pages = seqs * width + 1
    lead = () if layers is None else (layers,)
    k, v = (ids((*lead, pages, hkv, page, d), dev, seed=s) for s in (1, 2))
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(n))[:seqs * width]
    table = table.view(seqs, width)
    # strided: a slice of a fused projection
    qkv = ids((*lead, seqs, n, 2 * hkv, d), dev, seed=5)
    nk, nv = qkv[..., :hkv, :].transpose(-2, -3), qkv[..., hkv:, :].transpose(-2, -3)
    want = [bits(x).clone() for x in (k, v)]
    for s in range(seqs):
        for i in range(count[s]):
            t = start[s] + i
            at = (*([slice(None)] if lead else []), int(table[s, t // page]), slice(None), t % page)
            want[0][at] = bits(nk)[..., s, :, i, :]
            want[1][at] = bits(nv)[..., s, :, i, :]
    pbs.cache_append(nk, nv, k, v, table.to(dev, torch.int32), i32(start, dev), i32(count, dev))
    assert torch.equal(bits(k), want[0]) and torch.equal(bits(v), want[1])


def test_append_and_accept_refuse_pages_they_do_not_have(dev):
    k, v = (ids((4, 1, 16, 64), dev, seed=s) for s in (1, 2))
    k0, v0 = bits(k).clone(), bits(v).clone()
    new = ids((3, 1, 2, 64), dev, seed=3)
    table = i32([[0, -1], [4, 1], [3, 2]], dev)
    # no second page; a page outside; the last row behind the table
    pbs.cache_append(new, new, k, v, table, i32([15, 0, 31], dev))
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
    k0[0, 0, 15], v0[0, 0, 15] = bits(new)[0, 0, 0], bits(new)[0, 0, 0]
    k0[2, 0, 15], v0[2, 0, 15] = bits(new)[2, 0, 0], bits(new)[2, 0, 0]
    assert torch.equal(bits(k), k0) and torch.equal(bits(v), v0)
    for call in (lambda: pbs.cache_append(new, new, k, k, table, i32([0, 0, 0], dev)),
                 lambda: pbs.cache_accept(k, k, table, i32([0, 0, 0], dev), i32([[0]] * 3, dev))):
        with pytest.raises(pbs.PbsError):  # one pool for both
            call()
    lens = i32([7, 8, 9], dev)
    for start, path in (([14, 0, 31], [[1, 2], [0, 1], [1, 2]]),      # pages missing
                        ([0, 0, -1], [[1, 1], [1, 0], [0, 1]]),       # does not ascend; start < 0
                        ([0, 0, 0], [[-1, 1], [2, 3], [0, 32]])):     # before, a bad page, behind
        pbs.cache_accept(k, v, table, i32(start, dev), i32(path, dev)[:, :2].contiguous(),
                         lens=lens)
        assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
        assert torch.equal(bits(k), k0) and torch.equal(bits(v), v0)
        assert lens.tolist() == [7, 8, 9]


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("hkv,page,d,tree", [(1, 16, 8, 1), (3, 5, 24, 40), (8, 64, 128, 33),
                                             (2, 1, 64, 100)])
def test_accept(layers, hkv, page, d, tree, dev):
    """Rows move down over one another, in order, across pages."""
    seqs, r = 5, random.Random(tree)
    start = [0, 1, page, r.randint(0, 100), 2 * page - 1]
    count = [r.randint(0, tree) for _ in range(seqs)]
    count[0], count[2] = tree, 0
    path = [sorted(r.sample(range(tree), n)) + [-7] * (tree - n) for n in count]
    width = (max(start) + tree) // page + 1
    pages = seqs * width + 2
    lead = () if layers is None else (layers,)
    k, v = (ids((*lead, pages, hkv, page, d), dev, seed=s) for s in (1, 2))
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(tree))[:seqs * width]
    table = table.view(seqs, width)
    want = [bits(x).clone() for x in (k, v)]
    sl = (slice(None),) if lead else ()
    for w in want:
        for s in range(seqs):
            for i in range(count[s]):
                a, b = start[s] + path[s][i], start[s] + i
                w[(*sl, int(table[s, b // page]), slice(None), b % page)] = \
                    w[(*sl, int(table[s, a // page]), slice(None), a % page)].clone()
    lens = torch.zeros(seqs, dtype=torch.int32, device=dev)
    pbs.cache_accept(k, v, table.to(dev, torch.int32), i32(start, dev), i32(path, dev),
                     i32(count, dev), lens)
    assert torch.equal(bits(k), want[0]) and torch.equal(bits(v), want[1])
    assert lens.tolist() == [a + n for a, n in zip(start, count)]


def test_compact_moves_every_layer(dev):
    layers, pages, seqs, width = 3, 67, 4, 9
    k, v = (ids((layers, pages, 2, 16, 64), dev, seed=s) for s in (1, 2))
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(9))[:seqs * width]
    table = perm.view(seqs, width).clone()
    table[1, :4] = table[0, :4]
    table[2, 5:] = -1
    refs = torch.zeros(pages, dtype=torch.int32)
    for p in table.flatten().tolist():
        if p >= 0:
            refs[p] += 1
    n = int((refs > 0).sum())
    t, rf = table.to(dev, torch.int32), refs.to(dev)
    rows = [bits(x)[:, table.clamp(min=0)].clone() for x in (k, v)]
    pbs.cache_compact(k, v, t, rf)
    assert int(t.max()) < n and bool((rf[:n] > 0).all()) and not rf[n:].any()
    assert sorted(rf[:n].tolist()) == sorted(refs[refs > 0].tolist())
    assert torch.equal(t.cpu() < 0, table < 0)
    held = (table >= 0).to(dev)
    for x, w in zip((k, v), rows):
        assert torch.equal(bits(x)[:, t.clamp(min=0).long()][:, held], w[:, held])
    before = t.clone()
    src, _ = pbs.cache_compact(k, v, t, rf)  # nothing left to move
    assert torch.equal(t, before) and (src == -1).all()


# ------------------------------------------------------------------ tree masks
@pytest.mark.parametrize("tree", [1, 2, 31, 32, 33, 100, 1024])
def test_tree_mask(tree, dev):
    r = random.Random(tree)
    parents = [[-1 if i == 0 or r.random() < 0.1 else r.randrange(i) for i in range(tree)],
               list(range(-1, tree - 1)), [-1] * tree]
    mask, depth = pbs.tree_mask(i32(parents, dev))
    assert mask.shape == (3, tree, (tree + 31) // 32)
    on = (mask.cpu().numpy().view(np.uint32)[..., None] >> np.arange(32)) & 1
    for b in range(3):
        see = dec.visible(parents[b], tree)
        got = on[b].reshape(tree, -1)
        assert np.array_equal(got[:, :tree].astype(bool), see) and not got[:, tree:].any()
        assert depth[b].tolist() == (see.sum(1) - 1).tolist()


def test_tree_mask_reports_bad_parents(dev):
    mask, depth = pbs.tree_mask(i32([[-1, 1, 0, 7], [-2, 0, 1, 2]], dev))
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
    assert mask[..., 0].tolist() == [[1, 2, 5, 8], [1, 3, 7, 15]]
    assert depth.tolist() == [[0, 0, 1, 0], [0, 1, 2, 3]]


# ------------------------------------------------------------------- attention
class Tree:
    """A paged cache with drafts in it, junk wherever nothing was written."""

    def __init__(self, dev, dtype, d, page, hkv, start, count, tree, seed=0, junk=True):
        g = torch.Generator().manual_seed(seed)
        self.start, self.count, self.tree, self.page = start, count, tree, page
        self.len = [s + c for s, c in zip(start, count)]
        need = [-(-n // page) for n in self.len]
        width, pages = max(need + [1]) + 1, sum(need) + 3
        perm = torch.randperm(pages, generator=g).tolist()
        table = torch.full((len(start), width), -1, dtype=torch.int32)
        fill = float("nan") if junk else 0.0
        self.k, self.v = (torch.full((pages, hkv, page, d), fill) for _ in range(2))
        self.v[::2] = float("inf") if junk else 0.0
        self.rows = []
        for s, n in enumerate(self.len):
            for j in range(need[s]):
                table[s, j] = perm.pop()
            k, v = (torch.randn(hkv, n, d, generator=g).to(dtype).float() for _ in range(2))
            self.rows.append((k, v))
            for t in range(n):
                p, o = int(table[s, t // page]), t % page
                self.k[p, :, o], self.v[p, :, o] = k[:, t], v[:, t]
        self.k, self.v = self.k.to(dev, dtype), self.v.to(dev, dtype)
        self.table = table.to(dev)
        self.q = None

    def check(self, q, o, lse, see, sigma, dtype, wild=()):
        """Against the oracle. Logits: a sum of d products in fp32 (the tensor
        cores' sums may truncate: 2^-23 a step) of size at most |q||k|, then
        exponentials within 2^-21; P in 16 bits is off by half a step of itself
        (fp16: or half the smallest step, 2^-25, of a maximum of 1 that is part
        of the sum), so its sum with V by half a step of the spread (and n 2^-25
        of the largest V); the n weights times V are added in fp32. The result rounds by half a step,
        plus the smallest step in fp16."""
        hkv, g = self.k.shape[1], q.shape[1] // self.k.shape[1]
        d = q.shape[-1]
        for s, n in enumerate(self.len):
            for h in range(hkv):
                k, v = (f64(x[h]) for x in self.rows[s])
                for x in range(g):
                    hq, c = h * g + x, self.count[s]
                    qq = f64(q[s, hq, :c])
                    want, wl, spread = dec.attend(qq, k, v, self.start[s], see[s][:c, :c], sigma)
                    size = sigma * (np.abs(qq) @ np.abs(np.nan_to_num(k)).T).max(initial=0.0)
                    logit = size * d * 2.0 ** -23 + 2.0 ** -21
                    rel = 2 * logit + 2.0 ** -15 + n * 2.0 ** -23 + half_step(dtype)
                    got, gl = f64(o[s, hq, :c]), f64(lse[s, hq, :c])
                    if (s, h) in wild:
                        ok = ~np.isfinite(want)
                        assert np.array_equal(np.isnan(want), np.isnan(got))
                        assert np.array_equal(want[ok & ~np.isnan(want)], got[ok & ~np.isnan(want)])
                        fin = np.isfinite(want)
                    else:
                        fin = np.ones_like(want, dtype=bool)
                    tol = half_step(dtype) * np.abs(want) + rel * spread + 2.0 ** -24
                    if dtype is FP16:
                        tol += n * 2.0 ** -25 * np.abs(v[np.isfinite(v)]).max(initial=0.0)
                    assert (np.abs(got - want)[fin] <= tol[fin]).all(), (s, hq)
                    e = np.isneginf(wl)
                    assert np.array_equal(e, np.isneginf(gl))
                    f = np.isfinite(wl)
                    assert (np.abs(gl - wl)[f] <= logit + n * 2.0 ** -23
                            + 4 * 2.0 ** -23 * (1 + np.abs(wl[f]))).all()


def chains(t, count):
    return [np.tril(np.ones((t, t), dtype=bool)) for _ in count]


def pack_mask(see, t, dev):
    w = (t + 31) // 32
    out = np.zeros((len(see), t, w), dtype=np.uint32)
    for s, x in enumerate(see):
        for i, j in zip(*np.nonzero(x)):
            out[s, i, j >> 5] |= np.uint32(1 << (j & 31))
    return torch.from_numpy(out.view(np.int32)).to(dev)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP16, 64), (BF16, 64), (FP16, 128)])
@pytest.mark.parametrize("page,hkv,g", [(16, 1, 1), (64, 2, 4), (256, 3, 2), (128, 1, 8), (32, 2, 3)])
def test_decoding_step(page, hkv, g, dtype, d, dev):
    """One new token per sequence: lengths at every edge of pages and tiles."""
    start = [0, 1, 15, 16, 63, 64, 127, 128, 129, 700]
    t = Tree(dev, dtype, d, page, hkv, start, [1] * len(start), 1)
    q = (2 * torch.randn(len(start), hkv * g, 1, d, generator=torch.Generator().manual_seed(5)))
    q = q.to(dtype).to(dev)
    o, lse = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), lse=True)
    t.check(q, o, lse, chains(1, start), 1 / math.sqrt(d), dtype)


@pytest.mark.parametrize("dtype,d", [(BF16, 128), (FP16, 64)])
@pytest.mark.parametrize("tree,hkv,g", [(2, 2, 1), (5, 1, 3), (9, 2, 4), (17, 1, 1), (33, 2, 2),
                                        (40, 1, 8), (64, 1, 4), (130, 1, 3)])
@pytest.mark.parametrize("page", [16, 128])
def test_drafted_trees(page, tree, hkv, g, dtype, d, dev):
    """Random masks over ragged batches: empty rows, empty sequences, drafts
    without a prefix, counts below the width of the call; rows behind the
    count stay as they were."""
    r = np.random.default_rng(tree * page)
    start = [0, 3, 61, 200, 0, 300]
    count = [tree, max(tree - 1, 1), tree, tree // 2, 0, 1]
    see = [r.random((tree, tree)) < 0.4 for _ in start]
    see[0][tree // 2] = False  # sees nothing at all
    see[5][:] = False          # only the prefix
    t = Tree(dev, dtype, d, page, hkv, start, count, tree, seed=tree)
    q = torch.randn(len(start), tree, hkv * g, d, generator=torch.Generator().manual_seed(tree))
    q = (2 * q).to(dtype).to(dev).transpose(1, 2)  # strided, as a projection leaves it
    out = torch.full(q.shape, 7.0, dtype=dtype, device=dev)
    o, lse = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), pack_mask(see, tree, dev),
                           i32(count, dev), scale=0.11, lse=True, out=out)
    assert o is out
    t.check(q, o, lse, see, 0.11, dtype)
    assert (o[0, :, tree // 2] == 0).all() and torch.isneginf(lse[0, :, tree // 2]).all()
    for s, c in enumerate(count):
        assert (o[s, :, c:] == 7).all() and (lse[s, :, c:] == 0).all()
    again = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), pack_mask(see, tree, dev),
                          i32(count, dev), scale=0.11)
    for s, c in enumerate(count):
        assert torch.equal(again[s, :, :c], o[s, :, :c]) and not again[s, :, c:].any()


@pytest.mark.parametrize("tree,g", [(4, 1), (12, 2), (48, 4)])
def test_chain_without_a_mask_equals_its_mask(tree, g, dev):
    start = [5, 130]
    t = Tree(dev, BF16, 128, 16, 2, start, [tree] * 2, tree)
    q = torch.randn(2, 2 * g, tree, 128, device=dev).to(BF16)
    a = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev))
    chain = i32([list(range(-1, tree - 1))] * 2, dev)
    b = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), pbs.tree_mask(chain)[0])
    assert torch.equal(a, b)


@pytest.mark.parametrize("tree,g", [(6, 1), (6, 4), (48, 4)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_hidden_tokens_have_no_part(tree, g, dtype, dev):
    """NaN and infinities in drafts reach exactly the rows that see them."""
    start, count = [70, 0, 3000], [tree, tree, tree]
    t = Tree(dev, dtype, 64, 32, 2, start, count, tree)
    see = [np.tril(np.ones((tree, tree), dtype=bool)) for _ in start]
    for s in see:
        s[:, 2], s[:, 4], s[:, 5] = False, False, False
        s[2, 2], s[4, 4], s[5, 4], s[5, 5] = True, True, True, True
    bad = {2: ("v", float("inf")), 4: ("k", float("nan")), 5: ("v", float("nan"))}
    for s in range(3):
        for j, (what, x) in bad.items():
            n = start[s] + j
            p, o = int(t.table[s, n // 32]), n % 32
            (t.k if what == "k" else t.v)[p, :, o] = x
            t.rows[s][0 if what == "k" else 1][:, n] = x
    q = torch.randn(3, 2 * g, tree, 64, device=dev).to(dtype)
    o, lse = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), pack_mask(see, tree, dev),
                           i32(count, dev), lse=True)
    fine = [i for i in range(tree) if i not in (2, 4, 5)]
    assert torch.isfinite(o[:, :, fine]).all() and torch.isfinite(lse[:, :, fine]).all()
    assert torch.isinf(o[:, :, 2]).all() and torch.isnan(o[:, :, 4:6]).all()
    assert torch.isnan(lse[:, :, 4]).all()
    t.check(q, o, lse, see, 1 / 8, dtype, wild=set(itertools.product(range(3), range(2))))


def test_long_context_split_over_every_sm(dev):
    """One sequence, keys and values of one head: each SM takes a part; the
    largest logit sits in the last page, the second one in the first."""
    n, d = 100003, 128
    k = torch.randn(-(-n // 64), 1, 64, d, device=dev).to(BF16)
    v = torch.randn(k.shape, device=dev).to(BF16)
    table = torch.randperm(k.shape[0], device=dev).to(torch.int32)[None]
    q = torch.randn(1, 4, 1, d, device=dev).to(BF16)
    flat = lambda x: x[table[0].long()].view(-1, d)
    k[table[0, -1], 0, (n - 1) % 64] = 3 * q[0, 1, 0]
    k[table[0, 0], 0, 5] = 2.9 * q[0, 1, 0]
    o, lse = pbs.tree_attn(q, k, v, table.contiguous(), i32([n - 1], dev), lse=True)
    a = q[0, :, 0].double() @ flat(k)[:n].double().T / math.sqrt(d)
    want = torch.softmax(a, -1) @ flat(v)[:n].double()
    spread = torch.softmax(a, -1) @ flat(v)[:n].double().abs()
    size = float((q[0, :, 0].double().abs() @ flat(k)[:n].double().abs().T).max()) / math.sqrt(d)
    rel = 2 * (size * d * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -15 + 2.0 ** -12  # n 2^-23 < 2^-6;
    # the parts are summed tile by tile, 64 keys at a time: n / 64 + 64 steps
    # the weights round to 16 bits: half a step of the spread
    assert ((o[0, :, 0].double() - want).abs() <= half_step(BF16) * want.abs()
            + (rel + half_step(BF16)) * spread).all()
    assert ((lse[0, :, 0].double() - torch.logsumexp(a, -1)).abs() <= rel).all()


@pytest.mark.parametrize("tree,hq,hkv,b,most", [(64, 32, 8, 24, 900), (1, 32, 8, 150, 400),
                                                (20, 16, 8, 40, 3000), (100, 8, 2, 9, 2000),
                                                (1024, 2, 2, 2, 300), (3, 64, 1, 3, 700),
                                                (5, 1, 1, 70, 90)])
def test_many_items_in_a_run(tree, hq, hkv, b, most, dev):
    """Batches whose CTAs work through several items each, drafts that span key
    tiles in one after the other: against the formula in fp64 on the GPU, within
    a step of the result plus a step of the spread."""
    d, page, g = 128, 64, torch.Generator(dev).manual_seed(tree)
    r = random.Random(b)
    start = [r.randint(0, most) for _ in range(b)]
    count = [r.randint(0, tree) if tree > 1 else 1 for _ in range(b)]
    need = [-(-(s + c) // page) for s, c in zip(start, count)]
    pages, width = sum(need) + 1, max(need)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(b)).tolist()
    table = torch.full((b, width), -1, dtype=torch.int32)
    for s in range(b):
        for j in range(need[s]):
            table[s, j] = perm.pop()
    k, v = (torch.randn(pages, hkv, page, d, generator=g, device=dev).to(BF16) for _ in range(2))
    q = (2 * torch.randn(b, hq, tree, d, generator=g, device=dev)).to(BF16)
    parents = [[-1 if i == 0 else r.randrange(max(0, i - 5), i) for i in range(tree)]] * b
    mask = pbs.tree_mask(i32(parents, dev))[0]
    o, lse = pbs.tree_attn(q, k, v, table.to(dev), i32(start, dev), mask, i32(count, dev), lse=True)
    assert pbs.device_status() == 0
    see = torch.from_numpy(dec.visible(parents[0], tree)).to(dev)
    for s in range(b):
        c, n = count[s], start[s] + count[s]
        assert not o[s, :, c:].any() and not lse[s, :, c:].any()
        if not c:
            continue
        at = table[s, :need[s]].to(dev).long()
        kk, vv = (x[at].transpose(0, 1).reshape(hkv, -1, d)[:, :n].double().repeat_interleave(
            hq // hkv, 0) for x in (k, v))
        a = q[s, :, :c].double() @ kk.transpose(1, 2) / math.sqrt(d)
        a[:, :, start[s]:] = a[:, :, start[s]:].masked_fill(~see[:c, :c], -math.inf)
        p = torch.softmax(a, -1)
        tol = half_step(BF16) * (p @ vv).abs() + 2 * half_step(BF16) * (p @ vv.abs())
        assert ((o[s, :, :c].double() - p @ vv).abs() <= tol).all()
        assert (lse[s, :, :c].double() - torch.logsumexp(a, -1)).abs().max() < 1e-3


@pytest.mark.parametrize("tree,g", [(1, 4), (7, 4), (64, 4)])
def test_waits_are_bounded(tree, g, dev, monkeypatch):
    """Each kernel with every CTA's first K tile left out: the waits run out
    (about a second), the status says so, and the next call is right."""
    t = Tree(dev, BF16, 128, 64, 1, [300], [tree], tree, junk=False)
    q = torch.randn(1, g, tree, 128, device=dev).to(BF16)
    call = lambda: pbs.tree_attn(q, t.k, t.v, t.table, i32(t.start, dev))
    good = call()
    assert pbs.device_status() == 0
    monkeypatch.setenv("PBS_FAULT_INJECT", "tree")
    call()
    code, where = pbs.device_status(detail=True)
    monkeypatch.delenv("PBS_FAULT_INJECT")
    assert code == _lib.ERR_TIMEOUT and where > 0
    assert torch.equal(call(), good)


@pytest.mark.parametrize("d,seqs,hkv,g,tree,most,page", [
    (128, 65, 8, 4, 1, 200, 64), (128, 520, 1, 5, 3, 70, 16), (128, 33, 4, 1, 16, 500, 128),
    (128, 128, 1, 16, 1, 1023, 32), (64, 9, 1, 3, 5, 2500, 16), (64, 70, 2, 1, 12, 300, 64),
    (64, 4, 2, 16, 1, 5000, 256), (64, 300, 3, 2, 2, 40, 16)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_many_short_sequences(d, seqs, hkv, g, tree, most, page, dtype, dev):
    """Few rows and many items, ragged: empty sequences, drafts across tiles, and
    in every third sequence NaN in a draft that only its own row sees."""
    r = random.Random(seqs)
    start = [r.choice([0, r.randint(0, 70), r.randint(0, most)]) for _ in range(seqs)]
    start[0] = most
    count = [r.randint(0, tree) if tree > 1 else 1 for _ in range(seqs)]
    t = Tree(dev, dtype, d, page, hkv, start, count, tree, seqs)
    see, wild = [], set()
    for s in range(seqs):
        x = np.tril(np.ones((tree, tree), dtype=bool))
        if s % 3 == 0 and count[s] > 1:
            j = count[s] - 1
            n = start[s] + j
            p, o = int(t.table[s, n // page]), n % page
            t.v[p, :, o] = float("nan")
            t.rows[s][1][:, n] = float("nan")
            x[:, j] = False
            x[j, j] = True
            wild |= {(s, h) for h in range(hkv)}
        see.append(x)
    q = (2 * torch.randn(seqs, hkv * g, tree, d, generator=torch.Generator().manual_seed(3)))
    q = q.to(dtype).to(dev)
    call = lambda: pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), pack_mask(see, tree, dev),
                                 i32(count, dev), lse=True)
    o, lse = call()
    assert pbs.device_status() == 0
    t.check(q, o, lse, see, 1 / math.sqrt(d), dtype, wild=wild)
    for s in range(seqs):
        assert not o[s, :, count[s]:].any()
    again = call()  # the same on every run
    assert torch.equal(bits(o), bits(again[0])) and torch.equal(bits(lse), bits(again[1]))


@pytest.mark.parametrize("tree,g,most", [(12, 3, 300), (90, 3, 200), (64, 2, 150), (3, 2, 400)])
def test_drafts_of_many_sequences(tree, g, most, dev):
    """Far more items than CTAs, some of them cut, rows behind the counts zeroed
    or left as they were."""
    r, seqs, hkv, d = random.Random(tree), 221, 3, 64
    start = [r.randint(0, most) for _ in range(seqs)]
    count = [r.choice([0, 1, tree, r.randint(0, tree)]) for _ in range(seqs)]
    t = Tree(dev, BF16, d, 32, hkv, start, count, tree, tree)
    q = (2 * torch.randn(seqs, hkv * g, tree, d, generator=torch.Generator().manual_seed(4)))
    q = q.to(BF16).to(dev)
    o, lse = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), None, i32(count, dev), lse=True)
    assert pbs.device_status() == 0
    t.check(q, o, lse, chains(tree, count), 1 / math.sqrt(d), BF16)
    kept = torch.full_like(o, 7.0)
    pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), None, i32(count, dev), out=kept)
    for s in range(seqs):
        assert not o[s, :, count[s]:].any() and not lse[s, :, count[s]:].any()
        assert torch.equal(bits(kept[s, :, :count[s]]), bits(o[s, :, :count[s]]))
        assert (kept[s, :, count[s]:] == 7).all()


@pytest.mark.parametrize("d,seqs,hkv,tokens", [(64, 1, 8, 130), (128, 64, 8, 130), (128, 2, 8, 9000),
                                               (64, 2, 8, 9000)])
@pytest.mark.parametrize("tree", [1, 9, 64])
def test_waits_end_in_long_runs(tree, d, seqs, hkv, tokens, dev, monkeypatch):
    """The same where a CTA has more tiles, and more items, than its ring holds."""
    t = Tree(dev, BF16, d, 64, hkv, [tokens] * seqs, [tree] * seqs, tree, junk=False)
    q = torch.randn(seqs, 4 * hkv, tree, d, device=dev).to(BF16)
    call = lambda: pbs.tree_attn(q, t.k, t.v, t.table, i32(t.start, dev))
    good = call()
    assert pbs.device_status() == 0
    monkeypatch.setenv("PBS_FAULT_INJECT", "tree")
    call()
    code, where = pbs.device_status(detail=True)
    monkeypatch.delenv("PBS_FAULT_INJECT")
    assert code == _lib.ERR_TIMEOUT and where > 0
    assert torch.equal(call(), good)


def test_pools_beyond_32_bits(dev):
    """Pools of 4.5 GB each: copies, appends, accepts and attention at pages
    whose offsets pass 2^31 elements and 2^32 bytes."""
    hkv, page, d = 8, 64, 128
    pages = 2 ** 31 // (hkv * page * d) + 3000
    k, v = (torch.empty(pages, hkv, page, d, dtype=BF16, device=dev) for _ in range(2))
    top = [pages - 1, pages - 2, pages - 700]
    n, t = 150, 3
    table = i32([top], dev)
    rows = [torch.randn(1, hkv, n + t, d, device=dev).to(BF16) for _ in range(2)]
    pbs.cache_append(*rows, k, v, table, i32([0], dev))
    q = torch.randn(1, hkv * 2, t, d, device=dev).to(BF16)
    o = pbs.tree_attn(q, k, v, table, i32([n], dev))
    flat = [x.double().repeat_interleave(2, 1) for x in rows]
    a = q.double() @ flat[0].transpose(2, 3) / math.sqrt(d)
    a += torch.full((t, n + t), -math.inf, device=dev, dtype=torch.float64).triu(n + 1)
    p = torch.softmax(a, -1)
    tol = half_step(BF16) * ((p @ flat[1]).abs() + (1 + 2.0 ** -2) * (p @ flat[1].abs()))
    assert ((o.double() - p @ flat[1]).abs() <= tol).all()
    pbs.cache_copy(k, v, table[0].contiguous(), i32([0, 1, pages - 5], dev))
    assert torch.equal(bits(k[top]), bits(k[[0, 1, pages - 5]]))
    assert torch.equal(bits(v[top]), bits(v[[0, 1, pages - 5]]))
    pbs.cache_accept(k, v, table, i32([n], dev), i32([[0, 2]], dev))
    got = k[top].transpose(0, 1).reshape(hkv, -1, d)
    assert torch.equal(got[:, n + 1], rows[0][0, :, n + 2])
    m = k.clone()[:4]  # keep four pages, then compact the top ones down
    refs = torch.zeros(pages, dtype=torch.int32, device=dev)
    refs[top] = 1
    want = [x[top].clone() for x in (k, v)]
    pbs.cache_compact(k, v, table, refs)
    assert sorted(table[0].tolist()) == [0, 1, 2] and refs[:3].tolist() == [1, 1, 1]
    for x, w in zip((k, v), want):
        assert torch.equal(bits(x[table[0].long()]), bits(w))
    del m


def test_cache_calls_in_a_graph(dev):
    """Reserve, copy, append, attend, accept and trim captured together and
    replayed: each replay works on what the tables hold by then."""
    hkv, d, page = 2, 64, 16
    c = pbs.PagedCache(3, 200, 64, hkv, d, page, 1, BF16, dev)
    count, want, keep = i32([2, 2, 0], dev), i32([2, 2, 0], dev), i32([-1, -1, -1], dev)
    k, v = (torch.zeros(3, hkv, 2, d, dtype=BF16, device=dev) for _ in range(2))
    q = torch.zeros(3, 4, 2, d, dtype=BF16, device=dev)
    path, taken = i32([[1, 0], [0, 1], [0, 0]], dev), i32([1, 2, 0], dev)

    def step():
        c.reserve(want)
        c.append(0, k, v, count=count)
        o = c.attend(0, q, count=count)
        c.accept(path, taken)
        c.trim(keep)
        return o

    side = torch.cuda.Stream(dev)
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    c.trim(i32([0, 0, 0], dev))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    rows = [[], []]
    g = torch.Generator().manual_seed(3)
    for i in range(20):
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, generator=g).to(BF16))
        want.copy_(torch.where(count > 0, c.lens + 2, 0))
        graph.replay()
        for s in (0, 1):
            kk, vv = (np.concatenate([rows[s][j], f64(x[s])], 1) if len(rows[s]) else f64(x[s])
                      for j, x in enumerate((k, v)))
            n = kk.shape[1] - 2
            for h in range(4):
                w = dec.attend(f64(q[s, h]), kk[h // 2], vv[h // 2], n, np.tril(np.ones((2, 2), bool)),
                               1 / 8)[0]
                assert np.abs(f64(out[s, h]) - w).max() <= 2.0 ** -8 * np.abs(w).max() + 2.0 ** -9
            at = list(range(n)) + [n + j for j in ([1], [0, 1])[s]]
            rows[s] = [kk[:, at], vv[:, at]]
    assert c.lens.tolist() == [20, 40, 0] and pbs.device_status() == 0


def test_tree_attn_refuses(dev):
    t = Tree(dev, BF16, 64, 16, 2, [20, 5], [2, 2], 2, junk=False)
    q, start = torch.zeros(2, 4, 2, 64, dtype=BF16, device=dev), i32([20, 5], dev)
    ok = dict(q=q, k_pages=t.k, v_pages=t.v, table=t.table, start=start)
    for bad in (dict(q=q.half()), dict(q=q[:1]), dict(q=q[:, :3]), dict(q=q[..., :32]),
                dict(k_pages=t.k[None], v_pages=t.v[None]), dict(v_pages=t.v[:1]),
                dict(table=t.table.long()), dict(table=t.table[:, ::2]), dict(start=start[:1]),
                dict(mask=torch.zeros(2, 2, 2, dtype=torch.int32, device=dev)),
                dict(count=start.long()), dict(out=q), dict(out=q.transpose(1, 2)),
                dict(out=t.k.view(-1)[64:64 + q.numel()].view(q.shape)),
                dict(start=start.cpu()), dict(k_pages=t.k.transpose(1, 2), v_pages=t.v.transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            pbs.tree_attn(**dict(ok, **bad))
    with pytest.raises(pbs.PbsError):
        pbs.tree_attn(**dict(ok, k_pages=t.k[:, :, :12].contiguous(), v_pages=t.v[:, :, :12].contiguous()))
    assert pbs.tree_attn(**dict(ok, q=q[:, :, :0])).shape == (2, 4, 0, 64)


@pytest.mark.parametrize("tree", [1, 9, 70])
def test_nothing_to_do_and_large_pages(tree, dev):
    """A batch without drafts: allocated rows are 0, given ones stay. Then pages
    of 256 tokens that end inside tiles and hold several."""
    start, zero = [300, 0, 255, 1000], [0] * 4
    t = Tree(dev, FP16, 64, 256, 2, start, [tree] * 4, tree, seed=tree)
    q = torch.randn(4, 4, tree, 64, device=dev).half()
    o, lse = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), count=i32(zero, dev), lse=True)
    assert not o.any() and not lse.any()
    out = torch.full_like(o, 5)
    pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), count=i32(zero, dev), out=out)
    assert (out == 5).all()
    o, lse = pbs.tree_attn(q, t.k, t.v, t.table, i32(start, dev), lse=True)
    t.check(q, o, lse, chains(tree, start), 1 / 8, FP16)


def test_lengths_beyond_the_table_are_reported(dev):
    """Such a sequence is left alone; a page outside is reported, the others
    come out right."""
    t = Tree(dev, BF16, 64, 16, 1, [20, 5, 9], [1, 1, 1], 1)
    q = torch.randn(3, 2, 1, 64, device=dev).to(BF16)
    good = pbs.tree_attn(q, t.k, t.v, t.table, i32([20, 5, 9], dev))
    out = torch.full_like(good, 3)
    pbs.tree_attn(q, t.k, t.v, t.table, i32([16 * t.table.shape[1], 5, -1], dev), out=out)
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
    assert (out[0] == 3).all() and (out[2] == 3).all() and torch.equal(out[1], good[1])
    table = t.table.clone()
    table[0, 1] = 10000
    out = pbs.tree_attn(q, t.k, t.v, table, i32([20, 5, 9], dev))
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
    assert torch.equal(out[1:], good[1:])


# --------------------------------------------------------- streams, graphs, run
@pytest.mark.parametrize("tree,g", [(1, 4), (12, 2), (48, 4)])
def test_captured_steps_read_lengths_at_replay(tree, g, dev):
    """Two captured graphs that share one workspace, replayed in turn on
    another stream after the lengths, tables and queries changed."""
    start = [[700, 30], [64, 1000], [0, 129]]
    trees = [Tree(dev, BF16, 128, 64, 2, s, [tree] * 2, tree, seed=i) for i, s in enumerate(start)]
    pages = max(t.k.shape[0] for t in trees)
    width = max(t.table.shape[1] for t in trees)
    k, v = (torch.zeros(pages, 2, 64, 128, dtype=BF16, device=dev) for _ in range(2))
    table, st = torch.full((2, width), -1, dtype=torch.int32, device=dev), i32([0, 0], dev)
    q = torch.zeros(2, 2 * g, tree, 128, dtype=BF16, device=dev)
    c = _lib.Cache(1, pages, 2, 64, 128, 2, width)
    ws = torch.empty(pbs.lib().pbs_tree_workspace_bytes(2 * g, tree, c), dtype=torch.uint8, device=dev)
    call = lambda: pbs.tree_attn(q, k, v, table, st, lse=True, ws=ws)

    def load(t):
        k.zero_(), v.zero_(), table.fill_(-1)
        k[:t.k.shape[0]], v[:t.v.shape[0]] = t.k, t.v
        table[:, :t.table.shape[1]] = t.table
        st.copy_(i32(t.start, dev))
        q.copy_(torch.randn(q.shape, device=dev))

    load(trees[0])
    graphs = []
    call()
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        graphs.append((graph, out))
    side = torch.cuda.Stream(dev)
    for i in (1, 2, 0):
        load(trees[i])
        want = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for graph, out in graphs:
                graph.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


@pytest.mark.parametrize("tree,g", [(1, 4), (40, 2)])
def test_calls_right_behind_what_they_read(tree, g, dev):
    """Queries, lengths and rows written by the kernel just in front of each
    call, results read by the one just behind, over and over on one stream."""
    t = Tree(dev, BF16, 128, 64, 2, [900, 333], [tree] * 2, tree, junk=False)
    start = torch.zeros(2, dtype=torch.int32, device=dev)
    q = torch.zeros(2, 2 * g, tree, 128, dtype=BF16, device=dev)
    out, sums = torch.empty_like(q), torch.zeros_like(q, dtype=torch.float32)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device=dev)
    draws = [torch.randn(q.shape, device=dev).to(BF16) for _ in range(4)]
    lens = [i32(x, dev) for x in ([900, 333], [64, 200], [500, 1], [0, 128])]
    want = []
    for i in range(4):
        want.append(pbs.tree_attn(draws[i], t.k, t.v, t.table, lens[i]))
        torch.cuda.synchronize()
    for n in range(40):
        i = n % 4
        big = torch.ones(1 << 24, device=dev).cumsum(0)  # keeps the stream busy in front
        start.copy_(lens[i])
        q.copy_(draws[i])
        pbs.tree_attn(q, t.k, t.v, t.table, start, out=out, ws=ws)
        sums += (out.float() - want[i].float()).abs()
        out.fill_(9)
        del big
    assert not sums.any()


@pytest.mark.parametrize("tree,g", [(1, 4), (40, 2)])
def test_captured_behind_copies_and_joined_streams(tree, g, dev):
    """A graph in which the call stands behind a copy, behind a kernel of another
    stream and behind both, and two calls run side by side."""
    t = Tree(dev, BF16, 128, 64, 2, [900, 333], [tree] * 2, tree, junk=False)
    src = [torch.randn(2, 2 * g, tree, 128, device=dev).to(BF16) for _ in range(2)]
    lens = i32(t.start, dev)
    want = [pbs.tree_attn(x, t.k, t.v, t.table, lens) for x in src]
    q = [torch.zeros_like(x) for x in src]
    start = torch.zeros_like(lens)
    side, graph = torch.cuda.Stream(dev), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            start.copy_(lens)
            q[1].copy_(src[1])
        q[0].copy_(src[0])
        main.wait_stream(side)
        a = pbs.tree_attn(q[0], t.k, t.v, t.table, start)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            b = pbs.tree_attn(q[1], t.k, t.v, t.table, start)
        c = pbs.tree_attn(a * 0 + q[0], t.k, t.v, t.table, start)
        main.wait_stream(side)
        d = pbs.tree_attn(q[1] + b * 0, t.k, t.v, t.table, start)
    for _ in range(3):
        for x in (start, *q):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, i in ((a, 0), (b, 1), (c, 0), (d, 1)):
            assert torch.equal(got, want[i])


def test_two_calls_at_once_on_two_streams(dev):
    t = [Tree(dev, BF16, 128, 64, 2, [900, 333], [3, 2], 3, seed=i) for i in range(2)]
    q = [torch.randn(2, 8, 3, 128, device=dev).to(BF16) for _ in range(2)]
    call = lambda i: pbs.tree_attn(q[i], t[i].k, t[i].v, t[i].table, i32(t[i].start, dev),
                                   count=i32(t[i].count, dev))
    want = [call(0), call(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(i))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_prefill_then_drafts(dev):
    """Rotary positions, the prefill, the cache behind it, two rounds of drafted
    trees verified, accepted and continued, a fork and a compaction: every
    attention output against fp64 attention on the same rotated rows. The
    prefill kernel rounds P to 16 bits, so its outputs are held to the
    forward's tolerance (2e-2)."""
    g = torch.Generator().manual_seed(0)
    layers, b, hq, hkv, n, d, page = 2, 1, 4, 2, 512, 64, 32
    f, gain = pbs.rope_freqs(d, scaling=dict(type="yarn", factor=4, original=256))
    fd = f.to(dev)
    c = pbs.PagedCache(3, 700, 60, hkv, d, page, layers, BF16, dev)
    keys = [[None] * layers for _ in range(3)]  # rotated K, V in fp64 by sequence and layer

    def project(m, pos):
        q, k, v = (torch.randn(3, h, m, d, generator=g).to(BF16).to(dev) for h in (hq, hkv, hkv))
        qr, kr = pbs.rope(q, k, pos, fd, gain)
        for x, y in ((q, qr), (k, kr)):
            w = dec.rope(f64(x), pos.cpu().numpy(), f.numpy(), gain)
            assert (np.abs(f64(y) - w) <= rope_bound(f64(x), w, gain, BF16, d)).all()
        return qr, kr, v

    c.reserve(i32([n, 0, 0], dev))
    pos = torch.arange(n, dtype=torch.int32, device=dev).expand(3, n).contiguous()
    for l in range(layers):
        q, k, v = project(n, pos)
        o = pbs.pbs_attention(q[:1].contiguous(), k[:1].contiguous(), v[:1].contiguous(), 64, 64,
                              mode="dense_causal")
        c.append(l, k, v, count=i32([n, 0, 0], dev))
        keys[0][l] = (f64(k[0]), f64(v[0]))
        see = np.tril(np.ones((n, n), dtype=bool))
        for h in range(hq):
            want = dec.attend(f64(q[0, h, -3:]), *(x[h // 2] for x in keys[0][l]), 0, see[-3:],
                              1 / math.sqrt(d))[0]
            assert np.abs(f64(o[0, h, -3:]) - want).max() <= 2e-2
    c.lens += i32([n, 0, 0], dev)
    c.fork(i32([0], dev), i32([2], dev))
    keys[2] = list(keys[0])
    parents = [[-1, 0, 0, 1, 2, 2, -1]] * 3
    accepted = [[[0, 2, 5], [], [6]], [[0, 1, 3], [], [0, 2, 4]]]
    t = len(parents[0])
    for path in accepted:
        mask, depth = pbs.tree_mask(i32(parents, dev))
        count = i32([t, 0, t], dev)
        c.reserve(torch.where(count > 0, c.lens + t, 0).to(torch.int32))
        start = c.lens.tolist()
        for l in range(layers):
            q, k, v = project(t, c.lens[:, None] + depth)
            c.append(l, k, v, count=count)
            o, lse = c.attend(l, q, mask, count=count, lse=True)
            see = dec.visible(parents[0], t)
            for s in (0, 2):
                kk, vv = (np.concatenate([x, f64(y[s])], 1) for x, y in zip(keys[s][l], (k, v)))
                for h in range(hq):
                    want, wl, spread = dec.attend(f64(q[s, h]), kk[h // 2], vv[h // 2], start[s],
                                                  see, 1 / math.sqrt(d))
                    size = np.abs(f64(q[s, h])) @ np.abs(kk[h // 2]).T / math.sqrt(d)
                    rel = 2 * (size.max() * d * 2.0 ** -23 + 2.0 ** -21) + 2.0 ** -15 + \
                        kk.shape[1] * 2.0 ** -23
                    # half a step of the result, and of each weight
                    assert (np.abs(f64(o[s, h]) - want) <= 2.0 ** -8 * np.abs(want) +
                            (rel + 2.0 ** -8) * spread).all()
                    assert np.abs(f64(lse[s, h]) - wl).max() <= rel + 1e-5
                at = [start[s] + j for j in path[s]]
                keys[s][l] = tuple(np.concatenate([x[:, :start[s]], x[:, at]], 1)
                                   for x in (kk, vv))
        c.accept(i32([p + [0] * (t - len(p)) for p in path], dev), i32([len(p) for p in path], dev))
        assert c.lens.tolist() == [a + len(p) for a, p in zip(start, path)]
        c.compact()
    held = int((c.refs > 0).sum())
    assert int(c.table.max()) < held
    # everything that the cache holds is what went in
    for s, l in itertools.product((0, 2), range(layers)):
        m = int(c.lens[s])
        for pool, want in zip((c.k, c.v), keys[s][l]):
            rows = pool[l, c.table[s, :-(-m // page)].long()].transpose(0, 1).reshape(hkv, -1, d)
            assert np.array_equal(f64(rows[:, :m]), want)
    c.trim(i32([0, -1, 0], dev))
    assert not c.refs.any() and (c.table == -1).all() and not c.lens.any()
