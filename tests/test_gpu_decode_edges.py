"""The decoding operators where their calls meet: inputs that are outputs, calls
behind one that failed, sequences that a kernel refuses, and the far ends of
types and lengths."""
import random

import pytest
import torch

import long_context_sparse_segment_b200 as pbs
from long_context_sparse_segment_b200 import _lib
from test_gpu_decode import Tree, bits, i32, ids

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


# ----------------------------------------------------------------------- moves
@pytest.mark.parametrize("alias", ["start", "count", "both"])
@pytest.mark.parametrize("seqs,layers,n", [(1, 1, 5), (64, 32, 24), (200, 40, 12)])
def test_accept_into_the_lengths_it_reads(seqs, layers, n, alias, dev):
    """lens given as start (a draft's start is the length), as count, or as
    both: the same moves and lengths as with tensors of their own, over more
    blocks than the GPU holds at once."""
    hkv, page, d, tree, width, r = 8, 16, 128, 32, 3, random.Random(seqs)
    start = [r.randint(0, 12) for _ in range(seqs)]
    count = [min(x, n) for x in start] if alias == "both" else [r.randint(0, n) for _ in range(seqs)]
    start = count if alias == "both" else start
    path = i32([sorted(r.sample(range(tree), n)) + [0] * (tree - n) for _ in range(seqs)], dev)
    path[0, 0] = -1  # not good: its length stays
    count[0] = max(count[0], 1)
    table = torch.randperm(seqs * width, generator=torch.Generator().manual_seed(1))
    table = table.view(seqs, width).to(dev, torch.int32)
    k, v = (ids((layers, seqs * width, hkv, page, d), dev, seed=s) for s in (1, 2))
    k0, v0, wk, wv = k.clone(), v.clone(), k.clone(), v.clone()
    after = i32(count if alias == "count" else start, dev)
    pbs.cache_accept(wk, wv, table, i32(start, dev), path, i32(count, dev), after)
    assert pbs.device_status() != 0
    assert seqs == 1 or not torch.equal(bits(wk), bits(k0))
    want = [a + c for a, c in zip(start, count)]
    want[0] = (count if alias == "count" else start)[0]
    assert after.tolist() == want
    for _ in range(3):
        k.copy_(k0), v.copy_(v0)
        lens = i32(count if alias == "count" else start, dev)
        pbs.cache_accept(k, v, table, i32(start, dev) if alias == "count" else lens, path,
                         i32(count, dev) if alias == "start" else lens, lens)
        assert pbs.device_status() != 0
        assert torch.equal(lens, after)
        assert torch.equal(bits(k), bits(wk)) and torch.equal(bits(v), bits(wv))


def test_accept_refuses_lengths_inside_other_inputs(dev):
    k, v = (ids((4, 1, 16, 64), dev, seed=s) for s in (1, 2))
    x = i32([3, 3, 3, 3], dev)
    table, path = i32([[0, 1], [2, 3]], dev), i32([[0], [0]], dev)
    for kw in (dict(start=x[:2], lens=x[1:3]), dict(start=x[2:], count=x[:2], lens=x[1:3]),
               dict(start=x[:2], path=x[2:].view(2, 1), lens=x[2:]),
               dict(start=x[:2], lens=table.view(-1)[2:])):
        with pytest.raises(pbs.PbsError):
            pbs.cache_accept(k, v, table, **dict(dict(path=path), **kw))


@pytest.mark.parametrize("whole", [False, True])
def test_nothing_is_written_into_shared_pages_behind_a_failed_reserve(whole, dev):
    """A fork cut back to the middle of a shared page, a full pool, and the calls
    enqueued behind the reserve that fails: the other holder's rows stay, rows
    of pages that one sequence holds alone are written. By PagedCache and by the
    functions on every layer at once."""
    page, hkv, d, layers = 16, 2, 64, 3
    c = pbs.PagedCache(3, 112, 8, hkv, d, page, layers, BF16, dev)
    c.reserve(i32([100, 0, 12], dev))  # all 8 pages
    c.k.copy_(ids(c.k.shape, dev, seed=1)), c.v.copy_(ids(c.v.shape, dev, seed=2))
    c.lens.copy_(i32([100, 0, 10], dev))
    c.fork(i32([0], dev), i32([1], dev))
    c.trim(i32([-1, 50, -1], dev))
    assert pbs.device_status() == 0
    want = [bits(x).clone() for x in (c.k, c.v)]
    new = ids((layers, 3, hkv, 10, d), dev, seed=3)
    at = int(c.table[2, 0])
    for w in want:
        w[:, at, :, 10:12] = bits(new)[:, 2, :, :2]
    books = [x.clone() for x in (c.table, c.refs)]
    count = i32([0, 10, 2], dev)
    c.reserve(c.lens + count)
    if whole:
        pbs.cache_append(new, new, c.k, c.v, c.table, c.lens, count, refs=c.refs)
        for w in want:  # draft 1 behind token 9 + 1
            w[:, at, :, 10] = w[:, at, :, 11]
        pbs.cache_accept(c.k, c.v, c.table, c.lens, i32([[0, 2, 5], [0, 2, 5], [1, 0, 0]], dev),
                         i32([0, 3, 1], dev), c.lens, refs=c.refs)
        lens = [100, 50, 11]
    else:
        for l in range(layers):
            c.append(l, new[l], new[l], count=count)
        # a path that moves nothing makes no length of tokens that were not written
        c.accept(i32([[0, 1, 2]] * 3, dev), i32([0, 3, 2], dev))
        lens = [100, 50, 12]
    assert pbs.device_status() == _lib.ERR_PAGES
    assert all(torch.equal(a, b) for a, b in zip((c.table, c.refs), books))
    assert torch.equal(bits(c.k), want[0]) and torch.equal(bits(c.v), want[1])
    assert c.lens.tolist() == lens
    # with a page free the same calls go through
    c.trim(i32([-1, -1, 0], dev))
    c.reserve(i32([0, 60, 0], dev))
    c.append(0, new[0], new[0], count=i32([0, 10, 0], dev))
    assert pbs.device_status() == 0
    mine, theirs = int(c.table[1, 3]), int(c.table[0, 3])
    assert mine == at and torch.equal(bits(c.k)[:, theirs], want[0][:, theirs])
    assert torch.equal(bits(c.k)[0, mine, :, 2:12], bits(new)[0, 1])


# ------------------------------------------------------------------- attention
@pytest.mark.parametrize("tree", [1, 9, 70])
def test_refused_sequences_are_zero_in_what_is_allocated(tree, dev):
    """A sequence beyond its table and one of negative length, without a count:
    0 in allocated outputs, untouched in a given one, whose lse is 0."""
    t = Tree(dev, BF16, 64, 16, 1, [20, 5, 9], [tree] * 3, tree, junk=False)
    q = torch.randn(3, 2, tree, 64, device=dev).to(BF16)
    start = i32([16 * t.table.shape[1], 5, -1], dev)
    good, good_lse = pbs.tree_attn(q, t.k, t.v, t.table, i32([20, 5, 9], dev), lse=True)

    def junk():  # what the allocator hands out next
        for x in (q.shape, q.shape[:3]):
            torch.full(x, 7, dtype=q.dtype if len(x) == 4 else FP32, device=dev)

    for _ in range(3):
        junk()
        o, lse = pbs.tree_attn(q, t.k, t.v, t.table, start, lse=True)
        assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
        assert not o[[0, 2]].any() and not lse[[0, 2]].any()
        assert torch.equal(o[1], good[1]) and torch.equal(lse[1], good_lse[1])
    out = torch.full_like(q, 3)
    junk()
    _, lse = pbs.tree_attn(q, t.k, t.v, t.table, start, lse=True, out=out)
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT
    assert (out[[0, 2]] == 3).all() and not lse[[0, 2]].any() and torch.equal(out[1], good[1])
