"""The decoding operators where their calls meet: inputs that are outputs, calls
behind one that failed, sequences that a kernel refuses, and the far ends of
types and lengths."""
import random

import pytest
import torch

import long_context_sparse_segment_b200 as pbs
from test_gpu_decode import bits, i32, ids

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
