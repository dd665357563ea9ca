"""The decoding operators where their calls meet: inputs that are outputs, calls
behind one that failed, sequences that a kernel refuses, and the far ends of
types and lengths."""
import math
import random

import numpy as np
import pytest
import torch

import long_context_sparse_segment_b200 as pbs
from long_context_sparse_segment_b200 import _lib
from oracle import decode_oracle as dec
from pbs_testutil import f64
from test_gpu_decode import Tree, bits, i32, ids, rope_bound

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


def test_accept_of_an_empty_path_sets_the_lengths(dev):
    k, v = (ids((4, 1, 16, 64), dev, seed=s) for s in (1, 2))
    table, none = i32([[0, 1], [2, 3], [0, 1]], dev), torch.zeros(3, 0, dtype=torch.int32, device=dev)
    lens = i32([9, 9, 9], dev)
    pbs.cache_accept(k, v, table, i32([3, 4, -1], dev), none, lens=lens)
    assert pbs.device_status() == _lib.ERR_DEVICE_ASSERT  # the negative one
    assert lens.tolist() == [3, 4, 9]
    pbs.cache_accept(k, v, table, lens, none, lens=lens)
    pbs.cache_accept(k, v, table, i32([1, 2, 3], dev), none)
    pbs.cache_accept(k, v, table[:0], lens[:0], none[:0], lens=lens[:0])
    assert lens.tolist() == [3, 4, 9]
    with pytest.raises(pbs.PbsError):
        pbs.cache_accept(k, v, table[:2], lens[:2], none[:2], lens=lens[1:])
    # no row of a longer path
    pbs.cache_accept(k, v, table, i32([1, 2, 3], dev), i32([[0]] * 3, dev), i32([0, -2, 0], dev), lens)
    assert lens.tolist() == [1, 2, 3]


def test_tables_of_ones_own_need_no_reference_counts(dev):
    """A PagedCache whose table the caller fills, its counts left at 0."""
    c = pbs.PagedCache(2, 32, 4, 1, 64, 16, 1, BF16, dev)
    c.table.copy_(i32([[3, 1], [0, 2]], dev))
    new = ids((2, 1, 5, 64), dev, seed=1)
    c.append(0, new, new, start=i32([13, 2], dev))
    assert pbs.device_status() == 0
    for pool in (c.k, c.v):
        got = bits(pool)[0]
        assert torch.equal(got[3, :, 13:], bits(new)[0, :, :3])
        assert torch.equal(got[1, :, :2], bits(new)[0, :, 3:])
        assert torch.equal(got[0, :, 2:7], bits(new)[1])
    c.lens.copy_(i32([13, 2], dev))
    c.accept(i32([[1, 4], [0, 3]], dev))
    assert pbs.device_status() == 0 and c.lens.tolist() == [15, 4]
    assert torch.equal(bits(c.k)[0, 3, :, 13:15], bits(new)[0, :, [1, 4]])


@pytest.mark.parametrize("lead", [(), (2,)])
def test_append_refuses_rows_inside_the_pools(lead, dev):
    """k or v cut out of a pool, pools that share pages, and tables there; a
    neighbour of the pools in one allocation is taken."""
    size = (*lead, 4, 1, 16, 64)
    n = 2 * 64 * 16 * 4 // 2 * (lead[0] if lead else 1)
    big = ids((4 * n,), dev, seed=1)
    k, v, new = (big[i * n:(i + 1) * n].view(size) for i in range(3))
    rows = new.view(*lead, 2, 2, 16, 64)[..., :1, :3, :]  # [.., seqs, 1, 3, 64]
    table, start = i32([[0], [1]], dev), i32([2, 5], dev)
    inside = k.view(*lead, 2, 2, 16, 64)[..., :1, :3, :]
    ints = v.view(torch.int32).view(-1)
    before = bits(big).clone()
    for kw in (dict(k=inside), dict(v=inside), dict(v_pages=k),
               dict(v_pages=big[n // 4:n // 4 + n].view(size)), dict(table=ints[:2].view(2, 1)),
               dict(start=ints[2:4]), dict(count=ints[2:4])):
        with pytest.raises(pbs.PbsError):
            pbs.cache_append(**dict(dict(k=rows, v=rows, k_pages=k, v_pages=v, table=table,
                                         start=start), **kw))
    with pytest.raises(pbs.PbsError):
        pbs.cache_accept(k, big[n // 4:n // 4 + n].view(size), table, start, i32([[0], [0]], dev))
    assert torch.equal(bits(big), before)
    pbs.cache_append(rows, rows, k, v, table, start)
    for s in range(2):
        at = int(start[s])
        for pool in (k, v):
            assert torch.equal(bits(pool[..., s, :, at:at + 3, :]), bits(rows[..., s, :, :, :]))
    assert torch.equal(bits(big)[2 * n:], before[2 * n:])


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


# ------------------------------------------------------------------------ rope
def test_rope_outputs_beside_and_over_other_tensors(dev):
    """Head slices of one buffer: outputs that interleave with the inputs are
    taken, in place too; outputs that reach into an input or into one another
    are refused."""
    b, n, d = 2, 5, 64
    f = pbs.rope_freqs(d)[0].to(dev)
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    buf = torch.randn(b, n, 12, d, device=dev).to(BF16).transpose(1, 2)
    q, k, rest = buf[:, :4], buf[:, 4:6], buf[:, 6:]
    want = pbs.rope(q, k, pos, f)
    before = buf.clone()
    got = pbs.rope(q, k, pos, f, q_out=rest[:, :4], k_out=rest[:, 4:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(buf[:, :6], before[:, :6])
    assert torch.equal(rest[:, :4], want[0]) and torch.equal(rest[:, 4:], want[1])
    after = buf.clone()
    for kw in (dict(q_out=buf[:, 2:6]), dict(q_out=buf[:, 5:9]), dict(k_out=buf[:, 3:5]),
               dict(k_out=buf[:, 0:2]), dict(q_out=q, k_out=buf[:, 2:4]),
               dict(q_out=buf[:, 5:9], k_out=k), dict(q_out=rest[:, :4], k_out=rest[:, 3:5])):
        with pytest.raises((ValueError, pbs.PbsError)):
            pbs.rope(q, k, pos, f, **kw)
    with pytest.raises(pbs.PbsError):  # q and k the same rows, both turned in place
        pbs.rope(q, q[:, :2], pos, f, q_out=q, k_out=q[:, :2])
    assert torch.equal(buf, after)
    pbs.rope(q, k, pos, f, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(rest, after[:, 6:])


def test_rope_takes_just_the_outputs_that_are_apart(dev):
    """Random slices of one buffer as inputs and outputs, against their elements
    one by one."""
    r = random.Random(5)
    d = 16
    f = pbs.rope_freqs(d)[0].to(dev)
    base = torch.zeros(2 * 4 * 6 * d, dtype=FP32, device=dev)
    names = torch.arange(base.numel()).view(2, 4, 6, d)
    taken = 0
    for turn in range(400):
        layout = r.choice([(0, 2, 1, 3), (0, 1, 2, 3), (1, 0, 2, 3), (2, 0, 1, 3)])
        buf, num = base.view(2, 4, 6, d).permute(layout), names.permute(layout)
        size = [r.randint(1, buf.shape[0]), 0, r.randint(1, buf.shape[2])]
        hq, hkv = (r.randint(1, max(1, buf.shape[1] // 2)) for _ in range(2))

        def cut(h):
            b, n = size[0], size[2]
            at = [r.randint(0, x - y) for x, y in zip(buf.shape, (b, h, n))]
            return tuple(slice(a, a + y) for a, y in zip(at, (b, h, n)))

        q, k = cut(hq), cut(hkv)
        qo, ko = (x if r.random() < 0.3 else cut(h) for x, h in ((q, hq), (k, hkv)))
        if r.random() < 0.2:
            ko = None
        ids = {n: set(num[x].flatten().tolist()) for n, x in
               dict(q=q, k=k, qo=qo, ko=ko).items() if x is not None}
        bad = ids["qo"] & ids["k"] or (qo != q and ids["qo"] & ids["q"])
        if ko is not None:
            bad = bad or ids["ko"] & ids["q"] or ids["ko"] & ids["qo"] or \
                (ko != k and ids["ko"] & ids["k"])
        base.copy_(torch.randn(base.shape, generator=torch.Generator().manual_seed(turn)))
        before = base.clone()
        pos = torch.randint(0, 1000, (size[0], size[2]), dtype=torch.int32).to(dev)
        call = lambda **kw: pbs.rope(buf[q], buf[k], pos, f, **kw)
        want = call()
        kw = dict(q_out=buf[qo], **({} if ko is None else dict(k_out=buf[ko])))
        if bad:
            with pytest.raises((ValueError, pbs.PbsError)):
                call(**kw)
            assert torch.equal(base, before)
        else:
            got = call(**kw)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            written = ids["qo"] | ids.get("ko", set())
            rest = torch.ones(base.numel(), dtype=torch.bool)
            rest[list(written)] = False
            assert torch.equal(base[rest.to(dev)], before[rest.to(dev)])
            taken += 1
    assert 100 < taken < 300


def test_rope_rows_that_run_backwards(dev):
    """Rows from the last to the first through the C ABI: into their own places,
    into places behind them, and over one another (refused)."""
    n, d = 6, 64
    f, pos = pbs.rope_freqs(d)[0].to(dev), torch.arange(n, dtype=torch.int32, device=dev)
    buf = torch.randn(3 * n, d, device=dev).to(BF16)
    before = buf.clone()
    want = pbs.rope(before[:n].flip(0)[None, None], None, pos, f)[0, 0].flip(0)

    def call(src, dst):  # from row src and to row dst down
        rows = [_lib.Rows(buf[x].data_ptr(), 0, 0, 0, -d) for x in (src, dst)]
        none = _lib.Rows(None, 0, 0, 0, 0)
        return pbs.lib().pbs_rope(*rows, 1, none, none, 0, pos.data_ptr(), 0, f.data_ptr(), 1.0, 1, n,
                                  d, d, 0, 0, _lib.BF16, torch.cuda.current_stream(dev).cuda_stream)

    assert call(n - 1, n + 1) == _lib.ERR_INVALID_ARG and call(n + 1, n - 1) == _lib.ERR_INVALID_ARG
    assert torch.equal(buf, before)
    assert call(n - 1, 2 * n - 1) == 0 and torch.equal(buf[n:2 * n], want)
    assert torch.equal(buf[:n], before[:n]) and torch.equal(buf[2 * n:], before[2 * n:])
    assert call(n - 1, n - 1) == 0 and torch.equal(buf[:n], want)


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("transpose", [False, True])
def test_angles_of_rope_in_fp32(transpose, layout, dev):
    """The cosine and sine of angles all over the turn, close to and on the
    quarters among them: an eighth of a turn, cut to 2^-34 turns, rounds to fp32
    within pi 2^-27, and sincospif is within a step of 2^-24. The oracle's angle comes from the same
    fp64 frequency, reduced in whole numbers."""
    n = 1 << 18
    x = torch.zeros(1, 1, n, 16, device=dev)
    at = (0, 8) if layout == "half" else (0, 1)
    x[..., at[0]] = 1
    pos = torch.arange(n, dtype=torch.int32)
    pos[n // 2:] = torch.randint(-2 ** 31, 2 ** 31 - 1, (n // 2,),
                                 generator=torch.Generator().manual_seed(1)).int()
    for turn in (0.11637718, 1 / 8 + 2.0 ** -30, 1 / 4, 1 / 4 - 2.0 ** -33, 0.5, 3 / 16):
        f = torch.zeros(8, dtype=torch.float64)
        f[0] = turn * 2 * math.pi
        y = f64(pbs.rope(x, None, pos.to(dev), f.to(dev), 1.0, layout, transpose))[0, 0]
        # turns of the frequency as the call gets it, a whole number of 2^-64 as it keeps them
        whole = int(math.floor((float(f[0]) * 0.15915494309189535 % 1.0) * 2.0 ** 64))
        rest = [p * whole % 2 ** 64 for p in pos.tolist()]
        part = np.array([(z + 2 ** 61) % 2 ** 62 - 2 ** 61 for z in rest], dtype=np.float64)
        a = part * (2 * math.pi / 2.0 ** 64)
        cs, sn = np.cos(a), np.sin(a)
        quarter = np.array([(z + 2 ** 61) // 2 ** 62 % 4 for z in rest])
        cos = np.choose(quarter, [cs, -sn, -cs, sn])
        sin = np.choose(quarter, [sn, cs, -sn, -cs]) * (-1 if transpose else 1)
        tol = math.pi * (2.0 ** -27 + 2.0 ** -33) + 2.0 ** -24
        assert np.abs(y[:, at[0]] - cos).max() <= tol and np.abs(y[:, at[1]] - sin).max() <= tol


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_under_autograd(layout, dtype, dev):
    """Gradients of q and k against the transposed map in fp64, against
    differences, of one of the two alone, of expanded inputs, through expanded
    and strided gradients, and of a gradient."""
    b, hq, hkv, n, d, rot = 2, 6, 2, 11, 64, 48
    f, pos = pbs.rope_freqs(rot)[0].to(dev), i32(np.arange(22).reshape(2, 11) * 991, dev)
    make = lambda h: torch.randn(b, h, n, d, device=dev).to(dtype)
    q, k, gq, gk = make(hq).requires_grad_(), make(hkv).requires_grad_(), make(hq), make(hkv)
    how = dict(gain=1.25, layout=layout)
    exact = lambda g: dec.rope(f64(g), pos.cpu().numpy(), f.cpu().numpy(), 1.25, layout, True)
    near = lambda x, g: (np.abs(f64(x) - exact(g)) <= rope_bound(f64(g), exact(g), 1.25, dtype,
                                                                 rot)).all()
    y, z = pbs.rope(q, k, pos, f, **how)
    plain = pbs.rope(q.detach(), k.detach(), pos, f, **how)
    assert torch.equal(y, plain[0]) and torch.equal(z, plain[1]) and not plain[0].requires_grad
    dq, dk = torch.autograd.grad((y, z), (q, k), (gq, gk), retain_graph=True)
    assert near(dq, gq) and near(dk, gk) and dq.dtype == dtype
    # one of the two alone; neither asked for
    assert torch.equal(torch.autograd.grad(y, q, gq, retain_graph=True)[0], dq)
    assert torch.equal(torch.autograd.grad(z, k, gk, retain_graph=True)[0], dk)
    assert torch.autograd.grad(y, k, gq, allow_unused=True)[0] is None
    assert torch.equal(torch.autograd.grad(pbs.rope(q, None, pos, f, **how), q, gq)[0], dq)
    y, z = pbs.rope(q.detach(), k, pos, f, **how)
    assert torch.equal(torch.autograd.grad(z, k, gk)[0], dk)
    assert not y.requires_grad or torch.autograd.grad(y, k, gq, allow_unused=True)[0] is None
    # gradients that repeat an element, or lie across
    one = torch.ones((), dtype=dtype, device=dev)
    dq1, = torch.autograd.grad(pbs.rope(q, None, pos, f, **how).sum(), q)
    assert near(dq1, one.expand(b, hq, n, d))
    across = torch.randn(b, hq, d, n, device=dev).to(dtype).transpose(2, 3)
    assert near(torch.autograd.grad(pbs.rope(q, None, pos, f, **how), q, across)[0], across)
    # heads and a batch that share an input: the sums of their gradients
    s = make(hq)[:1, :1].requires_grad_()
    ds, = torch.autograd.grad(pbs.rope(s.expand(b, hq, n, d), None, pos, f, **how), s, gq)
    parts = f64(dq).sum((0, 1), keepdims=True)
    # torch sums b hq rounded parts in fp32 and rounds once for the heads, once for the batch
    size = np.abs(f64(dq)).sum((0, 1), keepdims=True)
    assert (np.abs(f64(ds) - parts) <= 2.5 * torch.finfo(dtype).eps * size + b * hq * 2.0 ** -23
            * size).all()
    if dtype is FP32:  # along a direction: the map is linear
        v = make(hq)
        diff = f64(pbs.rope(q.detach() + v, None, pos, f, **how)) - f64(plain[0])
        x, w = (diff * f64(gq)).sum(), (f64(v) * f64(dq)).sum()
        size = sum((np.abs(f64(t)) * np.abs(f64(gq))).sum() for t in (q, v))
        assert abs(x - w) <= 8 * 2.0 ** -23 * 1.25 * 2 * 6 * size
    # the gradient of a gradient is the map itself
    g = gq.clone().requires_grad_()
    dq, = torch.autograd.grad(pbs.rope(q, None, pos, f, **how), q, g, create_graph=True)
    assert torch.equal(torch.autograd.grad(dq, g, q.detach())[0], plain[0])


def test_rope_under_autograd_refuses_and_captures(dev):
    q = torch.randn(1, 4, 8, 64, device=dev, requires_grad=True)
    f, pos = pbs.rope_freqs(64)[0].to(dev), torch.arange(8, dtype=torch.int32, device=dev)
    for kw in (dict(q_out=torch.empty_like(q)), dict(inv_freq=f.clone().requires_grad_()),
               dict(k=q.detach(), k_out=torch.empty_like(q))):
        with pytest.raises(ValueError):
            pbs.rope(**dict(dict(q=q, k=None, pos=pos, inv_freq=f), **kw))
    with torch.no_grad():
        y = torch.empty_like(q)
        assert pbs.rope(q, None, pos, f, q_out=y) is y and not y.requires_grad
    assert not pbs.rope(q.detach(), None, pos, f).requires_grad
    with pytest.raises(ValueError):
        pbs.rope(q.detach(), None, pos, f, q_out=torch.empty_like(q).requires_grad_())
    # positions that change before the backward pass are noticed
    z = pbs.rope(q, None, pos, f)
    pos += 1
    with pytest.raises(RuntimeError):
        z.sum().backward()
    del z
    # forward and backward as one graph
    x, g = torch.randn_like(q), torch.randn_like(q)

    def step():
        leaf = x.detach().requires_grad_()
        y = pbs.rope(leaf, None, pos, f)
        return y.detach(), torch.autograd.grad(y, leaf, g)[0]

    side, graph = torch.cuda.Stream(dev), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(torch.randn_like(x)), g.copy_(torch.randn_like(g)), pos.add_(100)
    graph.replay()
    want = step()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


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


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("tree", [1, 8, 64])
def test_fp16_keeps_small_weights(tree, d, dev):
    """One key 2^25 above the 131071 others, which are 0.36 % of the softmax
    together, in batches whose CTAs work through whole items (300 sequences on
    the same pages). With the one's V row 0 the output is those 0.36 % alone. The
    result rounds by half a step, the weights by half a step of theirs; an item
    is summed in one, two (up to 128 rows), four or eight streams (16 rows: the
    warps of a CTA, d = 64 or 128), where each product may be a step within 2^-23
    of the sum so far (fp32, cut off: the tensor cores' sums need not round)."""
    g, b, n, page = 4, 300, 131072 - tree, 64
    pages = 131072 // page
    k = torch.zeros(pages, 1, page, d, device=dev).half()
    v = (0.5 + torch.rand(k.shape, generator=torch.Generator(dev).manual_seed(d), device=dev)).half()
    table = torch.arange(pages, device=dev, dtype=torch.int32).expand(b, pages).contiguous()
    q = torch.zeros(b, g, tree, d, device=dev).half()
    q[..., 0] = 1
    steps = 131072 / {1: d // 16, 8: 2, 64: 1}[tree] * 2.0 ** -23
    for at in (3, n // 2, n - 70):
        k.zero_()
        k[at // page, 0, at % page, 0] = 25.1 * math.log(2)
        e = k.view(-1, d)[:, 0].double().exp()
        total = e.cumsum(0)[n:]
        for alone in (False, True):
            vv = v.clone()
            if alone:
                vv[at // page, 0, at % page] = 0
            o, lse = pbs.tree_attn(q, k, vv, table, i32([n] * b, dev), scale=1.0, lse=True)
            want = (e[:, None] * vv.view(-1, d).double()).cumsum(0)[n:] / total[:, None]
            tol = 2.0 ** -11 * (2 if alone else 1.004) + steps
            assert ((o.double() / want - 1).abs().max()) <= tol
            assert ((lse.double() - total.log()).abs().max()) <= steps + 18 * 2.0 ** -23


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("tree,g", [(1, 4), (8, 4), (64, 4)])
def test_huge_logits_pick_the_largest(tree, g, dtype, dev):
    """Logits of up to 3e8, where a step of fp32 is 32: every row is the V row
    of its largest logit, and finite."""
    d, n = 64, 700
    k = torch.zeros(12, 2, 64, d, device=dev)
    at = torch.randperm(n, generator=torch.Generator().manual_seed(tree))[:16].to(dev)
    k[at // 64, :, at % 64, torch.arange(16, device=dev)] = 30.0
    k, v = k.to(dtype), torch.randn(k.shape, device=dev).to(dtype)
    pick = torch.randint(0, 16, (1, 2 * g, tree), device=dev)
    q = torch.nn.functional.one_hot(pick, d).to(dtype) * 20
    table = torch.arange(12, device=dev, dtype=torch.int32)[None]
    for scale in (1e3, 1e5, 5e5):
        o = pbs.tree_attn(q, k, v, table, i32([n], dev), scale=scale)
        where = at[pick]
        head = (torch.arange(2 * g, device=dev) // g)[None, :, None].expand_as(pick)
        want = v[where // 64, head, where % 64]
        assert ((o.float() - want.float()).abs() <= 2.0 ** -9 * want.float().abs()).all()


def test_tree_attn_outputs_and_workspaces_over_other_tensors(dev):
    t = Tree(dev, BF16, 64, 16, 1, [20], [2], 2, junk=False)
    c = _lib.Cache(1, t.k.shape[0], 1, 16, 64, 1, t.table.shape[1])
    need = pbs.lib().pbs_tree_workspace_bytes(2, 2, c)
    buf = torch.zeros(need + 8192, dtype=torch.uint8, device=dev)
    q = torch.randn(1, 2, 2, 64, device=dev).to(BF16)
    start, mask = i32([20], dev), i32([[[1], [3]]], dev)
    want = pbs.tree_attn(q, t.k, t.v, t.table, start, mask)
    ws, rest = buf[:need], buf[-(-need // 16) * 16:]
    out = rest[:512].view(BF16).view(q.shape)
    assert torch.equal(pbs.tree_attn(q, t.k, t.v, t.table, start, mask, out=out, ws=ws), want)
    ints = ws[:8].view(torch.int32)
    for kw in (dict(q=ws[:512].view(BF16).view(q.shape)), dict(out=ws[:512].view(BF16).view(q.shape)),
               dict(k_pages=t.k, v_pages=buf[1024:1024 + 2 * t.v.numel()].view(BF16).view(t.v.shape)),
               dict(start=ints[:1]), dict(count=ints[:1]), dict(mask=ints.view(1, 2, 1)),
               dict(table=ints.view(1, 2))):
        kw = dict(dict(q=q, k_pages=t.k, v_pages=t.v, table=t.table, start=start, mask=mask), **kw)
        with pytest.raises((ValueError, pbs.PbsError)):
            pbs.tree_attn(**kw, ws=ws)
    over = out.view(torch.int32)
    for kw in (dict(start=over.view(-1)[:1]), dict(mask=over.view(-1)[:2].view(1, 2, 1)),
               dict(table=over.view(-1)[:2].view(1, 2))):
        kw = dict(dict(table=t.table, start=start, mask=mask), **kw)
        with pytest.raises((ValueError, pbs.PbsError)):
            pbs.tree_attn(q, t.k, t.v, out=out, **kw)
