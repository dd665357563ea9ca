"""Decoding operators beside the prefill path, as they are timed and compared.

Rotary positions, the page table of a key/value cache (fork, reserve with
copy-on-write, append, copy, accept, compact, trim), and attention for trees
of drafted tokens over that cache (one drafted token is plain decoding).

With ``own`` false ``run`` computes each operator from elementary torch
operations in fp32 (angles in fp64); with ``own`` true it makes the library
calls. Shapes follow the package's workloads: 32 query heads on 8 KV heads
with d = 128, contexts of 8192 to 131072 tokens, and d = 64.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a batch: q and k of one new token per sequence
        dict(name="rope_step", op="rope", b=16, n=1, hq=32, hkv=8, d=128, rot=128, layout="half",
             base=500000.0, far=131072, scaled=True, transpose=False, dtype="bf16"),
        # the prompt of a 32K prefill, q and k as slices of one projection
        dict(name="rope_prompt", op="rope", b=1, n=32768, hq=32, hkv=8, d=128, rot=128,
             layout="half", base=500000.0, far=0, scaled=True, transpose=False, dtype="bf16"),
        # gradients of a batch of odd length, half of each head rotated in pairs
        dict(name="rope_grad", op="rope", b=3, n=1021, hq=12, hkv=3, d=128, rot=64,
             layout="pairs", base=10000.0, far=4096, scaled=False, transpose=True, dtype="fp32"),
        # beams: prompts forked, each copy extended by a few tokens, then dropped
        dict(name="pages_beam", op="beam", seqs=16, most=2000, new=5, layers=2, hkv=8, d=128,
             page=64, dtype="bf16", mix=1),
        # a prefix moved to other pages in all layers (swapping, defragmenting by hand)
        dict(name="pages_copy", op="copy", pairs=96, pages=256, layers=32, hkv=8, d=128, page=64,
             dtype="bf16"),
        # the accepted drafts of a batch moved behind their prefixes, in all layers
        dict(name="pages_accept", op="accept", seqs=32, most=700, tree=32, layers=32, hkv=8,
             d=128, page=32, dtype="bf16", mix=2),
        # a half-empty pool compacted to its low pages
        dict(name="pages_compact", op="compact", pages=1023, share=0.5, layers=4, hkv=4, d=128,
             page=32, seqs=24, dtype="bf16", mix=3),
        # one new token of one sequence at 8K
        dict(name="tree_single", op="tree", b=1, tree=1, least=8191, most=8191, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", mix=4),
        # one new token of every sequence of a ragged batch
        dict(name="tree_batch", op="tree", b=48, tree=1, least=100, most=32768, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", mix=5),
        # trees of 64 drafts verified over contexts up to 32K
        dict(name="tree_drafts", op="tree", b=8, tree=64, least=8192, most=32768, hq=32, hkv=8,
             d=128, page=128, dtype="bf16", mix=6),
        # odd sizes: fp16, d = 64, three query heads a group, small pages, short prefixes
        dict(name="tree_odd", op="tree", b=5, tree=13, least=0, most=1500, hq=6, hkv=2, d=64,
             page=16, dtype="fp16", mix=7),
        # a few drafts over one 128K context
        dict(name="tree_long", op="tree", b=1, tree=7, least=131072, most=131072, hq=32, hkv=8,
             d=128, page=64, dtype="bf16", mix=8),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "beam", "copy", "accept", "compact", "tree", "tree", "tree"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    mix = rng.randrange(1 << 20)
    if op == "rope":
        n, g = _log(rng, 1, 32768), rng.choice([1, 2, 3, 4])
        b = rng.randint(1, max(1, min(32, 32768 // n)))
        return dict(op=op, b=b, n=n, hq=hkv * g, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2]),
                    layout=rng.choice(["half", "pairs"]), base=rng.choice([10000.0, 500000.0]),
                    far=rng.choice([0, 4096, 131072]), scaled=rng.random() < 0.5,
                    transpose=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "beam":
        return dict(op=op, seqs=rng.randint(1, 48), most=_log(rng, 1, 2000), new=rng.randint(1, 40),
                    layers=rng.randint(1, 4), hkv=hkv, d=d, page=page, dtype=dtype, mix=mix)
    if op == "copy":
        layers = rng.randint(1, 32)
        pairs = _log(rng, 1, max(1, min(1000, 96 * 32 * 8 * 64 * 128 // (layers * hkv * page * d))))
        return dict(op=op, pairs=pairs, pages=2 * pairs + rng.randint(1, 64), layers=layers,
                    hkv=hkv, d=d, page=page, dtype=dtype)
    if op == "accept":
        return dict(op=op, seqs=rng.randint(1, 32), most=_log(rng, 1, 700),
                    tree=_log(rng, 1, 64), layers=rng.randint(1, 16), hkv=hkv, d=d, page=page,
                    dtype=dtype, mix=mix)
    if op == "compact":
        return dict(op=op, pages=_log(rng, 40, 1500), share=rng.uniform(0.1, 0.95),
                    layers=rng.randint(1, 4), hkv=min(hkv, 4), d=d, page=rng.choice([16, 32]),
                    seqs=rng.randint(2, 24), dtype=dtype, mix=mix)
    most, g = _log(rng, 1, 131072), rng.choice([1, 2, 3, 4, 8])
    b = rng.randint(1, max(1, min(48, 400000 // most)))
    tree = rng.choice([1, 1, 2, 5, _log(rng, 1, 100)])
    tree = max(1, min(tree, 400000000 // (b * most * hkv * g)))
    return dict(op="tree", b=b, tree=tree, least=rng.choice([0, most // 2, most]), most=most,
                hq=hkv * g, hkv=hkv, d=d, page=page, dtype=dtype, mix=mix)


# ------------------------------------------------------------ what follows from a case
def _lengths(c):
    """Tokens cached per sequence, the drafts of each, and the drafts' parents."""
    r = random.Random(c["mix"])
    b, t = c["b"], c["tree"]
    start = [r.randint(c["least"], c["most"]) for _ in range(b)]
    if t == 1:
        return start, [1] * b, [[-1]] * b
    count = [t if i == 0 else r.randint(t // 2, t) for i in range(b)]
    if b > 3:
        count[1] = 0
    # each draft continues an earlier one, or the cached prefix itself
    parents = [[-1 if i == 0 or r.random() < 0.1 else r.randrange(max(0, i - 8), i)
                for i in range(t)] for _ in range(b)]
    return start, count, parents


def _ceil(a, b):
    return -(-a // b)


def _beam(c):
    r = random.Random(c["mix"])
    return [r.randint(1, c["most"]) for _ in range(c["seqs"])]


def _accept(c):
    """Prefix lengths and accepted drafts. A draft that is not in place already
    comes from behind the accepted ones, so that a pass can be made again."""
    r = random.Random(c["mix"])
    t, start, path, count = c["tree"], [], [], []
    for _ in range(c["seqs"]):
        n = r.randint(1, max(1, t // 3))
        same = r.randint(0, n)
        rest = sorted(r.sample(range(n, t), min(n - same, t - n)))
        p = list(range(n - len(rest))) + rest
        start.append(r.randint(1, c["most"]))
        path.append(p + [0] * (t - len(p)))
        count.append(len(p))
    return start, path, count


def _compact(c):
    """A table whose rows hold pages all over the pool; some pages have two holders."""
    r = random.Random(c["mix"])
    live = r.sample(range(c["pages"]), max(c["seqs"], int(c["share"] * c["pages"])))
    rows = [live[i::c["seqs"]] for i in range(c["seqs"])]
    if len(rows) > 1:  # the second sequence shares the first one's first pages
        k = len(rows[0]) // 2
        rows[1] = rows[0][:k] + rows[1]
    m = max(len(x) for x in rows) + 3
    refs = [0] * c["pages"]
    for x in rows:
        for p in x:
            refs[p] += 1
    return [x + [-1] * (m - len(x)) for x in rows], refs


def work(c):
    e = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "rope":
        x = c["b"] * c["n"] * (c["hq"] + c["hkv"])
        return {"bytes": 2 * x * c["d"] * e + 4 * c["b"] * c["n"] + 4 * c["rot"],
                "flops": 3 * x * c["rot"]}
    row = c["hkv"] * c["d"] * e * 2  # a token's key and value in one layer
    if c["op"] == "beam":
        lens = _beam(c)
        partial = sum(n % c["page"] for n in lens)
        pages = sum(_ceil(n, c["page"]) for n in lens)
        rows = c["layers"] * row * 2
        return {"bytes": rows * (partial + c["new"] * len(lens)) + 16 * pages, "flops": 0}
    if c["op"] == "copy":
        return {"bytes": 2 * c["pairs"] * c["layers"] * row * c["page"], "flops": 0}
    if c["op"] == "accept":
        _, path, count = _accept(c)
        moved = sum(1 for p, n in zip(path, count) for i in range(n) if p[i] != i)
        return {"bytes": 2 * moved * c["layers"] * row + 4 * c["seqs"] * c["tree"], "flops": 0}
    if c["op"] == "compact":
        table, refs = _compact(c)
        n = sum(x > 0 for x in refs)
        moved = sum(x > 0 for x in refs[n:])
        return {"bytes": 2 * moved * c["layers"] * row * c["page"] + 8 * len(refs)
                + 8 * len(table) * len(table[0]), "flops": 0}
    start, count, _ = _lengths(c)
    keys = sum(s + n for s, n in zip(start, count) if n)
    rows = c["b"] * c["hq"] * c["tree"]
    return {"bytes": keys * row + rows * (2 * c["d"] * e + 4),
            "flops": 4 * c["d"] * c["hq"] * sum(n * (s + 1) for s, n in zip(start, count))}


# ------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(DEV).manual_seed(1000003 * (seed + 1))


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _freqs(c):
    """Angle per position of each rotated pair, and the factor on cos and sin.
    Scaled: low frequencies stretched by 8, high ones kept, a ramp between."""
    f = [c["base"] ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)]
    if not c["scaled"]:
        return torch.tensor(f, dtype=torch.float64, device=DEV), 1.0
    turns = [8192 * x / (2 * math.pi) for x in f]
    keep = [min(1.0, max(0.0, (t - 1.0) / 3.0)) for t in turns]
    f = [x * (k + (1 - k) / 8.0) for x, k in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64, device=DEV), 0.1 * math.log(8.0) + 1.0


def _pools(c, pages, gen):
    shape = (c["layers"], pages, c["hkv"], c["page"], c["d"])
    return [torch.randn(shape, generator=gen, device=DEV, dtype=TYPES[c["dtype"]])
            for _ in range(2)]


def _table(counts, width, pages, seed):
    """Rows of distinct pages in random order, counts[i] of them in row i."""
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    rows, at = [], 0
    for n in counts:
        rows.append(perm[at:at + n] + [-1] * (width - n))
        at += n
    return rows


def prepare(c, seed):
    gen = _gen(seed)
    t = TYPES[c["dtype"]]
    s = {"c": c}
    if c["op"] == "rope":
        b, n, hq, hkv, d = (c[x] for x in ("b", "n", "hq", "hkv", "d"))
        qkv = torch.randn(b, n, hq + 2 * hkv, d, generator=gen, device=DEV, dtype=t)
        s["q"] = qkv[:, :, :hq].transpose(1, 2)
        s["k"] = qkv[:, :, hq:hq + hkv].transpose(1, 2)
        first = torch.randint(0, c["far"] + 1, (b, 1), generator=gen, device=DEV)
        s["pos"] = (first + torch.arange(n, device=DEV)).to(torch.int32)
        s["inv_freq"], s["gain"] = _freqs(c)
        return s
    if c["op"] == "beam":
        lens, page, new = _beam(c), c["page"], c["new"]
        m = _ceil(c["most"] + new, page) + 1
        held = sum(_ceil(n, page) for n in lens)
        pages = held + len(lens) * (_ceil(new, page) + 2) + 7
        s["k"], s["v"] = _pools(c, pages, gen)
        rows = _table([_ceil(n, page) for n in lens] + [0] * len(lens), m, pages, seed)
        s["table"] = _i32(rows)
        refs = torch.zeros(pages, dtype=torch.int32)
        for r in rows:
            for p in r:
                if p >= 0:
                    refs[p] = 1
        s["refs"], k = refs.to(DEV), len(lens)
        s["lens"] = _i32(lens + [0] * k)
        s["src"], s["dst"] = _i32(range(k)), _i32(range(k, 2 * k))
        s["want"] = _i32([0] * k + [n + new for n in lens])
        s["start"] = _i32([0] * k + lens)
        s["count"] = _i32([0] * k + [new] * k)
        s["keep"] = _i32([-1] * k + [0] * k)
        shape = (c["layers"], 2 * k, c["hkv"], new, c["d"])
        s["new_k"] = torch.randn(shape, generator=gen, device=DEV, dtype=t)
        s["new_v"] = torch.randn(shape, generator=gen, device=DEV, dtype=t)
        return s
    if c["op"] == "copy":
        s["k"], s["v"] = _pools(c, c["pages"], gen)
        perm = torch.randperm(c["pages"], generator=torch.Generator().manual_seed(seed))
        s["src"] = perm[:c["pairs"]].to(DEV, torch.int32)
        s["dst"] = perm[c["pairs"]:2 * c["pairs"]].to(DEV, torch.int32)
        return s
    if c["op"] == "accept":
        start, path, count = _accept(c)
        need = [_ceil(n + c["tree"], c["page"]) for n in start]
        s["k"], s["v"] = _pools(c, sum(need) + 3, gen)
        s["table"] = _i32(_table(need, max(need) + 1, sum(need) + 3, seed))
        s["start"], s["path"], s["count"] = _i32(start), _i32(path), _i32(count)
        s["lens"] = s["start"] + c["tree"]
        return s
    if c["op"] == "compact":
        table, refs = _compact(c)
        s["k"], s["v"] = _pools(c, c["pages"], gen)
        s["table0"], s["refs0"] = _i32(table), _i32(refs)
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
        return s
    start, count, parents = _lengths(c)
    need = [_ceil(a + n, c["page"]) for a, n in zip(start, count)]
    pages = sum(need) + 5
    shape = (pages, c["hkv"], c["page"], c["d"])
    s["k"] = torch.randn(shape, generator=gen, device=DEV, dtype=t)
    s["v"] = torch.randn(shape, generator=gen, device=DEV, dtype=t)
    s["table"] = _i32(_table(need, max(need + [1]), pages, seed))
    q = 2.5 * torch.randn(c["b"], c["tree"], c["hq"], c["d"], generator=gen, device=DEV)
    s["q"] = q.to(t).transpose(1, 2)
    s["start"], s["count"], s["parents"] = _i32(start), _i32(count), _i32(parents)
    return s


# ------------------------------------------------------------ one pass
def run(s):
    c = s["c"]
    if own:
        return _own(s, c)
    return _PLAIN[c["op"]](s, c)


def _own(s, c):
    import long_context_sparse_segment_b200 as pbs
    if c["op"] == "rope":
        return pbs.rope(s["q"], s["k"], s["pos"], s["inv_freq"], gain=s["gain"],
                        layout=c["layout"], transpose=c["transpose"])
    if c["op"] == "beam":
        page = c["page"]
        pbs.cache_fork(s["table"], s["refs"], s["lens"], s["src"], s["dst"], page)
        src, dst = pbs.cache_reserve(s["table"], s["refs"], s["lens"], s["want"], page)
        pbs.cache_copy(s["k"], s["v"], src, dst)
        pbs.cache_append(s["new_k"], s["new_v"], s["k"], s["v"], s["table"], s["start"],
                         count=s["count"])
        pbs.cache_trim(s["table"], s["refs"], s["lens"], s["keep"], page)
        return s["k"], s["v"], s["table"], s["refs"], s["lens"], src, dst
    if c["op"] == "copy":
        pbs.cache_copy(s["k"], s["v"], s["src"], s["dst"])
        return s["k"], s["v"]
    if c["op"] == "accept":
        pbs.cache_accept(s["k"], s["v"], s["table"], s["start"], s["path"], count=s["count"],
                         lens=s["lens"])
        return s["k"], s["v"], s["lens"]
    if c["op"] == "compact":
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        src, dst = pbs.cache_compact(s["k"], s["v"], s["table"], s["refs"])
        return s["k"], s["v"], s["table"], s["refs"], src, dst
    if c["tree"] == 1:
        return pbs.tree_attn(s["q"], s["k"], s["v"], s["table"], s["start"], lse=True)
    mask, depth = pbs.tree_mask(s["parents"])
    o, lse = pbs.tree_attn(s["q"], s["k"], s["v"], s["table"], s["start"], mask=mask,
                           count=s["count"], lse=True)
    return o, lse, mask, depth


def _plain_rope(s, c):
    angle = s["pos"].double()[:, None, :, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["gain"]).float(), (angle.sin() * s["gain"]).float()
    sin = -sin if c["transpose"] else sin
    return _rotate(s["q"], cos, sin, c), _rotate(s["k"], cos, sin, c)


def _rotate(x, cos, sin, c):
    y, r = x.float(), c["rot"]
    if c["layout"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        z = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., r:]], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        z = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        z = torch.cat([z, y[..., r:]], -1)
    return z.to(x.dtype)


def _plain_beam(s, c):
    table, refs, lens, page = s["table"], s["refs"], s["lens"], c["page"]
    pages, (rows, m) = refs.numel(), table.shape
    col = torch.arange(m, device=DEV)
    src, dst = s["src"].long(), s["dst"].long()
    # fork: the copies hold the same pages
    held = torch.where(col < -(-lens[src] // page)[:, None], table[src], -1)
    table[dst] = held
    lens[dst] = lens[src]
    one = (held >= 0).to(torch.int32).flatten()
    refs.index_add_(0, held.clamp(min=0).flatten(), one)
    # reserve: new pages for what will be written; a shared page that holds tokens is copied
    first, last = lens // page, -(-s["want"] // page)
    write = (col >= first[:, None]) & (col < last[:, None]) & (s["want"] > lens)[:, None]
    same = (table[:, None] == table[None]) & write[None] & (table >= 0)[:, None]
    before = torch.ones(rows, rows, device=DEV).tril(-1).bool()
    earlier = (same & before[:, :, None]).sum(1)
    shared = (table >= 0) & (refs[table.clamp(min=0).long()] - earlier > 1)
    fresh = write & ((table < 0) | shared)
    order = torch.argsort((refs > 0).to(torch.int32), stable=True)
    page_of = order[(fresh.flatten().cumsum(0) - 1).clamp(min=0)].view(rows, m).to(torch.int32)
    copied = fresh & shared & (col == first[:, None]) & (lens % page > 0)[:, None]
    at = first.clamp(max=m - 1).long()[:, None]
    moved = copied.gather(1, at)[:, 0]
    from_page = torch.where(moved, table.gather(1, at)[:, 0], -1)
    to_page = torch.where(moved, page_of.gather(1, at)[:, 0], -1)
    old = fresh & shared
    refs.index_add_(0, table.clamp(min=0).flatten(), -old.to(torch.int32).flatten())
    refs.index_add_(0, page_of.flatten(), fresh.to(torch.int32).flatten())
    table.copy_(torch.where(fresh, page_of, table))
    # copy the shared pages, write the new tokens
    s["k"][:, to_page[moved]] = s["k"][:, from_page[moved]]
    s["v"][:, to_page[moved]] = s["v"][:, from_page[moved]]
    i = torch.arange(c["new"], device=DEV)
    valid = i < s["count"][:, None]
    pos = (s["start"][:, None] + i).long()
    p = table.gather(1, (pos // page).clamp(max=m - 1))[valid].long()
    s["k"][:, p, :, (pos % page)[valid]] = s["new_k"].transpose(2, 3)[:, valid].transpose(0, 1)
    s["v"][:, p, :, (pos % page)[valid]] = s["new_v"].transpose(2, 3)[:, valid].transpose(0, 1)
    # trim: the copies are dropped
    keep = s["keep"]
    lens.copy_(torch.where(keep >= 0, torch.minimum(lens, keep), lens))
    gone = (col >= -(-lens // page)[:, None]) & (keep >= 0)[:, None] & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).flatten(), -gone.to(torch.int32).flatten())
    table.copy_(torch.where(gone, -1, table))
    return s["k"], s["v"], table, refs, lens, from_page, to_page


def _plain_copy(s, c):
    src, dst = s["src"].long(), s["dst"].long()
    s["k"][:, dst] = s["k"][:, src]
    s["v"][:, dst] = s["v"][:, src]
    return s["k"], s["v"]


def _plain_accept(s, c):
    i = torch.arange(c["tree"], device=DEV)
    path = torch.where(i < s["count"][:, None], s["path"], i)
    a, b = (s["start"][:, None] + path).long(), (s["start"][:, None] + i).long()
    page = c["page"]
    pa, pb = s["table"].gather(1, a // page).long(), s["table"].gather(1, b // page).long()
    s["k"][:, pb, :, b % page] = s["k"][:, pa, :, a % page]
    s["v"][:, pb, :, b % page] = s["v"][:, pa, :, a % page]
    s["lens"].copy_(s["start"] + s["count"])
    return s["k"], s["v"], s["lens"]


def _plain_compact(s, c):
    table, refs = s["table"], s["refs"]
    table.copy_(s["table0"])
    refs.copy_(s["refs0"])
    n = (refs > 0).sum()
    at = torch.arange(refs.numel(), device=DEV)
    mover = torch.nonzero((refs > 0) & (at >= n))[:, 0]
    hole = torch.nonzero((refs == 0) & (at < n))[:, 0]
    s["k"][:, hole] = s["k"][:, mover]
    s["v"][:, hole] = s["v"][:, mover]
    to = at.to(torch.int32)
    to[mover] = hole.to(torch.int32)
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    refs[hole] = refs[mover]
    refs[mover] = 0
    src, dst = torch.full_like(refs, -1), torch.full_like(refs, -1)
    src[:mover.numel()], dst[:mover.numel()] = mover.to(torch.int32), hole.to(torch.int32)
    return s["k"], s["v"], table, refs, src, dst


def _plain_tree(s, c):
    b, t, hkv, d, page = c["b"], c["tree"], c["hkv"], c["d"], c["page"]
    g = c["hq"] // hkv
    # draft i sees draft j when j is i or one of its ancestors
    up = (s["parents"][:, :, None] == torch.arange(t, device=DEV)).double()
    sees = torch.linalg.matrix_power(up + torch.eye(t, device=DEV, dtype=torch.double), t) > 0.5
    cap = s["table"].shape[1] * page
    at = s["table"].clamp(min=0).long()
    k = s["k"][at].transpose(1, 2).reshape(b, hkv, cap, d).float()
    v = s["v"][at].transpose(1, 2).reshape(b, hkv, cap, d).float()
    j = torch.arange(cap, device=DEV)
    start, count = s["start"][:, None], s["count"][:, None]
    draft = (j - start).clamp(0, t - 1).long()
    vis = sees.gather(2, draft[:, None].expand(b, t, cap)) & ((j < start + count)[:, None])
    vis = torch.where((j < start)[:, None], True, vis)
    vis = vis & (torch.arange(t, device=DEV) < count)[:, :, None]
    x = (s["q"].float() / math.sqrt(d)).reshape(b, hkv, g * t, d) @ k.transpose(2, 3)
    x = x.view(b, hkv, g, t, cap).masked_fill(~vis[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (x - top).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hkv, g * t, cap) @ v).view(b, hkv, g, t, d) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0].view(b, c["hq"], t)
    o = o.view(b, c["hq"], t, d).to(s["q"].dtype)
    lse = torch.where((torch.arange(t, device=DEV) < count)[:, None], lse, 0.0)
    if t == 1:
        return o, lse
    words = _ceil(t, 32)
    bit = torch.zeros(b, t, words * 32, dtype=torch.int64, device=DEV)
    bit[..., :t] = sees
    mask = (bit.view(b, t, words, 32) << torch.arange(32, device=DEV)).sum(-1)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    return o, lse, mask, (sees.sum(-1) - 1).to(torch.int32)


_PLAIN = {"rope": _plain_rope, "beam": _plain_beam, "copy": _plain_copy,
          "accept": _plain_accept, "compact": _plain_compact, "tree": _plain_tree}


# ------------------------------------------------------------ in 64 bits
def exact(c, seed):
    return _EXACT[c["op"]](prepare(c, seed), c)


def _exact_rope(s, c):
    w = torch.outer(s["pos"].flatten().double(), s["inv_freq"])
    turn = s["gain"] * torch.complex(w.cos(), -w.sin() if c["transpose"] else w.sin())
    turn = turn.view(c["b"], 1, c["n"], c["rot"] // 2)
    out = []
    for x in (s["q"], s["k"]):
        y, h = x.double().clone(), c["rot"] // 2
        lo, hi = (slice(0, h), slice(h, 2 * h)) if c["layout"] == "half" else \
            (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
        z = torch.complex(y[..., lo].clone(), y[..., hi].clone()) * turn
        y[..., lo], y[..., hi] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_beam(s, c):
    page, lens = c["page"], s["lens"].tolist()
    table, refs = s["table"].tolist(), s["refs"].tolist()
    src, dst = [-1] * len(lens), [-1] * len(lens)
    k = len(lens) // 2
    free = [p for p, r in enumerate(refs) if r == 0]
    for i in range(k):  # each copy takes a page of its own for its open page, then new ones
        n, row, at = lens[i], table[i], k + i
        have = _ceil(n, page)
        own_pages = list(row[:have])
        if n % page:
            src[at], dst[at] = row[have - 1], free.pop(0)
            for pool in (s["k"], s["v"]):
                pool[:, dst[at]] = pool[:, src[at]]
            own_pages[-1] = dst[at]
        while len(own_pages) * page < n + c["new"]:
            own_pages.append(free.pop(0))
        for x in range(c["new"]):
            p, o = own_pages[(n + x) // page], (n + x) % page
            s["k"][:, p, :, o] = s["new_k"][:, at, :, x]
            s["v"][:, p, :, o] = s["new_v"][:, at, :, x]
    return (s["k"], s["v"], s["table"], s["refs"], s["lens"], _i32(src), _i32(dst))


def _exact_copy(s, c):
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        s["k"][:, b], s["v"][:, b] = s["k"][:, a].clone(), s["v"][:, a].clone()
    return s["k"], s["v"]


def _exact_accept(s, c):
    table, page = s["table"].tolist(), c["page"]
    start, path, count = s["start"].tolist(), s["path"].tolist(), s["count"].tolist()
    for i, n in enumerate(count):
        for x in range(n):
            a, b = start[i] + path[i][x], start[i] + x
            if a != b:
                for pool in (s["k"], s["v"]):
                    pool[:, table[i][b // page], :, b % page] = \
                        pool[:, table[i][a // page], :, a % page].clone()
    return s["k"], s["v"], _i32([a + n for a, n in zip(start, count)])


def _exact_compact(s, c):
    table, refs = s["table0"].tolist(), s["refs0"].tolist()
    n = sum(r > 0 for r in refs)
    holes = [p for p in range(n) if refs[p] == 0]
    to, src, dst = {}, [-1] * len(refs), [-1] * len(refs)
    for p in range(n, len(refs)):
        if refs[p]:
            src[len(to)], dst[len(to)] = p, holes[len(to)]
            to[p] = holes[len(to)]
    for a, b in to.items():
        for pool in (s["k"], s["v"]):
            pool[:, b] = pool[:, a].clone()
        refs[a], refs[b] = 0, refs[a]
    table = [[to.get(p, p) for p in row] for row in table]
    return s["k"], s["v"], _i32(table), _i32(refs), _i32(src), _i32(dst)


def _exact_tree(s, c):
    b, t, g, d, page = c["b"], c["tree"], c["hq"] // c["hkv"], c["d"], c["page"]
    start, count, parents = _lengths(c)
    o = torch.zeros(b, c["hq"], t, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(b, c["hq"], t, dtype=torch.float64, device=DEV)
    seen = [[] for _ in range(b)]
    for i in range(b):
        for r in range(t):
            p = parents[i][r]
            seen[i].append((seen[i][p] if p >= 0 else []) + [r])
        n = start[i] + count[i]
        if not count[i]:
            continue
        pages = s["table"][i, :_ceil(n, page)].long()
        hide = torch.zeros(t, n, dtype=torch.float64)
        for r in range(count[i]):
            hide[r, start[i]:] = -math.inf
            for x in seen[i][r]:
                hide[r, start[i] + x] = 0.0
        hide = hide[:count[i]].to(DEV)
        for h in range(c["hkv"]):
            k = s["k"][pages, h].reshape(-1, d)[:n].double()
            v = s["v"][pages, h].reshape(-1, d)[:n].double()
            for x in range(h * g, h * g + g):
                a = s["q"][i, x, :count[i]].double() @ k.T / d ** 0.5 + hide
                lse[i, x, :count[i]] = torch.logsumexp(a, -1)
                o[i, x, :count[i]] = torch.softmax(a, -1) @ v
    if t == 1:
        return o, lse
    mask = [[[sum(1 << (x & 31) for x in row if x >> 5 == w) for w in range(_ceil(t, 32))]
             for row in rows] for rows in seen]
    mask = torch.tensor(mask, dtype=torch.int64, device=DEV)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    return o, lse, mask, _i32([[len(row) - 1 for row in rows] for rows in seen])


_EXACT = {"rope": _exact_rope, "beam": _exact_beam, "copy": _exact_copy,
          "accept": _exact_accept, "compact": _exact_compact, "tree": _exact_tree}
