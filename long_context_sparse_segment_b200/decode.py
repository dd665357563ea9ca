"""PyTorch-facing calls of libpbs around the prefill: rotary positions, the
paged K/V cache, and attention for trees of drafted tokens over it.

As in ``ops.py`` every step runs in the library's CUDA kernels (csrc/rope.cu,
cache.cu, tree.cu); these functions check tensors, allocate outputs and pass
pointers and the current stream of the tensors' device through the C ABI
(include/pbs.h). Nothing here waits for the device: lengths, page tables and
reference counts are device tensors, so every call can be captured into a
CUDA graph. What a kernel refuses (a bad page, a pool without free pages) is
read with ``device_status``.
"""
from __future__ import annotations

import math

import torch

from . import _lib
from ._lib import Cache, Rows, check, lib

_TYPES = {torch.bfloat16: _lib.BF16, torch.float16: _lib.FP16, torch.float32: _lib.FP32}
_LAYOUTS = {"half": 0, "pairs": 1}
_HALVES = (torch.bfloat16, torch.float16)
_NONE = Rows(None, 0, 0, 0, 0)
_push, _pop = torch.cuda.nvtx.range_push, torch.cuda.nvtx.range_pop
_VEC = {torch.bfloat16: 7, torch.float16: 7, torch.float32: 3}  # elements of 16 bytes, less one


def _fresh(t):
    """A new contiguous tensor of t's shape, type and device."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _on(t, name, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _ints(t, name, shape, device):
    if (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.shape == shape
            and t.is_cuda and t.device == device and t.is_contiguous()):
        return
    _on(t, name, device)
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _call(name, dev, *args):
    """One C-ABI call on the current stream of device ``dev`` (its last
    argument), with that device current, inside an NVTX range of its name."""
    at = dev.index
    if at != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call(name, dev, *args)
    _push(name)
    try:
        status = getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(at))
    finally:
        _pop()
    if status:
        check(status, name)


def _rows(t, name, written=False):
    """[..., b, h, n, d] (4 or 5 dimensions) as pbs_rows: the head dimension
    contiguous, the others multiples of 16 bytes; a tensor that is written may
    not overlap itself."""
    stride, p, odd = t.stride(), t.data_ptr(), _VEC[t.dtype]
    if not written and stride[-1] == 1 and not p & 15:
        if len(stride) == 4:
            if not (stride[0] | stride[1] | stride[2]) & odd:
                return Rows(p, 0, stride[0], stride[1], stride[2])
        elif not (stride[0] | stride[1] | stride[2] | stride[3]) & odd:
            return Rows(p, *stride[:4])
    size = t.shape
    if size[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    step = [st if n > 1 else 0 for n, st in zip(size[:-1], stride[:-1])]
    if p & 15 or any(x & odd for x in step):
        raise ValueError(f"{name}: rows must be 16-byte aligned")
    if written:
        used = size[-1]
        for st, n in sorted((st, n) for st, n in zip(stride[:-1], size[:-1]) if n > 1):
            if st < used:
                raise ValueError(f"{name}: an output may not overlap itself")
            used = st * (n - 1) + used
    return Rows(p, step[0] if len(step) == 4 else 0, *step[-3:])


def _span(t):
    """The bytes from a tensor's first element to behind its last."""
    p, size = t.data_ptr(), t.element_size()
    if t.is_contiguous():
        return p, p + t.numel() * size
    last = sum(st * (n - 1) for st, n in zip(t.stride(), t.shape))
    return p, p + (last + 1) * size


def _meet(x, y):
    """Whether two tensors share memory. Slices of one buffer (equal strides) are
    compared element by element, so that interleaved ones are apart; others by
    their spans."""
    if not (x.numel() and y.numel()):
        return False
    (a, b), (c, d) = _span(x), _span(y)
    if b <= c or d <= a:
        return False
    size = x.element_size()
    if x.dim() != y.dim() or y.element_size() != size or (c - a) % size:
        return True
    dims = []
    for n, m, s, t in zip(x.shape, y.shape, x.stride(), y.stride()):
        s, t = (t, t) if n == 1 else (s, s) if m == 1 else (s, t)
        if s != t:
            return True
        if s and (n > 1 or m > 1):
            dims.append((s, n, m))
    dims.sort(reverse=True)

    def hits(k, off):
        """Whether sum_k (i - j) s = off for some i < n, j < m of dims[k:]."""
        if k == len(dims):
            return off == 0
        s, n, m = dims[k]
        rest = sum(st * (max(u, w) - 1) for st, u, w in dims[k + 1:])
        lo, hi = max(-((rest - off) // s), 1 - m), min((off + rest) // s, n - 1)
        return hi - lo > 3 or any(hits(k + 1, off - t * s) for t in range(lo, hi + 1))

    return hits(0, (c - a) // size)


def _apart(out, name, *others):
    """An output that a call was given may not reach into its inputs (the C call
    looks at the other pairs)."""
    for x in others:
        if _meet(out, x):
            raise ValueError(f"{name} overlaps an input")


def rope_freqs(rot, base=10000.0, scaling=None, device=None):
    """(inv_freq [rot/2] fp64, gain) for ``rope``: inv_freq[i] = base^(-2i/rot)
    radians per position, scaled for contexts longer than a model was trained
    on (``original`` tokens) by ``factor``:

    None                            as trained
    dict(type="linear", factor=)    every frequency divided by factor
    dict(type="ntk", factor=)       base * factor^(rot/(rot-2))
    dict(type="ramp", factor=, original=, low=1, high=4)
                                    pairs that turn more than ``high`` times in
                                    ``original`` tokens keep their frequency,
                                    those that turn less than ``low`` times
                                    have it divided, a linear ramp over the
                                    turns between
    dict(type="yarn", factor=, original=, fast=32, slow=1, gain=None)
                                    the same with the ramp over the pair's
                                    index, and gain 0.1 ln(factor) + 1
    """
    if rot < 0 or rot % 16:
        raise ValueError("rot must be a non-negative multiple of 16")
    if not base > 1:
        raise ValueError("base must be above 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    freq = lambda b: torch.pow(torch.tensor(float(b), dtype=torch.float64), -2.0 * i / max(rot, 1))
    f, gain = freq(base), 1.0
    if scaling is not None:
        s = dict(scaling)
        kind, factor = s.pop("type", None), float(s.pop("factor", 0))
        if not factor >= 1:
            raise ValueError("factor must be at least 1")
        if kind == "linear":
            f = f / factor
        elif kind == "ntk":
            f = freq(base * factor ** (rot / max(rot - 2, 1)))
        elif kind in ("ramp", "yarn") and not s.get("original", 0) > 0:
            raise ValueError(f"{kind} needs original, the tokens trained on")
        elif kind == "ramp":
            original, low, high = s.pop("original"), s.pop("low", 1.0), s.pop("high", 4.0)
            if not high > low:
                raise ValueError("high must be above low")
            keep = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
            f = f * keep + f / factor * (1 - keep)
        elif kind == "yarn":
            original, fast, slow = s.pop("original"), s.pop("fast", 32.0), s.pop("slow", 1.0)
            at = lambda turns: (rot * math.log(original / (turns * 2 * math.pi))
                                / (2 * math.log(base)))
            lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
            drop = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
            f = f / factor * drop + f * (1 - drop)
            gain = s.pop("gain", None)
            gain = 0.1 * math.log(factor) + 1.0 if gain is None else float(gain)
        else:
            raise ValueError(f"unknown scaling type {kind!r}")
        if s:
            raise ValueError(f"unknown scaling entries {sorted(s)}")
    return f.to(device), gain


def rope(q, k, pos, inv_freq, gain=1.0, layout="half", transpose=False, q_out=None, k_out=None):
    """Rotary positions of q [b, hq, n, d] and k [b, hkv, n, d] (or None) in
    one launch (pbs_rope): bf16, fp16 or fp32, any strides with contiguous
    16-byte-aligned rows (slices of one projection). pos is int32 [b, n] or
    [n]; the first 2 * len(inv_freq) elements of each head turn. ``transpose``
    turns back: the gradients of q and k from those of the results, which
    autograd takes where q or k requires one (then without q_out and k_out, and
    inv_freq gets none). Returns (q', k'), or q' alone without k. q_out may be q
    itself and k_out k, and they overlap nothing else."""
    _on(q, "q")
    dev, t, size = q.device, q.dtype, q.shape
    kind, order = _TYPES.get(t), _LAYOUTS.get(layout)
    if len(size) != 4:
        raise ValueError("q must be [b, hq, n, d]")
    if kind is None:
        raise TypeError(f"q must be bf16, fp16 or fp32, got {t}")
    if order is None:
        raise ValueError(f"layout must be 'half' or 'pairs', got {layout!r}")
    b, hq, n, d = size
    if d < 16 or d % 16 or d > 1024:
        raise ValueError("the head dimension must be a multiple of 16, at most 1024")
    hkv = 0
    if k is not None:
        _on(k, "k", dev)
        ksize = k.shape
        if len(ksize) != 4 or (ksize[0], ksize[2], ksize[3]) != (b, n, d) or k.dtype is not t:
            raise ValueError("k must be [b, hkv, n, d] of q's type")
        hkv = ksize[1]
    elif k_out is not None:
        raise ValueError("k_out without k")
    _on(inv_freq, "inv_freq", dev)
    if inv_freq.dtype is not torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be a contiguous fp64 vector")
    rot = 2 * inv_freq.numel()
    if rot % 16 or rot > d:
        raise ValueError("inv_freq: 2 * len must be a multiple of 16 and at most d")
    each = isinstance(pos, torch.Tensor) and pos.dim() == 1
    _ints(pos, "pos", (n,) if each else (b, n), dev)
    if (q.requires_grad or inv_freq.requires_grad or (k is not None and k.requires_grad)) and \
            torch.is_grad_enabled():
        if inv_freq.requires_grad:
            raise ValueError("inv_freq has no gradient")
        if not (q_out is None and k_out is None):
            raise ValueError("q_out and k_out are not for inputs that require a gradient")
        return _Rope.apply(q, k, pos, inv_freq, gain, layout, transpose)
    q_out, q_to = _rope_out(q, q_out, "q_out", hq, n, d)
    k_from = k_to = _NONE
    if k is not None:
        k_out, k_to = _rope_out(k, k_out, "k_out", hkv, n, d)
        k_from = _rows(k, "k") if hkv else _NONE
    if b and n and hq + hkv:
        _call("pbs_rope", dev, _rows(q, "q") if hq else _NONE, q_to, hq, k_from, k_to, hkv,
              pos.data_ptr(), 0 if each else n, inv_freq.data_ptr() if rot else None, gain, b, n,
              d, rot, order, 1 if transpose else 0, kind)
    return q_out if k is None else (q_out, k_out)


class _Rope(torch.autograd.Function):
    """rope under autograd. The map is linear, its gradient the transposed map,
    which is a rope again (and so has a gradient itself)."""

    @staticmethod
    def forward(ctx, q, k, pos, inv_freq, gain, layout, transpose):
        out = rope(q, k, pos, inv_freq, gain, layout, transpose)
        ctx.save_for_backward(pos, inv_freq)
        ctx.how = gain, layout, not transpose
        ctx.set_materialize_grads(False)
        return out

    @staticmethod
    def backward(ctx, *grads):
        need = ctx.needs_input_grad[:2]
        grads = [_readable(g) if n and g is not None else None
                 for g, n in zip((*grads, None), need)]
        there = [g for g in grads if g is not None]
        if not there:
            return (None,) * 7
        back = rope(there[0], there[1] if len(there) > 1 else None, *ctx.saved_tensors, *ctx.how)
        back = list(back) if len(there) > 1 else [back]
        return (*(None if g is None else back.pop(0) for g in grads), *(None,) * 5)


def _readable(g):
    """A gradient as rope reads it: contiguous rows, 16-byte aligned."""
    try:
        _rows(g, "gradient")
    except ValueError:
        return g.clone(memory_format=torch.contiguous_format)
    return g


def _rope_out(x, y, name, h, n, d):
    """The tensor that takes x's result, and its rows."""
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        return y, Rows(y.data_ptr(), 0, h * n * d, n * d, d)
    _on(y, name, x.device)
    if y.shape != x.shape or y.dtype is not x.dtype:
        raise ValueError(f"{name} must have the shape and type of its input")
    if y.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} may not require a gradient")
    if y.data_ptr() != x.data_ptr() or y.stride() != x.stride():
        _apart(y, name, x)
    return y, _rows(y, name, True) if y.numel() else _NONE


# ------------------------------------------------------------------ the cache
def _pools(k_pages, v_pages, table=None):
    """The pools [layers, pages, hkv, page, d] (or one layer's, 4-D)."""
    _on(k_pages, "k_pages")
    dev, size = k_pages.device, k_pages.shape
    n = len(size)
    _on(v_pages, "v_pages", dev)
    if n < 4 or n > 5 or k_pages.element_size() != 2:
        raise ValueError("k_pages must be [layers, pages, hkv, page, d] (or 4-D) of a 16-bit type")
    if v_pages.shape != size or v_pages.dtype is not k_pages.dtype:
        raise ValueError("v_pages must have the shape and type of k_pages")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    if not k_pages.numel():
        raise ValueError("k_pages is empty")
    layers, pages, hkv, page, d = size if n == 5 else (1, *size)
    if d % 8:
        raise ValueError("the head dimension must be a multiple of 8")
    if table is None:
        return Cache(layers, pages, hkv, page, d, 0, 1)
    seqs, width = _table(table, dev)
    return Cache(layers, pages, hkv, page, d, seqs, width)


def _table(table, device=None):
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        _on(table, "table", device)
        raise ValueError("table must be [seqs, width]")
    size = table.shape
    _ints(table, "table", size, table.device if device is None else device)
    seqs, width = size
    if width < 1:
        raise ValueError("table must have a column")
    return seqs, width


def _books(table, refs, lens, page):
    seqs, width = _table(table)
    dev = table.device
    _on(refs, "refs", dev)
    pages = refs.numel()
    _ints(refs, "refs", (pages,), dev)
    _ints(lens, "lens", (seqs,), dev)
    if pages < 1 or page < 1:
        raise ValueError("refs and page must not be empty")
    return Cache(1, pages, 1, page, 8, seqs, width)


def _pairs(src, dst, device):
    _on(src, "src", device)
    n = src.numel()
    _ints(src, "src", (n,), device)
    _ints(dst, "dst", (n,), device)
    return n


def _ws(op, c, n, device):
    need = lib().pbs_cache_workspace_bytes(c, op, n)
    return (torch.empty(need, dtype=torch.uint8, device=device) if need else None), need


def cache_reserve(table, refs, lens, want, page):
    """Pages for the tokens lens[s] .. want[s]-1 of every sequence, each held
    by it alone (pbs_cache_reserve). Returns (src, dst) int32 [seqs]: the
    pages to copy with ``cache_copy`` before writing, -1 where none. Too few
    free pages: nothing changes and device_status() is PBS_ERR_PAGES."""
    c = _books(table, refs, lens, page)
    dev = table.device
    _ints(want, "want", (c.seqs,), dev)
    src, dst = torch.empty_like(lens), torch.empty_like(lens)
    ws, need = _ws(_lib.CACHE_RESERVE, c, 0, dev)
    _call("pbs_cache_reserve", dev, _ptr(table), _ptr(refs), _ptr(lens), _ptr(want), _ptr(src),
          _ptr(dst), c, _ptr(ws), need)
    return src, dst


def _owned(c, refs, device):
    """``refs`` put into c: no writes into pages that several sequences hold."""
    if refs is not None:
        _ints(refs, "refs", (c.pages,), device)
        c.refs = refs.data_ptr()


def cache_append(k, v, k_pages, v_pages, table, start, count=None, refs=None):
    """Rows i < count[s] (all without count) of k, v [seqs, hkv, n, d] written
    at tokens start[s] + i of one layer's pools, or [layers, seqs, hkv, n, d]
    of all layers (pbs_cache_append). The pages must be reserved; with ``refs``
    rows whose page another sequence holds too, as behind a reserve that found
    too few free pages, are reported and skipped."""
    c = _pools(k_pages, v_pages, table)
    dev = k_pages.device
    for t, nm in ((k, "k"), (v, "v")):
        _on(t, nm, dev)
        if t.dtype != k_pages.dtype or t.dim() != k_pages.dim():
            raise ValueError(f"{nm} must have the type and dimensions of k_pages")
        lead = (c.layers,) if t.dim() == 5 else ()
        if t.shape != (*lead, c.seqs, c.hkv, k.shape[-2], c.d):
            raise ValueError(f"{nm} must be {[*lead, c.seqs, c.hkv, 'n', c.d]}, got {list(t.shape)}")
    _ints(start, "start", (c.seqs,), dev)
    if count is not None:
        _ints(count, "count", (c.seqs,), dev)
    _owned(c, refs, dev)
    if k.numel() == 0:
        return
    _call("pbs_cache_append", dev, _rows(k, "k"), _rows(v, "v"), k.shape[-2], _ptr(k_pages),
          _ptr(v_pages), _ptr(table), _ptr(start), _ptr(count), c)


def cache_copy(k_pages, v_pages, src, dst):
    """Page src[i] copied to page dst[i] in both pools and every layer; pairs
    of -1 are skipped (pbs_cache_copy). All pairs happen at once: a repeated
    destination, or a source that is also a destination, is refused on the
    device."""
    c = _pools(k_pages, v_pages)
    dev = k_pages.device
    n = _pairs(src, dst, dev)
    ws, need = _ws(_lib.CACHE_COPY, c, n, dev)
    _call("pbs_cache_copy", dev, _ptr(k_pages), _ptr(v_pages), _ptr(src), _ptr(dst), n, c,
          _ptr(ws), need)


def cache_fork(table, refs, lens, src, dst, page):
    """Sequence dst[i] (empty) becomes a second holder of sequence src[i]'s
    pages (pbs_cache_fork); no page is copied before one of them writes."""
    c = _books(table, refs, lens, page)
    dev = table.device
    n = _pairs(src, dst, dev)
    _call("pbs_cache_fork", dev, _ptr(table), _ptr(refs), _ptr(lens), _ptr(src), _ptr(dst),
          n, c)


def cache_trim(table, refs, lens, keep, page):
    """Sequence s keeps min(lens[s], keep[s]) tokens and releases the pages
    behind them; keep 0 frees it, a negative keep leaves it (pbs_cache_trim)."""
    c = _books(table, refs, lens, page)
    dev = table.device
    _ints(keep, "keep", (c.seqs,), dev)
    _call("pbs_cache_trim", dev, _ptr(table), _ptr(refs), _ptr(lens), _ptr(keep), c)


def cache_compact(k_pages, v_pages, table, refs):
    """The held pages moved to the low end of the pools; table and refs follow
    (pbs_cache_compact). Returns (src, dst) int32 [pages]: the moves, then -1."""
    c = _pools(k_pages, v_pages, table)
    dev = k_pages.device
    _ints(refs, "refs", (c.pages,), dev)
    src, dst = torch.empty_like(refs), torch.empty_like(refs)
    ws, need = _ws(_lib.CACHE_COMPACT, c, 0, dev)
    _call("pbs_cache_compact", dev, _ptr(k_pages), _ptr(v_pages), _ptr(table), _ptr(refs),
          _ptr(src), _ptr(dst), c, _ptr(ws), need)
    return src, dst


def cache_accept(k_pages, v_pages, table, start, path, count=None, lens=None, refs=None):
    """The accepted drafts moved behind their prefix: token start[s] +
    path[s][i] becomes token start[s] + i, i < count[s], in every layer
    (pbs_cache_accept). path [seqs, n] ascends strictly (n may be less than the
    drafts). With ``lens``, lens[s] becomes start[s] + count[s]; it may be
    ``start`` itself (the drafts' start is the length), or ``count``. With
    ``refs`` a sequence whose accepted tokens come to lie in a page that another
    one holds too is reported and left alone."""
    c = _pools(k_pages, v_pages, table)
    dev = k_pages.device
    _ints(start, "start", (c.seqs,), dev)
    if not isinstance(path, torch.Tensor) or path.dim() != 2:
        raise ValueError("path must be [seqs, n]")
    _ints(path, "path", (c.seqs, path.shape[1]), dev)
    for t, nm in ((count, "count"), (lens, "lens")):
        if t is not None:
            _ints(t, nm, (c.seqs,), dev)
    _owned(c, refs, dev)
    _call("pbs_cache_accept", dev, _ptr(k_pages), _ptr(v_pages), _ptr(table), _ptr(start),
          _ptr(path), _ptr(count), _ptr(lens), path.shape[1], c)


# ------------------------------------------------------------------ attention
def tree_mask(parents):
    """(mask, depth) of drafted trees (pbs_tree_mask). parents int32 [b, tree]:
    the draft that draft i continues (below i), or -1 for the cached prefix.
    mask int32 [b, tree, ceil(tree/32)]: bit j & 31 of word j >> 5 of row i is
    set when j is i or an ancestor of i; depth int32 [b, tree] counts the
    ancestors (draft i's position is start + depth)."""
    _on(parents, "parents")
    if parents.dim() != 2:
        raise ValueError("parents must be [b, tree]")
    _ints(parents, "parents", parents.shape, parents.device)
    b, t = parents.shape
    mask = torch.empty(b, t, (t + 31) // 32, dtype=torch.int32, device=parents.device)
    depth = torch.empty_like(parents)
    _call("pbs_tree_mask", parents.device, _ptr(parents), _ptr(mask), _ptr(depth), b, t)
    return mask, depth


def _tree_bytes(dev, hq, tree, c):
    """The workspace of tree_attn on device ``dev``: it grows with its SMs."""
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return lib().pbs_tree_workspace_bytes(hq, tree, c)
    return lib().pbs_tree_workspace_bytes(hq, tree, c)


def tree_attn(q, k_pages, v_pages, table, start, mask=None, count=None, scale=0.0, lse=False,
              out=None, ws=None):
    """Attention of q [seqs, hq, tree, d] (bf16 or fp16, strided rows) over one
    layer's pools [pages, hkv, page, d] (pbs_tree_attn). Draft i < count[s]
    (all without count) sees the first start[s] tokens and those tokens
    start[s] + j, j < count[s], whose bit is set in mask row i (see
    ``tree_mask``; without mask j <= i). With tree = 1 this is a decoding
    step. Returns o [seqs, hq, tree, d], and lse [seqs, hq, tree] fp32 when
    asked; rows i >= count[s], and a sequence that is refused on the device
    (a negative length, tokens beyond the table), are left as they were in
    ``out`` and are zero in what this call allocates (their lse too)."""
    c = _pools(k_pages, v_pages, table)
    dev, t, size = k_pages.device, k_pages.dtype, getattr(q, "shape", None)
    _on(q, "q", dev)
    if k_pages.dim() != 4:
        raise ValueError("k_pages must be one layer's: [pages, hkv, page, d]")
    if t not in _HALVES or q.dtype is not t:
        raise TypeError("q must be bf16 or fp16 and have the type of k_pages")
    seqs = c.seqs
    if len(size) != 4 or size[0] != seqs or size[3] != c.d:
        raise ValueError(f"q must be [{seqs}, hq, tree, {c.d}]")
    hq, tree = size[1], size[2]
    if hq < 1 or hq % c.hkv:
        raise ValueError("hq must be a multiple of hkv")
    _ints(start, "start", (seqs,), dev)
    if count is not None:
        _ints(count, "count", (seqs,), dev)
    if mask is not None:
        _ints(mask, "mask", (seqs, tree, (tree + 31) // 32), dev)
    zero = out is None  # sequences that the kernel refuses have rows behind their count too
    if zero:
        out = _fresh(q)
    else:
        _on(out, "out", dev)
        if out.shape != size or out.dtype is not t or not out.is_contiguous():
            raise ValueError("out must be contiguous, of q's shape and type")
        _apart(out, "out", q, k_pages, v_pages)
    l = None
    if lse:
        make = out.new_empty if zero else out.new_zeros
        l = make((seqs, hq, tree), dtype=torch.float32)
    if not (seqs and tree):
        return (out, l) if lse else out
    need = _tree_bytes(dev, hq, tree, c)
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _on(ws, "ws", dev)
        if not ws.is_contiguous() or ws.numel() * ws.element_size() < need:
            raise ValueError(f"ws must be contiguous, of {need} bytes at least")
    _call("pbs_tree_attn", dev, _rows(q, "q"), k_pages.data_ptr(), v_pages.data_ptr(),
          table.data_ptr(), start.data_ptr(), _ptr(count), _ptr(mask), out.data_ptr(), _ptr(l),
          hq, tree, c, scale, zero, _TYPES[t], ws.data_ptr(), need)
    return (out, l) if lse else out


class PagedCache:
    """The tensors of a paged cache, and the calls above on them: pools k, v
    [layers, pages, hkv, page, d], table [seqs, width], refs [pages], lens
    [seqs]. Made empty; everything it knows is in these tensors."""

    def __init__(self, seqs, max_len, pages, hkv, d, page=64, layers=1, dtype=torch.bfloat16,
                 device="cuda"):
        if min(seqs, max_len, pages, hkv, d, page, layers) < 1:
            raise ValueError("sizes must be positive")
        if dtype not in _HALVES:
            raise TypeError("dtype must be bf16 or fp16")
        self.page = page
        self.k = torch.zeros(layers, pages, hkv, page, d, dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        ints = lambda *n: torch.zeros(*n, dtype=torch.int32, device=self.k.device)
        self.table = ints(seqs, -(-max_len // page)) - 1
        self.refs, self.lens = ints(pages), ints(seqs)

    def reserve(self, want):
        """Room for want[s] tokens in every sequence, shared pages that will
        be written copied. Too few free pages: nothing changes, and what append
        and accept would then write into a shared page is reported and left out."""
        src, dst = cache_reserve(self.table, self.refs, self.lens, want, self.page)
        cache_copy(self.k, self.v, src, dst)

    def append(self, layer, k, v, start=None, count=None):
        """k, v [seqs, hkv, n, d] at tokens start[s].. (the length) of a layer.
        The length is not changed: every layer appends at the same tokens."""
        cache_append(k, v, self.k[layer], self.v[layer], self.table,
                     self.lens if start is None else start, count, self.refs)

    def attend(self, layer, q, mask=None, start=None, **kw):
        """tree_attn of a layer; ``start`` is the lengths when not given."""
        return tree_attn(q, self.k[layer], self.v[layer], self.table,
                         self.lens if start is None else start, mask, **kw)

    def accept(self, path, count=None):
        """The accepted drafts behind the lengths, which grow by their number."""
        cache_accept(self.k, self.v, self.table, self.lens, path, count, self.lens,
                     self.refs)

    def fork(self, src, dst):
        cache_fork(self.table, self.refs, self.lens, src, dst, self.page)

    def trim(self, keep):
        cache_trim(self.table, self.refs, self.lens, keep, self.page)

    def compact(self):
        return cache_compact(self.k, self.v, self.table, self.refs)
