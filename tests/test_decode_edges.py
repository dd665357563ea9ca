"""Host side of the decoding operators: what the C ABI and the binding refuse
beyond test_decode.py. Nothing here reaches a kernel."""
import ctypes
import itertools
import pathlib
import random
import re

import pytest
import torch

import long_context_sparse_segment_b200 as pbs
from long_context_sparse_segment_b200 import _lib
from test_decode import FAKE, cache, call_rope, call_tree, rows


def at(x):
    return ctypes.c_void_p((1 << 20) + x)


def test_reference_counts_are_aligned():
    lib, c, r = pbs.lib(), cache(), rows()
    c.refs = (1 << 20) + 2
    assert lib.pbs_cache_append(r, r, 1, FAKE, at(1 << 16), *[FAKE] * 2, None, c,
                                None) == _lib.ERR_INVALID_ARG
    assert lib.pbs_cache_accept(FAKE, at(1 << 16), FAKE, FAKE, FAKE, None, None, 1, c,
                                None) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("lens,refs", [(4, None), (-4, None), (1 << 12, 1 << 12),
                                       ((1 << 13) + 8, None), ((1 << 14) + 124, None)])
def test_accepted_lengths_inside_another_input_are_refused(lens, refs):
    """start, refs (64), path [4, 3] and table [4, 8] of 32-bit words."""
    c = cache()
    c.refs = (1 << 20) + refs if refs else None
    assert pbs.lib().pbs_cache_accept(
        at(1 << 16), at(1 << 18), at(1 << 14), at(0), at(1 << 13), None, at(lens), 3, c,
        None) == _lib.ERR_INVALID_ARG


def test_kernels_launched_early_read_nothing_as_read_only():
    """Kernels that start while the one in front may still write their inputs
    wait for its end; loads of the read-only path need not stay behind that."""
    csrc = pathlib.Path(_lib.LIB_PATH).parent / "csrc"
    for f in ("tree.cuh", "tree.cu", "tree_tc.cu"):
        code = re.sub(r"//[^\n]*", "", (csrc / f).read_text())
        assert "__ldg" not in code and "global.nc" not in code and "__ldcs" not in code, f
    # the compaction's copies, the one such kernel of cache.cu
    code = (csrc / "cache.cu").read_text()
    kernel = code[code.index("copy_kernel(uint4"):code.index("append, accept")]
    assert "griddepcontrol.wait" in kernel
    assert "__ldg" not in kernel and "__restrict__" not in kernel


def shares(x, y):
    """Whether two views of one buffer name a common element."""
    at = lambda t: {t.storage_offset() + sum(i * s for i, s in zip(ix, t.stride()))
                    for ix in itertools.product(*map(range, t.shape))}
    return bool(at(x) & at(y))


def test_overlaps_of_strided_tensors():
    """Slices of one buffer against their elements one by one."""
    from long_context_sparse_segment_b200.decode import _meet
    base = torch.zeros(2, 5, 12, 8, dtype=torch.bfloat16)
    buf = base.transpose(1, 2)
    cuts = [buf[:, a:b] for a, b in ((0, 4), (4, 6), (3, 5), (6, 12), (0, 12), (5, 6))]
    cuts += [buf[:, 4:8, 1:3], buf[:, 4:8, 3:], buf[:1, 2:9], buf[1:, 2:9], buf[..., :4],
             buf[..., 4:], buf[:, 0:12:2], buf[:, 1:12:2], buf[:, :0], base,
             base[:, :, :1].expand(2, 5, 12, 8), base.view(2, 5, 24, 4)[:, :, ::2]]
    seen = set()
    for x, y in itertools.product(cuts, cuts):
        if x.stride() == y.stride() or not _meet(x, y):
            assert _meet(x, y) == shares(x, y), (x.shape, x.stride(), y.shape, y.stride())
            seen.add(_meet(x, y))
    assert seen == {True, False}
    # other strides and other types: by spans
    assert _meet(base, base.view(torch.int32)) and not _meet(base, torch.zeros_like(base))
    assert not _meet(base[:1], base.view(torch.uint8)[1:])
    flat = torch.zeros(4096, dtype=torch.bfloat16)
    rng = random.Random(0)
    for _ in range(300):
        st = (rng.choice([512, 64, 520]), rng.choice([64, 16, 128]), rng.choice([16, 8, 256]), 1)
        view = lambda: flat.as_strided((rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3),
                                        rng.choice([4, 8])), st, rng.randrange(0, 1200, 4))
        x, y = view(), view()
        # nothing that overlaps is taken for apart, and the other way where no
        # dimension reaches into another
        if shares(x, y):
            assert _meet(x, y)
        elif st in ((512, 64, 16, 1), (512, 128, 16, 1), (512, 64, 8, 1)):
            assert not _meet(x, y)


def test_written_rows_that_meet_other_memory_are_refused():
    """The same rows for everything; one output over the other input; over the
    positions; a workspace over the table."""
    r, far = rows(), rows(p=1 << 30)
    for kw in (dict(), dict(q=far), dict(k=far, q=rows(p=1 << 32), ko=rows(p=1 << 34)),
               dict(q=far, k=rows(p=1 << 32), ko=rows(p=1 << 34)),
               dict(q=far, k=far, qo=rows(p=1 << 32), ko=rows(p=(1 << 32) + 64)),
               dict(q=rows(batch=2048), qo=rows(batch=2056), k=far, ko=rows(p=1 << 32))):
        assert call_rope(**kw) == _lib.ERR_INVALID_ARG
    apart = [ctypes.c_void_p(1 << x) for x in range(25, 33)]
    for i, name in enumerate(("k", "v", "table", "start", "count", "mask", "out", "lse")):
        p = list(apart)
        p[i] = FAKE  # the workspace's place
        assert call_tree(cache(), ptrs=p, q=rows(p=1 << 40)) == _lib.ERR_INVALID_ARG, name
    assert call_tree(cache(), ptrs=apart, q=rows(p=1 << 31)) == _lib.ERR_INVALID_ARG  # q is out


def test_grids_follow_the_device():
    """No launch of the decoding operators takes the SMs for a constant."""
    csrc = pathlib.Path(_lib.LIB_PATH).parent / "csrc"
    for f in ("rope.cu", "cache.cu", "tree.cu", "tree.cuh", "tree_tc.cu", "decode.h"):
        assert not re.search(r"\b148\b", re.sub(r"//[^\n]*", "", (csrc / f).read_text())), f


def test_workspaces_are_sized_on_the_tensors_device(monkeypatch):
    """Two devices of different SM counts, faked: the size is asked for with the
    tensors' device current, and the current one is put back."""
    from long_context_sparse_segment_b200 import decode
    now = [0]

    class Device:
        def __init__(self, dev):
            self.to = dev.index

        def __enter__(self):
            self.back, now[0] = now[0], self.to

        def __exit__(self, *_):
            now[0] = self.back

    class Lib:
        @staticmethod
        def pbs_tree_workspace_bytes(hq, tree, c):
            return (100, 132)[now[0]] * hq * tree

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(decode, "lib", Lib)
    sizes = [decode._tree_bytes(torch.device("cuda", i), 2, 3, cache()) for i in (0, 1, 0)]
    assert sizes == [600, 792, 600] and now == [0]
