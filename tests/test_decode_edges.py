"""Host side of the decoding operators: what the C ABI and the binding refuse
beyond test_decode.py. Nothing here reaches a kernel."""
import ctypes
import pathlib
import re

import pytest

import long_context_sparse_segment_b200 as pbs
from long_context_sparse_segment_b200 import _lib
from test_decode import FAKE, cache, rows


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
