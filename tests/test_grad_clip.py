"""Gradient clipping on the CPU: the library's refusals, which return before any launch."""
from __future__ import annotations

import ctypes as C
import os
from array import array

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "combine_top_router_amd", "libmoe.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libmoe.so not built")

MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from combine_top_router_amd import _lib
    return _lib.load()


def _refs(*rows):
    words = array("q")
    for data, out, numel, dtype in rows:
        words.extend((data, out, numel, dtype))
    return words, C.c_void_p(words.buffer_info()[0]), len(rows)


@pytest.mark.parametrize("row,status", [
    ((0, 0, 8, 0), 1), ((MB + 1, 0, 8, 0), 1), ((MB + 2, 0, 8, 2), 1), ((MB, MB + 1, 8, 1), 1),
    ((MB, 0, -1, 0), 1), ((MB, 0, 1 << 44, 0), 1), ((MB, 0, 8, 3), 2), ((MB, 0, 8, -1), 2),
    ((MB, 0, 8, 1 << 32), 1),  # reserved word set
])
def test_bad_tensors_are_refused(lib, row, status):
    keep, refs, n = _refs((MB, 0, 100, 0), row)
    fake = C.c_void_p(MB)
    assert lib.moe_grad_sumsq_workspace_bytes(refs, n) == 0
    assert lib.moe_grad_sumsq(refs, n, fake, fake, 1 << 30, None) == status
    assert lib.moe_grad_clip(refs, n, fake, 1.0, fake, None) == status


def test_bad_arguments_are_refused(lib):
    keep, refs, n = _refs((MB, 0, 100, 0))
    fake, odd = C.c_void_p(MB), C.c_void_p(MB + 4)
    need = lib.moe_grad_sumsq_workspace_bytes(refs, n)
    assert need >= 8
    assert lib.moe_grad_sumsq(None, 1, fake, fake, need, None) == 1
    assert lib.moe_grad_sumsq(refs, -1, fake, fake, need, None) == 1
    assert lib.moe_grad_sumsq(refs, n, None, fake, need, None) == 1
    assert lib.moe_grad_sumsq(refs, n, odd, fake, need, None) == 1
    assert lib.moe_grad_sumsq(refs, n, fake, None, need, None) == 1
    assert lib.moe_grad_sumsq(refs, n, fake, odd, need, None) == 1
    assert lib.moe_grad_sumsq(refs, n, fake, fake, need - 1, None) == 1
    assert lib.moe_grad_clip(refs, n, None, 1.0, fake, None) == 1
    for bound in (-1.0, float("nan")):
        assert lib.moe_grad_clip(refs, n, fake, bound, fake, None) == 1


@pytest.mark.parametrize("rows", [
    [(MB, 0, 100, 0), (MB, 0, 100, 0)],                    # the same tensor twice, in place
    [(MB, 0, 100, 0), (MB + 100, 0, 100, 0)],              # halves of each other
    [(MB, 4 * MB, 100, 2), (2 * MB, 4 * MB + 396, 8, 2)],  # outputs overlap
    [(MB, 4 * MB, 100, 0), (4 * MB + 2, 8 * MB, 100, 0)],  # an output over another's input
    [(MB, MB + 2, 100, 0)],                                # shifted over itself
    [(MB, 0, 1 << 20, 0), (8 * MB, 0, 4, 0), (MB + 64, 16 * MB, 4, 0)],
])
def test_shared_memory_that_is_written_is_refused(lib, rows):
    keep, refs, n = _refs(*rows)
    assert lib.moe_grad_clip(refs, n, C.c_void_p(64 * MB), 1.0, C.c_void_p(65 * MB), None) == 1


def test_workspace_counts_workgroups_not_elements(lib):
    keep, refs, n = _refs((MB, 0, 1, 0), (MB, 0, 0, 0), (MB, 0, 1 << 40, 1))
    assert 0 < lib.moe_grad_sumsq_workspace_bytes(refs, n) <= 1 << 20
    many = [(MB, 0, 5, 2)] * 1000
    keep, refs, n = _refs(*many)
    assert lib.moe_grad_sumsq_workspace_bytes(refs, n) == 8000  # one chunk each
    keep, refs, n = _refs((0, 0, 0, 0))
    assert lib.moe_grad_sumsq_workspace_bytes(refs, n) == 0
