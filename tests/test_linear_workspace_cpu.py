"""A workspace that linear_workspace_bytes gives for rows at any alignment serves rows
at every alignment."""

import itertools

import pytest

from memory_efficient_activation_amd import _lib

F32, BF16 = 0, 1
XW, DY = _lib.LINEAR_ALIGNED_XW, _lib.LINEAR_ALIGNED_DY


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("backward", [0, 1])
@pytest.mark.parametrize("act", [_lib.LINEAR_IDENTITY, 5])
def test_fewer_aligned_rows_need_no_less(act, backward, dtype):
    size = _lib.library().linear_workspace_bytes
    tokens = [0, *range(1, 34), 63, 64, 100, 129, 777, 2048, 16384]
    sides = [0, 1, 8, 64, 72, 100, 1000, 1024, 2730, 4096, 8192, 16384, 32768, 1 << 21]
    for t, dim, units in itertools.product(tokens, sides, sides):
        by = {a: size(t, dim, units, act, dtype, backward, a) for a in (0, XW, DY, XW | DY)}
        for a, b in itertools.product(by, by):
            if a & b == a:  # rows that are aligned as in b are so as in a
                assert by[a] >= by[b], (t, dim, units, a, b)


def test_rows_that_turn_out_aligned():
    """Aligned rows of 24 tokens take a split sum, others the kernel without a
    workspace: the call with the size for any rows is not refused for its size.
    (It is refused for what it overlaps, before anything is launched.)"""
    lib = _lib.library()
    x, w, ws = (0x100000000 * k for k in range(1, 4))
    for dtype, dim, units in ((BF16, 4096, 16384), (BF16, 16384, 4096), (F32, 4096, 16384)):
        need = lib.linear_workspace_bytes(24, dim, units, -1, dtype, 0, 0)

        def call(size):
            return lib.linear_fwd(-1, 0.0, x, dim, w, dim, None, None, 0, 24, dim, units, x, units,
                                  ws if size else None, size, dtype, None)

        assert call(need) == _lib.EALIAS
        assert call(lib.linear_workspace_bytes(24, dim, units, -1, dtype, 0, XW) - 1) == _lib.EINVAL
