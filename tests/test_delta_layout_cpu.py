"""The numbering of a packed batch's blocks, with the kernels' own block size and
the workspace that the library asks for."""

import ctypes
import os
import re

import numpy as np
import pytest

from retnet_retention_amd import binding

HEADER = os.path.join(os.path.dirname(binding.__file__), "csrc", "delta.hpp")


def block_size():
    return int(re.search(r"constexpr int kDeltaBlock = (\d+);", open(HEADER).read()).group(1))


@pytest.mark.parametrize("grad", [False, True])
def test_every_block_of_a_packed_batch_has_its_own_place(grad):
    """Block i of sequence b is cu[b] // size + b + i: no two are the same, and the
    workspace holds exactly as many as the largest number a batch can reach."""
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libretention.so not built (run __graft_entry__.build())")
    L, size, rng = binding.lib(), block_size(), np.random.default_rng(8)

    def need(batch, total):
        d = binding.DeltaDesc(batch, 1000, 2, 4, 128, 128, binding.RET_F32, 1.0)
        f = L.retention_delta_bwd_workspace_bytes if grad else L.retention_delta_workspace_bytes
        return f(ctypes.byref(d), 1, total)

    # bytes of one block and of one token (the backward keeps V' by rows)
    token = need(1, 1) - need(1, 0)
    block = need(1, size) - need(1, 0) - size * token
    assert block > 0 and (token > 0) == grad
    for _ in range(300):
        lens = rng.integers(0, 300, rng.integers(1, 9)) * rng.integers(0, 2)
        cu = np.concatenate([[0], np.cumsum(lens)])
        numbers = [cu[b] // size + b + i for b, n in enumerate(lens) for i in range(-(-n // size))]
        assert len(set(numbers)) == len(numbers)
        held = (need(len(lens), int(cu[-1])) - need(1, 0) - int(cu[-1]) * token) // block + 1
        assert held == cu[-1] // size + len(lens) and all(0 <= i < held for i in numbers)
