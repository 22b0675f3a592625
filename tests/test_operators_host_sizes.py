"""Sizes that the training operators ask for, on the host."""

import pytest

import double_binary_tree_gb300 as vr

A = 0x10000000


@pytest.mark.parametrize("T,D", [(300, 4096), (4096, 4096), (5000, 4096), (2048, 8192)])
def test_the_least_workspace_is_never_the_larger(T, D):
    """Around one piece of the vocabulary (256 MB of gradient factors) the sums
    of several pieces weigh more than what the pieces save."""
    size = vr.vr_linear_xent_workspace_bytes
    for V in list(range(24000, 44000, 250)) + [131072, 262144, 400000]:
        full, least = (size(A, D, A, D, T, D, V, vr.VR_BFLOAT16, g) for g in (1, 2))
        assert 0 < least <= full
    # far beyond it the pieces do take less
    assert size(A, D, A, D, T, D, 1 << 20, vr.VR_BFLOAT16, 2) < \
        size(A, D, A, D, T, D, 1 << 20, vr.VR_BFLOAT16, 1) or T > D
