"""Refusals at the ends of the policy objective's size range, before any launch (CPU only)."""
import ctypes

import pytest

from prefix_tree_packed_dfs_gb300 import binding as B

P = ctypes.c_void_p
MOST = 2 ** 31 - 8193


def _call(lib, R, F, n_seqs):
    o = B.PolicyOpts(0.2, 0.2, 0.0, 0.0)
    return lib.tpk_policy_loss(*[P(4096)] * 8, P(4096) if n_seqs else None, n_seqs, ctypes.byref(o), P(4096), P(4096), R,
                               F, None, 0, None)


@pytest.mark.parametrize("n", [MOST + 1, 2 ** 31 - 4000, 2 ** 31 - 32, 2 ** 31 - 1])
def test_policy_refuses_counts_whose_strides_pass_32_bits(lib, n):
    """Lists of raw tokens are read 32 entries at a time and partial sums 32 rows at a time, counted in 32 bits."""
    assert lib.tpk_policy_loss_workspace_bytes(n, 0) == 0
    assert lib.tpk_policy_loss_workspace_bytes(8, n) == 0
    assert _call(lib, n, 8, 0) == -1 and _call(lib, n, n, 0) == -1
    assert _call(lib, 8, 8, n) == -1


def test_policy_takes_counts_below_that(lib):
    assert lib.tpk_policy_loss_workspace_bytes(MOST, 0) > 4 * MOST
    assert lib.tpk_policy_loss_workspace_bytes(8, MOST) > 40 * MOST
    assert _call(lib, MOST, 8, 0) == -7 and _call(lib, 8, 8, MOST) == -7     # (there is no workspace)
