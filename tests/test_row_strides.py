"""One rule for tensors whose rows may lie apart, whichever wrapper takes them (CPU only: refused before any launch)."""
import pytest
import torch

from prefix_tree_packed_dfs_gb300 import ops

BF = torch.bfloat16


def _strided(rows, width, ld):
    return torch.zeros(rows * ld + width, dtype=BF).as_strided((rows, width), (ld, 1))


@pytest.mark.parametrize("ld", [8, 56, 60, 68, 100])
def test_every_wrapper_refuses_rows_that_overlap_or_are_not_aligned(lib, ld):
    bad, good = _strided(3, 64, ld), torch.zeros(3, 64, dtype=BF)
    w, ones = torch.zeros(64, 64, dtype=BF), torch.ones(64)
    wi, wo = torch.zeros(128, 64, dtype=BF), torch.zeros(64, 64, dtype=BF)
    depth, freqs = torch.zeros(3, dtype=torch.int32), ops.rope_freqs(64)
    heads, bad_heads = good.unflatten(1, (1, 64)), bad.as_strided((3, 1, 64), (ld, 64, 1))
    for fn in (lambda: ops.linear(bad, w), lambda: ops.linear(good, w, residual=bad), lambda: ops.linear(good, w, out=bad),
               lambda: ops.linear_bwd(bad, w, good), lambda: ops.linear_bwd(good, w, bad),
               lambda: ops.linear_bwd(good, w, good, dx=bad), lambda: ops.gated_ffn(bad, wi, wo),
               lambda: ops.gated_ffn(good, wi, wo, residual=bad), lambda: ops.gated_ffn(good, wi, wo, out=bad),
               lambda: ops.block_norm(good, ones, y=bad), lambda: ops.block_norm(good, ones, y=good, gate=bad),
               lambda: ops.rope_by_depth_ex(bad_heads, None, depth, freqs),
               lambda: ops.rope_by_depth_ex(heads, None, depth, freqs, q_out=bad_heads)):
        with pytest.raises(ValueError, match="rows must not overlap"):
            fn()


@pytest.mark.parametrize("ld", [64, 72, 8, 3])
def test_the_stride_of_one_row_is_of_no_account(lib, ld):
    one = torch.zeros(1000, dtype=BF).as_strided((1, 64), (ld, 1))
    with pytest.raises(ValueError, match="no CPU path"):     # past every check of shapes and strides
        ops.linear(one, torch.zeros(64, 64, dtype=BF), residual=one, out=one)
    with pytest.raises(ValueError, match="no CPU path"):
        ops.rope_by_depth_ex(one.as_strided((1, 1, 64), (ld, 64, 1)), None, torch.zeros(1, dtype=torch.int32),
                             ops.rope_freqs(64))
