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


def test_a_result_that_starts_where_the_residual_does_has_its_rows(lib):
    """In place on the residual means row for row: with another stride a row would be written before it was read."""
    import ctypes
    P = ctypes.c_void_p
    buf, w = torch.zeros(3 * 128, dtype=BF), torch.zeros(64, 64, dtype=BF)
    wi = torch.zeros(128, 64, dtype=BF)
    dense, apart = buf[:192].view(3, 64), buf.view(3, 128)[:, :64]
    x = torch.zeros(3, 64, dtype=BF)
    for r, o in ((dense, apart), (apart, dense)):
        with pytest.raises(ValueError, match="out starts where residual does"):
            ops.linear(x, w, residual=r, out=o)
        with pytest.raises(ValueError, match="out starts where residual does"):
            ops.gated_ffn(x, wi, w, residual=r, out=o)
    with pytest.raises(ValueError, match="no CPU path"):
        ops.linear(x, w, residual=apart, out=apart)
    with pytest.raises(ValueError, match="no CPU path"):      # one row has no stride
        ops.linear(x[:1], w, residual=apart[:1], out=dense[:1])
    for n in (3, 70):
        assert lib.tpk_linear(P(256), 64, P(512), None, 0, P(1024), 128, P(1024), 64, n, 64, 64, P(4096), 1 << 30, None,
                              None) == -1
        assert lib.tpk_gated_ffn(P(256), 64, P(512), P(768), 1, P(1024), 128, None, None, P(1024), 64, n, 64, 64, 64,
                                 P(4096), 1 << 30, None, None) == -1
