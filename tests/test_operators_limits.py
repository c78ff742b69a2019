"""Refusals at the ends of the operators' size ranges, before any launch (CPU only)."""
import ctypes


def test_lm_loss_refuses_rows_whose_strides_pass_32_bits(lib):
    """The gather's last loop starts up to 304 * 16 = 4,864 rows behind the last
    position and counts in 32 bits: 2^31 - 8192 positions and more are refused."""
    a, big = ctypes.c_void_p(4096), 1 << 62
    assert lib.tpk_lm_loss_workspace_bytes(2 ** 31 - 8193, 4, 8, 0) > 0
    for n in (2 ** 31 - 8192, 2 ** 31 - 4000, 2 ** 31 - 300):
        for backward in (0, 1):
            assert lib.tpk_lm_loss_workspace_bytes(n, 4, 8, backward) == 0
        assert lib.tpk_lm_loss(a, a, a, a, a, n, 4, 8, 1.0, a, big, None, None) == -1
        assert lib.tpk_lm_loss_bwd(a, a, a, a, a, a, a, n, 4, 8, 1.0, a, big, None, None) == -1
