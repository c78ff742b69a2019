"""gelu far below 0, where Phi is small: it keeps its relative precision in every
form of the products.

Tolerance: half a bf16 step, 2^-8 of the value at most, and the relative error of
the fit that Phi is formed with (Abramowitz and Stegun 7.1.26), from its
coefficients in fp64, with 2^-16 for fp32 arithmetic (the exponential's argument
is up to 36, off by 2^-23 of that).
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = 2.0 ** -8


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available()
    from prefix_tree_packed_dfs_gb300 import ops as o
    return o


def _tail(n):
    """n scores from -1.5 to -7, exact in bf16, their gelu, and the tolerance relative to it."""
    z = -(1.5 + (np.arange(n) % 89) / 16.0)
    phi = np.array([0.5 * math.erfc(-v / math.sqrt(2)) for v in z])
    x = -z / math.sqrt(2)
    t = 1 / (1 + 0.3275911 * x)
    fit = 0.5 * t * np.polyval([1.061405429, -1.453152027, 1.421413741, -0.284496736, 0.254829592], t) * np.exp(-x * x)
    return z, z * phi, BF + 2.0 ** -16 + np.abs(fit / phi - 1)


@pytest.mark.parametrize("n,c,o,form", [(60, 64, 8, "few"), (300, 64, 264, "narrow"), (4096, 256, 5000, "wide"),
                                        (4922, 8016, 200, "wide")])
def test_gelu_keeps_its_tail(ops, n, c, o, form):
    assert ops.linear_plan(n, c, o)["y"]["form"] == form
    z, want, rel = _tail(n)
    x, w = torch.zeros(n, c, device="cuda").bfloat16(), torch.zeros(o, c, device="cuda").bfloat16()
    x[:, 0], w[:, 0] = torch.from_numpy(z).cuda(), 1.0
    got = ops.linear(x, w, act="gelu").double().cpu().numpy()
    off = np.abs(got / want[:, None] - 1) - rel[:, None]
    assert (off <= 0).all(), (z[np.argmax(off) // o], off.max())


@pytest.mark.parametrize("n", [60, 300])
def test_a_gated_tail_that_a_large_factor_brings_back(ops, n):
    z, want, rel = _tail(n)
    c, i = 64, 136
    x, w_in = torch.zeros(n, c, device="cuda").bfloat16(), torch.zeros(2 * i, c, device="cuda").bfloat16()
    x[:, 0], x[:, 1] = torch.from_numpy(z).cuda(), 2.0 ** 20
    w_in[:i, 0], w_in[i:, 1] = 1.0, 1.0
    w_out = torch.zeros(8, i, device="cuda").bfloat16()
    w_out[:, 5] = 1.0
    y, pre, a = ops.gated_ffn(x, w_in, w_out, act="gelu", save=True)
    for got in (a, ops.gated_ffn(x, w_in, w_out, act="gelu"), y):   # (y rounds a once more, to itself)
        off = np.abs(got.double().cpu().numpy() / (want * 2.0 ** 20)[:, None] - 1) - rel[:, None]
        assert (off <= 0).all(), (z[np.argmax(off) // got.shape[1]], off.max())
    # du = dy w_out gelu(g), which is 8 gelu(g) in the one channel that w_out takes, and dx of the up channel their sum;
    # rounded twice, from g kept within 2^-11 of itself, whose |z phi / Phi| <= z^2 + 1 = 50 times enter gelu
    dx = ops.gated_ffn_bwd(x, w_in, w_out, torch.ones(n, 8, device="cuda").bfloat16(), pre, a, act="gelu")[0]
    off = np.abs(dx[:, 1].double().cpu().numpy() / (8 * want) - 1) - (rel + BF + 51 * 2.0 ** -11)
    assert (off <= 0).all(), off.max()
