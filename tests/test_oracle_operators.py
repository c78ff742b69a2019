"""Pins of the fp64 oracle of the operators around the token mixers, and the
wrappers' refusals before any launch (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import operators as oo

RNG = np.random.default_rng


def _diff(f, x, d, h=1e-5):
    """Central difference of the scalar f at x along d."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_embed_rows_and_transpose():
    g = RNG(1)
    table, tokens = g.normal(size=(7, 8)), np.array([3, 0, 6, 3, -1, 7, 3])
    out = oo.embed(table, tokens, 2.0)
    assert np.array_equal(out[0], 2 * table[3]) and np.array_equal(out[2], 2 * table[6])
    assert not out[4].any() and not out[5].any()
    y = g.normal(size=out.shape)
    # <embed(table), y> = <table, embed_bwd(y)>: the gradient is the transpose
    assert np.isclose((out * y).sum(), (table * oo.embed_bwd(tokens, y, 7, 2.0)).sum())


@pytest.mark.parametrize("post,gate,y", [(True, True, True), (True, False, True), (False, True, True),
                                         (False, False, True), (False, False, False)])
def test_block_norm_gradients_match_differences(post, gate, y):
    g = RNG(2)
    n, c = 5, 16
    a = {"res": g.normal(size=(n, c)), "w_pre": g.normal(size=c)}
    if y:
        a["y"] = g.normal(size=(n, c))
    if post:
        a["w_post"] = g.normal(size=c)
    if gate:
        a["gate"] = g.normal(size=(n, c))
    dr, dx = g.normal(size=(n, c)), g.normal(size=(n, c))
    names = ["res", "y", "gate", "w_post", "w_pre"]
    got = dict(zip(names, oo.block_norm_bwd(dx=dx, dres_out=dr, scale=0.7, eps=1e-3, **a)))
    for k in names:
        if k not in a:
            assert got[k] is None
            continue

        def total(v, k=k):
            r, x = oo.block_norm(scale=0.7, eps=1e-3, **dict(a, **{k: v}))
            return (r * dr).sum() + (x * dx).sum()
        d = g.normal(size=a[k].shape)
        assert np.isclose(_diff(total, a[k], d), (got[k] * d).sum(), rtol=1e-6, atol=1e-7), k


def test_block_norm_closed_form():
    # y with unit mean square, unit weights, eps 0: u = y, and a gate of zero halves it
    y = np.array([[1.0, -1.0] * 4])
    r, x = oo.block_norm(np.zeros((1, 8)), np.ones(8), y, np.ones(8), np.zeros((1, 8)), scale=4.0, eps=0.0)
    assert np.allclose(r, 2 * y) and np.allclose(x, y)


def test_lm_loss_uniform_and_gradients():
    n, v, c = 4, 9, 8
    loss, lse = oo.lm_loss(np.zeros((n, c)), np.ones((v, c)), np.array([0, 8, -1, 9]))
    assert np.allclose(loss[:2], np.log(v)) and np.allclose(lse[:2], np.log(v)) and not loss[2:].any()
    g = RNG(3)
    h, w, t, dl = g.normal(size=(n, c)), g.normal(size=(v, c)), np.array([2, -1, 0, 8]), g.normal(size=n)
    dh, dw = oo.lm_loss_bwd(h, w, t, dl, 1.3)
    assert not dh[1].any()
    d = g.normal(size=h.shape)
    assert np.isclose(_diff(lambda a: (dl * oo.lm_loss(a, w, t, 1.3)[0]).sum(), h, d), (dh * d).sum(), rtol=1e-6)
    d = g.normal(size=w.shape)
    assert np.isclose(_diff(lambda a: (dl * oo.lm_loss(h, a, t, 1.3)[0]).sum(), w, d), (dw * d).sum(), rtol=1e-6)
    # the scores' gradients of a position add up to zero
    assert np.allclose(oo.score_grads(h, w, t, dl, 1.3).sum(axis=1), 0)


# ---- refusals ------------------------------------------------------------------

def _b(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _i(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_embed_refusals(lib):
    from prefix_tree_packed_dfs_gb300 import ops
    with pytest.raises(TypeError):
        ops.embed(_b(4, 8).half(), _i(3))
    with pytest.raises(TypeError):
        ops.embed(_b(4, 8), _i(3).long())
    with pytest.raises(ValueError):
        ops.embed(_b(4, 12), _i(3))                       # width not a multiple of 8
    with pytest.raises(ValueError):
        ops.embed(_b(0, 8), _i(3))
    with pytest.raises(ValueError):
        ops.embed(_b(4, 16)[:, :8], _i(3))                # not contiguous
    with pytest.raises(ValueError):
        ops.embed(_b(4, 8), _i(3), out=_b(2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ops.embed(_b(4, 8), _i(3))
    with pytest.raises(ValueError):
        ops.embed_bwd(_i(3), _b(2, 8), 4)
    with pytest.raises(ValueError):
        ops.embed_bwd(_i(3), _b(3, 8), 0)
    with pytest.raises(TypeError):
        ops.embed_bwd(_i(3), _b(3, 8), 4, dtype=torch.float16)
    with pytest.raises(ValueError):
        ops.embed_bwd(_i(3), _b(3, 8), 4, dtable=torch.zeros(5, 8))
    with pytest.raises(ValueError, match="workspace"):
        ops.embed_bwd(_i(3), _b(3, 8), 4, workspace=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        ops.embed_bwd(_i(3), _b(3, 8), 4)


def test_block_norm_refusals(lib):
    from prefix_tree_packed_dfs_gb300 import ops
    w = torch.ones(16)
    with pytest.raises(TypeError):
        ops.block_norm(torch.zeros(2, 16), w)
    with pytest.raises(TypeError):
        ops.block_norm(_b(2, 16), w.double())
    with pytest.raises(ValueError):
        ops.block_norm(_b(2, 12), torch.ones(12))
    with pytest.raises(ValueError):
        ops.block_norm(_b(2, 16), torch.ones(8))
    with pytest.raises(ValueError):
        ops.block_norm(_b(2, 16), w, gate=_b(2, 16))      # a gate without y
    with pytest.raises(ValueError):
        ops.block_norm(_b(2, 16), w, y=_b(3, 16))
    with pytest.raises(ValueError):
        ops.block_norm(_b(2, 16), w, y=_b(1, 16).expand(2, 16))      # rows overlap
    with pytest.raises(ValueError):
        ops.block_norm(_b(2, 16), w, y=_b(2, 20)[:, :16])            # rows not 16-byte aligned
    with pytest.raises(ValueError):
        ops.block_norm(_b(2, 16), w, y=_b(16, 2).T)
    with pytest.raises(ValueError, match="CUDA"):
        ops.block_norm(_b(2, 16), w, y=_b(2, 32)[:, 16:])
    with pytest.raises(ValueError):
        ops.block_norm_bwd(_b(2, 16), w, _b(2, 16), dy=_b(2, 16))    # gradient of a missing input
    with pytest.raises(ValueError):
        ops.block_norm_bwd(_b(2, 16), w, _b(2, 16), y=_b(2, 16), dy=_b(1, 16).expand(2, 16))
    with pytest.raises(ValueError, match="CUDA"):
        ops.block_norm_bwd(_b(2, 16), w, _b(2, 16), y=_b(2, 16))


def test_lm_loss_refusals(lib):
    from prefix_tree_packed_dfs_gb300 import ops
    f = torch.zeros(3)
    with pytest.raises(TypeError):
        ops.lm_loss(torch.zeros(3, 8), _b(5, 8), _i(3))
    with pytest.raises(ValueError):
        ops.lm_loss(_b(3, 8), _b(5, 16), _i(3))
    with pytest.raises(ValueError):
        ops.lm_loss(_b(3, 8), _b(0, 8), _i(3))
    with pytest.raises(ValueError):
        ops.lm_loss(_b(3, 8), _b(5, 8), _i(2))
    with pytest.raises(ValueError):
        ops.lm_loss(_b(3, 12), _b(5, 12), _i(3))
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        with pytest.raises(ValueError):
            ops.lm_loss(_b(3, 8), _b(5, 8), _i(3), scale=bad)
    with pytest.raises(ValueError, match="CUDA"):
        ops.lm_loss(_b(3, 8), _b(5, 8), _i(3))
    with pytest.raises(TypeError):
        ops.lm_loss_bwd(_b(3, 8), _b(5, 8), _i(3), f.double(), f)
    with pytest.raises(ValueError):
        ops.lm_loss_bwd(_b(3, 8), _b(5, 8), _i(3), f, f, dw=_b(4, 8))
    with pytest.raises(ValueError, match="workspace"):
        ops.lm_loss_bwd(_b(3, 8), _b(5, 8), _i(3), f, f, workspace=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        ops.lm_loss_bwd(_b(3, 8), _b(5, 8), _i(3), f, f)


def test_entry_points_reject_bad_arguments_before_any_device_call(lib):
    P = ctypes.c_void_p
    a = P(4096)
    # sizes, types, NULL pointers, misalignment: TPK_E_ARG (-1); workspaces: TPK_E_WORKSPACE (-7)
    assert lib.tpk_embed(a, 0, a, a, 4, 4, 12, 1.0, None) == -1
    assert lib.tpk_embed(a, 2, a, a, 4, 4, 8, 1.0, None) == -1
    assert lib.tpk_embed(None, 0, a, a, 4, 4, 8, 1.0, None) == -1
    assert lib.tpk_embed(P(4104), 0, a, a, 4, 4, 8, 1.0, None) == -1
    assert lib.tpk_embed(a, 0, a, a, -1, 4, 8, 1.0, None) == -1
    assert lib.tpk_embed(a, 0, None, None, 0, 4, 8, 1.0, None) == 0
    assert lib.tpk_embed_bwd(a, a, None, 1, 4, 4, 8, 1.0, a, 1 << 20, None) == -1
    assert lib.tpk_embed_bwd(a, a, a, 1, 4, 4, 8, 1.0, None, 0, None) == -7
    assert lib.tpk_embed_bwd(a, a, a, 1, 4, 4, 8, 1.0, P(4112), 1 << 20, None) == -7
    assert lib.tpk_block_norm(a, None, 8, a, 8, None, a, a, a, 4, 8, 1.0, 1e-6, None) == -1     # gate without y
    assert lib.tpk_block_norm(a, a, 4, None, 8, None, a, a, a, 4, 8, 1.0, 1e-6, None) == -1     # rows overlap
    assert lib.tpk_block_norm(a, a, 8, None, 8, None, a, None, a, 4, 8, 1.0, 1e-6, None) == -1  # res_out missing
    assert lib.tpk_block_norm(a, a, 8, None, 8, None, a, a, a, 4, 8, 1.0, -1.0, None) == -1
    assert lib.tpk_block_norm(a, a, 16392, None, 8, None, a, a, a, 4, 16392, 1.0, 1e-6, None) == -4
    assert lib.tpk_block_norm(None, None, 8, None, 8, None, a, None, None, 0, 8, 1.0, 1e-6, None) == 0
    assert lib.tpk_block_norm_bwd(a, a, 8, None, 8, None, a, None, a, a, None, 8, None, 8, None, a, 4, 8, 1.0, 1e-6, a,
                                  1 << 30, None) == -1                                          # dy missing
    assert lib.tpk_block_norm_bwd(a, a, 8, None, 8, None, a, None, a, a, a, 8, None, 8, None, a, 4, 8, 1.0, 1e-6, None,
                                  0, None) == -7
    assert lib.tpk_lm_loss(a, a, a, a, a, 4, 4, 8, 0.0, a, 1 << 30, None, None) == -1
    assert lib.tpk_lm_loss(a, a, a, a, a, 4, 0, 8, 1.0, a, 1 << 30, None, None) == -1
    assert lib.tpk_lm_loss(a, a, a, None, a, 4, 4, 8, 1.0, a, 1 << 30, None, None) == -1
    assert lib.tpk_lm_loss(a, a, a, a, a, 4, 4, 8, 1.0, a, 16, None, None) == -7
    assert lib.tpk_lm_loss(None, a, None, None, None, 0, 4, 8, 1.0, None, 0, None, None) == 0
    assert lib.tpk_lm_loss_bwd(a, a, a, a, a, a, None, 4, 4, 8, 1.0, a, 1 << 40, None, None) == -1
    assert lib.tpk_lm_loss_bwd(a, a, a, a, a, a, a, 4, 4, 8, 1.0, a, 16, None, None) == -7


def test_workspace_sizes(lib):
    # larger problems never need less, and refused sizes ask for nothing
    assert lib.tpk_embed_bwd_workspace_bytes(10, 100, 12) == 0
    assert lib.tpk_lm_loss_workspace_bytes(10, 100, 12, 1) == 0
    assert lib.tpk_block_norm_bwd_workspace_bytes(10, 16392) == 0
    last = 0
    for n in (1, 100, 5000, 100000):
        need = lib.tpk_lm_loss_workspace_bytes(n, 32000, 512, 1)
        assert need >= last
        last = need
    # dz of one piece stays within 4 GiB where a piece of 4,096 ids allows it
    assert lib.tpk_lm_loss_workspace_bytes(100000, 131072, 512, 1) < (6 << 30)
