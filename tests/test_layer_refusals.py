"""Argument checks of the projections, the feed-forward block, the rotary forms
and the policy objective: every refusal comes before any launch (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from prefix_tree_packed_dfs_gb300 import binding as B
from prefix_tree_packed_dfs_gb300 import ops

P = ctypes.c_void_p
ARG, UNSUPPORTED, OVERFLOW, WORKSPACE = -1, -4, -3, -7
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _bf(*shape):
    return torch.zeros(*shape, dtype=BF)


def test_linear_refuses_on_the_host(lib):
    ok = dict(x=P(256), ld_x=64, w=P(512), b=None, act=0, r=None, ld_r=0, y=P(1024), ld_y=128, n=70, c=64, o=128,
              ws=P(4096), ws_bytes=1 << 30)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.tpk_linear(a["x"], a["ld_x"], a["w"], a["b"], a["act"], a["r"], a["ld_r"], a["y"], a["ld_y"], a["n"],
                              a["c"], a["o"], a["ws"], a["ws_bytes"], None, None)
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(x=P(8)), dict(w=P(24)), dict(y=P(1032)), dict(b=P(4)),
               dict(r=P(8), ld_r=128), dict(r=P(16), ld_r=120), dict(ld_x=56), dict(ld_x=68), dict(ld_y=120),
               dict(ld_y=132), dict(n=-1), dict(c=0), dict(c=60), dict(o=4), dict(o=130), dict(act=-1), dict(act=4),
               dict(o=(1 << 20) + 8, ld_y=1 << 21), dict(n=(1 << 31) - 8192), dict(y=P(256)), dict(y=P(512))):
        assert call(**kw) == ARG, kw
    assert call(c=32776, ld_x=32776) == UNSUPPORTED
    assert call(n=(1 << 31) - 8200, o=1 << 20, ld_y=1 << 20) == OVERFLOW
    assert call(n=0, x=None, w=None, y=None) == 0
    need = lib.tpk_linear_workspace_bytes(100, 8192, 256, 0, 0)
    if need:   # a split over K
        assert call(n=100, c=8192, ld_x=8192, o=256, ld_y=256, ws=None, ws_bytes=0) == WORKSPACE
        assert call(n=100, c=8192, ld_x=8192, o=256, ld_y=256, ws_bytes=need - 1) == WORKSPACE
    assert lib.tpk_linear_workspace_bytes(0, 64, 64, 0, 1) == 0
    assert lib.tpk_linear_workspace_bytes(10, 60, 64, 0, 1) == 0
    assert lib.tpk_linear_workspace_bytes(B.FEW_ROWS, 8192, 256, 0, 0) == 0       # a few rows need none


def test_linear_bwd_refuses_on_the_host(lib):
    ok = dict(x=P(256), ld_x=64, w=P(512), b=None, act=1, dy=P(768), ld_dy=128, dx=P(1024), ld_dx=64, dw=P(2048),
              db=None, n=70, c=64, o=128, ws=P(4096), ws_bytes=1 << 30)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.tpk_linear_bwd(a["x"], a["ld_x"], a["w"], a["b"], a["act"], a["dy"], a["ld_dy"], a["dx"], a["ld_dx"],
                                  a["dw"], a["db"], a["n"], a["c"], a["o"], a["ws"], a["ws_bytes"], None, None)
    for kw in (dict(x=None), dict(w=None), dict(dy=None), dict(dx=None), dict(dw=None), dict(db=P(4)), dict(ld_dy=120),
               dict(ld_dx=60), dict(ld_dx=56), dict(dw=P(8)), dict(dx=P(8)), dict(dx=P(256)), dict(dx=P(768)), dict(c=12, ld_x=16, ld_dx=16)):
        assert call(**kw) == ARG, kw
    assert call(ws=None) == WORKSPACE and call(ws=P(4100)) == WORKSPACE
    assert call(ws_bytes=lib.tpk_linear_workspace_bytes(70, 64, 128, 1, 1) - 1) == WORKSPACE


def test_gated_ffn_refuses_on_the_host(lib):
    ok = dict(x=P(256), ld_x=64, wi=P(512), wo=P(768), act=1, r=None, ld_r=0, saved=None, a=None, y=P(1024), ld_y=64,
              n=70, c=64, i=128, o=64, ws=P(4096), ws_bytes=1 << 30)

    def call(**kw):
        q = dict(ok, **kw)
        return lib.tpk_gated_ffn(q["x"], q["ld_x"], q["wi"], q["wo"], q["act"], q["r"], q["ld_r"], q["saved"], q["a"],
                                 q["y"], q["ld_y"], q["n"], q["c"], q["i"], q["o"], q["ws"], q["ws_bytes"], None, None)
    for kw in (dict(x=None), dict(wi=None), dict(wo=None), dict(y=None), dict(saved=P(8)), dict(a=P(8)), dict(i=100),
               dict(i=0), dict(o=12, ld_y=16), dict(act=7), dict(ld_x=60), dict(r=P(16), ld_r=8), dict(y=P(256))):
        assert call(**kw) == ARG, kw
    for kw in (dict(c=32776, ld_x=32776), dict(i=32776), dict(o=32776, ld_y=32776)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(ws=None) == WORKSPACE and call(ws_bytes=16) == WORKSPACE
    assert call(n=0, x=None) == 0
    bwd = lambda **kw: lib.tpk_gated_ffn_bwd(*[dict(
        x=P(256), ld_x=64, wi=P(512), wo=P(768), act=1, dy=P(1024), ld_dy=64, saved=P(2048), a=P(4096), dx=P(8192),
        ld_dx=64, dwi=P(16384), dwo=P(32768), n=70, c=64, i=128, o=64, ws=P(65536), ws_bytes=1 << 30,
        **{})[k] if k not in kw else kw[k] for k in ("x", "ld_x", "wi", "wo", "act", "dy", "ld_dy", "saved", "a", "dx",
                                                     "ld_dx", "dwi", "dwo", "n", "c", "i", "o", "ws", "ws_bytes")],
        None, None)
    for kw in (dict(saved=None), dict(a=None), dict(dwi=None), dict(dwo=P(8)), dict(dx=None), dict(ld_dy=56), dict(dx=P(256)), dict(dx=P(1024))):
        assert bwd(**kw) == ARG, kw
    assert bwd(ws=None) == WORKSPACE and bwd(ws_bytes=64) == WORKSPACE
    assert lib.tpk_gated_ffn_saved_bytes(70, 100) == 0 and lib.tpk_gated_ffn_saved_bytes(70, 128) > 70 * 128 * 4


def test_rope_forms_refuse_on_the_host(lib):
    freqs = (ctypes.c_double * 128)(*[0.1] * 128)

    def call(rot=64, inter=0, factor=1.0, fr=freqs, q=P(256), ldq=256, qo=P(512), ldqo=256, k=None, ko=None, F=3, Hq=2,
             Hkv=0, d=128, depth=P(64)):
        o = B.RopeOpts(rot, inter, factor, ctypes.cast(fr, P) if fr is not None else None)
        return lib.tpk_rope_by_depth_ex(q, ldq, k, 256, qo, ldqo, ko, 256, depth, F, Hq, Hkv, d, ctypes.byref(o), 0, None)
    bad = (ctypes.c_double * 128)(*[0.1] * 31 + [float("nan")] * 97)
    for kw in (dict(rot=8), dict(rot=24), dict(rot=144), dict(rot=0), dict(inter=2), dict(factor=float("inf")),
               dict(fr=None), dict(fr=bad), dict(q=P(8)), dict(qo=None), dict(ldq=248), dict(ldqo=260), dict(Hq=0),
               dict(d=100), dict(d=520), dict(depth=None), dict(F=-1), dict(qo=P(256), ldqo=512),
               dict(k=P(1024), ko=P(2048))):
        assert call(**kw) == ARG, kw
    assert call(F=0) == 0 and call(q=None, qo=None) == 0
    assert lib.tpk_rope_by_depth_ex(P(256), 256, None, 0, P(512), 256, None, 0, P(64), 3, 2, 0, 128, None, 0, None) == ARG


def test_policy_refuses_on_the_host(lib):
    def call(lo=0.2, hi=0.2, dual=0.0, kl=0.0, R=10, F=8, seq=None, n=0, ws=P(4096), ws_bytes=1 << 20, stats=P(64),
             drop=None, opts=True):
        o = B.PolicyOpts(lo, hi, dual, kl)
        a = [P(64)] * 8
        a[2] = None
        if drop is not None:
            a[drop] = None
        return lib.tpk_policy_loss(*a, seq, n, ctypes.byref(o) if opts else None, stats, P(64), R, F, ws, ws_bytes, None)
    for kw in (dict(lo=-0.1), dict(lo=1.5), dict(lo=float("nan")), dict(hi=-1.0), dict(dual=0.5), dict(dual=1.0),
               dict(kl=-1.0), dict(kl=float("inf")), dict(R=-1), dict(F=11), dict(stats=None), dict(opts=False),
               dict(n=3), dict(seq=P(64), n=0), dict(R=1 << 31), *[dict(drop=i) for i in (0, 1, 3, 4, 5, 6, 7)]):
        assert call(**kw) == ARG, kw
    assert call(ws=None) == WORKSPACE and call(ws=P(4100)) == WORKSPACE and call(ws_bytes=8) == WORKSPACE


def test_wrappers_name_what_is_wrong(lib):
    x, w = _bf(3, 64), _bf(16, 64)
    for err, text, fn in (
            (TypeError, "x", lambda: ops.linear(x.float(), w)),
            (TypeError, "w", lambda: ops.linear(x, w.half())),
            (ValueError, "w must have shape", lambda: ops.linear(x, _bf(16, 72))),
            (ValueError, "w must be contiguous", lambda: ops.linear(x, _bf(64, 16).T)),
            (ValueError, "multiple of 8 channels", lambda: ops.linear(_bf(3, 60), _bf(16, 60))),
            (ValueError, "multiple of 8 rows", lambda: ops.linear(x, _bf(12, 64))),
            (ValueError, "act", lambda: ops.linear(x, w, act="relu")),
            (ValueError, "bias", lambda: ops.linear(x, w, bias=torch.zeros(8))),
            (TypeError, "bias", lambda: ops.linear(x, w, bias=_bf(16))),
            (ValueError, "residual", lambda: ops.linear(x, w, residual=_bf(3, 24))),
            (ValueError, "out", lambda: ops.linear(x, w, out=_bf(16, 3).T)),
            (ValueError, "rows must not overlap", lambda: ops.linear(_bf(200).as_strided((3, 64), (8, 1)), w)),
            (ValueError, "no CPU path", lambda: ops.linear(x, w)),
            (ValueError, "db is given", lambda: ops.linear_bwd(x, w, _bf(3, 16), db=torch.zeros(16))),
            (ValueError, "dy", lambda: ops.linear_bwd(x, w, _bf(3, 24))),
            (ValueError, "no CPU path", lambda: ops.linear_bwd(x, w, _bf(3, 16))),
            (ValueError, "w_out must have shape", lambda: ops.gated_ffn(x, _bf(16, 64), _bf(64, 16))),
            (ValueError, "w_in must have shape", lambda: ops.gated_ffn(x, _bf(16, 72), _bf(64, 8))),
            (ValueError, "twice a multiple", lambda: ops.gated_ffn(x, _bf(24, 64), _bf(64, 12))),
            (ValueError, "save=True", lambda: ops.gated_ffn(x, _bf(32, 64), _bf(64, 16), a=_bf(3, 16))),
            (ValueError, "no CPU path", lambda: ops.gated_ffn(x, _bf(32, 64), _bf(64, 16))),
            (TypeError, "pre", lambda: ops.gated_ffn_bwd(x, _bf(32, 64), _bf(64, 16), x, _bf(3, 32), _bf(3, 16))),
            (TypeError, "3-d", lambda: ops.rope_by_depth_ex(x, None, torch.zeros(3, dtype=I32), ops.rope_freqs(16))),
            (ValueError, "freqs", lambda: ops.rope_by_depth_ex(_bf(3, 1, 64), None, torch.zeros(3, dtype=I32),
                                                               ops.rope_freqs(128))),
            (ValueError, "depth", lambda: ops.rope_by_depth_ex(_bf(3, 1, 64), None, torch.zeros(4, dtype=I32),
                                                               ops.rope_freqs(64))),
            (ValueError, "k_out is given", lambda: ops.rope_by_depth_ex(_bf(3, 1, 64), None, torch.zeros(3, dtype=I32),
                                                                        ops.rope_freqs(64), k_out=_bf(3, 1, 64))),
            (ValueError, "k must have shape", lambda: ops.rope_by_depth_ex(_bf(3, 1, 64), _bf(2, 1, 64),
                                                                           torch.zeros(3, dtype=I32), ops.rope_freqs(64))),
    ):
        with pytest.raises(err, match=text):
            fn()
    z, i = torch.zeros(3), torch.zeros(3, dtype=I32)
    b = torch.zeros(4, dtype=I32)
    for err, text, fn in (
            (TypeError, "tensors", lambda: ops.policy_loss([1.0], z, z, z, i, b, i)),
            (TypeError, "old_logp", lambda: ops.policy_loss(z, z.double(), z, z, i, b, i)),
            (ValueError, "advantage", lambda: ops.policy_loss(z, z, torch.zeros(2), z, i, b, i)),
            (ValueError, "fwd_raw_begin", lambda: ops.policy_loss(z, z, z, z, i, i, i)),
            (ValueError, "clip_low", lambda: ops.policy_loss(z, z, z, z, i, b, i, clip_low=2.0)),
            (ValueError, "clip_low", lambda: ops.policy_loss(z, z, z, z, i, b, i, dual_clip=0.5)),
            (ValueError, "at least one sequence", lambda: ops.policy_loss(z, z, z, z, i, b, i, seq_offsets=i[:1])),
            (ValueError, "more than", lambda: ops.policy_loss(torch.zeros(5), z, z, z, i, torch.zeros(6, dtype=I32), i)),
            (ValueError, "no CPU path", lambda: ops.policy_loss(z, z, z, z, i, b, i))):
        with pytest.raises(err, match=text):
            fn()


def test_rope_freqs():
    f = ops.rope_freqs(64, 1e4)
    assert np.allclose(f, 1e4 ** (-np.arange(32) / 32.0), rtol=1e-15)
    assert np.allclose(ops.rope_freqs(64, 1e4, stretch=4.0), f / 4)
    s = ops.rope_freqs(64, 1e4, stretch=4.0, trained=4096)
    turns = 4096 * f / (2 * np.pi)
    assert (s[turns >= 32] == f[turns >= 32]).all() and np.allclose(s[turns <= 1], f[turns <= 1] / 4)
    assert ((s <= f) & (s >= f / 4 * (1 - 1e-15))).all()
    with pytest.raises(ValueError):
        ops.rope_freqs(64, trained=10, fast=1.0, slow=2.0)
