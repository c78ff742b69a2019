"""The projections, the feed-forward block, the rotary forms and the policy
objective as a program uses them: long and wide sums, rows that hold no numbers,
dirty workspaces, other streams, graphs, calls at once, offsets past 32 bits, and a
whole training step over a packed tree.

References are formed in fp64 with torch on the GPU.  Tolerances as in
test_gpu_layer.py; the long sums here: the tensor core's truncation of a chunk of
8,192 elements is at most 512 steps of 2u of the running magnitude, and the chunks
(or splits) are added in fp32: (512 + chunks) 2^-23 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 2.0 ** -8
STEP = 514 * 2.0 ** -23


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available()
    from prefix_tree_packed_dfs_gb300 import ops as o
    return o


def _rnd(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _near(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(err).all(), what
    assert (err <= tol).all(), "%s: off by %.3g" % (what, float((err - tol).max()))


@pytest.mark.parametrize("n,c,o", [
    (70, 64, 9000), (300, 64, 20000),            # dx: a long sum shared by four pairs
    (8200, 64, 72), (20000, 136, 264),           # dw: the same
    (130, 9000, 256), (300, 20000, 64),          # forward: a sum that never stops, shared by four pairs
    (4096, 256, 5000), (19457, 512, 256),        # wide tiles in rounds; narrow ones, dw by four pairs
    (100000, 64, 64), (30000, 200, 72),          # dw: a tile's long column split many ways
])
def test_linear_long_sums(ops, n, c, o):
    x, w, dy = _rnd(1, n, c), _rnd(2, o, c, std=c ** -0.5), _rnd(3, n, o)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = _rnd(4, o, dtype=torch.float32)
    y = ops.linear(x, w, bias=b, residual=dy, dev_err=err)
    dx, dw, db = ops.linear_bwd(x, w, dy, bias=b, dev_err=err)
    assert int(err) == 0
    X, W, D = x.double(), w.double(), dy.double()
    ref = X @ W.T + b.double() + D
    mag = X.abs() @ W.abs().T + b.double().abs()
    _near(y, ref, BF * ref.abs() + (c + 4) * 2.0 ** -23 * (mag + D.abs()), "y")
    ref, mag = D @ W, D.abs() @ W.abs()
    _near(dx, ref, BF * ref.abs() + (STEP + o / 8192 * 2.0 ** -23) * mag, "dx")
    ref, mag = D.T @ X, D.abs().T @ X.abs()
    _near(dw, ref, BF * ref.abs() + (STEP + (n / 8192 + 40) * 2.0 ** -23) * mag, "dw")
    _near(db, D.sum(0), 1100 * U * D.abs().sum(0), "db")   # (at most 1,000 rows in a row per thread)


def test_sums_of_one_sign_do_not_drift(ops):
    """Truncation is a bias: sums of 65,536 positive terms stay within their bf16 rounding."""
    n = 65536
    x = torch.full((n, 64), 1.0, device="cuda").bfloat16()
    dy = _rnd(1, n, 64).abs().bfloat16() + 0.5
    _, dw, _ = ops.linear_bwd(x, _rnd(2, 64, 64), dy)
    ref = dy.double().sum(0)[:, None].expand(64, 64)
    _near(dw, ref, (BF / 2 * 2 + STEP) * ref, "dw")


def test_ffn_long_sums(ops):
    n, c, i = 9000, 264, 8328
    x, w_in, w_out = _rnd(1, n, c), _rnd(2, 2 * i, c, std=c ** -0.5), _rnd(3, c, i, std=i ** -0.5)
    dy = _rnd(4, n, c)
    y, pre, a = ops.gated_ffn(x, w_in, w_out, save=True)
    got = ops.gated_ffn_bwd(x, w_in, w_out, dy, pre, a)
    leaf = [t.double().requires_grad_() for t in (x, w_in, w_out)]
    gu = leaf[0] @ leaf[1].T
    ref = (torch.nn.functional.silu(gu[:, :i]) * gu[:, i:]) @ leaf[2].T
    want = torch.autograd.grad(ref, leaf, dy.double())
    # 2-norms: a, dg, du and the results in bf16 (each at most b / sqrt 3 of the root mean square)
    for p, q, name in zip((y,) + got, (ref.detach(),) + want, ("y", "dx", "dw_in", "dw_out")):
        rel = float((p.double() - q).norm() / q.norm())
        assert rel <= 3 * BF / 3 ** 0.5, (name, rel)


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1.0, 1e6, 1e15])
def test_ffn_gradients_at_any_scale(ops, scale):
    """What the forward keeps holds g and u at any scale, beside larger neighbours too."""
    n, c, i = 200, 64, 160
    x, w_in, w_out = _rnd(1, n, c), _rnd(2, 2 * i, c, std=c ** -0.5).float(), _rnd(3, c, i, std=i ** -0.5)
    w_in[i:] *= scale
    w_in[i::2] *= 1e-2
    w_in = w_in.bfloat16()
    dy = (_rnd(4, n, c).float() / max(scale, 1e-6)).bfloat16()
    y, pre, a = ops.gated_ffn(x, w_in, w_out, save=True)
    got = ops.gated_ffn_bwd(x, w_in, w_out, dy, pre, a)
    leaf = [t.double().requires_grad_() for t in (x, w_in, w_out)]
    gu = leaf[0] @ leaf[1].T
    ref = (torch.nn.functional.silu(gu[:, :i]) * gu[:, i:]) @ leaf[2].T
    want = torch.autograd.grad(ref, leaf, dy.double())
    for p, q, name in zip((y,) + got, (ref.detach(),) + want, ("y", "dx", "dw_in", "dw_out")):
        rel = float((p.double() - q).norm() / q.norm())
        assert rel <= 3 * BF / 3 ** 0.5, (name, rel)


@pytest.mark.parametrize("n", [3, 40, 70, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_hold_no_numbers_stay_alone(ops, n, bad):
    c, o, i = 136, 200, 264
    x, w, w_in, w_out = _rnd(1, n, c), _rnd(2, o, c), _rnd(3, 2 * i, c, std=0.1), _rnd(4, c, i, std=0.1)
    y, f = ops.linear(x, w, act="gelu"), ops.gated_ffn(x, w_in, w_out)
    x2 = x.clone()
    x2[n // 2] = bad
    rest = torch.arange(n, device="cuda") != n // 2
    y2, (f2, pre, a) = ops.linear(x2, w, act="gelu"), ops.gated_ffn(x2, w_in, w_out, save=True)
    f1 = ops.gated_ffn(x2, w_in, w_out)
    assert torch.equal(y2[rest], y[rest]) and torch.equal(f1[rest], f[rest])
    assert torch.isfinite(f2[rest].float()).all() and torch.isfinite(a[rest].float()).all()
    assert not torch.isfinite(f1[n // 2].float()).any()
    dy = _rnd(5, n, c)
    dx = ops.gated_ffn_bwd(x2, w_in, w_out, dy, pre, a)[0]
    clean = ops.gated_ffn(x, w_in, w_out, save=True)
    want = ops.gated_ffn_bwd(x, w_in, w_out, dy, clean[1], clean[2])[0]
    assert torch.equal(dx[rest], want[rest])
    # a channel of the weights that holds none reaches its own column alone
    w2 = w.clone()
    w2[7] = bad
    y3 = ops.linear(x, w2)
    cols = torch.arange(o, device="cuda") != 7
    assert torch.equal(y3[:, cols], ops.linear(x, w)[:, cols])


def test_infinite_and_extreme_scores(ops):
    z = torch.tensor([0.0, -0.0, 3e4, -3e4, 3e38, -3e38, 1e-38, 88.0, -88.0, -104.0], device="cuda")
    x = torch.zeros(len(z), 8, device="cuda")
    x[:, 0] = z
    w = torch.zeros(8, 8, device="cuda").bfloat16()
    w[:, 0] = 1.0
    xb = x.bfloat16()
    zb = xb[:, :1].double().expand(-1, 8)
    fn = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
          "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}
    for name, f in fn.items():
        ref = f(zb)
        _near(ops.linear(xb, w, act=name), ref, BF * ref.abs() + 2.0 ** -20 * (zb.abs().clamp(max=10) + 1), name)
        got = ops.linear_bwd(xb, w, torch.ones(len(z), 8, device="cuda").bfloat16(), act=name)
        assert all(torch.isfinite(t.float()).all() for t in got if t is not None), name


def test_nothing_and_one_row(ops):
    w, b = _rnd(1, 64, 72), _rnd(2, 64, dtype=torch.float32)
    e = _rnd(3, 0, 72)
    assert ops.linear(e, w, bias=b).shape == (0, 64)
    dw = torch.full((64, 72), 7.0, device="cuda").bfloat16()
    db = torch.full((64,), 7.0, device="cuda")
    dx, dw, db = ops.linear_bwd(e, w, _rnd(4, 0, 64), bias=b, act="silu", dw=dw, db=db)
    assert dx.shape == (0, 72) and not dw.any() and not db.any()
    w_in, w_out = _rnd(5, 64, 72), _rnd(6, 72, 32)
    y, pre, a = ops.gated_ffn(e, w_in, w_out, save=True)
    out = ops.gated_ffn_bwd(e, w_in, w_out, _rnd(7, 0, 72), pre, a)
    assert y.shape == (0, 72) and out[0].shape == (0, 72) and not out[1].any() and not out[2].any()
    q = _rnd(8, 0, 2, 64)
    assert ops.rope_by_depth_ex(q, None, torch.zeros(0, dtype=torch.int32, device="cuda"),
                                ops.rope_freqs(64))[0].shape == (0, 2, 64)
    z, i = torch.zeros(0, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    s, d = ops.policy_loss(z, z, z, z, i, torch.zeros(1, dtype=torch.int32, device="cuda"), i,
                           stats=torch.ones(5, device="cuda"))
    assert not s.any() and d.numel() == 0


def _state(seed, n=150, c=264, o=136, i=200):
    t = {"x": _rnd(seed, n, c), "w": _rnd(seed + 1, o, c, std=0.06), "b": _rnd(seed + 2, o, dtype=torch.float32),
         "r": _rnd(seed + 3, n, o), "dy": _rnd(seed + 4, n, o), "wi": _rnd(seed + 5, 2 * i, c, std=0.06),
         "wo": _rnd(seed + 6, c, i, std=0.07), "df": _rnd(seed + 7, n, c), "few": _rnd(seed + 8, 5, c),
         "q": _rnd(seed + 9, n, 4, 64), "k": _rnd(seed + 10, n, 2, 64),
         "depth": torch.randint(0, 5000, (n,), device="cuda", dtype=torch.int32,
                                generator=torch.Generator(device="cuda").manual_seed(seed)),
         "loss": _rnd(seed + 11, n, dtype=torch.float32).abs(), "adv": _rnd(seed + 12, 2 * n, dtype=torch.float32),
         "weight": _rnd(seed + 13, 2 * n, dtype=torch.float32).abs()}
    t["index"] = torch.arange(2 * n, device="cuda", dtype=torch.int32) % n
    t["begin"] = torch.arange(0, 2 * n + 1, 2, device="cuda", dtype=torch.int32)
    t["raw"] = torch.argsort(t["index"], stable=True).to(torch.int32)
    t["old"] = -t["loss"][t["index"].long()] + _rnd(seed + 14, 2 * n, std=0.2, dtype=torch.float32)
    t["seqs"] = torch.tensor([0, n // 3, n, 2 * n], dtype=torch.int32, device="cuda")
    return t


def _all(ops, s):
    f = ops.rope_freqs(32)
    out = [ops.linear(s["x"], s["w"], bias=s["b"], act="gelu", residual=s["r"]), ops.linear(s["few"], s["w"])]
    out += ops.linear_bwd(s["x"], s["w"], s["dy"], bias=s["b"], act="silu")
    y, pre, a = ops.gated_ffn(s["x"], s["wi"], s["wo"], save=True)
    out += [y, a, ops.gated_ffn(s["few"], s["wi"], s["wo"])]
    out += ops.gated_ffn_bwd(s["x"], s["wi"], s["wo"], s["df"], pre, a)
    out += ops.rope_by_depth_ex(s["q"], s["k"], s["depth"], f, interleaved=True)
    for seqs in (None, s["seqs"]):
        out += ops.policy_loss(s["loss"], s["old"], s["adv"], s["weight"], s["index"], s["begin"], s["raw"],
                               ref_logp=s["old"], kl_coef=0.1, seq_offsets=seqs)
    return out


def _same(a, b):
    assert len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))


def test_on_another_stream_and_in_a_graph(ops):
    s = _state(100)
    want = _all(ops, s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _all(ops, s)
    side.synchronize()
    _same(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = _all(ops, s)
    for seed in (200, 300):
        for k, t in _state(seed).items():
            s[k].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        _same(static, _all(ops, s))


def test_many_rounds_in_one_graph_and_beside_another(ops):
    """Two graphs on two streams, each call after call, replayed together."""
    a, b = _state(400), _state(500, n=70)
    wa, wb = _all(ops, a), _all(ops, b)
    graphs, outs = [], []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([_all(ops, s) for _ in range(3)])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, (wa, wb)):
        for rounds in got:
            _same(rounds, want)


def test_two_streams_at_once(ops):
    a, b = _state(600, n=1001), _state(700)
    wa, wb = _all(ops, a), _all(ops, b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ga, gb = [], []
    for _ in range(4):
        with torch.cuda.stream(s1):
            ga.append(_all(ops, a))
        with torch.cuda.stream(s2):
            gb.append(_all(ops, b))
    torch.cuda.synchronize()
    for g in ga:
        _same(g, wa)
    for g in gb:
        _same(g, wb)


def test_dirty_workspaces_of_the_exact_size_and_guarded_outputs(ops):
    lib = ops.B.load()
    s = _state(800, n=300, c=1000, o=552, i=264)
    n, c, o, i = 300, 1000, 552, 264
    y = ops.linear(s["x"], s["w"], bias=s["b"], act="gelu", residual=s["r"])
    g = ops.linear_bwd(s["x"], s["w"], s["dy"], bias=s["b"], act="gelu")
    f, pre, a = ops.gated_ffn(s["x"], s["wi"], s["wo"], save=True)
    h = ops.gated_ffn_bwd(s["x"], s["wi"], s["wo"], s["df"], pre, a)

    def room(nbytes):
        t = torch.full((nbytes + 512,), 0xFF, dtype=torch.uint8, device="cuda")
        return t, t[:nbytes] if nbytes else None

    def checked(nbytes, fn):
        whole, ws = room(int(nbytes))
        got = fn(ws)
        torch.cuda.synchronize()
        assert (whole[int(nbytes):] == 0xFF).all(), "wrote past its workspace"
        return got
    _same([checked(lib.tpk_linear_workspace_bytes(n, c, o, 2, 0),
                   lambda ws: ops.linear(s["x"], s["w"], bias=s["b"], act="gelu", residual=s["r"], workspace=ws))], [y])
    _same(checked(lib.tpk_linear_workspace_bytes(n, c, o, 2, 1),
                  lambda ws: ops.linear_bwd(s["x"], s["w"], s["dy"], bias=s["b"], act="gelu", workspace=ws)), g)
    _same(checked(lib.tpk_gated_ffn_workspace_bytes(n, c, i, c, 0),
                  lambda ws: ops.gated_ffn(s["x"], s["wi"], s["wo"], save=True, workspace=ws))[::2], [f, a])
    _same(checked(lib.tpk_gated_ffn_workspace_bytes(n, c, i, c, 1),
                  lambda ws: ops.gated_ffn_bwd(s["x"], s["wi"], s["wo"], s["df"], pre, a, workspace=ws)), h)
    # saved: of the exact size, guarded
    size = lib.tpk_gated_ffn_saved_bytes(n, i)
    whole, mine = room(int(size))
    ops.gated_ffn(s["x"], s["wi"], s["wo"], save=True, pre=mine)
    _same(ops.gated_ffn_bwd(s["x"], s["wi"], s["wo"], s["df"], mine, a), h)
    assert (whole[int(size):] == 0xFF).all()
    # dw, dx: guarded
    big = torch.full((o + 2, c), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.linear_bwd(s["x"], s["w"], s["dy"], bias=s["b"], act="gelu", dw=big[1:-1])
    assert torch.equal(big[1:-1], g[1]) and (big[0] == 7).all() and (big[-1] == 7).all()


def test_policy_of_one_element_alignment(ops):
    s = _state(900)
    names = ("loss", "old", "adv", "weight", "index", "begin", "raw")
    want = ops.policy_loss(*(s[k] for k in names), ref_logp=s["old"], kl_coef=0.1)
    for shift in (1, 2, 3):
        def moved(t):
            r = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
            r[shift:shift + t.numel()] = t
            return r[shift:shift + t.numel()]
        _same(ops.policy_loss(*(moved(s[k]) for k in names), ref_logp=moved(s["old"]), kl_coef=0.1), want)


def test_policy_long_lists_and_indices_out_of_range(ops):
    """Positions under 1 to 5,000 sequences; tokens that point nowhere carry nothing."""
    seqs, n = 5000, 6
    index = torch.arange(n, device="cuda", dtype=torch.int32).repeat(seqs)
    R = seqs * n
    raw = torch.argsort(index, stable=True).to(torch.int32)
    begin = torch.arange(0, R + 1, seqs, device="cuda", dtype=torch.int32)
    loss, adv, weight = (_rnd(k, m, dtype=torch.float32).abs() for k, m in ((1, n), (2, R), (3, R)))
    old = -loss[index.long()]
    index[::7] = -1
    index[1::7] = n
    _, d = ops.policy_loss(loss, old, adv, weight, index, begin, raw)
    on = ((index >= 0) & (index < n)).double()
    at = index.long().clamp(0, n - 1)
    want = torch.zeros(n, dtype=torch.float64, device="cuda").index_add_(0, at, on * (adv * weight).double())
    _near(d, want, (seqs / 8 + 8) * U * want, "dloss")


def test_offsets_past_32_bits(ops):
    """More than 2^31 elements in rows of y, dy, dx, of what the block keeps, and of the rotated heads."""
    n, c, o = 530000, 64, 4096
    x, w = _rnd(1, n, c), _rnd(2, o, c, std=0.125)
    y = ops.linear(x, w)
    at = torch.tensor([0, 1, 524287, 524288, 524289, n - 1], device="cuda")
    ref = x[at].double() @ w.double().T
    _near(y[at], ref, BF * ref.abs() + (c + 2) * 2.0 ** -23 * (x[at].double().abs() @ w.double().abs().T), "y")
    dx, dw, _ = ops.linear_bwd(x, w, y)
    ref = y[at].double() @ w.double()
    _near(dx[at], ref, BF * ref.abs() + STEP * (y[at].double().abs() @ w.double().abs()), "dx")
    ref = sum(p.double().T @ q.double() for p, q in zip(y.split(65536), x.split(65536)))
    mag = sum(p.double().abs().T @ q.double().abs() for p, q in zip(y.split(65536), x.split(65536)))
    _near(dw, ref, BF * ref.abs() + 2 * STEP * mag, "dw")
    del y, dx
    w_in, w_out = _rnd(3, o, c, std=0.125), _rnd(4, c, o // 2, std=0.02)
    f, pre, a = ops.gated_ffn(x, w_in, w_out, save=True)
    few = ops.gated_ffn(x[at].contiguous(), w_in, w_out)
    assert (f[at].float() - few.float()).abs().max() <= 4 * BF * few.float().abs().max()
    df = _rnd(5, n, c)
    dx = ops.gated_ffn_bwd(x, w_in, w_out, df, pre, a)[0]
    small = ops.gated_ffn(x[at].contiguous(), w_in, w_out, save=True)
    want = ops.gated_ffn_bwd(x[at].contiguous(), w_in, w_out, df[at].contiguous(), *small[1:])[0]
    assert (dx[at].float() - want.float()).abs().max() <= 4 * BF * want.float().abs().max()
    del f, pre, a, dx
    q = _rnd(6, n, 32, 128)
    depth = torch.arange(n, device="cuda", dtype=torch.int32)
    fr = ops.rope_freqs(128)
    got = ops.rope_by_depth_ex(q, None, depth, fr)[0]
    assert torch.equal(got[at], ops.rope_by_depth_ex(q[at].contiguous(), None, depth[at].contiguous(), fr)[0])
    ops.rope_by_depth_ex(q, None, depth, fr, q_out=q)
    assert torch.equal(q, got)


def test_training_step_of_a_layer_over_a_packed_tree(ops):
    """ids -> rows -> norm -> q, k, v -> rotary -> tree attention -> projection onto the residual stream -> norm ->
    feed-forward block -> norm -> vocabulary loss -> policy objective, and all the way back, against fp64 automatic
    differentiation of the same layer with the tree's mask written out.

    Tolerance, in 2-norms: some 10 results each way are rounded to bf16 (2.3e-3 of the root mean square at most) and
    each enters at most two sums further on: 40 x 2.3e-3 if all errors added up, 2^-3.4."""
    rng = np.random.default_rng(11)
    head = rng.integers(0, 300, 60)
    seqs = [np.concatenate([head, rng.integers(0, 300, k)]).astype(np.int32) for k in (40, 75, 22, 90)]
    plan = ops.Plan.from_sequences(seqs, row_capacity=1024, min_shared=8)
    dp = plan.to_device()
    F, R = plan.info["n_fwd"], plan.info["n_raw"]
    Hq, Hkv, d, V = 4, 2, 64, 304
    C, I = Hq * d, 328
    p = {"table": _rnd(1, V, C), "wqkv": _rnd(2, (Hq + 2 * Hkv) * d, C, std=C ** -0.5),
         "bqkv": _rnd(3, (Hq + 2 * Hkv) * d, std=0.1, dtype=torch.float32), "wo": _rnd(4, C, C, std=C ** -0.5),
         "w_in": _rnd(5, 2 * I, C, std=C ** -0.5), "w_out": _rnd(6, C, I, std=I ** -0.5),
         "n1": 1 + _rnd(7, C, std=0.1, dtype=torch.float32), "n2": 1 + _rnd(8, C, std=0.1, dtype=torch.float32),
         "n3": 1 + _rnd(9, C, std=0.1, dtype=torch.float32), "head": _rnd(10, V, C, std=C ** -0.5)}
    ids = ops.gather_to_forwarded(dp, torch.from_numpy(np.concatenate(seqs)).cuda())
    nxt = np.concatenate([np.append(s[1:], -1) for s in seqs]).astype(np.int32)
    target = ops.gather_to_forwarded(dp, torch.from_numpy(nxt).cuda())
    weight = torch.from_numpy((nxt >= 0).astype(np.float32) / R).cuda()
    adv = _rnd(12, R, dtype=torch.float32)
    freqs = ops.rope_freqs(32, 1e4, stretch=2.0)
    rope = dict(interleaved=True, factor=1.1)

    # forward
    emb = ops.embed(p["table"], ids)
    _, x1 = ops.block_norm(emb, p["n1"])
    qkv = ops.linear(x1, p["wqkv"], bias=p["bqkv"])
    q, k = qkv[:, :C].unflatten(1, (Hq, d)), qkv[:, C:C + Hkv * d].unflatten(1, (Hkv, d))
    v = qkv[:, C + Hkv * d:].unflatten(1, (Hkv, d)).contiguous()
    rq, rk = ops.rope_by_depth_ex(q, k, dp.depth, freqs, **rope)
    o, lse = ops.tree_attn_fwd(dp, rq, rk, v, precise=False)
    mid = ops.linear(o.flatten(1), p["wo"], residual=emb)
    _, x2 = ops.block_norm(mid, p["n2"])
    out, pre, a = ops.gated_ffn(x2, p["w_in"], p["w_out"], residual=mid, save=True)
    _, x3 = ops.block_norm(out, p["n3"])
    loss, lse_v = ops.lm_loss(x3, p["head"], target)
    old = -ops.scatter_token_index(dp.token_index, lse_src=loss[None])[1][0] + _rnd(13, R, std=0.1, dtype=torch.float32)
    ref = old + _rnd(14, R, std=0.1, dtype=torch.float32)
    # the clip's borders stay away from every ratio, on which side a token falls is not the question here
    stats, dloss = ops.policy_loss(loss, old, adv, weight, dp.token_index, dp.fwd_raw_begin, dp.fwd_raw, ref_logp=ref,
                                   clip_low=0.9, clip_high=9.0, kl_coef=0.05)
    # backward
    dx3, dhead = ops.lm_loss_bwd(x3, p["head"], target, lse_v, dloss)
    dout, _, _, _, dn3 = ops.block_norm_bwd(out, p["n3"], dx3)
    dx2, dw_in, dw_out = ops.gated_ffn_bwd(x2, p["w_in"], p["w_out"], dout, pre, a)
    dmid, _, _, _, dn2 = ops.block_norm_bwd(mid, p["n2"], dx2, dres_out=dout)
    do, dwo, _ = ops.linear_bwd(o.flatten(1), p["wo"], dmid)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = ops.tree_attn_bwd(dp, rq, rk, v, o, lse, do.unflatten(1, (Hq, d)))
    ops.rope_by_depth_ex(dq, dk, dp.depth, freqs, inverse=True, q_out=dqkv[:, :C].unflatten(1, (Hq, d)),
                         k_out=dqkv[:, C:C + Hkv * d].unflatten(1, (Hkv, d)), **rope)
    dqkv[:, C + Hkv * d:] = dv.flatten(1)
    dx1, dwqkv, dbqkv = ops.linear_bwd(x1, p["wqkv"], dqkv, bias=p["bqkv"])
    demb, _, _, _, dn1 = ops.block_norm_bwd(emb, p["n1"], dx1, dres_out=dmid)
    dtable = ops.embed_bwd(ids, demb, V)
    got = dict(table=dtable, wqkv=dwqkv, bqkv=dbqkv, wo=dwo, w_in=dw_in, w_out=dw_out, n1=dn1, n2=dn2, n3=dn3, head=dhead)

    # fp64
    w = {n: t.double().requires_grad_() for n, t in p.items()}

    def norm(t, s):
        return t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6) * s

    def turn(t):
        angle = dp.depth.double()[:, None] * torch.from_numpy(freqs).cuda()
        c, s = (1.1 * torch.cos(angle))[:, None], (1.1 * torch.sin(angle))[:, None]
        a_, b_ = t[..., 0:32:2], t[..., 1:32:2]
        return torch.cat([torch.stack([a_ * c - b_ * s, a_ * s + b_ * c], 3).flatten(2), t[..., 32:]], 2)
    e = w["table"][ids.long()]
    z = norm(e, w["n1"]) @ w["wqkv"].T + w["bqkv"]
    Q = turn(z[:, :C].unflatten(1, (Hq, d))).transpose(0, 1)
    K = turn(z[:, C:C + Hkv * d].unflatten(1, (Hkv, d))).repeat_interleave(Hq // Hkv, 1).transpose(0, 1)
    Vv = z[:, C + Hkv * d:].unflatten(1, (Hkv, d)).repeat_interleave(Hq // Hkv, 1).transpose(0, 1)
    i = torch.arange(F, device="cuda")
    sees = (i[None] <= i[:, None]) & (i[:, None] < dp.subtree_end.long()[None])
    scores = (Q @ K.transpose(1, 2) / d ** 0.5).masked_fill(~sees[None], float("-inf"))
    att = (torch.softmax(scores, 2) @ Vv).transpose(0, 1).flatten(1)
    m = e + att @ w["wo"].T
    gu = norm(m, w["n2"]) @ w["w_in"].T
    y = m + (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]) @ w["w_out"].T
    logp = torch.log_softmax(norm(y, w["n3"]) @ w["head"].T, 1).gather(1, target.long().clamp(min=0)[:, None])[:, 0]
    on = torch.nonzero(weight)[:, 0]
    lp = logp[dp.token_index.long()[on]]
    ratio, t = torch.exp(lp - old[on].double()), ref[on].double() - lp
    surr = torch.minimum(ratio * adv[on].double(), ratio.clamp(0.1, 10.0) * adv[on].double())
    total = (weight[on].double() * (0.05 * (torch.expm1(t) - t) - surr)).sum()
    grads = torch.autograd.grad(total, list(w.values()))
    for (name, _), g in zip(w.items(), grads):
        rel = float((got[name].double() - g).norm() / g.norm())
        assert rel <= 2.0 ** -3.4, (name, rel)
    assert abs(float(stats[0]) - float(total.detach())) <= 2.0 ** -3.4 * float((weight * adv.abs()).sum())
