"""What the operators around the token mixers are measured on.

A training step over packed rows is more than its token mixers: token ids
become hidden rows (``embed``), every block's output is normed, gated and
added to the residual stream and normed again for the next block
(``block_norm``), and the last hidden rows meet the vocabulary in the loss
(``lm_loss``).  Each case below is one call, or one forward and backward, of
one of them.  Sizes are those of the repository's own batches (32,000 token
ids; 2,048 = 16 heads of 128 and 4,096 = 32 heads of 128; 692, 32,768 and
96,888 forwarded positions) and generic odd ones.
"""
import math

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # the token rows of one short packed row, table in the compute type: latency
        {"name": "embed_row_692", "op": "embed", "n": 692, "c": 2048, "v": 32000, "table": "bf16", "pad": 0.0,
         "scale": 1.0},
        # a whole rollout batch, fp32 master table, rows scaled by sqrt(c), a few padding ids
        {"name": "embed_batch_fp32", "op": "embed", "n": 96888, "c": 2048, "v": 32000, "table": "fp32", "pad": 0.02,
         "scale": math.sqrt(2048.0)},
        # the gradient of that table: Zipf token ids, frequent ids hold thousands of rows
        {"name": "embed_bwd_batch", "op": "embed_bwd", "n": 96888, "c": 2048, "v": 32000, "table": "fp32", "pad": 0.02,
         "scale": math.sqrt(2048.0)},
        # a small odd batch against a small odd vocabulary, gradient in the compute type
        {"name": "embed_bwd_odd", "op": "embed_bwd", "n": 1001, "c": 1000, "v": 5003, "table": "bf16", "pad": 0.1,
         "scale": 1.0},
        # one sampled token through a block's norms: the smallest call
        {"name": "norm_token", "op": "norm", "n": 1, "c": 2048, "post": True, "gate": True, "scale": 1.0},
        # every position of a rollout batch, gate taken as a column slice of a fused projection
        {"name": "norm_batch", "op": "norm", "n": 96888, "c": 2048, "post": True, "gate": True, "scale": 0.5},
        # training a wide model on one 32k row
        {"name": "norm_bwd_row", "op": "norm_bwd", "n": 32768, "c": 4096, "post": True, "gate": True, "scale": 0.5},
        # odd rows and an odd width, no gate
        {"name": "norm_bwd_odd", "op": "norm_bwd", "n": 4099, "c": 1000, "post": True, "gate": False, "scale": 1.0},
        # the log-probability of one sampled token
        {"name": "loss_token", "op": "loss", "n": 1, "c": 2048, "v": 32000, "trained": 1.0, "run": 1, "scale": 1.0},
        # reference log-probabilities of a ragged batch, sampled at a temperature; tool output masked
        {"name": "loss_ragged", "op": "loss", "n": 5003, "c": 1024, "v": 50003, "trained": 0.7, "run": 61,
         "scale": 1.25},
        # loss and gradients of a rollout batch: prompts and tool turns carry no loss
        {"name": "loss_step_batch", "op": "loss_step", "n": 96888, "c": 2048, "v": 32000, "trained": 0.8, "run": 512,
         "scale": 1.0},
        # loss and gradients against a large vocabulary and a wide hidden state
        {"name": "loss_step_wide", "op": "loss_step", "n": 8192, "c": 4096, "v": 131072, "trained": 1.0, "run": 1,
         "scale": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_bwd", "norm", "norm_bwd", "loss", "loss", "loss_step", "loss_step"])
    c = 8 * _log(rng, 8, 512)
    if op.startswith("embed"):
        return {"op": op, "n": _log(rng, 1, 96888 * 2048 // max(c, 2048)), "c": c, "v": _log(rng, 100, 32000),
                "table": rng.choice(["bf16", "fp32"]), "pad": rng.choice([0.0, 0.05, 0.3]),
                "scale": rng.choice([1.0, math.sqrt(c)])}
    if op.startswith("norm"):
        return {"op": op, "n": _log(rng, 1, 32768), "c": c, "post": rng.random() < 0.8, "gate": rng.random() < 0.6,
                "scale": rng.choice([1.0, 0.5, 0.1767767])}
    v = _log(rng, 500, 131072)
    most = min(65536, int(2e9 / v), int(2e12 / (float(v) * c)))
    return {"op": op, "n": _log(rng, 1, max(1, most)), "c": c, "v": v, "trained": rng.choice([1.0, 0.8, 0.4, 0.05]),
            "run": _log(rng, 1, 700), "scale": rng.choice([1.0, 1.25, 0.7])}


def _ids(g, n, v):
    # log-uniform ids: the k-th most frequent id comes up about 1/k as often as the first
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return (torch.pow(float(v) + 1.0, u) - 1.0).long().clamp_(0, v - 1).to(torch.int32)


def _bf16(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n, c = case["n"], case["c"]
    s = {"case": case}
    if case["op"].startswith("embed"):
        v = case["v"]
        tok = _ids(g, n, v)
        pad = torch.rand(n, generator=g, device="cuda") < case["pad"]
        s["tokens"] = torch.where(pad, torch.full_like(tok, -1), tok)
        if case["op"] == "embed":
            table = torch.randn(v, c, generator=g, device="cuda") * 0.02
            s["table"] = table if case["table"] == "fp32" else table.bfloat16()
        else:
            s["dout"] = _bf16(g, n, c, std=1.0 / max(1, n))
    elif case["op"].startswith("norm"):
        s["res"] = _bf16(g, n, c, std=2.0)
        s["y"] = _bf16(g, n, c, std=0.7)
        # the gate is a column slice of a fused projection's output
        s["gate"] = _bf16(g, n, 2 * c)[:, c:] if case["gate"] else None
        s["w_post"] = 1.0 + 0.1 * torch.randn(c, generator=g, device="cuda") if case["post"] else None
        s["w_pre"] = 1.0 + 0.1 * torch.randn(c, generator=g, device="cuda")
        if case["op"] == "norm_bwd":
            s["dres_out"] = _bf16(g, n, c, std=1.0 / n)
            s["dx"] = _bf16(g, n, c, std=1.0 / n)
    else:
        v, run_len = case["v"], case["run"]
        w = torch.randn(v, c, generator=g, device="cuda") * (2.0 / math.sqrt(c))
        tgt = _ids(g, n, v)
        # a hidden row leans towards its target's row, as in a model that has learned something
        h = torch.randn(n, c, generator=g, device="cuda") + 1.5 * w[tgt.long()]
        trained = torch.rand((n + run_len - 1) // run_len, generator=g, device="cuda") < case["trained"]
        trained = trained.repeat_interleave(run_len)[:n]
        s["h"], s["w"] = h.bfloat16(), w.bfloat16()
        s["target"] = torch.where(trained, tgt, torch.full_like(tgt, -1))
        # weight of each position's loss: an advantage over the batch
        s["dloss"] = torch.randn(n, generator=g, device="cuda") / n
    return s


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    return {"embed": _embed, "embed_bwd": _embed_bwd, "norm": _norm, "norm_bwd": _norm_bwd, "loss": _loss,
            "loss_step": _loss_step}[case["op"]](state, case, torch.float32)


def _run_own(s):
    from prefix_tree_packed_dfs_gb300 import ops
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return ops.embed(s["table"], s["tokens"], scale=case["scale"])
    if op == "embed_bwd":
        return ops.embed_bwd(s["tokens"], s["dout"], case["v"], scale=case["scale"],
                             dtype=torch.float32 if case["table"] == "fp32" else torch.bfloat16)
    if op == "norm":
        return ops.block_norm(s["res"], s["w_pre"], y=s["y"], w_post=s["w_post"], gate=s["gate"], scale=case["scale"],
                              eps=EPS)
    if op == "norm_bwd":
        return [t for t in ops.block_norm_bwd(s["res"], s["w_pre"], s["dx"], dres_out=s["dres_out"], y=s["y"],
                                              w_post=s["w_post"], gate=s["gate"], scale=case["scale"], eps=EPS)
                if t is not None]
    loss, lse = ops.lm_loss(s["h"], s["w"], s["target"], scale=case["scale"])
    if op == "loss":
        return [loss, lse]
    dh, dw = ops.lm_loss_bwd(s["h"], s["w"], s["target"], lse, s["dloss"], scale=case["scale"])
    return [loss, lse, dh, dw]


# ---- plain forms: elementary operations in `t` (32 bits), rounded once at the end ----

def _table_type(case):
    return torch.float32 if case["table"] == "fp32" else torch.bfloat16


def _embed(s, case, t):
    tok = s["tokens"].long()
    rows = s["table"][tok.clamp(min=0)].to(t) * case["scale"]
    return torch.where((tok >= 0)[:, None], rows, torch.zeros((), dtype=t, device=rows.device)).bfloat16()


def _embed_bwd(s, case, t):
    tok = s["tokens"].long()
    v = case["v"]
    sums = torch.zeros(v + 1, case["c"], dtype=t, device=tok.device)   # row v takes the padding's
    sums.index_add_(0, torch.where(tok >= 0, tok, torch.full_like(tok, v)), s["dout"].to(t))
    return (sums[:v] * case["scale"]).to(_table_type(case))


def _norm(s, case, t):
    y = s["y"].to(t)
    if case["post"]:
        y = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["w_post"].to(t)
    if case["gate"]:
        y = y / (1.0 + torch.exp(-s["gate"].to(t)))
    r = s["res"].to(t) + case["scale"] * y
    x = r * torch.rsqrt((r * r).mean(1, keepdim=True) + EPS) * s["w_pre"].to(t)
    return [r.bfloat16(), x.bfloat16()]


def _norm_grad(x, rstd, w, d):
    """Gradients of x * rstd * w (rstd = 1/sqrt(mean x^2 + eps)) for the gradient d: (dx, dw)."""
    xn = x * rstd
    dw = (d * xn).sum(0)
    dn = d * w
    return rstd * (dn - xn * (dn * xn).mean(1, keepdim=True)), dw


def _norm_bwd(s, case, t):
    y, res, w_pre = s["y"].to(t), s["res"].to(t), s["w_pre"].to(t)
    u, sig = y, 1.0
    if case["post"]:
        w_post = s["w_post"].to(t)
        rstd_y = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        u = y * rstd_y * w_post
    if case["gate"]:
        sig = 1.0 / (1.0 + torch.exp(-s["gate"].to(t)))
    r = res + case["scale"] * (sig * u)
    dr, dw_pre = _norm_grad(r, torch.rsqrt((r * r).mean(1, keepdim=True) + EPS), w_pre, s["dx"].to(t))
    dr = dr + s["dres_out"].to(t)
    out = [dr.bfloat16(), None, None, None, dw_pre]     # dres, dy, dgate, dw_post, dw_pre
    dt = case["scale"] * dr
    if case["gate"]:
        out[2] = (dt * u * sig * (1.0 - sig)).bfloat16()
    dy = dt * sig
    if case["post"]:
        dy, out[3] = _norm_grad(y, rstd_y, w_post, dy)
    out[1] = dy.bfloat16()
    return [o for o in out if o is not None]


def _scores(s, case, t):
    tgt = s["target"].long()
    on = tgt >= 0
    logits = (s["h"].to(t) @ s["w"].to(t).T) * case["scale"]
    zero = torch.zeros((), dtype=t, device=tgt.device)
    top = logits.max(1, keepdim=True).values
    lse = (top + torch.exp(logits - top).sum(1, keepdim=True).log())[:, 0]
    at = logits.gather(1, tgt.clamp(min=0)[:, None])[:, 0]
    return logits, on, torch.where(on, lse - at, zero), torch.where(on, lse, zero)


def _loss(s, case, t):
    _, _, loss, lse = _scores(s, case, t)
    return [loss, lse]


def _loss_step(s, case, t):
    logits, on, loss, lse = _scores(s, case, t)
    tgt = s["target"].long()
    # d loss / d logits, weighted: weight * scale * (softmax - one at the target)
    d = torch.exp(logits - lse[:, None])
    d.scatter_add_(1, tgt.clamp(min=0)[:, None], torch.full((len(tgt), 1), -1.0, dtype=t, device=d.device))
    d = d * torch.where(on, s["dloss"].to(t) * case["scale"], torch.zeros((), dtype=t, device=d.device))[:, None]
    d = torch.where(on[:, None], d, torch.zeros((), dtype=t, device=d.device))
    return [loss, lse, (d @ s["w"].to(t)).bfloat16(), (d.T @ s["h"].to(t)).bfloat16()]


# ---- what a pass cannot do without ----

def work(case):
    n, c = case["n"], case["c"]
    if case["op"] == "embed":
        tab = 4 if case["table"] == "fp32" else 2
        # each distinct row once (at most the table), the ids, the output
        return {"bytes": min(n, case["v"]) * c * tab + 4 * n + 2 * n * c, "flops": n * c}
    if case["op"] == "embed_bwd":
        tab = 4 if case["table"] == "fp32" else 2
        return {"bytes": 2 * n * c + 4 * n + case["v"] * c * tab, "flops": n * c}
    if case["op"] == "norm":
        return {"bytes": 2 * n * c * (4 + case["gate"]) + 4 * c * (1 + case["post"]), "flops": 14 * n * c}
    if case["op"] == "norm_bwd":
        return {"bytes": 2 * n * c * (6 + 2 * case["gate"]) + 8 * c * (1 + case["post"]), "flops": 30 * n * c}
    v = case["v"]
    rows = max(1, int(n * case["trained"]))
    if case["op"] == "loss":
        return {"bytes": 2 * (rows + v) * c + 12 * n, "flops": 2 * rows * v * c}
    return {"bytes": 2 * (rows + v) * c + 16 * n + 2 * (n + v) * c, "flops": 6 * rows * v * c}


# ---- from the definitions, in 64 bits ----

def exact(case, seed):
    n, c = case["n"], case["c"]
    if case["op"].startswith("loss"):
        if (8.0 if case["op"] == "loss_step" else 2.0) * n * c * case["v"] > 8e12:
            return None
        return _exact_loss(case, prepare(case, seed))
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros(n, c, dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["tokens"] >= 0)[:, 0]
        out[at] = s["table"].double()[s["tokens"][at].long()] * case["scale"]
        return out
    if case["op"] == "embed_bwd":
        # the transpose of the lookup as sums over the ids in sorted order: differences of running sums
        tok, order = torch.sort(s["tokens"].long(), stable=True)
        run_sum = torch.zeros(n + 1, c, dtype=torch.float64, device="cuda")
        torch.cumsum(s["dout"].double()[order], 0, out=run_sum[1:])
        ids = torch.arange(case["v"], device="cuda")
        lo, hi = torch.searchsorted(tok, ids), torch.searchsorted(tok, ids, right=True)
        return (run_sum[hi] - run_sum[lo]) * case["scale"]
    # the norms by automatic differentiation of their definition
    names = [k for k in ("res", "y", "gate", "w_post", "w_pre") if s.get(k) is not None]
    leaf = {k: s[k].double().requires_grad_(case["op"] == "norm_bwd") for k in names}
    u = leaf["y"]
    if case["post"]:
        u = u / (u.square().mean(1, keepdim=True) + EPS).sqrt() * leaf["w_post"]
    if case["gate"]:
        u = u * torch.sigmoid(leaf["gate"])
    r = leaf["res"] + case["scale"] * u
    x = r / (r.square().mean(1, keepdim=True) + EPS).sqrt() * leaf["w_pre"]
    if case["op"] == "norm":
        return [r, x]
    total = (r * s["dres_out"].double()).sum() + (x * s["dx"].double()).sum()
    return list(torch.autograd.grad(total, [leaf[k] for k in names]))


def _exact_loss(case, s):
    on = torch.nonzero(s["target"] >= 0)[:, 0]
    n, c, v = case["n"], case["c"], case["v"]
    loss, lse = (torch.zeros(n, dtype=torch.float64, device="cuda") for _ in range(2))
    dh, dw = (torch.zeros(k, c, dtype=torch.float64, device="cuda") for k in (n, v))
    w, tgt = s["w"].double(), s["target"].long()
    for at in on.split(1024):
        h = s["h"][at].double()
        logp = torch.log_softmax(h @ w.T * case["scale"], 1)
        pick = torch.nn.functional.one_hot(tgt[at], v).double()
        loss[at] = -(logp * pick).sum(1)
        lse[at] = (h @ w.T * case["scale"])[:, 0] - logp[:, 0]
        if case["op"] == "loss_step":
            d = (logp.exp() - pick) * (s["dloss"][at].double() * case["scale"])[:, None]
            dh[at] = d @ w
            dw += d.T @ h
    return [loss, lse] if case["op"] == "loss" else [loss, lse, dh, dw]
