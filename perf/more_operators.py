"""What the operators that complete a step on packed rows are measured on.

Between the token mixers, the norms and the vocabulary loss a step needs its
projections (``linear``), its feed-forward block (``gated_ffn``), rotary
positions of every layout (``rope_by_depth_ex``), and at its end the objective
that turns log-probabilities into the weights of the loss (``policy_loss``).
Each case below is one call, or one forward and backward, of one of them.
Sizes are those of the repository's own batches (2,048 = 16 heads of 128 and
4,096 = 32 heads of 128; 8 key/value heads; 32,768 and 96,888 forwarded
positions; 64 sequences over a 512-token system prompt and 1,024-token
prompts) and generic odd ones.
"""
import math

import numpy as np
import torch

own = False


def listed():
    return [
        # q, k and v of one sampled token in one product: a read of the weights
        {"name": "linear_token", "op": "linear", "n": 1, "c": 2048, "o": 4096, "act": "none", "bias": False,
         "res": False},
        # the projection after the mixer over a rollout batch, onto the residual stream
        {"name": "linear_batch", "op": "linear", "n": 96888, "c": 2048, "o": 2048, "act": "none", "bias": False,
         "res": True},
        # a small odd batch through a biased projection with an activation, and back
        {"name": "linear_step_odd", "op": "linear_step", "n": 1001, "c": 1000, "o": 552, "act": "gelu", "bias": True,
         "res": True},
        # fused q, k, v projection of a wide model on one 32k row, and back
        {"name": "linear_step_row", "op": "linear_step", "n": 32768, "c": 4096, "o": 6144, "act": "none", "bias": True,
         "res": False},
        # one sampled token through a feed-forward block
        {"name": "ffn_token", "op": "ffn", "n": 1, "c": 2048, "i": 8192, "act": "silu", "res": True},
        # the next tokens of a few dozen rollouts at once, wide model
        {"name": "ffn_rollouts", "op": "ffn", "n": 40, "c": 4096, "i": 12288, "act": "silu", "res": True},
        # a ragged row and odd widths, forward and backward
        {"name": "ffn_step_odd", "op": "ffn_step", "n": 1003, "c": 1000, "i": 2728, "act": "gelu_tanh", "res": True},
        # training the block on one 32k row
        {"name": "ffn_step_row", "op": "ffn_step", "n": 32768, "c": 2048, "i": 8192, "act": "silu", "res": True},
        # every position of a rollout batch, frequencies stretched for a long context, q and k taken out of the
        # fused projection
        {"name": "rope_batch", "op": "rope", "n": 96888, "hq": 16, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "base": 1e6, "stretch": 8.0, "factor": 1.2079441541679836, "far": 131072,
         "inverse": False},
        # interleaved pairs in a part of the head: the gradients of a short ragged row
        {"name": "rope_part", "op": "rope", "n": 5003, "hq": 16, "hkv": 8, "d": 64, "rot": 32, "interleaved": True,
         "base": 1e4, "stretch": 1.0, "factor": 1.0, "far": 8192, "inverse": True},
        # a rollout batch: clipped token ratios with a KL term, prompts shared and without loss
        {"name": "policy_batch", "op": "policy", "groups": 8, "rollouts": 8, "system": 512, "prompt": 1024,
         "least": 256, "most": 2048, "joint": 0.0, "level": "token", "lo": 0.2, "hi": 0.28, "dual": 0.0, "kl": 0.04},
        # many short rollouts in pairs with a first turn in common, ratios of whole sequences
        {"name": "policy_sequences", "op": "policy", "groups": 32, "rollouts": 16, "system": 100, "prompt": 211,
         "least": 20, "most": 1500, "joint": 0.3, "level": "sequence", "lo": 0.02, "hi": 0.03, "dual": 3.0,
         "kl": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_step", "ffn", "ffn", "ffn_step", "rope", "policy"])
    act = rng.choice(["none", "silu", "gelu", "gelu_tanh"])
    if op.startswith("linear"):
        c, o = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 768)
        most = int(4.9e12 / (6.0 * c * o))
        return {"op": op, "n": _log(rng, 1, min(96888, most)), "c": c, "o": o, "act": act,
                "bias": rng.random() < 0.5, "res": rng.random() < 0.5}
    if op.startswith("ffn"):
        c, i = 8 * _log(rng, 8, 512), 8 * _log(rng, 8, 1536)
        most = int(9.8e12 / (18.0 * c * i))
        return {"op": op, "n": _log(rng, 1, min(32768, most)), "c": c, "i": i,
                "act": rng.choice(["silu", "gelu", "gelu_tanh"]), "res": rng.random() < 0.5}
    if op == "rope":
        d = rng.choice([64, 96, 128, 256])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4])
        return {"op": op, "n": _log(rng, 1, 96888 * 24 * 128 // (max(24, hq + hkv) * max(128, d))), "hq": hq,
                "hkv": hkv, "d": d, "rot": rng.choice([16, 32, d // 2, d]), "interleaved": rng.random() < 0.5,
                "base": rng.choice([1e4, 1e6]), "stretch": rng.choice([1.0, 4.0, 32.0]),
                "factor": rng.choice([1.0, 1.25]), "far": _log(rng, 100, 1000000), "inverse": rng.random() < 0.4}
    least = _log(rng, 1, 500)
    return {"op": op, "groups": _log(rng, 1, 32), "rollouts": _log(rng, 1, 16), "system": _log(rng, 1, 600),
            "prompt": _log(rng, 1, 1000), "least": least, "most": least + _log(rng, 1, 1500),
            "joint": rng.choice([0.0, 0.3, 1.0]), "level": rng.choice(["token", "sequence"]),
            "lo": rng.choice([0.2, 0.1, 0.003]), "hi": rng.choice([0.2, 0.28, 0.004]),
            "dual": rng.choice([0.0, 0.0, 3.0]), "kl": rng.choice([0.0, 0.04, 0.001])}


def _freqs(case):
    """Angle per position of each pair: slow pairs stretched by the context's growth, fast ones kept, a ramp between."""
    rot = case["rot"]
    f = case["base"] ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if case["stretch"] != 1.0:
        turns = 8192.0 * f / (2.0 * math.pi)              # turns over the context that the model was trained on
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = f * (keep + (1.0 - keep) / case["stretch"])
    return f


def _rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).bfloat16()


def _packed(case):
    """(token_index, fwd_raw_begin, fwd_raw, seq_offsets, own part's start in each sequence) of the case's tree:
    a system prompt under all, a prompt per group, and for some pairs of rollouts a first part in common."""
    rs = np.random.default_rng([case[k] for k in ("groups", "rollouts", "system", "prompt", "least", "most")])
    at, index, starts, offsets = 0, [], [], [0]

    def fresh(n):
        nonlocal at
        at += n
        return np.arange(at - n, at, dtype=np.int32)

    system = fresh(case["system"])
    for _ in range(case["groups"]):
        prompt = fresh(case["prompt"])
        common = None
        for k in range(case["rollouts"]):
            n = int(rs.integers(case["least"], case["most"] + 1))
            if k % 2 == 0:
                common = fresh(case["least"] // 2) if rs.random() < case["joint"] else None
            head = [system, prompt] + ([] if common is None else [common])
            index += head + [fresh(n - (0 if common is None else len(common)))]
            offsets.append(offsets[-1] + case["system"] + case["prompt"] + n)
            starts.append(offsets[-2] + case["system"] + case["prompt"])
    index = np.concatenate(index)
    begin = np.zeros(at + 1, dtype=np.int32)
    begin[1:] = np.cumsum(np.bincount(index, minlength=at))
    raw = np.argsort(index, kind="stable").astype(np.int32)
    return index, begin, raw, np.asarray(offsets, dtype=np.int32), np.asarray(starts)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    op = case["op"]
    if op.startswith("linear"):
        n, c, o = case["n"], case["c"], case["o"]
        s["x"], s["w"] = _rand(g, n, c), _rand(g, o, c, std=1.0 / math.sqrt(c))
        s["bias"] = 0.3 * torch.randn(o, generator=g, device="cuda") if case["bias"] else None
        s["res"] = _rand(g, n, o, std=2.0) if case["res"] else None
        if op == "linear_step":
            s["dy"] = _rand(g, n, o, std=1.0 / n)
    elif op.startswith("ffn"):
        n, c, i = case["n"], case["c"], case["i"]
        s["x"], s["w_in"] = _rand(g, n, c), _rand(g, 2 * i, c, std=1.0 / math.sqrt(c))
        s["w_out"] = _rand(g, c, i, std=1.0 / math.sqrt(i))
        s["res"] = _rand(g, n, c, std=2.0) if case["res"] else None
        if op == "ffn_step":
            s["dy"] = _rand(g, n, c, std=1.0 / n)
    elif op == "rope":
        n, hq, hkv, d = case["n"], case["hq"], case["hkv"], case["d"]
        qkv = _rand(g, n, (hq + 2 * hkv) * d)      # the fused projection's output
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["depth"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda", dtype=torch.int32)
        s["freqs"] = _freqs(case)
    else:
        index, begin, raw, offsets, starts = _packed(case)
        r, f = len(index), len(begin) - 1
        for k, v in (("index", index), ("begin", begin), ("raw", raw), ("offsets", offsets)):
            s[k] = torch.from_numpy(v).cuda()
        s["loss"] = 0.05 - 2.0 * torch.log(torch.rand(f, generator=g, device="cuda").clamp_(min=1e-4))
        logp = -s["loss"][s["index"].long()]
        # the policy that sampled is some steps older, the reference is further away
        s["old"] = logp + 0.15 * torch.randn(r, generator=g, device="cuda")
        s["ref"] = logp + 0.4 * torch.randn(r, generator=g, device="cuda") if case["kl"] else None
        # one advantage per sequence, weights: a mean over each completion's tokens, then over the sequences
        seq = torch.repeat_interleave(torch.arange(len(starts), device="cuda"),
                                      (s["offsets"][1:] - s["offsets"][:-1]).long())
        adv = torch.randn(len(starts), generator=g, device="cuda")
        s["adv"] = adv[seq].contiguous()
        mine = torch.arange(r, device="cuda") >= torch.from_numpy(starts).cuda()[seq]
        left = (s["offsets"][1:].long() - torch.from_numpy(starts).cuda())[seq]
        s["weight"] = torch.where(mine, 1.0 / (left * len(starts)).float(), torch.zeros((), device="cuda"))
        # tokens that carry no loss hold no numbers either
        for k in ("old", "ref"):
            if s[k] is not None:
                s[k] = torch.where(mine, s[k], torch.full_like(s[k], float("nan")))
    return s


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    return {"linear": _linear, "linear_step": _linear, "ffn": _ffn, "ffn_step": _ffn, "rope": _rope,
            "policy": _policy}[case["op"]](state, case)


def _run_own(s):
    from prefix_tree_packed_dfs_gb300 import ops
    case = s["case"]
    op = case["op"]
    if op == "linear":
        return ops.linear(s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["res"])
    if op == "linear_step":
        y = ops.linear(s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["res"])
        dx, dw, db = ops.linear_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], act=case["act"])
        return [t for t in (y, dx, dw, db) if t is not None]
    if op == "ffn":
        return ops.gated_ffn(s["x"], s["w_in"], s["w_out"], act=case["act"], residual=s["res"])
    if op == "ffn_step":
        y, pre, a = ops.gated_ffn(s["x"], s["w_in"], s["w_out"], act=case["act"], residual=s["res"], save=True)
        return [y, *ops.gated_ffn_bwd(s["x"], s["w_in"], s["w_out"], s["dy"], pre, a, act=case["act"])]
    if op == "rope":
        return list(ops.rope_by_depth_ex(s["q"], s["k"], s["depth"], s["freqs"], interleaved=case["interleaved"],
                                         factor=case["factor"], inverse=case["inverse"]))
    return list(ops.policy_loss(s["loss"], s["old"], s["adv"], s["weight"], s["index"], s["begin"], s["raw"],
                                ref_logp=s["ref"], clip_low=case["lo"], clip_high=case["hi"], dual_clip=case["dual"],
                                kl_coef=case["kl"], seq_offsets=s["offsets"] if case["level"] == "sequence" else None))


# ---- plain forms: elementary operations in 32 bits, rounded once at the end ----

def _act(z, name):
    """(act(z), its derivative)."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "gelu":
        half = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * half, half + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    k = 2.0 * math.sqrt(2.0 / math.pi)                      # 0.5 (1 + tanh(t)) = sigmoid(2 t)
    s = 1.0 / (1.0 + torch.exp(-k * (z + 0.044715 * z * z * z)))
    return z * s, s + z * s * (1.0 - s) * k * (1.0 + 3.0 * 0.044715 * z * z)


def _linear(s, case):
    x, w = s["x"].float(), s["w"].float()
    z = x @ w.T
    if case["bias"]:
        z = z + s["bias"]
    y, slope = _act(z, case["act"])
    if case["res"]:
        y = y + s["res"].float()
    if case["op"] == "linear":
        return y.bfloat16()
    dz = s["dy"].float() * slope
    out = [y.bfloat16(), (dz @ w).bfloat16(), (dz.T @ x).bfloat16()]
    return out + [dz.sum(0)] if case["bias"] else out


def _ffn(s, case):
    x, w_in, w_out = s["x"].float(), s["w_in"].float(), s["w_out"].float()
    gu = x @ w_in.T
    g, u = gu[:, :case["i"]], gu[:, case["i"]:]
    a, slope = _act(g, case["act"])
    h = a * u
    y = h @ w_out.T
    if case["res"]:
        y = y + s["res"].float()
    if case["op"] == "ffn":
        return y.bfloat16()
    dy = s["dy"].float()
    dh = dy @ w_out
    dgu = torch.cat([dh * u * slope, dh * a], 1)
    return [y.bfloat16(), (dgu @ w_in).bfloat16(), (dgu.T @ x).bfloat16(), (dy.T @ h).bfloat16()]


def _rope(s, case):
    rot = case["rot"]
    angle = s["depth"].double()[:, None] * torch.from_numpy(s["freqs"]).cuda()
    cos = (torch.cos(angle) * case["factor"]).float()[:, None]
    sin = (torch.sin(angle) * (-case["factor"] if case["inverse"] else case["factor"])).float()[:, None]
    out = []
    for t in (s["q"], s["k"]):
        y = t.float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if case["interleaved"] else (y[..., :rot // 2], y[..., rot // 2:rot])
        p, q = a * cos - b * sin, a * sin + b * cos
        turned = torch.stack([p, q], 3).flatten(2) if case["interleaved"] else torch.cat([p, q], 2)
        out.append(torch.cat([turned, y[..., rot:]], 2).bfloat16())
    return out


def _policy(s, case):
    w, adv, index = s["weight"], s["adv"], s["index"].long()
    on = w != 0
    zero = torch.zeros((), device=w.device)
    logp = -s["loss"][index]
    # borders of the clip: the difference of two 32-bit numbers and its comparison in 64 bits
    d = torch.where(on, logp.double() - s["old"].double(), torch.zeros((), dtype=torch.float64, device=w.device))
    if case["level"] == "sequence":
        off = s["offsets"].long()
        total = torch.zeros(len(d) + 1, dtype=torch.float64, device=w.device)
        many = torch.zeros(len(d) + 1, dtype=torch.float64, device=w.device)
        total[1:], many[1:] = torch.cumsum(d, 0), torch.cumsum(on.double(), 0)
        count = (many[off[1:]] - many[off[:-1]]).clamp(min=1.0)
        mean = (total[off[1:]] - total[off[:-1]]) / count
        seq = torch.searchsorted(off, torch.arange(len(d), device=w.device), right=True) - 1
        d = torch.where(on, mean[seq], torch.zeros_like(d))
    lo, hi = math.log1p(-case["lo"]), math.log1p(case["hi"])
    ratio = torch.exp(d).float()
    pos = adv >= 0
    held = torch.where(pos, d > hi, d < lo)
    used = torch.exp(torch.where(pos, d.clamp(max=hi), d.clamp(min=lo)))
    if case["dual"]:
        held = held | (~pos & (d > math.log(case["dual"])))
        used = torch.where(pos, used, used.clamp(max=case["dual"]))
    grad = torch.where(held, zero, adv * ratio)
    if case["level"] == "sequence":
        # every token moves its sequence's ratio by a share
        run_sum = torch.zeros(len(d) + 1, dtype=torch.float64, device=w.device)
        run_sum[1:] = torch.cumsum(torch.where(on, w * grad, zero).double(), 0)
        share = ((run_sum[off[1:]] - run_sum[off[:-1]]) / count).float()
        grad = torch.where(on, share[seq], zero)
    else:
        grad = torch.where(on, w * grad, zero)
    objective = torch.where(on, -adv * used.float(), zero)
    kl = torch.zeros_like(w)
    if case["kl"]:
        t = torch.where(on, s["ref"].double() - logp.double(), torch.zeros_like(d))
        kl = (torch.expm1(t) - t).float()
        objective = objective + case["kl"] * kl
        grad = grad + torch.where(on, w * case["kl"] * torch.expm1(t).float(), zero)
    stats = [(torch.where(on, w, zero).double() * v.double()).sum()
             for v in (objective, kl, (held & on).float(), ratio, torch.ones_like(w))]
    dloss = torch.zeros(len(s["begin"]) - 1, dtype=torch.float64, device=w.device)
    dloss.index_add_(0, index, grad.double())
    return [torch.stack(stats).float(), dloss.float()]


# ---- what a pass cannot do without ----

def work(case):
    op = case["op"]
    if op.startswith("linear"):
        n, c, o = case["n"], case["c"], case["o"]
        moved = 2 * (n * c + o * c + n * o * (1 + case["res"])) + 4 * o * case["bias"]
        if op == "linear":
            return {"bytes": moved, "flops": 2 * n * c * o}
        return {"bytes": moved + 2 * (n * o + n * c + o * c) + 4 * o * case["bias"], "flops": 6 * n * c * o}
    if op.startswith("ffn"):
        n, c, i = case["n"], case["c"], case["i"]
        moved = 2 * (n * c * (2 + case["res"]) + 3 * c * i)
        if op == "ffn":
            return {"bytes": moved, "flops": 6 * n * c * i}
        return {"bytes": moved + 2 * (2 * n * c + 3 * c * i), "flops": 18 * n * c * i}
    if op == "rope":
        elems = case["n"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": 4 * elems + 4 * case["n"], "flops": 3 * elems}
    mean = (case["least"] + case["most"]) // 2
    seqs = case["groups"] * case["rollouts"]
    raw = seqs * (case["system"] + case["prompt"] + mean)
    forwarded = case["system"] + case["groups"] * case["prompt"] + seqs * mean
    # index, order, weight of every token; old, reference and advantage of those that carry a loss; loss and its
    # gradient of every position
    return {"bytes": 12 * raw + seqs * mean * (8 + 4 * (case["kl"] != 0)) + 12 * forwarded, "flops": 20 * seqs * mean}


# ---- from the definitions, in 64 bits ----

def exact(case, seed):
    op = case["op"]
    if op.startswith(("linear", "ffn")):
        if work(case)["flops"] > 1.1e13:
            return None
        return _exact_products(case, prepare(case, seed))
    s = prepare(case, seed)
    if op == "rope":
        # as products of complex numbers
        rot = case["rot"]
        angle = s["depth"].double()[:, None] * torch.tensor(s["freqs"], device="cuda")
        turn = torch.polar(torch.full_like(angle, case["factor"]), -angle if case["inverse"] else angle)[:, None]
        out = []
        for t in (s["q"], s["k"]):
            y = t.double().clone()
            if case["interleaved"]:
                y[..., :rot] = torch.view_as_real(torch.view_as_complex(
                    y[..., :rot].unflatten(2, (rot // 2, 2)).contiguous()) * turn).flatten(2)
            else:
                z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
                y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
            out.append(y)
        return out
    return _exact_policy(case, s)


def _exact_products(case, s):
    fn = {"none": lambda z: z, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
          "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}[case["act"]]
    step = case["op"].endswith("step")
    names = [k for k in ("x", "w", "bias", "w_in", "w_out") if s.get(k) is not None]
    leaf = {k: s[k].double().requires_grad_(step) for k in names}
    if "w" in leaf:
        z = torch.nn.functional.linear(leaf["x"], leaf["w"], leaf.get("bias"))
        y = fn(z)
        wanted = [leaf[k] for k in ("x", "w", "bias") if k in leaf]
    else:
        gu = torch.nn.functional.linear(leaf["x"], leaf["w_in"])
        gate, up = gu.chunk(2, 1)
        y = torch.nn.functional.linear(fn(gate) * up, leaf["w_out"])
        wanted = [leaf[k] for k in ("x", "w_in", "w_out")]
    if s["res"] is not None:
        y = y + s["res"].double()
    if not step:
        return y
    return [y.detach(), *torch.autograd.grad(y, wanted, s["dy"].double())]


def _exact_policy(case, s):
    # by automatic differentiation of the objective, from the smaller of the two products
    on = torch.nonzero(s["weight"])[:, 0]
    loss = s["loss"].double().requires_grad_()
    w, adv = s["weight"][on].double(), s["adv"][on].double()
    logp = -loss[s["index"][on].long()]
    d = logp - s["old"][on].double()
    if case["level"] == "sequence":
        seqs = len(s["offsets"]) - 1
        seq = torch.bucketize(on, s["offsets"][1:].long(), right=True)
        count = torch.bincount(seq, minlength=seqs).double()
        d = (torch.zeros(seqs, dtype=torch.float64, device="cuda").index_add(0, seq, d) / count.clamp(min=1.0))[seq]
    ratio = torch.exp(d)
    bounded = torch.clamp(ratio, 1.0 - case["lo"], 1.0 + case["hi"])
    surrogate = torch.minimum(ratio * adv, bounded * adv)
    held = ratio.detach() * adv > bounded.detach() * adv
    if case["dual"]:
        floor = case["dual"] * adv
        held = held | ((adv < 0) & (surrogate.detach() < floor))
        surrogate = torch.where(adv < 0, torch.maximum(surrogate, floor), surrogate)
    kl = torch.zeros_like(w)
    if case["kl"]:
        t = s["ref"][on].double() - logp
        kl = torch.special.expm1(t) - t
    objective = (w * (case["kl"] * kl - surrogate)).sum()
    grad, = torch.autograd.grad(objective, loss)
    stats = torch.stack([objective.detach(), (w * kl.detach()).sum(), (w * held).sum(), (w * ratio.detach()).sum(),
                         w.sum()])
    return [stats, grad]
