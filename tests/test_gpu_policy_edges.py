"""The policy objective where its numbers end: infinite log-probabilities, ratios
past fp32's range, long sums.

The reference is the objective's formula in fp64, with s by the advantage's sign
(A > 0: A min(ratio, 1 + clip_high); A < 0: A max(ratio, 1 - clip_low), at most
the dual clip; A = 0: 0), so that infinities go through it.  Finite results:
2^-19 of the terms' magnitudes, as in test_gpu_layer.py.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

INF, LARGEST = np.inf, float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available()
    from prefix_tree_packed_dfs_gb300 import ops as o
    return o


def _formula(loss, old, adv, weight, index, offsets, ref, lo, hi, dual, kl_coef):
    """(stats, dloss, magnitudes of the terms of both)."""
    stats, smag, grad, mag = np.zeros(5), np.zeros(5), np.zeros(len(loss)), np.zeros(len(loss))
    bounds = [(r, r + 1) for r in range(len(old))] if offsets is None else list(zip(offsets[:-1], offsets[1:]))
    with np.errstate(all="ignore"):
        for b, e in bounds:
            on = [r for r in range(b, e) if weight[r] != 0]
            if not on:
                continue
            ratio = np.exp(np.mean([-loss[index[r]] - old[r] for r in on]))
            pull, pull_mag = 0.0, 0.0
            for r in on:
                A, w = adv[r], weight[r]
                if A > 0:
                    used, held = min(ratio, 1 + hi), ratio > 1 + hi
                else:
                    used, held = max(ratio, 1 - lo), ratio < 1 - lo
                    if dual and used > dual:
                        used, held = dual, True
                held = held and A != 0
                s, g = (0.0, 0.0) if A == 0 else (A * used, 0.0 if held else A * ratio)
                t = 0.0 if ref is None else ref[r] + loss[index[r]]
                kl = INF if np.isinf(t) else np.expm1(t) - t
                k = kl_coef * kl if kl_coef else 0.0
                terms = np.array([k - s, kl, float(held), ratio, 1.0])
                stats += w * terms
                smag += w * np.abs([k + abs(s), kl, float(held), ratio, 1.0])
                pull, pull_mag = pull + w * g, pull_mag + abs(w * g)
                if kl_coef and ref is not None:
                    grad[index[r]] += w * kl_coef * np.expm1(t)
                    mag[index[r]] += w * kl_coef * (np.exp(t) + 1)
            for r in on:
                grad[index[r]] += pull / len(on)
                mag[index[r]] += pull_mag / len(on)
    return stats, grad, smag, mag


def _matches(got, want, mag, what, rel=2.0 ** -19):
    got = got.double().cpu().numpy()
    want = np.where(np.abs(want) > LARGEST, np.copysign(INF, want), want)
    ends = ~np.isfinite(want)
    assert np.array_equal(got[ends], want[ends], equal_nan=True), (what, got, want)
    assert (np.abs(got[~ends] - want[~ends]) <= rel * mag[~ends] + 1e-30).all(), (what, got, want)


def _batch(level):
    """Two positions under three sequences of five own tokens each, the second sequence's third token for the tests."""
    index = np.concatenate([np.concatenate([[0, 1], np.arange(5) + 2 + 5 * k]) for k in range(3)]).astype(np.int32)
    g = np.random.default_rng(3)
    s = dict(loss=(0.1 + 2 * g.random(17)), index=index, at=7 + 4)
    s["old"] = -s["loss"][index] + 0.2 * g.normal(size=21)
    s["ref"] = -s["loss"][index] + 0.3 * g.normal(size=21)
    s["adv"], s["weight"] = 0.5 + g.random(21), 0.1 + g.random(21)
    s["offsets"] = np.arange(0, 22, 7, dtype=np.int32) if level == "sequence" else None
    return {k: v.astype(np.float32).astype(np.float64) if isinstance(v, np.ndarray) and v.dtype == np.float64 else v
            for k, v in s.items()}


def _run(ops, s, **kw):
    index = s["index"]
    begin = np.zeros(len(s["loss"]) + 1, np.int32)
    begin[1:] = np.cumsum(np.bincount(index, minlength=len(s["loss"])))
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    f = lambda a: t(np.asarray(a).astype(np.float32))
    return ops.policy_loss(f(s["loss"]), f(s["old"]), f(s["adv"]), f(s["weight"]), t(index), t(begin),
                           t(np.argsort(index, kind="stable").astype(np.int32)),
                           ref_logp=None if s["ref"] is None else f(s["ref"]),
                           seq_offsets=None if s["offsets"] is None else t(s["offsets"]), **kw)


def _check(ops, s, lo=0.2, hi=0.28, dual=0.0, kl=0.0):
    want = _formula(s["loss"], s["old"], s["adv"], s["weight"], s["index"], s["offsets"], s["ref"], lo, hi, dual, kl)
    stats, dloss = _run(ops, s, clip_low=lo, clip_high=hi, dual_clip=dual, kl_coef=kl)
    _matches(stats, want[0], want[2], "stats")
    _matches(dloss, want[1], want[3], "dloss")
    return dloss


@pytest.mark.parametrize("level", ["token", "sequence"])
@pytest.mark.parametrize("dual", [0.0, 3.0])
@pytest.mark.parametrize("which,value,kl,ref", [
    (which, value, kl, ref) for kl, ref in ((0.0, False), (0.0, True), (0.05, True))
    for which, value in (("old", -INF), ("old", INF), ("loss", INF)) + ((("ref", -INF), ("ref", INF)) if ref else ())])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_log_probabilities(ops, level, dual, kl, ref, which, value, sign):
    s = _batch(level)
    if not ref:
        s["ref"] = None
    s["adv"] = s["adv"] * sign
    plain = _check(ops, s, dual=dual, kl=kl)
    at = s["at"]
    s[which][s["index"][at] if which == "loss" else at] = value
    got = _check(ops, s, dual=dual, kl=kl)
    # what does not share the token's position or its sequence's ratio stays as it was
    lo, hi = (7, 14) if level == "sequence" else (at, at + 1)
    apart = np.ones(len(s["loss"]), bool)
    apart[s["index"][lo:hi]] = False
    assert torch.equal(got[torch.from_numpy(apart)], plain[torch.from_numpy(apart)])


@pytest.mark.parametrize("level", ["token", "sequence"])
@pytest.mark.parametrize("border", [dict(lo=1.0), dict(hi=INF), dict(lo=1.0, hi=INF), dict(dual=INF)])
@pytest.mark.parametrize("value", [-INF, INF])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_log_probabilities_at_borders_without_end(ops, level, border, value, sign):
    s = _batch(level)
    s["adv"] = s["adv"] * sign
    s["old"][s["at"]] = value
    _check(ops, s, kl=0.05, **border)


@pytest.mark.parametrize("level", ["token", "sequence"])
@pytest.mark.parametrize("value", [-INF, INF])
def test_an_infinite_log_probability_among_others_that_cancel_it_not(ops, level, value):
    """Two of a kind in a sequence, and advantages of both signs."""
    s = _batch(level)
    s["adv"][::2] *= -1
    s["old"][s["at"]] = s["old"][s["at"] + 1] = value
    _check(ops, s, dual=3.0)


@pytest.mark.parametrize("level", ["token", "sequence"])
@pytest.mark.parametrize("gap", [100.0, 1e30, INF])
@pytest.mark.parametrize("dual", [0.0, 3.0])
def test_no_advantage_beside_a_ratio_past_the_range(ops, level, gap, dual):
    """A group of equal rewards has advantages of 0: they add nothing, at a ratio that fp32 cannot hold too."""
    s = _batch(level)
    s["adv"][7:14] = 0.0
    s["old"][7:14] = np.float32(-gap)
    dloss = _check(ops, s, dual=dual)
    assert not dloss[torch.from_numpy(s["index"][9:14]).long().cuda()].any()
    s["adv"][8] = 0.5            # held at the border beside them
    _check(ops, s, dual=dual)


def test_ends_of_lists_that_lie_outside_the_batch(ops):
    """An end below 0 or above R counts as 0 or R, one below its list's start as that start; other positions are as they were."""
    index = np.repeat(np.arange(40), np.where(np.arange(40) % 5 == 0, 60, 3)).astype(np.int32)
    g = np.random.default_rng(4)
    R, F = len(index), 40
    begin = np.zeros(F + 1, np.int32)
    begin[1:] = np.cumsum(np.bincount(index))
    raw = np.arange(R, dtype=np.int32)
    t = lambda a: torch.from_numpy(a).cuda()
    f = lambda *s: g.normal(size=s).astype(np.float32)
    loss, adv, weight = np.abs(f(F)), f(R), np.abs(f(R))
    old = -loss[index] + 0.1 * f(R)
    run = lambda b: ops.policy_loss(t(loss), t(old), t(adv), t(weight), t(index), t(b), t(raw))[1].cpu().numpy()
    want = run(begin)
    share = lambda lo, hi: float(ops.policy_loss(t(loss), t(old), t(adv), t(weight), t(index),
                                                 t(np.array([lo] + [hi] * F, np.int32)), t(raw))[1][0])
    for at, value in ((0, -2 ** 31), (0, -1), (F, R + 1), (F, 2 ** 31 - 1), (17, 2 ** 31 - 1), (17, -2 ** 31), (20, -5)):
        b = begin.copy()
        b[at] = value
        got = run(b)
        touched = [k for k in (at - 1, at) if 0 <= k < F]
        rest = np.setdiff1d(np.arange(F), touched)
        assert np.array_equal(got[rest], want[rest])
        for k in touched:
            lo = min(max(int(b[k]), 0), R)
            hi = min(max(int(b[k + 1]), lo), R)
            assert abs(got[k] - share(lo, hi)) <= 2.0 ** -19 * np.abs(adv * weight).sum() * 2


@pytest.mark.parametrize("level", ["token", "sequence"])
@pytest.mark.parametrize("lengths", [(2000003,), (3, 1000000, 1, 999999), (8000000,)])
def test_statistics_of_many_tokens(ops, level, lengths):
    """Sums of thousands of terms per thread.  The sums of weights and of clipped tokens: up to six of a thread's
    terms at a time in fp32, 6 roundings, and these sums in pairs; a warp's 5, and one each for the pair and the result:
    13 x 2^-24 of the magnitudes.
    The others have the exponential's 2^-19 besides (here |d| < 2)."""
    R = sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(R)
    rnd = lambda: torch.rand(R, generator=g, device="cuda")
    index = torch.arange(R, dtype=torch.int32, device="cuda")
    begin = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    loss, weight = 0.1 + rnd(), torch.full((R,), 0.1, device="cuda")
    old, ref, adv = -loss + 0.8 * (rnd() - 0.4), -loss + rnd() - 0.5, 0.5 + rnd()
    stats, dloss = ops.policy_loss(loss, old, adv, weight, index, begin, index, ref_logp=ref, kl_coef=0.1,
                                   seq_offsets=off if level == "sequence" else None)
    d, t, w, A = -loss.double() - old.double(), ref.double() + loss.double(), weight.double(), adv.double()
    n = torch.tensor(lengths, device="cuda")
    if level == "sequence":
        seq = torch.repeat_interleave(torch.arange(len(lengths), device="cuda"), n)
        d = (torch.zeros(len(lengths), dtype=torch.float64, device="cuda").index_add_(0, seq, d) / n)[seq]
    ratio, kl = torch.exp(d), torch.expm1(t) - t
    terms = torch.stack([w * (0.1 * kl - A * ratio.clamp(max=1.2)), w * kl, w * (ratio > 1.2), w * ratio, w])
    mag = terms.abs().sum(1)
    mag[0] = (w * (0.1 * kl + A * ratio.clamp(max=1.2))).sum()
    rel = torch.tensor([2.0 ** -19] * 2 + [13 * 2.0 ** -24, 2.0 ** -19, 13 * 2.0 ** -24], dtype=torch.float64, device="cuda")
    off_by = (stats.double() - terms.sum(1)).abs() / mag.clamp(min=1e-30)
    assert (off_by <= rel).all(), off_by


@pytest.mark.parametrize("cut", [None, 1.0, 0.75])
def test_statistics_of_hundreds_of_millions_of_tokens(ops, cut):
    """Millions of terms per thread, all alike, so that their roundings do not cancel: 13 x 2^-24 as above (the ratio is
    exactly 1, and nothing else is rounded).  Token by token, as one sequence, and as two."""
    R = 600000000
    index = torch.arange(R + 1, dtype=torch.int32, device="cuda")
    full = lambda v: torch.full((R,), v, device="cuda")
    offsets = None if cut is None else torch.tensor([0, int(R * cut), R], dtype=torch.int32, device="cuda")
    w = np.float32(1e-3)
    stats, dloss = ops.policy_loss(full(0.5), full(-0.5), full(1.0), full(float(w)), index[:R], index, index[:R],
                                   seq_offsets=offsets)
    want = float(w) * R * np.array([-1.0, 0.0, 0.0, 1.0, 1.0])
    off = np.abs(stats.double().cpu().numpy() - want)
    assert (off <= 13 * 2.0 ** -24 * np.abs(want)).all(), off / want[-1]
    assert torch.equal(dloss[::1000003], full(float(w))[::1000003])
