"""Next-token targets of packed positions against the raw sequences: every raw
token finds its own next token at its packed position (a branch's last common
token is packed once per branch), and the weighted loss of the packed positions
is the loss of the raw tokens."""
import numpy as np
import pytest

import workloads

BF = 2.0 ** -8


def _plan(w):
    from prefix_tree_packed_dfs_gb300 import ops
    return ops.Plan.from_sequences(w.sequences, group_ids=w.group_ids, row_capacity=w.row_capacity,
                                   min_shared=w.min_shared)


def _next(sequences):
    return np.concatenate([np.append(s[1:], -1) for s in sequences]).astype(np.int32)


@pytest.mark.parametrize("name", ["tiny", "tiny_fit", "grpo", "deep_small"])
def test_a_packed_position_has_one_next_token(lib, name):
    w = workloads.get(name)
    plan = _plan(w)
    nxt = _next(w.sequences)
    begin, raw = plan.raw_of_forwarded()
    assert plan.info["n_fwd"] < plan.info["n_raw"]              # something is shared
    packed = nxt[raw[begin[:-1]]]                               # the owner's, as gather_to_forwarded takes it
    assert np.array_equal(packed[plan.export()["token_index"]], nxt)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["tiny", "tiny_fit"])
def test_packed_loss_and_gradient_are_those_of_the_raw_tokens(lib, name):
    """fp64 over the raw tokens, each with its own next token, against the loss
    and gradients over the packed positions.  A loss is off by at most twice
    e = 128 * 2^-23 sum|h w| + 2^-14 + |lse| 2^-21 (a score's additions, the
    softmax sum, roundings).  Gradients: two bf16 roundings, b sqrt(2/3) in the
    2-norm."""
    import torch
    from prefix_tree_packed_dfs_gb300 import ops
    w = workloads.get(name)
    plan = _plan(w)
    dp = plan.to_device()
    F, R, V, C = plan.info["n_fwd"], plan.info["n_raw"], workloads.VOCAB, 128
    g = torch.Generator().manual_seed(1)
    h = torch.randn(F, C, generator=g).bfloat16().cuda()
    table = (torch.randn(V, C, generator=g) * 0.2).bfloat16().cuda()
    weight = torch.randn(1, R, generator=g).cuda()
    nxt = torch.from_numpy(_next(w.sequences)).cuda()
    target = ops.gather_to_forwarded(dp, nxt)
    _, dl = ops.sum_to_forwarded(dp, lse_src=weight)
    loss, lse = ops.lm_loss(h, table, target)
    dh, dw = ops.lm_loss_bwd(h, table, target, lse, dl[0])

    at, on = torch.from_numpy(plan.export()["token_index"]).long().cuda(), nxt >= 0
    hr = h.double()[at]                                          # the raw tokens' hidden rows
    logp = torch.log_softmax(hr @ table.double().T, 1)
    one = torch.nn.functional.one_hot(nxt.long().clamp(min=0), V).double()
    wr = torch.where(on, weight[0].double(), 0.0)
    e = 128 * 2.0 ** -23 * (hr.abs() @ table.double().abs().T).amax(1) + 2.0 ** -14 + lse.double()[at].abs() * 2.0 ** -21
    raw_loss = torch.where(on, -(logp * one).sum(1), 0.0)
    assert ((loss.double()[at] - raw_loss).abs() <= 2 * e * on).all()
    off = (loss.double() * dl[0].double()).sum() - (wr * raw_loss).sum()
    # the weights' fp32 sums: some 2^-20 of their magnitudes, for up to 16 of them
    assert abs(float(off)) <= float((wr.abs() * (2 * e + 2.0 ** -20 * raw_loss)).sum())
    dz = (logp.exp() - one) * wr[:, None]
    ref_h = torch.zeros(F, C, dtype=torch.float64, device="cuda").index_add_(0, at, dz @ table.double())
    ref_w = dz.T @ hr
    for a, b in ((dh, ref_h), (dw, ref_w)):
        assert float((a.double() - b).norm()) <= BF * (2 / 3) ** 0.5 * float(b.norm())
