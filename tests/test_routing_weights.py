"""Budgeted routing where a token keeps only experts of weight 0, in moe_route and in
moe_layer_few: the weights stay 0 (nothing is left to renormalise) and the token's y is
its shared expert's alone."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_05_amd as moe
import workloads as W
from oracle import moe as O
from tests import harness as Hn

INF = float("inf")


def _routing(low):
    """Logits [4, 8] and the budgeted routing that follows: tokens 1 to 3 share experts 1
    and 2, which outweigh token 0's only expert; token 0 fills its picks with the first
    experts of weight 0."""
    z = torch.full((4, 8), low)
    z[0, 0] = 0.0
    z[1:, 1:3] = 0.0
    ids = [[1, 2, -1, -1]] + [[1, 2, -1, -1]] * 3
    w = [[0, 0, 0, 0]] + [[0.5, 0.5, 0, 0]] * 3
    # Union {0, 1, 2, 3}; tokens 1 to 3 fill up with experts 0 and 3.
    return z, np.array(ids), np.array(w), [4, 2, 8, 0]


def test_oracle_keeps_weights_of_zero():
    z, ids, w, stats = _routing(-INF)
    i, v = O.topk_softmax(z.double().numpy(), 4)
    i, v, s = O.expert_budget(i, v, 2)
    assert np.array_equal(i, ids) and np.array_equal(v, w) and s.tolist() == stats


@pytest.mark.gpu
@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("S", [0, 128])
@pytest.mark.parametrize("low", [-INF, torch.finfo(torch.float32).min])
def test_budget_leaves_only_masked_experts(low, S, few):
    print(f"\n[case] masked budget low={low} S={S} few={few}", flush=True)
    shape = W.LayerShape("masked_budget", 256, 8, 128, 4, S, "bf16", "bf16", expert_budget=2)
    case = Hn.make_case(shape, 4, 101, condition=False)
    case.inp.w_router.zero_()                              # the logits are the bias
    case.inp.logit_bias, ids, w, stats = _routing(low)
    wg = case.inp.w_shared_gate
    layer = moe.MoELayer(Hn.config(shape), case.weights, case.inp.w_router.cuda(), None if wg is None else wg.cuda(),
                         case.shared, max_tokens=4, few=few, stats=True)
    layer.y.fill_(float("nan"))
    y = layer(case.inp.x.cuda(), case.inp.logit_bias.cuda())
    torch.cuda.synchronize()
    assert np.array_equal(layer.topk_ids.cpu().numpy(), ids)
    assert np.array_equal(layer.topk_weights.cpu().numpy(), w)     # 1 / 2 and 0 are exact
    assert layer.route_stats.tolist() == stats
    sg = None if wg is None else O.sigmoid(O.shared_gate_logit(case.inp.x, wg))
    shared = None if case.shared is None else case.shared_cpu()
    # The three calls keep h in bf16, the two-launch form in float32: each against the
    # oracle that does the same, with the bounds derived for those pairs (a bf16 h moves a
    # token by up to half a step, 2^-8 relative, so the exact one is no reference there).
    ref = O.moe_combine(case.inp.x, ids, w, sg, case.expert_cpu, shared, "bf16", None, ["model", "bf16_h"])
    got = y.cpu().double().numpy()
    if S == 0:
        assert (got[0] == 0).all()
    err = Hn.token_rel_l2(got, ref["model" if few else "bf16_h"])
    assert err.size == (4 if S else 3) and err.max() <= (2.0 ** -16 if few else Hn.TOKEN_TOL["bf16"])


@pytest.mark.gpu
@pytest.mark.parametrize("few", [False, True])
def test_weights_that_underflow_stay_zero(few):
    """exp(-200) is 0 in float32: a token whose larger picks are dropped keeps weight 0."""
    shape = W.LayerShape("underflow_budget", 256, 8, 128, 4, 0, "bf16", "bf16", expert_budget=2)
    case = Hn.make_case(shape, 4, 102, condition=False)
    case.inp.w_router.zero_()
    z, ids, w, stats = _routing(-200.0)
    layer = moe.MoELayer(Hn.config(shape), case.weights, case.inp.w_router.cuda(), max_tokens=4, few=few, stats=True)
    y = layer(case.inp.x.cuda(), z.cuda())
    torch.cuda.synchronize()
    assert np.array_equal(layer.topk_ids.cpu().numpy(), ids)
    assert np.array_equal(layer.topk_weights.cpu().numpy(), w)
    assert layer.route_stats.tolist() == stats and (y[0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("few", [False, True])
def test_a_token_without_any_logit_stays_nan_under_a_budget(few):
    shape = W.LayerShape("nan_budget", 256, 8, 128, 4, 0, "bf16", "bf16", expert_budget=2)
    case = Hn.make_case(shape, 4, 103, condition=False)
    case.inp.w_router.zero_()
    z, ids, w, _ = _routing(-INF)
    z[0] = -INF
    layer = moe.MoELayer(Hn.config(shape), case.weights, case.inp.w_router.cuda(), max_tokens=4, few=few)
    y = layer(case.inp.x.cuda(), z.cuda())
    torch.cuda.synchronize()
    assert np.array_equal(layer.topk_ids.cpu().numpy(), ids)
    assert torch.isnan(layer.topk_weights[0, :2]).all() and torch.isnan(y[0]).all()
    assert np.array_equal(layer.topk_weights[1:].cpu().numpy(), w[1:]) and torch.isfinite(y[1:]).all()
