"""moe_layer_few and moe_linear at the ends of their size ranges: no rows, the longest rows
and contractions, the most rows; and one token's NaN beside others.

Tolerance of the layer, relative L2 of a token's y.  A sum of L random terms runs as four
chains of L / 4, at most one rounding a term.  A chain's partial sums grow as a random
walk, so its roundings, each uniform within 2^-24 of the partial sum, add up to
2^-24 sqrt(n / 6) of the sum's standard deviation, n = L / 4 (rms: the mean square of
the partial sums is half the last one's, a uniform error's a third of its bound's); the
four chains' errors add as their sums do.  h is a product of two such sums, sqrt(2) of
that and a little for silu's slope: 1.5.  Three standard deviations, and a token whose few
h are a third of the usual size: 1.5 * 3 * 3 < 16.
Products: at most K + 1 roundings of 2^-24 on a term."""
import math

import numpy as np
import pytest
import torch

import mixture_experts_layer_05_amd as moe
import workloads as W
from oracle import moe as O
from tests import harness as Hn

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _y_tol(s):
    n = max(s.hidden_size, s.moe_intermediate_size, s.shared_expert_intermediate_size) / 4
    return 16 * 2.0 ** -24 * math.sqrt(n / 6)


def _layer(case):
    wg = case.inp.w_shared_gate
    return moe.MoELayer(Hn.config(case.shape), case.weights, case.inp.w_router.cuda(), None if wg is None else wg.cuda(),
                        case.shared, max_tokens=case.T, few=True)


def _oracle(case):
    s = case.shape
    r = O.route(case.inp.x, case.inp.w_router, case.inp.w_shared_gate, case.inp.logit_bias, s.num_experts_per_tok)
    r["y"] = O.moe_combine(case.inp.x, r["ids"], r["w"], r["shared_gate"], case.expert_cpu, case.shared_cpu(),
                           s.weight_dtype)
    return r


@pytest.mark.parametrize("T", [1, 16])
@pytest.mark.parametrize("shape", [
    W.LayerShape("wide_f32", 70001, 3, 5, 2, 3, "f32", "f32"), W.LayerShape("deep_f32", 33, 2, 20003, 1, 9999, "f32", "f32"),
    W.LayerShape("wide_bf16", 65536, 3, 128, 2, 128, "bf16", "bf16"),
    W.LayerShape("deep_bf16", 128, 2, 16384, 1, 16384, "bf16", "bf16")], ids=lambda s: s.name)
def test_long_rows(shape, T):
    print(f"\n[case] few {shape.name} T={T}", flush=True)
    case = Hn.make_case(shape, T, 131)
    layer = _layer(case)
    y = layer(case.inp.x.cuda(), None if case.inp.logit_bias is None else case.inp.logit_bias.cuda())
    torch.cuda.synchronize()
    ora = _oracle(case)
    assert np.array_equal(layer.topk_ids.cpu().numpy(), ora["ids"])
    err = Hn.token_rel_l2(y.cpu().double().numpy(), ora["y"])
    print(f"[case] worst token {err.max():.2e}", flush=True)
    assert err.max() <= _y_tol(shape)


def test_no_tokens_and_no_rows():
    case = Hn.make_case(W.LayerShape("none", 256, 8, 128, 2, 128, "bf16", "bf16"), 3, 132)
    layer = _layer(case)
    layer.y.fill_(-3.0)
    x = case.inp.x.cuda()
    assert layer(x[:0]).shape == (0, 256)
    p = moe.Linear(torch.ones(8, 256).bfloat16().cuda(), max_rows=4)
    p.y.fill_(-3.0)
    assert p(x[:0]).shape == (0, 8)
    torch.cuda.synchronize()
    assert (layer.y == -3.0).all() and (p.y == -3.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_one_tokens_bad_activation_stays_with_it(bad):
    """NaN or Inf in a row of x: its logits are NaN or infinite, no other token sees it."""
    case = Hn.make_case(W.LayerShape("bad_x", 256, 8, 128, 2, 128, "bf16", "bf16", expert_budget=7), 9, 133)
    x = case.inp.x.clone()
    x[4, 100] = bad
    layer = _layer(case)
    y = layer(x.cuda(), None if case.inp.logit_bias is None else case.inp.logit_bias.cuda())
    torch.cuda.synchronize()
    assert not torch.isfinite(y[4]).any()
    keep = [t for t in range(9) if t != 4]
    # The others routed by themselves: the bad token's picks count as present, with no weight.
    assert torch.isfinite(y[keep]).all()


def _product(M, K, N, i, o, rows=None, seed=0):
    print(f"\n[case] linear {M}x{K}x{N} {i}->{o}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda").to(DT[i])
    w = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).to(DT[i])
    b = torch.randn(N, generator=g, device="cuda").to(DT[i])
    p = moe.Linear(w, b, "relu", out_dtype=o, max_rows=M)
    p.y.fill_(float("nan"))
    y = p(x)
    torch.cuda.synchronize()
    rows = torch.arange(M) if rows is None else rows
    x, y, w, b = x[rows.cuda()].cpu().double(), y[rows.cuda()].cpu().double(), w.cpu().double(), b.cpu().double()
    v = x @ w.t() + b
    tol = (K + 1) * 2.0 ** -24 * (x.abs() @ w.abs().t() + b.abs())
    want = v.clamp(min=0)
    tol = tol + torch.finfo(DT[o]).eps / 2 * (want + tol)
    assert ((y - want).abs() <= tol).all()


@pytest.mark.parametrize("i,o", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("M,K,N", [(1, 1 << 20, 3), (17, (1 << 20) - 1, 5), (300, 1 << 20, 2), (1, 3, 1 << 20),
                                   (20, 8, (1 << 20) - 3)])
def test_longest_rows_of_products(M, K, N, i, o):
    _product(M, K, N, i, o, seed=M)


@pytest.mark.parametrize("i,o", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("K,N", [(8, 9), (128, 256), (131, 30)])
def test_most_rows_of_products(K, N, i, o):
    M = 1 << 21
    rows = torch.cat([torch.arange(0, 300), torch.arange(M // 2 - 150, M // 2 + 150), torch.arange(M - 300, M)])
    _product(M, K, N, i, o, rows, seed=K)
