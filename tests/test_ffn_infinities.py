"""Infinite weights of the gated FFN's down projection, on either side of the row count up to
which h is a sum of two bf16 numbers: y is what the formula gives, an infinity where one
meets an h that is not 0, NaN where infinities of both signs meet, and finite elsewhere.
Tolerances are those of test_ffn.py."""
import pytest
import torch

import mixture_experts_layer_05_amd as moe
from tests import test_ffn as F


# One part of the contraction and several, eight and sixteen columns to a workgroup, odd rows.
@pytest.mark.gpu
@pytest.mark.parametrize("H,I", [(512, 640), (64, 4096), (41, 4097), (8256, 64)])
@pytest.mark.parametrize("T", [1, 3, 7, 8, 9, 16, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinite_down_weights(T, H, I, dtype):
    print(f"\n[case] ffn infinite weights T={T} H={H} I={I} {dtype}", flush=True)
    x, _, w = F._inputs(T, H, I, dtype, 32)
    inf = float("inf")
    w["down"][3, 5], w["down"][7, I - 1], w["down"][H - 1, 11] = inf, -inf, inf
    w["down"][9, 8], w["down"][9, 13] = inf, -inf
    finite = dict(w, down=torch.where(w["down"].isinf(), torch.zeros_like(w["down"]), w["down"]))
    want, tol = F._expect(x, finite, None, "silu", dtype)["y"]
    # h where an infinite weight meets it is off by less than it is large: its sign is certain.
    g, u = x.double() @ w["gate"].double().t(), x.double() @ w["up"].double().t()
    h = g * torch.sigmoid(g) * u
    at = [5, 8, 11, 13, I - 1]
    assert (h[:, at].abs() > 2.0 ** -14 * (g[:, at].abs() + 1) * (u[:, at].abs() + 1)).all()
    want = want.clone()
    want[:, 3], want[:, 7], want[:, H - 1] = (s * h[:, k].sign() * inf for s, k in ((1, 5), (-1, I - 1), (1, 11)))
    want[:, 9] = h[:, 8].sign() * inf - h[:, 13].sign() * inf
    for training in (False, True):
        op = moe.GatedFFN({n: t.cuda() for n, t in w.items()}, max_rows=T, training=training)
        op.workspace.fill_(0xFF)
        y = op(x.cuda()).cpu().double()
        odd = ~want.isfinite()
        assert torch.equal(y[odd].nan_to_num(7.0, 1.0, -1.0), want[odd].nan_to_num(7.0, 1.0, -1.0))
        err = (y - want).abs()[~odd]
        print(f"[case] worst error / tolerance {(err / tol[~odd]).max():.3f}", flush=True)
        assert (err <= tol[~odd]).all()
