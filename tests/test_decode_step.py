"""The operators as a decode step uses them: attention output projection onto the
residual stream, the few-token layer, a projection of its output; eager and as one
captured graph."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_05_amd as moe
import workloads as W
from oracle import moe as O
from tests import harness as Hn

pytestmark = pytest.mark.gpu


def test_projection_layer_projection():
    shape, T, A, V = W.LayerShape("step", 512, 16, 256, 2, 256, "bf16", "bf16"), 7, 768, 1000
    case = Hn.make_case(shape, T, 91)
    H = shape.hidden_size
    g = torch.Generator().manual_seed(92)
    attn = torch.randn(T, A, generator=g).bfloat16().cuda()
    # The stream starts so that the projection's result is the case's x, whose routing has margins.
    wo = (torch.randn(H, A, generator=g) / A ** 0.5).bfloat16().cuda()
    proj = (attn.double() @ wo.double().t())
    stream0 = (case.inp.x.cuda().double() - proj).bfloat16()
    wv = (torch.randn(V, H, generator=g) / H ** 0.5).bfloat16().cuda()
    up = moe.Linear(wo, max_rows=T)
    head = moe.Linear(wv, out_dtype="f32", max_rows=T)
    layer = moe.MoELayer(Hn.config(shape), case.weights, case.inp.w_router.cuda(), case.inp.w_shared_gate.cuda(),
                         case.shared, max_tokens=T, act_output=True, few=True)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")

    def step():
        x.copy_(stream0)
        up(attn, x, out=x)
        layer(x)
        return head(layer.y_act)

    logits = step().clone()
    torch.cuda.synchronize()
    xin = x.cpu()
    # x: one bf16 rounding of a float32 sum; the routing below takes the x that came out.
    want_x = proj + stream0.double()
    assert ((x.double() - want_x).abs() <= 2.0 ** -8 * want_x.abs() + 1e-5).all()
    r = O.route(xin, case.inp.w_router, case.inp.w_shared_gate, None, 2, True, 0, 0.0)
    y = O.moe_combine(xin, r["ids"], r["w"], r["shared_gate"], case.expert_cpu, case.shared_cpu(), "bf16", None,
                      ["model"])["model"]
    assert np.array_equal(layer.topk_ids.cpu().numpy(), r["ids"])
    assert Hn.rel_l2(layer.y.cpu().double().numpy(), y) <= 2.0 ** -16
    want = layer.y_act.double() @ wv.double().t()
    assert ((logits.double() - want).abs() <= 1e-4).all()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        head.y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(head.y, logits)
