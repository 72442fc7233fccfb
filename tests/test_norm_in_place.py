"""The norms' outputs in an input's place, where the interface allows it: z in the residual's,
and the residual's gradient in dz's."""
import pytest
import torch

import mixture_experts_layer_05_amd as moe
from tests import test_norm as N


# Rows of one wave and of several, of one chunk to a lane and of more; fewer rows than there
# are groups, and several to a group with a last round that not every group has a row in.
@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 64), (37, 200), (2100, 64), (9001, 320), (300, 1024), (4099, 1536), (1999, 5120), (700, 8200),
                                 (530, 12000)])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [0, 5])
def test_gradient_of_the_residual_in_place(T, H, stream, pad):
    print(f"\n[case] norm backward in place T={T} H={H} {stream} pad={pad}", flush=True)
    p = N._inputs(T, H, "bf16", stream, stream, stream, "channel", True, False, True, T + H, pad)
    c = {k: N._gpu(v) for k, v in p.items()}
    ws = torch.full((moe.norm_backward_workspace_size(H, T),), 0xFF, dtype=torch.uint8, device="cuda")

    def back(dz, dr):
        got = {n: torch.full_like(t, float("nan")) for n, t in (("dy", c["y"]), ("dgate", c["gate"]), ("dweight", c["w"]),
                                                                ("dpost_weight", c["pw"]))}
        moe.norm_backward(c["y"], c["z"], dz, c["dout"], ws, dresidual=dr, weight=c["w"], post_weight=c["pw"], gate=c["gate"],
                          residual_scale=0.75, block_scale=0.5, **got)
        return dict(got, dresidual=dr)

    want = back(c["dz"], torch.full_like(c["dz"], float("nan")))
    whole = torch.full((T, H + pad), 7.0, dtype=N.DT[stream], device="cuda")
    for k in range(4):
        dz = whole[:, :H].copy_(c["dz"])
        got = back(dz, dz)
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want), k
        assert (whole[:, H:] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(37, 200), (2100, 64), (300, 5120), (700, 8200), (257, 12000)])
@pytest.mark.parametrize("stream", ["bf16", "f32"])
def test_stream_in_place(T, H, stream):
    p = N._inputs(T, H, "f32", stream, stream, stream, "token", True, True, True, T + H, 3)
    c = {k: N._gpu(v) for k, v in p.items()}
    args = dict(weight=c["w"], bias=c["wb"], post_weight=c["pw"], post_bias=c["pb"], gate=c["gate"], kind="layer")
    z, out, out2 = (torch.empty(T, H, dtype=N.DT[stream], device="cuda") for _ in range(3))
    moe.norm(c["y"], c["r"], z, out, **args)
    r = c["r"].clone()
    moe.norm(c["y"], r, r, out2, **args)
    assert torch.equal(r, z) and torch.equal(out2, out)


def test_other_strides_in_place_are_refused():
    """z in the residual's place, or its gradient in dz's, with rows that lie elsewhere would
    overwrite rows that are still to be read (no GPU: nothing is launched)."""
    assert N._forward(r=N.FAKE, z=N.FAKE, ldr=64, ldz=72) == N.BAD_SHAPE
    assert N._forward(r=N.FAKE, z=N.FAKE, ldr=72, ldz=64) == N.BAD_SHAPE
    assert N._backward(dz=N.FAKE, dr=N.FAKE, lddz=64, lddr=72) == N.BAD_SHAPE
    assert N._backward(dz=N.FAKE, dr=N.FAKE, lddz=72, lddr=64) == N.BAD_SHAPE
    # Elsewhere strides differ as they like: the call gets as far as its other arguments.
    assert N._forward(r=2 * N.FAKE, z=N.FAKE, ldr=64, ldz=72, out=N.FAKE, c=N._cfg(out=4)) == N.NULL_PTR
    assert N._backward(dz=2 * N.FAKE, dr=N.FAKE, lddz=64, lddr=72, ws_bytes=16) == N.WS_SMALL
    assert N._backward(dz=None, dr=None, lddz=64, lddr=72, ws_bytes=16) == N.WS_SMALL
