"""moe_linear: y = act(x W^T + bias) + residual, against float64 on the host.

Tolerance, per element.  Products of two bf16 values are exact in float32; a float32
sum of K products in any order is off by at most (K - 1) steps of half an ulp of the
running sum, (K - 1) 2^-24 sum |x w|, and far less here, where the K terms are added
in groups: a chain is at most K / 16 + 32 long.  The activations' slope is at most
1.13 and their own error at most 2^-21 (|v| + 1).  Adding the residual rounds to
2^-24 of the result, storing y to half a step of its type."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_05_amd as moe

OK, NULL_PTR, BAD_SHAPE, BAD_DTYPE, UNSUPPORTED, WS_SMALL = 0, -1, -2, -3, -4, -5
FAKE = 0x1000
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------- refusals (no GPU)

def _call(M=4, K=64, N=32, in_dtype=1, out_dtype=1, act=0, **kw):
    p = dict(x=FAKE, ldx=K, w=FAKE, ldw=K, bias=None, residual=None, ldr=0, y=2 * FAKE, ldy=N, ws=FAKE, ws_bytes=1 << 40)
    p.update(kw)
    c = moe._LinearConfig(K, N, in_dtype, out_dtype, act)
    return moe.lib().moe_linear(ctypes.byref(c), M, p["x"], p["ldx"], p["w"], p["ldw"], p["bias"], p["residual"],
                                p["ldr"], p["y"], p["ldy"], p["ws"], p["ws_bytes"], None)


def test_refusals():
    assert _call(M=0, x=None, w=None, y=None, ws=None) == OK
    assert _call(M=-1) == BAD_SHAPE
    assert _call(K=0) == BAD_SHAPE and _call(N=0) == BAD_SHAPE and _call(N=-5) == BAD_SHAPE
    assert _call(M=(1 << 21) + 1) == UNSUPPORTED
    assert _call(K=(1 << 20) + 1) == UNSUPPORTED and _call(N=(1 << 20) + 1) == UNSUPPORTED
    for i, o in ((2, 1), (3, 1), (1, 2), (0, 1), (9, 1), (-1, 0)):
        assert _call(in_dtype=i, out_dtype=o) == BAD_DTYPE
    assert _call(act=5) == BAD_SHAPE and _call(act=-1) == BAD_SHAPE
    for name in ("x", "w", "y", "ws"):
        assert _call(**{name: None}) == NULL_PTR
    assert _call(ldx=63) == BAD_SHAPE and _call(ldw=63) == BAD_SHAPE and _call(ldy=31) == BAD_SHAPE
    assert _call(residual=FAKE, ldr=31) == BAD_SHAPE
    assert _call(residual=2 * FAKE, ldr=40) == BAD_SHAPE              # y itself, at another stride
    assert _call(ldx=(1 << 40) + 1) == UNSUPPORTED and _call(ldy=1 << 62) == UNSUPPORTED
    assert _call(M=224, K=5120, N=5120, ws_bytes=0) == WS_SMALL
    for name in ("x", "w", "y", "bias", "ws"):
        assert _call(**{name: FAKE + 1}) == UNSUPPORTED
    assert _call(residual=FAKE + 1, ldr=32) == UNSUPPORTED
    assert _call(in_dtype=0, out_dtype=0, x=FAKE + 2) == UNSUPPORTED
    assert _call(out_dtype=0, y=FAKE + 2) == UNSUPPORTED


def test_workspace_size_is_monotone_in_rows():
    for K, N, i, o in ((5120, 5120, "bf16", "bf16"), (64, 64, "f32", "f32"), (16384, 80, "bf16", "f32"), (1023, 515, "bf16", "f32")):
        sizes = [moe.linear_workspace_size(K, N, m, i, o) for m in
                 (0, 1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 224, 256, 257, 1000, 1024, 4096, 8192)]
        assert sizes == sorted(sizes), (K, N, sizes)
    with pytest.raises(moe.MoEError):
        moe.linear_workspace_size(0, 5, 1)


def test_binding_refusals():
    x = torch.zeros(2, 4)
    with pytest.raises(ValueError, match="activation"):
        moe.linear(x, x, None, None, x, x, activation="swish")
    with pytest.raises(ValueError, match="float32"):
        moe.linear(x.half(), x.half(), None, None, x, x)
    with pytest.raises(ValueError, match="GPU"):
        moe.linear(x, torch.zeros(3, 4), None, None, torch.zeros(2, 3), x)


# ----------------------------------------------------------------------------- GPU

def _act64(v, name):
    if name == "relu":
        return v.clamp(min=0)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v * torch.sigmoid(v)
    return v


def _inputs(M, K, N, i, o, bias, residual, seed, padx=0, padw=0, padr=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K + padx, generator=g).to(DT[i])[:, :K]
    w = (torch.randn(N, K + padw, generator=g) / math.sqrt(K)).to(DT[i])[:, :K]
    b = torch.randn(N, generator=g).to(DT[i]) if bias else None
    r = torch.randn(M, N + padr, generator=g).to(DT[o])[:, :N] if residual else None
    return x, w, b, r


def _gpu(t):
    """The same matrix at the same stride on the GPU."""
    if t is None:
        return None
    base = t if t._base is None else t._base
    return base.cuda()[tuple(slice(0, n) for n in t.shape)]


def _expect(x, w, b, r, act, o):
    v = x.double() @ w.double().t()
    mag = x.double().abs() @ w.double().abs().t()
    K = x.shape[1]
    if b is not None:
        v, mag = v + b.double(), mag + b.double().abs()
    tol = 1.13 * (K / 16 + 32) * 2.0 ** -24 * mag + 2.0 ** -21 * (v.abs() + 1)
    y = _act64(v, act)
    if r is not None:
        y = y + r.double()
    return y, tol + (2.0 ** -24 + torch.finfo(DT[o]).eps / 2) * (y.abs() + tol)


def _run(M, K, N, i, o, act="none", bias=False, residual=False, seed=0, pads=(0, 0, 0, 0), rows=None):
    print(f"\n[case] linear {M}x{K}x{N} {i}->{o} {act} bias={bias} residual={residual} pads={pads}", flush=True)
    x, w, b, r = _inputs(M, K, N, i, o, bias, residual, seed, *pads[:3])
    ws = torch.full((moe.linear_workspace_size(K, N, M, i, o),), 0xFF, dtype=torch.uint8, device="cuda")
    full = torch.full((M, N + pads[3]), 77.0, dtype=DT[o], device="cuda")
    y = full[:, :N]
    moe.linear(_gpu(x), _gpu(w), _gpu(b), _gpu(r), y, ws, act)
    torch.cuda.synchronize()
    assert (full[:, N:] == 77.0).all()                    # between the rows
    if rows is not None:                                  # check some rows of a large product
        x, r, y = x[rows], None if r is None else r[rows], y[rows.cuda()]
    want, tol = _expect(x, w, b, r, act, o)
    err = (y.cpu().double() - want).abs()
    print(f"[case] worst error / tolerance {(err / tol).max():.3f}", flush=True)
    assert (err <= tol).all()


SIZES = [(1, 1, 1), (1, 5120, 64), (1, 128, 5120), (2, 8, 7), (3, 129, 33), (7, 640, 515), (15, 256, 48), (16, 128, 16),
         (16, 4097, 31), (17, 64, 64), (33, 1000, 130), (63, 96, 65), (64, 64, 64), (65, 2048, 100), (128, 512, 256),
         (129, 136, 257), (224, 1280, 640), (256, 256, 256), (257, 1023, 515), (300, 72, 1025), (1, 16384, 16),
         (40, 8192, 24)]


@pytest.mark.gpu
@pytest.mark.parametrize("i,o", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_sizes(M, K, N, i, o):
    _run(M, K, N, i, o, bias=True, residual=True, act="silu", seed=M + K + N)


@pytest.mark.gpu
@pytest.mark.parametrize("i,o", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("M", [3, 50, 300])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_epilogues(act, M, i, o):
    for bias, residual in ((False, False), (True, False), (False, True)):
        _run(M, 192, 160, i, o, act, bias, residual, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("i,o", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("pads", [(8, 0, 0, 0), (0, 8, 0, 8), (1, 0, 0, 0), (0, 3, 0, 0), (0, 0, 1, 3), (5, 5, 5, 5)])
@pytest.mark.parametrize("M", [1, 9, 70, 400])
def test_strides(M, pads, i, o):
    _run(M, 320, 200, i, o, "gelu", True, True, seed=4, pads=pads)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(1024, 1024, 2048), (2048, 4096, 1024), (1001, 1537, 2049), (4100, 520, 776)])
@pytest.mark.parametrize("o", ["bf16", "f32"])
def test_large(M, K, N, o):
    _run(M, K, N, "bf16", o, "gelu_tanh", True, True, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N", [(8192, 1536, 4096), (5000, 5120, 5120)])
def test_largest(M, K, N):
    rows = torch.cat([torch.arange(0, 40), torch.arange(M - 300, M), torch.arange(2000, 2300)])
    _run(M, K, N, "bf16", "bf16", "none", True, True, seed=6, rows=rows)


# More parts of tiles than run at a time.
@pytest.mark.gpu
@pytest.mark.parametrize("M,K,N,pads", [(1529, 2048, 1920, (0, 0, 0, 0)), (1300, 2501, 2051, (1, 3, 5, 7))])
def test_large_f32(M, K, N, pads):
    rows = torch.cat([torch.arange(0, 140), torch.arange(M - 140, M)])
    _run(M, K, N, "f32", "f32", "silu", True, True, seed=12, pads=pads, rows=rows)


# 256 x 256 tiles, cut at both edges; rows of x and W further apart than they are long, y and
# the residual aligned to four elements or not.
@pytest.mark.gpu
@pytest.mark.parametrize("o", ["bf16", "f32"])
@pytest.mark.parametrize("N,pads", [(3900, (8, 8, 4, 4)), (3900, (0, 0, 1, 3)), (3897, (64, 8, 3, 7))])
def test_wide_tiles(N, pads, o):
    M = 4001
    rows = torch.cat([torch.arange(0, 300), torch.arange(M - 200, M)])
    _run(M, 256, N, "bf16", o, "silu", True, True, seed=10, pads=pads, rows=rows)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 200, 1500])
def test_in_place_on_the_residual(M):
    """residual may be y: the residual stream updated where it stands."""
    x, w, b, r = _inputs(M, 512, 384, "bf16", "bf16", True, True, 7)
    y = r.cuda()
    ws = torch.empty(moe.linear_workspace_size(512, 384, M), dtype=torch.uint8, device="cuda")
    moe.linear(x.cuda(), w.cuda(), b.cuda(), y, y, ws)
    want, tol = _expect(x, w, b, r, "none", "bf16")
    assert ((y.cpu().double() - want).abs() <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 20, 300])
def test_infinities_and_nan_stay_in_their_rows_and_columns(M):
    x, w, _, _ = _inputs(M, 200, 90, "bf16", "f32", False, False, 8)
    x[0, 199], w[50, 3] = float("inf"), float("nan")
    ws = torch.empty(moe.linear_workspace_size(200, 90, M, "bf16", "f32"), dtype=torch.uint8, device="cuda")
    y = torch.empty(M, 90, device="cuda")
    moe.linear(x.cuda(), w.cuda(), None, None, y, ws, "silu")
    y = y.cpu()
    assert torch.isnan(y[:, 50]).all()
    rest = torch.arange(90) != 50
    want, tol = _expect(x[1:], w[rest], None, None, "silu", "f32")
    assert ((y[1:, rest].double() - want).abs() <= tol).all()
    s = x[0].double() @ w[rest].double().t()                # +inf or -inf: silu gives +inf or NaN
    assert (torch.isposinf(y[0, rest]) == torch.isposinf(s)).all()


@pytest.mark.gpu
def test_saturated_activations():
    """Sums far out on either side: exp and tanh overflow, the activations do not."""
    v = torch.tensor([-1e30, -1e4, -200.0, -90.0, -30.0, -1e-20, 0.0, 1e-20, 30.0, 90.0, 200.0, 1e4, 1e12])
    w = torch.eye(13)
    ws = torch.empty(moe.linear_workspace_size(13, 13, 1, "f32"), dtype=torch.uint8, device="cuda")
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        y = torch.empty(1, 13, device="cuda")
        moe.linear(v[None].cuda(), w.cuda(), None, None, y, ws, act)
        want = _act64(v.double().clamp(min=-1e20), act)
        assert ((y.cpu()[0].double() - want).abs() <= 2.0 ** -20 * want.abs() + 1e-30).all(), (act, y, want)


@pytest.mark.gpu
def test_projection_class_and_graph():
    x, w, b, r = _inputs(20, 256, 192, "bf16", "bf16", True, True, 9)
    p = moe.Linear(w.cuda(), b.cuda(), "gelu", max_rows=24)
    xg, rg = x.cuda(), r.cuda()
    want, tol = _expect(x, w, b, r, "gelu", "bf16")
    p.y.fill_(5.0)
    assert ((p(xg, rg).cpu().double() - want).abs() <= tol).all()
    assert (p.y[20:] == 5.0).all()
    out = torch.empty(20, 192, dtype=torch.bfloat16, device="cuda")
    assert p(xg, rg, out=out) is out and torch.equal(out, p.y[:20])
    with pytest.raises(ValueError):
        p(torch.zeros(25, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        p(xg.t())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        p(xg, rg)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p(xg, rg)
    for k in range(4):
        xg.copy_(x.roll(k, 0))
        eager = p(xg, rg, out=out).clone()
        p.y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p.y[:20], eager)


@pytest.mark.gpu
def test_replaced_parameters_are_checked():
    w, x = torch.zeros(16, 8).cuda(), torch.ones(2, 8).cuda()
    p = moe.Linear(w, torch.zeros(16).cuda(), max_rows=2)
    p(x)
    p.bias = torch.zeros(8).cuda()
    with pytest.raises(ValueError, match="bias"):
        p(x)
    p.bias = None
    p.weight = w.bfloat16()
    with pytest.raises(ValueError, match="weight"):
        p(x)
    p.weight = w
    with pytest.raises(ValueError, match="GPU"):
        p(x, residual=torch.zeros(2, 16))
    p.bias = torch.zeros(16)
    with pytest.raises(ValueError, match="GPU"):
        p(x)
    p.bias = torch.full((16,), 3.0).cuda()
    assert (p(x) == 3).all()
