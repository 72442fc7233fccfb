"""moe_ffn_forward and moe_ffn_backward against float64 on the host.

Tolerance, per element, u = 2^-24.  A float32 sum of K products of exact factors is off by
at most `chain` u sum |products|: 16 products meet in one bf16 matrix instruction and 2 in
a float32 one, parts and their sums add less than 40.  The activations are good to 2^-21
(|v| + 1) with the hardware's exponential and reciprocal, their slopes to 2^-20 (|v| + 1);
|act'| <= 1.13, |act''| <= 1 (relu's slope is undefined where the gate's sign is).  h, the
gradients of gate and up, and the results are rounded to the type: half a step each.
Errors of a factor pass through a product with the other factors' magnitudes."""
import ctypes
import math

import pytest
import torch

import mixture_experts_layer_05_amd as moe

OK, NULL_PTR, BAD_SHAPE, BAD_DTYPE, UNSUPPORTED, WS_SMALL = 0, -1, -2, -3, -4, -5
FAKE = 0x1000
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


# ----------------------------------------------------------------------------- refusals (no GPU)

def _cfg(H=64, I=32, dtype=1, act=4):
    from mixture_experts_layer_05_amd.dense import _FfnConfig
    return _FfnConfig(H, I, dtype, act)


def _forward(T=4, c=None, **kw):
    c = c or _cfg()
    p = dict(x=FAKE, ldx=c.hidden_size, g=FAKE, u=FAKE, d=FAKE, y=2 * FAKE, ldy=c.hidden_size, kept=None, kept_bytes=0,
             ws=FAKE, ws_bytes=1 << 50)
    p.update(kw)
    return moe.lib().moe_ffn_forward(ctypes.byref(c), T, p["x"], p["ldx"], p["g"], p["u"], p["d"], p["y"], p["ldy"],
                                     p["kept"], p["kept_bytes"], p["ws"], p["ws_bytes"], None)


def _backward(T=4, c=None, **kw):
    c = c or _cfg()
    H = c.hidden_size
    p = dict(x=FAKE, ldx=H, g=FAKE, u=FAKE, d=FAKE, kept=FAKE, kept_bytes=1 << 50, dy=FAKE, lddy=H, dx=2 * FAKE, lddx=H,
             dg=2 * FAKE, du=2 * FAKE, dd=2 * FAKE, ws=FAKE, ws_bytes=1 << 50)
    p.update(kw)
    return moe.lib().moe_ffn_backward(ctypes.byref(c), T, p["x"], p["ldx"], p["g"], p["u"], p["d"], p["kept"],
                                      p["kept_bytes"], p["dy"], p["lddy"], p["dx"], p["lddx"], p["dg"], p["du"], p["dd"],
                                      p["ws"], p["ws_bytes"], None)


def test_refusals():
    for call in (_forward, _backward):
        assert call(T=-1) == BAD_SHAPE
        for kw in (dict(H=0), dict(I=0), dict(H=-3), dict(act=5), dict(act=-1)):
            assert call(c=_cfg(**kw)) == BAD_SHAPE
        for d in (2, 3, 4, -1, 9):
            assert call(c=_cfg(dtype=d)) == BAD_DTYPE
        assert call(c=_cfg(H=(1 << 20) + 1)) == UNSUPPORTED and call(c=_cfg(I=(1 << 18) + 1)) == UNSUPPORTED
        assert call(T=(1 << 21) + 1) == UNSUPPORTED
        for name in ("x", "g", "u", "d", "ws"):
            assert call(**{name: None}) == NULL_PTR
            assert call(**{name: FAKE + 1}) == UNSUPPORTED
        assert call(ldx=63) == BAD_SHAPE and call(ldx=(1 << 40) + 1) == UNSUPPORTED
        assert call(ws=FAKE + 8) == UNSUPPORTED and call(ws_bytes=100) == WS_SMALL
    assert _forward(T=0, x=None, g=None, u=None, d=None, y=None, ws=None) == OK
    assert _forward(y=None) == NULL_PTR and _forward(y=FAKE + 1) == UNSUPPORTED and _forward(ldy=63) == BAD_SHAPE
    assert _forward(kept=FAKE, kept_bytes=100) == WS_SMALL and _forward(kept=FAKE + 8, kept_bytes=1 << 30) == UNSUPPORTED
    assert _backward(kept=None) == NULL_PTR and _backward(dy=None) == NULL_PTR
    assert _backward(dg=None) == NULL_PTR and _backward(du=None) == NULL_PTR
    assert _backward(kept_bytes=100) == WS_SMALL and _backward(kept=FAKE + 8) == UNSUPPORTED
    assert _backward(lddy=63) == BAD_SHAPE and _backward(lddx=63) == BAD_SHAPE
    for name in ("dy", "dx", "dg", "du", "dd"):
        assert _backward(**{name: FAKE + 1}) == UNSUPPORTED
    assert _backward(T=0, x=None, g=None, u=None, d=None, kept=None, dy=None, dx=None, dg=None, du=None, dd=None, ws=None) == OK


def test_sizes_grow_with_the_rows():
    for H, I in ((1, 1), (5120, 2048), (1537, 2049)):
        for f in (lambda n: moe.ffn_workspace_size(H, I, n), lambda n: moe.ffn_workspace_size(H, I, n, "f32", True),
                  lambda n: moe.ffn_kept_size(H, I, n)):
            sizes = [f(n) for n in (1, 2, 7, 64, 1000, 8192)]
            assert sizes == sorted(sizes) and sizes[0] > 0


def test_the_binding_checks_its_arguments():
    w = {"gate": torch.zeros(8, 4), "up": torch.zeros(8, 4), "down": torch.zeros(4, 8)}
    with pytest.raises(ValueError, match="activation"):
        moe.GatedFFN(w, activation="tanh")
    with pytest.raises(ValueError, match="GPU"):
        moe.GatedFFN(w)
    for n in w:
        bad = dict(w, **{n: torch.zeros(5, 5)})
        with pytest.raises(ValueError):
            moe.GatedFFN(bad)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        moe.GatedFFN({n: t.half() for n, t in w.items()})


# ----------------------------------------------------------------------------- the formula

def _act64(v, name):
    """act, act' in float64."""
    if name == "relu":
        return v.clamp(min=0), (v > 0).double()
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(v / math.sqrt(2)))
        return v * c, c + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)
    if name == "silu":
        s = torch.sigmoid(v)
        return v * s, s * (1 + v * (1 - s))
    return v, torch.ones_like(v)


def _chain(K, dtype):
    return K / 16 + 56 if dtype == "bf16" else K / 2 + 56


def _expect(x, w, dy, act, dtype):
    """{name: (value, tolerance)} in float64."""
    half = torch.finfo(DT[dtype]).eps / 2
    x, wg, wu, wd = x.double(), w["gate"].double(), w["up"].double(), w["down"].double()
    H, I, T = x.shape[1], wg.shape[0], x.shape[0]
    cH, cI = _chain(H, dtype) * U, _chain(I, dtype) * U

    def rounded(v, e):
        return v, e + half * (v.abs() + e)

    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = cH * (x.abs() @ wg.abs().t()), cH * (x.abs() @ wu.abs().t())
    a, s = _act64(g, act)
    ea = 1.13 * eg + 2.0 ** -21 * (g.abs() + 1)
    es = (g.abs() <= eg).double() if act == "relu" else eg + 2.0 ** -20 * (g.abs() + 1)
    h = a * u
    _, eh = rounded(h, a.abs() * eu + ea * (u.abs() + eu) + 4 * U * h.abs())
    y = h @ wd.t()
    got = {"y": rounded(y, eh @ wd.abs().t() + cI * ((h.abs() + eh) @ wd.abs().t()))}
    if dy is None:
        return got
    dy = dy.double()
    dh = dy @ wd
    edh = cH * (dy.abs() @ wd.abs())
    du, dg = dh * a, dh * u * s
    _, edu = rounded(du, dh.abs() * ea + edh * (a.abs() + ea) + 4 * U * du.abs())
    b, eb = u * s, u.abs() * es + eu * (s.abs() + es)
    _, edg = rounded(dg, dh.abs() * eb + edh * (b.abs() + eb) + 4 * U * dg.abs())
    cT, c2I = _chain(T, dtype) * U, _chain(2 * I + 16, dtype) * U
    dx = dg @ wg + du @ wu
    mag = (dg.abs() + edg) @ wg.abs() + (du.abs() + edu) @ wu.abs()
    got["x"] = rounded(dx, edg @ wg.abs() + edu @ wu.abs() + c2I * mag)
    for n, d, e in (("gate", dg, edg), ("up", du, edu)):
        got[n] = rounded(d.t() @ x, e.t() @ x.abs() + cT * ((d.abs() + e).t() @ x.abs()))
    got["down"] = rounded(dy.t() @ h, dy.abs().t() @ eh + cT * (dy.abs().t() @ (h.abs() + eh)))
    return got


def _inputs(T, H, I, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H + pad, generator=g).to(DT[dtype])
    dy = torch.randn(T, H + pad, generator=g).to(DT[dtype])
    w = {"gate": torch.randn(I, H, generator=g) / H ** 0.5, "up": torch.randn(I, H, generator=g) / H ** 0.5,
         "down": torch.randn(H, I, generator=g) / I ** 0.5}
    return x, dy, {n: t.to(DT[dtype]) for n, t in w.items()}


def _compare(got, want, what):
    for n, (v, tol) in want.items():
        err = (got[n].cpu().double() - v).abs()
        print(f"[case] {what} {n}: worst error / tolerance {(err / tol).max() if err.numel() else 0:.3f}", flush=True)
        assert (err <= tol).all(), n


def _run(T, H, I, dtype, act="silu", seed=0, pad=0):
    print(f"\n[case] ffn T={T} H={H} I={I} {dtype} {act} pad={pad}", flush=True)
    x, dy, w = _inputs(T, H, I, dtype, seed, pad)
    xg, dyg, wg = x.cuda()[:, :H], dy.cuda()[:, :H], {n: t.cuda() for n, t in w.items()}
    want = _expect(x[:, :H], w, dy[:, :H], act, dtype)
    # Through the functions, with rows that lie apart and buffers that hold NaN before.
    full = torch.full((2, T, H + pad), 77.0, dtype=DT[dtype], device="cuda")
    y, dx = full[0][:, :H], full[1][:, :H]
    ws = torch.full((moe.ffn_workspace_size(H, I, T, dtype, True),), 0xFF, dtype=torch.uint8, device="cuda")
    kept = torch.full((moe.ffn_kept_size(H, I, T, dtype),), 0xFF, dtype=torch.uint8, device="cuda")
    grads = {n: torch.full_like(t, float("nan")) for n, t in wg.items()}
    serve = torch.full((T, H), float("nan"), dtype=DT[dtype], device="cuda")
    moe.ffn(xg, wg, serve, ws[:moe.ffn_workspace_size(H, I, T, dtype)], act)
    moe.ffn(xg, wg, y, ws, act, kept)
    ws.fill_(0xFF)
    moe.ffn_backward(xg, wg, kept, dyg, dx, grads, ws, act)
    torch.cuda.synchronize()
    assert torch.equal(serve, y)                         # keeping changes nothing
    assert (full[:, :, H:] == 77.0).all()                # between the rows
    _compare(dict(grads, x=dx, y=y), want, "functions")
    # Through the class, sized for more rows.
    op = moe.GatedFFN(wg, act, max_rows=T + 3, training=True)
    y2 = op(xg)
    d = op.backward(xg, dyg)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(d["x"], dx)
    for n in wg:
        assert torch.equal(d[n], grads[n])


SIZES = [(1, 1, 1), (1, 5120, 64), (1, 64, 2048), (2, 8, 7), (3, 129, 33), (7, 640, 515), (15, 256, 48), (16, 136, 16),
         (17, 64, 64), (33, 1000, 130), (64, 64, 64), (65, 2048, 100), (128, 512, 256), (129, 136, 257), (224, 1280, 640),
         (257, 1023, 515), (300, 72, 1025), (1, 31, 4097)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_sizes(T, H, I, dtype):
    _run(T, H, I, dtype, seed=T + H + I)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 150])
@pytest.mark.parametrize("act", ACTS)
def test_activations(act, T, dtype):
    _run(T, 192, 160, dtype, act, seed=3)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad", [1, 3, 8, 40])
@pytest.mark.parametrize("T", [1, 9, 70, 400])
def test_strides(T, pad, dtype):
    _run(T, 320, 200, dtype, "gelu", seed=4, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,act", [(1024, 512, 1024, "silu"), (1001, 1537, 2049, "gelu_tanh"), (2050, 1024, 1536, "gelu"),
                                       (4100, 264, 776, "relu")])
def test_large(T, H, I, act):
    _run(T, H, I, "bf16", act, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_against_differences(dtype):
    """d/dt of sum(dy * y) at x + t v, and likewise for each weight, from the forward pass
    itself in float32 (the bf16 backward is compared where its inputs are exact in bf16)."""
    T, H, I = 37, 48, 56
    x, dy, w = _inputs(T, H, I, "bf16", 11)
    x, dy, w = x[:, :H].float(), dy[:, :H].float(), {n: t.float() for n, t in w.items()}
    cast = {n: t.to(DT[dtype]).cuda() for n, t in w.items()}
    op = moe.GatedFFN(cast, "silu", max_rows=T, training=True)
    op(x.to(DT[dtype]).cuda())
    d = op.backward(x.to(DT[dtype]).cuda(), dy.to(DT[dtype]).cuda())

    def loss(x, w):
        f = moe.GatedFFN({n: t.float().cuda().contiguous() for n, t in w.items()}, "silu", max_rows=T)
        return (f(x.float().cuda()).double().cpu() * dy.double()).sum().item()

    g = torch.Generator().manual_seed(12)
    for n in ("x", "gate", "up", "down"):
        v = torch.randn(d[n].shape, generator=g)
        e = 2.0 ** -6 / v.abs().max().item()
        if n == "x":
            diff = (loss(x + e * v, w) - loss(x - e * v, w)) / (2 * e)
        else:
            diff = (loss(x, dict(w, **{n: w[n] + e * v})) - loss(x, dict(w, **{n: w[n] - e * v}))) / (2 * e)
        grad = d[n].double().cpu()
        # The difference: float32 sums of about 2^11 terms of size 1, 2^-24 2^11 / e; its
        # third derivative, of the order of the slope, times e^2 / 6.  The gradient: two
        # roundings of its type to each element, whose signs are independent of v.
        slope = (grad.abs() * v.abs().double()).sum().item()
        tol = 2.0 ** -13 / e + slope * e * e + (2.0 ** -6 if dtype == "bf16" else 2.0 ** -18) * (grad * v).norm().item()
        assert abs(diff - (grad * v.double()).sum().item()) <= tol, n


# ----------------------------------------------------------------------------- use

@pytest.mark.gpu
def test_parts_of_the_gradients():
    x, dy, w = _inputs(50, 96, 72, "bf16", 6)
    x, dy, w = x.cuda(), dy.cuda(), {n: t.cuda() for n, t in w.items()}
    op = moe.GatedFFN(w, max_rows=64, training=True)
    op(x)
    every = {n: t.clone() for n, t in op.backward(x, dy).items()}
    only = op.backward(x, dy, weights=False)
    assert set(only) == {"x"} and torch.equal(only["x"], every["x"])
    only = op.backward(x, dy, inputs=False)
    assert set(only) == {"gate", "up", "down"} and all(torch.equal(only[n], every[n]) for n in only)
    # Through the function, the down projection's alone.
    down = torch.full_like(w["down"], float("nan"))
    kept = op.kept
    moe.ffn_backward(x, w, kept, dy, None, {"down": down}, op.workspace)
    assert torch.equal(down, every["down"])
    with pytest.raises(ValueError, match="together"):
        moe.ffn_backward(x, w, kept, dy, None, {"gate": every["gate"]}, op.workspace)


@pytest.mark.gpu
def test_no_rows():
    _, _, w = _inputs(1, 96, 72, "bf16", 7)
    w = {n: t.cuda() for n, t in w.items()}
    op = moe.GatedFFN(w, max_rows=4, training=True)
    x = torch.empty(0, 96, dtype=torch.bfloat16, device="cuda")
    assert op(x).shape == (0, 96)
    for t in op.grads.values():
        t.fill_(float("nan"))
    d = op.backward(x, x)
    torch.cuda.synchronize()
    assert d["x"].shape == (0, 96) and all((d[n] == 0).all() for n in w)


@pytest.mark.gpu
def test_the_class_refuses():
    _, _, w = _inputs(1, 96, 72, "bf16", 7)
    w = {n: t.cuda() for n, t in w.items()}
    x = torch.zeros(3, 96, dtype=torch.bfloat16, device="cuda")
    serve, train = moe.GatedFFN(w, max_rows=4), moe.GatedFFN(w, max_rows=4, training=True)
    with pytest.raises(ValueError, match="training"):
        serve(x)
        serve.backward(x, x)
    with pytest.raises(ValueError, match="after a call"):
        train.backward(x, x)
    train(x)
    with pytest.raises(ValueError, match="after a call"):
        train.backward(x[:2], x[:2])
    with pytest.raises(ValueError, match="sized for"):
        serve(torch.zeros(5, 96, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        serve(x.float())
    with pytest.raises(ValueError):
        serve(torch.zeros(3, 95, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        serve(torch.zeros(96, 3, dtype=torch.bfloat16, device="cuda").t())
    with pytest.raises(ValueError, match="GPU"):
        serve(x.cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 20, 300])
def test_infinities_and_nan_stay_in_their_rows(T):
    """A row of x with a NaN, a row of dy with an infinity: other rows of y and dx are as
    without them."""
    x, dy, w = _inputs(T + 2, 72, 88, "bf16", 8)
    w = {n: t.cuda() for n, t in w.items()}
    op = moe.GatedFFN(w, max_rows=T + 2, training=True)
    y0 = op(x.cuda()).clone()
    dx0 = op.backward(x.cuda(), dy.cuda())["x"].clone()
    x[T, 71], dy[T + 1, 3] = float("nan"), float("inf")
    y1 = op(x.cuda())
    dx1 = op.backward(x.cuda(), dy.cuda())["x"]
    assert torch.equal(y1[:T], y0[:T]) and torch.equal(y1[T + 1], y0[T + 1]) and y1[T].isnan().all()
    assert torch.equal(dx1[:T], dx0[:T])
    assert dx1[T].isnan().all() and not dx1[T + 1].isfinite().any()


@pytest.mark.gpu
def test_training_step_in_a_graph_and_on_a_stream():
    """Forward and backward captured into one graph replay the eager bits, with eager work
    of another block between the replays; so does a run on another stream."""
    T, H, I = 300, 520, 392
    x, dy, w = _inputs(T, H, I, "bf16", 9)
    x, dy, w = x.cuda(), dy.cuda(), {n: t.cuda() for n, t in w.items()}
    op, other = (moe.GatedFFN(w, max_rows=T, training=True) for _ in range(2))

    def step(f):
        y = f(x)
        return dict(f.backward(x, dy), y=y)

    want = {n: t.clone() for n, t in step(other).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(op)
    side.synchronize()
    assert all(torch.equal(got[n], want[n]) for n in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(op)
    for k in range(4):
        for t in got.values():
            t.fill_(float("nan"))
        again = step(other)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) and torch.equal(again[n], want[n]) for n in want), k


# ----------------------------------------------------------------------------- every tile, every end

def _check_on_the_gpu(T, H, I, act, seed, pad=0, train=True):
    """As _run for bf16, the float64 results taken on the GPU for sizes that the host would
    take long for, through the class alone."""
    print(f"\n[case] ffn T={T} H={H} I={I} bf16 {act} pad={pad}", flush=True)
    x, dy, w = _inputs(T, H, I, "bf16", seed, pad)
    x, dy, w = x.cuda()[:, :H], dy.cuda()[:, :H], {n: t.cuda() for n, t in w.items()}
    want = _expect(x, w, dy if train else None, act, "bf16")
    op = moe.GatedFFN(w, act, max_rows=T, training=train)
    op.workspace.fill_(0xFF)
    got = {"y": op(x)}
    if train:
        op.workspace.fill_(0xFF)
        got.update(op.backward(x, dy))
    torch.cuda.synchronize()
    for n, (v, tol) in want.items():
        worst = ((got[n].double() - v).abs() / tol).max().item()
        print(f"[case] {n}: worst error / tolerance {worst:.3f}", flush=True)
        assert worst <= 1, n


# Rows, widths and contractions that end inside tiles, stages and pieces of 8, around every
# tile height, with rows aligned (the DMA kernels), laid out afresh (odd sizes or strides)
# and too small for that.
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(17, 72, 40), (31, 136, 200), (40, 264, 328), (64, 1024, 2048), (65, 2040, 1544), (100, 520, 72),
                                   (129, 4096, 264), (191, 1000, 2056), (250, 3000, 1000), (255, 64, 4096), (256, 256, 8), (257, 8, 256),
                                   (500, 2056, 1032), (1000, 1032, 2080), (1023, 4104, 1096)])
def test_ends_of_tiles(T, H, I):
    _check_on_the_gpu(T, H, I, "silu", seed=T)
    _check_on_the_gpu(T, H, I, "gelu_tanh", seed=T + 1, pad=5)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(20, 31, 35), (33, 129, 257), (200, 1001, 777), (300, 1025, 65), (513, 2049, 1027)])
def test_odd_ends(T, H, I):
    _check_on_the_gpu(T, H, I, "gelu", seed=T, pad=3)


# Whole rounds of 256 x 256 tiles and a rest in parts, in every product of a step.
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,pad", [(4200, 2056, 4104, 0), (5000, 4096, 2560, 8), (4099, 2049, 4101, 1)])
def test_rounds_of_tiles_and_their_rest(T, H, I, pad):
    _check_on_the_gpu(T, H, I, "silu", seed=14, pad=pad)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [2, 16, 150])
def test_far_strides(T):
    """Rows 2^23 elements and more apart: beyond the aligned kernels' offsets."""
    H, I = 64, 96
    x, dy, w = _inputs(T, H, I, "bf16", 15)
    far = torch.zeros(2, T * ((1 << 23) + 8), dtype=torch.bfloat16, device="cuda")
    xs, ds = (far[i].view(T, -1)[:, :H] for i in range(2))
    xs.copy_(x[:, :H])
    ds.copy_(dy[:, :H])
    op = moe.GatedFFN({n: t.cuda() for n, t in w.items()}, max_rows=T, training=True)
    want = _expect(x[:, :H], w, dy[:, :H], "silu", "bf16")
    y = op(xs)
    _compare(dict(op.backward(xs, ds), y=y), want, "far")


@pytest.mark.gpu
def test_weights_off_their_boundaries():
    """Weights and rows that start two bytes behind a 16-byte boundary."""
    for T, H, I in ((5, 64, 72), (300, 264, 520)):
        x, dy, w = _inputs(T, H, I, "bf16", 16)

        def shifted(t):
            buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
            return buf[1:].view(t.shape).copy_(t)

        op = moe.GatedFFN({n: shifted(t) for n, t in w.items()}, max_rows=T, training=True)
        y = op(shifted(x))
        want = _expect(x, w, dy, "silu", "bf16")
        _compare(dict(op.backward(shifted(x), shifted(dy)), y=y), want, "shifted")


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 300])
def test_an_infinity_behind_the_end_stays_there(T):
    """Padding between the rows of x and dy that holds infinities and NaN: nothing of it
    reaches a result, whichever way the rows are read."""
    for H, I, pad in ((72, 88, 8), (264, 520, 8), (71, 88, 9), (265, 519, 3)):
        x, dy, w = _inputs(T, H, I, "bf16", 17, pad)
        x[:, H:], dy[:, H:] = float("inf"), float("nan")
        op = moe.GatedFFN({n: t.cuda() for n, t in w.items()}, max_rows=T, training=True)
        want = _expect(x[:, :H], w, dy[:, :H], "silu", "bf16")
        y = op(x.cuda()[:, :H])
        _compare(dict(op.backward(x.cuda()[:, :H], dy.cuda()[:, :H]), y=y), want, "padding")


# Up to eight rows h keeps what its rounding leaves as a second bf16 number: y's own rounding is
# the only one.  What remains of h is half a step of a half step: 2^-8 2^-8 |h|, and sums of
# twice as many products (32 to a pair of matrix instructions).
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I,pad", [(1, 64, 64, 0), (1, 5120, 2048, 0), (7, 515, 1023, 3), (8, 256, 512, 8), (8, 41, 4097, 0),
                                       (3, 16, 1, 0), (2, 5120, 17408, 0)])
@pytest.mark.parametrize("train", [False, True])
def test_few_rows_round_once(T, H, I, pad, train):
    print(f"\n[case] ffn rounds once T={T} H={H} I={I} pad={pad} train={train}", flush=True)
    x, _, w = _inputs(T, H, I, "bf16", T + H + I, pad)
    x = x[:, :H]
    op = moe.GatedFFN({n: t.cuda() for n, t in w.items()}, "gelu_tanh", max_rows=T, training=train)
    op.workspace.fill_(0xFF)
    y = op(x.cuda()).cpu().double()
    x, wg, wu, wd = x.double(), w["gate"].double(), w["up"].double(), w["down"].double()
    cH, cI = _chain(H, "bf16") * U, (2 * I / 16 + 56) * U
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = cH * (x.abs() @ wg.abs().t()), cH * (x.abs() @ wu.abs().t())
    a, _ = _act64(g, "gelu_tanh")
    ea = 1.13 * eg + 2.0 ** -21 * (g.abs() + 1)
    h = a * u
    eh = a.abs() * eu + ea * (u.abs() + eu) + (4 * U + 2.0 ** -16) * h.abs()
    want = h @ wd.t()
    e = eh @ wd.abs().t() + cI * ((h.abs() + eh) @ wd.abs().t())
    tol = e + 2.0 ** -8 * (want.abs() + e)
    err = (y - want).abs()
    print(f"[case] worst error / tolerance {(err / tol).max():.3f}", flush=True)
    assert (err <= tol).all()


# Few rows and many weights, which go through tiles; the functions' and the training form's
# results are the same bits.
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(5, 5120, 17408), (12, 5120, 8192), (16, 4096, 16384)])
def test_few_rows_and_many_weights(T, H, I):
    print(f"\n[case] ffn T={T} H={H} I={I} many weights", flush=True)
    x, _, w = _inputs(T, H, I, "bf16", T)
    wg = {n: t.cuda() for n, t in w.items()}
    op, train = (moe.GatedFFN(wg, "silu", max_rows=T, training=k) for k in (False, True))
    op.workspace.fill_(0xFF)
    y = op(x.cuda())
    assert torch.equal(y, train(x.cuda()))
    _compare({"y": y}, _expect(x, w, None, "silu", "bf16"), "many weights")
