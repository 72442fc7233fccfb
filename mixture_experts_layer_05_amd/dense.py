"""Binding of the operators around the MoE layer beside `Linear`: the dense gated FFN
with its backward pass, the norms before and after a block, and products in 8-bit
integers.  As in the rest of the binding every step runs in the HIP kernels behind the C
ABI of include/moe_mi355x.h, on the current stream, and nothing falls back.

autograd does not see these calls: results have no grad_fn, and gradients come from the
backward passes' own calls (GatedFFN.backward, ResidualNorm.backward)."""
from __future__ import annotations

import ctypes
import warnings
from typing import Dict, Optional

import torch

from . import (ACTIVATIONS, DTYPES, _check, _dtype_code, _expect, _on, _ptr, _rows, _stream_of, _together, lib)

_BACK = {v: k for k, v in DTYPES.items()}


class _FfnConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden_size", "intermediate_size", "dtype", "activation")]


def _activation(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation: expected one of {sorted(ACTIVATIONS)}, got {name!r}")
    return ACTIVATIONS[name]


def _bytes_of(fn: str, *args) -> int:
    n = ctypes.c_size_t(0)
    _check(getattr(lib(), fn)(*args, ctypes.byref(n)), fn)
    return n.value


def _outside_autograd(what: str, gradients: str) -> None:
    """Warns of an input whose gradient autograd would look for in vain."""
    if torch.is_grad_enabled():
        warnings.warn(f"{what}: an input requires gradients, but autograd does not see this call: its results have no "
                      f"grad_fn ({gradients})", stacklevel=3)


# ----------------------------------------------------------------------------- gated FFN

def _ffn_config(x_dtype: int, gate: torch.Tensor, activation: str) -> _FfnConfig:
    intermediate, hidden = gate.shape
    return _FfnConfig(hidden, intermediate, x_dtype, _activation(activation))


def ffn_workspace_size(hidden_size: int, intermediate_size: int, max_rows: int, dtype: str = "bf16",
                       backward: bool = False) -> int:
    c = _FfnConfig(hidden_size, intermediate_size, DTYPES[dtype], 0)
    return _bytes_of("moe_ffn_workspace_size", ctypes.byref(c), int(max_rows), int(backward))


def ffn_kept_size(hidden_size: int, intermediate_size: int, max_rows: int, dtype: str = "bf16") -> int:
    c = _FfnConfig(hidden_size, intermediate_size, DTYPES[dtype], 0)
    return _bytes_of("moe_ffn_kept_size", ctypes.byref(c), int(max_rows))


def _ffn_weights(weights: Dict[str, torch.Tensor], H: int, I: int, dtype, device, what: str = ""):
    for n, shape in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I))):
        _expect(weights[n], shape, dtype, what + n)
    _together(device, weights["gate"], weights["up"], weights["down"])
    return _ptr(weights["gate"]), _ptr(weights["up"]), _ptr(weights["down"])


def ffn(x, weights: Dict[str, torch.Tensor], y, workspace, activation: str = "silu", kept=None, stream=None) -> None:
    """y = (act(x gate^T) * (x up^T)) down^T (moe_ffn_forward).  x and y [T, H] may be
    views with rows further apart than they are long; weights {gate [I, H], up [I, H],
    down [H, I]} are contiguous and share x's dtype.  `kept`, a buffer of ffn_kept_size
    bytes, takes what ffn_backward needs."""
    T, H = x.shape
    c = _ffn_config(_dtype_code(x, "x"), weights["gate"], activation)
    wp = _ffn_weights(weights, H, c.intermediate_size, x.dtype, x.device)
    xp, ldx = _rows(x, (T, H), x.dtype, "x")
    yp, ldy = _rows(y, (T, H), x.dtype, "y")
    _together(x.device, y, workspace, kept)
    with _on(x.device):
        _check(lib().moe_ffn_forward(ctypes.byref(c), T, xp, ldx, *wp, yp, ldy, _ptr(kept),
                                     0 if kept is None else kept.numel(), _ptr(workspace), workspace.numel(),
                                     _stream_of(x.device, stream)), "moe_ffn_forward")


def ffn_backward(x, weights: Dict[str, torch.Tensor], kept, dy, dx, grads: Dict[str, Optional[torch.Tensor]], workspace,
                 activation: str = "silu", stream=None) -> None:
    """The gradients of ffn for a gradient dy of y, from what that call kept
    (moe_ffn_backward).  dx may be None; grads {gate, up, down} as the weights, of which
    down, and gate together with up, may be None or absent."""
    T, H = x.shape
    c = _ffn_config(_dtype_code(x, "x"), weights["gate"], activation)
    I = c.intermediate_size
    wp = _ffn_weights(weights, H, I, x.dtype, x.device)
    xp, ldx = _rows(x, (T, H), x.dtype, "x")
    gp, ldg = _rows(dy, (T, H), x.dtype, "dy")
    dp, ldd = (None, 0) if dx is None else _rows(dx, (T, H), x.dtype, "dx")
    g = [grads.get(n) for n in ("gate", "up", "down")]
    for t, shape, n in zip(g, ((I, H), (I, H), (H, I)), ("gate", "up", "down")):
        _expect(t, shape, x.dtype, "gradient of " + n)
    if (g[0] is None) != (g[1] is None):
        raise ValueError("the gradients of gate and up are computed together")
    _together(x.device, kept, dy, dx, *g, workspace)
    with _on(x.device):
        _check(lib().moe_ffn_backward(ctypes.byref(c), T, xp, ldx, *wp, _ptr(kept), kept.numel(), gp, ldg, dp, ldd,
                                      *[_ptr(t) for t in g], _ptr(workspace), workspace.numel(),
                                      _stream_of(x.device, stream)), "moe_ffn_backward")


class GatedFFN:
    """The dense gated feed-forward block y = (act(x gate^T) * (x up^T)) down^T, with
    weights {gate [I, H], up [I, H], down [H, I]} as a shared expert has them.  Owns y and
    the workspace for up to `max_rows` rows and runs on the current stream; a call returns
    its rows of `y`, or `out` if that is given.

    With `training=True` a call also keeps what the backward pass of its rows needs, and
    `backward(x, dy)` returns {x, gate, up, down}, the gradients for the rows of the last
    call, in the weights' type and in buffers that the next backward overwrites.  The
    buffers serve one call (one forward and its backward) at a time: calls that overlap
    (other streams, graphs replayed side by side) need a GatedFFN each.  autograd does not
    see the calls; an input that requires gradients is warned of."""

    def __init__(self, weights: Dict[str, torch.Tensor], activation: str = "silu", max_rows: int = 1,
                 training: bool = False):
        _activation(activation)
        self.weights, self.activation, self.max_rows, self.training = weights, activation, max_rows, training
        self.I, self.H = weights["gate"].shape
        self.dtype = weights["gate"].dtype
        dtype = _BACK[_dtype_code(weights["gate"], "gate")]
        dev = weights["gate"].device
        _ffn_weights(weights, self.H, self.I, self.dtype, dev)
        rows = max(max_rows, 1)
        self.workspace = torch.empty(ffn_workspace_size(self.H, self.I, rows, dtype, training), dtype=torch.uint8, device=dev)
        self.y = torch.empty(max_rows, self.H, dtype=self.dtype, device=dev)
        self.kept = self.dx = self.grads = None
        self.rows = None                       # of the last call, whose kept tensors are there
        if training:
            self.kept = torch.empty(ffn_kept_size(self.H, self.I, rows, dtype), dtype=torch.uint8, device=dev)
            self.dx = torch.empty(max_rows, self.H, dtype=self.dtype, device=dev)
            self.grads = {n: torch.empty_like(weights[n]) for n in ("gate", "up", "down")}

    def __call__(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        T = x.shape[0]
        if T > self.max_rows:
            raise ValueError("more rows than the block was sized for")
        if x.dtype != self.dtype:
            raise ValueError(f"x: expected {self.dtype}, got {x.dtype}")
        if getattr(x, "requires_grad", False):
            _outside_autograd("GatedFFN", "`backward` of a block made with training=True gives the gradients")
        y = out if out is not None else self.y if T == self.max_rows else self.y[:T]
        self.rows = None
        ffn(x, self.weights, y, self.workspace, self.activation, self.kept, stream)
        self.rows = T
        return y

    def backward(self, x: torch.Tensor, dy: torch.Tensor, inputs: bool = True, weights: bool = True,
                 stream=None) -> Dict[str, torch.Tensor]:
        """The gradients for x, the rows of the last call, and dy.  `inputs=False` leaves
        out that of x, `weights=False` those of the weights."""
        if not self.training:
            raise ValueError("a backward pass needs a block made with training=True")
        T = x.shape[0]
        if T != self.rows:
            raise ValueError(f"a backward pass of {T} rows after a call of {self.rows}")
        dx = None if not inputs else self.dx if T == self.max_rows else self.dx[:T]
        grads = self.grads if weights else {}
        ffn_backward(x, self.weights, self.kept, dy, dx, grads, self.workspace, self.activation, stream)
        got = dict(grads)
        if inputs:
            got["x"] = dx
        return got


# ----------------------------------------------------------------------------- norms

NORMS = {"rms": 0, "layer": 1}
GATES = {"none": 0, "channel": 1, "token": 2, "full": 3}


class _NormConfig(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("hidden_size", "kind", "gate", "block_dtype", "stream_dtype", "out_dtype",
                                              "param_dtype")] + \
               [(n, ctypes.c_float) for n in ("eps", "residual_scale", "block_scale")]


_OUT_TYPES = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"], torch.int8: DTYPES["i8"]}


def _gate_kind(gate: Optional[torch.Tensor], T: int, H: int) -> int:
    """The kind of a gate by its shape: [H] or [1, H], [T, 1], or [T, H].  A gate that
    could be several (T = 1 or H = 1) is taken as the first of them."""
    if gate is None:
        return GATES["none"]
    shape = tuple(gate.shape)
    if shape in ((H,), (1, H)):
        return GATES["channel"]
    if shape == (T, 1):
        return GATES["token"]
    if shape == (T, H):
        return GATES["full"]
    raise ValueError(f"gate: expected [H], [1, H], [T, 1] or [T, H] with T = {T}, H = {H}, got {list(shape)}")


def _gate_rows(gate, kind: int, T: int, H: int, dtype):
    if gate is None:
        return None, 0
    if kind == GATES["full"]:
        return _rows(gate, (T, H), dtype, "gate")
    if gate.dtype != dtype:
        raise ValueError(f"gate: expected {dtype}, got {gate.dtype}")
    return _ptr(gate), 0


def _vector(t, H: int, dtype, name: str):
    if t is None:
        return None
    if t.shape != (H,) or t.dtype != dtype:
        raise ValueError(f"{name}: expected {(H,)} {dtype}, got {tuple(t.shape)} {t.dtype}")
    return _ptr(t)


def _norm_kind(kind: str) -> int:
    if kind not in NORMS:
        raise ValueError(f"kind: expected one of {sorted(NORMS)}, got {kind!r}")
    return NORMS[kind]


def _opt_rows(t, shape, dtype, name: str):
    return (None, 0) if t is None else _rows(t, shape, dtype, name)


def norm(y, residual, z, out, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, kind: str = "rms",
         eps: float = 1e-6, residual_scale: float = 1.0, block_scale: float = 1.0, out_scale=None, stream=None) -> None:
    """z = residual_scale residual + block_scale gate * post(y), out = norm(z) (moe_norm).
    y, residual, z and out [T, H] may be views with rows further apart than they are long;
    residual, and z or out, may be None.  residual and z share a dtype, weights, biases and
    gate another; out in torch.int8 takes codes, with a float32 out_scale [T]."""
    T, H = y.shape
    stream_t = (z if z is not None else residual if residual is not None else y).dtype
    c, pt = _norm_struct(T, H, _norm_kind(kind), gate, y.dtype, stream_t, None if out is None else out.dtype,
                         (weight, bias, post_weight, post_bias, gate), eps, residual_scale, block_scale)
    _norm_call(c, T, H, y, residual, z, out, out_scale, weight, bias, post_weight, post_bias, gate, stream_t, pt, stream)


def _norm_struct(T, H, kind, gate, block_t, stream_t, out_t, params, eps, a, b):
    pt = next((p.dtype for p in params if p is not None), stream_t)
    codes = []
    for t, name in ((block_t, "y"), (stream_t, "the residual stream"), (out_t or stream_t, "out"), (pt, "weights")):
        if t not in _OUT_TYPES or (t == torch.int8 and name != "out"):
            raise ValueError(f"{name}: {t} is not supported")
        codes.append(_OUT_TYPES[t])
    return _NormConfig(H, kind, _gate_kind(gate, T, H), *codes, eps, a, b), pt


def _norm_call(c, T, H, y, residual, z, out, out_scale, weight, bias, post_weight, post_bias, gate, stream_t, pt,
               stream) -> None:
    zp, ldz = _opt_rows(z, (T, H), stream_t, "z")
    op, ldo = _opt_rows(out, (T, H), out.dtype if out is not None else None, "out")
    _expect(out_scale, (T,), torch.float32, "out_scale")
    _together(y.device, z, out, out_scale)
    _norm_to(c, T, H, y, residual, (zp, ldz, op, ldo, _ptr(out_scale)), weight, bias, post_weight, post_bias, gate,
             stream_t, pt, stream)


def _norm_to(c, T, H, y, residual, outputs, weight, bias, post_weight, post_bias, gate, stream_t, pt, stream) -> None:
    """moe_norm with the addresses and strides of its outputs, whose device the caller has
    compared with y's; the others' is compared here."""
    shape, device = (T, H), y.device
    yp, ldy = _rows(y, shape, y.dtype, "y")
    rp, ldr = (None, 0) if residual is None else _rows(residual, shape, stream_t, "residual")
    gp, ldg = (None, 0) if gate is None else _gate_rows(gate, c.gate, T, H, pt)
    wp = bp = pp = qp = None
    if weight is not None:
        wp = _vector(weight, H, pt, "weight")
    if bias is not None:
        bp = _vector(bias, H, pt, "bias")
    if post_weight is not None:
        pp = _vector(post_weight, H, pt, "post_weight")
    if post_bias is not None:
        qp = _vector(post_bias, H, pt, "post_bias")
    _together(device, residual, gate, weight, bias, post_weight, post_bias)
    with _on(device):
        status = lib().moe_norm(ctypes.byref(c), T, yp, ldy, rp, ldr, gp, ldg, wp, bp, pp, qp, *outputs,
                                _stream_of(device, stream))
    if status:
        _check(status, "moe_norm")


def norm_backward_workspace_size(hidden_size: int, max_rows: int) -> int:
    c = _NormConfig(hidden_size, 0, 0, 0, 0, 0, 0, 1e-6, 1.0, 1.0)
    return _bytes_of("moe_norm_backward_workspace_size", ctypes.byref(c), int(max_rows))


def norm_backward(y, z, dz, dout, workspace, dy=None, dresidual=None, dgate=None, dweight=None, dbias=None,
                  dpost_weight=None, dpost_bias=None, weight=None, post_weight=None, post_bias=None, gate=None,
                  kind: str = "rms", eps: float = 1e-6, residual_scale: float = 1.0, block_scale: float = 1.0,
                  stream=None) -> None:
    """The gradients of norm from dz and dout, of which one may be None, for the z that it
    stored (moe_norm_backward).  Each result is written to the tensor that is given for
    it; dgate has the gate's shape."""
    T, H = y.shape
    stream_t = next(t for t in (z, dz, dresidual, dout) if t is not None).dtype
    c, pt = _norm_struct(T, H, _norm_kind(kind), gate, y.dtype, stream_t, None if dout is None else dout.dtype,
                         (weight, post_weight, post_bias, gate, dweight, dbias), eps, residual_scale, block_scale)
    shape = (T, H)
    yp, ldy = _rows(y, shape, y.dtype, "y")
    zp, ldz = _opt_rows(z, shape, stream_t, "z")
    zg, ldzg = _opt_rows(dz, shape, stream_t, "dz")
    og, ldog = _opt_rows(dout, shape, dout.dtype if dout is not None else None, "dout")
    yg, ldyg = _opt_rows(dy, shape, y.dtype, "dy")
    rg, ldrg = _opt_rows(dresidual, shape, stream_t, "dresidual")
    gp, ldg = _gate_rows(gate, c.gate, T, H, pt)
    if dgate is not None and (gate is None or dgate.shape != gate.shape):
        raise ValueError("dgate: expected the gate's shape")
    gg, ldgg = _gate_rows(dgate, c.gate, T, H, pt)
    _together(y.device, z, dz, dout, workspace, dy, dresidual, dgate, dweight, dbias, dpost_weight, dpost_bias, weight,
              post_weight, post_bias, gate)
    with _on(y.device):
        status = lib().moe_norm_backward(
            ctypes.byref(c), T, yp, ldy, zp, ldz, gp, ldg, _vector(weight, H, pt, "weight"),
            _vector(post_weight, H, pt, "post_weight"), _vector(post_bias, H, pt, "post_bias"), zg, ldzg, og, ldog, yg,
            ldyg, rg, ldrg, gg, ldgg, _vector(dweight, H, pt, "dweight"), _vector(dbias, H, pt, "dbias"),
            _vector(dpost_weight, H, pt, "dpost_weight"), _vector(dpost_bias, H, pt, "dpost_bias"), _ptr(workspace),
            workspace.numel(), _stream_of(y.device, stream))
    _check(status, "moe_norm_backward")


class ResidualNorm:
    """The norms after a block and before the next one:
        z = residual_scale residual + block_scale gate * post(y),  out = norm(z)
    with `weight` and `bias` for norm, `post_weight` and `post_bias` for post (no post norm
    without a post_weight).  Owns z and out for up to `max_rows` rows and runs on the
    current stream; a call returns its rows of both.  `stream_dtype` ("f32" / "bf16", by
    default the weight's) is that of the residual and z, `block_dtype` that of y, `out_dtype` that
    of out: "i8" gives (codes, scales) for LinearI8.  The gate is an argument of the call
    and multiplies by channel [H], token [T, 1] or element [T, H].

    With `training=True`, `backward` returns the gradients in buffers that the next
    backward overwrites.  The buffers serve one call at a time: calls that overlap (other
    streams, graphs replayed side by side) need a ResidualNorm each.  autograd does not see
    the calls; an input that requires gradients is warned of."""

    def __init__(self, hidden_size: int, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                 post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None, kind: str = "rms",
                 eps: float = 1e-6, residual_scale: float = 1.0, block_scale: float = 1.0,
                 block_dtype: Optional[str] = None, stream_dtype: Optional[str] = None, out_dtype: Optional[str] = None,
                 max_rows: int = 1, training: bool = False, device: str = "cuda"):
        if post_bias is not None and post_weight is None:
            raise ValueError("post_bias needs a post_weight")
        self.H, self.max_rows, self.training = hidden_size, max_rows, training
        self.weight, self.bias, self.post_weight, self.post_bias = weight, bias, post_weight, post_bias
        self.kind, self.eps, self.residual_scale, self.block_scale = kind, eps, residual_scale, block_scale
        types = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}
        params = [p for p in (weight, bias, post_weight, post_bias) if p is not None]
        default = params[0].dtype if params else torch.bfloat16
        self.stream_t = types[stream_dtype] if stream_dtype else default
        self.block_t = types[block_dtype] if block_dtype else self.stream_t
        self.out_t = types[out_dtype] if out_dtype else self.stream_t
        self.param_t = params[0].dtype if params else self.stream_t
        self._c, _ = _norm_struct(max_rows, hidden_size, _norm_kind(kind), None, self.block_t, self.stream_t, self.out_t,
                                  params, eps, residual_scale, block_scale)
        self._set = self._mine = None
        dev = params[0].device if params else torch.device(device)
        self.z = torch.empty(max_rows, hidden_size, dtype=self.stream_t, device=dev)
        self.out = torch.empty(max_rows, hidden_size, dtype=self.out_t, device=dev)
        self.out_scale = torch.empty(max_rows, dtype=torch.float32, device=dev) if self.out_t == torch.int8 else None
        if training:
            if self.out_t == torch.int8:
                raise ValueError("there is no backward pass through 8-bit codes")
            self.workspace = torch.empty(norm_backward_workspace_size(hidden_size, max(max_rows, 1)), dtype=torch.uint8,
                                         device=dev)
            self.dy = torch.empty(max_rows, hidden_size, dtype=self.block_t, device=dev)
            self.dresidual = torch.empty_like(self.z)
            self.grads = {n: torch.empty_like(p) for n, p in (("weight", weight), ("bias", bias),
                                                              ("post_weight", post_weight), ("post_bias", post_bias))
                          if p is not None}
            self.dgate = {}                    # by the buffer's shape and type

    def _here(self, t: torch.Tensor, T: int) -> torch.Tensor:
        return t if T == self.max_rows else t[:T]

    def _config(self, T: int, gate) -> _NormConfig:
        now = (self.kind, self.eps, self.residual_scale, self.block_scale, 0 if gate is None else _gate_kind(gate, T, self.H))
        c = self._c
        if now != self._set:
            c.kind, c.eps, c.residual_scale, c.block_scale, c.gate = _norm_kind(self.kind), *now[1:]
            self._set = now
        return c

    def __call__(self, y: torch.Tensor, residual: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                 stream=None):
        T = y.shape[0]
        if T > self.max_rows:
            raise ValueError("more rows than the norm was sized for")
        if y.dtype != self.block_t:
            raise ValueError(f"y: expected {self.block_t}, got {y.dtype}")
        if getattr(y, "requires_grad", False) or getattr(residual, "requires_grad", False):
            _outside_autograd("ResidualNorm", "`backward` of a norm made with training=True gives the gradients")
        c = self._config(T, gate)
        # The rows of the norm's own buffers, and their addresses, of the last call's length.
        mine = self._mine
        if mine is None or mine[0] != T or mine[1] is not self.z or mine[2] is not self.out or mine[3] is not self.out_scale:
            z, out = self._here(self.z, T), self._here(self.out, T)
            scale = None if self.out_scale is None else self._here(self.out_scale, T)
            _together(z.device, out, scale)
            outputs = (*_rows(z, (T, self.H), self.stream_t, "z"), *_rows(out, (T, self.H), self.out_t, "out"), _ptr(scale))
            mine = self._mine = (T, self.z, self.out, self.out_scale, (z, out if scale is None else (out, scale)), outputs)
        if mine[1].device != y.device:
            _together(y.device, mine[1])
        _norm_to(c, T, self.H, y, residual, mine[5], self.weight, self.bias, self.post_weight,
                 self.post_bias, gate, self.stream_t, self.param_t, stream)
        return mine[4]

    def backward(self, y: torch.Tensor, z: torch.Tensor, dz: Optional[torch.Tensor], dout: Optional[torch.Tensor],
                 gate: Optional[torch.Tensor] = None, has_residual: bool = True, stream=None) -> Dict[str, torch.Tensor]:
        """{y, residual, gate, weight, bias, post_weight, post_bias}, of these what there
        is, from the gradients of z and out (either may be None: then what hangs on it
        alone is left out).  y, gate and z are those of the call."""
        if not self.training:
            raise ValueError("a backward pass needs a norm made with training=True")
        T = y.shape[0]
        if T > self.max_rows:
            raise ValueError("more rows than the norm was sized for")
        if y.dtype != self.block_t:
            raise ValueError(f"y: expected {self.block_t}, got {y.dtype}")
        got = {"y": self._here(self.dy, T)}
        if has_residual:
            got["residual"] = self._here(self.dresidual, T)
        if gate is not None:
            # A buffer for each shape and type of gate, kept from its first call on: captured
            # graphs hold its address.
            rows = gate.shape[0] if _gate_kind(gate, T, self.H) == GATES["channel"] else self.max_rows
            shape = (rows, *gate.shape[1:])
            buf = self.dgate.get((shape, gate.dtype))
            if buf is None:
                buf = self.dgate[shape, gate.dtype] = torch.empty(*shape, dtype=gate.dtype, device=self.z.device)
            got["gate"] = buf if buf.shape[0] == gate.shape[0] else buf[:gate.shape[0]]
        for n in ("weight", "bias") if dout is not None else ():
            if n in self.grads:
                got[n] = self.grads[n]
        for n in ("post_weight", "post_bias"):
            if n in self.grads:
                got[n] = self.grads[n]
        if dout is not None and dout.dtype != self.out_t:
            raise ValueError(f"dout: expected {self.out_t}, got {dout.dtype}")
        norm_backward(y, z, dz, dout, self.workspace, got["y"], got.get("residual"), got.get("gate"), got.get("weight"),
                      got.get("bias"), got.get("post_weight"), got.get("post_bias"), self.weight, self.post_weight,
                      self.post_bias, gate, self.kind, self.eps, self.residual_scale, self.block_scale, stream)
        return got


# ----------------------------------------------------------------------------- 8-bit products

class _LinearI8Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("in_features", "out_features", "in_dtype", "bias_dtype", "out_dtype",
                                              "activation")]


def quantize_i8(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, stream=None):
    """(codes, scale) of the rows of x [M, K], a batch's or a weight's (moe_quant_i8):
    scale = max(amax / 127, 2^-126), codes = x / scale rounded, ties to even."""
    M, K = x.shape
    xp, ldx = _rows(x, (M, K), x.dtype, "x")
    if codes is None:
        codes = torch.empty(M, K, dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=x.device)
    cp, ldc = _rows(codes, (M, K), torch.int8, "codes")
    _expect(scale, (M,), torch.float32, "scale")
    _together(x.device, codes, scale)
    with _on(x.device):
        _check(lib().moe_quant_i8(_dtype_code(x, "x"), M, K, xp, ldx, cp, ldc, _ptr(scale), _stream_of(x.device, stream)),
               "moe_quant_i8")
    return codes, scale


def linear_i8_workspace_size(in_features: int, out_features: int, max_rows: int, in_dtype: str = "bf16") -> int:
    c = _LinearI8Config(in_features, out_features, DTYPES[in_dtype], 0, 0, 0)
    return _bytes_of("moe_linear_i8_workspace_size", ctypes.byref(c), int(max_rows))


def linear_i8(x, weight, weight_scale, bias, residual, y, workspace, activation: str = "none", x_scale=None,
              stream=None) -> None:
    """y = activation(x_scale weight_scale (x weight^T) + bias) + residual (moe_linear_i8).
    x [M, K] holds codes (torch.int8, with x_scale [M]) or float32 or bfloat16 values, which are
    quantised row by row; weight [N, K] holds codes; residual and y [M, N] share a dtype."""
    (M, K), N = x.shape, weight.shape[0]
    if (x.dtype == torch.int8) != (x_scale is not None):
        raise ValueError("x_scale goes with codes, and codes with an x_scale")
    if x.dtype not in _OUT_TYPES:
        raise ValueError(f"x: {x.dtype} is not supported")
    c = _LinearI8Config(K, N, _OUT_TYPES[x.dtype], DTYPES["f32"] if bias is None else _dtype_code(bias, "bias"),
                        _dtype_code(y, "y"), _activation(activation))
    _linear_i8_call(c, M, N, K, x, x_scale, weight, weight_scale, bias, residual, y, workspace, stream)


def _linear_i8_call(c, M, N, K, x, x_scale, weight, weight_scale, bias, residual, y, workspace, stream) -> None:
    xp, ldx = _rows(x, (M, K), x.dtype, "x")
    wp, ldw = _rows(weight, (N, K), torch.int8, "weight")
    rp, ldr = _opt_rows(residual, (M, N), y.dtype, "residual")
    yp, ldy = _rows(y, (M, N), y.dtype, "y")
    _expect(x_scale, (M,), torch.float32, "x_scale")
    sp = _vector(weight_scale, N, torch.float32, "weight_scale")
    bp = None if bias is None else _vector(bias, N, bias.dtype, "bias")
    _together(x.device, x_scale, weight, weight_scale, bias, residual, y, workspace)
    with _on(x.device):
        status = lib().moe_linear_i8(ctypes.byref(c), M, xp, ldx, _ptr(x_scale), wp, ldw, sp, bp, rp, ldr, yp, ldy,
                                     _ptr(workspace), workspace.numel(), _stream_of(x.device, stream))
    _check(status, "moe_linear_i8")


class LinearI8:
    """A projection in 8-bit integers, y = activation(sx sw (q weight^T) + bias) + residual:
    `weight` [N, K] holds codes with a scale for each row (quantize_i8 of a weight gives
    both), x is quantised row by row, or comes as (codes, scales), as a ResidualNorm with
    out_dtype="i8" gives them.  Owns the output and the workspace for up to `max_rows`
    rows and runs on the current stream; `out_dtype` ("f32" / "bf16") is that of y and of
    the residual.  A call returns its rows of `y`, or `out` if that is given.  The
    workspace serves one call at a time: calls that overlap (other streams, graphs
    replayed side by side) need a LinearI8 each."""

    def __init__(self, weight: torch.Tensor, weight_scale: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 activation: str = "none", out_dtype: str = "bf16", max_rows: int = 1):
        self.weight, self.weight_scale, self.bias = weight, weight_scale, bias
        self.activation, self.max_rows = activation, max_rows
        self.N, self.K = weight.shape
        _expect(weight, (self.N, self.K), torch.int8, "weight")
        _expect(weight_scale, (self.N,), torch.float32, "weight_scale")
        self.out_t = {"f32": torch.float32, "bf16": torch.bfloat16}[out_dtype]
        dev = weight.device
        self.workspace = torch.empty(linear_i8_workspace_size(self.K, self.N, max(max_rows, 1)), dtype=torch.uint8, device=dev)
        self.y = torch.empty(max_rows, self.N, dtype=self.out_t, device=dev)
        self._c = _LinearI8Config(self.K, self.N, 0, DTYPES["f32"] if bias is None else _dtype_code(bias, "bias"),
                                  DTYPES[out_dtype], _activation(activation))

    def __call__(self, x, residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
        x, scale = x if isinstance(x, tuple) else (x, None)
        M = x.shape[0]
        if M > self.max_rows:
            raise ValueError("more rows than the projection was sized for")
        if (x.dtype == torch.int8) != (scale is not None) or x.dtype not in _OUT_TYPES:
            raise ValueError(f"x: expected float32, bfloat16 or (int8 codes, scales), got {x.dtype}")
        if getattr(x, "requires_grad", False):
            _outside_autograd("LinearI8", "there is no backward pass through 8-bit codes")
        y = out if out is not None else self.y if M == self.max_rows else self.y[:M]
        if y.dtype != self.out_t:
            raise ValueError(f"out: expected {self.out_t}, got {y.dtype}")
        c = self._c
        c.in_dtype, c.activation = _OUT_TYPES[x.dtype], _activation(self.activation)
        if self.bias is not None:
            c.bias_dtype = _dtype_code(self.bias, "bias")
        _linear_i8_call(c, M, self.N, self.K, x, scale, self.weight, self.weight_scale, self.bias, residual, y,
                        self.workspace, stream)
        return y
