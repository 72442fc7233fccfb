"""Binding of the operators around the MoE layer beside `Linear`: the dense gated FFN
with its backward pass, the norms before and after a block, and products in 8-bit
integers.  As in the rest of the binding every step runs in the HIP kernels behind the C
ABI of include/moe_mi355x.h, on the current stream, and nothing falls back."""
from __future__ import annotations

import ctypes
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
    (other streams, graphs replayed side by side) need a GatedFFN each."""

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
