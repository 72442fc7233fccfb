"""The binding refuses tensors of a call, and streams, on different GPUs before it calls the
library.  Stand-ins for tensors: no GPU is needed, none is asked."""
import types

import pytest
import torch

import mixture_experts_layer_05_amd as moe

HERE, THERE = torch.device("cuda:0"), torch.device("cuda:1")


class _Tensor:
    """A contiguous tensor on a GPU, as far as the binding looks at it."""

    def __init__(self, shape, dtype, device=HERE):
        self.shape, self.dtype, self.device, self.is_cuda = tuple(shape), dtype, device, True

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000

    def numel(self):
        return 1 << 40

    def stride(self):
        return self.shape[1], 1

    def __getitem__(self, rows):
        return _Tensor((rows.stop,) + self.shape[1:], self.dtype, self.device)


@pytest.fixture
def calls(monkeypatch):
    """The library calls that get past the checks (none is made)."""
    seen = []

    def record(name):
        return lambda *a: seen.append(name) or 0

    fake = types.SimpleNamespace(moe_layer_few=record("layer_few"), moe_linear=record("linear"))
    real = moe.lib()
    for name in ("moe_layer_few_workspace_size", "moe_linear_workspace_size", "moe_workspace_size"):
        setattr(fake, name, getattr(real, name))
    monkeypatch.setattr(moe, "lib", lambda: fake)
    monkeypatch.setattr(moe, "_on", lambda device: moe._HERE_CTX)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    return seen


CFG = moe.MoEConfig(256, 4, 128, 2, 128, "fp8_e4m3_g128", "bf16")
U8, F32, BF16, I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


def _experts(lead):
    H, I = 256, 128
    out = {}
    for n, r, c in (("gate", I, H), ("up", I, H), ("down", H, I)):
        out[n], out[n + "_s"] = _Tensor(lead + (r, c), U8), _Tensor(lead + (r, c // 128), F32)
    return out


def _layer(monkeypatch, weights, shared, router, gate):
    def empty(*shape, dtype, device):
        return _Tensor(shape, dtype, HERE)

    monkeypatch.setattr(moe.torch, "empty", empty)
    layer = moe.MoELayer(CFG, weights, router, gate, shared, max_tokens=4, few=True)
    monkeypatch.undo()
    return layer


X = _Tensor((2, 256), BF16)


def _parts():
    return dict(weights=_experts((4,)), shared=_experts(()), router=_Tensor((4, 256), BF16), gate=_Tensor((256,), BF16))


def _one_there(p, where):
    """One tensor of the layer's moved to the other GPU."""
    group, _, name = where.partition(".")
    t = p[group][name] if name else p[group]
    t.device = THERE


PLACES = (["router", "gate"] + [f"weights.{n}{s}" for n in ("gate", "up", "down") for s in ("", "_s")]
          + [f"shared.{n}{s}" for n in ("gate", "up", "down") for s in ("", "_s")])


def _few(p, x=X, stream=None, **kw):
    a = dict(y=_Tensor((2, 256), F32), workspace=_Tensor((1 << 20,), U8))
    a.update(kw)
    moe.layer_few(CFG, x, p["router"], p["gate"], a.pop("bias", None), moe.expert_weights_struct(CFG, p["weights"], p["shared"]),
                  a.pop("y"), a.pop("workspace"), stream=stream, **a)


def test_layer_few_takes_tensors_of_one_gpu(calls):
    _few(_parts())
    p = _parts()
    for group in ("weights", "shared"):
        for t in p[group].values():
            t.device = THERE
    p["router"].device = p["gate"].device = THERE
    _few(p, _Tensor((2, 256), BF16, THERE), y=_Tensor((2, 256), F32, THERE), workspace=_Tensor((1 << 20,), U8, THERE))
    assert calls == ["layer_few"] * 2


@pytest.mark.parametrize("where", PLACES)
def test_layer_few_refuses_a_tensor_elsewhere(where, calls):
    p = _parts()
    _one_there(p, where)
    with pytest.raises(ValueError, match="one GPU"):
        _few(p)
    assert not calls


@pytest.mark.parametrize("name,shape,dtype", [
    ("y", (2, 256), F32), ("workspace", (1 << 20,), U8), ("y_act", (2, 256), BF16), ("topk_ids", (2, 2), I32),
    ("topk_weights", (2, 2), F32), ("shared_gate", (2,), F32), ("route_stats", (4,), I32), ("bias", (2, 4), F32)])
def test_layer_few_refuses_outputs_elsewhere(name, shape, dtype, calls):
    with pytest.raises(ValueError, match="one GPU"):
        _few(_parts(), **{name: _Tensor(shape, dtype, THERE)})
    assert not calls


@pytest.mark.parametrize("where", PLACES)
def test_layer_refuses_a_tensor_elsewhere(where, calls, monkeypatch):
    p = _parts()
    _one_there(p, where)
    with monkeypatch.context() as m:
        layer = _layer(m, **p)
    with pytest.raises(ValueError, match="one GPU"):
        layer(X)
    assert not calls


@pytest.mark.parametrize("name", ["y", "topk_ids", "topk_weights", "shared_gate", "few_workspace"])
def test_layer_refuses_buffers_elsewhere(name, calls, monkeypatch):
    """As made: the layer's own buffers on the current GPU, the weights and x on another;
    as changed later: one buffer."""
    p = _parts()
    with monkeypatch.context() as m:
        layer = _layer(m, **p)
    layer(X)
    assert calls == ["layer_few"]
    t = getattr(layer, name)
    setattr(layer, name, _Tensor(t.shape, t.dtype, THERE))
    with pytest.raises(ValueError, match="one GPU"):
        layer(X)
    setattr(layer, name, t)
    layer(X)
    for group in ("weights", "shared"):
        for v in p[group].values():
            v.device = THERE
    layer.weights = moe.expert_weights_struct(CFG, p["weights"], p["shared"])
    layer.w_router, layer.w_shared_gate = _Tensor((4, 256), BF16, THERE), _Tensor((256,), BF16, THERE)
    with pytest.raises(ValueError, match="one GPU"):
        layer(_Tensor((2, 256), BF16, THERE))
    assert calls == ["layer_few"] * 2


def _linear(weight_there=False):
    p = moe.Linear.__new__(moe.Linear)
    p.weight, p.bias, p.activation, p.max_rows = _Tensor((64, 256), BF16), None, "none", 4
    p.N, p.K, p.in_dtype, p.out_dtype = 64, 256, BF16, BF16
    p.workspace, p.y = _Tensor((1 << 20,), U8), _Tensor((4, 64), BF16)
    p._cfg = moe._LinearConfig(256, 64, 1, 1, 0)
    return p


def test_linear_refuses_tensors_elsewhere(calls):
    p = _linear()
    p(X)
    with pytest.raises(ValueError, match="one GPU"):
        p(_Tensor((2, 256), BF16, THERE))
    with pytest.raises(ValueError, match="one GPU"):
        p(X, out=_Tensor((2, 64), BF16, THERE))
    p.weight = _Tensor((64, 256), BF16, THERE)
    with pytest.raises(ValueError, match="one GPU"):
        p(X)
    # All but the workspace on the other GPU.
    with pytest.raises(ValueError, match="one GPU"):
        p(_Tensor((2, 256), BF16, THERE), out=_Tensor((2, 64), BF16, THERE))
    assert calls == ["linear"]


def test_streams_of_another_gpu_are_refused(calls):
    there = types.SimpleNamespace(device=THERE, cuda_stream=0x10)
    here = types.SimpleNamespace(device=HERE, cuda_stream=0x10)
    with pytest.raises(ValueError, match="stream"):
        _few(_parts(), stream=there)
    with pytest.raises(ValueError, match="stream"):
        _linear()(X, stream=there)
    _few(_parts(), stream=here)
    _linear()(X, stream=here)
    _linear()(X, stream=0x10)                              # a bare handle says nothing
    assert calls == ["layer_few", "linear", "linear"]
