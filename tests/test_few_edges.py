"""moe_layer_few at the ends of its weight formats."""
import pytest
import torch

import mixture_experts_layer_05_amd as moe
import workloads as W
from oracle import moe as O
from tests import harness as Hn

# As for the layer's other sizes: exact products, float32 sums.
Y_TOL = 2.0 ** -16


def _mx_layer(T, names, codes, nibbles=None):
    """One expert's layer whose matrices `names` take their scale codes from `codes` in
    turn; their elements are drawn from `nibbles` (any E2M1 code if None)."""
    shape = W.LayerShape("mx_codes", 256, 1, 256, 1, 0, W.DT_MXFP4, "bf16")
    case = Hn.make_case(shape, T, 111, condition=False)
    g = torch.Generator().manual_seed(112)
    for n in names:
        s = case.weights[n + "_s"]
        s.copy_(torch.tensor(codes, dtype=torch.uint8)[torch.randint(len(codes), s.shape, generator=g)])
        if nibbles is not None:
            d = torch.tensor(nibbles, dtype=torch.uint8)
            pick = lambda: d[torch.randint(len(nibbles), case.weights[n].shape, generator=g)]  # noqa: E731
            case.weights[n].copy_(pick() | pick() << 4)
    case.inp.x = (torch.randint(-8, 9, (T, 256), generator=g).float()).bfloat16()
    layer = moe.MoELayer(Hn.config(shape), case.weights, case.inp.w_router.cuda(), max_tokens=T, few=True)
    return case, layer


def _check(case, layer):
    y = layer(case.inp.x.cuda())
    torch.cuda.synchronize()
    s = case.shape
    r = O.route(case.inp.x, case.inp.w_router, None, None, 1, True, 0, 0.0)
    ref = O.moe_combine(case.inp.x, r["ids"], r["w"], None, case.expert_cpu, None, s.weight_dtype, None,
                        ["plain"])["plain"]
    err = Hn.token_rel_l2(y.cpu().double().numpy(), ref)
    print(f"[case] worst token {err.max():.2e}", flush=True)
    assert err.max() <= Y_TOL


# E2M1 codes of 0, 0.5, 1, 1.5 and their negatives.
SMALL = [0, 1, 2, 3, 8, 9, 10, 11]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16])
def test_mxfp4_smallest_scale_codes(T):
    """Codes 0 to 2 (2^-127 to 2^-125): x or h is large and brings the products back."""
    print(f"\n[case] smallest codes T={T}", flush=True)
    case, layer = _mx_layer(T, ("gate", "up"), [0, 1, 2])
    case.inp.x *= 2.0 ** 116
    _check(case, layer)
    case, layer = _mx_layer(T, ("down",), [0, 1, 2])
    case.inp.x *= 2.0 ** 30                                # h of about 2^60
    _check(case, layer)


@pytest.mark.gpu
@pytest.mark.parametrize("codes,nibbles", [([250, 252], None), ([253], [0, 1, 2, 3, 4, 5, 10, 12, 13]), ([254], SMALL)])
def test_mxfp4_largest_scale_codes(codes, nibbles):
    """Codes up to 254 (2^127), for elements whose weight stays below 2^128."""
    print(f"\n[case] largest codes {codes}", flush=True)
    case, layer = _mx_layer(5, ("gate", "up"), codes, nibbles)
    case.inp.x *= 2.0 ** -126                              # gate and up sums of about 2^8
    _check(case, layer)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["gate", "up", "down"])
def test_mxfp4_scale_code_255_is_nan(name):
    print(f"\n[case] code 255 in {name}", flush=True)
    case, layer = _mx_layer(3, (), [])
    if name == "down":
        case.weights["down_s"][0, 7, 3] = 255               # a block of row 7
    else:
        case.weights[name + "_s"][0, 9, 5] = 255            # one element of h
    y = layer(case.inp.x.cuda())
    torch.cuda.synchronize()
    if name == "down":
        assert torch.isnan(y[:, 7]).all()
        rest = torch.arange(256) != 7
        assert torch.isfinite(y[:, rest]).all()
    else:
        assert torch.isnan(y).all()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["gate", "down"])
@pytest.mark.parametrize("code,nibble", [(253, 6), (253, 7), (254, 4), (254, 15)])
def test_mxfp4_weights_of_2_to_128_are_infinite(code, nibble, name):
    """As the header states: an element times its scale at 2^128 or more is no bf16."""
    print(f"\n[case] code {code} element {nibble} in {name}", flush=True)
    case, layer = _mx_layer(2, (), [])
    case.weights[name + "_s"][0, 9, 5] = code
    case.weights[name][0, 9, 5 * 16:6 * 16] = nibble | nibble << 4
    case.inp.x = torch.full((2, 256), 2.0 ** -100).bfloat16()
    y = layer(case.inp.x.cuda())
    torch.cuda.synchronize()
    if name == "down":
        assert not torch.isfinite(y[:, 9]).any() and torch.isfinite(y[:, torch.arange(256) != 9]).all()
    else:
        assert not torch.isfinite(y).any()
