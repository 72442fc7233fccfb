"""moe_layer_few's limits: offsets within x, a matrix, the router and h are 32 bits.  A
layer past one of them is refused where its workspace is asked for, and by the call."""
import ctypes

import pytest

import mixture_experts_layer_05_amd as moe

OK, UNSUPPORTED = 0, -4
FAKE = 0x1000


def _size(T, H, E, I, K, S, dtype):
    c = moe.MoEConfig(H, E, I, K, S, dtype, "f32" if dtype == "f32" else "bf16").c()
    n = ctypes.c_size_t(0)
    st = moe.lib().moe_layer_few_workspace_size(ctypes.byref(c), T, ctypes.byref(n))
    if st != OK:                                        # the call refuses it too, before any launch
        ew = moe._Weights(*[FAKE] * 12)
        assert moe.lib().moe_layer_few(ctypes.byref(c), T, FAKE, FAKE, FAKE, None, ctypes.byref(ew), None, None, None,
                                       None, FAKE, None, FAKE, 1 << 62, None) == st
    return st


@pytest.mark.parametrize("T,H", [(16, 1 << 26), (16, 71582789), (9, 1 << 27), (13, (1 << 30) // 13 + 1), (2, 1 << 29)])
def test_x_of_4_gib_is_refused(T, H):
    assert _size(T, H, 1, 1, 1, 0, "f32") == UNSUPPORTED
    assert _size(((1 << 30) - 1) // H, H, 1, 1, 1, 0, "f32") == OK      # the most tokens that fit
    assert _size(T, ((1 << 30) - 1) // T, 1, 1, 1, 0, "f32") == OK      # the widest rows that fit


@pytest.mark.parametrize("H,E,I,K,S,dtype", [
    (1 << 15, 1, 1 << 15, 1, 0, "f32"),                  # a routed matrix of 4 GiB
    (1 << 15, 1, 1 << 16, 1, 0, "bf16"),
    (1 << 15, 1, 1, 1, 1 << 15, "f32"),                  # a shared one
    (1 << 15, 1, 128, 1, 1 << 16, "bf16"),
    (1 << 23, 256, 128, 1, 0, "bf16"),                   # the router
    (1, 1, 1 << 22, 1, 0, "f32"),                        # h
    (128, 1, 1 << 23, 1, 0, "bf16"),
])
def test_matrices_and_h_of_4_gib_are_refused(H, E, I, K, S, dtype):
    assert _size(16, H, E, I, K, S, dtype) == UNSUPPORTED


def test_sizes_below_the_limits_are_taken():
    assert _size(16, 1 << 15, 1, (1 << 15) - 1, 1, 0, "f32") == OK
    assert _size(16, 1 << 15, 1, (1 << 16) - 128, 1, 0, "bf16") == OK
    assert _size(16, (1 << 23) - 128, 256, 128, 1, 0, "bf16") == OK
    assert _size(16, 1, 1, (1 << 22) - 1, 1, 0, "f32") == OK
