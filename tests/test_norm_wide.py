"""The norms at their widest rows, 8193 to 16384 elements, of more rows than a backward pass has
groups.  Against float64 as in test_norm.py, whose tolerances these are."""
import pytest

from tests import test_norm as N


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(300, 8193), (700, 12288), (521, 16384), (600, 16377)])
@pytest.mark.parametrize("kind,types,gate,post,bias", [
    ("rms", ("bf16", "bf16", "bf16", "bf16"), "channel", True, False), ("rms", ("bf16", "f32", "bf16", "bf16"), "none", False, False),
    ("rms", ("f32", "f32", "f32", "f32"), "token", True, False), ("layer", ("f32", "f32", "f32", "f32"), "channel", True, True),
    ("layer", ("bf16", "bf16", "f32", "bf16"), "full", True, True)])
def test_wide_rows(T, H, kind, types, gate, post, bias):
    N._run(T, H, kind, *types, gate=gate, post=post, bias=bias, seed=T + H, pad=3)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(300, 8193), (521, 16384)])
def test_wide_rows_to_codes(T, H):
    N._run(T, H, "rms", out="i8", post=True, seed=T)
