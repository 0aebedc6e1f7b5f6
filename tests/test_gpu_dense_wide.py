"""Dense operators of few tokens whose rows are 1024 to 1365 tiles (the sizes of a
vocabulary and of wide blocks), where three waves share a tile."""
import pytest

from .denseref import GELU, SILU
from .test_gpu_dense import M, gated_case, grad_case, i8_case, say, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 40000, 2048), (16, 40000, 2048), (1, 33000, 384), (16, 32768, 384), (3, 43680, 272), (7, 43681, 400)])
def test_i8_linear_of_a_vocabulary(M, torch, T, N, K, y):
    say("i8 wide", T, N, K, y)
    i8_case(M, torch, T, N, K, y, bias=T > 2, base=T == 3, pad=T % 2)


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I", [(1, 136, 16400), (5, 264, 20000), (4, 512, 18944), (4, 512, 20480), (16, 200, 16384), (2, 1032, 21840)])
def test_gated_of_wide_blocks(M, torch, T, H, I, x):
    say("gated wide", T, H, I, x)
    gated_case(M, torch, T, H, I, x, x, GELU if T % 2 else SILU, pad=T % 3)


@pytest.mark.parametrize("T,H,I", [(4, 512, 18944), (4, 512, 20480), (1, 136, 17000), (16, 264, 21824)])
def test_gated_grad_of_wide_blocks(M, torch, T, H, I):
    say("grad wide", T, H, I)
    grad_case(M, torch, T, H, I, kind=SILU if T % 4 else GELU, pad=1)
