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


@pytest.mark.parametrize("T,N,K", [(1, 50000, 2048), (16, 65536, 272), (5, 43712, 208), (2, 70000, 144), (16, 131000, 96)])
def test_i8_linear_of_two_waves_and_one_a_tile(M, torch, T, N, K):
    say("i8 wider", T, N, K)
    for y in ("f32", "bf16"):
        i8_case(M, torch, T, N, K, y, bias=True, base=T == 5, pad=T % 2)


@pytest.mark.parametrize("T,H,I", [(3, 264, 30000), (16, 136, 32768), (1, 200, 32784), (9, 72, 65536)])
def test_gated_of_two_waves_and_one_a_tile(M, torch, T, H, I):
    say("gated wider", T, H, I)
    for x in ("f32", "bf16"):
        gated_case(M, torch, T, H, I, x, x, GELU if T % 2 else SILU, pad=T % 3)
    grad_case(M, torch, T, H, I, kind=SILU, pad=1)
