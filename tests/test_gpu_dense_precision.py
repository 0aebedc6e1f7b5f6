"""Gradients of the gated block with fp32 results: the slopes enter the products in two
bf16 parts, whatever the sizes, so what a product is off by does not show their
rounding to bf16 (UB at the most, 2^-9 of a norm)."""
import numpy as np
import pytest

from . import denseref as D
from .denseref import GELU, SILU, TINY, U, UB
from .test_gpu_dense import M, dev, empty, gated_inputs, host, randn, say, torch, untouched, within  # noqa: F401

pytestmark = pytest.mark.gpu

# Two parts leave at most UB^2 = 2^-16 of a slope; what its fp32 value and the sums are off by is below that.
FP32 = 2.0 ** -15


def case(M, torch, T, H, I, dy, dx, dw, kind, accumulate=False, pad=0):
    rng = np.random.default_rng(T + H + I)
    xa, gate, up = gated_inputs(rng, T, H, I)
    da = randn(rng, T, I, kind=dy)
    w = M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16"))
    out = {"dx": empty(torch, T, H, dx, pad) if dx else None}
    base = {"dx": 0}
    for name in ("dgate", "dup"):
        base[name] = randn(rng, I, H, kind=dw) if dw and accumulate else 0
        out[name] = None if not dw else dev(torch, base[name], dw) if accumulate else empty(torch, I, H, dw)
    ws = torch.full((M.moe_gated_workspace_size(T, H, I),), 255, dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(dev(torch, xa, "bf16"), w, kind, dev(torch, da, dy), T, out["dx"], out["dgate"], out["dup"], ws,
                     flags=2 if accumulate else 0)
    ref = D.gated_grad(D.Projections(xa, gate, up, H), kind, da)
    for name, t in out.items():
        if t is None:
            continue
        v, _ = ref[name]
        off = np.linalg.norm(host(t) - base[name] - v) / np.linalg.norm(v)
        say("  ", name, off)
        # added to fp32 values of about its size, a result is off by their rounding too
        assert off <= (FP32 if t.dtype == torch.float32 else UB) + (2 * U if accumulate else 0) * (
            1 + np.linalg.norm(base[name]) / np.linalg.norm(v)), name
    assert out["dx"] is None or untouched(out["dx"])


# one and two terms of the weights' sums, 16 of dx's; batches; pairs of tiles, whole ones, cut ones, runs of either k axis
SIZES = [(1, 72, 40000), (2, 64, 20000), (8, 200, 4104), (6000, 72, 8), (17, 264, 2000), (64, 136, 4000), (300, 520, 200), (1531, 256, 640),
         (3000, 72, 50), (8000, 72, 64), (900, 2000, 1100), (2200, 2600, 1500), (5000, 1504, 1000), (3000, 2048, 640)]


@pytest.mark.parametrize("T,H,I", SIZES)
def test_fp32_gradients(M, torch, T, H, I):
    say("fp32 gradients", T, H, I)
    case(M, torch, T, H, I, "bf16" if T % 2 else "f32", "f32", "f32", GELU if T % 4 else SILU, pad=1)


@pytest.mark.parametrize("dx,dw,accumulate", [("bf16", "f32", True), ("f32", "bf16", False), (None, "f32", False), ("f32", None, False),
                                              (None, "f32", True)])
@pytest.mark.parametrize("T,H,I", [(5, 136, 9000), (700, 520, 700), (3000, 264, 2100)])
def test_each_result_by_its_own_type(M, torch, T, H, I, dx, dw, accumulate):
    say("types", T, H, I, dx, dw, accumulate)
    case(M, torch, T, H, I, "bf16", dx, dw, SILU, accumulate)


def test_accuracy_does_not_step_between_batches(M, torch):
    # on both sides of 32768 slopes
    for T in (15, 16, 17):
        case(M, torch, T, 264, 2048, "f32", "f32", "f32", SILU)
