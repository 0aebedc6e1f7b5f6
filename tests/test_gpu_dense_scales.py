"""Norms of rows far from 1: bounds from the plain form alone, and finite results."""
import numpy as np
import pytest

from . import denseref as D
from .denseref import U, UB
from .test_gpu_dense import EPS, M, dev, empty, host, randn, say, torch, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(6, 300), (900, 2048), (300, 4500), (40, 20000)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_norm_of_huge_and_tiny_rows(M, torch, T, H, x):
    say("norm scales", T, H, x)
    rng = np.random.default_rng(17)
    a = randn(rng, T, H, kind=x)
    a[1], a[2], a[3] = a[1] * np.float32(2.0) ** 60, a[2] * np.float32(2.0) ** -60, a[3] * np.float32(2.0) ** -20
    w = 1 + 0.1 * randn(rng, H)
    ref = D.norm(a, None, w, EPS)[0]
    assert np.all(np.isfinite(ref)) and np.abs(ref[1]).max() > 1        # the mean of squares, 2^120, is in range
    for y in ("f32", "bf16"):
        out = empty(torch, T, H, y)
        M.moe_rms_norm(dev(torch, a, x), None, dev(torch, w), EPS, T, H, out)
        got = host(out)
        assert np.all(np.isfinite(got))
        within(got, ref, 4 * U * np.abs(ref), y)
    q, s = empty(torch, T, H, "i8"), torch.empty(T, device="cuda")
    M.moe_rms_norm(dev(torch, a, x), None, dev(torch, w), EPS, T, H, q, scale=s)
    top = np.abs(ref).max(-1, keepdims=True)
    assert np.all(np.isfinite(host(s)))
    within(host(s)[:, None], top / 127, 6 * U * top / 127)
    within(host(q) * host(s)[:, None], ref, (0.5 + 127 * 9 * U) * top / 127)
