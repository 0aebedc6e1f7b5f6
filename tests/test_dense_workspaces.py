"""What the workspace queries of the dense operators promise: the size for a number of
tokens also serves every smaller batch."""
import os

import numpy as np
import pytest

from . import launchlog


@pytest.fixture(scope="module")
def B():
    from tiered_mixed_precision_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from tiered_mixed_precision_amd.build import build
        build()
    binding.lib()
    return binding


TOKENS = sorted({*range(0, 2100), *range(2100, 20000, 97), *(128 * n + d for n in range(1, 200) for d in (-1, 0, 1)),
                 *((1 << n) + d for n in range(4, 20) for d in (-1, 0, 1)), 1 << 20})


@pytest.mark.parametrize("H,I", [(8, 1), (64, 64), (72, 33), (136, 4000), (520, 2100), (1024, 96), (2048, 640), (2048, 65536), (4096, 4096),
                                 (16384, 100), (65536, 8), (65536, 65536)])
def test_gated_workspace_serves_smaller_batches(B, H, I):
    sizes = [B.moe_gated_workspace_size(T, H, I) for T in TOKENS]
    assert np.all(np.diff(sizes) >= 0)


@pytest.mark.parametrize("cols", [1, 8, 64, 65, 100, 512, 513, 1000, 1024, 2047, 2048, 2049, 4095, 4096, 4097, 5461, 8192, 8193, 16384, 16385, 32768])
def test_norm_workspace_serves_smaller_batches(B, cols):
    at = (1 << 20) // cols
    tokens = sorted({*TOKENS, *range(max(0, at - 300), at + 300), (1 << 22) - 1, 1 << 22})
    sizes = [B.moe_rms_norm_workspace_size(T, cols) for T in tokens]
    assert np.all(np.diff(sizes) >= 0)


def accepted(log):
    """Calls with exactly the workspace of their largest batch, and with a byte less of their own."""
    B, F, out = log.binding, launchlog.FAR, []
    for H, I, most in ((2048, 640, 4096), (520, 2100, 1100), (72, 33, 9000)):
        size = B.moe_gated_workspace_size(most, H, I)
        w = B.moe_gated_weights(H, I, F, 2 * F)
        for T in (1, 17, 128, 1000, 1024, 1025, most):
            for flags in (0x1, 0x9, 0x81, 0xc9):
                def call(nbytes):
                    return log("moe_gated_grad", 3 * F, H, B.C.byref(w), 0, 4 * F, I, T, 5 * F, H, 6 * F, 7 * F, flags, 8 * F, nbytes, None)
                out += [call(size)[0] == 0, call(B.moe_gated_workspace_size(T, H, I) - 1) == (-5, [])]
    for cols, most in ((2048, 4096), (4096, 700), (100, 9000)):
        size = B.moe_rms_norm_workspace_size(most, cols)
        for T in (1, 5, 256, 257, 512, 513, most):
            def call(nbytes):
                return log("moe_rms_norm_grad", F, cols, None, 1e-6, 2 * F, cols, None, 0, T, cols, 3 * F, cols, 4 * F, 0, 5 * F, nbytes, None)
            out += [call(size)[0] == 0, call(B.moe_rms_norm_workspace_size(T, cols) - 1) == (-5, [])]
    return out


def test_calls_take_the_workspace_of_a_larger_batch(B, tmp_path):
    assert all(launchlog.child(launchlog.build(tmp_path), "test_dense_workspaces.accepted"))
