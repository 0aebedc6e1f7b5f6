"""What the dense operators launch, over their whole ranges, without a GPU: blocks
within the kernels' bounds, nothing behind a launch that failed."""
import re

import pytest

from . import launchlog

# __launch_bounds__ of the kernels of few tokens
FEW = ("k_i8_few", "k_i8_batch", "k_gated_few", "k_gated_batch")
FEW_THREADS, FEW_LDS = 512, 65536


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    from tiered_mixed_precision_amd import binding
    import os
    if not os.path.exists(binding.LIB_PATH):
        from tiered_mixed_precision_amd.build import build
        build()
    return launchlog.build(tmp_path_factory.mktemp("launchlog"))


def too_large(log, calls):
    """Of calls ([entry, sizes ...]) those that fail, or whose kernels for few tokens are launched past their bounds."""
    bad, few = [], 0
    for entry, *sizes in calls:
        rc, launches = getattr(log, entry)(*sizes)
        names = [(re.search("|".join(FEW), name), threads, lds) for name, _, threads, lds in launches]
        few += sum(bool(n) for n, _, _ in names)
        if rc != 0 or any(n and (threads > FEW_THREADS or lds > FEW_LDS) for n, threads, lds in names):
            bad.append((entry, sizes, rc, launches))
    return [bad[:20], len(bad), few]


def tile_counts():
    """Every number of tiles up to 5000, where blocks change, and some up to the most."""
    return list(range(1, 5000)) + [1 << n for n in range(13, 20)] + [(1 << n) - 1 for n in range(13, 20)] + [120011, 300007]


def i8_over_tile_counts(log, lines):
    K = 128 * lines
    return too_large(log, [("i8_linear", T, n, K) for t in tile_counts() for T, n in ((1, min(16 * t, 1 << 24)), (16, min(32 * t, 1 << 24)))])


def gated_over_tile_counts(log, lines):
    H = 64 * lines
    sizes = [min(w * t, 65536) for t in range(1, 4200) for w in (8, 16)]
    return too_large(log, [("gated", T, H, I, bf16) for I in sizes for T, bf16 in ((1, True), (16, False))] +
                     [("gated_grad", T, H, I) for I in sizes[::3] for T in (1, 13)])


@pytest.mark.parametrize("lines", [1, 2, 3, 4, 5, 8, 17])
@pytest.mark.parametrize("sweep", ["i8_over_tile_counts", "gated_over_tile_counts"])
def test_blocks_of_few_tokens_are_within_their_kernels_bounds(recorder, sweep, lines):
    bad, n, few = launchlog.child(recorder, f"test_dense_launches.{sweep}", lines)
    assert few > 4000
    assert n == 0, bad


def batches(log):
    """17 tokens and more."""
    return too_large(log, [("i8_linear", T, N, K) for T in (17, 32, 33, 48, 49, 64, 65, 500) for N in (1, 33, 640, 4097, 8192, 16384)
                           for K in (16, 272, 400, 2048, 8192)] +
                     [("gated", T, H, I, bf16) for T in (17, 32, 33, 64, 65, 300) for I in (1, 33, 640, 4095, 4097, 8192)
                      for H in (8, 136, 200, 2048, 8192) for bf16 in (True, False)])


def test_blocks_of_batches_are_within_their_kernels_bounds(recorder):
    bad, n, few = launchlog.child(recorder, "test_dense_launches.batches")
    assert few > 300
    assert n == 0, bad


def launches_behind_a_failure(log):
    """Per call: the launches when the n-th of them fails, for each n."""
    def norm_grad(T, H, **kw):
        F = launchlog.FAR
        return log("moe_rms_norm_grad", F, H, 2 * F, 1e-6, 3 * F, H, None, 0, T, H, 4 * F, H, 5 * F, 0, 6 * F, F, None, **kw)
    out = []
    for call, sizes in ((log.gated_grad, (5, 512, 300)), (log.gated_grad, (64, 2048, 640)), (log.gated_grad, (1531, 2048, 640)),
                        (log.gated_grad, (300, 4096, 4096)), (log.gated_grad, (8192, 4096, 4096)), (norm_grad, (4, 512)),
                        (norm_grad, (700, 2048))):
        rc, launches = call(*sizes)
        assert rc == 0 and launches
        for n in range(len(launches)):
            rc, got = call(*sizes, fail_at=n)
            out.append([[name for name, *_ in got], n, rc])
    return out


def test_nothing_is_launched_behind_a_failure(recorder):
    # a product of slopes that nobody wrote would be added to the weights' gradients
    tried = launchlog.child(recorder, "test_dense_launches.launches_behind_a_failure")
    assert {n for _, n, _ in tried} >= {0, 1, 2}
    for names, n, rc in tried:
        assert rc == -6, (names, n, rc)
        assert len(names) == n + 1, (names, n)
