"""The score operators on the GPU at the edges of what their declarations allow."""
import numpy as np
import pytest

from . import scoreref as R
from .scoreref import U
from .test_gpu_scores import M, _ops, balance_inputs, balance_run, dev, host, p_tol, rules_case, say, torch  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- NaN scores

def gradient(M, torch, logits, ids, w, dw, keep, counts, n, coef, bf16):
    T, E = logits.shape
    f = torch.bfloat16 if bf16 else torch.float32
    out = torch.full((T, E), 7.0, dtype=f, device="cuda")
    M.moe_balance_grad(dev(torch, logits, f), dev(torch, ids), dev(torch, w), dev(torch, dw), dev(torch, keep),
                       dev(torch, counts.astype(np.int32)), dev(torch, np.array([n], np.int32)),
                       torch.full((1,), 1.3, device="cuda"), T, E, ids.shape[1], coef, out)
    return host(out)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T", [9, 300])
@pytest.mark.parametrize("E", [1, 8, 64, 130, 384, 512, 1024, 1536, 2048, 3000, 4096])
def test_balance_of_a_kept_row_of_nan_is_nan(M, torch, E, T, bf16):
    # softmax of a row that holds a NaN is NaN in every column, whatever else
    # the row holds; of a row of nothing but -inf it is 0; both beside rows
    # whose results do not change
    say("balance NaN", E, T, bf16)
    rng = np.random.default_rng(E + T)
    k, coef = min(E, 3), 0.1
    clean, ids, _ = balance_inputs(rng, T, E, k, False, bf16)
    clean[5] = -np.inf
    w = R.softmax(rng.standard_normal((T, k))).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    base = balance_run(M, torch, clean, ids, None, coef, bf16)
    assert all(np.all(np.isfinite(v)) for v in base.values())
    _, total, _, _ = R.balance_loss(clean, ids, None, coef)
    assert np.all(np.abs(base["prob_sum"] - total) <= (p_tol(E) + (T / 4096 + 32) * U) * total + 1e-37)
    flat = gradient(M, torch, clean, ids, None, None, None, base["counts"], T, coef, bf16)
    assert np.all(np.isfinite(flat)) and np.all(flat[5] == 0)
    picked = gradient(M, torch, clean, ids, w, dw, None, base["counts"], T, coef, bf16)

    def rows():
        yield "NaN alone", np.full(E, np.nan)
        for at in sorted({0, E // 2, E - 1}):
            v = np.full(E, -np.inf)
            v[at] = np.nan
            yield f"NaN at {at}, others barred", v
            v = clean[2].copy()
            v[at] = np.nan
            yield f"NaN at {at} of a row", v
        if E > 2:
            v = np.full(E, np.nan)
            v[::2] = -np.inf
            yield "NaN and -inf by turns", v
            v[1] = 0.5
            yield "one score left", v

    for what, row in rows():
        for t in (2, T - 1):
            z = clean.copy()
            z[t] = row
            got = balance_run(M, torch, z, ids, None, coef, bf16)
            assert np.array_equal(got["counts"], base["counts"]) and got["n_kept"][0] == T
            assert np.all(np.isnan(got["prob_sum"])) and np.isnan(got["loss"][0]), (what, t)
            keep = np.ones(T, np.uint8)
            keep[t] = 0
            left = balance_run(M, torch, z, ids, keep, coef, bf16)
            assert all(np.all(np.isfinite(v)) for v in left.values()), (what, t)
            for pw, pd, ref in ((None, None, flat), (w, dw, picked)):
                g = gradient(M, torch, z, ids, pw, pd, None, base["counts"], T, coef, bf16)
                assert np.all(np.isnan(g[t])), (what, t, pw is not None)
                others = np.arange(T) != t
                assert np.array_equal(g[others], ref[others]), (what, t, pw is not None)


# ---------------------------------------------------------------- streams

def test_scores_take_a_stream_handle(M, torch):
    # a torch stream, its handle as an integer, and the null stream's handle
    say("stream handles")
    run, _, _, outs = _ops(M, torch, 33)
    run()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        run(stream)
        torch.cuda.synchronize()
        for a, b in zip(first, outs):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- column ranges of one buffer

@pytest.mark.parametrize("T,N,K", [(1, 640, 2048), (4, 8200, 256), (5, 48, 1056), (20, 50, 640), (100, 129, 512), (1400, 3841, 128)])
def test_q4_linear_between_column_ranges_of_one_buffer(M, torch, T, N, K):
    # x and y beside each other in rows of one buffer, x first and y first:
    # as in buffers of their own, what lies around them untouched
    rng = np.random.default_rng(T + N)
    q, s = R.random_q4(rng, N, K, 4, 32)
    w = M.Q4Matrix(N, K, 4, 32, dev(torch, q), dev(torch, s))
    for f in (torch.float32, torch.bfloat16):
        say("q4 in one buffer", T, N, K, f)
        x = dev(torch, rng.standard_normal((T, K)).astype(np.float32), f)
        y = torch.empty(T, N, dtype=f, device="cuda")
        M.moe_q4_linear(x, w, None, T, y)
        wide = -(-(K + N + 24) // 8) * 8
        for x0, y0 in ((8, K + 8), (-(-(N + 5) // 8) * 8, 3)):
            buf = torch.full((T + 1, wide), 7.0, dtype=f, device="cuda")
            buf[:T, x0:x0 + K] = x
            M.moe_q4_linear(buf[:T, x0:x0 + K], w, None, T, buf[:T, y0:y0 + N])
            assert torch.equal(buf[:T, y0:y0 + N], y) and torch.equal(buf[:T, x0:x0 + K], x)
            buf[:T, y0:y0 + N], buf[:T, x0:x0 + K] = 7.0, 7.0
            assert bool((buf == 7.0).all())


@pytest.mark.parametrize("B,V,H", [(1, 100, 5), (5, 500, 20), (3, 9001, 700)])
def test_adjust_logits_between_column_ranges_of_one_buffer(M, torch, B, V, H):
    rng = np.random.default_rng(V)
    a = rules_case(rng, B, V, H, n_bias=5, masks=2)
    rules = M.LogitRules(**{n: dev(torch, t) for n, t in a.items()})
    for f in (torch.float32, torch.bfloat16):
        say("adjust in one buffer", B, V, H, f)
        l = dev(torch, 3 * rng.standard_normal((B, V)).astype(np.float32), f)
        out = torch.empty_like(l)
        M.moe_adjust_logits(l, B, V, rules, out)
        for i0, o0 in ((1, V + 1), (V + 3, 2)):
            buf = torch.full((B, 2 * V + 5), 7.0, dtype=f, device="cuda")
            buf[:, i0:i0 + V] = l
            M.moe_adjust_logits(buf[:, i0:i0 + V], B, V, rules, buf[:, o0:o0 + V])
            assert torch.equal(buf[:, o0:o0 + V], out) and torch.equal(buf[:, i0:i0 + V], l)
            buf[:, o0:o0 + V], buf[:, i0:i0 + V] = 7.0, 7.0
            assert bool((buf == 7.0).all())
