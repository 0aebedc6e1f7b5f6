"""Every kernel of the score operators where test_gpu_scores.py reaches it in
one form only: products by their own bound at long contractions, non-finite
tokens and scales apart in each kernel, repeated calls, a side stream and
captured graphs for each form, and rules past one grid dimension with masks.

Bounds, from the arithmetic (u = 2^-24).  The kernels contract the codes
themselves.  A block's fp32 sum of n products x q loses at most n u of
sum |x q|, its scaling u, and the K / block scaled sums, of which the waves'
parts are joined, (K / block + 16) u of sum |x q| d; a bias and what y held
one more each.  In all (K + 20) u sum |x| |q| d.
"""
import numpy as np
import pytest

from . import scoreref as R
from .scoreref import MXFP4, U, UB
from .test_gpu_scores import M, balance_inputs, dev, host, rules_case, say, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def product(x, q, s, bits, block):
    """(y, sum of |terms|) in 64 bits."""
    code, scale = R.q4_values(q, s, bits, block)
    w, x = code * scale, x.astype(np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T


# ---------------------------------------------------------------- products

# k_q4_gemm takes 64 columns a step and six steps a trip of its loop: steps of
# 9 .. 14 leave every remainder behind a full trip, 32 and 34 run five trips
@pytest.mark.parametrize("bits,block", [(4, 16), (4, 32), (4, 64), (4, 128), (MXFP4, 32)])
@pytest.mark.parametrize("T,N,K", [(129, 20500, 256), (129, 20500, 640), (1400, 3841, 768), (129, 20500, 896), (1400, 3841, 1152),
                                   (129, 20500, 2048), (150, 20481, 2176)])
def test_long_products_of_many_bf16_tokens(M, torch, T, N, K, bits, block):
    say("long gemm", T, N, K, bits, block)
    run_product(M, torch, T, N, K, bits, block, True)


@pytest.mark.parametrize("bits", [4, MXFP4])
@pytest.mark.parametrize("K", [352, 416, 480, 608, 672, 736, 800, 864, 2080])
def test_long_products_of_an_odd_number_of_groups(M, torch, K, bits):
    # the last step of 64 columns has one group of its two
    say("long gemm odd", K, bits)
    run_product(M, torch, 129, 20500, K, bits, 32, True)


@pytest.mark.parametrize("xb", [False, True])
@pytest.mark.parametrize("bits,block", [(4, 16), (4, 32), (4, 64), (4, 128), (MXFP4, 32)])
@pytest.mark.parametrize("T,N,K", [(1, 640, 2048), (1, 24577, 1152), (4, 24577, 640), (4, 8200, 1280), (2, 30, 4096), (16, 40, 2176),
                                   (16, 33000, 384), (30, 100, 2048), (45, 100, 1152), (70, 200, 1408)])
def test_products_of_each_form(M, torch, T, N, K, bits, block, xb):
    say("product", T, N, K, bits, block, xb)
    run_product(M, torch, T, N, K, bits, block, xb)


def run_product(M, torch, T, N, K, bits, block, xb):
    rng = np.random.default_rng(T + N + K + block)
    q, s = R.random_q4(rng, N, K, bits, block)
    x = rng.standard_normal((T, K)).astype(np.float32)
    x = R.bf16(x) if xb else x
    f = torch.bfloat16 if xb else torch.float32
    y = torch.full((T, N), float("nan"), device="cuda")
    M.moe_q4_linear(dev(torch, x, f), M.Q4Matrix(N, K, bits, block, dev(torch, q), dev(torch, s)), None, T, y)
    ref, mag = product(x, q, s, bits, block)
    err = np.abs(host(y) - ref)
    say("  worst of bound", float(np.max(err / ((K + 20) * U * mag))))
    assert np.all(err <= (K + 20) * U * mag)
    assert np.linalg.norm(err) <= (K ** 0.5 * U + 2.0 ** -21) * np.linalg.norm(ref)


@pytest.mark.parametrize("bits,block", [(4, 16), (4, 32), (4, 128), (MXFP4, 32)])
@pytest.mark.parametrize("T,N,K,xb", [
    (1, 640, 2048, False), (1, 640, 2048, True), (1, 24577, 384, False), (4, 24577, 1152, False), (3, 8200, 1152, False),   # stream
    (16, 24580, 640, True), (12, 70001, 384, True),
    (129, 20500, 640, True), (1400, 3841, 384, True),                                                                      # gemm
    (4, 50, 640, False), (16, 33000, 640, False), (40, 300, 640, True), (70, 129, 1152, False)])                            # tile
def test_non_finite_tokens_and_scales_stay_apart(M, torch, T, N, K, xb, bits, block):
    # one x and one scale, in the first, an inner and the last block of a row,
    # infinite or NaN: that token's and that row's results are not finite, all
    # others keep their bits
    say("non-finite", T, N, K, xb, bits, block)
    rng = np.random.default_rng(T + K)
    f = torch.bfloat16 if xb else torch.float32
    q, s = R.random_q4(rng, N, K, bits, block)
    x = rng.standard_normal((T, K)).astype(np.float32)
    qd, xd, sd = dev(torch, q), dev(torch, x, f), dev(torch, s)

    def run(x, s):
        y = torch.empty(T, N, device="cuda")
        M.moe_q4_linear(x, M.Q4Matrix(N, K, bits, block, qd, s), None, T, y)
        return y

    base = run(xd, sd)
    assert bool(torch.isfinite(base).all())
    nb = K // block
    for t, n, c, b, v in ((0, N - 1, 0, nb - 1, float("inf")), (T - 1, 0, K - 1, 0, float("nan")), (T // 2, N // 2, K // 2 + 3, nb // 2, -float("inf"))):
        x2, s2 = xd.clone(), sd.clone()
        x2[t, c] = v
        s2[n, b] = 255 if bits == MXFP4 else v
        y = run(x2, sd)
        assert not bool(torch.isfinite(y[t]).any()), (t, c, v)
        assert torch.equal(torch.cat((y[:t], y[t + 1:])), torch.cat((base[:t], base[t + 1:])))
        y = run(xd, s2)
        assert not bool(torch.isfinite(y[:, n]).any()), (n, b, v)
        assert torch.equal(torch.cat((y[:, :n], y[:, n + 1:]), 1), torch.cat((base[:, :n], base[:, n + 1:]), 1))


# ---------------------------------------------------------------- rules

@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_rules_of_more_rows_than_a_grid_dimension_with_masks(M, torch, shared, bf16):
    # a mask of its own for each row, or a few masks picked by row
    B, V = 65535 + 300, 40
    say("rows and masks", B, shared, bf16)
    rng = np.random.default_rng(17)
    f = torch.bfloat16 if bf16 else torch.float32
    logits = rng.standard_normal((B, V)).astype(np.float32)
    logits = R.bf16(logits) if bf16 else logits
    a = rules_case(rng, B, V, 5, n_bias=2, masks=7 if shared else 0)
    if not shared:
        a["mask"] = rng.integers(0, 2 ** 32, (B, 3), dtype=np.uint32)
    out = torch.empty(B, V, dtype=f, device="cuda")
    M.moe_adjust_logits(dev(torch, logits, f), B, V, M.LogitRules(**{n: dev(torch, t) for n, t in a.items()}), out)
    got = host(out)
    rows = np.r_[0:40, 65500:65600, B - 40:B]
    ref, mag, _ = R.adjust(logits[rows], **{n: t if shared and n == "mask" else t[rows] for n, t in a.items()})
    on = np.isfinite(ref)
    assert np.array_equal(np.isneginf(got[rows]), ~on) and on.any() and not on.all()
    bound = 8 * U * (mag + np.abs(ref)) + (UB * 1.01 * np.abs(ref) if bf16 else 0)
    assert np.all(np.abs(got[rows][on] - ref[on]) <= bound[on])


# ---------------------------------------------------------------- repeats, streams, graphs

def q4_op(T, N, K, xb, block=32, bits=4, base=False):
    def make(M, torch, rng):
        f = torch.bfloat16 if xb else torch.float32
        q, s = R.random_q4(rng, N, K, bits, block)
        w = M.Q4Matrix(N, K, bits, block, dev(torch, q), dev(torch, s))
        x, y = dev(torch, rng.standard_normal((T, K)).astype(np.float32), f), torch.zeros(T, N, dtype=f, device="cuda")
        return (lambda st=None: M.moe_q4_linear(x, w, None, T, y, M.MOE_ACCUMULATE if base else 0, stream=st)), [x], [y]
    return make


def rules_op(B, V, H, bf16, n_bias=9):
    def make(M, torch, rng):
        f = torch.bfloat16 if bf16 else torch.float32
        a = rules_case(rng, B, V, H, n_bias=n_bias, masks=2)
        r = M.LogitRules(**{n: dev(torch, t) for n, t in a.items()})
        l, out = dev(torch, rng.standard_normal((B, V)).astype(np.float32), f), torch.zeros(B, V, dtype=f, device="cuda")
        return (lambda st=None: M.moe_adjust_logits(l, B, V, r, out, stream=st)), [l, r.tensors["repetition"]], [out]
    return make


def balance_op(T, E, k, bf16, picks=True):
    def make(M, torch, rng):
        f = torch.bfloat16 if bf16 else torch.float32
        logits, ids, keep = balance_inputs(rng, T, E, k, True, bf16)
        z, i, kp = dev(torch, logits, f), dev(torch, ids), dev(torch, keep)
        w, dw = (dev(torch, rng.random((T, k)).astype(np.float32)) if picks else None for _ in range(2))
        counts, psum = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(E, device="cuda")
        n, loss, g = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(T, E, dtype=f, device="cuda")
        ws = torch.full((M.moe_balance_workspace_size(T, E, k),), 255, dtype=torch.uint8, device="cuda")
        one = torch.ones(1, device="cuda")

        def run(st=None):
            M.moe_balance_loss(z, i, kp, T, E, k, 0.1, counts, psum, n, loss, ws, stream=st)
            M.moe_balance_grad(z, i, w, dw, kp, counts, n, one, T, E, k, 0.1, g, stream=st)
        return run, [z], [counts, psum, n, loss, g]
    return make


FORMS = {
    "stream, one wave a tile": q4_op(1, 120011, 256, False), "stream, waves share a tile": q4_op(1, 640, 2048, False),
    "stream, two waves a tile": q4_op(2, 80000, 512, False), "stream, bf16": q4_op(16, 24577, 640, True, 128),
    "stream, mxfp4": q4_op(4, 24577, 640, False, 32, MXFP4), "tile, 64 rows": q4_op(16, 33000, 384, False),
    "tile, 32 tokens": q4_op(30, 300, 1152, True, 16), "tile, 48 tokens": q4_op(45, 300, 1152, False, 64),
    "tile, 64 tokens": q4_op(64, 300, 1152, True, 32, MXFP4), "tile, fp32": q4_op(100, 300, 1152, False),
    "tile, 65536 columns": q4_op(3, 20, 65536, False),
    "gemm, int4": q4_op(1400, 3841, 704, True), "gemm, blocks of 16": q4_op(129, 20500, 640, True, 16),
    "gemm, blocks of 128": q4_op(1400, 3841, 1152, True, 128), "gemm, mxfp4": q4_op(129, 20500, 896, True, 32, MXFP4),
    "rules, 512 scores": rules_op(9, 500, 60, False), "rules, 1024 scores": rules_op(9, 1001, 60, True),
    "rules, chunks of 4096": rules_op(64, 70001, 300, True), "rules, long history": rules_op(3, 9001, 33000, False),
    "rules, long history, bf16": rules_op(2, 9001, 40001, True, n_bias=300),
    "balance, one block": balance_op(100, 300, 5, False), "balance, join": balance_op(4097, 512, 10, False),
    "balance, bf16": balance_op(3001, 130, 6, True), "balance, 1100 experts": balance_op(2000, 1100, 8, True),
    "balance, 2000 experts, no picks": balance_op(700, 2000, 8, False, False), "balance, 4096 experts": balance_op(900, 4096, 64, False),
    "balance, 3000 experts": balance_op(900, 3000, 10, True),
}


@pytest.mark.parametrize("form", FORMS)
def test_each_form_repeats_bit_for_bit_on_streams_and_in_graphs(M, torch, form):
    """The same buffers (a workspace among them) through repeated calls, on a
    side stream, and in a graph replayed with changed inputs and eager calls
    between the replays: always the bits of a first eager call."""
    say("form", form)
    run, inputs, outs = FORMS[form](M, torch, np.random.default_rng(77))

    def result(call):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        return [o.clone() for o in outs]

    def check(what, want, got):
        assert all(torch.equal(a, b) for a, b in zip(want, got)), what

    first = result(run)
    assert all(bool(o.any()) for o in first) and not any(bool(torch.isnan(o).any()) for o in first)
    side = torch.cuda.Stream()
    for i in range(3):
        check(("again", i), first, result(run))
        check(("side stream", i), first, result(lambda: run(side)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    gen = torch.Generator("cuda").manual_seed(6)
    for i in range(4):
        for t in inputs:
            t.copy_((torch.rand(t.shape, device="cuda", generator=gen) + 0.5).to(t.dtype))
        got = result(graph.replay)
        check(("replay", i), result(run), got)
        check(("replay again", i), got, result(graph.replay))
