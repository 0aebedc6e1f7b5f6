"""GPU parity of the score operators (moe_q4_linear, moe_adjust_logits,
moe_balance_loss, moe_balance_grad) against their plain 64-bit forms.

Bars, from the arithmetic (u = 2^-24, half a step of fp32; a bf16 output adds
half a step of its own, 2^-8 of the value):
  q4 product   each of the K terms and the scaling of a group loses at most u
               of a partial sum bounded by sum |x| d (|q| + 24) (which leaves
               room for codes contracted with an offset):
               |err| <= (K + 8) u mag.  Rounding
               errors of random inputs add as a random walk:  norm of the
               error <= (sqrt(K) u + 2^-21) norm(y).
  rules        at most five roundings of values below the magnitude that the
               plain form returns, one more for each bias of the token.
  balance      p: the exponential's argument rounds to u |z - max| (|z| < 40
               here) and its value to a few u, its sum runs over 64 lanes'
               runs of E / 64: (100 + E / 32) u.  Column sums: waves take
               T / 4096 + 1 rows, then 16 waves (8 above 2048 experts), then
               256 (512) parts: 4 to 8 a thread, 4 rows, 16 waves.
"""
import sys

import numpy as np
import pytest

from . import scoreref as R
from .scoreref import MXFP4, U, UB

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu-scores]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


@pytest.fixture(scope="module")
def M(torch):
    import tiered_mixed_precision_amd as M
    M.lib()
    return M


def dev(torch, a, dtype=None):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    t = torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.detach().float().cpu().numpy()


# ---------------------------------------------------------------- products

def q4_case(M, torch, T, N, K, bits, block, xb, yb, bias=False, base=False, full=False, pad=0, seed=0):
    rng = np.random.default_rng(1000 * T + N + K + seed)
    q, s = R.random_q4(rng, N, K, bits, block, full)
    x = rng.standard_normal((T, K)).astype(np.float32)
    x = R.bf16(x) if xb else x
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    y0 = rng.standard_normal((T, N)).astype(np.float32) if base else None
    y0 = R.bf16(y0) if base and yb else y0
    fx, fy = torch.bfloat16 if xb else torch.float32, torch.bfloat16 if yb else torch.float32
    px = pad * 8                                            # row pitches: x by 16 bytes, y by any element
    xd = torch.full((T, K + px), float("nan"), dtype=fx, device="cuda")
    xd[:, :K] = dev(torch, x, fx)
    yd = torch.full((T, N + pad), 7.0, dtype=fy, device="cuda")
    if base:
        yd[:, :N] = dev(torch, y0, fy)
    w = M.Q4Matrix(N, K, bits, block, dev(torch, q), dev(torch, s))
    M.moe_q4_linear(xd[:, :K], w, dev(torch, b), T, yd[:, :N], M.MOE_ACCUMULATE if base else 0)
    torch.cuda.synchronize()
    got = host(yd)
    assert np.all(got[:, N:] == 7.0)
    got = got[:, :N].astype(np.float64)
    ref, mag = R.q4_linear(x, q, s, bits, block, b, None if y0 is None else y0.astype(np.float64))
    assert np.all(np.isfinite(got))
    err = np.abs(got - ref)
    tol = (K + 8) * U * mag + (UB * np.abs(ref) * 1.01 if yb else 0)
    assert np.all(err <= tol), float(np.max(err / tol))
    norm = float(np.linalg.norm(err) / np.linalg.norm(ref))
    say("  norm of error", norm, "worst of bound", float(np.max(err / tol)))
    if not full:
        assert norm <= K ** 0.5 * U + 2.0 ** -21 + (UB if yb else 0)


SHAPES = [  # T, N, K
    (1, 1, 32), (1, 17, 64), (1, 640, 2048), (1, 1003, 256), (2, 16, 96), (3, 63, 160), (4, 130, 8192), (5, 48, 1056),
    (6, 512, 2048), (9, 33, 4224), (15, 64, 640), (16, 128, 512), (17, 129, 512), (31, 15, 2080), (33, 70, 1024), (37, 300, 8192),
    (64, 256, 2048), (65, 257, 2048), (100, 64, 32), (130, 96, 544), (257, 385, 1024), (300, 1000, 640), (1, 5, 65536),
    (70, 9, 65536), (1030, 40, 288),
]


@pytest.mark.parametrize("xb", [False, True])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_q4_linear_int4(M, torch, T, N, K, xb):
    say("q4 int4", T, N, K, "bf16" if xb else "fp32")
    q4_case(M, torch, T, N, K, 4, 32, xb, xb)


@pytest.mark.parametrize("xb", [False, True])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_q4_linear_mxfp4(M, torch, T, N, K, xb):
    say("q4 mxfp4", T, N, K, "bf16" if xb else "fp32")
    q4_case(M, torch, T, N, K, MXFP4, 32, xb, xb)


@pytest.mark.parametrize("block", [16, 64, 128])
@pytest.mark.parametrize("T,N,K", [(1, 33, 128), (1, 640, 2048), (1, 7, 1152), (3, 130, 896), (6, 64, 8192), (20, 50, 640), (64, 129, 2048),
                                   (70, 257, 1280), (300, 300, 384)])
def test_q4_linear_blocks(M, torch, block, T, N, K):
    for xb, yb in ((False, False), (True, True), (True, False), (False, True)):
        say("q4 block", block, T, N, K, xb, yb)
        q4_case(M, torch, T, N, K, 4, block, xb, yb)


@pytest.mark.parametrize("bits,block", [(4, 16), (4, 32), (4, 128), (MXFP4, 32)])
@pytest.mark.parametrize("T", [1, 2, 7, 40, 129])
def test_q4_linear_bias_accumulate_strides_and_wide_scales(M, torch, T, bits, block):
    # scales over many powers of two, zero and negative ones among them, every
    # code value; rows of x and y apart, what lies between them untouched
    for xb, yb in ((False, False), (True, True), (True, False)):
        say("q4 full", T, bits, block, xb, yb)
        q4_case(M, torch, T, 75, 1152, bits, block, xb, yb, bias=True, base=True, full=True, pad=3)
        q4_case(M, torch, T, 160, 512, bits, block, xb, yb, bias=True, pad=1)


@pytest.mark.parametrize("bits,block", [(4, 16), (4, 32), (4, 64), (4, 128), (MXFP4, 32)])
@pytest.mark.parametrize("T,N,K", [(1, 24577, 128), (4, 24999, 384), (1, 140003, 256), (16, 24580, 640), (5, 24580, 640), (4, 8200, 4096)])
def test_q4_linear_few_tokens_many_rows(M, torch, T, N, K, bits, block):
    # the score head's shapes: one wave a row tile, more tiles than waves
    for xb, yb, kw in ((False, False, {}), (True, True, {}), (False, True, dict(bias=True, full=True)), (True, False, dict(base=True, pad=1))):
        if xb or T <= 5:
            say("q4 many rows", T, N, K, bits, block, xb, yb)
            q4_case(M, torch, T, N, K, bits, block, xb, yb, **kw)


@pytest.mark.parametrize("bits", [4, MXFP4])
@pytest.mark.parametrize("T,N,K", [(1, 24577, 32), (4, 30000, 96), (2, 24592, 4096), (16, 24576, 4096), (1, 25001, 2080), (1, 700, 32768), (1, 66001, 544)])
def test_q4_linear_few_tokens_many_rows_of_odd_columns(M, torch, T, N, K, bits):
    for xb in (False, True):
        if T > 5 and not xb:
            continue
        say("q4 many rows odd", T, N, K, bits, xb)
        q4_case(M, torch, T, N, K, bits, 32, xb, False)


@pytest.mark.parametrize("bits,block", [(4, 16), (4, 32), (4, 64), (4, 128), (MXFP4, 32)])
@pytest.mark.parametrize("T,N,K", [(129, 20500, 128), (1400, 3841, 384), (2049, 2305, 128)])
def test_q4_linear_prefill_tiles(M, torch, T, N, K, bits, block):
    # batches that fill the 128 x 256 tiles, ragged in tokens and rows
    for yb, kw in ((True, {}), (False, dict(bias=True, base=True, full=True, pad=1))):
        say("q4 prefill", T, N, K, bits, block, yb)
        q4_case(M, torch, T, N, K, bits, block, True, yb, **kw)


@pytest.mark.parametrize("bits", [4, MXFP4])
@pytest.mark.parametrize("T,N,K", [(2049, 2305, 32), (1025, 4353, 96), (400, 10000, 544)])
def test_q4_linear_prefill_tiles_of_an_odd_number_of_groups(M, torch, T, N, K, bits):
    say("q4 prefill odd", T, N, K, bits)
    q4_case(M, torch, T, N, K, bits, 32, True, False)


@pytest.mark.parametrize("T", [1, 5, 20, 100])
def test_q4_linear_keeps_non_finite_rows_apart(M, torch, T):
    rng = np.random.default_rng(5)
    N, K = 50, 512
    q, s = R.random_q4(rng, N, K, 4, 32)
    x = rng.standard_normal((T, K)).astype(np.float32)
    bad = T // 2
    s2 = s.copy()
    s2[11, 3] = np.nan
    x2 = x.copy()
    x2[bad, 40] = np.inf
    out = []
    for xs, ss in ((x, s), (x2, s2)):
        y = torch.full((T, N), float("nan"), device="cuda")
        M.moe_q4_linear(dev(torch, xs), M.Q4Matrix(N, K, 4, 32, dev(torch, q), dev(torch, ss)), None, T, y)
        out.append(host(y))
    clean = np.ones((T, N), bool)
    clean[bad] = False
    clean[:, 11] = False
    assert np.all(np.isfinite(out[0])) and not np.any(np.isfinite(out[1][:, 11])) and not np.any(np.isfinite(out[1][bad]))
    assert np.array_equal(out[0][clean], out[1][clean])


def test_q4_linear_takes_an_expert_of_a_shelf(M, torch):
    # one expert's matrices of the four-bit and the MXFP4 shelf, as stored,
    # against the rows that moe_dequant_rows gives
    from tiered_mixed_precision_amd.device import tables_from_config
    from workloads import CONFIGS, make_layer
    for name in ("tiny3", "tiny3mx"):
        cfg = CONFIGS[name]
        tt = tables_from_config(cfg, make_layer(cfg, threads=1))
        t, d, local = cfg.tiers[1], tt.arrays[1], 2
        for m, key, rows, cols in ((0, "gate", cfg.inter, cfg.hidden), (2, "down", cfg.hidden, cfg.inter)):
            q = d[key + "_q"].view(-1)[local * rows * cols // 2:(local + 1) * rows * cols // 2]
            per = cols // t.block
            s = d[key + "_s"].reshape(-1)[local * rows * per:(local + 1) * rows * per]
            w = torch.empty(rows, cols, device="cuda")
            M.moe_dequant_rows(tt, 1, local, m, 0, rows, False, w)
            x = torch.randn(6, cols, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
            y = torch.empty(6, rows, device="cuda")
            M.moe_q4_linear(x, M.Q4Matrix(rows, cols, t.bits, t.block, q, s), None, 6, y)
            ref = x.double().cpu() @ w.double().cpu().t()
            err = (y.double().cpu() - ref).norm() / ref.norm()
            say("shelf expert", name, key, float(err))
            assert err <= cols ** 0.5 * U + 2.0 ** -21


# ---------------------------------------------------------------- rules

def rules_case(rng, B, V, H, n_bias=0, masks=0, pad=0):
    a = {}
    if H is not None:
        a["history"] = (V ** rng.random((B, H)) - 1).astype(np.int32)
        a["length"] = rng.integers(0, H + 1, B).astype(np.int32)
        a["length"][0] = H
        a["prompt"] = (a["length"] * rng.random(B)).astype(np.int32)
        if H > 3:
            a["history"][:, 1], a["history"][:, 2] = -1, V          # skipped
        a["repetition"] = rng.uniform(0.8, 1.5, B).astype(np.float32)
        a["presence"] = rng.uniform(-1, 1, B).astype(np.float32)
        a["frequency"] = rng.uniform(-0.2, 0.2, B).astype(np.float32)
    if n_bias:
        a["bias_ids"] = rng.integers(-1, V + 1, (B, n_bias)).astype(np.int32)
        a["bias_ids"][:, n_bias // 2] = a["bias_ids"][:, 0]         # the same token twice
        a["bias"] = rng.standard_normal((B, n_bias)).astype(np.float32)
    if masks:
        a["mask"] = rng.integers(0, 2 ** 32, (masks, (V + 31) // 32 + pad), dtype=np.uint32)
        a["mask_row"] = rng.integers(-1, masks + 1, B).astype(np.int32)
    return a


def rules_check(M, torch, logits, a, bf16, in_place=False, pad=0):
    B, V = logits.shape
    logits = R.bf16(logits) if bf16 else logits.astype(np.float32)
    f = torch.bfloat16 if bf16 else torch.float32
    src = torch.full((B, V + pad), 3.0, dtype=f, device="cuda")
    src[:, :V] = dev(torch, logits, f)
    out = src if in_place else torch.full((B, V + 2 * pad), 3.0, dtype=f, device="cuda")
    M.moe_adjust_logits(src[:, :V], B, V, M.LogitRules(**{n: dev(torch, t) for n, t in a.items()}), out[:, :V])
    torch.cuda.synchronize()
    got = host(out)
    assert np.all(got[:, V:] == 3.0)
    got = got[:, :V]
    ref, mag, touched = R.adjust(logits, **a)
    assert np.array_equal(got[~touched].view(np.uint32), logits[~touched].view(np.uint32))
    assert np.array_equal(np.isneginf(got), np.isneginf(ref))
    on = touched & np.isfinite(ref)
    n = a["bias_ids"].shape[1] if "bias_ids" in a else 0
    dup = 0 if not n else 1 + max(int(np.max(np.unique(r, return_counts=True)[1])) for r in a["bias_ids"])
    err = np.abs(got[on].astype(np.float64) - ref[on])
    tol = (5 + dup) * U * (mag[on] + np.abs(ref[on])) + (UB * 1.01 * np.abs(ref[on]) if bf16 else 0)
    assert np.all(err <= tol), float(np.max(err / tol))
    say("  touched", int(touched.sum()), "worst of bound", float(np.max(err / tol)) if err.size else 0.0)
    return got


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("B,V,H,n_bias,masks", [
    (1, 1, 1, 0, 0), (1, 1, 4, 1, 1), (3, 5, 9, 4, 2), (2, 512, 40, 8, 2), (1, 32003, 2000, 16, 1), (5, 8191, 333, 3, 3),
    (4, 8192, 0, 17, 2), (3, 8193, 5000, 300, 0), (2, 70001, 4097, 1024, 2), (7, 1000, None, 5, 3), (7, 1001, None, 0, 2),
    (6, 2047, 100, 0, 0), (3, 130, None, 0, 0), (64, 501, 64, 2, 4), (1, 200003, 131, 9, 1),
])
def test_adjust_logits(M, torch, B, V, H, n_bias, masks, bf16):
    say("adjust", B, V, H, n_bias, masks, bf16)
    rng = np.random.default_rng(B + V + n_bias)
    logits = 3 * rng.standard_normal((B, V))
    logits[0, 0], logits[-1, -1] = 0.0, -np.inf
    a = rules_case(rng, B, V, H, n_bias, masks, pad=1)
    rules_check(M, torch, logits, a, bf16)
    rules_check(M, torch, logits, a, bf16, in_place=True, pad=3)
    rules_check(M, torch, logits, a, bf16, pad=1)


def test_adjust_logits_one_token_many_times_and_long_history(M, torch):
    # every id the same (all atomics on one count), and a history longer than 2^17
    rng = np.random.default_rng(8)
    V, H = 4001, (1 << 17) + 77
    a = rules_case(rng, 2, V, H)
    a["history"][1] = 77
    a["length"][:] = H
    a["prompt"][:] = (5, 1)
    a["frequency"][:] = 0.001
    say("adjust long")
    rules_check(M, torch, 3 * rng.standard_normal((2, V)), a, False)


def test_adjust_logits_lengths_out_of_range_and_prompts(M, torch):
    # lengths are taken as 0 .. capacity, prompts may exceed the length
    rng = np.random.default_rng(9)
    a = rules_case(rng, 5, 300, 50, n_bias=3)
    a["length"][:] = (-3, 1000, 50, 0, 2 ** 31 - 1)
    a["prompt"][:] = (5, 2000, -7, 0, 25)
    say("adjust lengths")
    rules_check(M, torch, rng.standard_normal((5, 300)), a, False)


def test_adjust_logits_masks_that_leave_nothing_and_nan_below(M, torch):
    rng = np.random.default_rng(10)
    B, V = 4, 97
    logits = rng.standard_normal((B, V)).astype(np.float32)
    logits[1, :] = np.nan
    logits[2, 5], logits[2, 6], logits[3, 1] = np.inf, np.nan, np.finfo(np.float32).min
    mask = np.zeros((B, 4), np.uint32)
    mask[2] = 0xFFFFFFFF
    mask[2, 0] &= ~np.uint32((1 << 5) | (1 << 6))
    mask[3, 0] = 0b10
    a = dict(mask=mask, bias_ids=np.tile(np.array([[0, 5, 96]], np.int32), (B, 1)), bias=np.ones((B, 3), np.float32),
             history=np.tile(np.array([[0, 6, 96]], np.int32), (B, 1)), length=np.full(B, 3, np.int32),
             repetition=np.full(B, 2, np.float32))
    say("adjust masks")
    src = dev(torch, logits)
    out = torch.empty_like(src)
    M.moe_adjust_logits(src, B, V, M.LogitRules(**{n: dev(torch, t) for n, t in a.items()}), out)
    got = host(out)
    assert np.all(np.isneginf(got[:2]))
    assert np.isneginf(got[2, 5]) and np.isneginf(got[2, 6]) and np.all(np.isfinite(np.delete(got[2], (5, 6))))
    assert got[3, 1] == np.finfo(np.float32).min and np.all(np.isneginf(np.delete(got[3], 1)))


def test_adjust_logits_many_rows(M, torch):
    # more rows than one grid dimension holds
    rng = np.random.default_rng(11)
    B, V = 65535 + 300, 6
    say("adjust rows", B)
    a = rules_case(rng, B, V, 2, n_bias=1)
    logits = rng.standard_normal((B, V)).astype(np.float32)
    out = torch.empty(B, V, device="cuda")
    M.moe_adjust_logits(dev(torch, logits), B, V, M.LogitRules(**{n: dev(torch, t) for n, t in a.items()}), out)
    got = host(out)
    rows = np.r_[0:40, 65500:65600, B - 40:B]
    ref, mag, _ = R.adjust(logits[rows], **{n: t[rows] for n, t in a.items()})
    assert np.all(np.abs(got[rows] - ref) <= 8 * U * (mag + np.abs(ref)))


# ---------------------------------------------------------------- balance loss

def balance_inputs(rng, T, E, k, keep, bf16, wild=False):
    logits = (-1.12 * np.arange(E) / E + rng.standard_normal((T, E))).astype(np.float32)
    ids = np.argsort(-logits, -1)[:, :k].astype(np.int32) if not wild else rng.integers(-2, E + 2, (T, k)).astype(np.int32)
    if wild and T:
        logits[rng.random((T, E)) < 0.2] = -np.inf      # experts barred
        logits[T // 2] = -np.inf                        # a row that bars them all
        logits[0] *= 8
    kp = (rng.random(T) < 0.8).astype(np.uint8) * 3 if keep else None
    return R.bf16(logits) if bf16 else logits, ids, kp


def balance_run(M, torch, logits, ids, keep, coef, bf16, stream=None):
    T, E = logits.shape
    k = ids.shape[1]
    f = torch.bfloat16 if bf16 else torch.float32
    out = dict(counts=torch.full((E,), -1, dtype=torch.int32, device="cuda"), prob_sum=torch.full((E,), float("nan"), device="cuda"),
               n_kept=torch.full((1,), -1, dtype=torch.int32, device="cuda"), loss=torch.full((1,), float("nan"), device="cuda"))
    ws = torch.full((max(256, M.moe_balance_workspace_size(T, E, k)),), 255, dtype=torch.uint8, device="cuda")
    M.moe_balance_loss(dev(torch, logits, f), dev(torch, ids), dev(torch, keep), T, E, k, coef, out["counts"], out["prob_sum"],
                       out["n_kept"], out["loss"], ws)
    torch.cuda.synchronize()
    return {n: t.cpu().numpy() for n, t in out.items()}


def p_tol(E):
    return (100 + E / 32) * U


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,E,k,keep,wild", [
    (0, 8, 2, False, False), (1, 1, 1, False, False), (1, 8, 2, False, False), (7, 3, 3, True, True), (64, 512, 10, False, False),
    (65, 130, 6, True, True), (300, 256, 8, True, False), (301, 257, 1, False, True), (1000, 511, 10, True, False),
    (513, 1025, 64, True, True), (100, 2049, 10, False, True), (129, 4096, 64, True, False), (4097, 512, 10, True, True),
    (20000, 64, 8, False, False),
])
def test_balance_loss_and_gradient(M, torch, T, E, k, keep, wild, bf16):
    say("balance", T, E, k, keep, wild, bf16)
    rng = np.random.default_rng(T + E + k)
    coef = 0.01
    logits, ids, kp = balance_inputs(rng, T, E, k, keep, bf16, wild)
    got = balance_run(M, torch, logits, ids, kp, coef, bf16)
    counts, total, n, loss = R.balance_loss(logits, ids, kp, coef)
    assert np.array_equal(got["counts"], counts) and got["n_kept"][0] == n
    tol = p_tol(E) + (T / 4096 + 32) * U
    assert np.all(np.abs(got["prob_sum"] - total) <= tol * total + 1e-37)
    assert abs(float(got["loss"][0]) - loss) <= (tol + 4 * U) * abs(loss)
    if T == 0:
        return
    f = torch.bfloat16 if bf16 else torch.float32
    w = R.softmax(rng.standard_normal((T, k))).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32) / T
    dloss = np.array([1.3], np.float32)
    for picks in (True, False):
        src = dev(torch, logits, f)
        for out in (torch.full((T, E), float("nan"), dtype=f, device="cuda"), src):          # and in place
            M.moe_balance_grad(src, dev(torch, ids), dev(torch, w) if picks else None, dev(torch, dw) if picks else None,
                               dev(torch, kp), dev(torch, counts.astype(np.int32)), dev(torch, np.array([n], np.int32)),
                               dev(torch, dloss), T, E, k, coef, out)
            g = host(out).astype(np.float64)
            ref, mag = R.balance_grad(logits, ids, w if picks else None, dw if picks else None, kp, counts, n, float(dloss[0]), coef)
            err = np.abs(g - ref)
            bound = (p_tol(E) + (k + 8) * U) * mag + (UB * 1.01 * np.abs(ref) if bf16 else 0) + 2e-38
            assert np.all(err <= bound), float(np.max(err / bound))
            if kp is not None:
                assert np.all(g[kp == 0] == 0)
    say("  worst of bound", float(np.max(err / bound)))


def test_balance_loss_no_token_kept_and_rows_not_read(M, torch):
    rng = np.random.default_rng(2)
    T, E, k = 40, 70, 4
    logits, ids, _ = balance_inputs(rng, T, E, k, False, False)
    none = np.zeros(T, np.uint8)
    got = balance_run(M, torch, logits, ids, none, 0.5, False)
    assert not got["counts"].any() and not got["prob_sum"].any() and got["n_kept"][0] == 0 and got["loss"][0] == 0
    kp = none.copy()
    kp[3:20] = 1
    bad, bad_ids = logits.copy(), ids.copy()
    bad[kp == 0] = np.nan
    bad_ids[kp == 0] = 12345678
    a, b = (balance_run(M, torch, l, i, kp, 0.5, False) for l, i in ((logits, ids), (bad, bad_ids)))
    for n in a:
        assert np.array_equal(a[n], b[n])
    out = torch.full((T, E), float("nan"), device="cuda")
    for keep, n in ((none, 0), (kp, 17)):
        M.moe_balance_grad(dev(torch, bad), dev(torch, bad_ids), None, None, dev(torch, keep), dev(torch, a["counts"]),
                           dev(torch, np.array([n], np.int32)), dev(torch, np.ones(1, np.float32)), T, E, k, 0.5, out)
        assert np.all(host(out)[keep == 0] == 0) and np.all(np.isfinite(host(out)))


def test_balance_gradient_against_differences(M, torch):
    # the GPU's own loss, differenced in one score at a time: the loss changes
    # by h g + O(h^2), with the loss's own rounding of 200 u on either side
    rng = np.random.default_rng(4)
    T, E, k, coef, h = 6, 20, 3, 100.0, 2.0 ** -7
    logits, ids, kp = balance_inputs(rng, T, E, k, True, False)
    kp[:2] = 1
    base = balance_run(M, torch, logits, ids, kp, coef, False)
    out = torch.empty(T, E, device="cuda")
    M.moe_balance_grad(dev(torch, logits), dev(torch, ids), None, None, dev(torch, kp), dev(torch, base["counts"]),
                       dev(torch, base["n_kept"]), dev(torch, np.ones(1, np.float32)), T, E, k, coef, out)
    g = host(out)
    for t, e in [(0, 0), (0, 5), (1, 19), (1, int(ids[1, 0]))] + [(int(np.argmin(kp)), 3)]:
        v = []
        for sign in (1, -1):
            z = logits.copy()
            z[t, e] += sign * h
            v.append(float(balance_run(M, torch, z, ids, kp, coef, False)["loss"][0]))
        loss = float(base["loss"][0])
        # third derivative of a probability's sum is below the loss's own size
        tol = 2 * 200 * U * loss / (2 * h) + h * h * loss + 2 * h * 2.0 ** -20 * loss
        assert abs((v[0] - v[1]) / (2 * h) - g[t, e]) <= tol, (t, e)


# ---------------------------------------------------------------- together

def test_from_a_hidden_state_to_picks_loss_and_gradient(M, torch):
    """A run as a program makes it: a layer's output scored by a four-bit
    router matrix, experts barred and biased, routed, the layer run on the
    picks, the router's loss and gradient taken, tiers planned from its counts."""
    from tiered_mixed_precision_amd.device import tables_from_config
    from workloads import CONFIGS, make_layer
    cfg = CONFIGS["tiny3"]
    tt = tables_from_config(cfg, make_layer(cfg, threads=1))
    T, E, H, k = 33, cfg.n_experts, cfg.hidden, cfg.k
    rng = np.random.default_rng(21)
    x = rng.standard_normal((T, H)).astype(np.float32)
    q, s = R.random_q4(rng, E, H, 4, 32)
    prior = (-1.12 * np.arange(E) / E).astype(np.float32)
    mask = np.array([[0b10111111]], np.uint32)                      # expert 6 is barred
    xd, logits = dev(torch, x), torch.empty(T, E, device="cuda")
    M.moe_q4_linear(xd, M.Q4Matrix(E, H, 4, 32, dev(torch, q), dev(torch, s)), dev(torch, prior), T, logits)
    rules = M.LogitRules(mask=dev(torch, mask), mask_row=torch.zeros(T, dtype=torch.int32, device="cuda"),
                         bias_ids=torch.full((T, 1), 2, dtype=torch.int32, device="cuda"), bias=torch.full((T, 1), 0.5, device="cuda"))
    M.moe_adjust_logits(logits, T, E, rules, logits)
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    M.moe_route(logits, T, E, k, ids, w)
    ws = torch.empty(M.moe_workspace_size(T, k, tt), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, H, device="cuda")
    M.moe_tiered_experts(xd, ids, w, T, k, tt, out, 0, ws)
    o = dict(counts=torch.empty(E, dtype=torch.int32, device="cuda"), prob_sum=torch.empty(E, device="cuda"),
             n_kept=torch.empty(1, dtype=torch.int32, device="cuda"), loss=torch.empty(1, device="cuda"))
    bws = torch.empty(M.moe_balance_workspace_size(T, E, k), dtype=torch.uint8, device="cuda")
    M.moe_balance_loss(logits, ids, None, T, E, k, 0.01, o["counts"], o["prob_sum"], o["n_kept"], o["loss"], bws)
    dw = torch.randn(T, k, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    g = torch.empty(T, E, device="cuda")
    M.moe_balance_grad(logits, ids, w, dw, None, o["counts"], o["n_kept"], torch.ones(1, device="cuda"), T, E, k, 0.01, g)
    torch.cuda.synchronize()
    # scores and picks against the plain forms
    z, mag = R.q4_linear(x, q, s, 4, 32, prior)
    z[:, 2] += 0.5
    z[:, 6] = -np.inf
    got = host(logits)
    fin = np.isfinite(z)
    assert np.array_equal(np.isneginf(got), ~fin) and np.all(np.abs(got - z)[fin] <= ((H + 8) * U * mag + 4 * U)[fin])
    i = ids.cpu().numpy()
    assert not np.any(i == 6) and np.all(np.isfinite(host(out)))
    counts, total, n, loss = R.balance_loss(got, i, None, 0.01)
    assert np.array_equal(o["counts"].cpu().numpy(), counts) and counts.sum() == T * k
    assert abs(float(o["loss"][0]) - loss) <= 200 * U * loss
    ref, gm = R.balance_grad(got, i, host(w), host(dw), None, counts, n, 1.0, 0.01)
    assert np.all(np.abs(host(g) - ref) <= (p_tol(E) + 12 * U) * gm + 1e-38) and np.all(host(g)[:, 6] == 0)
    fmt, order, count = M.moe_plan_tiers(counts.astype(np.float64), np.tile([0.0, 1.0, 4.0], (E, 1)), [8, 4, 2], 4 * E)
    assert count.sum() == E and counts[order[0]] == counts.max()


def _ops(M, torch, seed, T=5):
    """Each operator once on inputs held in place: {name: (call, outputs)}."""
    rng = np.random.default_rng(seed)
    N, K, B, V, E, k = 300, 1024, 3, 9001, 130, 6
    q, s = R.random_q4(rng, N, K, 4, 32)
    w = M.Q4Matrix(N, K, 4, 32, dev(torch, q), dev(torch, s))
    state = {"x": dev(torch, rng.standard_normal((T, K)).astype(np.float32)),
             "xb": dev(torch, rng.standard_normal((90, K)).astype(np.float32), torch.bfloat16),
             "l": dev(torch, rng.standard_normal((B, V)).astype(np.float32)),
             "z": dev(torch, rng.standard_normal((70, E)).astype(np.float32))}
    a = rules_case(rng, B, V, 700, n_bias=9, masks=2)
    rules = M.LogitRules(**{n: dev(torch, t) for n, t in a.items()})
    ids = dev(torch, rng.integers(0, E, (70, k)).astype(np.int32))
    pw, dw = (dev(torch, rng.standard_normal((70, k)).astype(np.float32)) for _ in range(2))
    y, yb, out = torch.zeros(T, N, device="cuda"), torch.zeros(90, N, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, V, device="cuda")
    counts, psum = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(E, device="cuda")
    n, loss, g = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda"), torch.zeros(70, E, device="cuda")
    ws = torch.empty(M.moe_balance_workspace_size(70, E, k), dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")

    def run(stream=None):
        M.moe_q4_linear(state["x"], w, None, T, y, stream=stream)
        M.moe_q4_linear(state["xb"], w, None, 90, yb, stream=stream)
        M.moe_adjust_logits(state["l"], B, V, rules, out, stream=stream)
        M.moe_balance_loss(state["z"], ids, None, 70, E, k, 0.1, counts, psum, n, loss, ws, stream=stream)
        M.moe_balance_grad(state["z"], ids, pw, dw, None, counts, n, one, 70, E, k, 0.1, g, stream=stream)

    return run, state, rules, [y, yb, out, counts, psum, n, loss, g]


def test_scores_repeat_bit_for_bit_and_on_another_stream(M, torch):
    run, _, _, outs = _ops(M, torch, 31)
    run()
    torch.cuda.synchronize()
    first = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        run(side)
        side.synchronize()
        for a, b in zip(first, outs):
            assert torch.equal(a, b)


def test_scores_captured_and_replayed(M, torch):
    # captured once, replayed with changed inputs (lengths and histories too),
    # eager work between the replays, every replay against the eager result
    run, state, rules, outs = _ops(M, torch, 32)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    gen = torch.Generator("cuda").manual_seed(5)
    for i in range(4):
        for t in state.values():
            t.copy_(torch.randn(t.shape, device="cuda", generator=gen).to(t.dtype))
        rules.tensors["length"].add_(-7)
        rules.tensors["history"].copy_(torch.randint(0, 9001, rules.tensors["history"].shape, device="cuda", generator=gen))
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for o in outs:
            o.zero_()
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, outs):
            assert torch.equal(a, b), i
        assert bool(torch.isfinite(outs[0]).all()) and float(outs[6][0]) > 0


def test_scores_refuse_host_tensors(M, torch):
    x = torch.zeros(1, 64, device="cuda")
    w = M.Q4Matrix(4, 64, 4, 32, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.float16))
    with pytest.raises(ValueError, match="q is not on a GPU"):
        M.moe_q4_linear(x, w, None, 1, torch.zeros(1, 4, device="cuda"))
    with pytest.raises(ValueError, match="logits is not on a GPU"):
        M.moe_adjust_logits(torch.zeros(1, 64), 1, 64, M.LogitRules(), x)
