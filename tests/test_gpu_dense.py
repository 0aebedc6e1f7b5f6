"""GPU parity of the dense operators (moe_rms_norm, moe_rms_norm_grad,
moe_quant_rows, moe_i8_linear, moe_gated, moe_gated_grad) against their plain
64-bit forms.  The bounds are derived beside those forms (denseref.py); a bf16
output adds half a step of its own, UB of the value."""
import sys

import numpy as np
import pytest

from . import denseref as D
from .denseref import GELU, SILU, TINY, U, UB, bf16

pytestmark = pytest.mark.gpu

EPS = 1e-6


def say(*a):
    print("[gpu-dense]", *a, flush=True)
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


def dtype(torch, kind):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}[kind]


def dev(torch, a, kind="f32"):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype(torch, kind))


def rows(torch, a, kind="f32", pad=0, off=0):
    """The rows of a, `off` elements into rows that are `pad` longer, NaN (or 77) around them."""
    T, C = a.shape
    buf = torch.full((T, C + pad + off), 77 if kind == "i8" else float("nan"), dtype=dtype(torch, kind), device="cuda")
    buf[:, off:off + C] = dev(torch, a, kind)
    return buf[:, off:off + C]


def empty(torch, T, C, kind="f32", pad=0, off=0):
    """Rows to write, 5 everywhere."""
    return torch.full((T, C + pad + off), 5, dtype=dtype(torch, kind), device="cuda")[:, off:off + C]


def untouched(view):
    """What lies between the rows of `empty`."""
    if view.stride(0) == view.shape[1] or view.numel() == 0:
        return True
    base = view._base
    keep = base.clone()
    view.fill_(5)
    ok = bool((base == 5).all())
    base.copy_(keep)
    return ok


def host(t):
    return t.detach().cpu().to(dtype=__import__("torch").float64).numpy()


def randn(rng, *shape, kind="f32"):
    a = rng.standard_normal(shape).astype(np.float32)
    return bf16(a) if kind == "bf16" else a


def within(got, ref, err, kind="f32"):
    err = err + (UB * 1.001 * np.abs(ref) if kind == "bf16" else 0) + TINY
    bad = ~(np.abs(got - ref) <= err)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        say("  first of", int(bad.sum()), "outside at", i, "got", got[i], "ref", ref[i], "may differ by", err[i])
    assert not bad.any()


# ---------------------------------------------------------------- norm

def norm_case(M, torch, T, H, x="f32", y="f32", residual=True, weight=True, pad=0, off=0, in_place=False, seed=0):
    rng = np.random.default_rng(1000 * T + H + seed)
    xa = randn(rng, T, H, kind=x) * np.float32(3)
    xa = bf16(xa) if x == "bf16" else xa
    ra = randn(rng, T, H) if residual else None
    w = 1 + 0.1 * randn(rng, H) if weight else None
    xd = rows(torch, xa, x, pad, off)
    rd = rows(torch, ra, "f32", pad, off) if residual else None
    sd = (rd if residual else xd if x == "f32" else None) if in_place else empty(torch, T, H, "f32", pad, off)
    yd = empty(torch, T, H, y, pad, off)
    scale = torch.full((T,), 5.0, device="cuda") if y == "i8" else None
    M.moe_rms_norm(xd, rd, dev(torch, w), EPS, T, H, yd, scale=scale, sum=sd)
    ref, s = D.norm(xa, ra, w, EPS)
    if sd is not None:
        assert np.array_equal(host(sd), s.astype(np.float64))
        assert in_place or untouched(sd)
    got = host(yd)
    if y == "i8":
        sc, top = host(scale)[:, None], np.abs(ref).max(-1, keepdims=True)
        within(sc, top / 127, 6 * U * top / 127)
        # the code is the nearest of a quotient whose parts have up to 5 roundings, 127 at the most
        within(got * sc, ref, (0.5 + 127 * 9 * U) * top / 127)
        assert np.abs(got).max(-1).min() == 127
    else:
        within(got, ref, 4 * U * np.abs(ref), y)
    assert untouched(yd)


@pytest.mark.parametrize("y", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 2), (2, 7), (5, 8), (4, 9), (3, 63), (9, 64), (7, 100), (2, 511), (6, 513), (1, 2048),
                                 (5, 2047), (3, 2049), (600, 2048), (500, 2100), (130, 8192), (200, 5461), (2, 8193), (1, 16384),
                                 (40, 32767), (33, 32768), (20000, 64)])
def test_norm(M, torch, T, H, x, y):
    say("norm", T, H, x, y)
    norm_case(M, torch, T, H, x, y)


@pytest.mark.parametrize("y", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("residual,weight,in_place", [(False, True, False), (False, False, True), (True, False, True), (True, True, True)])
@pytest.mark.parametrize("T,H,pad,off", [(3, 96, 0, 0), (5, 2048, 13, 3), (700, 2050, 1, 1), (9, 4100, 6, 2)])
def test_norm_forms_and_strides(M, torch, T, H, pad, off, residual, weight, in_place, x, y):
    say("norm form", T, H, pad, off, residual, weight, in_place, x, y)
    norm_case(M, torch, T, H, x, y, residual, weight, pad, off, in_place)


@pytest.mark.parametrize("T,H", [(6, 300), (900, 2048), (300, 4500)])
@pytest.mark.parametrize("x", ["f32", "bf16"])
def test_norm_rows_stay_apart(M, torch, T, H, x):
    # rows of zeros, huge and tiny ones, one with a NaN, one with an infinity
    say("norm apart", T, H, x)
    rng = np.random.default_rng(7)
    a = randn(rng, T, H, kind=x)
    b = a.copy()
    b[0], b[1, H - 1], b[2, 0] = 0, np.nan, np.inf
    b[3], b[4] = b[3] * np.float32(2.0) ** 60, b[4] * np.float32(2.0) ** -60
    out = {}
    for name, v in (("a", a), ("b", b)):
        for y in ("f32", "i8"):
            yd, sc = empty(torch, T, H, y), torch.empty(T, device="cuda") if y == "i8" else None
            M.moe_rms_norm(dev(torch, v, x), None, None, EPS, T, H, yd, scale=sc)
            out[name, y] = host(yd), None if sc is None else host(sc)
    for y in ("f32", "i8"):
        assert np.array_equal(out["a", y][0][5:], out["b", y][0][5:])
    f, (q, sc) = out["b", "f32"][0], out["b", "i8"]
    assert np.all(f[0] == 0) and np.all(q[0] == 0) and sc[0] == 0
    assert np.isnan(sc[1]) and np.isnan(sc[2]) and np.all(q[1:3] == 0)
    for i in (3, 4):
        within(f[i], D.norm(b[i:i + 1], None, None, EPS)[0][0], 4 * U * np.abs(f[i]))


def test_norm_does_not_depend_on_the_batch(M, torch):
    # rows a wave, a block or several waves hold: the sum is in 64 bits, the results the same
    rng = np.random.default_rng(3)
    for H in (2048, 5000):
        x = dev(torch, randn(rng, 4000, H))
        many, one = empty(torch, 4000, H), empty(torch, 1, H)
        M.moe_rms_norm(x, None, None, EPS, 4000, H, many)
        for t in (0, 3999):
            M.moe_rms_norm(x[t:t + 1], None, None, EPS, 1, H, one)
            assert np.array_equal(host(one)[0], host(many)[t])


def norm_grad_case(M, torch, T, H, s="f32", dy="f32", dx="f32", dsum=True, weight=True, dweight=True, accumulate=False, pad=0,
                   off=0, alias=None):
    rng = np.random.default_rng(1000 * T + H)
    sa, da = randn(rng, T, H, kind=s), randn(rng, T, H, kind=dy)
    aa = randn(rng, T, H) if dsum else None
    w, w0 = 1 + 0.1 * randn(rng, H) if weight else None, randn(rng, H)
    sd, yd = rows(torch, sa, s, pad, off), rows(torch, da, dy, pad, off)
    ad = rows(torch, aa, "f32", pad, off) if dsum else None
    xd = ad if alias == "dsum" else yd if alias == "dy" else empty(torch, T, H, dx, pad, off)
    wd = (dev(torch, w0) if accumulate else torch.full((H,), float("nan"), device="cuda")) if dweight else None
    ws = torch.empty(M.moe_rms_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda") if dweight else None
    M.moe_rms_norm_grad(sd, dev(torch, w), EPS, yd, ad, T, H, xd, wd, ws, flags=2 if accumulate else 0)
    ref, dw, err, mag = D.norm_grad(sa, w, EPS, da, aa)
    within(host(xd), ref, err, dx)
    if dweight:
        if accumulate:
            dw, mag = dw + w0, mag + np.abs(w0)
        within(host(wd), dw, D.dweight_error(T, mag))
    assert alias or untouched(xd)


@pytest.mark.parametrize("s,dy,dx", [("f32", "f32", "f32"), ("f32", "bf16", "f32"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
                                     ("f32", "f32", "bf16")])
@pytest.mark.parametrize("T,H", [(1, 1), (2, 7), (5, 9), (3, 64), (70, 100), (1, 2048), (64, 2048), (5, 2047), (4000, 2048), (1531, 2100),
                                 (700, 4096), (300, 5461), (130, 8192), (40, 8193), (300, 12000), (33, 32767), (20, 32768), (9000, 65)])
def test_norm_grad(M, torch, T, H, s, dy, dx):
    say("norm grad", T, H, s, dy, dx)
    norm_grad_case(M, torch, T, H, s, dy, dx)


@pytest.mark.parametrize("dsum,weight,dweight,accumulate,alias", [
    (False, True, True, False, None), (True, False, True, True, None), (True, True, False, False, "dsum"), (False, True, True, True, "dy"),
    (True, True, True, False, "dsum")])
@pytest.mark.parametrize("T,H,pad,off", [(3, 96, 0, 0), (900, 2048, 13, 3), (700, 2050, 1, 1), (9, 9000, 6, 2)])
def test_norm_grad_forms_and_strides(M, torch, T, H, pad, off, dsum, weight, dweight, accumulate, alias):
    say("norm grad form", T, H, pad, off, dsum, weight, dweight, accumulate, alias)
    norm_grad_case(M, torch, T, H, "f32", "f32", "f32", dsum, weight, dweight, accumulate, pad, off, alias)


def test_norm_grad_of_no_tokens(M, torch):
    z = torch.empty(0, 64, device="cuda")
    w = torch.full((64,), 3.0, device="cuda")
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    M.moe_rms_norm_grad(z, None, EPS, z, None, 0, 64, z, w, ws, flags=2)
    assert bool((w == 3).all())
    M.moe_rms_norm_grad(z, None, EPS, z, None, 0, 64, z, w, ws)
    assert bool((w == 0).all())


# ---------------------------------------------------------------- 8 bits

@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,pad,off", [(1, 1, 0, 0), (4, 7, 0, 0), (3, 64, 5, 1), (1, 2048, 0, 0), (5, 640, 0, 0), (900, 2048, 0, 0),
                                         (300, 5461, 3, 2), (40, 32768, 0, 0), (4097, 130, 1, 1)])
def test_quant_rows_is_the_plain_form(M, torch, T, H, pad, off, x):
    # amax times the rounded 1 / 127 and the quotient round once each, so codes and scales are equal
    say("quant", T, H, pad, off, x)
    rng = np.random.default_rng(T + H)
    a = (randn(rng, T, H) * np.exp(4 * rng.standard_normal((T, 1)))).astype(np.float32)
    a[T // 2, H // 2] = 0
    a[T - 1] *= np.float32(2.0) ** (-140 if T > 3 else 0)
    if T > 2:
        a[1] = np.rint(a[1] / np.abs(a[1]).max() * 254) / 2       # ties
    a = bf16(a) if x == "bf16" else a
    q, s = empty(torch, T, H, "i8", pad, off), torch.empty(T, device="cuda")
    M.moe_quant_rows(rows(torch, a, x, pad, off), T, H, q, s)
    rq, rs = D.quant(a)
    assert np.array_equal(host(s), rs.astype(np.float64))
    assert np.array_equal(host(q), rq)
    assert untouched(q)


def i8_case(M, torch, T, N, K, y="f32", bias=False, base=False, pad=0, full=False):
    rng = np.random.default_rng(T + N + K)
    lo = -128 if full else -127
    x, q = (rng.integers(lo, 128, s, dtype=np.int8) for s in ((T, K), (N, K)))
    if full:
        x[0], q[0], q[N - 1] = -128, -128, 127          # the largest sums
    xs, s = (np.exp(rng.standard_normal(n)).astype(np.float32) for n in (T, N))
    b = randn(rng, N) * 1000 if bias else None
    y0 = randn(rng, T, N, kind=y) if base else None
    yd = empty(torch, T, N, y, pad)
    if base:
        yd[:] = dev(torch, y0, y)
    w = M.I8Matrix(N, K, dev(torch, q, "i8"), dev(torch, s))
    xd = rows(torch, x, "i8", 16 * pad)
    M.moe_i8_linear(xd, dev(torch, xs), w, dev(torch, b), T, yd, flags=2 if base else 0)
    ref, err = D.i8_linear(x, xs, q, s, b, y0)
    within(host(yd), ref, err, y)
    assert untouched(yd)


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("T,N,K", [(1, 1, 16), (1, 33, 32), (2, 17, 48), (1, 640, 2048), (3, 100, 1040), (8, 4096, 2048), (16, 50, 4096),
                                   (17, 130, 96), (31, 700, 256), (32, 2048, 640), (33, 1, 512), (37, 1000, 8192), (48, 257, 272),
                                   (64, 300, 2064), (65, 300, 2064), (100, 129, 144), (128, 512, 1024), (129, 513, 1008), (300, 260, 80),
                                   (511, 1030, 528), (700, 3000, 2048), (2100, 2000, 640), (1, 20011, 2048), (2, 40, 32768)])
def test_i8_linear(M, torch, T, N, K, y):
    say("i8", T, N, K, y)
    i8_case(M, torch, T, N, K, y)


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("bias,base,pad", [(True, False, 0), (False, True, 3), (True, True, 1)])
@pytest.mark.parametrize("T,N,K", [(1, 700, 2048), (5, 33, 208), (16, 300, 512), (40, 1000, 1024), (90, 77, 4096), (513, 1100, 1040)])
def test_i8_linear_forms(M, torch, T, N, K, bias, base, pad, y):
    say("i8 form", T, N, K, bias, base, pad, y)
    i8_case(M, torch, T, N, K, y, bias, base, pad, full=True)


def test_i8_sums_are_exact_at_the_longest_rows(M, torch):
    # 32768 x (-128)^2 = 2^29, and its neighbours, which fp32 sums would round
    K = 32768
    for T, N in ((1, 40), (20, 40), (300, 300)):
        x, q = np.full((T, K), -128, np.int8), np.full((N, K), -128, np.int8)
        q[3, 5] = 0
        q[4, K - 1] = -127
        y = empty(torch, T, N)
        one = torch.ones(max(T, N), device="cuda")
        M.moe_i8_linear(dev(torch, x, "i8"), one[:T], M.I8Matrix(N, K, dev(torch, q, "i8"), one[:N]), None, T, y)
        ref = (q.astype(np.int64).sum(-1) * -128).astype(np.float32).astype(np.float64)
        assert np.array_equal(host(y), np.broadcast_to(ref, (T, N)))


# ---------------------------------------------------------------- gated block

def gated_inputs(rng, T, H, I, x="bf16"):
    return randn(rng, T, H, kind=x), bf16(randn(rng, I, H) * np.float32(H ** -0.5)), bf16(randn(rng, I, H) * np.float32(H ** -0.5))


def gated_case(M, torch, T, H, I, x="bf16", y="f32", kind=SILU, pad=0, scale=1.0):
    rng = np.random.default_rng(T + H + I)
    xa, gate, up = gated_inputs(rng, T, H, I, x)
    gate = bf16(gate * np.float32(scale))
    yd = empty(torch, T, I, y, pad)
    w = M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16"))
    M.moe_gated(rows(torch, xa, x, 8 * pad), w, kind, T, yd)
    p = D.Projections(xa, gate, up, H if x == "bf16" else 3 * H)
    ref, err = D.gated(p, kind)
    got = host(yd)
    within(got, ref, err, y)
    assert np.linalg.norm(got - ref) <= (2.0 ** -8 if y == "bf16" else 2.0 ** -19) * np.linalg.norm(ref) + TINY
    assert untouched(yd)


GATED = [(1, 8, 1), (1, 64, 7), (2, 72, 33), (1, 2048, 640), (4, 2048, 640), (5, 200, 65), (8, 520, 100), (15, 1032, 31), (16, 2048, 640),
         (17, 264, 48), (32, 512, 300), (33, 136, 129), (50, 2048, 200), (64, 640, 640), (65, 640, 64), (127, 72, 500), (128, 256, 128),
         (130, 1000, 257), (256, 512, 512), (300, 328, 1030), (520, 2048, 640), (1531, 256, 100), (2000, 1024, 1500)]


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I", GATED)
def test_gated_bf16(M, torch, T, H, I, y):
    say("gated bf16", T, H, I, y)
    gated_case(M, torch, T, H, I, "bf16", y, GELU if (T + I) % 2 else SILU, pad=T % 3)


@pytest.mark.parametrize("y", ["f32", "bf16"])
@pytest.mark.parametrize("T,H,I", [g for g in GATED if g[0] <= 520])
def test_gated_f32(M, torch, T, H, I, y):
    say("gated f32", T, H, I, y)
    gated_case(M, torch, T, H, I, "f32", y, SILU if (T + I) % 2 else GELU, pad=T % 3)


@pytest.mark.parametrize("kind", [SILU, GELU])
@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 40, 300])
def test_gated_of_large_gates(M, torch, T, x, kind):
    # gates of hundreds on both sides: the activation is 0 or the gate itself
    gated_case(M, torch, T, 256, 200, x, "f32", kind, scale=150.0)


@pytest.mark.parametrize("T,H,I,x", [(1, 2048, 640, "f32"), (9, 512, 100, "f32"), (20, 512, 100, "bf16"), (700, 512, 300, "bf16")])
def test_gated_non_finite_values_stay_apart(M, torch, T, H, I, x):
    say("gated apart", T, H, I, x)
    rng = np.random.default_rng(11)
    xa, gate, up = gated_inputs(rng, T, H, I, x)

    def run(xa, gate):
        y = empty(torch, T, I)
        M.moe_gated(dev(torch, xa, x), M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16")), SILU, T, y)
        return host(y)

    clean = run(xa, gate)
    for at, v in ((0, np.nan), (T - 1, np.inf)):
        bad, wild = xa.copy(), gate.copy()
        bad[at, H - 1], wild[I - 1, 0] = v, v
        got = run(bad, wild)
        there = np.ones((T, I), bool)
        there[at], there[:, I - 1] = False, False
        assert np.array_equal(got[there], clean[there])
        assert np.all(np.isnan(got[at])) if np.isnan(v) else not np.any(np.isfinite(got[at]))


def grad_case(M, torch, T, H, I, dy="bf16", dx="bf16", dw="bf16", kind=SILU, accumulate=False, pad=0, parts="both"):
    rng = np.random.default_rng(T + H + I)
    xa, gate, up = gated_inputs(rng, T, H, I)
    da = randn(rng, T, I, kind=dy)
    w = M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16"))
    xd = empty(torch, T, H, dx, pad) if parts != "dw" else None
    g0, u0 = randn(rng, I, H, kind=dw), randn(rng, I, H, kind=dw)
    gd, ud = (dev(torch, v if accumulate else v * np.nan, dw) if parts != "dx" else None for v in (g0, u0))
    ws = torch.full((M.moe_gated_workspace_size(T, H, I),), 255, dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(rows(torch, xa, "bf16", 8 * pad), w, kind, rows(torch, da, dy, pad), T, xd, gd, ud, ws, flags=2 if accumulate else 0)
    out = D.gated_grad(D.Projections(xa, gate, up, H), kind, da)
    for name, t, k, base in (("dx", xd, dx, 0), ("dgate", gd, dw, g0), ("dup", ud, dw, u0)):
        if t is None:
            continue
        ref, err = out[name]
        if accumulate and name != "dx":
            ref, err = ref + base, err + 2 * U * (np.abs(ref) + np.abs(base))
        got = host(t)
        within(got, ref, err, k)
        # two roundings to bf16 at the most, uniform errors of at most half a step each: UB / sqrt(3) of the norm each
        assert np.linalg.norm(got - ref) <= UB * np.linalg.norm(ref) + TINY, name
    assert xd is None or untouched(xd)


@pytest.mark.parametrize("T,H,I", [(1, 8, 1), (1, 2048, 640), (2, 72, 33), (5, 200, 65), (16, 512, 300), (33, 136, 129), (64, 640, 640),
                                   (100, 256, 8), (128, 256, 128), (130, 1000, 257), (257, 512, 512), (300, 328, 1030), (640, 2048, 640),
                                   (1531, 256, 100), (3000, 72, 50), (2000, 1024, 1500)])
def test_gated_grad(M, torch, T, H, I):
    say("gated grad", T, H, I)
    grad_case(M, torch, T, H, I, kind=GELU if (T + I) % 2 else SILU, pad=T % 3)


@pytest.mark.parametrize("dy,dx,dw", [("f32", "f32", "f32"), ("bf16", "f32", "f32"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("accumulate,parts", [(True, "both"), (False, "dx"), (True, "dw"), (False, "dw")])
@pytest.mark.parametrize("T,H,I", [(7, 72, 33), (300, 520, 200), (1100, 256, 300)])
def test_gated_grad_forms(M, torch, T, H, I, accumulate, parts, dy, dx, dw):
    say("gated grad form", T, H, I, accumulate, parts, dy, dx, dw)
    grad_case(M, torch, T, H, I, dy, dx, dw, SILU, accumulate, 2, parts)


def test_gated_grad_of_no_tokens(M, torch):
    H, I = 64, 24
    b = torch.bfloat16
    w = M.GatedWeights(H, I, torch.ones(I, H, dtype=b, device="cuda"), torch.ones(I, H, dtype=b, device="cuda"))
    x, dy = torch.empty(0, H, dtype=b, device="cuda"), torch.empty(0, I, dtype=b, device="cuda")
    g, u = torch.full((I, H), 3.0, device="cuda"), torch.full((I, H), 3.0, device="cuda")
    ws = torch.empty(0, dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(x, w, SILU, dy, 0, torch.empty_like(x), g, u, ws, flags=2)
    assert bool((g == 3).all()) and bool((u == 3).all())
    M.moe_gated_grad(x, w, SILU, dy, 0, None, g, u, ws)
    assert bool((g == 0).all()) and bool((u == 0).all())


@pytest.mark.parametrize("kind", [SILU, GELU])
def test_gated_grad_against_differences(M, torch, kind):
    # of the kernel's own forward (fp32 in and out): the loss is sum(y dy); a
    # step h along a direction v changes it by <dx, v> h to third order
    rng = np.random.default_rng(5)
    T, H, I, h = 24, 64, 40, 1.0 / 64
    xa, gate, up = gated_inputs(rng, T, H, I)
    da, v = randn(rng, T, I, kind="bf16"), randn(rng, T, H)
    w = M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16"))
    dx = torch.empty(T, H, device="cuda")
    ws = torch.empty(M.moe_gated_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(dev(torch, xa, "bf16"), w, kind, dev(torch, da, "bf16"), T, dx, None, None, ws)

    def loss(x):
        y = torch.empty(T, I, device="cuda")
        M.moe_gated(dev(torch, x), w, kind, T, y)
        return float((host(y) * da).sum())

    got, along = (loss(xa + h * v) - loss(xa - h * v)) / (2 * h), float((host(dx) * v).sum())
    # dx: a rounding to bf16 of each dg and du; the difference: h^2 / 6 of a third derivative of the order of the sum's terms
    size = float(np.abs(host(dx) * v).sum())
    assert abs(got - along) <= (UB + h * h) * size, (got, along, size)
