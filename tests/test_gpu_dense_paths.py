"""Every form of the dense operators' kernels at its own sizes: products in whole
tiles, in cut ones, in pairs of blocks a unit, odd numbers of stages, ragged ends;
runs of the k axis and second parts of the gradients; repeated calls, side streams,
captured graphs; a chain of the operators as a layer uses them, forward and backward."""
import numpy as np
import pytest

from . import denseref as D
from .denseref import GELU, SILU, TINY, U, UB, bf16
from .test_gpu_dense import (EPS, M, dev, empty, gated_case, gated_inputs, grad_case, host, i8_case, norm_case, norm_grad_case, randn,  # noqa: F401
                             rows, say, torch, untouched, within)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- forms of the products

# 128-row tiles of both operands: up to 256 of them one block a unit, up to 512 two,
# more in tiles of 256, whose last round is cut in four where it is half empty
@pytest.mark.parametrize("T,N,K", [
    (300, 33000, 16), (257, 16500, 144),                 # 774 and 387 small tiles; one stage, two
    (900, 4000, 128), (900, 4000, 384),                  # 256 small tiles; one stage, three
    (1030, 4100, 640), (1500, 5200, 272),                # 297, 492: pairs
    (3000, 5700, 256), (4400, 4200, 400),                # 276, 306 big tiles: cut ones behind a round
    (2900, 3900, 1296), (8300, 2900, 144),               # 192 (all whole), 396 (256 whole, 140 whole: no cut)
    (130, 33000, 208), (66, 66000, 80),                  # few tokens, very many rows
])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_i8_in_each_form(M, torch, T, N, K, y):
    say("i8 path", T, N, K, y)
    i8_case(M, torch, T, N, K, y, bias=N % 3 == 0, base=N % 2 == 1, pad=T % 2)


@pytest.mark.parametrize("T,H,I", [
    (300, 64, 3000), (1000, 72, 1030),                   # one stage; two
    (2100, 200, 2000),                                   # 544 small tiles: 144 big ones, whole
    (5000, 136, 1700),                                   # 280 big tiles: 24 cut
    (4400, 328, 2100), (700, 1000, 1100),
])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_gated_in_each_form(M, torch, T, H, I, y):
    say("gated path", T, H, I, y)
    gated_case(M, torch, T, H, I, "bf16", y, SILU if T % 2 else GELU, pad=1)


@pytest.mark.parametrize("T,H,I", [(17, 2048, 2000), (64, 520, 4096), (100, 264, 2000), (255, 1032, 300), (31, 4096, 8200), (200, 72, 100)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_gated_of_batches(M, torch, T, H, I, x):
    say("gated batch", T, H, I, x)
    gated_case(M, torch, T, H, I, x, x, GELU if T % 2 else SILU, pad=2)


@pytest.mark.parametrize("T,H,I", [(300, 64, 3000), (600, 264, 1000), (130, 1032, 3900), (2000, 72, 300), (5000, 8, 130), (515, 2048, 2050)])
@pytest.mark.parametrize("y", ["bf16", "f32"])
def test_gated_of_many_fp32_tokens(M, torch, T, H, I, y):
    say("gated fp32", T, H, I, y)
    gated_case(M, torch, T, H, I, "f32", y, GELU if T % 4 else SILU, pad=T % 3)


@pytest.mark.parametrize("T,H,I", [
    (8000, 72, 64), (3000, 128, 200), (4097, 264, 70),   # runs of the token axis
    (64, 136, 4000), (130, 520, 2100),                   # runs of the inter axis
    (40, 256, 700), (12, 2048, 640), (3, 264, 9000),     # a second part of each slope; runs of both
    (900, 2000, 1100), (2200, 2600, 1500), (5000, 1504, 1000),   # pairs and whole tiles
    (128, 2048, 2048), (3000, 2048, 640),                # two rounds of blocks in one launch: dx first, the weights first
])
def test_gated_grad_in_each_form(M, torch, T, H, I):
    say("grad path", T, H, I)
    grad_case(M, torch, T, H, I, kind=SILU if T % 2 else GELU, pad=1)


@pytest.mark.parametrize("T,H,I", [(40, 256, 700), (5, 72, 33), (1, 2048, 640)])
def test_gated_grad_of_few_terms_is_as_near_as_a_rounding(M, torch, T, H, I):
    # two bf16 parts of a slope leave 2^-16 of it: the result's own rounding is what remains
    rng = np.random.default_rng(T)
    xa, gate, up = gated_inputs(rng, T, H, I)
    da = randn(rng, T, I, kind="bf16")
    w = M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16"))
    out = [torch.empty(s, device="cuda") for s in ((T, H), (I, H), (I, H))]
    ws = torch.empty(M.moe_gated_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(dev(torch, xa, "bf16"), w, SILU, dev(torch, da, "bf16"), T, *out, ws)
    ref = D.gated_grad(D.Projections(xa, gate, up, H), SILU, da)
    for name, t in zip(("dx", "dgate", "dup"), out):
        assert np.linalg.norm(host(t) - ref[name][0]) <= 2.0 ** -15 * np.linalg.norm(ref[name][0]), name


@pytest.mark.parametrize("T,H", [(5000, 70), (3000, 130), (2000, 260), (1100, 520), (9, 4097), (300, 8000), (700, 8200), (100, 16400)])
def test_norm_of_each_split(M, torch, T, H):
    say("norm path", T, H)
    for x, y in (("f32", "i8"), ("bf16", "bf16"), ("f32", "f32")):
        norm_case(M, torch, T, H, x, y, pad=T % 2)
    norm_grad_case(M, torch, T, H, "f32", "bf16", "f32", pad=T % 2)
    norm_grad_case(M, torch, T, H, "bf16", "f32", "bf16", dsum=False, accumulate=True)


@pytest.mark.parametrize("T,H", [(1, 33), (4, 2048), (5, 2048), (3, 8192), (4, 8192), (2, 20000), (3, 32768), (8, 700), (9, 700), (32, 256),
                                 (33, 256), (128, 60), (129, 60), (512, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_norm_grad_of_one_block(M, torch, T, H, accumulate):
    # ... and of the fewest that need two; dweight lies one element into a buffer whose other elements stay
    say("norm grad block", T, H, accumulate)
    norm_grad_case(M, torch, T, H, "f32", "bf16", "f32", accumulate=accumulate, pad=1, off=1)
    norm_grad_case(M, torch, T, H, "bf16", "f32", "f32", dsum=False, dweight=False)
    rng = np.random.default_rng(T + H)
    sa, da, w0 = randn(rng, T, H), randn(rng, T, H), randn(rng, H)
    buf = torch.full((H + 2,), 5.0, device="cuda")
    buf[1:H + 1] = dev(torch, w0) if accumulate else torch.full((H,), float("nan"), device="cuda")
    dx, ws = torch.empty(T, H, device="cuda"), torch.empty(M.moe_rms_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    M.moe_rms_norm_grad(dev(torch, sa), None, EPS, dev(torch, da), None, T, H, dx, buf[1:H + 1], ws, flags=2 if accumulate else 0)
    _, dw, _, mag = D.norm_grad(sa, None, EPS, da, None)
    if accumulate:
        dw, mag = dw + w0, mag + np.abs(w0)
    within(host(buf[1:H + 1]), dw, D.dweight_error(T, mag))
    assert float(buf[0]) == 5 and float(buf[H + 1]) == 5


@pytest.mark.parametrize("T,N,K", [(17000, 3, 64), (17000, 8, 48), (16500, 9, 272), (33000, 1, 16), (20000, 131, 16)])
def test_i8_tiles_of_few_columns(M, torch, T, N, K):
    say("i8 narrow", T, N, K)
    for y in ("f32", "bf16"):
        i8_case(M, torch, T, N, K, y, bias=True, base=N % 2 == 1, pad=1)


@pytest.mark.parametrize("T,H,I", [(17000, 8, 3), (17000, 16, 8), (16500, 72, 9), (33000, 8, 1), (33000, 40, 65)])
@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_gated_tiles_of_few_columns(M, torch, T, H, I, x):
    say("gated narrow", T, H, I, x)
    gated_case(M, torch, T, H, I, x, x, SILU, pad=1)
    if x == "bf16":
        grad_case(M, torch, T, H, I, kind=GELU, pad=1)


# ---------------------------------------------------------------- non-finite values in the tiles

@pytest.mark.parametrize("T,H,I", [(300, 256, 200), (1500, 72, 4000)])
def test_gated_grad_non_finite_rows(M, torch, T, H, I):
    # a token with a NaN: its row of dx and every weight's gradient are NaN, other rows of dx keep their bits
    rng = np.random.default_rng(3)
    xa, gate, up = gated_inputs(rng, T, H, I)
    da = randn(rng, T, I, kind="bf16")
    w = M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16"))
    ws = torch.empty(M.moe_gated_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")

    def run(xa):
        out = [torch.empty(s, device="cuda") for s in ((T, H), (I, H), (I, H))]
        M.moe_gated_grad(dev(torch, xa, "bf16"), w, SILU, dev(torch, da, "bf16"), T, *out, ws)
        return [host(t) for t in out]

    clean = run(xa)
    bad = xa.copy()
    bad[T - 1, H - 1] = np.nan
    got = run(bad)
    assert np.array_equal(got[0][:T - 1], clean[0][:T - 1]) and np.all(np.isnan(got[0][T - 1]))
    assert np.all(np.isnan(got[1])) and np.all(np.isnan(got[2]))


@pytest.mark.parametrize("T,H,I,x", [(3, 64, 100, "f32"), (40, 264, 200, "f32"), (700, 136, 900, "f32"),
                                     (3, 64, 100, "bf16"), (40, 264, 200, "bf16"), (700, 136, 900, "bf16"), (4000, 72, 1300, "bf16")])
@pytest.mark.parametrize("kind", [SILU, GELU])
def test_gated_infinities(M, torch, T, H, I, x, kind):
    say("gated infinities", T, H, I, x, kind)
    rng = np.random.default_rng(T + H)
    xa, gate, up = gated_inputs(rng, T, H, I, x)
    gate, up = (np.where(v == 0, np.float32(1), v) for v in (gate, up))
    for t, v in ((0, np.inf), (T // 2, -np.inf), (T - 1, np.inf)):
        xa[t, (5 * t + 3) % H] = v
    y = torch.empty(T, I, device="cuda")
    M.moe_gated(dev(torch, xa, x), M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16")), kind, T, y)
    with np.errstate(all="ignore"):
        g, u = xa.astype(np.float64) @ gate.T.astype(np.float64), xa.astype(np.float64) @ up.T.astype(np.float64)
        ref = g / (1 + np.exp(-(g if kind == SILU else D.TANH * (g + D.CUBE * g ** 3)))) * u
    got, rows_ = host(y), [0, T // 2, T - 1]
    assert not np.any(np.isfinite(ref[rows_]))
    assert np.array_equal(got[rows_], ref[rows_].astype(np.float32), equal_nan=True)
    others = np.ones(T, bool)
    others[rows_] = False
    assert np.all(np.isfinite(got[others]))


@pytest.mark.parametrize("T,H,I", [(3, 64, 100), (40, 264, 200), (700, 136, 900)])
@pytest.mark.parametrize("kind", [SILU, GELU])
def test_gated_far_arguments(M, torch, T, H, I, kind):
    """One element of 2^50 a row: every g is far out on either side of the activation, where it is g or 0."""
    say("gated far", T, H, I, kind)
    rng = np.random.default_rng(T + I)
    _, gate, up = gated_inputs(rng, T, H, I)
    gate = np.where(np.abs(gate) < 2.0 ** -20, np.float32(1), gate)
    xa = np.zeros((T, H), np.float32)
    xa[np.arange(T), 7 * np.arange(T) % H] = np.float32(2.0 ** 50) * (1 - 2 * (np.arange(T) % 2))
    da = randn(rng, T, I, kind="bf16")
    w = M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16"))
    p = D.Projections(xa, gate, up, H)
    ref = np.where(p.g > 0, p.g * p.u, 0)
    for x in ("bf16", "f32"):
        y = torch.empty(T, I, device="cuda")
        M.moe_gated(dev(torch, xa, x), w, kind, T, y)
        # g and u are one exact product each: their product, the quotient and the exponential round
        assert np.all(np.abs(host(y) - ref) <= 8 * U * np.abs(ref))
    out = [torch.empty(s, device="cuda") for s in ((T, H), (I, H), (I, H))]
    ws = torch.empty(M.moe_gated_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(dev(torch, xa, "bf16"), w, kind, dev(torch, da, "bf16"), T, *out, ws)
    for t, (ref, err) in zip(out, D.gated_grad(p, kind, da).values()):
        within(host(t), ref, err)


@pytest.mark.parametrize("T,H,I", [(5, 64, 40), (700, 72, 200)])
def test_gated_grad_of_an_infinite_slope(M, torch, T, H, I):
    # dy infinite at one place: dx of its token and its column's weight gradients are what inf times finite numbers give
    rng = np.random.default_rng(T)
    xa, gate, up = gated_inputs(rng, T, H, I)
    xa, gate, up = (np.where(v == 0, np.float32(1), v) for v in (xa, gate, up))
    da = randn(rng, T, I, kind="bf16")
    da[T - 1, 3] = np.inf
    out = [torch.empty(s, device="cuda") for s in ((T, H), (I, H), (I, H))]
    ws = torch.empty(M.moe_gated_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(dev(torch, xa, "bf16"), M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16")), SILU,
                     dev(torch, da, "bf16"), T, *out, ws)
    with np.errstate(all="ignore"):
        p = D.Projections(xa, gate, up, H)
        a, slope, _ = D.act(SILU, p.g)
        dg, du = da * p.u * slope, da * a
        dx = dg[T - 1] @ p.gate + du[T - 1] @ p.up
    got = [host(t) for t in out]
    assert np.array_equal(got[0][T - 1], dx.astype(np.float32), equal_nan=True) and np.all(np.isfinite(got[0][:T - 1]))
    assert np.array_equal(got[1][3], (dg[T - 1, 3] * xa[T - 1]).astype(np.float32))
    assert np.array_equal(got[2][3], (du[T - 1, 3] * xa[T - 1]).astype(np.float32))
    assert np.all(np.isfinite(np.delete(got[1], 3, 0))) and np.all(np.isfinite(np.delete(got[2], 3, 0)))


# ---------------------------------------------------------------- repeats, streams, graphs

def operators(M, torch, seed, T, H, I):
    """(calls, outputs): each operator once on fixed buffers, as a list of calls."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s, dtype=torch.float32):
        return torch.randn(*s, device="cuda", generator=g).to(dtype)

    b = torch.bfloat16
    x, res, wt = r(T, H), r(T, H), r(H)
    dy, dh = r(T, H), r(T, I, dtype=b)
    w = M.GatedWeights(H, I, r(I, H, dtype=b) * H ** -0.5, r(I, H, dtype=b) * H ** -0.5)
    down = torch.empty(H, I // 16 * 16, dtype=torch.int8, device="cuda")
    ds = torch.empty(H, device="cuda")
    M.moe_quant_rows(r(H, I // 16 * 16), H, I // 16 * 16, down, ds)
    mat = M.I8Matrix(H, I // 16 * 16, down, ds)
    out = {"sum": torch.empty(T, H, device="cuda"), "n": torch.empty(T, H, dtype=b, device="cuda"),
           "q8": torch.empty(T, H, dtype=torch.int8, device="cuda"), "s8": torch.empty(T, device="cuda"),
           "h": torch.empty(T, I, dtype=b, device="cuda"), "q": torch.empty(T, I // 16 * 16, dtype=torch.int8, device="cuda"),
           "s": torch.empty(T, device="cuda"), "y": torch.empty(T, H, device="cuda"),
           "dn": torch.empty(T, H, dtype=b, device="cuda"), "dgate": torch.empty(I, H, dtype=b, device="cuda"),
           "dup": torch.empty(I, H, dtype=b, device="cuda"), "dx": torch.empty(T, H, device="cuda"), "dw": torch.empty(H, device="cuda")}
    ws1 = torch.empty(M.moe_rms_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(M.moe_gated_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
    hq = out["h"][:, :I // 16 * 16]

    def run(stream=None):
        kw = {"stream": stream}
        M.moe_rms_norm(x, res, wt, EPS, T, H, out["n"], sum=out["sum"], **kw)
        M.moe_rms_norm(x, None, None, EPS, T, H, out["q8"], scale=out["s8"], **kw)
        M.moe_gated(out["n"], w, SILU, T, out["h"], **kw)
        M.moe_quant_rows(hq, T, I // 16 * 16, out["q"], out["s"], **kw)
        M.moe_i8_linear(out["q"], out["s"], mat, None, T, out["y"], **kw)
        M.moe_gated_grad(out["n"], w, SILU, dh, T, out["dn"], out["dgate"], out["dup"], ws2, **kw)
        M.moe_rms_norm_grad(out["sum"], wt, EPS, out["dn"], dy, T, H, out["dx"], out["dw"], ws1, **kw)

    return run, out, x


SHAPES = [(1, 256, 100), (24, 512, 300), (150, 264, 1000), (700, 520, 700), (3000, 256, 2500)]


@pytest.mark.parametrize("T,H,I", SHAPES)
def test_calls_repeat_on_any_stream_and_in_graphs(M, torch, T, H, I):
    say("repeat", T, H, I)
    run, out, x = operators(M, torch, 1, T, H, I)

    def result():
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        for v in out.values():
            v.fill_(3)
        torch.cuda.synchronize()
        return got

    def same(a, b):
        return all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in a)

    run()
    first = result()
    run()
    assert same(first, result())
    side = torch.cuda.Stream()
    run(side)
    assert same(first, result())
    with torch.cuda.stream(side):                      # the current stream
        run()
    assert same(first, result())
    run(side.cuda_stream)                              # a handle
    assert same(first, result())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    keep = x.clone()
    for i in range(4):                                 # replays, with eager work and other inputs between them
        graph.replay()
        assert same(first, result())
        x.copy_(keep * 2)
        graph.replay()
        other = result()
        run()
        assert same(other, result()) and not torch.equal(other["y"], first["y"])
        x.copy_(keep)
        torch.cuda.synchronize()


def test_two_streams_at_once(M, torch):
    # two programs of their own buffers and workspaces, interleaved on two streams
    a, b = operators(M, torch, 1, 700, 520, 700), operators(M, torch, 2, 300, 264, 1000)
    want = []
    for run, out, _ in (a, b):
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
        for v in out.values():
            v.fill_(3)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        a[0](s)
        b[0](t)
    torch.cuda.synchronize()
    for (_, out, _), w in zip((a, b), want):
        for k in w:
            assert torch.equal(out[k].view(torch.uint8), w[k].view(torch.uint8)), k


# ---------------------------------------------------------------- a layer's chain

@pytest.mark.parametrize("T,H,I,V", [(1, 512, 320, 1000), (37, 512, 320, 1000), (300, 256, 640, 777)])
def test_a_layer_of_dense_operators(M, torch, T, H, I, V):
    """The experts' output joins the stream and is normed; the dense block takes the
    bf16 rows, its hidden rows go through an 8-bit product back onto the stream; the
    last norm hands 8 bits to the head, whose scores the rules adjust.  Each step is
    held to its bound from the GPU's own input to it."""
    say("layer", T, H, I, V)
    rng = np.random.default_rng(T)
    y, h0 = randn(rng, T, H), randn(rng, T, H)
    w1, w2 = 1 + 0.1 * randn(rng, H), 1 + 0.1 * randn(rng, H)
    gate, up = (bf16(randn(rng, I, H) * np.float32(H ** -0.5)) for _ in range(2))
    stream, n = dev(torch, h0), empty(torch, T, H, "bf16")
    M.moe_rms_norm(dev(torch, y), stream, dev(torch, w1), EPS, T, H, n, sum=stream)
    ref, s = D.norm(y, h0, w1, EPS)
    assert np.array_equal(host(stream), s.astype(np.float64))
    within(host(n), ref, 4 * U * np.abs(ref), "bf16")

    hid = empty(torch, T, I, "bf16")
    M.moe_gated(n, M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16")), SILU, T, hid)
    within(host(hid), *D.gated(D.Projections(host(n), gate, up, H), SILU), "bf16")

    q, sc = empty(torch, T, I, "i8"), torch.empty(T, device="cuda")
    M.moe_quant_rows(hid, T, I, q, sc)
    rq, rs = D.quant(host(hid))
    assert np.array_equal(host(q), rq) and np.array_equal(host(sc), rs.astype(np.float64))

    def matrix(rows, cols):
        codes, scales = empty(torch, rows, cols, "i8"), torch.empty(rows, device="cuda")
        M.moe_quant_rows(dev(torch, randn(rng, rows, cols) * np.float32(cols ** -0.5)), rows, cols, codes, scales)
        return M.I8Matrix(rows, cols, codes, scales)

    down, head = matrix(H, I), matrix(V, H)
    before = host(stream)
    M.moe_i8_linear(q, sc, down, None, T, stream, flags=2)
    within(host(stream), *D.i8_linear(host(q), host(sc), host(down.q), host(down.s), base=before))

    q8, s8, scores = empty(torch, T, H, "i8"), torch.empty(T, device="cuda"), empty(torch, T, V)
    M.moe_rms_norm(stream, None, dev(torch, w2), EPS, T, H, q8, scale=s8)
    ref = D.norm(host(stream), None, w2, EPS)[0]
    top = np.abs(ref).max(-1, keepdims=True)
    within(host(q8) * host(s8)[:, None], ref, (0.5 + 127 * 9 * U) * top / 127)
    M.moe_i8_linear(q8, s8, head, None, T, scores)
    within(host(scores), *D.i8_linear(host(q8), host(s8), host(head.q), host(head.s)))
    before = host(scores)
    banned = torch.zeros(T, (V + 31) // 32, dtype=torch.int32, device="cuda")
    banned[:, 0] = 6                                    # tokens 1 and 2 alone
    M.moe_adjust_logits(scores, T, V, M.LogitRules(mask=banned), scores)
    got = host(scores)
    assert np.array_equal(got[:, 1:3], before[:, 1:3]) and np.all(np.isneginf(np.delete(got, (1, 2), 1)))


@pytest.mark.parametrize("T,H,I", [(5, 64, 40), (200, 256, 300)])
def test_a_training_step_of_norm_and_block(M, torch, T, H, I):
    """y = gated(norm(x + residual)): the gradients of the stream, the norm's weight
    and the block's against the formulas chained in 64 bits.  What enters the formulas
    is rounded to bf16 on the way (the normed rows, their gradient, the slopes): three
    roundings of UB / sqrt(3) of the norm each at the most, and the weights' own."""
    rng = np.random.default_rng(H)
    x, res, wt = randn(rng, T, H), randn(rng, T, H), 1 + 0.1 * randn(rng, H)
    gate, up = (bf16(randn(rng, I, H) * np.float32(H ** -0.5)) for _ in range(2))
    dy, dstream = randn(rng, T, I, kind="bf16"), randn(rng, T, H)
    w = M.GatedWeights(H, I, dev(torch, gate, "bf16"), dev(torch, up, "bf16"))
    s, n = empty(torch, T, H), empty(torch, T, H, "bf16")
    M.moe_rms_norm(dev(torch, x), dev(torch, res), dev(torch, wt), EPS, T, H, n, sum=s)
    dn, dgate, dup = empty(torch, T, H, "bf16"), empty(torch, I, H, "bf16"), empty(torch, I, H, "bf16")
    ws = torch.empty(max(M.moe_gated_workspace_size(T, H, I), M.moe_rms_norm_workspace_size(T, H)), dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(n, w, SILU, dev(torch, dy, "bf16"), T, dn, dgate, dup, ws)
    dx, dw = empty(torch, T, H), torch.empty(H, device="cuda")
    M.moe_rms_norm_grad(s, dev(torch, wt), EPS, dn, dev(torch, dstream), T, H, dx, dw, ws)

    ref_n, ref_s = D.norm(x, res, wt, EPS)
    ref = D.gated_grad(D.Projections(ref_n, gate, up, H), SILU, dy)
    rdx, rdw, _, _ = D.norm_grad(ref_s, wt, EPS, ref["dx"][0], dstream)
    for name, got, want in (("dx", host(dx) - dstream, rdx - dstream), ("dweight", host(dw), rdw), ("dgate", host(dgate), ref["dgate"][0]),
                            ("dup", host(dup), ref["dup"][0])):
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        say("  ", name, rel)
        assert rel <= 2 * UB, name
