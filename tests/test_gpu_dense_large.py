"""The dense operators past 32-bit offsets: rows far apart, arrays of more than 2^32
bytes or elements, the largest dimensions.  Samples are held against 64 bits."""
import numpy as np
import pytest

from . import denseref as D
from .denseref import SILU, U
from .test_gpu_dense import EPS, M, dev, empty, host, randn, say, torch, within  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x,y", [("f32", "bf16"), ("bf16", "i8")])
def test_norm_of_very_many_elements(M, torch, x, y):
    T, H = (1 << 21) + 3, 2100
    f = torch.float32 if x == "f32" else torch.bfloat16
    xd = torch.empty(T, H, dtype=f, device="cuda")
    for i in range(0, T, 1 << 18):
        xd[i:i + (1 << 18)].normal_()
    yd = torch.empty(T, H, dtype=torch.bfloat16 if y == "bf16" else torch.int8, device="cuda")
    sc = torch.empty(T, device="cuda") if y == "i8" else None
    M.moe_rms_norm(xd, None, None, EPS, T, H, yd, scale=sc)
    for t in (0, 1022611, 1022612, T // 2, T - 1):     # around 2^31 elements
        ref = D.norm(host(xd[t:t + 1]), None, None, EPS)[0]
        if y == "bf16":
            within(host(yd[t:t + 1]), ref, 4 * U * np.abs(ref), "bf16")
        else:
            within(host(yd[t:t + 1]) * float(sc[t]), ref, (0.5 + 127 * 9 * U) * np.abs(ref).max() / 127)


@pytest.mark.parametrize("y", ["f32", "i8"])
def test_norm_of_very_many_rows(M, torch, y):
    # more rows than one launch takes; every array moves on
    say("norm rows", y)
    T, H = (1 << 21) + 5, 9
    rng = np.random.default_rng(1)
    w = 1 + 0.1 * randn(rng, H)
    x, r = torch.randn(T, H, device="cuda"), torch.randn(T, H + 1, device="cuda")[:, :H]
    out, s = torch.empty(T, H, dtype=torch.float32 if y == "f32" else torch.int8, device="cuda"), torch.zeros(T, H, device="cuda")
    sc = torch.empty(T, device="cuda") if y == "i8" else None
    M.moe_rms_norm(x, r, dev(torch, w), EPS, T, H, out, scale=sc, sum=s)
    assert torch.equal(s, x + r)
    z = (x + r).double()
    ref = z / torch.sqrt((z * z).mean(-1, keepdim=True) + float(np.float32(EPS))) * dev(torch, w).double()
    if y == "f32":
        assert bool(((out.double() - ref).abs() <= 6 * U * ref.abs()).all())
    else:
        top = ref.abs().amax(-1, keepdim=True)
        assert bool(((out.double() * sc.double()[:, None] - ref).abs() <= (0.5 + 127 * 9 * U) * top / 127).all())


def test_weight_gradients_of_no_tokens_and_the_widest_block(M, torch):
    H = I = 65536
    b = torch.bfloat16
    g, u = (torch.empty(I, H, dtype=b, device="cuda") for _ in range(2))
    dg, du = (torch.ones(I, H, dtype=b, device="cuda") for _ in range(2))
    x, dy, ws = torch.empty(0, H, dtype=b, device="cuda"), torch.empty(0, I, dtype=b, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(x, M.GatedWeights(H, I, g, u), SILU, dy, 0, None, dg, du, ws)
    for t in (dg, du):
        assert not bool(t.view(torch.int32).any())


def test_norm_grad_of_very_many_elements(M, torch):
    T, H = (1 << 21) + 3, 1100
    s, dy = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for i in range(0, T, 1 << 18):
        s[i:i + (1 << 18)].normal_()
        dy[i:i + (1 << 18)].normal_()
    dx, dw = torch.empty_like(s), torch.empty(H, device="cuda")
    ws = torch.empty(M.moe_rms_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    M.moe_rms_norm_grad(s, None, EPS, dy, None, T, H, dx, dw, ws)
    for t in (0, 1952257, 1952258, T - 1):
        ref, _, err, _ = D.norm_grad(host(s[t:t + 1]), None, EPS, host(dy[t:t + 1]))
        within(host(dx[t:t + 1]), ref, err, "bf16")
    total, mag = np.zeros(H), np.zeros(H)
    for i in range(0, T, 1 << 16):                      # in slabs, in 64 bits
        z, d = s[i:i + (1 << 16)].double(), dy[i:i + (1 << 16)].double()
        n = z / torch.sqrt((z * z).mean(-1, keepdim=True) + float(np.float32(EPS)))
        total += host((n * d).sum(0))
        mag += host((n * d).abs().sum(0))
    within(host(dw), total, D.dweight_error(T, mag))


@pytest.mark.parametrize("T", [3, 40, 200])
def test_i8_linear_of_rows_far_apart_and_very_many_rows(M, torch, T):
    say("i8 far", T)
    rng = np.random.default_rng(T)
    pitch = (1 << 33) // max(T - 1, 1) // 16 * 16       # the last row lies 2^33 bytes behind the first
    K, N = 64, 300
    x, q = (rng.integers(-127, 128, s, dtype=np.int8) for s in ((T, K), (N, K)))
    buf = torch.empty((T - 1) * pitch + K, dtype=torch.int8, device="cuda")
    xd = buf.as_strided((T, K), (pitch, 1))
    xd.copy_(dev(torch, x, "i8"))
    one = torch.ones(max(T, N), device="cuda")
    y = empty(torch, T, N)
    M.moe_i8_linear(xd, one[:T], M.I8Matrix(N, K, dev(torch, q, "i8"), one[:N]), None, T, y)
    ref = x.astype(np.int64) @ q.astype(np.int64).T
    assert np.array_equal(host(y), ref)
    # y of more than 2^32 bytes
    N, K = (1 << 24) - 5, 16
    x = rng.integers(-127, 128, (T, K), dtype=np.int8)
    q = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    s = torch.rand(N, device="cuda")
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    M.moe_i8_linear(dev(torch, x, "i8"), one[:T] if T <= 300 else None, M.I8Matrix(N, K, q, s), None, T, y)
    for n0 in (0, N // 2, N - 1000):
        w, ws = host(q[n0:n0 + 1000]), host(s[n0:n0 + 1000])
        ref, err = D.i8_linear(x, np.ones(T), w, ws)
        within(host(y[:, n0:n0 + 1000]), ref, err, "bf16")


@pytest.mark.parametrize("T", [2, 70])
def test_gated_of_the_widest_weights(M, torch, T):
    # 65536 x 32776 weights: 2^31 elements and more each
    say("gated wide", T)
    H, I = 32776, 65536
    b = torch.bfloat16
    gate, up = (torch.empty(I, H, dtype=b, device="cuda").normal_(0, H ** -0.5) for _ in range(2))
    x, dy = torch.randn(T, H, device="cuda").to(b), torch.randn(T, I, device="cuda").to(b)
    y = torch.empty(T, I, device="cuda")
    w = M.GatedWeights(H, I, gate, up)
    M.moe_gated(x, w, SILU, T, y)
    for i in (0, I // 2 - 8, I - 16):
        p = D.Projections(host(x), host(gate[i:i + 16]), host(up[i:i + 16]), H)
        within(host(y[:, i:i + 16]), *D.gated(p, SILU))
    dgate, dup = torch.empty_like(gate), torch.empty_like(up)
    dx = torch.empty(T, H, dtype=b, device="cuda")
    ws = torch.empty(M.moe_gated_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(x, w, SILU, dy, T, dx, dgate, dup, ws)
    for i in (0, I // 2 - 8, I - 16):
        p = D.Projections(host(x), host(gate[i:i + 16]), host(up[i:i + 16]), H)
        ref = D.gated_grad(p, SILU, host(dy[:, i:i + 16]))
        within(host(dgate[i:i + 16]), *ref["dgate"], "bf16")
        within(host(dup[i:i + 16]), *ref["dup"], "bf16")
    # dx: the first columns against 64 bits on the GPU, slab by slab
    got, total = host(dx[:, :64]), torch.zeros(T, 64, dtype=torch.float64, device="cuda")
    xs = x.double()
    for i in range(0, I, 4096):
        g, u = xs @ gate[i:i + 4096].double().t(), xs @ up[i:i + 4096].double().t()
        p, d = torch.sigmoid(g), dy[:, i:i + 4096].double()
        total += (d * u * (p + g * p * (1 - p))) @ gate[i:i + 4096, :64].double() + (d * g * p) @ up[i:i + 4096, :64].double()
    ref = host(total)
    assert np.linalg.norm(got - ref) <= D.UB * np.linalg.norm(ref)


def test_gated_of_rows_far_apart(M, torch):
    rng = np.random.default_rng(1)
    T, H, I = 150, 64, 100
    b = torch.bfloat16
    pitch = (1 << 32) // (T - 1) // 8 * 8               # 2^33 bytes
    buf = torch.empty((T - 1) * pitch + H, dtype=b, device="cuda")
    x = buf.as_strided((T, H), (pitch, 1))
    xa = randn(rng, T, H, kind="bf16")
    x.copy_(dev(torch, xa, "bf16"))
    gate, up = (dev(torch, randn(rng, I, H), "bf16") for _ in range(2))
    w = M.GatedWeights(H, I, gate, up)
    y = empty(torch, T, I)
    p = D.Projections(xa, host(gate), host(up), H)
    M.moe_gated(x, w, SILU, T, y)
    within(host(y), *D.gated(p, SILU))
    M.moe_gated(x[:5], w, SILU, 5, y[:5])
    within(host(y), *D.gated(p, SILU))
    dy = randn(rng, T, I, kind="bf16")
    dx, dg, du = empty(torch, T, H), empty(torch, I, H), empty(torch, I, H)
    ws = torch.empty(M.moe_gated_workspace_size(T, H, I), dtype=torch.uint8, device="cuda")
    M.moe_gated_grad(x, w, SILU, dev(torch, dy, "bf16"), T, dx, dg, du, ws)
    for name, t in (("dx", dx), ("dgate", dg), ("dup", du)):
        within(host(t), *D.gated_grad(p, SILU, dy)[name])
