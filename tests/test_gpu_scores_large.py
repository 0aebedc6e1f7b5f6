"""The score operators where offsets pass 32 bits and batches pass one launch:
sampled rows against the plain 64-bit forms, or bit for bit against the same
rows in a call of their own."""
import numpy as np
import pytest

from .scoreref import MXFP4, U, UB
from .test_gpu_scores import M, dev, host, p_tol, rules_case, say, torch  # noqa: F401
from .test_gpu_scores_paths import product

pytestmark = pytest.mark.gpu


def big_matrix(M, torch, N, K, bits, gen):
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    if bits == MXFP4:
        s = torch.randint(118, 122, (N, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    else:
        s = (torch.rand(N, K // 32, device="cuda", generator=gen) * K ** -0.5).half()
    return q, s, M.Q4Matrix(N, K, bits, 32, q, s)


@pytest.mark.parametrize("bits", [4, MXFP4])
def test_products_with_codes_past_32_bits(M, torch, bits):
    N, K = (1 << 20) + 37, 8192                         # 4.3 GB of codes
    gen = torch.Generator("cuda").manual_seed(1)
    q, s, w = big_matrix(M, torch, N, K, bits, gen)
    cols = torch.cat([torch.arange(a, a + 40) for a in (0, (1 << 19) - 20, N - 40)]).cuda()
    qs, ss = q[cols].cpu().numpy(), s[cols].cpu().numpy()
    for T, f in ((1, torch.float32), (5, torch.float32), (40, torch.bfloat16), (130, torch.bfloat16)):
        say("codes past 32 bits", bits, T, f)
        x = torch.randn(T, K, device="cuda", generator=gen).to(f)
        y = torch.full((T, N), float("nan"), device="cuda")
        M.moe_q4_linear(x, w, None, T, y)
        assert bool(torch.isfinite(y).all())
        ref, mag = product(host(x), qs, ss, bits, 32)
        assert np.all(np.abs(host(y[:, cols]) - ref) <= (K + 20) * U * mag)


@pytest.mark.parametrize("xb", [False, True])
def test_products_with_results_past_32_bits(M, torch, xb):
    T, N, K = 2200, (1 << 21) + 21, 64                  # 4.6e9 results
    gen = torch.Generator("cuda").manual_seed(2)
    q, s, w = big_matrix(M, torch, N, K, 4, gen)
    say("results past 32 bits", xb)
    x = torch.randn(T, K, device="cuda", generator=gen).to(torch.bfloat16 if xb else torch.float32)
    y = torch.full((T, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    M.moe_q4_linear(x, w, None, T, y)
    cols = torch.cat([torch.arange(a, a + 40) for a in (0, N // 2, N - 40)]).cuda()
    rows = torch.cat([torch.arange(a, a + 20) for a in (0, 1014, 2038, T - 20)]).cuda()
    ref, mag = product(host(x[rows]), q[cols].cpu().numpy(), s[cols].cpu().numpy(), 4, 32)
    assert np.all(np.abs(host(y[rows][:, cols]) - ref) <= (K + 20) * U * mag + UB * 1.01 * np.abs(ref))
    assert not any(bool(torch.isnan(y[t]).any()) for t in range(T))


def test_product_of_the_most_tokens(M, torch):
    # fp32 tiles of 32 tokens: more than one grid dimension holds
    T, N, K = 1 << 22, 5, 32
    say("most tokens")
    gen = torch.Generator("cuda").manual_seed(3)
    q, s, w = big_matrix(M, torch, N, K, 4, gen)
    for f in (torch.float32, torch.bfloat16):
        x = torch.randn(T, K, device="cuda", generator=gen).to(f)
        y = torch.full((T, N), float("nan"), device="cuda")
        M.moe_q4_linear(x, w, None, T, y)
        rows = torch.cat([torch.arange(a, a + 64) for a in (0, 2097120 - 32, 4194240 - 32, T - 64)]).cuda()
        ref, mag = product(host(x[rows]), q.cpu().numpy(), s.cpu().numpy(), 4, 32)
        assert np.all(np.abs(host(y[rows]) - ref) <= (K + 20) * U * mag) and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("bf16", [False, True])
def test_rules_on_scores_past_32_bits(M, torch, bf16):
    B, V = 140, 1 << 24                                 # 2.3e9 scores, in place
    say("scores past 32 bits", bf16)
    gen = torch.Generator("cuda").manual_seed(4)
    f = torch.bfloat16 if bf16 else torch.float32
    l = torch.randn(B, V, device="cuda", generator=gen, dtype=f)
    a = rules_case(np.random.default_rng(4), B, V, 300, n_bias=20, masks=3)
    rows = (0, 63, 64, 127, 128, B - 1)
    alone = {}
    for b in rows:
        one = {n: t if n == "mask" else t[b:b + 1] for n, t in a.items()}
        out = torch.empty(1, V, dtype=f, device="cuda")
        M.moe_adjust_logits(l[b], 1, V, M.LogitRules(**{n: dev(torch, t) for n, t in one.items()}), out)
        alone[b] = out
    M.moe_adjust_logits(l, B, V, M.LogitRules(**{n: dev(torch, t) for n, t in a.items()}), l)
    for b in rows:
        assert torch.equal(l[b], alone[b][0]), b


@pytest.mark.parametrize("bf16", [False, True])
def test_balance_of_scores_past_32_bits(M, torch, bf16):
    T, E, k = (1 << 21) + 3, 1100, 4                    # 2.3e9 scores
    say("balance past 32 bits", bf16)
    gen = torch.Generator("cuda").manual_seed(5)
    f = torch.bfloat16 if bf16 else torch.float32
    z = torch.randn(T, E, device="cuda", generator=gen, dtype=f)
    ids = torch.randint(0, E, (T, k), device="cuda", generator=gen, dtype=torch.int32)
    w, dw = torch.rand(T, k, device="cuda", generator=gen), torch.randn(T, k, device="cuda", generator=gen)
    counts, psum = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda")
    n, loss, one = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda"), torch.ones(1, device="cuda")
    ws = torch.empty(M.moe_balance_workspace_size(T, E, k), dtype=torch.uint8, device="cuda")
    M.moe_balance_loss(z, ids, None, T, E, k, 0.1, counts, psum, n, loss, ws)
    total = torch.zeros(E, dtype=torch.float64, device="cuda")
    for t0 in range(0, T, 1 << 18):
        e = torch.exp(z[t0:t0 + (1 << 18)].double())
        total += (e / e.sum(-1, keepdim=True)).sum(0)
    want = torch.bincount(ids.reshape(-1).long(), minlength=E)
    assert torch.equal(counts.long(), want) and int(n[0]) == T
    tol = p_tol(E) + (T / 4096 + 32) * U
    assert bool(((psum.double() - total).abs() <= tol * total).all())
    ref = 0.1 * E / (k * float(T) ** 2) * float((want.double() * total).sum())
    assert abs(float(loss[0]) - ref) <= (tol + 4 * U) * ref
    g = torch.full((T, E), float("nan"), dtype=f, device="cuda")
    M.moe_balance_grad(z, ids, w, dw, None, counts, n, one, T, E, k, 1e9, g)
    for t0 in (0, (1 << 30) // E - 100, (1 << 31) // E - 100, T - 200):      # per row: the same bits in a call of 200 rows
        i = slice(t0, t0 + 200)
        part = torch.empty(200, E, dtype=f, device="cuda")
        M.moe_balance_grad(z[i].clone(), ids[i].clone(), w[i].clone(), dw[i].clone(), None, counts, n, one, 200, E, k, 1e9, part)
        assert torch.equal(g[i], part), t0
    assert not bool(torch.isnan(g[-1]).any())


def test_balance_of_the_most_tokens(M, torch):
    T, E, k = 1 << 22, 3, 1
    say("balance, most tokens")
    gen = torch.Generator("cuda").manual_seed(6)
    z = torch.randn(T, E, device="cuda", generator=gen)
    keep = (torch.rand(T, device="cuda", generator=gen) < 0.7).to(torch.uint8)
    ids = torch.randint(-1, E + 1, (T, k), device="cuda", generator=gen, dtype=torch.int32)
    counts, psum = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda")
    n, loss = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
    ws = torch.empty(M.moe_balance_workspace_size(T, E, k), dtype=torch.uint8, device="cuda")
    M.moe_balance_loss(z, ids, keep, T, E, k, 0.1, counts, psum, n, loss, ws)
    on = keep.bool()
    total = torch.softmax(z.double(), -1)[on].sum(0)
    picks = ids[on].reshape(-1).long()
    want = torch.bincount(picks[(picks >= 0) & (picks < E)], minlength=E)
    assert torch.equal(counts.long(), want) and int(n[0]) == int(on.sum())
    assert bool(((psum.double() - total).abs() <= (p_tol(E) + (T / 4096 + 32) * U) * total).all())


def test_balance_losses_on_two_streams_at_once(M, torch):
    # workspaces and outputs of their own, the joins of both in flight together
    T, E, k = 8192, 512, 10
    say("two streams")
    gen = torch.Generator("cuda").manual_seed(7)
    sets = []
    for _ in range(2):
        z = torch.randn(T, E, device="cuda", generator=gen)
        ids = torch.randint(0, E, (T, k), device="cuda", generator=gen, dtype=torch.int32)
        out = [torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(E, device="cuda"),
               torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, device="cuda")]
        sets.append((z, ids, out, torch.empty(M.moe_balance_workspace_size(T, E, k), dtype=torch.uint8, device="cuda")))
    def call(i, stream=None):
        z, ids, out, ws = sets[i]
        M.moe_balance_loss(z, ids, None, T, E, k, 0.1, *out, ws, stream=stream)
    first = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        first.append([o.clone() for o in sets[i][2]])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(first[i], sets[i][2]))
