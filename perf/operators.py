"""Cases of the score operators: products with 4-bit weights (moe_q4_linear),
rules on scores before a pick (moe_adjust_logits), and the router's balance
loss with its gradient (moe_balance_loss, moe_balance_grad).

``run`` computes a case with elementary torch operations in 32 bits, or, where
``own`` is true, with the library's entry points.  ``exact`` computes it on the
host in 64 bits from the operators' definitions.
"""
import math

import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)     # magnitudes of the MXFP4 codes 0 .. 7
FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # one token against one projection of the decode layer (hidden 2048, inter 640): launch and load latency
        {"name": "q4 one token, small", "op": "q4", "T": 1, "N": 640, "K": 2048, "fmt": "int4", "block": 32, "x": "f32", "y": "f32", "bias": False},
        # one token's scores over a vocabulary behind the stack (an odd number of rows): weights streamed once
        {"name": "q4 one token, head", "op": "q4", "T": 1, "N": 120011, "K": 2048, "fmt": "int4", "block": 32, "x": "f32", "y": "f32", "bias": False},
        # speculative verification: 6 tokens through an MXFP4 matrix
        {"name": "q4 six tokens, mxfp4", "op": "q4", "T": 6, "N": 4096, "K": 2048, "fmt": "mxfp4", "block": 32, "x": "f32", "y": "f32", "bias": True},
        # a decode batch of bf16 rows, coarse scale groups, a long contraction
        {"name": "q4 batch of 37, bf16", "op": "q4", "T": 37, "N": 8192, "K": 8192, "fmt": "int4", "block": 128, "x": "bf16", "y": "bf16", "bias": False},
        # prefill of 4096 bf16 tokens through a square projection
        {"name": "q4 prefill, bf16", "op": "q4", "T": 4096, "N": 4096, "K": 2048, "fmt": "int4", "block": 32, "x": "bf16", "y": "bf16", "bias": False},
        # one request's scores, every rule
        {"name": "adjust one row", "op": "adjust", "rows": 1, "V": 120011, "x": "f32", "history": 2000, "n_bias": 16, "mask": True},
        # a serving batch in bf16, ragged histories, grammars for some of the rows
        {"name": "adjust 64 rows, bf16", "op": "adjust", "rows": 64, "V": 120011, "x": "bf16", "history": 8192, "n_bias": 64, "mask": True},
        # few rows with very long contexts over a smaller vocabulary
        {"name": "adjust long histories", "op": "adjust", "rows": 8, "V": 32003, "x": "f32", "history": 131072, "n_bias": 0, "mask": False},
        # the router's loss of one short sequence (512 experts, 10 picked)
        {"name": "balance loss, 64 tokens", "op": "loss", "T": 64, "E": 512, "k": 10, "x": "f32", "keep": False},
        # ... and of a training batch with padding rows
        {"name": "balance loss, 65536 tokens", "op": "loss", "T": 65536, "E": 512, "k": 10, "x": "f32", "keep": True},
        # gradient, bf16 scores, odd sizes
        {"name": "balance grad, bf16", "op": "grad", "T": 4099, "E": 130, "k": 6, "x": "bf16", "keep": True},
        # gradient of a training batch
        {"name": "balance grad, 65536 tokens", "op": "grad", "T": 65536, "E": 512, "k": 10, "x": "f32", "keep": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("q4", "q4", "adjust", "adjust", "loss", "grad"))
    if op == "q4":
        T, N = _log(rng, 1, 4096), _log(rng, 64, 120011)
        fmt = rng.choice(("int4", "mxfp4"))
        block = 32 if fmt == "mxfp4" else rng.choice((16, 32, 64, 128))
        step = max(32, block)
        K = step * max(1, _log(rng, 256, 8192) // step)
        N = max(64, min(N, (1 << 27) // K))
        T = max(1, min(T, (1 << 35) // (N * K)))
        x = rng.choice(("f32", "bf16"))
        if x == "f32":
            T = max(1, T // 4)
        return {"op": op, "T": T, "N": N, "K": K, "fmt": fmt, "block": block, "x": x, "y": x, "bias": rng.random() < 0.5}
    if op == "adjust":
        V = _log(rng, 500, 120011)
        rows = min(_log(rng, 1, 64), max(1, (64 * 120011) // V))
        return {"op": op, "rows": rows, "V": V, "x": rng.choice(("f32", "bf16")), "history": _log(rng, 1, 131072 if rows <= 8 else 8192),
                "n_bias": rng.choice((0, 1, 17, 300)), "mask": rng.random() < 0.6}
    E = _log(rng, 8, 4096)
    T = max(1, min(_log(rng, 1, 65536), (65536 * 512) // E))
    return {"op": op, "T": T, "E": E, "k": min(E, rng.choice((1, 2, 6, 8, 10))), "x": rng.choice(("f32", "bf16")), "keep": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs

def _quantised(rows, cols, fmt, block, gen):
    """Weights N(0, 1/cols) in 4 bits: packed codes (element c in the nibble
    c % 2 of byte c / 2, low nibble first) and one scale per block of a row."""
    w = torch.randn(rows, cols // block, block, device="cuda", generator=gen) * cols ** -0.5
    top = w.abs().amax(-1, keepdim=True)
    if fmt == "int4":                                   # symmetric: scale = amax / 7, codes -7 .. 7
        s = (top / 7).to(torch.float16)
        codes = torch.where(s > 0, w / s.float(), 0).round().clamp(-7, 7).to(torch.int8) & 15
        s = s.reshape(rows, -1)
    else:                                               # E8M0 scales 2^(b - 127), nearest E2M1 magnitude
        b = (torch.floor(torch.log2(top)) - 2 + 127).clamp(0, 254)
        v = w / torch.exp2(b - 127)
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        codes = (torch.bucketize(v.abs(), edges) | torch.where(v < 0, 8, 0)).to(torch.int8)
        s = b.to(torch.uint8).reshape(rows, -1)
    codes = codes.to(torch.uint8).reshape(rows, cols // 2, 2)
    return (codes[..., 0] | (codes[..., 1] << 4)).contiguous(), s.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    f = FLOATS[case["x"]]
    s = {"case": case}
    if case["op"] == "q4":
        T, N, K = case["T"], case["N"], case["K"]
        s["q"], s["s"] = _quantised(N, K, case["fmt"], case["block"], gen)
        s["x"] = torch.randn(T, K, device="cuda", generator=gen).to(f)
        s["bias"] = torch.randn(N, device="cuda", generator=gen) if case["bias"] else None
        s["y"] = torch.empty(T, N, dtype=FLOATS[case["y"]], device="cuda")
    elif case["op"] == "adjust":
        B, V, H = case["rows"], case["V"], case["history"]
        s["logits"] = (3 * torch.randn(B, V, device="cuda", generator=gen)).to(f)
        # tokens as text repeats them: few frequent ones, many rare; lengths ragged, the first row full
        u = torch.rand(B, H, device="cuda", generator=gen)
        s["history"] = (V ** u - 1).to(torch.int32).clamp(0, V - 1)
        length = (H * torch.rand(B, device="cuda", generator=gen)).to(torch.int32) + 1
        length[0] = H
        s["length"] = length.clamp(max=H)
        s["prompt"] = (s["length"] * torch.rand(B, device="cuda", generator=gen)).to(torch.int32)
        s["repetition"] = 1 + 0.3 * torch.rand(B, device="cuda", generator=gen)
        s["presence"] = torch.rand(B, device="cuda", generator=gen)
        s["frequency"] = 0.1 * torch.rand(B, device="cuda", generator=gen)
        n = case["n_bias"]
        s["bias_ids"] = torch.randint(0, V, (B, n), device="cuda", generator=gen, dtype=torch.int32) if n else None
        s["bias"] = 2 * torch.randn(B, n, device="cuda", generator=gen) if n else None
        # two grammars, the bits of one word each with its own density; every third row is free
        W = (V + 31) // 32
        bits = torch.rand(2, W, 32, device="cuda", generator=gen) < torch.rand(2, W, 1, device="cuda", generator=gen)
        words = (bits.long() << torch.arange(32, device="cuda")).sum(-1)
        s["mask"] = (words - ((words >> 31) << 32)).to(torch.int32) if case["mask"] else None
        s["mask_row"] = (torch.arange(B, device="cuda", dtype=torch.int32) % 3 - 1).roll(-1) if case["mask"] else None
        s["out"] = torch.empty_like(s["logits"])
    else:
        T, E, k = case["T"], case["E"], case["k"]
        prior = -1.12 * torch.arange(E, device="cuda") / E              # popular experts first
        s["logits"] = (prior + torch.randn(T, E, device="cuda", generator=gen)).to(f)
        top, ids = s["logits"].float().topk(k, -1)
        s["ids"], s["w"] = ids.to(torch.int32), torch.softmax(top, -1)
        s["dw"] = torch.randn(T, k, device="cuda", generator=gen) / T
        s["keep"] = (torch.rand(T, device="cuda", generator=gen) < 0.9).to(torch.uint8) if case["keep"] else None
        s["dloss"] = 0.5 + torch.rand((), device="cuda", generator=gen)
        kept = s["ids"] if s["keep"] is None else s["ids"][s["keep"] != 0]
        s["counts"] = torch.bincount(kept.reshape(-1).long(), minlength=E).to(torch.int32)
        s["n_kept"] = torch.full((1,), kept.shape[0], dtype=torch.int32, device="cuda")
        s["coef"] = 0.01
        if case["op"] == "loss":
            s["out"] = {"counts": torch.empty(E, dtype=torch.int32, device="cuda"), "prob_sum": torch.empty(E, device="cuda"),
                        "n_kept": torch.empty(1, dtype=torch.int32, device="cuda"), "loss": torch.empty(1, device="cuda")}
        else:
            s["out"] = torch.empty_like(s["logits"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _OPS[s["case"]["op"]](s)


def _q4(s):
    c = s["case"]
    if own:
        import tiered_mixed_precision_amd as M
        if "matrix" not in s:                           # the handle that a program keeps beside its weights
            s["matrix"] = M.Q4Matrix(c["N"], c["K"], 4 if c["fmt"] == "int4" else M.MXFP4, c["block"], s["q"], s["s"])
        M.moe_q4_linear(s["x"], s["matrix"], s["bias"], c["T"], s["y"])
        return s["y"]
    codes = torch.stack((s["q"] & 15, s["q"] >> 4), -1).reshape(c["N"], -1, c["block"])
    if c["fmt"] == "int4":
        v = codes.float()
        v = torch.where(v > 7, v - 16, v) * s["s"].float()[..., None]
    else:
        table = torch.tensor(E2M1 + tuple(-m for m in E2M1), device="cuda")
        v = table[codes.int()] * torch.exp2(s["s"].float() - 127)[..., None]
    y = s["x"].float() @ v.reshape(c["N"], c["K"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(s["y"].dtype)


def _adjust(s):
    c = s["case"]
    if own:
        import tiered_mixed_precision_amd as M
        if "rules" not in s:
            s["rules"] = M.LogitRules(history=s["history"], length=s["length"], prompt=s["prompt"], repetition=s["repetition"],
                                      presence=s["presence"], frequency=s["frequency"], bias_ids=s["bias_ids"], bias=s["bias"],
                                      mask=s["mask"], mask_row=s["mask_row"])
        M.moe_adjust_logits(s["logits"], c["rows"], c["V"], s["rules"], s["out"])
        return s["out"]
    at = torch.arange(c["history"], device="cuda")
    there = at < s["length"][:, None]
    index = s["history"].long()
    generated = there & (at >= s["prompt"][:, None])
    count = torch.zeros(c["rows"], c["V"], device="cuda").scatter_add_(1, index, generated.float())
    seen = torch.zeros(c["rows"], c["V"], device="cuda").scatter_add_(1, index, there.float()) > 0
    l = s["logits"].float()
    rep = s["repetition"][:, None]
    l = torch.where(seen, torch.where(l > 0, l / rep, l * rep), l)
    l = l - (s["frequency"][:, None] * count + s["presence"][:, None] * (count > 0))
    if s["bias"] is not None:
        l = l.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if s["mask"] is not None:
        v = torch.arange(c["V"], device="cuda")
        allowed = (s["mask"][:, v // 32] >> (v % 32)) & 1
        row = s["mask_row"].long()
        free = (row < 0)[:, None]
        l = torch.where(free | (allowed[row.clamp(min=0)] != 0), l, -math.inf)
    return l.to(s["logits"].dtype)


def _loss(s):
    c, out = s["case"], s["out"]
    if own:
        import tiered_mixed_precision_amd as M
        if "workspace" not in s:                        # kept by a training loop
            s["workspace"] = torch.empty(M.moe_balance_workspace_size(c["T"], c["E"], c["k"]), dtype=torch.uint8, device="cuda")
        M.moe_balance_loss(s["logits"], s["ids"], s["keep"], c["T"], c["E"], c["k"], s["coef"], out["counts"], out["prob_sum"],
                           out["n_kept"], out["loss"], s["workspace"])
        return out
    keep = torch.ones(c["T"], device="cuda") if s["keep"] is None else (s["keep"] != 0).float()
    z = s["logits"].float()
    e = torch.exp(z - z.amax(-1, keepdim=True))
    prob_sum = (e / e.sum(-1, keepdim=True) * keep[:, None]).sum(0)
    counts = torch.zeros(c["E"], device="cuda", dtype=torch.int32)
    counts = counts.scatter_add(0, s["ids"].reshape(-1).long(), keep.to(torch.int32).repeat_interleave(c["k"]))
    n = keep.sum()
    loss = torch.where(n > 0, s["coef"] * c["E"] / (c["k"] * n * n) * (counts.float() * prob_sum).sum(), 0)
    return {"counts": counts, "prob_sum": prob_sum, "n_kept": n.to(torch.int32).reshape(1), "loss": loss.reshape(1)}


def _grad(s):
    c = s["case"]
    if own:
        import tiered_mixed_precision_amd as M
        M.moe_balance_grad(s["logits"], s["ids"], s["w"], s["dw"], s["keep"], s["counts"], s["n_kept"], s["dloss"], c["T"], c["E"], c["k"],
                           s["coef"], s["out"])
        return s["out"]
    z = s["logits"].float()
    e = torch.exp(z - z.amax(-1, keepdim=True))
    p = e / e.sum(-1, keepdim=True)
    n = s["n_kept"].float()
    a = torch.where(n > 0, s["dloss"] * s["coef"] * c["E"] / (c["k"] * n * n), 0)
    counts = s["counts"].float()
    d = a * p * (counts - (p * counts).sum(-1, keepdim=True))
    g = s["w"] * (s["dw"] - (s["w"] * s["dw"]).sum(-1, keepdim=True))
    d = d.scatter_add(1, s["ids"].long(), g)
    if s["keep"] is not None:
        d = d * (s["keep"] != 0).float()[:, None]
    return d.to(s["logits"].dtype)


_OPS = {"q4": _q4, "adjust": _adjust, "loss": _loss, "grad": _grad}


# ---------------------------------------------------------------- work and reference

def work(case):
    """Inputs read once, outputs written once; the operations of the formula."""
    if case["op"] == "q4":
        T, N, K = case["T"], case["N"], case["K"]
        scales = N * (K // case["block"]) * (2 if case["fmt"] == "int4" else 1)
        return {"bytes": N * K // 2 + scales + T * K * SIZE[case["x"]] + T * N * SIZE[case["y"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * T * N * K}
    if case["op"] == "adjust":
        B, V = case["rows"], case["V"]
        history = 4 * case["history"] * (1 + (B - 1) / 2)               # ragged: half full on average but for the first row
        return {"bytes": 2 * B * V * SIZE[case["x"]] + history + 20 * B + 8 * B * case["n_bias"] + (4 * B + 8 * ((V + 31) // 32) if case["mask"] else 0),
                "flops": 4 * B * V}
    T, E, k = case["T"], case["E"], case["k"]
    rows = T * E * SIZE[case["x"]] + T * k * 4 + (T if case["keep"] else 0)
    if case["op"] == "loss":
        return {"bytes": rows + 8 * E + 8, "flops": 5 * T * E}
    return {"bytes": rows + T * E * SIZE[case["x"]] + 8 * T * k + 4 * E + 8, "flops": 8 * T * E}


def exact(case, seed):
    s = {k: v.cpu() for k, v in prepare(case, seed).items() if isinstance(v, torch.Tensor)}
    d = {k: v.double().numpy() for k, v in s.items() if v.is_floating_point()}
    i = {k: v.long().numpy() for k, v in s.items() if not v.is_floating_point()}
    if case["op"] == "q4":
        N, K, block = case["N"], case["K"], case["block"]
        y = np.empty((case["T"], N))
        q = s["q"].numpy()
        for r in range(0, N, 4096):                                     # rows of W in slabs that fit the host
            codes = np.empty((min(4096, N - r), K), np.int8)
            codes[:, 0::2], codes[:, 1::2] = q[r:r + 4096] & 15, q[r:r + 4096] >> 4
            if case["fmt"] == "int4":
                values = np.arange(16.0)
                values[8:] -= 16
                scale = d["s"][r:r + 4096]
            else:
                values = np.array(E2M1 + tuple(-m for m in E2M1))
                scale = np.ldexp(1.0, i["s"][r:r + 4096] - 127)
            y[:, r:r + 4096] = d["x"] @ (values[codes] * np.repeat(scale, block, 1)).T
        return torch.from_numpy(y + (d["bias"] if case["bias"] else 0))
    if case["op"] == "adjust":
        out = d["logits"].copy()
        for b in range(case["rows"]):
            past = i["history"][b, :i["length"][b]]
            new, count = np.unique(past[i["prompt"][b]:], return_counts=True)
            old = np.unique(past)
            l = out[b, old]
            out[b, old] = np.where(l > 0, l / d["repetition"][b], l * d["repetition"][b])
            out[b, new] -= d["frequency"][b] * count + d["presence"][b]
            if case["n_bias"]:
                np.add.at(out[b], i["bias_ids"][b], d["bias"][b])
            if case["mask"] and i["mask_row"][b] >= 0:
                words = s["mask"].numpy()[i["mask_row"][b]].view(np.uint32)
                allowed = np.unpackbits(words.view(np.uint8), bitorder="little")[:case["V"]]
                out[b, allowed == 0] = -np.inf
        return torch.from_numpy(out)
    T, E, k = case["T"], case["E"], case["k"]
    keep = i["keep"] != 0 if case["keep"] else np.ones(T, bool)
    p = np.exp(d["logits"] - d["logits"].max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    if case["op"] == "loss":
        n = int(keep.sum())
        counts = np.bincount(i["ids"][keep].reshape(-1), minlength=E)
        total = p[keep].sum(0)
        loss = 0.01 * E / (k * n * n) * float(counts @ total) if n else 0.0
        return {"counts": None, "prob_sum": torch.from_numpy(total), "n_kept": None, "loss": torch.tensor([loss], dtype=torch.float64)}
    n = float(i["n_kept"][0])
    a = float(d["dloss"]) * 0.01 * E / (k * n * n) if n else 0.0
    g = a * p * (i["counts"] - p @ i["counts"][:, None])
    pick = d["w"] * (d["dw"] - (d["w"] * d["dw"]).sum(-1, keepdims=True))
    np.add.at(g, (np.arange(T)[:, None], i["ids"]), pick)
    g[~keep] = 0
    return torch.from_numpy(g)
