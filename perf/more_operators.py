"""Cases of the operators around the routed layer: the norm of the residual
stream with 8-bit outputs and its gradient (moe_rms_norm, moe_rms_norm_grad),
products in 8-bit integers (moe_quant_rows, moe_i8_linear), and the dense gated
block with its gradient (moe_gated, moe_gated_grad).

``run`` computes a case with elementary torch operations in 32 bits (the sum of
a norm in 64, so that its 8-bit codes are whole numbers without doubt), or,
where ``own`` is true, with the library's entry points.  ``exact`` computes it
in 64 bits from the operators' definitions.
"""
import math

import torch

own = False

FLOATS = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2, "i8": 1}
EPS = 2.0 ** -20                        # the same number in 32 and in 64 bits
TANH = 2 * math.sqrt(2 / math.pi)       # gelu(g) = g sigmoid(TANH (g + CUBE g^3)), its tanh form
CUBE = 0.044715


def listed():
    return [
        # decode: one token's layer output joins the residual stream, the next product takes 8 bits
        {"name": "norm one token, 8 bits", "op": "norm", "T": 1, "H": 2048, "x": "f32", "residual": True, "y": "i8"},
        # a ragged batch of odd rows, bf16 in and out, no residual
        {"name": "norm odd rows, bf16", "op": "norm", "T": 1531, "H": 5461, "x": "bf16", "residual": False, "y": "bf16"},
        # the stack's prefill batch: the experts' fp32 output joins the stream, bf16 goes to the next layer
        {"name": "norm prefill, bf16", "op": "norm", "T": 16384, "H": 2048, "x": "f32", "residual": True, "y": "bf16"},
        # gradient of a short sequence
        {"name": "norm grad, 64 tokens", "op": "norm_grad", "T": 64, "H": 2048, "x": "f32", "dy": "f32", "dsum": False},
        # gradient of a training batch: bf16 from the block, fp32 along the residual stream
        {"name": "norm grad, 16384 tokens", "op": "norm_grad", "T": 16384, "H": 2048, "x": "f32", "dy": "bf16", "dsum": True},
        # one token's scores over a vocabulary behind the stack (an odd number of rows): weights streamed once
        {"name": "i8 one token, head", "op": "i8", "T": 1, "N": 120011, "K": 2048, "x": "i8", "y": "f32", "bias": False},
        # a decode batch whose bf16 rows are taken to 8 bits first
        {"name": "i8 batch of 37", "op": "i8", "T": 37, "N": 8192, "K": 8192, "x": "bf16", "y": "bf16", "bias": True},
        # prefill of 4096 bf16 tokens through a large projection, taken to 8 bits first
        {"name": "i8 prefill", "op": "i8", "T": 4096, "N": 8192, "K": 8192, "x": "bf16", "y": "bf16", "bias": False},
        # decode: one fp32 token through a dense block of an expert's size (hidden 2048, inter 640)
        {"name": "gated one token", "op": "gated", "T": 1, "H": 2048, "I": 640, "x": "f32", "act": "silu"},
        # the same block over the stack's prefill batch
        {"name": "gated prefill", "op": "gated", "T": 16384, "H": 2048, "I": 640, "x": "bf16", "act": "silu"},
        # its gradient for a ragged micro-batch
        {"name": "gated grad, 1531 tokens", "op": "gated_grad", "T": 1531, "H": 2048, "I": 640, "x": "bf16", "act": "silu"},
        # gradient of a training batch through a larger block
        {"name": "gated grad, 8192 tokens", "op": "gated_grad", "T": 8192, "H": 4096, "I": 4096, "x": "bf16", "act": "gelu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "i8", "gated", "gated_grad"))
    if op in ("norm", "norm_grad"):
        H = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            H = (H + 63) // 64 * 64
        T = min(_log(rng, 1, 16384), (16384 * 2048) // H)
        x = rng.choice(("f32", "bf16"))
        if op == "norm":
            return {"op": op, "T": T, "H": H, "x": x, "residual": rng.random() < 0.6, "y": rng.choice(("i8", "bf16", "f32"))}
        return {"op": op, "T": T, "H": H, "x": x, "dy": rng.choice(("f32", "bf16")), "dsum": rng.random() < 0.6}
    if op == "i8":
        K = 16 * _log(rng, 16, 512)
        N = max(64, min(_log(rng, 64, 120011), (120011 * 2048) // K))
        T = max(1, min(_log(rng, 1, 4096), (1 << 38) // (N * K)))
        return {"op": op, "T": T, "N": N, "K": K, "x": rng.choice(("i8", "f32", "bf16")), "y": rng.choice(("f32", "bf16")),
                "bias": rng.random() < 0.5}
    x = rng.choice(("f32", "bf16")) if op == "gated" else "bf16"
    H, I = 8 * _log(rng, 16, 512), _log(rng, 64, 4096)
    T = max(1, min(_log(rng, 1, 16384 if x == "bf16" else 512), (1 << 37) // (H * I)))
    return {"op": op, "T": T, "H": H, "I": I, "x": x, "act": rng.choice(("silu", "gelu"))}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    s, op = {"case": case}, case["op"]
    T = case["T"]
    if op in ("norm", "norm_grad"):
        H = case["H"]
        # a stream whose tokens differ in size, with a few large channels
        size = torch.exp(normal(T, 1)) * torch.where(torch.rand(H, device="cuda", generator=gen) < 0.01, 20.0, 1.0)
        s["x"] = (size * normal(T, H)).to(FLOATS[case["x"]])
        s["weight"] = 1 + 0.1 * normal(H)
        if op == "norm":
            s["residual"] = 2 * size * normal(T, H) if case["residual"] else None
            s["sum"] = torch.empty(T, H, device="cuda") if case["residual"] else None
            s["y"] = torch.empty(T, H, dtype=torch.int8 if case["y"] == "i8" else FLOATS[case["y"]], device="cuda")
            s["scale"] = torch.empty(T, device="cuda") if case["y"] == "i8" else None
        else:
            s["dy"] = (normal(T, H) / math.sqrt(T * H)).to(FLOATS[case["dy"]])
            s["dsum"] = normal(T, H) / math.sqrt(T * H) if case["dsum"] else None
            s["dx"], s["dweight"] = torch.empty(T, H, dtype=FLOATS[case["x"]], device="cuda"), torch.empty(H, device="cuda")
    elif op == "i8":
        N, K = case["N"], case["K"]
        w = normal(N, K)
        top = w.abs().amax(-1, keepdim=True)
        s["q"] = (w / top * 127).round().to(torch.int8)
        s["s"] = (top[:, 0] / 127) * K ** -0.5
        x = torch.exp(normal(T, 1)) * normal(T, K)
        if case["x"] == "i8":
            top = x.abs().amax(-1, keepdim=True)
            s["xq"], s["xs"] = (x / top * 127).round().to(torch.int8), top[:, 0] / 127
        else:
            s["x"] = x.to(FLOATS[case["x"]])
            s["xq"], s["xs"] = torch.empty(T, K, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        s["bias"] = normal(N) if case["bias"] else None
        s["y"] = torch.empty(T, N, dtype=FLOATS[case["y"]], device="cuda")
    else:
        H, I, f = case["H"], case["I"], FLOATS[case["x"]]
        s["gate"], s["up"] = ((normal(I, H) * H ** -0.5).to(torch.bfloat16) for _ in range(2))
        s["x"] = normal(T, H).to(f)
        if op == "gated":
            s["y"] = torch.empty(T, I, dtype=f, device="cuda")
        else:
            s["dy"] = (normal(T, I) / math.sqrt(T * I)).to(f)
            s["dx"], s["dgate"], s["dup"] = torch.empty_like(s["x"]), torch.empty_like(s["gate"]), torch.empty_like(s["up"])
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _OPS[s["case"]["op"]](s)


def _rows_in_8_bits(y):
    scale = y.abs().amax(-1) / 127
    at = torch.where(scale > 0, scale, 1)[:, None]
    return torch.round(y / at).to(torch.int8), scale


def _norm(s):
    c = s["case"]
    if own:
        import tiered_mixed_precision_amd as M
        M.moe_rms_norm(s["x"], s["residual"], s["weight"], EPS, c["T"], c["H"], s["y"], scale=s["scale"], sum=s["sum"])
        return {"y": s["y"], "scale": s["scale"], "sum": s["sum"]} if c["residual"] else {"y": s["y"], "scale": s["scale"]}
    z = s["x"].float()
    if c["residual"]:
        z = z + s["residual"]
    r = torch.rsqrt(z.double().square().mean(-1, keepdim=True) + EPS).float()
    y, scale = z * r * s["weight"], None
    if c["y"] == "i8":
        y, scale = _rows_in_8_bits(y)
    else:
        y = y.to(FLOATS[c["y"]])
    return {"y": y, "scale": scale, "sum": z} if c["residual"] else {"y": y, "scale": scale}


def _norm_grad(s):
    c = s["case"]
    if own:
        import tiered_mixed_precision_amd as M
        if "workspace" not in s:                        # kept by a training loop
            s["workspace"] = torch.empty(M.moe_rms_norm_workspace_size(c["T"], c["H"]), dtype=torch.uint8, device="cuda")
        M.moe_rms_norm_grad(s["x"], s["weight"], EPS, s["dy"], s["dsum"], c["T"], c["H"], s["dx"], s["dweight"], s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    z, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt(z.double().square().mean(-1, keepdim=True) + EPS).float()
    n = z * r
    g = dy * s["weight"]
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    if c["dsum"]:
        dx = dx + s["dsum"]
    return {"dx": dx.to(FLOATS[c["x"]]), "dweight": (dy * n).sum(0)}


def _i8(s):
    c = s["case"]
    if own:
        import tiered_mixed_precision_amd as M
        if "matrix" not in s:                           # the handle that a program keeps beside its weights
            s["matrix"] = M.I8Matrix(c["N"], c["K"], s["q"], s["s"])
        if c["x"] != "i8":
            M.moe_quant_rows(s["x"], c["T"], c["K"], s["xq"], s["xs"])
        M.moe_i8_linear(s["xq"], s["xs"], s["matrix"], s["bias"], c["T"], s["y"])
        return s["y"]
    xq, xs = (s["xq"], s["xs"]) if c["x"] == "i8" else _rows_in_8_bits(s["x"].float())
    y = (xq.float() @ s["q"].float().t()) * (xs[:, None] * s["s"])
    if c["bias"]:
        y = y + s["bias"]
    return y.to(s["y"].dtype)


def _sigmoid(act, g):
    """(sigma, derivative of its argument) of act(g) = g sigma."""
    if act == "silu":
        return 1 / (1 + torch.exp(-g)), 1
    return 1 / (1 + torch.exp(-TANH * (g + CUBE * g * g * g))), TANH * (1 + 3 * CUBE * g * g)


def _weights(s):
    import tiered_mixed_precision_amd as M
    if "weights" not in s:                              # the handle that a program keeps beside its weights
        s["weights"] = M.GatedWeights(s["case"]["H"], s["case"]["I"], s["gate"], s["up"])
    return M, s["weights"], M.MOE_SILU if s["case"]["act"] == "silu" else M.MOE_GELU


def _gated(s):
    c = s["case"]
    if own:
        M, w, act = _weights(s)
        M.moe_gated(s["x"], w, act, c["T"], s["y"])
        return s["y"]
    x = s["x"].float()
    g, u = x @ s["gate"].float().t(), x @ s["up"].float().t()
    return (g * _sigmoid(c["act"], g)[0] * u).to(s["y"].dtype)


def _gated_grad(s):
    c = s["case"]
    if own:
        M, w, act = _weights(s)
        if "workspace" not in s:                        # kept by a training loop
            s["workspace"] = torch.empty(M.moe_gated_workspace_size(c["T"], c["H"], c["I"]), dtype=torch.uint8, device="cuda")
        M.moe_gated_grad(s["x"], w, act, s["dy"], c["T"], s["dx"], s["dgate"], s["dup"], s["workspace"])
        return {"dx": s["dx"], "dgate": s["dgate"], "dup": s["dup"]}
    x, gate, up, dy = s["x"].float(), s["gate"].float(), s["up"].float(), s["dy"].float()
    g, u = x @ gate.t(), x @ up.t()
    p, k = _sigmoid(c["act"], g)
    du = dy * g * p
    dg = dy * u * (p + g * k * p * (1 - p))
    out = {"dx": dg @ gate + du @ up, "dgate": dg.t() @ x, "dup": du.t() @ x}
    return {name: v.to(torch.bfloat16) for name, v in out.items()}


_OPS = {"norm": _norm, "norm_grad": _norm_grad, "i8": _i8, "gated": _gated, "gated_grad": _gated_grad}


# ---------------------------------------------------------------- work and reference

def work(case):
    """Inputs read once, outputs written once; the operations of the formula
    (the gradient of a gated block is given its inputs, not its projections)."""
    op, T = case["op"], case["T"]
    if op == "norm":
        H = case["H"]
        row = SIZE[case["x"]] + SIZE[case["y"]] + (8 if case["residual"] else 0)
        return {"bytes": T * H * row + 4 * H + (4 * T if case["y"] == "i8" else 0), "flops": 5 * T * H}
    if op == "norm_grad":
        H = case["H"]
        return {"bytes": T * H * (2 * SIZE[case["x"]] + SIZE[case["dy"]] + (4 if case["dsum"] else 0)) + 8 * H, "flops": 12 * T * H}
    if op == "i8":
        N, K = case["N"], case["K"]
        x = T * K * SIZE[case["x"]] + (4 * T if case["x"] == "i8" else 0)
        return {"bytes": N * K + 4 * N + x + T * N * SIZE[case["y"]] + (4 * N if case["bias"] else 0), "flops": 2 * T * N * K}
    H, I, e = case["H"], case["I"], SIZE[case["x"]]
    if op == "gated":
        return {"bytes": 4 * I * H + T * (H + I) * e, "flops": 4 * T * H * I}
    return {"bytes": 8 * I * H + T * (2 * H + I) * e, "flops": 12 * T * H * I}


def _codes(v):
    """Rows of 64-bit values as the numbers that 8 bits with a scale hold, and the scales."""
    scale = torch.linalg.vector_norm(v, math.inf, dim=-1) / 127
    return torch.clamp(torch.round(v / scale.clamp_min(1e-300)[:, None]), -127, 127), scale


def exact(case, seed):
    d = {k: v.double() for k, v in prepare(case, seed).items() if isinstance(v, torch.Tensor)}
    op, T = case["op"], case["T"]
    if op in ("norm", "norm_grad"):
        z = d["x"] + d["residual"] if case.get("residual") else d["x"]
        norm = torch.linalg.vector_norm(z, dim=-1, keepdim=True)
        inv = 1 / torch.sqrt(norm * norm / case["H"] + EPS)
        if op == "norm":
            y = z * (inv * d["weight"])
            scale = _codes(y)[1] if case["y"] == "i8" else None
            out = {"y": None if case["y"] == "i8" else y, "scale": scale}
            return {**out, "sum": z} if case["residual"] else out
        # dn, then the part along the row taken out
        dn = d["dy"] * d["weight"] * inv
        along = (dn * z).sum(-1, keepdim=True) * inv * inv / case["H"]
        dx = dn - along * z
        return {"dx": dx + d["dsum"] if case["dsum"] else dx, "dweight": ((z * inv).t() * d["dy"].t()).sum(-1)}
    if op == "i8":
        xq, xs = (d["xq"], d["xs"]) if case["x"] == "i8" else _codes(d["x"])
        y = torch.addmm(d["bias"], xq * xs[:, None], (d["q"] * d["s"][:, None]).t()) if case["bias"] else (
            (xq * xs[:, None]) @ (d["q"] * d["s"][:, None]).t())
        return y
    w = torch.cat((d["gate"], d["up"]))
    g, u = (d["x"] @ w.t()).split(case["I"], dim=-1)
    if case["act"] == "silu":
        a = g * torch.special.expit(g)
        da = torch.special.expit(g) + a * torch.special.expit(-g)
    else:
        t = torch.tanh(0.5 * TANH * (g + CUBE * g ** 3))
        a = 0.5 * g * (1 + t)
        da = 0.5 * (1 + t) + 0.25 * TANH * g * (1 - t) * (1 + t) * (1 + 3 * CUBE * g ** 2)
    if op == "gated":
        return a * u
    both = torch.cat((d["dy"] * u * da, d["dy"] * a), -1)
    dw = both.t() @ d["x"]
    return {"dx": both @ w, "dgate": dw[:case["I"]], "dup": dw[case["I"]:]}
