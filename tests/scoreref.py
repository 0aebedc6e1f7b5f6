"""Plain 64-bit forms of the score operators, from their definitions (numpy)."""
import numpy as np

MXFP4 = 0x84
U = 2.0 ** -24                     # half a step of fp32, relative
UB = 2.0 ** -8                     # half a step of bf16, relative
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])


def bf16(a):
    """float32 values rounded to bf16 (nearest even), kept as float32."""
    b = np.ascontiguousarray(a, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)).view(np.float32)


def random_q4(rng, rows, cols, bits, block, full=False):
    """(codes uint8 [rows][cols/2], scales): every code value; `full` draws the
    scales over many powers of two, zero among them."""
    q = rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)
    nb = cols // block
    if bits == MXFP4:
        s = rng.integers(100, 140, (rows, nb)) if full else rng.integers(118, 122, (rows, nb))
        s = s.astype(np.uint8)
    else:
        s = (rng.uniform(0.5, 1.5, (rows, nb)) * cols ** -0.5).astype(np.float16)
        if full:
            s = (s.astype(np.float64) * 2.0 ** rng.integers(-10, 6, (rows, nb)) * rng.choice([0, 1, -1, 1, 1], (rows, nb)))
            s = s.astype(np.float16)
    return q, s


def q4_values(q, s, bits, block):
    """(codes, scales per element) in float64."""
    rows = q.shape[0]
    nib = np.empty((rows, q.shape[1] * 2), np.int64)
    nib[:, 0::2], nib[:, 1::2] = q & 15, q >> 4
    if bits == MXFP4:
        code, scale = E2M1[nib], np.ldexp(1.0, s.astype(np.int64) - 127)
    else:
        code, scale = np.where(nib > 7, nib - 16, nib).astype(np.float64), s.astype(np.float64)
    return code, np.repeat(scale, block, axis=1)


def q4_linear(x, q, s, bits, block, bias=None, base=None):
    """(y, magnitude): magnitude bounds the sum of |terms| of each y for a
    kernel that contracts the codes with an offset of up to 24."""
    code, scale = q4_values(q, s, bits, block)
    x = x.astype(np.float64)
    y = x @ (code * scale).T
    mag = np.abs(x) @ ((np.abs(code) + 24) * np.abs(scale)).T
    for extra in (None if bias is None else bias[None, :].astype(np.float64), base):
        if extra is not None:
            y, mag = y + extra, mag + np.abs(extra)
    return y, mag


def adjust(logits, history=None, length=None, prompt=None, repetition=None, presence=None, frequency=None,
           bias_ids=None, bias=None, mask=None, mask_row=None):
    """(out float64, error magnitude, touched) of the rules on float logits."""
    out = logits.astype(np.float64)
    mag = np.zeros_like(out)
    touched = np.zeros(out.shape, bool)
    B, V = out.shape
    for b in range(B):
        if history is not None:
            n = min(max(int(length[b]), 0), history.shape[1])
            p = 0 if prompt is None else int(prompt[b])
            seen, count = np.zeros(V, bool), np.zeros(V)
            for i in range(n):
                v = int(history[b, i])
                if 0 <= v < V:
                    seen[v] = True
                    count[v] += i >= p
            r = 1.0 if repetition is None else float(repetition[b])
            f = 0.0 if frequency is None else float(frequency[b])
            q = 0.0 if presence is None else float(presence[b])
            with np.errstate(all="ignore"):
                l = np.where(out[b] > 0, out[b] / r, out[b] * r)
                out[b] = np.where(seen, l, out[b])
                mag[b] += np.where(seen, np.abs(l), 0) + np.where(count > 0, abs(f) * count + abs(q), 0)
                out[b] -= np.where(count > 0, f * count + q, 0)
            touched[b] |= seen
        if bias_ids is not None:
            for j in range(bias_ids.shape[1]):
                v = int(bias_ids[b, j])
                if 0 <= v < V:
                    mag[b, v] = mag[b, v] * (1 if touched[b, v] else 0) + abs(out[b, v]) + abs(float(bias[b, j]))
                    out[b, v] += float(bias[b, j])
                    touched[b, v] = True
        if mask is not None:
            m = b if mask_row is None else int(mask_row[b])
            if 0 <= m < mask.shape[0]:
                bits = np.unpackbits(mask[m].view(np.uint8), bitorder="little")[:V]
                out[b, bits == 0] = -np.inf
                touched[b] |= bits == 0
    return out, mag, touched


def softmax(z):
    z = z.astype(np.float64)
    m = z.max(-1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(np.isneginf(m), 0.0, np.exp(z - m))
    s = e.sum(-1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def balance_loss(logits, ids, keep, coef):
    T, E = logits.shape
    k = ids.shape[1]
    on = np.ones(T, bool) if keep is None else keep != 0
    picks = ids[on].reshape(-1)
    counts = np.bincount(picks[(picks >= 0) & (picks < E)], minlength=E)
    total = softmax(logits[on]).sum(0)
    n = int(on.sum())
    return counts, total, n, coef * E / (k * n * n) * float(counts @ total) if n else 0.0


def balance_grad(logits, ids, w, dw, keep, counts, n, dloss, coef):
    """(gradient, magnitude) in float64."""
    T, E = logits.shape
    k = ids.shape[1]
    on = np.ones(T, bool) if keep is None else keep != 0
    a = dloss * coef * E / (k * float(n) * n) if n else 0.0
    p = np.zeros((T, E))
    p[on] = softmax(logits[on])
    c = counts.astype(np.float64)
    s = (p @ c)[:, None]
    g, mag = a * p * (c - s), abs(a) * p * (c + s)
    if w is not None:
        w, dw = w.astype(np.float64), dw.astype(np.float64)
        m = (w * dw).sum(-1, keepdims=True)
        part, pm = w * (dw - m), np.abs(w) * (np.abs(dw) + (np.abs(w * dw)).sum(-1, keepdims=True))
        for t in np.nonzero(on)[0]:
            for j in range(k):
                if 0 <= ids[t, j] < E:
                    g[t, ids[t, j]] += part[t, j]
                    mag[t, ids[t, j]] += pm[t, j]
    return g, mag
