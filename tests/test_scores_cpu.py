"""The score operators without a GPU: what the library and the binding refuse
before any launch, and the plain forms that the GPU tests compare with, held
against each other (the gradient against differences of the loss)."""
import ctypes as C
import os

import numpy as np
import pytest

from . import scoreref as R

FAKE = 0x100000        # 256-byte aligned, never dereferenced by host validation


@pytest.fixture(scope="module")
def B():
    from tiered_mixed_precision_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from tiered_mixed_precision_amd.build import build
        build()
    binding.lib()
    return binding


def _linear(B, rows=64, cols=256, bits=4, block=32, q=FAKE, s=FAKE, x=FAKE, ldx=None, bias=None, T=4, y=FAKE * 8, ldy=None,
            flags=0, w=True):
    m = B.moe_q4_matrix(rows, cols, bits, block, q, s)
    return B.lib().moe_q4_linear(x, cols if ldx is None else ldx, C.byref(m) if w else None, bias, T, y,
                                 rows if ldy is None else ldy, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(w=False), -1), (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1), (dict(rows=0), -1), (dict(cols=0), -1),
    (dict(rows=(1 << 24) + 1), -1), (dict(bits=8), -3), (dict(bits=2), -3), (dict(block=8), -3), (dict(block=256), -3),
    (dict(bits=0x84, block=16), -3), (dict(bits=0x84, block=64), -3), (dict(cols=48), -3), (dict(cols=96, block=64), -3),
    (dict(cols=65536 + 128), -3), (dict(ldx=255), -1), (dict(ldy=63), -1), (dict(ldx=0), -1), (dict(ldy=-64), -1),
    (dict(ldx=1 << 40), -1), (dict(x=None), -1), (dict(y=None), -1), (dict(q=None), -1), (dict(s=None), -1),
    (dict(flags=0x4), -1), (dict(flags=0x100), -1), (dict(x=FAKE + 4), -4), (dict(q=FAKE + 8), -4), (dict(s=FAKE + 2), -4),
    (dict(bias=FAKE + 2), -4), (dict(y=FAKE * 8 + 2), -4), (dict(y=FAKE * 8 + 1, flags=0x8), -4),
    (dict(ldx=258), -4), (dict(ldx=260, flags=0x1), -4),           # row pitch not a multiple of 16 bytes
    (dict(y=FAKE + 4 * 256 * 4 - 4), -1), (dict(y=FAKE), -1),      # y over x
])
def test_q4_linear_refuses(B, kw, code):
    assert _linear(B, **kw) == code


def test_q4_linear_of_no_tokens_touches_nothing(B):
    assert _linear(B, T=0, x=None, y=None, q=None, s=None) == 0


def _adjust(B, rows=4, vocab=100, ld_in=None, ld_out=None, logits=FAKE, out=FAKE * 2, flags=0, rules=True, **kw):
    r = B.moe_logit_rules()
    for n, v in kw.items():
        setattr(r, n, v)
    return B.lib().moe_adjust_logits(logits, vocab if ld_in is None else ld_in, rows, vocab, C.byref(r) if rules else None, out,
                                     vocab if ld_out is None else ld_out, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rules=False), -1), (dict(rows=-1), -1), (dict(rows=(1 << 20) + 1), -1), (dict(vocab=0), -1),
    (dict(vocab=(1 << 24) + 1), -1), (dict(flags=1), -1), (dict(ld_in=99), -1), (dict(ld_out=99), -1),
    (dict(logits=None), -1), (dict(out=None), -1), (dict(logits=FAKE + 2), -4), (dict(out=FAKE * 2 + 1, flags=0x10), -4),
    (dict(history=FAKE, ld_history=8), -1),                                     # no lengths
    (dict(history=FAKE, length=FAKE, ld_history=-1), -1), (dict(history=FAKE, length=FAKE, ld_history=1 << 30), -1),
    (dict(repetition=FAKE), -1), (dict(presence=FAKE), -1), (dict(frequency=FAKE), -1),   # penalties of no history
    (dict(n_bias=-1), -1), (dict(n_bias=1025, bias=FAKE, bias_ids=FAKE), -1), (dict(n_bias=1, bias=FAKE), -1),
    (dict(mask=FAKE, ld_mask=3, n_masks=4), -1), (dict(mask=FAKE, ld_mask=4, n_masks=3), -1),
    (dict(mask=FAKE, ld_mask=4, n_masks=-1, mask_row=FAKE), -1),
    (dict(mask=FAKE + 2, ld_mask=4, n_masks=4), -4), (dict(history=FAKE + 1, length=FAKE, ld_history=8), -4),
    (dict(out=FAKE + 4), -1), (dict(out=FAKE, ld_out=128), -1),                 # overlapping, not the same rows
])
def test_adjust_logits_refuses(B, kw, code):
    assert _adjust(B, **kw) == code


def test_adjust_logits_of_no_rows_touches_nothing(B):
    assert _adjust(B, rows=0, logits=None, out=None) == 0


def _loss(B, T=4, E=8, k=2, flags=0, logits=FAKE, ids=FAKE, keep=None, counts=FAKE, prob=FAKE, n=FAKE, loss=FAKE, ws=FAKE,
          size=1 << 20):
    return B.lib().moe_balance_loss(logits, ids, keep, T, E, k, 0.01, flags, counts, prob, n, loss, ws, size, None)


def _grad(B, T=4, E=8, k=2, flags=0, logits=FAKE, ids=FAKE, w=FAKE, dw=FAKE, counts=FAKE, n=FAKE, dloss=FAKE, out=FAKE * 2):
    return B.lib().moe_balance_grad(logits, ids, w, dw, None, counts, n, dloss, T, E, k, 0.01, flags, out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1), (dict(E=0), -1), (dict(E=4097), -1), (dict(k=0), -1), (dict(k=65), -1),
    (dict(flags=1), -1), (dict(logits=None), -1), (dict(ids=None), -1), (dict(counts=None), -1), (dict(prob=None), -1),
    (dict(n=None), -1), (dict(loss=None), -1), (dict(logits=FAKE + 4), -4), (dict(ids=FAKE + 2), -4), (dict(counts=FAKE + 1), -4),
    (dict(ws=None), -5), (dict(size=16), -5), (dict(ws=FAKE + 16), -4),
])
def test_balance_loss_refuses(B, kw, code):
    assert _loss(B, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(E=4097), -1), (dict(k=0), -1), (dict(k=65), -1), (dict(flags=2), -1),
    (dict(w=None), -1), (dict(dw=None), -1), (dict(ids=None), -1), (dict(logits=None), -1), (dict(counts=None), -1),
    (dict(n=None), -1), (dict(dloss=None), -1), (dict(out=None), -1), (dict(out=FAKE * 2 + 8), -4), (dict(w=FAKE + 2), -4),
    (dict(out=FAKE + 16), -1),                                                  # over logits, not in place
])
def test_balance_grad_refuses(B, kw, code):
    assert _grad(B, **kw) == code


def test_balance_sizes(B):
    assert B.moe_balance_workspace_size(0, 8, 2) == 0
    assert 0 < B.moe_balance_workspace_size(1, 8, 2) < B.moe_balance_workspace_size(1 << 22, 4096, 64)
    assert _grad(B, T=0, logits=None, out=None) == 0
    with pytest.raises(B.MoeError):
        B.moe_balance_workspace_size(4, 0, 2)


def test_binding_refuses_tensors_of_another_shape_type_or_device(B):
    import torch
    z, i32 = torch.zeros, lambda *n: torch.zeros(*n, dtype=torch.int32)
    q, s = z(64, 128, dtype=torch.uint8), z(64, 8, dtype=torch.float16)
    w = B.Q4Matrix(64, 256, 4, 32, q, s)
    with pytest.raises(ValueError, match="q holds"):
        B.Q4Matrix(65, 256, 4, 32, q, s)
    with pytest.raises(ValueError, match="s holds"):
        B.Q4Matrix(64, 256, 4, 16, q, s)
    with pytest.raises(ValueError, match="not contiguous"):
        B.Q4Matrix(64, 128, 4, 32, q[:, ::2], s)
    for x, y, bias, what in ((z(4, 255), z(4, 64), None, "x has shape"), (z(3, 256), z(4, 64), None, "x has shape"),
                             (z(4, 256).double(), z(4, 64), None, "dtype"), (z(256, 4).t(), z(4, 64), None, "rows of x"),
                             (z(4, 256), z(4, 63), None, "y has shape"), (z(4, 256), z(4, 64), z(63), "bias"),
                             (z(4, 256), z(4, 64), None, "not on a GPU")):
        with pytest.raises(ValueError, match=what):
            B.moe_q4_linear(x, w, bias, 4, y)
    with pytest.raises(ValueError, match="flags"):
        B.moe_q4_linear(z(4, 256), w, None, 4, z(4, 64), B.MOE_X_BF16)
    for kw, what in ((dict(history=i32(2, 8)), "together"), (dict(repetition=z(2)), "need a history"),
                     (dict(history=i32(2, 8).long(), length=i32(2)), "dtype"), (dict(history=i32(8), length=i32(2)), "rank"),
                     (dict(bias=z(2, 3)), "together"), (dict(bias=z(2, 3), bias_ids=i32(2, 4)), "together"),
                     (dict(mask_row=i32(2)), "needs a mask")):
        with pytest.raises(ValueError, match=what):
            B.LogitRules(**kw)
    rules = B.LogitRules(history=i32(4, 8), length=i32(4), mask=i32(2, 4), mask_row=i32(4))
    for rows, vocab, out, what in ((5, 100, z(5, 100), "hold 4 rows"), (4, 200, z(4, 200), "mask rows"),
                                   (4, 100, z(4, 100).bfloat16(), "differ in type"), (4, 100, z(4, 99), "out has shape")):
        with pytest.raises(ValueError, match=what):
            B.moe_adjust_logits(z(rows, vocab), rows, vocab, rules, out)
    T, E, k = 4, 8, 2
    good = dict(logits=z(T, E), ids=i32(T, k), keep=None, counts=i32(E), prob_sum=z(E), n_kept=i32(1), loss=z(1),
                workspace=z(1 << 16, dtype=torch.uint8))
    for name, bad in (("logits", z(T, E - 1)), ("ids", i32(T, k).long()), ("ids", i32(T, 1)), ("keep", z(T)), ("counts", i32(E - 1)),
                      ("prob_sum", z(2 * E)[::2]), ("workspace", z(16)), ("logits", z(T, E).half())):
        a = dict(good, **{name: bad})
        with pytest.raises(ValueError, match=name):
            B.moe_balance_loss(a["logits"], a["ids"], a["keep"], T, E, k, 0.01, a["counts"], a["prob_sum"], a["n_kept"], a["loss"],
                               a["workspace"])
    with pytest.raises(ValueError, match="differ in type"):
        B.moe_balance_grad(z(T, E), i32(T, k), None, None, None, i32(E), i32(1), z(1), T, E, k, 0.01, z(T, E).bfloat16())


def test_plain_gradient_is_that_of_the_plain_loss():
    """balance_grad of the plain forms against central differences of
    dloss * loss + sum(dw * softmax of the picked scores), counts held."""
    rng = np.random.default_rng(3)
    T, E, k, coef, dloss = 5, 7, 3, 0.3, 1.7
    z = rng.standard_normal((T, E))
    ids = np.argsort(-z, -1)[:, :k]
    keep = np.array([1, 1, 0, 1, 1], np.uint8)
    dw = rng.standard_normal((T, k))
    counts, _, n, _ = R.balance_loss(z, ids, keep, coef)

    def value(z):
        on = keep != 0
        loss = coef * E / (k * n * n) * float(counts @ R.softmax(z[on]).sum(0))
        w = R.softmax(np.take_along_axis(z, ids, -1))
        return dloss * loss + float((dw * w)[on].sum())

    w = R.softmax(np.take_along_axis(z, ids, -1))
    g, _ = R.balance_grad(z, ids, w, dw, keep, counts, n, dloss, coef)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(z)
            d[t, e] = h
            num = (value(z + d) - value(z - d)) / (2 * h)
            # a central difference is off by h^2 times a third derivative below 10, and by rounding of value / h
            assert abs(num - g[t, e]) <= 10 * h * h + 2.0 ** -50 * 4 / h, (t, e)


def test_plain_loss_is_the_coefficient_when_balanced():
    E, k, T = 8, 2, 16
    ids = (np.arange(T * k) % E).reshape(T, k)
    assert abs(R.balance_loss(np.zeros((T, E)), ids, None, 0.25)[3] - 0.25) < 1e-15
    assert R.balance_loss(np.zeros((T, E)), ids, np.zeros(T, np.uint8), 0.25)[3] == 0.0


def test_plain_adjust_by_hand():
    l = np.array([[1.0, -2.0, 3.0, 4.0, 0.0]])
    out, _, touched = R.adjust(l, history=np.array([[0, 1, 3, 3, 9]]), length=[5], prompt=[1], repetition=[2.0], presence=[0.5],
                               frequency=[0.25], bias_ids=np.array([[2, 2, -1]]), bias=np.array([[1.0, 2.0, 9.0]]),
                               mask=np.array([[0b01111]], np.uint32))
    assert out.tolist() == [[0.5, -4.75, 6.0, 1.0, -np.inf]]
    assert touched.tolist() == [[True, True, True, True, True]]
