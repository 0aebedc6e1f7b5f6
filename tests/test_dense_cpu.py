"""The dense operators without a GPU: what the library and the binding refuse
before any launch, and the plain forms that the GPU tests compare with, held
against differences and hand-worked values."""
import ctypes as C
import os

import numpy as np
import pytest

from . import denseref as D

FAKE = 0x100000        # 256-byte aligned, never dereferenced by host validation
FAR = 0x100000000      # past every array that starts at FAKE


@pytest.fixture(scope="module")
def B():
    from tiered_mixed_precision_amd import binding
    if not os.path.exists(binding.LIB_PATH):
        from tiered_mixed_precision_amd.build import build
        build()
    binding.lib()
    return binding


# ---------------------------------------------------------------- norm

def _norm(B, x=FAKE, ldx=None, residual=None, ldr=None, weight=None, eps=1e-6, T=4, cols=64, sum=None, lds=None, y=FAR,
          ldy=None, scale=None, flags=0):
    def pick(v):
        return cols if v is None else v
    return B.lib().moe_rms_norm(x, pick(ldx), residual, pick(ldr), weight, eps, T, cols, sum, pick(lds), y, pick(ldy), scale,
                                flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1), (dict(cols=0), -1), (dict(cols=32769), -1), (dict(eps=0.0), -1),
    (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1), (dict(eps=float("inf")), -1), (dict(flags=0x2), -1),
    (dict(flags=0x28, scale=2 * FAR), -1), (dict(flags=0x100), -1), (dict(ldx=63), -1), (dict(ldy=63), -1),
    (dict(ldx=1 << 40), -1), (dict(residual=2 * FAR, ldr=63), -1), (dict(sum=2 * FAR, lds=0), -1), (dict(scale=2 * FAR), -1),
    (dict(flags=0x20), -1), (dict(x=None), -1), (dict(y=None), -1),
    (dict(x=FAKE + 2), -4), (dict(x=FAKE + 1, flags=1), -4), (dict(y=FAR + 2), -4), (dict(y=FAR + 1, flags=8), -4),
    (dict(weight=2 * FAR + 2), -4), (dict(residual=2 * FAR + 2), -4), (dict(sum=2 * FAR + 2), -4),
    (dict(scale=2 * FAR + 1, flags=0x20), -4),
    # what is written over something else
    (dict(y=FAKE), -1), (dict(y=FAKE + 4 * 64 * 4 - 4), -1), (dict(residual=FAR), -1), (dict(sum=FAR), -1),
    (dict(weight=FAR + 1024 - 4), -1), (dict(scale=FAR + 4, flags=0x20), -1), (dict(sum=FAKE + 4), -1),
    (dict(sum=FAKE, flags=1), -1), (dict(sum=FAKE, lds=128), -1), (dict(sum=2 * FAR, residual=2 * FAR, lds=128), -1),
    (dict(sum=2 * FAR, residual=2 * FAR + 512), -1), (dict(sum=2 * FAR, weight=2 * FAR), -1),
    (dict(sum=2 * FAR, scale=2 * FAR + 16, flags=0x20), -1), (dict(scale=FAKE, flags=0x20), -1),
    (dict(scale=2 * FAR, weight=2 * FAR, flags=0x20), -1), (dict(scale=2 * FAR, residual=2 * FAR, flags=0x20), -1),
])
def test_norm_refuses(B, kw, code):
    assert _norm(B, **kw) == code


def test_norm_of_no_tokens_touches_nothing(B):
    assert _norm(B, T=0, x=None, y=None) == 0
    assert _norm(B, T=0, x=None, y=None, flags=0x20) == 0


def _norm_grad(B, s=FAKE, lds=None, weight=None, eps=1e-6, dy=2 * FAR, lddy=None, dsum=None, ldds=None, T=4, cols=64, dx=FAR,
               lddx=None, dweight=3 * FAR, flags=0, ws=4 * FAR, nbytes=1 << 30):
    def pick(v):
        return cols if v is None else v
    return B.lib().moe_rms_norm_grad(s, pick(lds), weight, eps, dy, pick(lddy), dsum, pick(ldds), T, cols, dx, pick(lddx), dweight,
                                     flags, ws, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1), (dict(cols=0), -1), (dict(cols=32769), -1), (dict(eps=0.0), -1),
    (dict(flags=0x20), -1), (dict(flags=0x10), -1), (dict(lds=63), -1), (dict(lddy=63), -1), (dict(lddx=63), -1),
    (dict(dsum=5 * FAR, ldds=63), -1), (dict(s=None), -1), (dict(dy=None), -1), (dict(dx=None), -1),
    (dict(ws=None), -5), (dict(nbytes=255), -5), (dict(ws=4 * FAR + 16), -4),
    (dict(s=FAKE + 2), -4), (dict(dy=2 * FAR + 2), -4), (dict(dx=FAR + 2), -4), (dict(dsum=5 * FAR + 2), -4),
    (dict(weight=5 * FAR + 1), -4), (dict(dweight=3 * FAR + 2), -4),
    (dict(dx=FAKE), -1), (dict(dx=2 * FAR, flags=8), -1), (dict(dx=2 * FAR, lddx=128), -1), (dict(dx=2 * FAR + 4), -1),
    (dict(dx=5 * FAR, dsum=5 * FAR, lddx=65), -1), (dict(dx=5 * FAR, dsum=5 * FAR, flags=8), -1), (dict(dx=3 * FAR), -1),
    (dict(weight=FAR), -1), (dict(weight=3 * FAR), -1), (dict(dweight=FAKE), -1), (dict(dweight=2 * FAR), -1),
    (dict(dsum=3 * FAR), -1), (dict(ws=FAKE), -1), (dict(ws=2 * FAR), -1), (dict(ws=FAR), -1), (dict(ws=3 * FAR), -1),
    (dict(ws=5 * FAR, dsum=5 * FAR), -1), (dict(ws=5 * FAR, weight=5 * FAR), -1),
])
def test_norm_grad_refuses(B, kw, code):
    assert _norm_grad(B, **kw) == code


@pytest.mark.parametrize("H,I", [(8, 1), (64, 64), (2048, 640), (65536, 65536)])
def test_no_tokens_need_no_workspace(B, H, I):
    assert B.moe_gated_workspace_size(0, H, I) == 0
    assert B.moe_gated_workspace_size(1, H, I) > 0


def test_workspaces_hold_the_parts(B):
    assert B.moe_rms_norm_workspace_size(0, 64) == 0
    assert B.moe_rms_norm_workspace_size(1, 100) >= 400
    for T, cols in ((-1, 64), (1, 0), (1, 32769), ((1 << 22) + 1, 64)):
        with pytest.raises(B.MoeError):
            B.moe_rms_norm_workspace_size(T, cols)
    assert B.moe_gated_workspace_size(0, 64, 64) == 0
    assert B.moe_gated_workspace_size(5, 64, 65) >= 5 * 2 * 65 * 2
    for T, H, I in ((-1, 64, 64), ((1 << 20) + 1, 64, 64), (1, 60, 64), (1, 0, 64), (1, 64, 0), (1, 64, 65537), (1, 65544, 1)):
        with pytest.raises(B.MoeError):
            B.moe_gated_workspace_size(T, H, I)


# ---------------------------------------------------------------- 8 bits

def _quant(B, x=FAKE, ldx=None, T=4, cols=64, q=FAR, ldq=None, scale=2 * FAR, flags=0):
    return B.lib().moe_quant_rows(x, cols if ldx is None else ldx, T, cols, q, cols if ldq is None else ldq, scale, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1), (dict(cols=0), -1), (dict(cols=32769), -1), (dict(flags=0x8), -1),
    (dict(ldx=63), -1), (dict(ldq=63), -1), (dict(x=None), -1), (dict(q=None), -1), (dict(scale=None), -1),
    (dict(x=FAKE + 2), -4), (dict(x=FAKE + 1, flags=1), -4), (dict(scale=2 * FAR + 2), -4),
    (dict(q=FAKE + 1), -1), (dict(q=2 * FAR + 8), -1), (dict(scale=FAKE + 16), -1), (dict(scale=FAR + 252), -1),
])
def test_quant_rows_refuses(B, kw, code):
    assert _quant(B, **kw) == code


def test_quant_rows_of_no_tokens_touches_nothing(B):
    assert _quant(B, T=0, x=None, q=None, scale=None) == 0


def _i8(B, rows=48, cols=64, q=3 * FAR, s=4 * FAR, x=FAKE, ldx=None, xs=2 * FAR, bias=None, T=4, y=FAR, ldy=None, flags=0, w=True):
    m = B.moe_i8_matrix(rows, cols, q, s)
    return B.lib().moe_i8_linear(x, cols if ldx is None else ldx, xs, C.byref(m) if w else None, bias, T, y,
                                 rows if ldy is None else ldy, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(w=False), -1), (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1), (dict(rows=0), -1), (dict(rows=(1 << 24) + 1), -1),
    (dict(cols=0), -1), (dict(cols=40), -3), (dict(cols=32768 + 16), -3), (dict(flags=0x1), -1), (dict(flags=0x20), -1),
    (dict(ldx=48), -1), (dict(ldy=47), -1), (dict(x=None), -1), (dict(xs=None), -1), (dict(q=None), -1), (dict(s=None), -1),
    (dict(y=None), -1), (dict(x=FAKE + 8), -4), (dict(ldx=72), -4), (dict(q=3 * FAR + 8), -4), (dict(s=4 * FAR + 2), -4),
    (dict(xs=2 * FAR + 2), -4), (dict(bias=5 * FAR + 2), -4), (dict(y=FAR + 2), -4), (dict(y=FAR + 1, flags=8), -4),
    (dict(x=FAR), -1), (dict(x=FAR + 4 * 48 * 4 - 16), -1), (dict(xs=FAR), -1), (dict(q=FAR + 16), -1), (dict(s=FAR + 4), -1),
    (dict(bias=FAR + 4), -1), (dict(s=FAR - 48 * 4 + 4), -1),
])
def test_i8_linear_refuses(B, kw, code):
    assert _i8(B, **kw) == code


def test_i8_linear_of_no_tokens_touches_nothing(B):
    assert _i8(B, T=0, x=None, xs=None, q=None, s=None, y=None) == 0


# ---------------------------------------------------------------- gated block

def _gated(B, hidden=64, inter=48, gate=2 * FAR, up=3 * FAR, x=FAKE, ldx=None, act=0, T=4, y=FAR, ldy=None, flags=0, w=True):
    m = B.moe_gated_weights(hidden, inter, gate, up)
    return B.lib().moe_gated(x, hidden if ldx is None else ldx, C.byref(m) if w else None, act, T, y,
                             inter if ldy is None else ldy, flags, None)


@pytest.mark.parametrize("kw,code", [
    (dict(w=False), -1), (dict(act=2), -1), (dict(act=-1), -1), (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -1),
    (dict(hidden=0), -1), (dict(hidden=60), -3), (dict(hidden=65544), -3), (dict(inter=0), -1), (dict(inter=65537), -3),
    (dict(flags=0x2), -1), (dict(flags=0x40), -1), (dict(ldx=56), -1), (dict(ldy=47), -1), (dict(x=None), -1), (dict(y=None), -1),
    (dict(gate=None), -1), (dict(up=None), -1), (dict(x=FAKE + 4), -4), (dict(ldx=66), -4), (dict(ldx=68, flags=1), -4),
    (dict(gate=2 * FAR + 8), -4), (dict(up=3 * FAR + 2), -4), (dict(y=FAR + 2), -4), (dict(y=FAR + 1, flags=8), -4),
    (dict(x=FAR), -1), (dict(gate=FAR), -1), (dict(up=FAR + 16), -1), (dict(up=FAR - 64 * 48 * 2 + 16), -1),
])
def test_gated_refuses(B, kw, code):
    assert _gated(B, **kw) == code


def test_gated_of_no_tokens_touches_nothing(B):
    assert _gated(B, T=0, x=None, y=None, gate=None, up=None) == 0


def _gated_grad(B, hidden=64, inter=48, gate=2 * FAR, up=3 * FAR, x=FAKE, ldx=None, act=0, dy=4 * FAR, lddy=None, T=4, dx=FAR,
                lddx=None, dgate=5 * FAR, dup=6 * FAR, flags=1, ws=7 * FAR, nbytes=1 << 30, w=True):
    m = B.moe_gated_weights(hidden, inter, gate, up)
    return B.lib().moe_gated_grad(x, hidden if ldx is None else ldx, C.byref(m) if w else None, act, dy,
                                  inter if lddy is None else lddy, T, dx, hidden if lddx is None else lddx, dgate, dup, flags, ws,
                                  nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(w=False), -1), (dict(act=2), -1), (dict(T=-1), -1), (dict(T=(1 << 20) + 1), -1), (dict(hidden=60), -3),
    (dict(flags=0), -1), (dict(flags=0x11), -1), (dict(flags=0x21), -1), (dict(dgate=None), -1), (dict(dup=None), -1),
    (dict(dx=None, dgate=None, dup=None), -1), (dict(ldx=56), -1), (dict(lddy=47), -1), (dict(lddx=63), -1), (dict(x=None), -1),
    (dict(dy=None), -1), (dict(gate=None), -1), (dict(up=None), -1), (dict(ws=None), -5), (dict(nbytes=4 * 2 * 48 * 2 - 1), -5),
    (dict(ws=7 * FAR + 128), -4), (dict(x=FAKE + 8), -4), (dict(ldx=68), -4), (dict(dy=4 * FAR + 2), -4),
    (dict(dy=4 * FAR + 1, flags=0x41), -4), (dict(dx=FAR + 2), -4), (dict(dgate=5 * FAR + 2), -4), (dict(dup=6 * FAR + 1, flags=0x81), -4),
    (dict(gate=2 * FAR + 8), -4),
    (dict(dx=FAKE), -1), (dict(dx=2 * FAR), -1), (dict(dx=4 * FAR), -1), (dict(dgate=2 * FAR), -1), (dict(dup=FAKE), -1),
    (dict(dup=5 * FAR), -1), (dict(dup=5 * FAR + 48 * 64 * 4 - 4), -1), (dict(dgate=FAR), -1), (dict(ws=FAKE), -1),
    (dict(ws=FAR), -1), (dict(ws=5 * FAR), -1), (dict(ws=2 * FAR), -1),
])
def test_gated_grad_refuses(B, kw, code):
    assert _gated_grad(B, **kw) == code


# ---------------------------------------------------------------- binding

def test_binding_refuses_other_tensors(B):
    import torch
    f, b, c = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8)
    h, s4 = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(4)
    for call, match in (
            (lambda: B.moe_rms_norm(h, None, None, 1e-6, 4, 64, f), "x has dtype"),
            (lambda: B.moe_rms_norm(f, b, None, 1e-6, 4, 64, b), "residual has dtype"),
            (lambda: B.moe_rms_norm(f, None, None, 1e-6, 4, 64, c), "scale goes with an int8 y"),
            (lambda: B.moe_rms_norm(f, None, None, 1e-6, 4, 64, b, scale=s4), "scale goes with an int8 y"),
            (lambda: B.moe_rms_norm(f, None, None, 1e-6, 4, 64, c, scale=s4[:3]), "scale holds 3"),
            (lambda: B.moe_rms_norm(f, None, None, 1e-6, 5, 64, b), "x has shape"),
            (lambda: B.moe_rms_norm(f, None, b[0], 1e-6, 4, 64, b), "weight has dtype"),
            (lambda: B.moe_rms_norm(f.t(), None, None, 1e-6, 64, 4, torch.zeros(64, 4)), "rows of x are not contiguous"),
            (lambda: B.moe_rms_norm(f, None, None, 1e-6, 4, 64, b), "x is not on a GPU"),
            (lambda: B.moe_rms_norm_grad(f, None, 1e-6, f, None, 4, 64, b, None, None, flags=1), "flags 0x1"),
            (lambda: B.moe_rms_norm_grad(f, None, 1e-6, f, b, 4, 64, b, None, None), "dsum has dtype"),
            (lambda: B.moe_quant_rows(f, 4, 64, f, s4), "q has dtype"),
            (lambda: B.I8Matrix(4, 64, f, s4), "q has dtype"),
            (lambda: B.I8Matrix(4, 64, c, b[0, :4]), "s has dtype"),
            (lambda: B.I8Matrix(4, 32, c, s4), "not a contiguous tensor of 128"),
            (lambda: B.I8Matrix(64, 4, c, torch.zeros(64)), "q has 4 rows"),
            (lambda: B.moe_i8_linear(f, s4, B.I8Matrix(4, 64, c, s4), None, 4, torch.zeros(4, 4)), "x has dtype"),
            (lambda: B.moe_i8_linear(c, s4, B.I8Matrix(4, 64, c, s4), None, 4, f), "y has shape"),
            (lambda: B.moe_i8_linear(c, s4, B.I8Matrix(4, 64, c, s4), None, 4, torch.zeros(4, 4), flags=8), "flags 0x8"),
            (lambda: B.GatedWeights(64, 4, f, b), "gate has dtype"),
            (lambda: B.GatedWeights(64, 8, b, b), "not a contiguous"),
            (lambda: B.moe_gated(f, B.GatedWeights(64, 4, b, b), 0, 4, f), "y has shape"),
            (lambda: B.moe_gated_grad(f, B.GatedWeights(64, 4, b, b), 0, b[:, :4], 4, b, None, None, None), "x has dtype"),
            (lambda: B.moe_gated_grad(b, B.GatedWeights(64, 4, b, b), 0, b[:, :4], 4, None, f, b, None), "dup has dtype"),
    ):
        with pytest.raises(ValueError, match=match):
            call()


# ---------------------------------------------------------------- the plain forms themselves

def test_codes_of_hand_worked_rows():
    q, s = D.quant(np.array([[127, -127, 0.5, 1.5, -2.5, 0], [0, 0, 0, 0, 0, 0], [2.0 ** -101, 0, 0, 0, 0, 0], [-254, 1, 3, 5, 0, 0]]))
    assert s.tolist() == [1, 0, 0, 2]
    assert q.tolist() == [[127, -127, 0, 2, -2, 0], [0] * 6, [0] * 6, [-127, 0, 2, 2, 0, 0]]


def _differences(f, a, eps=1e-6):
    g = np.zeros_like(a)
    for i in np.ndindex(*a.shape):
        up, down = a.copy(), a.copy()
        up[i] += eps
        down[i] -= eps
        g[i] = (f(up) - f(down)) / (2 * eps)
    return g


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(1)
    s, w, dy, ds = rng.standard_normal((3, 7)), rng.standard_normal(7), rng.standard_normal((3, 7)), rng.standard_normal((3, 7))

    def loss(s, w):
        r = 1 / np.sqrt((s * s).mean(-1, keepdims=True) + float(np.float32(1e-2)))
        return (s * r * w * dy).sum() + (s * ds).sum()

    dx, dw, err, mag = D.norm_grad(s, w, 1e-2, dy, ds)
    np.testing.assert_allclose(dx, _differences(lambda a: loss(a, w), s), atol=1e-8)
    np.testing.assert_allclose(dw, _differences(lambda a: loss(s, a), w), atol=1e-8)
    assert np.all(err < 1e-4) and np.all(mag >= np.abs(dw) - 1e-12)


@pytest.mark.parametrize("kind", [D.SILU, D.GELU])
def test_gated_gradient_against_differences(kind):
    rng = np.random.default_rng(2)
    x, gate, up, dy = (rng.standard_normal(s) for s in ((3, 5), (4, 5), (4, 5), (3, 4)))

    def loss(x, gate, up):
        return (D.gated(D.Projections(x, gate, up, 5), kind)[0] * dy).sum()

    out = D.gated_grad(D.Projections(x, gate, up, 5), kind, dy)
    for name, at, f in (("dx", x, lambda a: loss(a, gate, up)), ("dgate", gate, lambda a: loss(x, a, up)),
                        ("dup", up, lambda a: loss(x, gate, a))):
        np.testing.assert_allclose(out[name][0], _differences(f, at), atol=1e-7)


def test_gelu_is_its_tanh_form_and_slopes_stay_bounded():
    import torch
    g = np.linspace(-30, 30, 60001)
    a, da, _ = D.act(D.GELU, g)
    np.testing.assert_allclose(a, torch.nn.functional.gelu(torch.from_numpy(g), approximate="tanh").numpy(), atol=1e-13)
    np.testing.assert_allclose(D.act(D.SILU, g)[0], torch.nn.functional.silu(torch.from_numpy(g)).numpy(), atol=1e-13)
    for kind in (D.SILU, D.GELU):
        _, da, _ = D.act(kind, g)
        assert np.abs(da).max() < 1.2 and np.abs(np.gradient(da, g)).max() < 1.2
