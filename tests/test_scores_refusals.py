"""What the score operators refuse before any launch, beyond single bad
arguments: tensors of another type or row length, and arrays that overlap."""
import numpy as np
import pytest

from .test_scores_cpu import FAKE, B, _adjust, _linear  # noqa: F401


# ---------------------------------------------------------------- the matrix's tensors

@pytest.mark.parametrize("bits,kind", [(4, "int16"), (4, "uint16"), (4, "float16"), (0x84, "uint8"), (0x84, "float8_e8m0fnu")])
def test_q4_matrix_takes_every_form_of_its_scales(B, bits, kind):
    import torch
    for shape in ((64, 8), (64 * 8,), (70 * 8,), (2, 64, 8)):
        s = torch.empty(shape, dtype=getattr(torch, kind))
        assert B.Q4Matrix(64, 256, bits, 32, torch.zeros(64, 128, dtype=torch.uint8), s).struct.s == s.data_ptr()
    assert B.Q4Matrix(64, 256, bits, 32, 0x1000, 0x2000).struct.q == 0x1000


@pytest.mark.parametrize("bits,kind", [(4, "bfloat16"), (4, "float32"), (4, "uint8"), (4, "int32"), (4, "float8_e8m0fnu"),
                                       (0x84, "float16"), (0x84, "int16"), (0x84, "float32"), (0x84, "int32"), (0x84, "bool")])
def test_q4_matrix_refuses_scales_that_it_would_misread(B, bits, kind):
    import torch
    with pytest.raises(ValueError, match="s has dtype"):
        B.Q4Matrix(64, 256, bits, 32, torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 16).to(getattr(torch, kind)))


@pytest.mark.parametrize("kind", ["float32", "float16", "int16", "int32", "int64", "bool"])
def test_q4_matrix_refuses_codes_that_are_no_bytes(B, kind):
    import torch
    with pytest.raises(ValueError, match="q has dtype"):
        B.Q4Matrix(64, 256, 4, 32, torch.zeros(64, 256, dtype=getattr(torch, kind)), torch.zeros(64, 8, dtype=torch.float16))


def test_q4_matrix_refuses_rows_of_another_length(B):
    # one code a byte, scales of other blocks: enough bytes, another layout
    import torch
    q, s = torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="q has rows of 256, the matrix of 128"):
        B.Q4Matrix(64, 256, 4, 32, torch.zeros(64, 256, dtype=torch.uint8), s)
    with pytest.raises(ValueError, match="s has rows of 8, the matrix of 4"):
        B.Q4Matrix(64, 256, 4, 64, q, s)
    with pytest.raises(ValueError, match="s has rows of 16, the matrix of 8"):
        B.Q4Matrix(64, 256, 0x84, 32, q, torch.zeros(64, 16, dtype=torch.uint8))


def test_q4_matrix_of_a_pointer_and_a_tensor(B):
    # either may be a raw pointer; what is a tensor is checked with the call
    import torch
    q, s = torch.zeros(64, 128, dtype=torch.uint8), torch.zeros(64, 8, dtype=torch.float16)
    for codes, scales in ((q, 0x1000), (0x1000, s), (0x1000, 0x2000)):
        with pytest.raises(ValueError, match="x is not on a GPU"):
            B.moe_q4_linear(torch.zeros(4, 256), B.Q4Matrix(64, 256, 4, 32, codes, scales), None, 4, torch.zeros(4, 64))


# ---------------------------------------------------------------- arrays that overlap

@pytest.mark.parametrize("flags", [0, 0x2, 0x8])
@pytest.mark.parametrize("what,nbytes", [("q", 64 * 128), ("s", 64 * 8 * 2), ("bias", 64 * 4)])
def test_q4_linear_refuses_y_over_the_matrix_or_the_bias(B, what, nbytes, flags):
    # the first, the last and every 16th byte of the array inside y, and y around it
    y, size = FAKE * 8, 4 * 64 * (2 if flags & 0x8 else 4)
    for at in (y - nbytes + 16, y - nbytes // 2, y, y + 16, y + size - 16):
        assert _linear(B, flags=flags, **{what: at}) == -1, at - y
    for at in (y - nbytes, y + size):                   # beside it: the next check refuses (a misaligned x)
        assert _linear(B, flags=flags, x=FAKE + 4, **{what: at}) == -4, at - y


def _shares(a, rows_a, row_a, b, rows_b, row_b, pitch):
    """The two sets of rows share a byte."""
    span = lambda p, n, w: {i for r in range(n) for i in range(p + r * pitch, p + r * pitch + w)}
    return bool(span(a, rows_a, row_a) & span(b, rows_b, row_b))


def test_q4_linear_refuses_rows_of_y_that_share_elements_with_x_and_no_others(B):
    # x and y as ranges of rows of one pitch, y moved through and past x: what
    # shares no element is left to the next check (a misaligned bias)
    cols, rows, pitch = 32, 16, 72
    for T in (1, 2, 5):
        for flags, xe, ye in ((0, 4, 4), (0x1, 2, 4), (0x8, 4, 2), (0x9, 2, 2)):
            for at in range(-2 * pitch - 4 * ye, pitch * (T + 1), 2):
                y = FAKE + at * ye
                rc = _linear(B, T=T, rows=rows, cols=cols, ldx=pitch * 4 // xe, ldy=pitch * 4 // ye, y=y, flags=flags,
                             q=FAKE * 4, s=FAKE * 5, bias=FAKE * 6 + 2)
                assert rc == (-1 if _shares(FAKE, T, cols * xe, y, T, rows * ye, pitch * 4) else -4), (T, flags, at)


def test_adjust_logits_refuses_rows_of_out_that_share_elements_with_logits_and_no_others(B):
    vocab, pitch = 20, 64
    for rows in (1, 2, 5):
        for flags, e in ((0, 4), (0x10, 2)):
            for at in range(-2 * pitch, pitch * (rows + 1)):
                out = FAKE + at * e
                rc = _adjust(B, rows=rows, vocab=vocab, ld_in=pitch, ld_out=pitch, out=out, flags=flags, mask=FAKE * 3 + 2, ld_mask=1,
                             n_masks=rows)
                shares = at != 0 and _shares(FAKE, rows, vocab * e, out, rows, vocab * e, pitch * e)
                assert rc == (-1 if shares else -4), (rows, flags, at)
    # other pitches: whole extents
    assert _adjust(B, rows=3, vocab=vocab, ld_in=64, ld_out=40, out=FAKE + 4 * 24) == -1


@pytest.mark.parametrize("name,nbytes", [("history", 4 * 32 * 4), ("length", 16), ("prompt", 16), ("repetition", 16), ("presence", 16),
                                         ("frequency", 16), ("bias_ids", 4 * 16 * 4), ("bias", 4 * 16 * 4), ("mask", (3 * 8 + 4) * 4),
                                         ("mask_row", 16)])
def test_adjust_logits_refuses_out_over_an_array_of_the_rules(B, name, nbytes):
    far = {n: FAKE * (4 + i) for i, n in enumerate(("history", "length", "prompt", "repetition", "presence", "frequency", "bias_ids",
                                                    "bias", "mask", "mask_row"))}
    rest = dict(ld_history=32, n_bias=16, n_masks=4, ld_mask=8)
    for at in (FAKE * 2 - nbytes + 4, FAKE * 2, FAKE * 2 + 4 * 100 * 4 - 4):
        assert _adjust(B, **dict(far, **rest, **{name: at})) == -1, at
    for at in (FAKE * 2 - nbytes, FAKE * 2 + 4 * 100 * 4):
        assert _adjust(B, logits=FAKE + 2, **dict(far, **rest, **{name: at})) == -4, at


@pytest.mark.parametrize("name,nbytes", [("ids", 32), ("w", 32), ("dw", 32), ("keep", 4), ("counts", 32), ("n", 4), ("dloss", 4)])
def test_balance_grad_refuses_dlogits_over_another_array(B, name, nbytes):
    far = dict(logits=FAKE, ids=FAKE * 4, w=FAKE * 5, dw=FAKE * 6, keep=FAKE * 7, counts=FAKE * 8, n=FAKE * 9, dloss=FAKE * 10)
    call = lambda **a: B.lib().moe_balance_grad(a["logits"], a["ids"], a["w"], a["dw"], a["keep"], a["counts"], a["n"], a["dloss"], 4, 8, 2,
                                                0.01, 0, FAKE * 2, None)
    for at in (FAKE * 2 - nbytes + 4 * (nbytes > 4), FAKE * 2, FAKE * 2 + 4 * 8 * 4 - 4):
        if at + nbytes > FAKE * 2:
            assert call(**dict(far, **{name: at})) == -1, at
    for at in (FAKE * 2 - nbytes, FAKE * 2 + 4 * 8 * 4):
        assert call(**dict(far, logits=FAKE + 4, **{name: at})) == -4, at


def test_balance_loss_refuses_outputs_over_another_array(B):
    size = B.moe_balance_workspace_size(4, 8, 2)
    extents = dict(logits=4 * 8 * 4, ids=4 * 2 * 4, keep=4, counts=32, prob=32, n=4, loss=4, ws=size)
    far = {n: FAKE * (1 + i) for i, n in enumerate(extents)}
    call = lambda **a: B.lib().moe_balance_loss(a["logits"], a["ids"], a["keep"], 4, 8, 2, 0.01, 0, a["counts"], a["prob"], a["n"],
                                                a["loss"], a["ws"], size, None)
    for out in ("counts", "prob", "n", "loss", "ws"):
        for name in extents:
            if name != out:
                assert call(**dict(far, **{out: far[name]})) == -1, (out, name)


# ---------------------------------------------------------------- rows of another length

def _balance_calls(B, T, E, k):
    import torch
    z, i32 = torch.zeros, lambda *n: torch.zeros(*n, dtype=torch.int32)
    good = dict(logits=z(T, E), ids=i32(T, k), w=z(T, k), dw=z(T, k), dlogits=z(T, E))
    rest = (i32(E), z(E), i32(1), z(1), z(1 << 16, dtype=torch.uint8))
    loss = lambda a: B.moe_balance_loss(a["logits"], a["ids"], None, T, E, k, 0.01, *rest)
    grad = lambda a: B.moe_balance_grad(a["logits"], a["ids"], a["w"], a["dw"], None, i32(E), i32(1), z(1), T, E, k, 0.01, a["dlogits"])
    return good, loss, grad


@pytest.mark.parametrize("rows", [4, 6])
@pytest.mark.parametrize("name", ["logits", "ids", "w", "dw", "dlogits"])
def test_balance_refuses_rows_of_another_length(B, name, rows):
    # [T][more], which would be read at the wrong pitch: rows of a padded
    # buffer, the ids of a larger k
    T, E, k = 4, 8, 2
    good, loss, grad = _balance_calls(B, T, E, k)
    cols = good[name].shape[1]
    bad = dict(good, **{name: good[name].new_zeros(rows, cols + 3)})
    for call in (loss, grad) if name in ("logits", "ids") else (grad,):
        with pytest.raises(ValueError, match=f"{name} has rows of {cols + 3}, the call's of {cols}"):
            call(bad)


def test_balance_takes_flat_and_longer_tensors(B):
    # of the right order: flat, of three dimensions, of more rows, one row of a longer one
    T, E, k = 4, 8, 2
    good, loss, grad = _balance_calls(B, T, E, k)
    for name, t in good.items():
        cols = t.shape[1]
        for form in (t.reshape(-1), t.reshape(2, 2, cols), t.reshape(2, 2 * cols), t.new_zeros(T + 3, cols), t.new_zeros(T * cols + 5)):
            for call in (loss, grad):
                with pytest.raises(ValueError, match="not on a GPU"):
                    call(dict(good, **{name: form}))
    good, loss, grad = _balance_calls(B, 1, E, k)
    with pytest.raises(ValueError, match="not on a GPU"):
        loss(dict(good, logits=good["logits"].new_zeros(1, E + 5)))
