"""Frequencies and arguments of the rotation of queries and keys (CPU only)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

import nf4_quantize_amd as nq
from nf4_quantize_amd import heads

FAKE = 0x10000  # a 16-byte-aligned, never dereferenced address
OK, NULL, SIZE, UNSUPPORTED, ALIGN, WORKSPACE = range(6)


def test_plain_frequencies():
    f, scale = nq.rotary_frequencies(8, base=10000.0)
    assert scale == 1.0 and np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-15)


def test_scaled_frequencies():
    plain, _ = nq.rotary_frequencies(64)
    linear, s = nq.rotary_frequencies(64, scaling=dict(kind="linear", factor=4))
    assert s == 1.0 and np.allclose(np.array(linear) * 4, plain, rtol=1e-15)
    ntk, _ = nq.rotary_frequencies(64, scaling=dict(kind="ntk", factor=4))
    assert ntk[0] == plain[0] and math.isclose(ntk[-1] * 4, plain[-1], rel_tol=1e-12)
    assert nq.rotary_frequencies(2, scaling=dict(kind="ntk", factor=4))[0] == [1.0]
    for kind, first, last in (("yarn", 32.0, 1.0), ("wavelength", 4.0, 1.0)):
        got, s = nq.rotary_frequencies(64, scaling=dict(kind=kind, factor=8, length=4096))
        assert math.isclose(s, 0.1 * math.log(8) + 1 if kind == "yarn" else 1.0)
        turns = np.array(plain) * 4096 / (2 * math.pi)
        ratio = np.array(plain) / np.array(got)
        # well inside the two ends; yarn's places are rounded to whole pairs
        assert np.allclose(ratio[turns > 2 * first], 1.0) and np.allclose(ratio[turns < last / 2], 8.0)
        assert (np.diff(ratio) >= -1e-9).all() and ((ratio > 1.01) & (ratio < 7.99)).any()
    assert nq.rotary_frequencies(64, scaling=dict(kind="yarn", factor=8, length=4096, attention=1.0))[1] == 1.0


@pytest.mark.parametrize("dim, base, scaling", [
    (7, 1e4, None), (0, 1e4, None), (8, -1.0, None), (8, float("inf"), None), (8, 1e4, dict(kind="other", factor=2)),
    (8, 1e4, dict(factor=2)), (8, 1e4, dict(kind="linear")), (8, 1e4, dict(kind="linear", factor=0)),
    (8, 1e4, dict(kind="linear", factor=2, length=3)), (8, 1e4, dict(kind="yarn", factor=2)),
    (8, 1e4, dict(kind="yarn", factor=2, length=100, slow=2, fast=1)),
    (8, 1.0, dict(kind="yarn", factor=2, length=100)),
    (8, 1e4, dict(kind="wavelength", factor=2, length=100, low=4, high=4))])
def test_frequencies_refused(dim, base, scaling):
    with pytest.raises(ValueError):
        nq.rotary_frequencies(dim, base, scaling)


def test_turns():
    rope = nq.NF4Rotary(64, device="cpu")
    for f, t in zip(rope.frequencies, rope.turns.tolist()):
        exact = Fraction(f) / heads.TWO_PI
        assert abs(Fraction(t % 2 ** 64, 2 ** 64) - exact % 1) <= Fraction(1, 2 ** 65)
    # negative frequencies and such above a turn a position turn by their remainder
    rope = nq.NF4Rotary(4, frequencies=[-0.5, 20.0], device="cpu")
    assert math.isclose(rope.turns[0].item() / 2 ** 64, -0.5 / (2 * math.pi), rel_tol=1e-12)
    assert math.isclose((rope.turns[1].item() % 2 ** 64) / 2 ** 64, (20 / (2 * math.pi)) % 1, rel_tol=1e-12)
    for kw in (dict(dim=6, frequencies=[1.0]), dict(dim=3), dict(dim=4, layout="pairs"), dict(dim=2, scale=float("nan")),
               dict(dim=2, frequencies=[float("inf")]), dict(dim=2, frequencies=[1.0], scaling=dict(kind="linear", factor=2))):
        with pytest.raises(ValueError):
            nq.NF4Rotary(device="cpu", **kw)


def shape(**c):
    f = dict(batch=2, tokens=3, heads_q=4, heads_k=1, dim=64, rotated=64, layout=0, dtype=1, w_dtype=1, eps=1e-6,
             w_offset=0.0, scale=1.0)
    f.update(c)
    return ctypes.byref(heads.nf4_rotary_shape(**f))


BAD_SHAPES = ((dict(batch=-1), SIZE), (dict(tokens=-1), SIZE), (dict(batch=1 << 30, tokens=2), SIZE),
              (dict(batch=1 << 62, tokens=1 << 62), SIZE), (dict(heads_q=-1), SIZE), (dict(heads_q=65537), SIZE),
              (dict(heads_k=-1), SIZE), (dict(heads_k=65537), SIZE), (dict(dim=0), SIZE), (dict(dim=513), SIZE),
              (dict(rotated=0), SIZE), (dict(rotated=66), SIZE), (dict(rotated=31), SIZE), (dict(layout=2), UNSUPPORTED),
              (dict(layout=-1), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(w_dtype=-1), UNSUPPORTED),
              (dict(eps=-1.0), SIZE), (dict(eps=float("nan")), SIZE), (dict(w_offset=float("inf")), SIZE),
              (dict(scale=float("nan")), SIZE))


def view(**c):
    f = dict(data=FAKE, batch_stride=768, token_stride=256, head_stride=64)
    f.update(c)
    return ctypes.byref(heads.nf4_heads(**f))


BAD_VIEWS = ((None, NULL), (view(data=None), NULL), (view(data=FAKE + 1), ALIGN), (view(batch_stride=-1), SIZE),
             (view(token_stride=-1), SIZE), (view(head_stride=-1), SIZE), (view(head_stride=(1 << 40) + 1), SIZE))


def test_structures():
    """The bytes that the binding packs are the structures'."""
    assert heads._SHAPE.size == ctypes.sizeof(heads.nf4_rotary_shape) == 56
    assert heads._HEADS.size == ctypes.sizeof(heads.nf4_heads) == 32
    fields = [(n, getattr(heads.nf4_rotary_shape, n).offset) for n, _ in heads.nf4_rotary_shape._fields_]
    s = heads.nf4_rotary_shape.from_buffer_copy(heads._SHAPE.pack(*range(1, 10), 10.0, 11.0, 12.0))
    assert [float(getattr(s, n)) for n, _ in fields] == [float(i) for i in range(1, 13)]


def test_forward_refusals():
    L = nq.lib()
    names = ("turns", "positions", "code", "stride", "q", "k", "w_q", "w_k", "q_out", "k_out")

    def fwd(sh, **c):
        f = dict(turns=FAKE, positions=FAKE, code=1, stride=0, q=view(), k=view(), w_q=FAKE, w_k=FAKE, q_out=view(),
                 k_out=view())
        f.update(c)
        return L.nf4_rotary_forward(sh, *(f[n] for n in names), None)

    for c, want in BAD_SHAPES:
        assert fwd(shape(**c)) == want, c
        assert L.nf4_rotary_backward_workspace_size(shape(**c)) == ctypes.c_size_t(-1).value
    assert fwd(None) == NULL
    for c in (dict(batch=0), dict(tokens=0), dict(heads_q=0, heads_k=0)):
        assert fwd(shape(**c), turns=None, q=None) == OK, c
    for n in ("q", "k", "q_out", "k_out"):
        for bad, want in BAD_VIEWS:
            assert fwd(shape(), **{n: bad}) == want, n
    assert fwd(shape(dtype=0), q=view(data=FAKE + 2)) == ALIGN
    assert fwd(shape(), turns=None) == NULL
    assert fwd(shape(), turns=FAKE + 4) == ALIGN
    assert fwd(shape(), positions=FAKE + 4) == ALIGN
    assert fwd(shape(), positions=FAKE + 2, code=0) == ALIGN
    assert fwd(shape(), code=2) == UNSUPPORTED
    assert fwd(shape(), stride=-1) == SIZE
    assert fwd(shape(), w_q=FAKE + 2) == ALIGN
    assert fwd(shape(), w_k=FAKE + 8) == ALIGN


def test_backward_refusals():
    L = nq.lib()
    names = ("turns", "positions", "code", "stride", "dq_out", "dk_out", "q", "k", "w_q", "w_k", "dq", "dk", "dw_q", "dw_k",
             "ws", "size")
    need = L.nf4_rotary_backward_workspace_size(shape())
    assert 0 < need < 1 << 24

    def bwd(sh, **c):
        f = {n: view() for n in ("dq_out", "dk_out", "q", "k", "dq", "dk")}
        f.update({n: FAKE for n in ("turns", "positions", "w_q", "w_k", "dw_q", "dw_k", "ws")})
        f.update(dict(code=1, stride=0, size=need))
        f.update(c)
        return L.nf4_rotary_backward(sh, *(f[n] for n in names), None)

    for c, want in BAD_SHAPES:
        assert bwd(shape(**c)) == want, c
    assert bwd(None) == NULL
    for n in ("dq_out", "dk_out", "q", "k", "dq", "dk"):
        for bad, want in BAD_VIEWS:
            assert bwd(shape(), **{n: bad}) == want, n
    assert bwd(shape(), turns=None) == NULL
    assert bwd(shape(), code=-1) == UNSUPPORTED
    assert bwd(shape(), w_q=None) == NULL  # its gradient is asked for
    assert bwd(shape(), dw_k=FAKE + 8) == ALIGN
    assert bwd(shape(), ws=None) == WORKSPACE
    assert bwd(shape(), size=need - 1) == WORKSPACE
    assert bwd(shape(), ws=FAKE + 128) == ALIGN
    assert bwd(shape(tokens=0), dw_q=None, dw_k=None, dq=None, turns=None) == OK


def test_binding_refuses_host_tensors():
    import torch

    rope = nq.NF4Rotary(8, device="cpu")
    q = torch.zeros(3, 2, 8)
    with pytest.raises(ValueError, match="device tensors"):
        nq.rotary_forward(q, None, None, rope)
    with pytest.raises(ValueError):
        nq.rotary_forward(None, q, None, rope)
    with pytest.raises(ValueError):
        nq.rotary_forward(q.view(-1), None, None, rope)
    with pytest.raises(ValueError):
        nq.rotary_backward(None, None, None, rope)


def test_slices_of_one_row_are_apart():
    """The host's question whether two tensors share an element, against the sets of their elements' addresses."""
    import torch

    rng = np.random.default_rng(5)
    seen = set()
    for _ in range(400):
        base = torch.zeros(4000, dtype=torch.float32)
        sizes = rng.integers(1, 4, 2)
        token = int(rng.integers(8, 40))
        batch = int(rng.choice([token * sizes[1], token * sizes[1] + 7, token]))

        def one():
            n, d = int(rng.integers(1, 4)), int(rng.integers(1, 5))
            return base.as_strided((int(sizes[0]), int(sizes[1]), n, d), (batch, token, d, 1), int(rng.integers(0, 30)))

        x, y = one(), one()
        at = [{t.storage_offset() + int(i) for i in (np.add.outer(np.add.outer(np.arange(t.shape[0]) * t.stride(0), np.arange(
            t.shape[1]) * t.stride(1)), np.arange(t.shape[2] * t.shape[3]))).ravel()} for t in (x, y)]
        said = heads._apart(x, y)
        seen.add((said, not (at[0] & at[1])))
        if said:
            assert not at[0] & at[1]
    assert (True, True) in seen and (False, False) in seen
