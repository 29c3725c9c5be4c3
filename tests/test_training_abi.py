"""Refusals of the training-step operators: bad arguments are turned away on the
host before any HIP call (CPU only: no call here reaches a kernel launch)."""
import ctypes
import os

import numpy as np
import pytest

import nf4_quantize_amd as nq
from nf4_quantize_amd import training

FAKE = 0x10000  # a 16-byte-aligned, never dereferenced address
OK, NULL, SIZE, UNSUPPORTED, ALIGN, WORKSPACE = range(6)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nq.LIB_PATH):
        from nf4_quantize_amd import build

        build.build()
    return nq.lib()


def entries(*changes):
    e = np.zeros(max(1, len(changes)), training._ENTRY)
    for name in ("w", "grad", "m", "v", "m_scale", "v_scale"):
        e[name] = FAKE
    e["n"], e["lr"] = 1000, 1e-3
    for row, ch in zip(e, changes):
        for k, x in ch.items():
            row[k] = x
    return e


def adamw(L, e, count=None, wt=1, gt=1, moments=8, norm=None, cfg=True, ws=None, wsb=0, **c):
    f = dict(beta1=0.9, beta2=0.999, eps=1e-8, max_norm=0.0, step=1, seed=0)
    f.update(c)
    config = training.nf4_adamw_config(**f)
    return L.nf4_adamw_step(e.ctypes.data, len(e) if count is None else count, wt, gt, moments,
                            ctypes.byref(config) if cfg else None, norm, ws, wsb, None)


def test_adamw_refusals(L):
    assert ctypes.sizeof(training.nf4_adamw_config) == 40 and training._ENTRY.itemsize == 72
    bad = {}  # the last entry of each list is the bad one: those before it launch nothing either
    assert adamw(L, entries({}), count=0) == OK
    assert adamw(L, entries({"n": 0, "w": 0, "grad": 0})) == OK
    assert adamw(L, entries({}), count=-1) == SIZE
    assert L.nf4_adamw_step(None, 2, 1, 1, 8, None, None, None, 0, None) == NULL
    assert adamw(L, entries(bad), cfg=False) == NULL
    assert adamw(L, entries(bad), wt=2) == UNSUPPORTED
    assert adamw(L, entries(bad), gt=-1) == UNSUPPORTED
    assert adamw(L, entries(bad), moments=16) == UNSUPPORTED
    for k in ("w", "grad", "m", "v", "m_scale", "v_scale"):
        assert adamw(L, entries({}, {k: 0})) == NULL, k
        off = FAKE + (2 if "scale" in k else 8)
        assert adamw(L, entries({}, {k: off})) == ALIGN, k
    assert adamw(L, entries({}, {"n": -1})) == SIZE
    assert adamw(L, entries({}, {"n": (1 << 33) + 1})) == SIZE
    assert adamw(L, entries({}, {"lr": float("nan")})) == SIZE
    assert adamw(L, entries({}, {"weight_decay": float("inf")})) == SIZE
    assert adamw(L, entries({}, {"master": FAKE}), wt=0) == UNSUPPORTED
    assert adamw(L, entries({}, {"master": FAKE + 4})) == ALIGN
    for c in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1.0),
              dict(step=0), dict(max_norm=float("nan"))):
        assert adamw(L, entries(bad), **c) == SIZE, c
    assert adamw(L, entries(bad), max_norm=1.0) == NULL       # clipping without a norm
    assert adamw(L, entries(bad), norm=FAKE + 2) == ALIGN
    # more entries than the kernel arguments hold go through the workspace
    size = L.nf4_adamw_workspace_size
    assert size(48) == 0 and size(49) == 49 * 84 and size(-1) == ctypes.c_size_t(-1).value
    many = entries(*[{}] * 49)
    assert adamw(L, many) == WORKSPACE
    assert adamw(L, many, ws=FAKE, wsb=size(49) - 1) == WORKSPACE
    assert adamw(L, many, ws=FAKE + 128, wsb=size(49)) == ALIGN
    # 32-bit moments have no scales: the refusal of the entry after shows that this one passed
    assert adamw(L, entries({"m_scale": 0, "v_scale": 0}, {"w": 0}), moments=32) == NULL


def test_grad_norm_refusals(L):
    e = entries({}, {"n": 16385}, {"n": 0})
    size = L.nf4_grad_norm_workspace_size
    assert size(e.ctypes.data, 3) == 8 * (1 + 2)
    assert size(None, 0) == 0
    assert size(None, 1) == ctypes.c_size_t(-1).value
    assert size(entries({"n": -1}).ctypes.data, 1) == ctypes.c_size_t(-1).value

    def norm(e, gt=1, out=FAKE, ws=FAKE, b=24):
        return L.nf4_grad_norm(e.ctypes.data, len(e), gt, out, ws, b, None)

    assert norm(e, gt=3) == UNSUPPORTED
    assert norm(e, out=None) == NULL
    assert norm(e, out=FAKE + 1) == ALIGN
    assert norm(e, ws=None) == WORKSPACE
    assert norm(e, b=23) == WORKSPACE
    assert norm(e, ws=FAKE + 16) == ALIGN
    assert norm(entries({}, {"grad": 0})) == NULL
    assert norm(entries({}, {"grad": FAKE + 2})) == ALIGN
    assert norm(entries({"n": -2})) == SIZE


def shape(**c):
    f = dict(rows=4, dim=64, dtype=1, res_dtype=1, w_dtype=1, gate_kind=1, eps=1e-6, alpha=1.0, w_offset=0.0)
    f.update(c)
    return ctypes.byref(training.nf4_residual_norm_shape(**f))


BAD_SHAPES = ((dict(rows=-1), SIZE), (dict(dim=0), SIZE), (dict(dim=32769), SIZE), (dict(rows=1 << 32, dim=64), SIZE),
              (dict(dtype=2), UNSUPPORTED), (dict(res_dtype=5), UNSUPPORTED), (dict(w_dtype=-1), UNSUPPORTED),
              (dict(dtype=0, res_dtype=1), UNSUPPORTED), (dict(gate_kind=3), UNSUPPORTED), (dict(eps=-1.0), SIZE),
              (dict(alpha=float("inf")), SIZE), (dict(w_offset=float("nan")), SIZE))


def test_residual_norm_refusals(L):
    names = ("y", "h", "w_post", "gate", "w_pre", "h_out", "x_out", "rstd_post", "rstd_pre")

    def fwd(sh, **c):
        return L.nf4_residual_norm_forward(sh, *(c.get(k, FAKE) for k in names), None)

    for c, want in BAD_SHAPES:
        assert fwd(shape(**c)) == want, c
        assert L.nf4_residual_norm_backward_workspace_size(shape(**c)) == ctypes.c_size_t(-1).value
    assert fwd(None) == NULL
    assert fwd(shape(rows=0), h=None) == OK
    for k in ("h", "w_pre", "x_out", "h_out", "gate"):
        assert fwd(shape(), **{k: None}) == NULL, k
    for k in names:
        assert fwd(shape(), **{k: FAKE + 2}) == ALIGN, k
    names_b = ("dx", "dh_out", "y", "h_out", "w_post", "gate", "w_pre", "rstd_post", "rstd_pre", "dy", "dh", "dgate",
               "dw_pre", "dw_post")
    need = L.nf4_residual_norm_backward_workspace_size(shape())
    assert need > 0

    def bwd(sh, ws=FAKE, b=need, **c):
        return L.nf4_residual_norm_backward(sh, *(c.get(k, FAKE) for k in names_b), ws, b, None)

    for c, want in BAD_SHAPES:
        assert bwd(shape(**c)) == want, c
    for k in ("h_out", "w_pre", "rstd_pre", "rstd_post", "gate", "w_post"):  # dw_post needs w_post
        assert bwd(shape(), **{k: None}) == NULL, k
    assert bwd(shape(gate_kind=0)) == NULL  # dgate without a gate
    for k in names_b:
        assert bwd(shape(), **{k: FAKE + 2}) == ALIGN, k
    assert bwd(shape(), ws=None) == WORKSPACE
    assert bwd(shape(), b=need - 1) == WORKSPACE
    assert bwd(shape(), ws=FAKE + 64) == ALIGN
    assert bwd(shape(rows=0), ws=None, b=0, dw_pre=None, dw_post=None, dgate=None) == OK


def test_embedding_refusals(L):
    def fwd(ids=FAKE, it=1, tokens=10, table=FAKE, dt=1, vocab=100, dim=64, out=FAKE, ot=1):
        return L.nf4_embedding_forward(ids, it, tokens, table, dt, vocab, dim, 1.0, out, ot, None)

    def bwd(ids=FAKE, it=1, tokens=10, dy=FAKE, dt=1, vocab=100, dim=64, grad=FAKE, gt=1, ws=FAKE, b=1 << 20):
        return L.nf4_embedding_backward(ids, it, tokens, dy, dt, vocab, dim, 1.0, -1, grad, gt, 0, ws, b, None)

    for call in (fwd, bwd):
        assert call(tokens=-1) == SIZE
        assert call(tokens=(1 << 28) + 1) == SIZE
        assert call(vocab=0) == SIZE
        assert call(vocab=(1 << 28) + 1) == SIZE
        assert call(dim=0) == SIZE
        assert call(vocab=1 << 28, dim=1 << 10) == SIZE
        assert call(it=2) == UNSUPPORTED
        assert call(dt=7) == UNSUPPORTED
        assert call(ids=None) == NULL
        assert call(ids=FAKE + 4) == ALIGN
    assert fwd(tokens=0, ids=None, table=None) == OK
    assert fwd(ot=9) == UNSUPPORTED
    assert fwd(table=None) == NULL and fwd(out=None) == NULL
    assert fwd(table=FAKE + 8) == ALIGN and fwd(out=FAKE + 2) == ALIGN
    assert fwd(it=0, ids=FAKE + 2) == ALIGN
    assert bwd(gt=9) == UNSUPPORTED
    assert bwd(dy=None) == NULL and bwd(grad=None) == NULL
    assert bwd(dy=FAKE + 8) == ALIGN and bwd(grad=FAKE + 4) == ALIGN
    need = L.nf4_embedding_backward_workspace_size(10, 100, 64)
    assert need > 0 and L.nf4_embedding_backward_workspace_size(0, 100, 64) == 0
    assert L.nf4_embedding_backward_workspace_size(-1, 100, 64) == ctypes.c_size_t(-1).value
    assert bwd(ws=None) == WORKSPACE and bwd(b=need - 1) == WORKSPACE and bwd(ws=FAKE + 16) == ALIGN

    def packed(w, ids=FAKE, it=1, tokens=10, out=FAKE, ot=1):
        return L.nf4_embedding_forward_packed(ids, it, tokens, w, 1.0, out, ot, None)

    def weight(n=100, k=128, codes=FAKE, aq=FAKE, asc=FAKE, am=None, bs=64, dq=256):
        return ctypes.byref(nq.nf4_weight(codes=codes, absmax_q=aq, absmax_scale=asc, absmax=am, n_out=n, k_in=k,
                                          blocksize=bs, dq_blocksize=dq))

    assert packed(None) == NULL
    assert packed(weight(k=100)) == SIZE and packed(weight(n=0)) == SIZE
    assert packed(weight(bs=32)) == UNSUPPORTED and packed(weight(dq=64)) == UNSUPPORTED
    assert packed(weight(), it=5) == UNSUPPORTED and packed(weight(), ot=5) == UNSUPPORTED
    assert packed(weight(), tokens=0, ids=None) == OK
    for w in (weight(codes=None), weight(aq=None), weight(aq=None, asc=None)):
        assert packed(w) == NULL
    assert packed(weight(), ids=None) == NULL and packed(weight(), out=None) == NULL
    assert packed(weight(codes=FAKE + 4)) == ALIGN and packed(weight(asc=FAKE + 1)) == ALIGN
    assert packed(weight(aq=None, asc=None, am=FAKE + 2)) == ALIGN and packed(weight(), out=FAKE + 8) == ALIGN


def test_binding_refusals():
    """What the Python side refuses before it calls the library: host tensors, lists
    that do not fit, wrong shapes and types."""
    import torch

    w = torch.zeros(4, 4)
    for bad in (dict(params=[]), dict(params=[w], state_bits=4), dict(params=[w]),
                dict(params=[dict(params=[w], masters=[])])):
        with pytest.raises(ValueError):
            nq.NF4AdamW(**bad)
    with pytest.raises(TypeError):
        nq.NF4AdamW([torch.zeros(4, dtype=torch.float16)])
    with pytest.raises(ValueError):
        nq.residual_norm_forward(w, w, torch.ones(4))
    with pytest.raises(ValueError):
        training._norm_shape(w, torch.zeros(4, 5), torch.ones(5), None, None, 1.0, 1e-6, 0.0)
    with pytest.raises(ValueError):
        training._norm_shape(w, w, torch.ones(5), None, None, 1.0, 1e-6, 0.0)
    with pytest.raises(ValueError):
        training._norm_shape(w, w, torch.ones(4), torch.ones(4).double(), None, 1.0, 1e-6, 0.0)
    with pytest.raises(ValueError):
        training._norm_shape(w, w, torch.ones(4), None, torch.ones(3), 1.0, 1e-6, 0.0)
    with pytest.raises(TypeError):
        training._norm_shape(w, w, torch.ones(4), None, torch.ones(4).bfloat16(), 1.0, 1e-6, 0.0)
    with pytest.raises(ValueError):
        nq.embedding_forward(torch.zeros(3, dtype=torch.int64), w)
    with pytest.raises(ValueError):
        nq.embedding_forward(torch.zeros(3, dtype=torch.int64), torch.zeros(4))
    with pytest.raises(ValueError):
        nq.embedding_backward(torch.zeros(3, dtype=torch.int64), torch.zeros(2, 4), 10)
    with pytest.raises(TypeError):
        training._index_code(torch.zeros(3, dtype=torch.int16))


def test_adamw_clip_refusals(L):
    """What the norm's call and the step refuse; the norm is written, so it has to be there."""
    def clip(e, norm=FAKE, ws=FAKE, b=1 << 20, wt=1, gt=1, **c):
        f = dict(beta1=0.9, beta2=0.999, eps=1e-8, max_norm=1.0, step=1, seed=0)
        f.update(c)
        return L.nf4_adamw_clip_step(e.ctypes.data, len(e), wt, gt, 8, ctypes.byref(training.nf4_adamw_config(**f)),
                                     norm, ws, b, None)

    assert L.nf4_adamw_clip_step(None, 2, 1, 1, 8, None, None, None, 0, None) == NULL
    assert clip(entries({}), norm=None) == NULL
    assert clip(entries({}), norm=None, max_norm=0.0) == NULL
    assert clip(entries({}), norm=FAKE + 2) == ALIGN
    assert clip(entries({}), ws=None) == WORKSPACE
    assert clip(entries({}, {"n": 16385}), b=23) == WORKSPACE
    assert clip(entries(*[{}] * 49), b=49 * 84 - 1) == WORKSPACE
    assert clip(entries({}), ws=FAKE + 64) == ALIGN
    assert clip(entries({}), gt=2) == UNSUPPORTED
    assert clip(entries({}), beta1=1.0) == SIZE
    for k in ("w", "grad", "m", "v", "m_scale", "v_scale"):
        assert clip(entries({}, {k: 0})) == NULL, k
