"""Refusals of the Muon step and of the orthogonalising alone, and sizes of their
workspace (CPU only: no call here reaches a kernel launch)."""
import ctypes

import numpy as np
import pytest

import nf4_quantize_amd as nq
from nf4_quantize_amd import muon

FAKE = 0x10000  # a 256-byte-aligned, never dereferenced address
OK, NULL, SIZE, UNSUPPORTED, ALIGN, WORKSPACE = range(6)
BAD = ctypes.c_size_t(-1).value


def entries(*changes):
    e = np.zeros(max(1, len(changes)), muon._ENTRY)
    for name in ("w", "grad", "m"):
        e[name] = FAKE
    e["rows"], e["cols"], e["lr"], e["scale"] = 100, 16, 1e-3, 1.0
    for row, ch in zip(e, changes):
        for k, x in ch.items():
            row[k] = x
    return e


def config(**c):
    f = dict(momentum=0.95, eps=1e-7, a=3.4445, b=-4.775, c=2.0315, nesterov=1, iterations=5)
    f.update(c)
    return muon.nf4_muon_config(**f)


def size(e, count=None):
    return nq.lib().nf4_muon_workspace_size(e.ctypes.data, len(e) if count is None else count)


def step(e, count=None, wt=1, gt=1, mt=0, cfg=None, ws=FAKE, wsb=1 << 40):
    cfg = config() if cfg is None else cfg
    return nq.lib().nf4_muon_step(e.ctypes.data, len(e) if count is None else count, wt, gt, mt,
                                  ctypes.byref(cfg) if cfg else None, ws, wsb, None)


def orth(e, dt=1, cfg=None, ws=FAKE, wsb=1 << 40):
    cfg = config() if cfg is None else cfg
    return nq.lib().nf4_orthogonalize(e.ctypes.data, len(e), dt, ctypes.byref(cfg) if cfg else None, ws, wsb, None)


def test_layouts():
    assert ctypes.sizeof(muon.nf4_muon_config) == 48 and muon._ENTRY.itemsize == 64


def test_sizes():
    assert size(entries({}), count=0) == 0 and nq.lib().nf4_muon_workspace_size(None, 0) == 0
    assert nq.lib().nf4_muon_workspace_size(None, 1) == BAD and size(entries({}), count=-1) == BAD
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=257, cols=257), dict(rows=1 << 40), dict(rows=1 << 26), dict(rows=4, cols=1 << 28), dict(rows=1 << 62, cols=1 << 62)):
        assert size(entries({}, bad)) == BAD, bad
    small, large = size(entries({})), size(entries(dict(rows=4096, cols=256)))
    assert 0 < small < 1 << 16 and 5 * 256 * 256 * 8 < large < 64 << 20
    assert size(entries(dict(rows=0))) == size(entries(dict(cols=0)))
    # 448 adapters of rank 64
    many = entries(*[dict(rows=4096, cols=64), dict(rows=64, cols=14336)] * 224)
    assert size(many) < 160 << 20


@pytest.mark.parametrize("call", [step, orth])
def test_lists_refused(call):
    assert call(entries(dict(rows=0, w=0, grad=0))) == OK
    for ch, want in ((dict(rows=-1), SIZE), (dict(rows=300, cols=300), SIZE), (dict(w=0), NULL), (dict(grad=0), NULL),
                     (dict(w=FAKE + 8), ALIGN), (dict(grad=FAKE + 2), ALIGN)):
        assert call(entries({}, ch)) == want, ch
    for c in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(a=float("nan")), dict(b=float("inf")),
              dict(c=float("nan")), dict(iterations=0), dict(iterations=17)):
        assert call(entries({}), cfg=config(**c)) == SIZE, c
    assert call(entries({}), cfg=False) == NULL
    need = size(entries({}, {}))
    assert call(entries({}, {}), ws=None) == WORKSPACE
    assert call(entries({}, {}), wsb=need - 1) == WORKSPACE
    assert call(entries({}, {}), ws=FAKE + 128) == ALIGN
    # the list's last entry is looked at before anything is launched, however long it is
    for n in (33, 34, 35, 1000):
        assert call(entries(*[{}] * n, dict(w=0))) == NULL


def test_step_refused():
    assert step(entries({}), count=0) == OK and step(entries({}), count=-1) == SIZE
    assert nq.lib().nf4_muon_step(None, 1, 1, 1, 0, ctypes.byref(config()), FAKE, 1 << 40, None) == NULL
    for k in ("wt", "gt", "mt"):
        assert step(entries({}), **{k: 2}) == UNSUPPORTED
    for ch, want in ((dict(m=0), NULL), (dict(m=FAKE + 4), ALIGN), (dict(master=FAKE + 4), ALIGN), (dict(lr=float("nan")), SIZE),
                     (dict(weight_decay=float("inf")), SIZE), (dict(scale=float("nan")), SIZE)):
        assert step(entries({}, ch)) == want, ch
    assert step(entries(dict(master=FAKE)), wt=0) == UNSUPPORTED
    for c, want in ((dict(momentum=1.0), SIZE), (dict(momentum=-0.1), SIZE), (dict(momentum=float("nan")), SIZE),
                    (dict(nesterov=2), UNSUPPORTED)):
        assert step(entries({}), cfg=config(**c)) == want, c


def test_orthogonalize_refused():
    assert orth(entries({}), dt=2) == UNSUPPORTED
    # what the step alone reads is not looked at: the refusal is the next entry's
    assert orth(entries(dict(m=0, lr=float("nan"), master=FAKE + 1), dict(w=0))) == NULL


def test_binding_refuses():
    import torch

    with pytest.raises(ValueError):
        nq.NF4Muon([])
    with pytest.raises(ValueError, match="device tensors"):
        nq.NF4Muon([torch.zeros(3, 4)])
    for kw in (dict(state_bits=8), dict(momentum=1.0), dict(iterations=0), dict(eps=0.0), dict(coefficients=(1.0, 2.0))):
        with pytest.raises(ValueError):
            nq.NF4Muon([torch.zeros(3, 4)], **kw)
    assert nq.orthogonalize([]) == []
    with pytest.raises(ValueError, match="device tensors"):
        nq.orthogonalize([torch.zeros(3, 4)])
