"""The training step around the 4-bit linears: AdamW over a list of adapter
tensors (``NF4AdamW``), the residual norms between blocks (``residual_norm``)
and the token embedding (``nf4_embedding``). Formulas, storage and limits are
in ``include/nf4.h``; every step of the computation runs in the library's HIP
kernels, torch supplies device memory and the current stream.
"""
import array
import ctypes
import operator

import numpy as np

import nf4_quantize_amd as _nq

MOMENT_BLOCK = 256
GATE_KINDS = {"none": 0, "channel": 1, "token": 2}

# nf4_adamw_entry, as one row of a host array.
_ENTRY = np.dtype([("w", "u8"), ("master", "u8"), ("grad", "u8"), ("m", "u8"), ("v", "u8"), ("m_scale", "u8"),
                   ("v_scale", "u8"), ("n", "i8"), ("lr", "f4"), ("weight_decay", "f4")])


class nf4_adamw_config(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_float),
                ("max_norm", ctypes.c_float), ("step", ctypes.c_int64), ("seed", ctypes.c_uint64)]


class nf4_residual_norm_shape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("eps", ctypes.c_float), ("alpha", ctypes.c_float), ("w_offset", ctypes.c_float)]


def declare(L):
    """argtypes and restypes of this module's entry points."""
    p, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    shape, weight = ctypes.POINTER(nf4_residual_norm_shape), ctypes.POINTER(_nq.nf4_weight)
    for name, restype, args in (
            ("nf4_grad_norm_workspace_size", sz, [p, i32]),
            ("nf4_grad_norm", i32, [p, i32, i32, p, p, sz, p]),
            ("nf4_adamw_step", i32, [p, i32, i32, i32, i32, ctypes.POINTER(nf4_adamw_config), p, p, sz, p]),
            ("nf4_adamw_clip_step", i32, [p, i32, i32, i32, i32, ctypes.POINTER(nf4_adamw_config), p, p, sz, p]),
            ("nf4_adamw_workspace_size", sz, [i32]),
            ("nf4_residual_norm_forward", i32, [shape] + [p] * 10),
            ("nf4_residual_norm_backward_workspace_size", sz, [shape]),
            ("nf4_residual_norm_backward", i32, [shape] + [p] * 15 + [sz, p]),
            ("nf4_embedding_forward", i32, [p, i32, i64, p, i32, i64, i64, f32, p, i32, p]),
            ("nf4_embedding_forward_packed", i32, [p, i32, i64, weight, f32, p, i32, p]),
            ("nf4_embedding_backward_workspace_size", sz, [i64, i64, i64]),
            ("nf4_embedding_backward", i32, [p, i32, i64, p, i32, i64, i64, f32, i64, p, i32, i32, p, sz, p])):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = restype, args


def _size(value, what):
    if value == ctypes.c_size_t(-1).value:
        raise _nq.NF4Error(2, what)
    return int(value)


def _addr(t):
    return None if t is None else t.data_ptr()


def _check_tensors(first, *ts):
    """Contiguous tensors of the first one's device (None: absent). Returns the
    device's index. These checks run before every call: they ask each tensor two
    plain questions and build no objects."""
    index = first.get_device()
    if index < 0 or not first.is_contiguous():
        raise ValueError("tensors must be contiguous device tensors")
    for t in ts:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous device tensors"
                             if t.get_device() < 0 or not t.is_contiguous() else
                             f"tensors of one call are on one device, got {first.device} and {t.device}")
    return index


def _check_apart(ts):
    """No two of the tensors share memory: a launch updates them all at once."""
    end = 0
    for at, size in sorted([(t.data_ptr(), t.nbytes) for t in ts]):
        if size and at < end:
            raise ValueError("two of an optimizer's weights, masters and moments share memory")
        end = max(end, at + size)


_TORCH = {}


def _torch(name):
    """Functions of torch that every call needs (torch is imported by the first one)."""
    if not _TORCH:
        import torch

        _TORCH.update(stream=torch._C._cuda_getCurrentRawStream, changed=torch.autograd.graph.increment_version)
    return _TORCH[name]


def _stream(index):
    """The current stream of a device, as _nq._stream without its objects."""
    return _torch("stream")(index)


def _changed(ts):
    """Tells autograd that this tensor, or these, were written: a graph that saved one
    of them refuses to run backward from then on."""
    _torch("changed")(ts)


_CODES = {}


def _code(dtype):
    """_nq._dtype_code, looked up."""
    if not _CODES:
        import torch

        _CODES.update({torch.float32: _nq.NF4_F32, torch.bfloat16: _nq.NF4_BF16})
    code = _CODES.get(dtype)
    return _nq._dtype_code(dtype) if code is None else code


# ------------------------------------------------------------------ AdamW

def _taken(name):
    """The list of the tensors whose addresses a step takes, made on first use. A step
    refuses to run where the caller has put others in."""

    def tensors(self):
        if name not in self._taken:
            raise AttributeError(f"32-bit moments have no {name}")
        return self._given.setdefault(name, list(self._taken[name]))

    return property(tensors)


class NF4AdamW:
    """AdamW over a list of device tensors in a few launches, with the moments in
    8 bits (E4M3 codes with one fp32 scale per 256 elements, rounded
    stochastically) or in 32, and clipping by the norm of all its list's gradients
    (each optimizer by its own: a list has one dtype).

    ``params``: tensors, or groups ``dict(params=[...], lr=..., weight_decay=...,
    masters=[...])``; all have one dtype (bfloat16 or float32), and no two share
    memory. ``masters`` are the fp32 weights of bfloat16 parameters: the step
    updates them and rounds them into the parameters (``masters=True``: made here
    from the parameters). ``max_grad_norm`` > 0 clips; a step whose norm is not
    finite then changes none of these tensors and no moment, but it counts in
    ``steps``, the step number of the bias corrections, like any other (``step=``
    gives a call another number). ``seed`` starts the random bits of the stochastic
    rounding; each step takes the next ones.

    ``m``, ``v`` (and ``m_scale``, ``v_scale``) are the lists of the tensors'
    moments in the order of the parameters. A step writes at these tensors' addresses,
    so ``bind_state`` replaces them, and a step refuses lists whose tensors are others,
    ``params`` and ``masters`` too (a parameter's ``data`` may change). ``grad_norm`` is
    the last norm (a device tensor of one float)."""

    params, masters, m, v, m_scale, v_scale = map(_taken, ("params", "masters", "m", "v", "m_scale", "v_scale"))

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, state_bits=8,
                 max_grad_norm=0.0, seed=0, masters=None):
        import torch

        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        params = list(params)
        if not params:
            raise ValueError("no parameters")
        if not isinstance(params[0], dict):
            params = [dict(params=params, masters=masters)]
        elif masters is not None:
            raise ValueError("masters belong to the groups")
        self.groups = []
        self._params, self._masters = [], []
        for g in params:
            ps = list(g["params"])
            ms = g.get("masters")
            if ms is True:
                ms = [p.detach().float().contiguous() for p in ps]
            ms = [None] * len(ps) if ms is None else list(ms)
            if len(ms) != len(ps):
                raise ValueError(f"{len(ms)} masters for {len(ps)} parameters")
            self.groups.append(dict(lr=float(g.get("lr", lr)), weight_decay=float(g.get("weight_decay", weight_decay)),
                                    first=len(self._params), count=len(ps)))
            self._params += ps
            self._masters += ms
        if not self._params:
            raise ValueError("no parameters")
        self._taken, self._given = dict(params=tuple(self._params), masters=tuple(self._masters)), {}
        self.dtype, self.device = self._params[0].dtype, self._params[0].device
        _nq._dtype_code(self.dtype)
        self._tensor = torch.Tensor
        self._entries = np.zeros(len(self._params), _ENTRY)
        self._at = self._entries.ctypes.data
        self._numels = [p.numel() for p in self._params]
        self._weights = self._params + [mw for mw in self._masters if mw is not None]
        self._rates = None
        self._held_state = []
        self._bind()
        self.betas, self.eps, self.state_bits = (float(betas[0]), float(betas[1])), float(eps), state_bits
        self.max_grad_norm, self.seed, self.steps = float(max_grad_norm), int(seed), 0
        self.grad_norm = torch.zeros(1, dtype=torch.float32, device=self.device)
        self._written = self._weights + [self.grad_norm]
        e = self._entries
        e["n"] = self._numels
        L = _nq.lib()
        size = max(_size(L.nf4_grad_norm_workspace_size(e.ctypes.data, len(e)), "nf4_grad_norm_workspace_size"),
                   _size(L.nf4_adamw_workspace_size(len(e)), "nf4_adamw_workspace_size"))
        self._workspace = torch.empty(max(1, size), dtype=torch.uint8, device=self.device)
        self._new_state()

    def _new_state(self):
        import torch

        # one buffer for each part of the state; a tensor's share starts at a whole block
        starts = np.concatenate(([0], np.cumsum([-(-n // MOMENT_BLOCK) * MOMENT_BLOCK for n in self._numels])))
        dt = torch.float8_e4m3fn if self.state_bits == 8 else torch.float32

        def part(dtype, per):
            flat = torch.zeros(int(starts[-1]) // per, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype,
                               device=self.device).view(dtype)
            return [flat[int(a) // per:int(a) // per + -(-n // per)] for a, n in zip(starts, self._numels)]

        state = [part(dt, 1), part(dt, 1)]
        if self.state_bits == 8:
            state += [part(torch.float32, MOMENT_BLOCK), part(torch.float32, MOMENT_BLOCK)]
        self.bind_state(*state)

    def bind_state(self, m, v, m_scale=None, v_scale=None):
        """Uses these tensors as the moments (a checkpoint's, or shares of buffers of
        the caller's): per parameter, m and v of its number of elements (E4M3
        codes, or float32), with 8-bit moments one float32 scale per 256."""
        import torch

        lists = dict(m=list(m), v=list(v))
        if self.state_bits == 8:
            if m_scale is None or v_scale is None:
                raise ValueError("8-bit moments have scales")
            lists.update(m_scale=list(m_scale), v_scale=list(v_scale))
        dt = torch.float8_e4m3fn if self.state_bits == 8 else torch.float32
        for name, ts in lists.items():
            if len(ts) != len(self._params):
                raise ValueError(f"{name}: {len(ts)} tensors for {len(self._params)} parameters")
            scale = name.endswith("scale")
            want = torch.float32 if scale else dt
            for t, n in zip(ts, self._numels):
                _check_tensors(self._params[0], t)
                if t.dtype != want or t.numel() != (-(-n // MOMENT_BLOCK) if scale else n):
                    raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} for a parameter of {n} elements")
        _check_apart(self._weights + [t for ts in lists.values() for t in ts])
        # held as well, so that their memory stays where a tensor of the list gets other data
        self._held_state = [t.detach() for ts in lists.values() for t in ts]
        for name, ts in lists.items():
            self._taken[name] = tuple(ts)
            self._given.pop(name, None)
            self._entries[name] = [t.data_ptr() for t in ts]

    def zero_grad(self, set_to_none=True):
        for p in self._params:
            if set_to_none:
                p.grad = None
            elif p.grad is not None:
                p.grad.zero_()

    def _bind(self):
        """Takes the weights' addresses, once they are what the step can update."""
        import torch

        for p, n, mw in zip(self._params, self._numels, self._masters):
            if p.dtype != self.dtype:
                raise TypeError(f"parameters of one dtype, got {self.dtype} and {p.dtype}")
            _check_tensors(self._params[0], p, mw)
            if p.numel() != n or p.device != self.device:
                raise ValueError("a parameter's size or device has changed")
            if mw is not None and (mw.dtype != torch.float32 or self.dtype != torch.bfloat16 or mw.numel() != n):
                raise TypeError("a master weight is float32, of a bfloat16 parameter of its size")
        if self._held_state:  # at construction bind_state asks this
            _check_apart(self._weights + self._held_state)
        self._entries["w"] = [p.data_ptr() for p in self._params]
        self._entries["master"] = [0 if mw is None else mw.data_ptr() for mw in self._masters]
        # held, so that no other memory can have their addresses
        self._held = [t.detach() for t in self._weights]
        self._bound = [t.data_ptr() for t in self._held]

    def _check_given(self):
        for name, ts in self._given.items():
            taken = self._taken[name]
            if len(ts) != len(taken) or any(map(operator.is_not, ts, taken)):
                raise ValueError(f"{name} has other tensors than the step writes: bind_state gives it other moments, a "
                                 "parameter's data another weight")

    def step(self, grads=None, step=None, seed=None):
        """One step with the parameters' ``.grad``, or with ``grads`` (a tensor for
        each parameter, all bfloat16 or all float32). ``step`` and ``seed``
        override the step number (the count of calls) and the random seed."""
        L = _nq.lib()
        if self._given:
            self._check_given()
        grads = [p.grad for p in self._params] if grads is None else grads
        if len(grads) != len(self._params):
            raise ValueError(f"{len(grads)} gradients for {len(self._params)} parameters")
        T = self._tensor  # the methods over the list: a third less time than a loop, for hundreds of tensors
        try:
            devices, sizes = set(map(T.get_device, grads)), list(map(T.numel, grads))
        except TypeError:
            raise ValueError("a parameter has no gradient") from None
        dt = grads[0].dtype
        if (devices != {self._params[0].get_device()} or sizes != self._numels or not all(map(T.is_contiguous, grads))
                or {g.dtype for g in grads} != {dt}):
            raise ValueError(f"gradients: contiguous, of the parameters' sizes, one dtype, on {self.device}; got "
                             + ", ".join(f"{tuple(g.shape)} {g.dtype} {g.device}" for g in grads[:4]) + " ...")
        if list(map(T.data_ptr, self._weights)) != self._bound or not all(map(T.is_contiguous, self._weights)):
            self._bind()  # a weight has new memory, or lies in another order, which this refuses
        grad_dtype = _code(dt)
        e = self._entries
        e["grad"] = array.array("Q", map(T.data_ptr, grads))
        rates = [(g["lr"], g["weight_decay"]) for g in self.groups]
        if rates != self._rates:
            for g in self.groups:
                part = slice(g["first"], g["first"] + g["count"])
                e["lr"][part], e["weight_decay"][part] = g["lr"], g["weight_decay"]
            self._rates = rates
        number = self.steps + 1 if step is None else int(step)
        stream = _stream(devices.pop())
        config = nf4_adamw_config(*self.betas, self.eps, self.max_grad_norm, number,
                                  (self.seed + number if seed is None else int(seed)) & 0xFFFFFFFFFFFFFFFF)
        call, norm = ((L.nf4_adamw_clip_step, self.grad_norm.data_ptr()) if self.max_grad_norm > 0
                      else (L.nf4_adamw_step, None))
        _nq._check(call(self._at, len(grads), _code(self.dtype), grad_dtype, self.state_bits, ctypes.byref(config), norm,
                        self._workspace.data_ptr(), self._workspace.numel(), stream), call.__name__)
        _changed(self._written)
        self.steps = number

    def __reduce_ex__(self, protocol):
        raise TypeError("an NF4AdamW holds its tensors' addresses and is not copied: state_dict carries its state")

    def state_dict(self):
        d = dict(steps=self.steps, seed=self.seed, state_bits=self.state_bits,
                 groups=[dict(lr=g["lr"], weight_decay=g["weight_decay"]) for g in self.groups],
                 m=[t.clone() for t in self._taken["m"]], v=[t.clone() for t in self._taken["v"]],
                 masters=[None if t is None else t.clone() for t in self._masters])
        if self.state_bits == 8:
            d.update(m_scale=[t.clone() for t in self._taken["m_scale"]],
                     v_scale=[t.clone() for t in self._taken["v_scale"]])
        return d

    def load_state_dict(self, d):
        import torch

        names = ["m", "v"] + (["m_scale", "v_scale"] if self.state_bits == 8 else [])
        if (d["state_bits"] != self.state_bits or len(d["groups"]) != len(self.groups)
                or any(len(d[k]) != len(self._params) for k in names + ["masters"])):
            raise ValueError("the state of another optimizer")
        pairs = [(x, y) for k in names for x, y in zip(self._taken[k], d[k])]
        for x, y in zip(self._masters, d["masters"]):
            if (x is None) != (y is None):
                raise ValueError("the state of another optimizer: master weights")
            pairs += [] if x is None else [(x, y)]
        for x, y in pairs:
            if x.dtype != y.dtype or x.numel() != y.numel():
                raise ValueError("the state of another optimizer: sizes")
        for x, y in pairs:
            x.reshape(-1).view(torch.uint8).copy_(y.reshape(-1).to(x.device).view(torch.uint8))
        self.steps, self.seed = int(d["steps"]), int(d["seed"])
        for g, new in zip(self.groups, d["groups"]):
            g.update(lr=float(new["lr"]), weight_decay=float(new["weight_decay"]))


# ------------------------------------------------------------------ residual norms

def _norm_shape(y, h, w_pre, w_post, gate, alpha, eps, w_offset):
    """The call's shape: y None leaves only the norm of h."""
    act = h if y is None else y
    shape = h.shape
    if not shape or act.shape != shape:
        raise ValueError(f"y {tuple(act.shape)} and h {tuple(shape)} have one shape")
    dim, wt = shape[-1], w_pre.dtype
    kind = 0
    if gate is not None and y is not None:
        kind = GATE_KINDS["token" if len(shape) > 1 and gate.shape == shape else "channel"]
        if kind == 1 and gate.shape != (dim,):
            raise ValueError(f"gate {tuple(gate.shape)}: ({dim},) or the shape of y")
        if gate.dtype != (act.dtype if kind == 2 else wt):
            raise TypeError("a token gate has the dtype of y, a channel gate that of the norms' weights")
    if w_pre.shape != (dim,) or (w_post is not None and (w_post.shape != (dim,) or w_post.dtype != wt)):
        raise ValueError(f"norm weights are ({dim},) of one dtype")
    return nf4_residual_norm_shape(h.numel() // max(dim, 1), dim, _code(act.dtype), _code(h.dtype), _code(wt), kind, eps,
                                   alpha, w_offset)


def residual_norm_forward(y, h, w_pre, w_post=None, gate=None, alpha=1.0, eps=1e-6, w_offset=0.0, h_out=None, x_out=None):
    """h' = h + alpha gate norm(y; w_post), x = norm(h'; w_pre) over the last
    dimension (nf4_residual_norm_forward). ``y`` bfloat16 or float32, ``h`` the
    same or float32; without ``w_post`` y is added as it is; ``y=None``: x =
    norm(h) and h' = h, which no other ``h_out`` receives. ``gate``: one value a
    channel, or one an element. Returns (h', x, rstd_pre, rstd_post or None);
    ``h_out=h`` updates the residual stream in place."""
    import torch

    index = _check_tensors(h, y, w_pre, w_post, gate, h_out, x_out)
    shape = _norm_shape(y, h, w_pre, w_post, gate, alpha, eps, w_offset)
    act = h if y is None else y
    if y is None and h_out is not None and h_out.data_ptr() != h.data_ptr():
        raise ValueError("h_out without y: h' is h, and nothing is written")
    given = [t for t in (None if y is None else h_out, x_out) if t is not None]
    for t, like in ((h_out, h), (x_out, act)):
        if t is not None and (t.shape != like.shape or t.dtype != like.dtype):
            raise ValueError("outputs have the shape and dtype of h and y")
    if h_out is None and y is not None:
        h_out = torch.empty_like(h)
    if x_out is None:
        x_out = torch.empty_like(act)
    rows = shape.rows
    rstd_pre = torch.empty(rows, dtype=torch.float32, device=h.device)
    rstd_post = torch.empty_like(rstd_pre) if w_post is not None and y is not None else None
    st = _nq.lib().nf4_residual_norm_forward(ctypes.byref(shape), _addr(y), h.data_ptr(), _addr(w_post), _addr(gate),
                                             w_pre.data_ptr(), _addr(h_out), x_out.data_ptr(), _addr(rstd_post),
                                             rstd_pre.data_ptr(), _stream(index))
    _nq._check(st, "nf4_residual_norm_forward")
    if given:
        _changed(given)
    return (h if y is None else h_out), x_out, rstd_pre, rstd_post


def residual_norm_backward(dx, dh_out, y, h_out, rstd_pre, w_pre, rstd_post=None, w_post=None, gate=None, alpha=1.0,
                           w_offset=0.0, want=(True, True, True, True, True)):
    """Gradients of residual_norm_forward from those of x and h' (either may be
    None) and the forward's h' and statistics: (dy, dh, dw_pre, dw_post, dgate),
    None where ``want`` is false or the input is absent."""
    import torch

    index = _check_tensors(h_out, dx, dh_out, y, rstd_pre, w_pre, rstd_post, w_post, gate)
    shape = _norm_shape(y, h_out, w_pre, w_post, gate, alpha, 0.0, w_offset)
    act = h_out if y is None else y
    for t, like in ((dx, act), (dh_out, h_out)):
        if t is not None and (t.shape != like.shape or t.dtype != like.dtype):
            raise ValueError("dx has the shape and dtype of y, dh_out those of h")
    post, kind, rows = w_post is not None and y is not None, shape.gate_kind, shape.rows
    for r, need in ((rstd_pre, True), (rstd_post, post)):
        if need and (r is None or r.dtype != torch.float32 or r.numel() != rows):
            raise ValueError("rstd_pre and, with w_post, rstd_post hold one float32 a row")
    dy = torch.empty_like(y) if want[0] and y is not None else None
    dh = torch.empty_like(h_out) if want[1] else None
    dw_pre = torch.empty_like(w_pre) if want[2] else None
    dw_post = torch.empty_like(w_post) if want[3] and post else None
    dgate = torch.empty_like(gate) if want[4] and kind else None
    L, shape_p = _nq.lib(), ctypes.byref(shape)
    ws, size = None, 0
    if shape.dim > 8192 or dw_pre is not None or dw_post is not None or (dgate is not None and kind == 1):
        size = max(_size(L.nf4_residual_norm_backward_workspace_size(shape_p),
                         "nf4_residual_norm_backward_workspace_size"), 1)
        ws = torch.empty(size, dtype=torch.uint8, device=h_out.device)
    st = L.nf4_residual_norm_backward(shape_p, _addr(dx), _addr(dh_out), _addr(y), h_out.data_ptr(), _addr(w_post),
                                      _addr(gate), w_pre.data_ptr(), _addr(rstd_post), rstd_pre.data_ptr(), _addr(dy),
                                      _addr(dh), _addr(dgate), _addr(dw_pre), _addr(dw_post), _addr(ws), size,
                                      _stream(index))
    _nq._check(st, "nf4_residual_norm_backward")
    return dy, dh, dw_pre, dw_post, dgate


# ------------------------------------------------------------------ token embedding

def _index_code(ids):
    import torch

    if ids.dtype == torch.int64:
        return 1
    if ids.dtype == torch.int32:
        return 0
    raise TypeError(f"token numbers are int32 or int64, got {ids.dtype}")


def embedding_forward(ids, table, scale=1.0, out_dtype=None, out=None):
    """scale * table[ids] (nf4_embedding_forward): ``table`` a [vocab x dim] tensor,
    or an NF4Tensor of that shape whose rows are dequantized as they are read.
    Ids outside the table give rows of zeros. The output has ``out_dtype``, by
    default the table's (bfloat16 for an NF4 table)."""
    import torch

    packed = isinstance(table, _nq.NF4Tensor)
    if len(table.shape) != 2:
        raise ValueError("a table is 2-D [vocab x dim]")
    if ids.get_device() < 0:
        raise ValueError("tensors must be contiguous device tensors")
    vocab, dim = table.shape
    given = out is not None
    if not given:
        out_dtype = out_dtype or (torch.bfloat16 if packed else table.dtype)
        out = torch.empty((*ids.shape, dim), dtype=out_dtype, device=ids.device)
    elif out.shape != (*ids.shape, dim) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError(f"out: {(*ids.shape, dim)} is wanted")
    L, code, count, od = _nq.lib(), _index_code(ids), ids.numel(), _code(out.dtype)
    if packed:
        stream = _stream(_check_tensors(ids, out, table.codes, table.absmax, table.absmax_q, table.absmax_scale))
        try:
            w = table.weight_struct()
        except ValueError:  # the table is 2-D, so its format is another one
            raise ValueError("the embedding takes NF4 tables in the default storage format "
                             "(B1 = 64, B2 = 256, E4M3, no mean offset)") from None
        st = L.nf4_embedding_forward_packed(ids.data_ptr(), code, count, ctypes.byref(w), scale, out.data_ptr(), od, stream)
    else:
        stream = _stream(_check_tensors(ids, out, table))
        st = L.nf4_embedding_forward(ids.data_ptr(), code, count, table.data_ptr(), _code(table.dtype), vocab, dim, scale,
                                     out.data_ptr(), od, stream)
    _nq._check(st, "nf4_embedding_forward")
    if given:
        _changed(out)
    return out


def embedding_backward(ids, dy, vocab, scale=1.0, padding_id=None, grad=None, grad_dtype=None, workspace=None):
    """Gradient of a [vocab x dim] table from dy [*ids.shape x dim]
    (nf4_embedding_backward): a new tensor of ``grad_dtype`` (by default dy's), or
    added to ``grad`` where one is given. Deterministic."""
    import torch

    dim = dy.shape[-1]
    if dy.get_device() < 0:
        raise ValueError("tensors must be contiguous device tensors")
    if dy.shape != (*ids.shape, dim):
        raise ValueError(f"dy {tuple(dy.shape)} for ids {tuple(ids.shape)}")
    accumulate = grad is not None
    if not accumulate:
        grad = torch.empty((vocab, dim), dtype=grad_dtype or dy.dtype, device=dy.device)
    elif tuple(grad.shape) != (vocab, dim) or (grad_dtype is not None and grad.dtype != grad_dtype):
        raise ValueError(f"grad {tuple(grad.shape)} {grad.dtype}: ({vocab}, {dim}) is wanted")
    index = _check_tensors(dy, ids, grad, workspace)
    L, count, code = _nq.lib(), ids.numel(), _index_code(ids)
    if workspace is None:
        size = max(_size(L.nf4_embedding_backward_workspace_size(count, vocab, dim),
                         "nf4_embedding_backward_workspace_size"), 1)
        workspace = torch.empty(size, dtype=torch.uint8, device=dy.device)
    else:
        size = workspace.numel() * workspace.element_size()
    st = L.nf4_embedding_backward(ids.data_ptr(), code, count, dy.data_ptr(), _code(dy.dtype), vocab, dim, scale,
                                  -1 if padding_id is None else int(padding_id), grad.data_ptr(), _code(grad.dtype),
                                  1 if accumulate else 0, workspace.data_ptr(), size, _stream(index))
    _nq._check(st, "nf4_embedding_backward")
    if accumulate:
        _changed(grad)
    return grad


# ------------------------------------------------------------------ autograd

_FUNCTIONS = None


def _functions():
    """The autograd functions (made on first use: importing this module does not
    import torch)."""
    global _FUNCTIONS
    if _FUNCTIONS is not None:
        return _FUNCTIONS
    import torch
    from torch.autograd.function import once_differentiable

    class ResidualNormFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, y, h, w_pre, w_post, gate, alpha, eps, w_offset):
            y = None if y is None else y.contiguous()
            h = h.contiguous()
            gate = None if gate is None else gate.contiguous()
            h_out, x, rstd_pre, rstd_post = residual_norm_forward(y, h, w_pre, w_post, gate, alpha, eps, w_offset)
            ctx.save_for_backward(y, h_out, rstd_pre, w_pre, rstd_post, w_post, gate)
            ctx.alpha, ctx.w_offset = alpha, w_offset
            ctx.set_materialize_grads(False)
            return (h_out if y is not None else h.view_as(h)), x

        @staticmethod
        @once_differentiable
        def backward(ctx, dh_out, dx):
            y, h_out, rstd_pre, w_pre, rstd_post, w_post, gate = ctx.saved_tensors
            act = h_out if y is None else y
            dx = None if dx is None else dx.to(act.dtype).contiguous()
            dh_out = None if dh_out is None else dh_out.to(h_out.dtype).contiguous()
            need = ctx.needs_input_grad
            dy, dh, dw_pre, dw_post, dgate = residual_norm_backward(
                dx, dh_out, y, h_out, rstd_pre, w_pre, rstd_post, w_post, gate, ctx.alpha, ctx.w_offset,
                want=(need[0], need[1], need[2], need[3], need[4]))
            return dy, dh, dw_pre, dw_post, dgate, None, None, None

    class EmbeddingFunction(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ids, table, scale, padding_id, out_dtype):
            ids = ids.contiguous()
            ctx.save_for_backward(ids)
            ctx.scale, ctx.padding_id, ctx.vocab, ctx.dtype = scale, padding_id, table.shape[0], table.dtype
            return embedding_forward(ids, table.contiguous(), scale, out_dtype)

        @staticmethod
        @once_differentiable
        def backward(ctx, dy):
            grad = embedding_backward(ctx.saved_tensors[0], dy.contiguous(), ctx.vocab, ctx.scale, ctx.padding_id,
                                      grad_dtype=ctx.dtype)
            return None, grad, None, None, None

    _FUNCTIONS = (ResidualNormFunction, EmbeddingFunction)
    return _FUNCTIONS


def residual_norm(y, h, w_pre, w_post=None, gate=None, alpha=1.0, eps=1e-6, w_offset=0.0):
    """Differentiable residual step: (h', x) of residual_norm_forward. Gradients
    flow to y, h, both norms' weights and the gate."""
    return _functions()[0].apply(y, h, w_pre, w_post, gate, float(alpha), float(eps), float(w_offset))


def nf4_embedding(ids, table, scale=1.0, padding_id=None, out_dtype=None):
    """Differentiable scale * table[ids]. A dense table receives a dense gradient
    (none for ``padding_id``); an NF4Tensor is frozen."""
    if isinstance(table, _nq.NF4Tensor):
        return embedding_forward(ids.contiguous(), table, scale, out_dtype)
    return _functions()[1].apply(ids, table, float(scale), padding_id, out_dtype)
