"""Operators around an expert layer (include/bmoe_adamw.h, bmoe_block.h,
bmoe_ffn.h): argument marshalling only, as in the package's other calls."""
from __future__ import annotations

import contextlib
import ctypes
import functools

import numpy as np

from . import BF16, F32, _check, _on_device, _operand, _raw_stream, _torch, _workspace_bytes, lib

# bmoe_adamw_tensor of include/bmoe_adamw.h
_ADAMW_TENSOR = np.dtype([
    ("param", np.uint64), ("grad", np.uint64), ("m", np.uint64), ("v", np.uint64), ("m_exp", np.uint64), ("v_exp", np.uint64),
    ("copy", np.uint64), ("n", np.int64), ("lr_scale", np.float32), ("weight_decay", np.float32), ("grad_dtype", np.int32),
    ("bits", np.int32)])


class _AdamWArgs(ctypes.Structure):
    """bmoe_adamw_args of include/bmoe_adamw.h."""
    _fields_ = [
        ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
        ("step", ctypes.c_int64), ("step_device", ctypes.c_void_p), ("lr_device", ctypes.c_void_p),
        ("grad_scale", ctypes.c_void_p), ("seed", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


def _listed(name, what, count, default=None):
    """`what` as a list of `count`: a number (or None) is everybody's."""
    if what is None:
        return [default] * count
    if isinstance(what, (list, tuple)):
        if len(what) != count:
            raise ValueError(f"{name} has {len(what)} entries for {count} parameters")
        return list(what)
    return [what] * count


def _tensor(name, t, kind, shape, device):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is {t!r}, expected a tensor")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected a GPU tensor on {device}")
    if t.dtype != kind:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {kind}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_HERE = contextlib.nullcontext()


def _device(index: int):
    """The GPU `index` as the current one (2 us less where it is)."""
    torch = _torch()
    return _HERE if index == torch._C._cuda_getDevice() else torch.cuda.device(index)


class AdamW:
    """AdamW over a list of fp32 tensors on one GPU, all of them in one launch for
    every 40 (bmoe_adamw_step): what `Layer.backward` gives gradients for besides the
    latent substrates (angles, gate matrix), norm weights, dense projections.

        opt = bmoe.AdamW([layer.theta[0], layer.phi[0], gamma], lr=1e-3, weight_decay=[0.0, 0.0, 0.0])
        opt.step([grads["theta"][0], grads["phi"][0], dgamma])

    params           the tensors, updated in place by every step (autograd is told: a graph
                     that saved one for its backward before refuses to run it).
    weight_decay, lr_scale, bits, copies   one for all tensors or a list of them: the
                     decoupled decay, a factor on lr, 32 or 8 bits for the moments (8:
                     bmoe_adamw.h's codes), a bf16 tensor that gets the new values.
    lr               a number, which may be set anew between steps (`opt.lr`; a captured
                     step keeps its own), or a one-element fp32 tensor that every step
                     reads on the GPU.
    m, v             the moments to go on from (fp32; with 8 bits uint8 codes and their
                     blocks' exponents m_exp, v_exp [ceil(n / 256)] uint8), used as they
                     are and updated in place; None: zeros.  `opt.m`, `opt.v` and so on
                     list the tensors in use, whose values may be set.  (Parameters and
                     copies may get other memory between steps, the moments not.)
    steps            the steps already taken.
    capturable       count the steps on the GPU, so that a step captured in a graph
                     counts on in every replay; without, a step in a capture is refused.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay=0.01, *, lr_scale=1.0, bits=32,
                 copies=None, seed: int = 0, m=None, v=None, m_exp=None, v_exp=None, steps: int = 0, capturable: bool = False):
        torch = _torch()
        self.params = list(params)
        if not self.params:
            raise ValueError("AdamW needs at least one parameter")
        if not isinstance(self.params[0], torch.Tensor) or not self.params[0].is_cuda:
            raise ValueError("AdamW needs GPU tensors")
        count, dev = len(self.params), self.params[0].device
        self.device, self.lr, self.betas, self.eps, self.seed = dev, lr, tuple(betas), float(eps), int(seed)
        if len(self.betas) != 2:
            raise ValueError("betas are two numbers")
        if not 0 <= self.seed < 1 << 32:
            raise ValueError("seed must fit 32 bits")
        if steps < 0:
            raise ValueError("steps must not be negative")
        f32, u8 = torch.float32, torch.uint8
        self.bits = _listed("bits", bits, count)
        self._decay, self._scale = _listed("weight_decay", weight_decay, count, 0.0), _listed("lr_scale", lr_scale, count, 1.0)
        self.copies = _listed("copies", [copies] if isinstance(copies, torch.Tensor) else copies, count)
        given = [_listed(n, [x] if isinstance(x, torch.Tensor) else x, count) for n, x in
                 (("m", m), ("v", v), ("m_exp", m_exp), ("v_exp", v_exp))]
        self.m, self.v, self.m_exp, self.v_exp = [], [], [], []
        for i, p in enumerate(self.params):
            _tensor(f"params[{i}]", p, f32, p.shape, dev)
            if self.copies[i] is not None:
                _tensor(f"copies[{i}]", self.copies[i], torch.bfloat16, p.shape, dev)
            if self.bits[i] not in (32, 8):
                raise ValueError(f"bits[{i}] is {self.bits[i]}, expected 32 or 8")
            eight = self.bits[i] == 8
            blocks = torch.Size([(p.numel() + 255) // 256])
            for name, have, out, kind, shape, wanted in (
                    ("m", given[0], self.m, u8 if eight else f32, p.shape, True), ("v", given[1], self.v, u8 if eight else f32, p.shape, True),
                    ("m_exp", given[2], self.m_exp, u8, blocks, eight), ("v_exp", given[3], self.v_exp, u8, blocks, eight)):
                x = have[i]
                if not wanted:
                    if x is not None:
                        raise ValueError(f"{name}[{i}] is for moments in 8 bits")
                    out.append(None)
                elif x is None:
                    out.append(torch.zeros(shape, dtype=kind, device=dev))
                else:
                    out.append(_tensor(f"{name}[{i}]", x, kind, shape, dev).detach())   # this memory, whatever x is given later
            if len({x[i] is None for x in (given if eight else given[:2])}) > 1:
                raise ValueError(f"{'m, v, m_exp and v_exp' if eight else 'm and v'} of parameter {i} go together")
        # what its owner may give other memory or another layout (`tensor.data = ..`, a module's `.to`)
        self._owned = [(f"{name}[{i}]", x, x.dtype, x.shape) for name, tensors in (("params", self.params), ("copies", self.copies))
                       for i, x in enumerate(tensors) if x is not None]
        self._owned_tensors, self._owned_kinds, self._owned_shapes = ([o[k] for o in self._owned] for k in (1, 2, 3))
        t = np.zeros(count, dtype=_ADAMW_TENSOR)
        self._table = t
        for name, tensors in (("m", self.m), ("v", self.v), ("m_exp", self.m_exp), ("v_exp", self.v_exp)):
            t[name] = [0 if x is None else x.data_ptr() for x in tensors]
        self._take_addresses()
        t["n"] = [p.numel() for p in self.params]
        t["lr_scale"], t["weight_decay"], t["bits"] = self._scale, self._decay, self.bits
        self._table_at = t.ctypes.data
        self._grad, self._grad_dtype = t["grad"], t["grad_dtype"]   # views of it
        self._shapes = [p.shape for p in self.params]
        self._coded = [i for i, b in enumerate(self.bits) if b == 8]
        self._coded_shapes = [self._shapes[i] for i in self._coded]
        self._steps = int(steps)
        self._counter = torch.full((1,), self._steps, dtype=torch.int64, device=dev) if capturable else None

    def _take_addresses(self):
        for name, tensors in (("param", self.params), ("copy", self.copies)):
            self._table[name] = [0 if x is None else x.data_ptr() for x in tensors]
        self._addresses = [x.data_ptr() for x in self._owned_tensors]

    @property
    def steps(self) -> int:
        """The steps taken (capturable: read from the GPU, which waits for it)."""
        return self._steps if self._counter is None else int(self._counter.item())

    def _fit(self, tensors, shapes):
        """The types of tensors that all are of these shapes, dense and on this GPU (a tenth of
        a microsecond for each, where checks that name what is wrong take one); None where
        one is not, or is of a class of its own."""
        torch = _torch()
        t = torch.Tensor
        if (set(map(type, tensors)) <= {t, torch.nn.Parameter} and set(map(t.get_device, tensors)) == {self.device.index} and
                list(map(t.size, tensors)) == shapes and all(map(t.is_contiguous, tensors))):
            return set(map(t.dtype.__get__, tensors))
        return None

    def step(self, grads, grad_scale=None) -> None:
        """One step: grads a list like params (fp32 or bf16; None: that tensor is left
        as it is), grad_scale a one-element fp32 tensor that multiplies all of them
        (what clips them, or takes a loss's scale out again)."""
        torch = _torch()
        f32, bf16, table, dev = torch.float32, torch.bfloat16, self._table, self.device
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        index = dev.index
        t, own = torch.Tensor, self._owned_tensors
        # (0.1 us a tensor for sizes, types and layouts beside the addresses: 45 -> 58 us at 120)
        if (list(map(t.data_ptr, own)) != self._addresses or list(map(t.size, own)) != self._owned_shapes or
                list(map(t.dtype.__get__, own)) != self._owned_kinds or not all(map(t.is_contiguous, own))):
            for name, x, kind, shape in self._owned:   # taken where they are now
                _tensor(name, x, kind, shape, dev)
            self._take_addresses()
        kinds = self._fit(grads, self._shapes)
        if kinds is None or not kinds <= {f32, bf16}:
            for i, (g, s) in enumerate(zip(grads, self._shapes)):
                if g is not None:
                    _tensor(f"grads[{i}]", g, bf16 if getattr(g, "dtype", None) == bf16 else f32, s, dev)
            kinds = None
        if kinds is None or len(kinds) > 1:
            self._grad[:] = [0 if g is None else g.data_ptr() for g in grads]
            self._grad_dtype[:] = [F32 if g is None or g.dtype is f32 else BF16 for g in grads]
        else:
            self._grad[:] = list(map(torch.Tensor.data_ptr, grads))
            self._grad_dtype[:] = F32 if f32 in kinds else BF16
        a = _AdamWArgs()
        a.beta1, a.beta2 = self.betas
        a.eps, a.seed = self.eps, self.seed
        if isinstance(self.lr, torch.Tensor):
            a.lr_device = _tensor("lr", self.lr.reshape(-1), f32, torch.Size([1]), dev).data_ptr()
        else:
            a.lr = float(self.lr)
        if grad_scale is not None:
            a.grad_scale = _tensor("grad_scale", grad_scale.reshape(-1), f32, torch.Size([1]), dev).data_ptr()
        with _device(index):
            if self._counter is not None:
                a.step_device = self._counter.data_ptr()
            elif torch.cuda.is_current_stream_capturing():
                raise ValueError("a captured step counts on the GPU: AdamW(capturable=True)")
            else:
                a.step = self._steps + 1
            _check(lib().bmoe_adamw_step(self._table_at, len(table), ctypes.byref(a), _raw_stream(self.params[0])))
        self._steps += 1
        # autograd's count of changes, as torch's own updates in place raise it
        torch.autograd.graph.increment_version(own if kinds is not None else [
            x for tensors in (self.params, self.copies) for x, g in zip(tensors, grads) if x is not None and g is not None])

    def moments(self, m_out=None, v_out=None):
        """The moments' values as two lists: the fp32 tensors themselves, and for codes of
        8 bits those of m_out and v_out (lists of tensors, None for a new one; not for
        moments of 32 bits) or new ones.  All of one type: that of the first given, fp32
        without any, or bf16, which holds the values exactly too (from 2^-130 on; smaller
        ones to the nearest of its numbers)."""
        torch = _torch()
        coded, kind, bf16 = self._coded, torch.float32, torch.bfloat16
        index, count = self.device.index, len(self.params)
        for name, outs in (("m_out", m_out), ("v_out", v_out)):
            if outs is not None and len(outs) != count:
                raise ValueError(f"{name} has {len(outs)} entries for {count} parameters")
        first = next((o[i] for o in (m_out, v_out) if o is not None for i in coded if o[i] is not None), None)
        if getattr(first, "dtype", None) == bf16:
            kind = bf16
        whole = len(coded) == count
        ms, vs = list(self.m), list(self.v)
        pointers = []
        for name, outs, out in (("m_out", m_out, ms), ("v_out", v_out, vs)):
            if outs is None:
                outs = [None] * count
            elif not whole and any(x is not None and b != 8 for x, b in zip(outs, self.bits)):
                raise ValueError(f"{name} is for moments in 8 bits: None elsewhere")
            given = list(outs) if whole else [outs[i] for i in coded]
            if self._fit(given, self._coded_shapes) != {kind}:
                for k, (i, x) in enumerate(zip(coded, given)):
                    given[k] = (torch.empty(self._shapes[i], dtype=kind, device=self.device) if x is None else
                                _tensor(f"{name}[{i}]", x, kind, self._shapes[i], self.device))
            if whole:
                out[:] = given
            else:
                for i, x in zip(coded, given):
                    out[i] = x
            pointers.append(np.array(list(map(torch.Tensor.data_ptr, given)), dtype=np.uint64))
        if coded:
            table = self._table if whole else self._table[coded]
            with _device(index):
                _check(lib().bmoe_adamw_moments(table.ctypes.data, len(table), BF16 if kind == torch.bfloat16 else F32,
                                                pointers[0].ctypes.data, pointers[1].ctypes.data, _raw_stream(self.params[0])))
        return ms, vs


class _BlockNorm(ctypes.Structure):
    """bmoe_block_norm of include/bmoe_block.h."""
    _fields_ = [
        ("rows", ctypes.c_int32), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32), ("kind", ctypes.c_int32),
        ("post", ctypes.c_int32), ("gate_kind", ctypes.c_int32), ("alpha", ctypes.c_float), ("scale", ctypes.c_float),
        ("eps", ctypes.c_float), ("reserved", ctypes.c_int32), ("gate", ctypes.c_void_p), ("gamma_post", ctypes.c_void_p),
        ("beta_post", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p)]


class _BlockNormGrads(ctypes.Structure):
    """bmoe_block_norm_grads of include/bmoe_block.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("gamma_post", "beta_post", "gate", "gamma", "beta")]


_NORM_KINDS = {"layer": 0, "rms": 1}


def _block_norm(b, gate, alpha, scale, post, kind, gamma_post, beta_post, gamma, beta, eps):
    """Check the weights and describe the call."""
    torch = _torch()
    dev, f32 = b.device, (torch.float32,)
    rows, width = b.shape
    _operand("b", b, b.shape, (torch.float32, torch.bfloat16), dev)
    if kind not in _NORM_KINDS:
        raise ValueError(f"kind is {kind!r}, expected 'layer' or 'rms'")
    n = _BlockNorm()
    n.rows, n.width, n.dtype, n.kind, n.post = rows, width, BF16 if b.dtype is torch.bfloat16 else F32, _NORM_KINDS[kind], 1 if post else 0
    n.alpha, n.scale, n.eps = alpha, scale, eps
    if gate is not None:
        if gate.dim() == 1:
            n.gate_kind = 1
            _operand("gate", gate, (width,), f32, dev)
        else:
            n.gate_kind = 2
            _operand("gate", gate, b.shape, (b.dtype,), dev)
        n.gate = gate.data_ptr()
    if gamma_post is not None:
        n.gamma_post = _operand("gamma_post", gamma_post, (width,), f32, dev).data_ptr()
    if beta_post is not None:
        n.beta_post = _operand("beta_post", beta_post, (width,), f32, dev).data_ptr()
    if gamma is not None:
        n.gamma = _operand("gamma", gamma, (width,), f32, dev).data_ptr()
    if beta is not None:
        n.beta = _operand("beta", beta, (width,), f32, dev).data_ptr()
    return n


@_on_device
def block_norm_forward(b, residual=None, gate=None, alpha: float = 1.0, scale: float = 1.0, post: bool = True, kind: str = "layer",
                       gamma_post=None, beta_post=None, gamma=None, beta=None, eps: float = 1e-5, stats: bool = True, s_out=None,
                       y=None):
    """From a block's output b [rows][width] (fp32 or bf16) to the next block's input:
        z = norm(b) gamma_post + beta_post   (z = b with post=False)
        s = alpha residual + scale gate z,   y = norm(s) gamma + beta
    with layer norms or (kind="rms", without betas) RMS norms.  gate: None, [width] fp32
    or [rows][width] like b; gammas and betas [width] fp32 or None (ones, zeros).  Returns
    (y, s, stats): stats [rows][4] fp32 for the backward (None with stats=False).  s_out may be
    residual itself, and y either input that is not needed any more."""
    torch = _torch()
    n = _block_norm(b, gate, alpha, scale, post, kind, gamma_post, beta_post, gamma, beta, eps)
    dev, shape, own = b.device, b.shape, (b.dtype,)
    if residual is not None:
        _operand("residual", residual, shape, own, dev)
    s_out = torch.empty_like(b) if s_out is None else _operand("s_out", s_out, shape, own, dev)
    y = torch.empty_like(b) if y is None else _operand("y", y, shape, own, dev)
    st = torch.empty((shape[0], 4), dtype=torch.float32, device=dev) if stats else None
    _check(lib().bmoe_block_norm_forward(ctypes.byref(n), b.data_ptr(), None if residual is None else residual.data_ptr(),
                                         s_out.data_ptr(), y.data_ptr(), None if st is None else st.data_ptr(), _raw_stream(b)))
    return y, s_out, st


@functools.lru_cache(maxsize=4096)
def _block_norm_workspace(rows: int, width: int) -> int:
    """bmoe_block_norm_backward_workspace: sizes alone decide."""
    n, size = _BlockNorm(), ctypes.c_size_t(0)
    n.rows, n.width = rows, width
    _check(lib().bmoe_block_norm_backward_workspace(ctypes.byref(n), ctypes.byref(size)))
    return int(size.value)


@_on_device
def block_norm_backward(dy, b, s, stats, gate=None, alpha: float = 1.0, scale: float = 1.0, post: bool = True, kind: str = "layer",
                        gamma_post=None, beta_post=None, gamma=None, d_sum=None, residual: bool = True, weight_grads: bool = True,
                        db=None, dr=None):
    """Backward of block_norm_forward at its s and stats: dy [rows][width] fp32 or of b's
    dtype, d_sum like b or None (gradient that reaches s past the norm in front of the next
    block).  Returns a dict of b, residual (None with residual=False), gate, gamma_post,
    beta_post, gamma and beta: the gradients, like b the first two and a gate of rows, fp32
    [width] the others, None for what the forward has no use for (betas of an RMS norm,
    post's without it, a gate that was not given; weight_grads=False: all but the first
    two).  db and dr may be b, s, d_sum or a dy of their dtype themselves."""
    torch = _torch()
    if b.dim() != 2:
        raise ValueError(f"b has shape {tuple(b.shape)}, expected two dimensions")
    dev, own = dy.device, (b.dtype,)
    if b.device != dev:
        raise ValueError(f"b is on {b.device}, expected {dev}")
    n = _block_norm(b, gate, alpha, scale, post, kind, gamma_post, beta_post, gamma, None, 0.0)
    shape = b.shape
    rows, width = shape
    _operand("dy", dy, shape, (torch.float32, b.dtype), dev)
    _operand("s", s, shape, own, dev)
    _operand("stats", stats, (rows, 4), (torch.float32,), dev)
    if d_sum is not None:
        _operand("d_sum", d_sum, shape, own, dev)
    out = dict.fromkeys(("b", "residual", "gate", "gamma_post", "beta_post", "gamma", "beta"))
    out["b"] = torch.empty_like(b) if db is None else _operand("db", db, shape, own, dev)
    if residual:
        out["residual"] = torch.empty_like(b) if dr is None else _operand("dr", dr, shape, own, dev)
    elif dr is not None:
        raise ValueError("dr needs residual=True")
    g, ws, nbytes = None, None, 0
    if weight_grads:
        layer = kind == "layer"
        names = ["gamma"] + (["beta"] if layer else []) + (["gamma_post"] if post else []) + (["beta_post"] if post and layer else [])
        if gate is not None and gate.dim() == 1:
            names.append("gate")
        for name, x in zip(names, torch.empty((len(names), width), dtype=torch.float32, device=dev).unbind(0)):
            out[name] = x
        if gate is not None and gate.dim() == 2:
            out["gate"] = torch.empty_like(b)
        g = _BlockNormGrads(*[None if out[k] is None else out[k].data_ptr() for k in ("gamma_post", "beta_post", "gate", "gamma", "beta")])
        nbytes = _block_norm_workspace(rows, width)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib().bmoe_block_norm_backward(
        ctypes.byref(n), BF16 if dy.dtype is torch.bfloat16 else F32, dy.data_ptr(), b.data_ptr(), s.data_ptr(), stats.data_ptr(),
        None if d_sum is None else d_sum.data_ptr(), out["b"].data_ptr(), None if out["residual"] is None else out["residual"].data_ptr(),
        None if g is None else ctypes.byref(g), None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dy)))
    return out


_GATED_ACTS = {"silu": 0, "gelu": 1}


def _ffn(x, w_in, w_down, act):
    """Check what all three calls have: (tokens, d, ff, act's number, bf16)."""
    torch = _torch()
    bf16, dev = (torch.bfloat16,), x.device
    tokens, d = x.shape
    _operand("x", x, x.shape, bf16, dev)
    if w_down.dim() != 2:
        raise ValueError(f"w_down has shape {tuple(w_down.shape)}, expected two dimensions")
    ff = w_down.shape[1]
    _operand("w_down", w_down, (d, ff), bf16, dev)
    _operand("w_in", w_in, (2 * ff, d), bf16, dev)
    if act not in _GATED_ACTS:
        raise ValueError(f"act is {act!r}, expected 'silu' or 'gelu'")
    return tokens, d, ff, _GATED_ACTS[act], bf16


def _ffn_forward(x, w_in, w_down, act, add, y, train):
    torch = _torch()
    tokens, d, ff, kind, bf16 = _ffn(x, w_in, w_down, act)
    dev = x.device
    if add is not None:
        _operand("add", add, x.shape, bf16, dev)
    y = torch.empty_like(x) if y is None else _operand("y", y, x.shape, bf16, dev)
    state = torch.empty(7 * tokens * ff, dtype=torch.uint8, device=dev) if train else None
    nbytes = _workspace_bytes("bmoe_gated_ffn_forward_workspace", tokens, d, ff, 1 if train else 0)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _check(lib().bmoe_gated_ffn_forward(tokens, d, ff, kind, x.data_ptr(), w_in.data_ptr(), w_down.data_ptr(),
                                        None if add is None else add.data_ptr(), y.data_ptr(), None if state is None else state.data_ptr(),
                                        7 * tokens * ff, None if ws is None else ws.data_ptr(), nbytes, _raw_stream(x)))
    return y, state


@_on_device
def gated_ffn_forward(x, w_in, w_down, act: str = "silu", add=None, y=None):
    """Dense gated feed-forward block on the rows of x [tokens][d]: with Wg the first and Wu
    the second half of w_in [2 ff][d],
        y = (act(x Wg^T) * (x Wu^T)) w_down^T (+ add)
    for act "silu" or "gelu" (exact).  Everything bf16, d and ff multiples of 8; w_down [d][ff].
    add [tokens][d] is added before the one rounding (a ButterflyMoE layer's output, to
    which this is the shared expert); y may be add itself."""
    return _ffn_forward(x, w_in, w_down, act, add, y, False)[0]


@_on_device
def gated_ffn_forward_train(x, w_in, w_down, act: str = "silu", add=None, y=None):
    """gated_ffn_forward and the state that gated_ffn_backward reads (an opaque device
    buffer, 7 bytes for each token and hidden unit).  Returns (y, state)."""
    return _ffn_forward(x, w_in, w_down, act, add, y, True)


@_on_device
def gated_ffn_backward(x, w_in, w_down, dy, state, act: str = "silu", dx_add=None, input_grad: bool = True, weight_grads: bool = True,
                       dx=None, dw_in=None, dw_down=None):
    """Gradients of sum(dy * y) at the state of gated_ffn_forward_train: (dx [tokens][d],
    dw_in, dw_down like the weights), bf16, None for those not wanted.  The activation is the
    one that the state was made with, whichever act names.  dx_add [tokens][d] fp32 is added
    into dx before its rounding (the input gradient of Layer.backward for the same x).  The
    gradient of the forward's add is dy."""
    torch = _torch()
    tokens, d, ff, kind, bf16 = _ffn(x, w_in, w_down, act)
    dev = x.device
    _operand("dy", dy, x.shape, bf16, dev)
    _operand("state", state, (7 * tokens * ff,), (torch.uint8,), dev)
    if dx_add is not None:
        _operand("dx_add", dx_add, x.shape, (torch.float32,), dev)
    if input_grad:
        dx = torch.empty_like(x) if dx is None else _operand("dx", dx, x.shape, bf16, dev)
    if weight_grads:
        dw_in = torch.empty_like(w_in) if dw_in is None else _operand("dw_in", dw_in, w_in.shape, bf16, dev)
        dw_down = torch.empty_like(w_down) if dw_down is None else _operand("dw_down", dw_down, w_down.shape, bf16, dev)
    if (not input_grad and dx is not None) or (not weight_grads and (dw_in is not None or dw_down is not None)):
        raise ValueError("an output is given for a gradient that is not wanted")
    nbytes = _workspace_bytes("bmoe_gated_ffn_backward_workspace", tokens, d, ff)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    at = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _check(lib().bmoe_gated_ffn_backward(tokens, d, ff, kind, x.data_ptr(), w_in.data_ptr(), w_down.data_ptr(), dy.data_ptr(), state.data_ptr(),
                                         7 * tokens * ff, at(dx_add), at(dx), at(dw_in), at(dw_down), at(ws), nbytes, _raw_stream(x)))
    return dx, dw_in, dw_down
