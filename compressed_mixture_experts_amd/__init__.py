"""ButterflyMoE expert layer on AMD MI355X (gfx950): Python binding.

The computation runs in ``libbmoe.so`` (hand-written HIP kernels behind the C
ABI of ``include/bmoe.h``, ``bmoe_trace.h``, ``bmoe_grad.h``, ``bmoe_train.h``,
``bmoe_norm.h`` and ``bmoe_update.h``).  The test
hooks of ``include/bmoe_debug.h`` live only in ``libbmoe_debug.so`` (the same
kernels, built with -DBMOE_DEBUG_EXPORTS), loaded on first use of a
``dbg_*`` function.  This module only marshals arguments: torch tensors
provide device memory and the current HIP stream.  There is no fallback path;
if a library is missing, loading it raises.  The environment variable
BMOE_LIBRARY names another build of the debug library to load for both (the
CPU ABI tests use it for the sanitized host build).

    import compressed_mixture_experts_amd as bmoe
    layer = bmoe.Layer.from_inputs(inputs, device="cuda")   # uploads + packs
    y = layer.forward(x)                                     # x: [T][d] on the GPU
"""
from __future__ import annotations

import ctypes
import functools
import inspect
import os
from typing import List, Optional, Sequence, Tuple

import numpy as np

__all__ = [
    "BmoeError", "lib", "library_path", "pack_ternary", "packed_words", "Layer",
    "dbg_butterfly", "dbg_ternary_gemm", "dbg_ternary_gemm_fp4", "butterfly_backward", "substrate_grad",
    "combine_backward", "router_backward", "gelu_backward", "substrate_input_grad",
    "layer_norm_forward", "layer_norm_backward", "orthogonalize", "substrate_step", "STATUS",
    "EXPORTED_SYMBOLS", "DEBUG_SYMBOLS", "debug_lib",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libbmoe.so")
_DEBUG_LIB_PATH = os.path.join(_PKG, "libbmoe_debug.so")

STATUS = {
    0: "BMOE_OK", 1: "BMOE_ERR_NULL", 2: "BMOE_ERR_SHAPE", 3: "BMOE_ERR_DTYPE",
    4: "BMOE_ERR_ALIGN", 5: "BMOE_ERR_ALIAS", 6: "BMOE_ERR_WORKSPACE",
    7: "BMOE_ERR_TERNARY", 8: "BMOE_ERR_HIP", 9: "BMOE_ERR_DEVICE",
}
F32, BF16 = 0, 1
NOALLOC_SCRATCH_BYTES = 64 << 20   # BMOE_NOALLOC_SCRATCH_BYTES of include/bmoe.h
ACT_NONE, ACT_GELU_ERF = 0, 1

# exports of libbmoe.so (include/bmoe.h, bmoe_trace.h, bmoe_grad.h, bmoe_train.h,
# bmoe_norm.h, bmoe_update.h)
EXPORTED_SYMBOLS = [
    "bmoe_packed_words", "bmoe_pack_ternary", "bmoe_workspace_size", "bmoe_prepared_bytes",
    "bmoe_prepare", "bmoe_route", "bmoe_forward", "bmoe_forward_noalloc", "bmoe_status_string",
    "bmoe_last_error", "bmoe_forward_kernels", "bmoe_forward_marked",
    "bmoe_butterfly_backward_workspace", "bmoe_butterfly_backward",
    "bmoe_substrate_grad_workspace", "bmoe_substrate_grad", "bmoe_combine_backward",
    "bmoe_router_backward_workspace", "bmoe_router_backward", "bmoe_gelu_backward",
    "bmoe_substrate_input_grad",
    "bmoe_train_state_size", "bmoe_forward_train_workspace", "bmoe_forward_train",
    "bmoe_layer_backward_workspace", "bmoe_layer_backward",
    "bmoe_layer_norm_forward", "bmoe_layer_norm_backward_workspace", "bmoe_layer_norm_backward",
    "bmoe_orthogonalize_workspace", "bmoe_orthogonalize",
    "bmoe_substrate_step_workspace", "bmoe_substrate_step",
]
# exported by libbmoe_debug.so only (include/bmoe_debug.h)
DEBUG_SYMBOLS = ["bmoe_dbg_butterfly", "bmoe_dbg_ternary_gemm", "bmoe_dbg_ternary_gemm_fp4"]


class BmoeError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {detail}")


class LayerGrads(ctypes.Structure):
    """bmoe_layer_grads of include/bmoe_train.h (device pointers)."""
    _fields_ = [
        ("dx", ctypes.c_void_p), ("d_w_gate", ctypes.c_void_p),
        ("d_theta", ctypes.c_void_p * 2), ("d_phi", ctypes.c_void_p * 2), ("d_w_base", ctypes.c_void_p * 2),
    ]


class LayerStruct(ctypes.Structure):
    _fields_ = [
        ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
        ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32), ("ffn_act", ctypes.c_int32),
        ("renorm_gates", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("w_gate", ctypes.c_void_p),
        ("w_base", ctypes.c_void_p * 2),
        ("theta", ctypes.c_void_p * 2),
        ("phi", ctypes.c_void_p * 2),
        ("w_scale", ctypes.c_float * 2),
        ("prepared", ctypes.c_void_p),
        ("prepared_bytes", ctypes.c_size_t),
    ]


_lib = None
_debug_lib = None


def library_path() -> str:
    return os.environ.get("BMOE_LIBRARY") or _LIB_PATH


def _load(path: str, debug: bool) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m compressed_mixture_experts_amd.build`")
    L = ctypes.CDLL(path)
    c_i32, c_sz, c_vp, c_f = ctypes.c_int32, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    pL = ctypes.POINTER(LayerStruct)
    L.bmoe_packed_words.argtypes = [c_i32, c_i32]
    L.bmoe_packed_words.restype = c_sz
    L.bmoe_pack_ternary.argtypes = [c_vp, c_i32, c_i32, c_vp, c_sz]
    L.bmoe_workspace_size.argtypes = [pL, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_prepared_bytes.argtypes = [pL]
    L.bmoe_prepared_bytes.restype = c_sz
    L.bmoe_prepare.argtypes = [pL, c_vp, c_sz, c_vp]
    L.bmoe_route.argtypes = [pL, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]
    L.bmoe_forward.argtypes = [pL, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]
    L.bmoe_forward_noalloc.argtypes = [pL, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp]
    L.bmoe_status_string.argtypes = [c_i32]
    L.bmoe_status_string.restype = ctypes.c_char_p
    L.bmoe_last_error.argtypes = []
    L.bmoe_last_error.restype = ctypes.c_char_p
    L.bmoe_forward_kernels.argtypes = [pL, ctypes.POINTER(c_i32), ctypes.c_char_p, c_sz]
    L.bmoe_forward_marked.argtypes = [pL, c_vp, c_i32, c_vp, c_vp, c_sz, c_vp, c_vp, c_i32]
    L.bmoe_butterfly_backward_workspace.argtypes = [c_i32, c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_butterfly_backward.argtypes = [c_i32, c_i32, c_i32, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp,
                                          c_vp, c_vp, c_sz, c_vp]
    L.bmoe_substrate_grad_workspace.argtypes = [c_i32, c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_substrate_grad.argtypes = [c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_f, c_vp, c_vp, c_sz, c_vp]
    L.bmoe_combine_backward.argtypes = [c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp]
    L.bmoe_router_backward_workspace.argtypes = [c_i32, c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_router_backward.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                       c_vp, c_sz, c_vp]
    L.bmoe_gelu_backward.argtypes = [c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp]
    L.bmoe_substrate_input_grad.argtypes = [c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_f, c_vp, c_vp]
    L.bmoe_train_state_size.argtypes = [pL, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_forward_train_workspace.argtypes = [pL, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_forward_train.argtypes = [pL, c_vp, c_i32, c_vp, c_vp, c_sz, c_vp, c_sz, c_vp]
    L.bmoe_layer_backward_workspace.argtypes = [pL, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_layer_backward.argtypes = [pL, c_vp, c_i32, c_vp, c_vp, c_sz, ctypes.POINTER(LayerGrads), c_vp, c_sz,
                                      c_vp]
    c_d = ctypes.c_double
    L.bmoe_layer_norm_forward.argtypes = [c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_f, c_vp, c_vp, c_vp, c_vp, c_vp]
    L.bmoe_layer_norm_backward_workspace.argtypes = [c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_layer_norm_backward.argtypes = [c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp, c_vp,
                                           c_vp, c_vp, c_sz, c_vp]
    L.bmoe_orthogonalize_workspace.argtypes = [c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_orthogonalize.argtypes = [c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_f, c_i32, c_vp, c_vp, c_sz, c_vp]
    L.bmoe_substrate_step_workspace.argtypes = [c_i32, c_i32, ctypes.POINTER(c_sz)]
    L.bmoe_substrate_step.argtypes = [c_i32, c_i32, c_vp, c_vp, c_d, c_d, c_vp, c_vp, c_vp, c_vp, c_sz, c_vp]
    ret = [n for n in EXPORTED_SYMBOLS if n not in ("bmoe_packed_words", "bmoe_prepared_bytes",
                                                    "bmoe_status_string", "bmoe_last_error")]
    if debug:
        L.bmoe_dbg_butterfly.argtypes = [c_i32, c_i32, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp]
        L.bmoe_dbg_ternary_gemm.argtypes = [c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_f, c_vp, c_vp]
        L.bmoe_dbg_ternary_gemm_fp4.argtypes = [c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_f, c_vp, c_vp]
        ret += DEBUG_SYMBOLS
    for name in ret:
        getattr(L, name).restype = c_i32
    return L


def lib() -> ctypes.CDLL:
    """Load libbmoe.so (built in-tree by compressed_mixture_experts_amd.build)."""
    global _lib
    if _lib is None:
        alt = os.environ.get("BMOE_LIBRARY")
        _lib = debug_lib() if alt else _load(_LIB_PATH, debug=False)
    return _lib


def debug_lib() -> ctypes.CDLL:
    """Load libbmoe_debug.so: the product exports plus the test hooks of
    include/bmoe_debug.h (or the library BMOE_LIBRARY names)."""
    global _debug_lib
    if _debug_lib is None:
        _debug_lib = _load(os.environ.get("BMOE_LIBRARY") or _DEBUG_LIB_PATH, debug=True)
    return _debug_lib


def _check(status: int, L: Optional[ctypes.CDLL] = None) -> None:
    """Raise BmoeError for a nonzero status; the detail comes from the
    thread-local error string of the library that returned it."""
    if status != 0:
        detail = (L or lib()).bmoe_last_error().decode(errors="replace")
        raise BmoeError(status, detail)


def packed_words(rows: int, cols: int) -> int:
    return int(lib().bmoe_packed_words(rows, cols))


def pack_ternary(w: np.ndarray) -> np.ndarray:
    """int8 [rows][cols] in {-1,0,1} -> uint32 [rows][cols/16] (host, via the C ABI)."""
    w = np.ascontiguousarray(w, dtype=np.int8)
    if w.ndim != 2:
        raise ValueError("pack_ternary expects a 2-D array")
    rows, cols = w.shape
    nw = packed_words(rows, cols)
    out = np.zeros(max(nw, 1), dtype=np.uint32)
    _check(lib().bmoe_pack_ternary(w.ctypes.data, rows, cols, out.ctypes.data, nw))
    return out[:nw].reshape(rows, cols // 16)


# --------------------------------------------------------------------------- torch glue
def _torch():
    import torch
    return torch


def _stream_handle(stream=None) -> int:
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _to_device_act(a: np.ndarray, act: str, device):
    torch = _torch()
    if act == "bf16":
        t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.uint16).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32))
    return t.to(device).contiguous()


class Layer:
    """A ButterflyMoE layer resident on one GPU (weights packed and uploaded)."""

    def __init__(self, *, d_model: int, d_ff: int, n_experts: int, top_k: int, act: str,
                 ffn_act: str, renorm_gates: bool, w_gate, w_base_packed: Sequence,
                 theta: Sequence, phi: Sequence, w_scale: Sequence[float]):
        self.d_model, self.d_ff, self.n_experts, self.top_k = d_model, d_ff, n_experts, top_k
        self.act = act
        self.w_gate = w_gate
        self.w_base = list(w_base_packed)
        self.theta = list(theta)
        self.phi = list(phi)
        s = LayerStruct()
        s.d_model, s.d_ff, s.n_experts, s.top_k = d_model, d_ff, n_experts, top_k
        s.act_dtype = BF16 if act == "bf16" else F32
        s.ffn_act = ACT_GELU_ERF if ffn_act == "gelu" else ACT_NONE
        s.renorm_gates = 1 if renorm_gates else 0
        s.reserved = 0
        s.w_gate = _ptr(w_gate)
        for m in range(2):
            s.w_base[m] = _ptr(self.w_base[m]) if m < len(self.w_base) else None
            s.theta[m] = _ptr(self.theta[m]) if m < len(self.theta) else None
            s.phi[m] = _ptr(self.phi[m]) if m < len(self.phi) else None
            s.w_scale[m] = float(w_scale[m]) if m < len(w_scale) else 1.0
        s.prepared, s.prepared_bytes = None, 0
        self.struct = s
        self._ws = None
        self._prep = None

    @classmethod
    def from_inputs(cls, inp, device="cuda") -> "Layer":
        """Pack and upload the arrays of a workloads.LayerInputs."""
        torch = _torch()
        cfg = inp.cfg
        packed = [torch.from_numpy(pack_ternary(w).view(np.int32)).to(device).contiguous()
                  for w in inp.w_base]
        th = [torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device) for a in inp.theta]
        ph = [torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(device) for a in inp.phi]
        wg = _to_device_act(inp.w_gate, cfg.act, device)
        nsub = len(inp.w_base)
        return cls(d_model=cfg.d_model, d_ff=cfg.d_ff, n_experts=cfg.n_experts, top_k=cfg.top_k,
                   act=cfg.act, ffn_act=cfg.ffn_act, renorm_gates=cfg.renorm_gates, w_gate=wg,
                   w_base_packed=packed, theta=th, phi=ph, w_scale=[cfg.w_scale] * nsub)

    # ---------------------------------------------------------------- prepared weights
    def prepared_bytes(self) -> int:
        return int(lib().bmoe_prepared_bytes(ctypes.byref(self.struct)))

    def prepare(self):
        """Build the prepared weights once (bmoe_prepare) and use them from now
        on; a no-op for layers whose forward uses none."""
        torch = _torch()
        need = self.prepared_bytes()
        self.struct.prepared, self.struct.prepared_bytes = None, 0
        if need == 0:
            self._prep = None
            return self
        buf = torch.empty(need + 256, dtype=torch.uint8, device=self.w_gate.device)
        off = (-int(buf.data_ptr())) % 256
        view = buf[off:off + need]
        _check(lib().bmoe_prepare(ctypes.byref(self.struct), _ptr(view), need, _stream_handle()))
        self._prep = buf
        self.struct.prepared, self.struct.prepared_bytes = _ptr(view), need
        return self

    def unprepare(self):
        """Go back to building the prepared data inside every forward."""
        self.struct.prepared, self.struct.prepared_bytes = None, 0
        self._prep = None
        return self

    # ---------------------------------------------------------------- workspace
    def workspace_size(self, T: int) -> int:
        n = ctypes.c_size_t(0)
        _check(lib().bmoe_workspace_size(ctypes.byref(self.struct), int(T), ctypes.byref(n)))
        return int(n.value)

    def workspace(self, T: int, device=None):
        """A cached device workspace large enough for T tokens."""
        torch = _torch()
        need = self.workspace_size(T)
        if self._ws is None or self._ws.numel() < need:
            dev = device if device is not None else self.w_gate.device
            self._ws = torch.empty(max(need, 256) + 256, dtype=torch.uint8, device=dev)
        ws = self._ws
        off = (-int(ws.data_ptr())) % 256
        return ws[off:], need

    # ---------------------------------------------------------------- calls
    def route(self, x, with_buckets: bool = False):
        """Top-k routing of x [T][d_model].  Returns (idx [T][k] int32, gate [T][k]
        fp32[, offsets [N+1], bucket_slots [T*k]])."""
        torch = _torch()
        T = int(x.shape[0])
        dev = x.device
        idx = torch.empty((T, self.top_k), dtype=torch.int32, device=dev)
        gate = torch.empty((T, self.top_k), dtype=torch.float32, device=dev)
        off = slots = None
        if with_buckets:
            off = torch.empty(self.n_experts + 1, dtype=torch.int32, device=dev)
            slots = torch.empty(max(T * self.top_k, 1), dtype=torch.int32, device=dev)
        ws, nbytes = self.workspace(T, dev)
        _check(lib().bmoe_route(ctypes.byref(self.struct), _ptr(x), T, _ptr(idx), _ptr(gate),
                                _ptr(off), _ptr(slots), _ptr(ws), nbytes, _stream_handle()))
        if with_buckets:
            return idx, gate, off, slots[:T * self.top_k]
        return idx, gate

    def forward(self, x, y=None, return_routing: bool = False):
        """y [T][d_model] = ButterflyMoE layer(x)."""
        torch = _torch()
        T = int(x.shape[0])
        if y is None:
            y = torch.empty_like(x)
        idx = gate = None
        if return_routing:
            idx = torch.empty((T, self.top_k), dtype=torch.int32, device=x.device)
            gate = torch.empty((T, self.top_k), dtype=torch.float32, device=x.device)
        ws, nbytes = self.workspace(T, x.device)
        _check(lib().bmoe_forward(ctypes.byref(self.struct), _ptr(x), T, _ptr(y), _ptr(idx),
                                  _ptr(gate), _ptr(ws), nbytes, _stream_handle()))
        if return_routing:
            return y, idx, gate
        return y

    def forward_noalloc(self, x, y, idx=None, gate=None):
        """bmoe_forward_noalloc: the forward into caller-given y (and optional
        idx / gate [T][top_k]) with the library's fixed device scratch as the
        workspace; nothing is allocated by the call."""
        T = int(x.shape[0])
        _check(lib().bmoe_forward_noalloc(ctypes.byref(self.struct), _ptr(x), T, _ptr(y), _ptr(idx),
                                          _ptr(gate), _stream_handle()))
        return y

    def _sized(self, fn, T: int, device) -> Tuple[object, int]:
        torch = _torch()
        n = ctypes.c_size_t(0)
        _check(fn(ctypes.byref(self.struct), T, ctypes.byref(n)))
        return torch.empty(max(int(n.value), 256), dtype=torch.uint8, device=device), int(n.value)

    def forward_train(self, x, y=None):
        """bmoe_forward_train: y = layer(x) and the state the layer backward
        reads (an opaque device buffer).  Returns (y, state)."""
        torch = _torch()
        T = int(x.shape[0])
        if y is None:
            y = torch.empty_like(x)
        state, ns = self._sized(lib().bmoe_train_state_size, T, x.device)
        ws, nw = self._sized(lib().bmoe_forward_train_workspace, T, x.device)
        _check(lib().bmoe_forward_train(ctypes.byref(self.struct), _ptr(x), T, _ptr(y), _ptr(state), ns, _ptr(ws), nw,
                                        _stream_handle()))
        return y, state

    def backward(self, x, dy, state) -> dict:
        """bmoe_layer_backward: fp32 gradients of sum(dy * y) in x, the gate
        matrix, every rotation's angles and the latent substrates, at the
        state of forward_train(x).  Returns dict(x, w_gate, theta [list],
        phi [list], w_base [list]) of device tensors."""
        torch = _torch()
        T = int(x.shape[0])
        dev = x.device
        nm = 2 if self.struct.d_ff else 1
        out = {"x": torch.empty((T, self.d_model), dtype=torch.float32, device=dev),
               "w_gate": torch.empty((self.n_experts, self.d_model), dtype=torch.float32, device=dev),
               "theta": [], "phi": [], "w_base": []}
        g = LayerGrads()
        g.dx = _ptr(out["x"])
        g.d_w_gate = _ptr(out["w_gate"])
        for m in range(nm):
            th, ph = self.theta[m], self.phi[m]
            out["theta"].append(torch.empty_like(th, dtype=torch.float32))
            out["phi"].append(torch.empty_like(ph, dtype=torch.float32))
            d_out = 1 << (ph.shape[1])
            d_in = 1 << (th.shape[1])
            out["w_base"].append(torch.empty((d_out, d_in), dtype=torch.float32, device=dev))
            g.d_theta[m] = _ptr(out["theta"][m])
            g.d_phi[m] = _ptr(out["phi"][m])
            g.d_w_base[m] = _ptr(out["w_base"][m])
        ws, nw = self._sized(lib().bmoe_layer_backward_workspace, T, dev)
        _check(lib().bmoe_layer_backward(ctypes.byref(self.struct), _ptr(x), T, _ptr(dy), _ptr(state),
                                         int(state.numel()), ctypes.byref(g), _ptr(ws), nw, _stream_handle()))
        return out

    def set_scale(self, m: int, scale) -> "Layer":
        """The factor of substrate m's codes (bmoe_layer's w_scale) in every call
        from now on: a number, or a one-element tensor, whose reading waits for its
        GPU.  The factor is an argument of the launches: a forward captured before
        replays with the one it was captured with."""
        if not 0 <= m < len(self.w_base):
            raise ValueError(f"the layer has no substrate {m}")
        scale = float(scale)
        if not abs(scale) <= float(np.finfo(np.float32).max):
            raise ValueError(f"substrate {m}'s scale must be finite in fp32, got {scale}")
        self.struct.w_scale[m] = scale
        return self

    def step_substrate(self, m: int, w, o=None, step: float = 0.0, decay: float = 0.0, w_out=None,
                       rescale: bool = False):
        """substrate_step of latent substrate m ([d_out][d_in] fp32) with the
        codes written into this layer; weights prepared before are prepared
        again in the same buffer, which graphs captured from this layer read.
        Returns (W', scale).

        scale * codes stand for W'.  With rescale the layer's factor
        follows (set_scale with the step's scale, which waits for the GPU and is
        refused in a capture), so that the layer computes with scale * codes.
        Without, the factor stays what it is: the layer's output and the gradient
        of its substrate keep that factor whatever |W'| is, which is what a step
        in a captured graph can do."""
        if not 0 <= m < len(self.w_base):
            raise ValueError(f"the layer has no substrate {m}")
        d_out, d_in = 1 << int(self.phi[m].shape[1]), 1 << int(self.theta[m].shape[1])
        if tuple(w.shape) != (d_out, d_in):
            raise ValueError(f"w has shape {tuple(w.shape)}, substrate {m} is {(d_out, d_in)}")
        if rescale and w.is_cuda and _torch().cuda.is_current_stream_capturing():
            raise ValueError("rescale reads the scale on the host, which a captured step cannot do")
        w, _, scale = substrate_step(w, o, step, decay, w_out=w_out, packed=self.w_base[m])
        if self._prep is not None:
            with _torch().cuda.device(w.device):
                _check(lib().bmoe_prepare(ctypes.byref(self.struct), self.struct.prepared, self.struct.prepared_bytes,
                                          _stream_handle()))
        if rescale:
            self.set_scale(m, scale)
        return w, scale

    def kernel_names(self) -> List[str]:
        """Names of the kernel launches of one forward, in order."""
        n = ctypes.c_int32(0)
        buf = ctypes.create_string_buffer(512)
        _check(lib().bmoe_forward_kernels(ctypes.byref(self.struct), ctypes.byref(n), buf, 512))
        return buf.value.decode().split(",")[: n.value]

    def forward_marked(self, x, y, marks):
        """Forward into y, recording the raw hipEvent_t handles in `marks`
        (list of ints or None) before the first and after each kernel launch."""
        T = int(x.shape[0])
        ws, nbytes = self.workspace(T, x.device)
        arr = (ctypes.c_void_p * max(len(marks), 1))(*[m if m else None for m in marks])
        _check(lib().bmoe_forward_marked(ctypes.byref(self.struct), _ptr(x), T, _ptr(y),
                                             _ptr(ws), nbytes, _stream_handle(), arr, len(marks)))
        return y


def dbg_butterfly(angles, x, transpose: bool = False, out=None):
    """Rows of x [rows][n] -> B(angles) row (or B^T row); angles [log2 n][n/2] fp32."""
    torch = _torch()
    rows, n = int(x.shape[0]), int(x.shape[1])
    log2n = n.bit_length() - 1
    dtype = BF16 if x.dtype == torch.bfloat16 else F32
    if out is None:
        out = torch.empty_like(x)
    D = debug_lib()
    _check(D.bmoe_dbg_butterfly(log2n, rows, _ptr(angles), 1 if transpose else 0, dtype,
                                _ptr(x), _ptr(out), _stream_handle()), D)
    return out


def butterfly_backward(angles, offsets, x, dy, transpose: bool = False, dx=None):
    """Backward of the bucketed rotation pass y_r = B(angles_e) x_r (or B^T x_r)
    for rows r of expert e (rows offsets[e] .. offsets[e+1]-1).  angles
    [N][L][n/2] fp32, offsets [N+1] int32, x and dy [rows][n] (fp32 or bf16).
    Returns (dx [rows][n] like x, dangles [N][L][n/2] fp32)."""
    torch = _torch()
    N, L = int(angles.shape[0]), int(angles.shape[1])
    rows = int(x.shape[0])
    dtype = BF16 if x.dtype == torch.bfloat16 else F32
    if dx is None:
        dx = torch.empty_like(x)
    dang = torch.empty_like(angles)
    nb = ctypes.c_size_t(0)
    _check(lib().bmoe_butterfly_backward_workspace(L, N, rows, ctypes.byref(nb)))
    ws = torch.empty(max(int(nb.value), 16), dtype=torch.uint8, device=x.device)
    _check(lib().bmoe_butterfly_backward(L, N, rows, _ptr(offsets), _ptr(angles), 1 if transpose else 0, dtype,
                                         _ptr(x), _ptr(dy), _ptr(dx), _ptr(dang), _ptr(ws), int(nb.value),
                                         _stream_handle()))
    return dx, dang


def substrate_grad(dz, u, alpha: float = 1.0, dw=None):
    """Latent substrate gradient through the straight-through estimator:
    dw [d_out][d_in] fp32 = alpha * dz^T u over all rows; dz [rows][d_out] and
    u [rows][d_in] bf16."""
    torch = _torch()
    rows, d_out, d_in = int(dz.shape[0]), int(dz.shape[1]), int(u.shape[1])
    if dw is None:
        dw = torch.empty((d_out, d_in), dtype=torch.float32, device=dz.device)
    nb = ctypes.c_size_t(0)
    _check(lib().bmoe_substrate_grad_workspace(d_out, d_in, rows, ctypes.byref(nb)))
    ws = torch.empty(max(int(nb.value), 16), dtype=torch.uint8, device=dz.device)
    _check(lib().bmoe_substrate_grad(d_out, d_in, rows, BF16 if dz.dtype == torch.bfloat16 else F32, _ptr(dz),
                                     _ptr(u), float(alpha), _ptr(dw), _ptr(ws), int(nb.value), _stream_handle()))
    return dw


def combine_backward(dy, bucket_slots, topk_gate, top_k: int, o=None):
    """Backward of the gated combine: d_rows [T*k][d] = gate * dy[token] in
    bucket order, and (with the experts' outputs o in bucket order) d_gate
    [T*k] by flat slot.  Returns (d_rows, d_gate or None)."""
    torch = _torch()
    T, d = int(dy.shape[0]), int(dy.shape[1])
    d_rows = torch.empty((T * top_k, d), dtype=dy.dtype, device=dy.device)
    d_gate = torch.empty(T * top_k, dtype=torch.float32, device=dy.device) if o is not None else None
    _check(lib().bmoe_combine_backward(T, top_k, d, BF16 if dy.dtype == torch.bfloat16 else F32, _ptr(dy),
                                       _ptr(bucket_slots), _ptr(topk_gate), _ptr(o), _ptr(d_rows), _ptr(d_gate),
                                       _stream_handle()))
    return d_rows, d_gate


def router_backward(x, w_gate, topk_idx, d_gate, renorm: bool = False):
    """Gating network's backward with the chosen experts held: returns
    (dx [T][d] fp32, dw_gate [N][d] fp32)."""
    torch = _torch()
    T, d, N, k = int(x.shape[0]), int(x.shape[1]), int(w_gate.shape[0]), int(topk_idx.shape[1])
    dx = torch.empty((T, d), dtype=torch.float32, device=x.device)
    dwg = torch.empty((N, d), dtype=torch.float32, device=x.device)
    nb = ctypes.c_size_t(0)
    _check(lib().bmoe_router_backward_workspace(T, d, N, ctypes.byref(nb)))
    ws = torch.empty(max(int(nb.value), 16), dtype=torch.uint8, device=x.device)
    _check(lib().bmoe_router_backward(T, d, N, k, 1 if renorm else 0, BF16 if x.dtype == torch.bfloat16 else F32,
                                      _ptr(x), _ptr(w_gate), _ptr(topk_idx), _ptr(d_gate), _ptr(dx), _ptr(dwg),
                                      _ptr(ws), int(nb.value), _stream_handle()))
    return dx, dwg


def gelu_backward(h, da, dh=None):
    """dh = da * GELU'(h) (exact erf GELU), elementwise; h, da [rows][width]."""
    torch = _torch()
    rows, width = int(h.shape[0]), int(h.shape[1])
    if dh is None:
        dh = torch.empty_like(h)
    _check(lib().bmoe_gelu_backward(rows, width, BF16 if h.dtype == torch.bfloat16 else F32, _ptr(h), _ptr(da),
                                    _ptr(dh), _stream_handle()))
    return dh


def substrate_input_grad(dz, wt_packed, d_in: int, alpha: float = 1.0):
    """du [rows][d_in] = alpha * dz [rows][d_out] * W_base, with W_base^T packed
    ([d_in][d_out/16] words)."""
    torch = _torch()
    rows, d_out = int(dz.shape[0]), int(dz.shape[1])
    du = torch.empty((rows, d_in), dtype=dz.dtype, device=dz.device)
    _check(lib().bmoe_substrate_input_grad(rows, d_out, d_in, BF16 if dz.dtype == torch.bfloat16 else F32, _ptr(dz),
                                           _ptr(wt_packed), float(alpha), _ptr(du), _stream_handle()))
    return du


def _operand(name: str, t, shape, dtypes, device):
    """Check one tensor of a training-step operator: dense, on `device`, of the
    given shape and one of the dtypes."""
    if t.device == device and t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.is_cuda:
        return t
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected a GPU tensor on {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _on_device(fn):
    """Run fn(matrix, ...) with the first argument's GPU as the current device."""
    sig = inspect.signature(fn)
    name = next(iter(sig.parameters))

    @functools.wraps(fn)
    def run(*args, **kw):
        torch = _torch()
        first = args[0] if args else kw.get(name)
        if isinstance(first, torch.Tensor):
            index = first.get_device()
            if index >= 0 and first.dim() == 2:
                if index == torch._C._cuda_getDevice():
                    return fn(*args, **kw)
                with torch.cuda.device(index):
                    return fn(*args, **kw)
        sig.bind(*args, **kw)      # a missing argument is Python's own TypeError
        if isinstance(first, torch.Tensor) and first.is_cuda:
            raise ValueError(f"{fn.__name__} expects a 2-D tensor, got {tuple(first.shape)}")
        what = f"{name} on {first.device}" if isinstance(first, torch.Tensor) else f"{name} = {first!r}"
        raise ValueError(f"{fn.__name__} needs GPU tensors, got {what}")
    return run


def _raw_stream(t) -> int:
    """Handle of the current stream of t's GPU, without a torch Stream object (0.1
    instead of 2.7 us of a call whose kernel takes 3)."""
    return _torch()._C._cuda_getCurrentRawStream(t.get_device())


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(name: str, a: int, b: int) -> int:
    """What the library's size query `name` says for (a, b): sizes alone decide."""
    n = ctypes.c_size_t(0)
    _check(getattr(lib(), name)(a, b, ctypes.byref(n)))
    return int(n.value)


@_on_device
def layer_norm_forward(x, gamma=None, beta=None, eps: float = 1e-5, residual=None, stats: bool = True, y=None,
                       sum_out=None):
    """Row norm of s = x (+ residual): y = (s - mean) rstd gamma + beta.
    x, residual [rows][width] fp32 or bf16; gamma, beta [width] fp32 or None
    (ones, zeros).  Returns (y, s, mean, rstd): s is x itself without a
    residual (None where y is written over x: the row that a backward reads is
    gone), mean and rstd ([rows] fp32) are None with stats=False."""
    torch = _torch()
    dev, kind, shape = x.device, x.dtype, x.shape
    rows, width = shape
    _operand("x", x, shape, (torch.float32, torch.bfloat16), dev)
    if gamma is not None:
        _operand("gamma", gamma, (width,), (torch.float32,), dev)
    if beta is not None:
        _operand("beta", beta, (width,), (torch.float32,), dev)
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out needs a residual")
    else:
        _operand("residual", residual, shape, (kind,), dev)
        sum_out = torch.empty_like(x) if sum_out is None else _operand("sum_out", sum_out, shape, (kind,), dev)
    y = torch.empty_like(x) if y is None else _operand("y", y, shape, (kind,), dev)
    mean = rstd = None
    if stats:
        mean, rstd = torch.empty(rows, dtype=torch.float32, device=dev), torch.empty(rows, dtype=torch.float32, device=dev)
    _check(lib().bmoe_layer_norm_forward(
        rows, width, BF16 if kind is torch.bfloat16 else F32, x.data_ptr(), None if residual is None else residual.data_ptr(),
        None if gamma is None else gamma.data_ptr(), None if beta is None else beta.data_ptr(), eps,
        None if residual is None else sum_out.data_ptr(), y.data_ptr(), mean.data_ptr() if stats else None,
        rstd.data_ptr() if stats else None, _raw_stream(x)))
    if residual is None:
        return y, None if y.data_ptr() == x.data_ptr() and x.numel() else x, mean, rstd
    return y, sum_out, mean, rstd


@_on_device
def layer_norm_backward(dy, s, gamma, mean, rstd, d_sum=None, weight_grads: bool = True, dx=None):
    """Backward of layer_norm_forward at its s, mean and rstd: dy [rows][width]
    fp32 or of s's dtype, d_sum [rows][width] like s or None (gradient that
    reaches s past the norm, added into dx).  Returns (dx like s, dgamma,
    dbeta [width] fp32; None with weight_grads=False)."""
    torch = _torch()
    if s is None:
        raise ValueError("s is None: the forward wrote y over the row that the backward reads")
    dev, kind, shape, f32 = dy.device, s.dtype, dy.shape, (torch.float32,)
    rows, width = shape
    _operand("s", s, shape, (torch.float32, torch.bfloat16), dev)
    _operand("dy", dy, shape, (torch.float32, kind), dev)
    if gamma is not None:
        _operand("gamma", gamma, (width,), f32, dev)
    _operand("mean", mean, (rows,), f32, dev)
    _operand("rstd", rstd, (rows,), f32, dev)
    if d_sum is not None:
        _operand("d_sum", d_sum, shape, (kind,), dev)
    dx = torch.empty_like(s) if dx is None else _operand("dx", dx, shape, (kind,), dev)
    dgamma = dbeta = ws = None
    nbytes = 0
    if weight_grads:
        dgamma, dbeta = torch.empty(width, dtype=torch.float32, device=dev), torch.empty(width, dtype=torch.float32, device=dev)
        nbytes = _workspace_bytes("bmoe_layer_norm_backward_workspace", rows, width)
        if nbytes:
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib().bmoe_layer_norm_backward(
        rows, width, BF16 if kind is torch.bfloat16 else F32, BF16 if dy.dtype is torch.bfloat16 else F32, dy.data_ptr(),
        s.data_ptr(), None if gamma is None else gamma.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        None if d_sum is None else d_sum.data_ptr(), dx.data_ptr(), dgamma.data_ptr() if weight_grads else None,
        dbeta.data_ptr() if weight_grads else None, None if ws is None else ws.data_ptr(), nbytes, _raw_stream(dy)))
    return dx, dgamma, dbeta


@_on_device
def orthogonalize(grad, momentum=None, mu: float = 0.95, nesterov: bool = True, momentum_out=None, out=None):
    """Orthogonalised update of a matrix gradient [rows][cols] (fp32 or bf16):
    momentum step M' = mu M + G (fp32, when momentum is given) and five
    Newton-Schulz steps on G + mu M' (or M', or G).  Returns (out bf16
    [rows][cols], M' or None); momentum_out may be momentum itself."""
    torch = _torch()
    dev, shape, f32 = grad.device, grad.shape, (torch.float32,)
    rows, cols = shape
    _operand("grad", grad, shape, (torch.float32, torch.bfloat16), dev)
    if momentum is None:
        if momentum_out is not None:
            raise ValueError("momentum_out needs a momentum")
    else:
        _operand("momentum", momentum, shape, f32, dev)
        momentum_out = (torch.empty_like(momentum) if momentum_out is None else
                        _operand("momentum_out", momentum_out, shape, f32, dev))
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    else:
        _operand("out", out, shape, (torch.bfloat16,), dev)
    nbytes = _workspace_bytes("bmoe_orthogonalize_workspace", rows, cols)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _check(lib().bmoe_orthogonalize(rows, cols, BF16 if grad.dtype is torch.bfloat16 else F32, grad.data_ptr(),
                                    _ptr(momentum), _ptr(momentum_out), float(mu), 1 if nesterov else 0, out.data_ptr(),
                                    ws.data_ptr(), nbytes, _raw_stream(grad)))
    return out, momentum_out


@_on_device
def substrate_step(w, o=None, step: float = 0.0, decay: float = 0.0, w_out=None, packed=None):
    """Latent substrate step W' = (1 - decay) W - step O (W [rows][cols] fp32, O
    bf16; W' = W without O) and its ternary codes at threshold mean |W'| / 2.
    Returns (W', packed [rows][cols / 16] int32 in pack_ternary's format,
    scale: 0-d fp32 tensor mean |W'|, the factor under which the codes stand for
    W').  w_out may be w itself (Layer.step_substrate writes the codes into a
    layer)."""
    torch = _torch()
    dev, shape = w.device, w.shape
    rows, cols = shape
    _operand("w", w, shape, (torch.float32,), dev)
    if o is None:
        if w_out is not None:
            raise ValueError("w_out needs an update o")
    else:
        _operand("o", o, shape, (torch.bfloat16,), dev)
        w_out = torch.empty_like(w) if w_out is None else _operand("w_out", w_out, shape, (torch.float32,), dev)
    nbytes = _workspace_bytes("bmoe_substrate_step_workspace", rows, cols)
    if packed is None:
        packed = torch.empty((rows, cols // 16), dtype=torch.int32, device=dev)
    else:
        _operand("packed", packed, (rows, cols // 16), (torch.int32,), dev)
    scale = torch.empty((), dtype=torch.float32, device=dev)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _check(lib().bmoe_substrate_step(rows, cols, w.data_ptr(), _ptr(o), float(step), float(decay), _ptr(w_out),
                                     packed.data_ptr(), scale.data_ptr(), _ptr(ws), nbytes, _raw_stream(w)))
    return w if o is None else w_out, packed, scale


def dbg_ternary_gemm(a, w_packed, n_out: int, alpha: float = 1.0):
    """z [M][n_out] = alpha * a [M][K] @ W^T with W packed [n_out][K/16]."""
    torch = _torch()
    M, K = int(a.shape[0]), int(a.shape[1])
    dtype = BF16 if a.dtype == torch.bfloat16 else F32
    z = torch.empty((M, n_out), dtype=a.dtype, device=a.device)
    D = debug_lib()
    _check(D.bmoe_dbg_ternary_gemm(M, n_out, K, dtype, _ptr(a), _ptr(w_packed), float(alpha),
                                   _ptr(z), _stream_handle()), D)
    return z


def dbg_ternary_gemm_fp4(a, w_packed, n_out: int, alpha: float = 1.0):
    """Matrix-core form of dbg_ternary_gemm for bf16 `a` (substrate re-encoded as
    paired 2-bit codes in a scratch buffer first)."""
    torch = _torch()
    M, K = int(a.shape[0]), int(a.shape[1])
    z = torch.empty((M, n_out), dtype=a.dtype, device=a.device)
    scratch = torch.empty((n_out * K // 4,), dtype=torch.uint8, device=a.device)
    D = debug_lib()
    _check(D.bmoe_dbg_ternary_gemm_fp4(M, n_out, K, _ptr(a), _ptr(w_packed), _ptr(scratch),
                                       float(alpha), _ptr(z), _stream_handle()), D)
    return z
