"""Argument errors of the operators around a layer (include/bmoe_adamw.h, bmoe_block.h,
bmoe_ffn.h): each is
found on the host before anything is enqueued, so the pointers here are never followed.
No GPU needed."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import compressed_mixture_experts_amd as bm
from compressed_mixture_experts_amd import blocks
from compressed_mixture_experts_amd import build as bbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, DTYPE, ALIGN, ALIAS, WORKSPACE = 1, 2, 3, 4, 5, 6
MB = 1 << 20


def ptr(k):
    """Made-up address of array k, far from every other one."""
    return (k + 1) * 64 * MB


def tensors(changes=(), second=()):
    """Two tensors of 1000 values, of 32 and 8 bits."""
    t = np.zeros(2, dtype=blocks._ADAMW_TENSOR)
    for i, (bits, change) in enumerate(((32, changes), (8, second))):
        row = dict(param=ptr(10 * i), grad=ptr(10 * i + 1), m=ptr(10 * i + 2), v=ptr(10 * i + 3), m_exp=ptr(10 * i + 4) if bits == 8 else 0,
                   v_exp=ptr(10 * i + 5) if bits == 8 else 0, copy=ptr(10 * i + 6), n=1000, lr_scale=1.0, weight_decay=0.0, grad_dtype=0,
                   bits=bits)
        row.update(change)
        for k, x in row.items():
            t[k][i] = x
    return t


ARGS = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, step_device=None, lr_device=None, grad_scale=None, seed=0, reserved=0)


def step(t, **change):
    a = blocks._AdamWArgs(**dict(ARGS, **change))
    return bm.lib().bmoe_adamw_step(t.ctypes.data, len(t), ctypes.byref(a), None)


REFUSED_TENSORS = [
    (dict(n=-1), {}, SHAPE), (dict(n=(1 << 33) + 1), {}, SHAPE), (dict(lr_scale=float("nan")), {}, SHAPE),
    (dict(weight_decay=float("inf")), {}, SHAPE), (dict(bits=16), {}, DTYPE), (dict(grad_dtype=2), {}, DTYPE),
    (dict(param=0), {}, NULL), (dict(m=0), {}, NULL), (dict(v=0), {}, NULL), ({}, dict(m_exp=0), NULL), ({}, dict(v_exp=0), NULL),
    (dict(param=ptr(0) + 2), {}, ALIGN), (dict(grad=ptr(1) + 1), {}, ALIGN), (dict(m=ptr(2) + 2), {}, ALIGN), (dict(copy=ptr(6) + 1), {}, ALIGN),
    (dict(grad=ptr(1) + 1, grad_dtype=1), {}, ALIGN),
    # within a tensor, and between two
    (dict(grad=ptr(0) + 4), {}, ALIAS), (dict(m=ptr(0)), {}, ALIAS), (dict(v=ptr(2)), {}, ALIAS), (dict(copy=ptr(1) + 2), {}, ALIAS),
    ({}, dict(m_exp=ptr(15)), ALIAS), ({}, dict(v_exp=ptr(12) + 999), ALIAS), ({}, dict(param=ptr(0) + 3996), ALIAS),
    ({}, dict(grad=ptr(3)), ALIAS), ({}, dict(copy=ptr(6) + 1998), ALIAS), (dict(grad=ptr(13)), {}, ALIAS), ({}, dict(m=ptr(0) - 999), ALIAS),
]


@pytest.mark.parametrize("first,second,status", REFUSED_TENSORS, ids=lambda v: str(v)[:50])
def test_adamw_tensor_refusals(first, second, status):
    assert step(tensors(first, second)) == status
    assert bm.lib().bmoe_last_error() != b""


REFUSED_ARGS = [
    (dict(lr=float("nan")), SHAPE), (dict(lr=float("inf")), SHAPE), (dict(beta1=1.0), SHAPE), (dict(beta1=-0.1), SHAPE),
    (dict(beta2=1.0), SHAPE), (dict(beta2=float("nan")), SHAPE), (dict(eps=-1e-8), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(eps=1e-40), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(step=0), SHAPE), (dict(reserved=1), SHAPE),
    (dict(step_device=ptr(40) + 4), ALIGN), (dict(lr_device=ptr(40) + 2), ALIGN), (dict(grad_scale=ptr(40) + 1), ALIGN),
    (dict(step_device=ptr(0)), ALIAS), (dict(lr_device=ptr(0) + 8), ALIAS), (dict(grad_scale=ptr(2)), ALIAS),
    (dict(step_device=ptr(40), lr_device=ptr(40) + 4), ALIAS),
]


@pytest.mark.parametrize("change,status", REFUSED_ARGS, ids=lambda v: str(v)[:50])
def test_adamw_argument_refusals(change, status):
    assert step(tensors(), **change) == status


def test_adamw_nothing_to_do():
    """No tensors, no values, no gradients: nothing is launched, no GPU is needed."""
    L = bm.lib()
    a = blocks._AdamWArgs(**ARGS)
    assert L.bmoe_adamw_step(None, 0, ctypes.byref(a), None) == 0
    assert step(tensors(dict(n=0, param=0, m=0, v=0), dict(grad=0))) == 0
    assert L.bmoe_adamw_step(None, 2, ctypes.byref(a), None) == NULL
    assert L.bmoe_adamw_step(None, 0, None, None) == NULL
    assert L.bmoe_adamw_step(None, -1, ctypes.byref(a), None) == SHAPE
    # what is read may be read twice: refused for another reason
    t = tensors(dict(grad=ptr(11)))
    assert step(t, beta1=2.0) == SHAPE


def moments(t, m_out, v_out, kind=0):
    m, v = np.array(m_out, dtype=np.uint64), np.array(v_out, dtype=np.uint64)
    return bm.lib().bmoe_adamw_moments(t.ctypes.data, len(t), kind, m.ctypes.data, v.ctypes.data, None)


def test_adamw_moments_refusals():
    t = tensors(second={})[1:].copy()
    assert moments(t, [ptr(30)], [ptr(31)], kind=2) == DTYPE
    assert moments(tensors(), [ptr(30), ptr(31)], [ptr(32), ptr(33)]) == DTYPE   # the first has no codes
    assert moments(t, [ptr(30) + 2], [ptr(31)]) == ALIGN and moments(t, [ptr(30)], [ptr(31) + 1], kind=1) == ALIGN
    assert moments(t, [ptr(30)], [ptr(30) + 4]) == ALIAS and moments(t, [ptr(12)], [0]) == ALIAS
    assert moments(t, [0], [ptr(15) - 4]) == ALIAS
    assert moments(t, [0], [0]) == 0
    assert bm.lib().bmoe_adamw_moments(None, 1, 0, None, None, None) == NULL
    assert bm.lib().bmoe_adamw_moments(None, -1, 0, None, None, None) == SHAPE


def test_adamw_struct_is_the_header_s():
    """Sizes of the two structures as the C compiler lays them out: 7 pointers, a 64-bit
    number and four 32-bit ones; 4 doubles, a 64-bit number, 3 pointers, two 32-bit numbers."""
    assert blocks._ADAMW_TENSOR.itemsize == 7 * 8 + 8 + 4 * 4 and ctypes.sizeof(blocks._AdamWArgs) == 4 * 8 + 8 + 3 * 8 + 2 * 4


def test_adamw_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    for params in ([torch.zeros(4)], [], [None]):
        with pytest.raises(ValueError):
            bm.AdamW(params)


NORM = dict(rows=2000, width=64, dtype=0, kind=0, post=1, gate_kind=1, alpha=1.0, scale=1.0, eps=1e-5, reserved=0, gate=ptr(0),
            gamma_post=ptr(1), beta_post=ptr(2), gamma=ptr(3), beta=ptr(4))
FWD = dict(b=ptr(5), r=ptr(6), s=ptr(7), y=ptr(8), stats=ptr(9))
BWD = dict(dy_dtype=0, dy=ptr(5), b=ptr(6), s=ptr(7), stats=ptr(8), d_sum=ptr(9), db=ptr(10), dr=ptr(11), grads=None, ws=ptr(12), ws_bytes=1 << 40)
GRADS = dict(gamma_post=ptr(13), beta_post=ptr(14), gate=ptr(15), gamma=ptr(16), beta=ptr(17))


def block_forward(norm={}, **change):
    n = blocks._BlockNorm(**dict(NORM, **norm))
    return bm.lib().bmoe_block_norm_forward(ctypes.byref(n), *dict(FWD, **change).values(), None)


def block_backward(norm={}, grads={}, **change):
    n = blocks._BlockNorm(**dict(NORM, beta=None, **norm) if "beta" not in norm else dict(NORM, **norm))
    g = blocks._BlockNormGrads(**dict(GRADS, **grads))
    args = dict(BWD, grads=ctypes.addressof(g))
    args.update(change)
    return bm.lib().bmoe_block_norm_backward(ctypes.byref(n), *args.values(), None)


BLOCK_NORM_REFUSED = [
    (dict(rows=-1), SHAPE), (dict(rows=(1 << 24) + 1), SHAPE), (dict(width=0), SHAPE), (dict(width=16385), SHAPE), (dict(post=2), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(alpha=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(reserved=1), SHAPE), (dict(post=0), SHAPE), (dict(post=0, gamma_post=None), SHAPE), (dict(kind=1), SHAPE), (dict(gate_kind=0), SHAPE),
    (dict(dtype=2), DTYPE), (dict(kind=2), DTYPE), (dict(gate_kind=3), DTYPE), (dict(gate_kind=-1), DTYPE), (dict(gate=None), NULL),
    (dict(gate=ptr(0) + 2), ALIGN), (dict(gate=ptr(0) + 1, gate_kind=2, dtype=1), ALIGN), (dict(gamma=ptr(3) + 2), ALIGN),
    (dict(beta_post=ptr(2) + 1), ALIGN),
]


@pytest.mark.parametrize("change,status", BLOCK_NORM_REFUSED, ids=lambda v: str(v)[:60])
def test_block_norm_description_refusals(change, status):
    assert block_forward(change) == status
    assert block_backward(change) == status
    assert bm.lib().bmoe_last_error() != b""


BLOCK_FORWARD_REFUSED = [
    (dict(b=None), NULL), (dict(s=None), NULL), (dict(y=None), NULL), (dict(b=ptr(5) + 2), ALIGN), (dict(r=ptr(6) + 1), ALIGN), (dict(stats=ptr(9) + 8), ALIGN),
    (dict(y=ptr(7)), ALIAS), (dict(y=ptr(5) + 4), ALIAS), (dict(s=ptr(6) - 4), ALIAS), (dict(s=ptr(3)), ALIAS), (dict(y=ptr(0)), ALIAS),
    (dict(stats=ptr(5)), ALIAS), (dict(stats=ptr(7) + 16), ALIAS), (dict(stats=ptr(1)), ALIAS), (dict(y=ptr(9) + 16), ALIAS),
]


@pytest.mark.parametrize("change,status", BLOCK_FORWARD_REFUSED, ids=lambda v: str(v)[:60])
def test_block_norm_forward_refusals(change, status):
    assert block_forward(**change) == status


BLOCK_BACKWARD_REFUSED = [
    ({}, {}, dict(dy_dtype=1), DTYPE), ({}, {}, dict(dy_dtype=2), DTYPE), ({}, {}, dict(dy=None), NULL), ({}, {}, dict(b=None), NULL),
    ({}, {}, dict(s=None), NULL), ({}, {}, dict(stats=None), NULL), ({}, {}, dict(db=None), NULL), ({}, {}, dict(ws=None), NULL),
    ({}, {}, dict(ws_bytes=100), WORKSPACE), ({}, {}, dict(ws=ptr(12) + 8), ALIGN), ({}, {}, dict(stats=ptr(8) + 4), ALIGN),
    ({}, {}, dict(dr=ptr(11) + 2), ALIGN), ({}, dict(gamma=ptr(16) + 2), {}, ALIGN),
    (dict(kind=1, beta_post=None), {}, {}, SHAPE), (dict(post=0, gamma_post=None, beta_post=None), {}, {}, SHAPE),
    (dict(gate_kind=0, gate=None), {}, {}, SHAPE),
    ({}, {}, dict(db=ptr(6) + 4), ALIAS), ({}, {}, dict(db=ptr(11)), ALIAS), ({}, {}, dict(dr=ptr(8)), ALIAS), ({}, {}, dict(dr=ptr(12)), ALIAS),
    ({}, {}, dict(db=ptr(0)), ALIAS), ({}, dict(gamma=ptr(5)), {}, ALIAS), ({}, dict(beta=ptr(16)), {}, ALIAS), ({}, dict(gate=ptr(0)), {}, ALIAS),
    ({}, dict(gate=ptr(10)), {}, ALIAS), ({}, {}, dict(ws=ptr(9)), ALIAS), ({}, {}, dict(ws=ptr(3) - 16), ALIAS), (dict(dtype=1), {}, dict(db=ptr(5)), ALIAS),
]


@pytest.mark.parametrize("norm,grads,change,status", BLOCK_BACKWARD_REFUSED, ids=lambda v: str(v)[:60])
def test_block_norm_backward_refusals(norm, grads, change, status):
    assert block_backward(norm, grads, **change) == status


def test_block_norm_nothing_to_do_and_sizes():
    n = ctypes.c_size_t(77)
    none = dict.fromkeys(GRADS)
    assert block_forward(dict(rows=0), b=None, s=None, y=None) == 0
    assert block_backward(dict(rows=0), none, dy=None, b=None, s=None, stats=None, db=None, dr=None, ws=None, ws_bytes=0) == 0
    for rows, width, status in ((-1, 64, SHAPE), (4, 0, SHAPE), (1 << 24, 16384, 0), (0, 64, 0)):
        d = blocks._BlockNorm(**dict(NORM, rows=rows, width=width))
        assert bm.lib().bmoe_block_norm_backward_workspace(ctypes.byref(d), ctypes.byref(n)) == status
    assert n.value == 0   # of no rows
    assert bm.lib().bmoe_block_norm_backward_workspace(None, ctypes.byref(n)) == NULL
    assert bm.lib().bmoe_block_norm_backward_workspace(ctypes.byref(d), None) == NULL
    assert ctypes.sizeof(blocks._BlockNorm) == 10 * 4 + 5 * 8 and ctypes.sizeof(blocks._BlockNormGrads) == 5 * 8


FFN = dict(tokens=100, d=64, ff=128, act=0, x=ptr(0), w_in=ptr(1), w_down=ptr(2), add=ptr(3), y=ptr(4), state=ptr(5), state_bytes=1 << 40,
           ws=ptr(6), ws_bytes=1 << 40, stream=None)
FFN_BWD = dict(tokens=100, d=64, ff=128, act=0, x=ptr(0), w_in=ptr(1), w_down=ptr(2), dy=ptr(3), state=ptr(4), state_bytes=1 << 40, dx_add=ptr(5),
               dx=ptr(6), dw_in=ptr(7), dw_down=ptr(8), ws=ptr(9), ws_bytes=1 << 40, stream=None)

FFN_SHAPES = [dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(d=0), dict(d=12), dict(d=16392), dict(ff=0), dict(ff=20), dict(ff=65544),
              dict(d=16384, ff=65536), dict(tokens=1 << 24, ff=4104), dict(d=-8)]
FFN_REFUSED = [(c, SHAPE) for c in FFN_SHAPES] + [
    (dict(act=2), DTYPE), (dict(act=-1), DTYPE), (dict(x=None), NULL), (dict(w_in=None), NULL), (dict(w_down=None), NULL), (dict(y=None), NULL),
    (dict(state=None, ws=None), NULL), (dict(x=ptr(0) + 8), ALIGN), (dict(add=ptr(3) + 2), ALIGN), (dict(state=ptr(5) + 4), ALIGN),
    (dict(state=None, ws=ptr(6) + 8), ALIGN), (dict(state_bytes=100 * 7 * 128 - 1), WORKSPACE), (dict(state=None, ws_bytes=100), WORKSPACE),
    (dict(y=ptr(0)), ALIAS), (dict(y=ptr(3) + 16), ALIAS), (dict(y=ptr(5)), ALIAS), (dict(state=ptr(1)), ALIAS), (dict(state=ptr(2) - 16), ALIAS),
    (dict(state=None, ws=ptr(0)), ALIAS), (dict(state=None, ws=ptr(4)), ALIAS),
]


@pytest.mark.parametrize("change,status", FFN_REFUSED, ids=lambda v: str(v)[:60])
def test_gated_ffn_forward_refusals(change, status):
    assert bm.lib().bmoe_gated_ffn_forward(*dict(FFN, **change).values()) == status
    assert bm.lib().bmoe_last_error() != b""


FFN_BWD_REFUSED = [(c, SHAPE) for c in FFN_SHAPES] + [
    (dict(act=3), DTYPE), (dict(x=None), NULL), (dict(dy=None), NULL), (dict(state=None), NULL), (dict(ws=None), NULL), (dict(w_in=None), NULL),
    (dict(dx=ptr(6) + 8), ALIGN), (dict(dw_in=ptr(7) + 2), ALIGN), (dict(dx_add=ptr(5) + 4), ALIGN), (dict(ws=ptr(9) + 8), ALIGN),
    (dict(state_bytes=100), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE), (dict(dx=ptr(3)), ALIAS), (dict(dx=ptr(5)), ALIAS), (dict(dw_in=ptr(1)), ALIAS),
    (dict(dw_down=ptr(7) + 64), ALIAS), (dict(ws=ptr(4)), ALIAS), (dict(ws=ptr(8)), ALIAS), (dict(dw_down=ptr(0) + 16), ALIAS),
]


@pytest.mark.parametrize("change,status", FFN_BWD_REFUSED, ids=lambda v: str(v)[:60])
def test_gated_ffn_backward_refusals(change, status):
    assert bm.lib().bmoe_gated_ffn_backward(*dict(FFN_BWD, **change).values()) == status


def test_gated_ffn_sizes_and_nothing_to_do():
    L, n = bm.lib(), ctypes.c_size_t(77)
    assert L.bmoe_gated_ffn_forward(*dict(FFN, tokens=0, x=None, y=None).values()) == 0
    assert L.bmoe_gated_ffn_backward(*dict(FFN_BWD, dx=None, dw_in=None, dw_down=None, x=None).values()) == 0
    assert L.bmoe_gated_ffn_state_size(10, 64, ctypes.byref(n)) == 0 and n.value == 10 * 7 * 64
    assert L.bmoe_gated_ffn_state_size(10, 64, None) == NULL and L.bmoe_gated_ffn_state_size(10, 63, ctypes.byref(n)) == SHAPE
    assert L.bmoe_gated_ffn_forward_workspace(10, 64, 64, 2, ctypes.byref(n)) == SHAPE
    # few tokens keep the activated product in fp32, with a state or without
    for tokens in (1, 4):
        for with_state in (0, 1):
            assert L.bmoe_gated_ffn_forward_workspace(tokens, 64, 64, with_state, ctypes.byref(n)) == 0 and n.value == tokens * 256
    for tokens, d, ff in ((1, 8, 8), (33, 2048, 8192), (1 << 20, 2048, 8192), (4096, 16384, 32768)):
        for call in ((L.bmoe_gated_ffn_forward_workspace, (tokens, d, ff, 0)), (L.bmoe_gated_ffn_backward_workspace, (tokens, d, ff))):
            assert call[0](*call[1], ctypes.byref(n)) == 0 and tokens * ff * 2 <= n.value < tokens * ff * 4 + (4 << 30)


def test_refusals_under_host_sanitizers():
    """This file again against the library whose host code is sanitized."""
    rt = bbuild.sanitizer_runtime()
    if os.environ.get("BMOE_LIBRARY"):
        pytest.skip("already running against a chosen library")
    if not os.path.exists(bbuild.LIB_HOSTSAN) or not rt:
        pytest.skip("libbmoe_hostsan.so or the sanitizer runtime is missing (build with the package build)")
    env = dict(os.environ, BMOE_LIBRARY=bbuild.LIB_HOSTSAN, LD_PRELOAD=rt,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1",
               HIP_VISIBLE_DEVICES=os.environ.get("HIP_VISIBLE_DEVICES", ""))
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider", "-k", "not binding",
                        os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = (r.stdout + r.stderr)[-3000:]
    assert r.returncode == 0 and "passed" in r.stdout and "ERROR: AddressSanitizer" not in r.stderr, tail
