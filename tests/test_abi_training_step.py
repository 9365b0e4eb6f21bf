"""Argument errors of the training-step operators (include/bmoe_norm.h,
include/bmoe_update.h): each is found on the host before anything is enqueued,
so the pointers here are never followed.  No GPU needed."""
import ctypes
import os
import subprocess
import sys

import pytest

import compressed_mixture_experts_amd as bm
from compressed_mixture_experts_amd import build as bbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHAPE, DTYPE, NULL, ALIGN, ALIAS, WORKSPACE = 2, 3, 1, 4, 5, 6
MB = 1 << 20
BIG = 1 << 40


def ptr(k):
    """Made-up address of array k, far from every other one."""
    return (k + 1) * 64 * MB


FWD = dict(rows=8, width=64, dtype=0, x=ptr(0), residual=ptr(1), gamma=ptr(2), beta=ptr(3), eps=1e-5, sum=ptr(4),
           y=ptr(5), mean=ptr(6), rstd=ptr(7), stream=None)
BWD = dict(rows=2000, width=64, dtype=0, dy_dtype=0, dy=ptr(0), s=ptr(1), gamma=ptr(2), mean=ptr(3), rstd=ptr(4),
           d_sum=ptr(5), dx=ptr(6), dgamma=ptr(7), dbeta=ptr(8), ws=ptr(9), ws_bytes=BIG, stream=None)
ORTHO = dict(rows=40, cols=72, dtype=0, grad=ptr(0), momentum=ptr(1), momentum_out=ptr(2), mu=0.9, nesterov=1, out=ptr(3),
             ws=ptr(4), ws_bytes=BIG, stream=None)
STEP = dict(rows=2000, cols=64, w=ptr(0), o=ptr(1), step=0.1, decay=0.0, w_out=ptr(2), packed=ptr(3), scale=ptr(4),
            ws=ptr(5), ws_bytes=BIG, stream=None)
CALLS = {"bmoe_layer_norm_forward": FWD, "bmoe_layer_norm_backward": BWD, "bmoe_orthogonalize": ORTHO,
         "bmoe_substrate_step": STEP}

REFUSED = [
    ("bmoe_layer_norm_forward", dict(rows=-1), SHAPE), ("bmoe_layer_norm_forward", dict(rows=(1 << 24) + 1), SHAPE),
    ("bmoe_layer_norm_forward", dict(width=0), SHAPE), ("bmoe_layer_norm_forward", dict(width=16385), SHAPE),
    ("bmoe_layer_norm_forward", dict(eps=-1e-5), SHAPE), ("bmoe_layer_norm_forward", dict(eps=float("nan")), SHAPE),
    ("bmoe_layer_norm_forward", dict(eps=float("inf")), SHAPE), ("bmoe_layer_norm_forward", dict(dtype=2), DTYPE),
    ("bmoe_layer_norm_forward", dict(x=None), NULL), ("bmoe_layer_norm_forward", dict(y=None), NULL),
    ("bmoe_layer_norm_forward", dict(sum=None), NULL), ("bmoe_layer_norm_forward", dict(residual=None), NULL),
    ("bmoe_layer_norm_forward", dict(mean=None), NULL), ("bmoe_layer_norm_forward", dict(rstd=None), NULL),
    ("bmoe_layer_norm_forward", dict(x=ptr(0) + 2), ALIGN), ("bmoe_layer_norm_forward", dict(y=ptr(5) + 1), ALIGN),
    ("bmoe_layer_norm_forward", dict(gamma=ptr(2) + 2), ALIGN), ("bmoe_layer_norm_forward", dict(rstd=ptr(7) + 1), ALIGN),
    ("bmoe_layer_norm_forward", dict(y=ptr(0) + 4), ALIAS), ("bmoe_layer_norm_forward", dict(y=ptr(4)), ALIAS),
    ("bmoe_layer_norm_forward", dict(y=ptr(2)), ALIAS), ("bmoe_layer_norm_forward", dict(sum=ptr(1) - 4), ALIAS),
    ("bmoe_layer_norm_forward", dict(sum=ptr(3)), ALIAS), ("bmoe_layer_norm_forward", dict(mean=ptr(0)), ALIAS),
    ("bmoe_layer_norm_forward", dict(mean=ptr(7)), ALIAS), ("bmoe_layer_norm_forward", dict(rstd=ptr(5)), ALIAS),
    ("bmoe_layer_norm_backward", dict(rows=-1), SHAPE), ("bmoe_layer_norm_backward", dict(width=0), SHAPE),
    ("bmoe_layer_norm_backward", dict(width=16385), SHAPE), ("bmoe_layer_norm_backward", dict(dtype=7), DTYPE),
    ("bmoe_layer_norm_backward", dict(dy_dtype=1), DTYPE), ("bmoe_layer_norm_backward", dict(dy_dtype=2), DTYPE),
    ("bmoe_layer_norm_backward", dict(dy=None), NULL), ("bmoe_layer_norm_backward", dict(s=None), NULL),
    ("bmoe_layer_norm_backward", dict(mean=None), NULL), ("bmoe_layer_norm_backward", dict(rstd=None), NULL),
    ("bmoe_layer_norm_backward", dict(dx=None), NULL), ("bmoe_layer_norm_backward", dict(dgamma=None), NULL),
    ("bmoe_layer_norm_backward", dict(dbeta=None), NULL), ("bmoe_layer_norm_backward", dict(ws=None), NULL),
    ("bmoe_layer_norm_backward", dict(dx=ptr(6) + 2), ALIGN), ("bmoe_layer_norm_backward", dict(ws=ptr(9) + 8), ALIGN),
    ("bmoe_layer_norm_backward", dict(dgamma=ptr(7) + 1), ALIGN), ("bmoe_layer_norm_backward", dict(ws_bytes=0), WORKSPACE),
    ("bmoe_layer_norm_backward", dict(dx=ptr(1) + 4), ALIAS), ("bmoe_layer_norm_backward", dict(dx=ptr(2)), ALIAS),
    ("bmoe_layer_norm_backward", dict(dx=ptr(9)), ALIAS), ("bmoe_layer_norm_backward", dict(dgamma=ptr(8)), ALIAS),
    ("bmoe_layer_norm_backward", dict(dgamma=ptr(0)), ALIAS), ("bmoe_layer_norm_backward", dict(dbeta=ptr(3)), ALIAS),
    ("bmoe_layer_norm_backward", dict(ws=ptr(5)), ALIAS),
    # a bf16 row gradient over an fp32 dy of the same address is not in place
    ("bmoe_layer_norm_backward", dict(dtype=1, dx=ptr(0)), ALIAS),
    ("bmoe_orthogonalize", dict(rows=0), SHAPE), ("bmoe_orthogonalize", dict(cols=0), SHAPE),
    ("bmoe_orthogonalize", dict(rows=16385), SHAPE), ("bmoe_orthogonalize", dict(cols=16385), SHAPE),
    ("bmoe_orthogonalize", dict(mu=-0.1), SHAPE), ("bmoe_orthogonalize", dict(mu=1.1), SHAPE),
    ("bmoe_orthogonalize", dict(mu=float("nan")), SHAPE), ("bmoe_orthogonalize", dict(nesterov=2), SHAPE),
    ("bmoe_orthogonalize", dict(dtype=3), DTYPE), ("bmoe_orthogonalize", dict(grad=None), NULL),
    ("bmoe_orthogonalize", dict(out=None), NULL), ("bmoe_orthogonalize", dict(ws=None), NULL),
    ("bmoe_orthogonalize", dict(momentum=None), NULL), ("bmoe_orthogonalize", dict(momentum_out=None), NULL),
    ("bmoe_orthogonalize", dict(grad=ptr(0) + 2), ALIGN), ("bmoe_orthogonalize", dict(out=ptr(3) + 1), ALIGN),
    ("bmoe_orthogonalize", dict(ws=ptr(4) + 128), ALIGN), ("bmoe_orthogonalize", dict(ws_bytes=1024), WORKSPACE),
    ("bmoe_orthogonalize", dict(momentum_out=ptr(1) + 4), ALIAS), ("bmoe_orthogonalize", dict(momentum_out=ptr(0)), ALIAS),
    ("bmoe_orthogonalize", dict(out=ptr(0)), ALIAS), ("bmoe_orthogonalize", dict(out=ptr(1)), ALIAS),
    ("bmoe_orthogonalize", dict(ws=ptr(0)), ALIAS), ("bmoe_orthogonalize", dict(ws=ptr(3) - 256), ALIAS),
    ("bmoe_substrate_step", dict(rows=0), SHAPE), ("bmoe_substrate_step", dict(cols=0), SHAPE),
    ("bmoe_substrate_step", dict(cols=24), SHAPE), ("bmoe_substrate_step", dict(rows=1 << 16, cols=1 << 15), SHAPE),
    ("bmoe_substrate_step", dict(step=float("inf")), SHAPE), ("bmoe_substrate_step", dict(decay=float("nan")), SHAPE),
    ("bmoe_substrate_step", dict(w=None), NULL), ("bmoe_substrate_step", dict(packed=None), NULL),
    ("bmoe_substrate_step", dict(ws=None), NULL), ("bmoe_substrate_step", dict(o=None), NULL),
    ("bmoe_substrate_step", dict(w_out=None), NULL), ("bmoe_substrate_step", dict(w=ptr(0) + 4), ALIGN),
    ("bmoe_substrate_step", dict(o=ptr(1) + 8), ALIGN), ("bmoe_substrate_step", dict(packed=ptr(3) + 4), ALIGN),
    ("bmoe_substrate_step", dict(scale=ptr(4) + 2), ALIGN), ("bmoe_substrate_step", dict(ws=ptr(5) + 8), ALIGN),
    ("bmoe_substrate_step", dict(ws_bytes=0), WORKSPACE), ("bmoe_substrate_step", dict(w_out=ptr(0) + 16), ALIAS),
    ("bmoe_substrate_step", dict(w_out=ptr(1)), ALIAS), ("bmoe_substrate_step", dict(packed=ptr(0)), ALIAS),
    ("bmoe_substrate_step", dict(scale=ptr(3)), ALIAS), ("bmoe_substrate_step", dict(ws=ptr(1)), ALIAS),
]


@pytest.mark.parametrize("name,change,status", REFUSED, ids=lambda v: str(v)[:60])
def test_refusals(name, change, status):
    args = dict(CALLS[name], **change)
    assert getattr(bm.lib(), name)(*args.values()) == status
    assert bm.lib().bmoe_last_error() != b""


SIZES = [("bmoe_layer_norm_backward_workspace", (-1, 8)), ("bmoe_layer_norm_backward_workspace", (8, 0)),
         ("bmoe_orthogonalize_workspace", (0, 8)), ("bmoe_orthogonalize_workspace", (8, 1 << 20)),
         ("bmoe_substrate_step_workspace", (4, 20)), ("bmoe_substrate_step_workspace", (-4, 16))]


@pytest.mark.parametrize("name,shape", SIZES)
def test_workspace_sizes(name, shape):
    n = ctypes.c_size_t(77)
    assert getattr(bm.lib(), name)(*shape, ctypes.byref(n)) == SHAPE and n.value == 77
    assert getattr(bm.lib(), name)(64, 64, None) == NULL
    assert getattr(bm.lib(), name)(2000, 64, ctypes.byref(n)) == 0 and 0 < n.value < 64 * MB


def test_few_rows_and_weights_need_no_workspace():
    n = ctypes.c_size_t(77)
    for rows, cols, none in ((1, 16, True), (256, 64, True), (257, 64, False)):
        assert bm.lib().bmoe_substrate_step_workspace(rows, cols, ctypes.byref(n)) == 0 and (n.value == 0) == none
    for rows, width, none in ((0, 64, True), (1024, 2048, True), (1025, 8, False), (1024, 2049, False)):
        assert bm.lib().bmoe_layer_norm_backward_workspace(rows, width, ctypes.byref(n)) == 0 and (n.value == 0) == none


def test_nothing_to_do():
    """No rows and no weight gradients: nothing is launched, no GPU is needed."""
    L = bm.lib()
    assert L.bmoe_layer_norm_forward(*dict(FWD, rows=0, x=None, y=None).values()) == 0
    assert L.bmoe_layer_norm_backward(*dict(BWD, rows=0, dgamma=None, dbeta=None, dy=None, dx=None).values()) == 0


def test_binding_refuses_cpu_and_misfit_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 32)
    for call in (lambda: bm.layer_norm_forward(x), lambda: bm.layer_norm_backward(x, x, None, x[:, 0], x[:, 0]),
                 lambda: bm.orthogonalize(x), lambda: bm.substrate_step(x), lambda: bm.layer_norm_forward(x=x)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    # the checks behind the device check, on CPU tensors
    with pytest.raises(ValueError, match="GPU tensor"):
        bm._operand("t", x, x.shape, (torch.float32,), x.device)


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


def test_layer_scale():
    """The factor of a substrate's codes, and what is refused for one."""
    torch = pytest.importorskip("torch")
    z = torch.zeros
    layer = bm.Layer(d_model=64, d_ff=0, n_experts=2, top_k=1, act="f32", ffn_act="none", renorm_gates=False,
                     w_gate=z(2, 64), w_base_packed=[z(64, 4, dtype=torch.int32)], theta=[z(2, 6, 32)], phi=[z(2, 6, 32)],
                     w_scale=[1.0])
    assert layer.set_scale(0, 0.25) is layer and layer.struct.w_scale[0] == 0.25
    layer.set_scale(0, torch.tensor(0.5))
    for m, scale in ((1, 1.0), (-1, 1.0), (0, float("nan")), (0, float("inf")), (0, 1e39), (0, torch.tensor(float("-inf")))):
        with pytest.raises(ValueError):
            layer.set_scale(m, scale)
    assert layer.struct.w_scale[0] == 0.5
