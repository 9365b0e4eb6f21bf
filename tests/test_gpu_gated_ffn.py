"""The gated feed-forward block (include/bmoe_ffn.h) on the GPU against 64-bit products.

Bars, elementwise, with u = 2^-24 and b = 2^-8 (half a step of bf16): a sum of K products of
bf16 values is off by (K + 64) u times the sum of their magnitudes (every order of fp32
additions, and the matrix cores' own roundings).  The activations' slopes are at most 1.13, so
what g is off by counts 1.13-fold in act(g), which the hardware's exp2 and reciprocal leave off by
8 u of itself and the GELU's tail by 2e-6 |g| + 1e-6 more; act' changes by at most 0.8 of what g
is off by (|act''| <= 0.8) and is off by 2e-6 (1 + |g|) itself.  h, dg and du are rounded to bf16, dg's and
du's factors u act'(g) and act(g) to 12 bits (2^-12 of themselves).  Every later product adds its sum's bar and carries what its operands are off by.

These bars add roundings up as if all had one sign.  They have not: a rounding's root mean
square is b / sqrt(3) of its value at most, so what two of them in a row do to a product of
many terms is 0.82 b relative to it by norm; b is asked of every output beside.
"""
import numpy as np
import pytest

import compressed_mixture_experts_amd as bm
from gpu_helpers import log

pytestmark = pytest.mark.gpu
U, B = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


def draw(tokens, d, ff, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    return dict(x=n(tokens, d).to(bf), w_in=(n(2 * ff, d) / d ** 0.5).to(bf), w_down=(n(d, ff) / ff ** 0.5).to(bf), add=n(tokens, d).to(bf),
                dy=(n(tokens, d) * torch.exp(0.5 * n(tokens, 1))).to(bf), dx_add=n(tokens, d))


def act64(g, act):
    import torch
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    cdf = torch.special.ndtr(g)
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / (2 * np.pi) ** 0.5


def near(name, got, want, off):
    """Elementwise within off plus the stored rounding, and by norm."""
    import torch
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), f"{name} is not finite"
    assert (err <= off + B * (want.abs() + off)).all(), f"{name}: {float((err / (off + B * want.abs())).max())}"
    norm = float(torch.linalg.vector_norm(want))
    if norm > 0:
        assert float(torch.linalg.vector_norm(err)) <= B * norm, f"{name} by norm: {float(torch.linalg.vector_norm(err)) / norm}"


class Want:
    """Everything in 64 bits, and what each may be off by."""

    def __init__(self, c, act):
        x, wi, wd = c["x"].double(), c["w_in"].double(), c["w_down"].double()
        (m, d), ff = x.shape, wd.shape[1]
        self.act, self.x, self.wi, self.wd, self.ff, self.m = act, x, wi, wd, ff, m
        gu = x @ wi.T
        e = (d + 64) * U * (x.abs() @ wi.abs().T)
        self.g, self.u, self.eg, self.eu = gu[:, :ff], gu[:, ff:], e[:, :ff], e[:, ff:]
        self.a, self.slope = act64(self.g, act)
        tail = 0 if act == "silu" else 2e-6 * self.g.abs() + 1e-6
        self.ea = 1.13 * self.eg + 8 * U * self.a.abs() + tail
        self.h = self.a * self.u
        eh = self.ea * self.u.abs() + self.a.abs() * self.eu + self.ea * self.eu + 2 * U * self.h.abs()
        self.eh = eh + B * (self.h.abs() + eh)
        self.y = self.h @ wd.T
        self.ey = self.eh @ wd.abs().T + (ff + 64) * U * (self.h.abs() @ wd.abs().T)

    def backward(self, dy):
        import torch
        dy = dy.double()
        ff, d = self.ff, self.x.shape[1]
        dh = dy @ self.wd
        edh = (d + 64) * U * (dy.abs() @ self.wd.abs())
        # the factors as kept
        es = 0.8 * self.eg + 2e-6 * (1 + self.g.abs())
        f, a = self.u * self.slope, self.a
        ef = self.eu * self.slope.abs() + (self.u.abs() + self.eu) * es + 2 * U * f.abs()
        ef, ea = ef + 2.0 ** -12 * (f.abs() + ef), self.ea + 2.0 ** -12 * (a.abs() + self.ea)
        du, dg = dh * a, dh * f
        edu = (dh.abs() + edh) * ea + edh * a.abs() + 2 * U * du.abs()
        edg = (dh.abs() + edh) * ef + edh * f.abs() + 2 * U * dg.abs()
        dgu, e = torch.cat([dg, du], 1), torch.cat([edg, edu], 1)
        e = e + B * (dgu.abs() + e)
        mag = dgu.abs() + e
        dx = dgu @ self.wi
        dwi, dwd = dgu.T @ self.x, dy.T @ self.h
        return ((dx, e @ self.wi.abs() + (2 * ff + 64) * U * (mag @ self.wi.abs())),
                (dwi, e.T @ self.x.abs() + (self.m + 64) * U * (mag.T @ self.x.abs())),
                (dwd, dy.abs().T @ self.eh + (self.m + 64) * U * (dy.abs().T @ (self.h.abs() + self.eh))))


SHAPES = [
    # few tokens, one by one: depths below and beside whole steps of 512, shared among 1 to 8 waves
    (1, 8, 8), (1, 64, 128), (2, 72, 40), (1, 520, 1032), (3, 512, 4104), (4, 2048, 264), (1, 1000, 16), (4, 8, 3000),
    # the fewest of the others
    (15, 24, 264), (16, 128, 64), (17, 200, 136), (32, 512, 1000), (31, 1024, 2048), (5, 2048, 24),
    # tiles of 64 and 128, ragged in every direction, depths below one step
    (33, 8, 8), (64, 64, 64), (65, 72, 136), (100, 16, 32), (127, 136, 8), (128, 128, 256), (129, 520, 264), (257, 264, 72), (300, 40, 1000),
    (1000, 256, 512), (1001, 512, 1368), (2000, 24, 56), (77, 1024, 2048),
    # tiles of 256
    (4001, 512, 1368), (8197, 264, 1000), (2049, 1024, 4104), (5000, 1032, 2056),
]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,d,ff", SHAPES)
def test_forward_and_backward(tokens, d, ff, act):
    log(f"gated ffn tokens={tokens} d={d} ff={ff} {act}")
    c = draw(tokens, d, ff, tokens + d + ff)
    w = Want(c, act)
    y = bm.gated_ffn_forward(c["x"], c["w_in"], c["w_down"], act)
    near("y", y, w.y, w.ey)
    y2, state = bm.gated_ffn_forward_train(c["x"], c["w_in"], c["w_down"], act, add=c["add"])
    near("y + add", y2, w.y + c["add"].double(), w.ey + 2 * U * (w.y.abs() + c["add"].double().abs()))
    (dx, ex), (dwi, ewi), (dwd, ewd) = w.backward(c["dy"])
    got = bm.gated_ffn_backward(c["x"], c["w_in"], c["w_down"], c["dy"], state, act, dx_add=c["dx_add"])
    add = c["dx_add"].double()
    near("dx", got[0], dx + add, ex + 2 * U * (dx.abs() + add.abs()))
    near("dw_in", got[1], dwi, ewi)
    near("dw_down", got[2], dwd, ewd)
    only = bm.gated_ffn_backward(c["x"], c["w_in"], c["w_down"], c["dy"], state, act, weight_grads=False)
    assert only[1] is None and only[2] is None
    near("dx alone", only[0], dx, ex)
    weights = bm.gated_ffn_backward(c["x"], c["w_in"], c["w_down"], c["dy"], state, act, input_grad=False)
    assert weights[0] is None and (weights[1] == got[1]).all() and (weights[2] == got[2]).all()


def test_gate_closed_and_open():
    """Gates far from 0: act is 0 or the identity there, and everything is exact on small
    whole numbers."""
    import torch
    tokens, d, ff = 70, 32, 64
    r = np.random.default_rng(0)
    x = torch.zeros(tokens, d)
    x[:, 0] = 1.0
    x[:, 1:] = torch.from_numpy(r.integers(-1, 2, (tokens, d - 1)).astype(np.float32)) * (torch.arange(1, d) < 4)
    wi = torch.zeros(2 * ff, d)
    wi[:ff, 0] = torch.where(torch.arange(ff) % 2 == 0, 128.0, -256.0)
    wi[ff:, 1:4] = torch.from_numpy(r.integers(-1, 2, (ff, 3)).astype(np.float32))
    wd = torch.from_numpy(r.integers(-1, 2, (d, ff)).astype(np.float32))
    x, wi, wd = (t.to(torch.bfloat16).cuda() for t in (x, wi, wd))
    u = x.double() @ wi[ff:].double().T
    h = 128.0 * u * (torch.arange(ff, device="cuda") % 2 == 0)
    for act in ("silu", "gelu"):
        for n in (2, 7, tokens):
            y, state = bm.gated_ffn_forward_train(x[:n], wi, wd, act)
            want = h[:n] @ wd.double().T
            assert (y.double() == want.to(torch.bfloat16).double()).all()
            dx, dwi, dwd = bm.gated_ffn_backward(x[:n], wi, wd, x[:n], state, act)
            dh = x[:n].double() @ wd.double()
            on = (torch.arange(ff, device="cuda") % 2 == 0).double()
            dgu = torch.cat([dh * u[:n] * on, dh * 128.0 * on], 1).to(torch.bfloat16).double()
            assert (dwi.double() == (dgu.T @ x[:n].double()).to(torch.bfloat16).double()).all()
            assert (dwd.double() == (x[:n].double().T @ h[:n]).to(torch.bfloat16).double()).all()


def test_bad_rows_stay_alone():
    """NaN and infinity in one token reach its own rows alone, at every tile's edge."""
    import torch
    for tokens in (4, 20, 100, 300):
        c = draw(tokens, 72, 136, 5)
        want, _ = bm.gated_ffn_forward_train(c["x"], c["w_in"], c["w_down"])
        for row, bad in ((0, float("nan")), (tokens - 1, float("inf")), (tokens // 2, float("nan"))):
            x = c["x"].clone()
            x[row, 71] = bad
            y, state = bm.gated_ffn_forward_train(x, c["w_in"], c["w_down"])
            keep = [i for i in range(tokens) if i != row]
            assert (y[keep] == want[keep]).all() and not torch.isfinite(y[row]).all()
            dx, _, _ = bm.gated_ffn_backward(x, c["w_in"], c["w_down"], c["dy"], state)
            assert torch.isfinite(dx[keep]).all() and not torch.isfinite(dx[row]).all()


def test_no_tokens_and_in_place():
    import torch
    c = draw(50, 64, 128, 8)
    z = c["x"][:0]
    y, state = bm.gated_ffn_forward_train(z, c["w_in"], c["w_down"])
    dx, dwi, dwd = bm.gated_ffn_backward(z, c["w_in"], c["w_down"], z, state)
    assert y.shape == dx.shape == (0, 64) and (dwi == 0).all() and (dwd == 0).all()
    for tokens in (3, 9, 50):
        want = bm.gated_ffn_forward(c["x"][:tokens], c["w_in"], c["w_down"], add=c["add"][:tokens])
        add = c["add"][:tokens].clone()
        assert bm.gated_ffn_forward(c["x"][:tokens], c["w_in"], c["w_down"], add=add, y=add) is add and (add == want).all()
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens,d,ff", [(3, 256, 512), (77, 512, 1024), (1000, 256, 1024)])
def test_same_results_every_time_and_captured(tokens, d, ff):
    import torch
    c = draw(tokens, d, ff, 3)

    def step():
        y, state = bm.gated_ffn_forward_train(c["x"], c["w_in"], c["w_down"], "gelu", add=c["add"])
        return (y, state) + bm.gated_ffn_backward(c["x"], c["w_in"], c["w_down"], c["dy"], state, "gelu", dx_add=c["dx_add"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        c["x"].mul_(-1.25)
        c["dy"].mul_(0.5)
        graph.replay()
        want, again = step(), step()
        torch.cuda.synchronize()
        assert all((a == b).all() and (b == d2).all() for a, b, d2 in zip(out, want, again))


def test_binding_refusals():
    import torch
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
    x, wi, wd = z(4, 16), z(64, 16), z(16, 32)
    for args in ((z(4, 16, dtype=torch.float32), wi, wd), (x, z(63, 16), wd), (x, z(64, 8), wd), (x, wi, z(8, 32)), (x, wi, z(16)),
                 (x, wi.cpu(), wd), (x, wi.float(), wd), (z(16, 4).t(), wi, wd), (x.cpu(), wi, wd), (z(4), wi, wd)):
        with pytest.raises(ValueError):
            bm.gated_ffn_forward(*args)
    for kw in (dict(act="relu"), dict(add=z(4, 8)), dict(add=z(4, 16, dtype=torch.float32)), dict(y=z(3, 16))):
        with pytest.raises(ValueError):
            bm.gated_ffn_forward(x, wi, wd, **kw)
    state = z(7 * 4 * 32, dtype=torch.uint8)
    for kw in (dict(dx_add=z(4, 16)), dict(input_grad=False, dx=z(4, 16)), dict(weight_grads=False, dw_in=z(64, 16))):
        with pytest.raises(ValueError):
            bm.gated_ffn_backward(x, wi, wd, x, state, **kw)
    with pytest.raises(ValueError):
        bm.gated_ffn_backward(x, wi, wd, x, state[:-1])
    with pytest.raises(bm.BmoeError, match="SHAPE"):
        bm.gated_ffn_forward(z(4, 12), z(64, 12), z(12, 32))
    with pytest.raises(bm.BmoeError, match="ALIGN"):
        bm.gated_ffn_forward(z(65)[1:].view(4, 16), wi, wd)
    with pytest.raises(bm.BmoeError, match="ALIAS"):
        bm.gated_ffn_forward(x, wi, wd, y=x)
    with pytest.raises(bm.BmoeError, match="ALIAS"):
        bm.gated_ffn_backward(x, wi, wd, x, state, dx=x)


@pytest.mark.parametrize("tokens,d,ff", [(3, 256, 512), (300, 40, 1000), (1000, 256, 512), (4001, 512, 1368), (257, 264, 72)])
def test_each_gradient_alone(tokens, d, ff):
    """The C call with any of dx, dw_in and dw_down left out: the others as with all of them,
    in one launch or in several."""
    import ctypes
    import itertools
    import torch
    c = draw(tokens, d, ff, 21)
    y, state = bm.gated_ffn_forward_train(c["x"], c["w_in"], c["w_down"])
    want = bm.gated_ffn_backward(c["x"], c["w_in"], c["w_down"], y, state)
    n = ctypes.c_size_t(0)
    assert bm.lib().bmoe_gated_ffn_backward_workspace(tokens, d, ff, ctypes.byref(n)) == 0
    for keep in itertools.product((False, True), repeat=3):
        ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
        out = [torch.full_like(w, 7.0) for w in want]
        assert bm.lib().bmoe_gated_ffn_backward(
            tokens, d, ff, 0, c["x"].data_ptr(), c["w_in"].data_ptr(), c["w_down"].data_ptr(), y.data_ptr(), state.data_ptr(),
            state.numel(), None, *[o.data_ptr() if k else None for o, k in zip(out, keep)], ws.data_ptr(), n.value,
            torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        for o, w, k in zip(out, want, keep):
            assert (o == w).all() if k else (o == 7.0).all()
