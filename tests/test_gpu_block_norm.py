"""Norms around a block (include/bmoe_block.h) on the GPU against the fp64 oracle,
elementwise.

Bars, with u = 2^-24 and h = finfo(dtype).eps / 2 for the stored outputs, as for the layer norm
(test_gpu_norm.py): a row sum (16 values a thread at most, 6 levels over the wave, 16 waves)
is off by 54 u sum|.| at most, the mean by that over the width and u |mean|, 1 / deviation by 40 u
relatively, the normed value by 44 u of itself and what the mean is off by.  The product with
scale and gate and the sum with alpha r add 4 u and 2 u of their parts.  Backward at given
statistics: xhat is off by 2 u, a row sum of products by 59 u of its magnitudes, which makes
ds off by e = u rstd (6 |v| + 64 mean|v| + 68 |xhat| mean|v xhat|) + u |d_sum|; through the norm
behind the block e goes like the gradient itself, with its own roundings of the same form.
Column sums are off by their depth (+ 6) u of their magnitudes and by their terms' e.
"""
import numpy as np
import pytest

import compressed_mixture_experts_amd as bm
from oracle import ref
from gpu_helpers import log, to_f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


def half(dt):
    import torch
    return torch.finfo(dt).eps / 2


def draw(rows, width, act, kind, gate, post, seed, offset=0):
    """Inputs on the GPU, each `offset` elements from an aligned place."""
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if act == "bf16" else torch.float32

    def n(*shape, kind=torch.float32, f=lambda x: x):
        count = int(np.prod(shape))
        flat = torch.empty(count + offset, dtype=kind)
        flat[offset:] = f(torch.randn(*shape, generator=g)).reshape(-1).to(kind)
        return flat.cuda()[offset:].view(shape)

    c = dict(b=n(rows, width, kind=dt, f=lambda x: x * torch.exp(0.5 * torch.randn(rows, 1, generator=g)) + 0.5),
             r=n(rows, width, kind=dt, f=lambda x: 2 * x - 0.7), dy=n(rows, width), ds=n(rows, width, kind=dt), dt=dt, kind=kind, post=post,
             gate={"none": None, "channel": n(width, f=lambda x: 0.6 + 0.3 * x), "rows": n(rows, width, kind=dt, f=torch.sigmoid)}[gate],
             ga=n(width, f=lambda x: 1 + 0.3 * x), be=n(width) if kind == "layer" else None, gp=None, bp=None)
    if post:
        c["gp"], c["bp"] = n(width, f=lambda x: 1 + 0.3 * x), n(width) if kind == "layer" else None
    return c


def wide(x):
    return None if x is None else to_f64(x)


def mag(x, otherwise):
    return otherwise if x is None else np.abs(wide(x))


def norm_bar(a, mean, rstd, gamma, beta):
    """What a normed row times gamma plus beta is off by."""
    em = 54 * U * np.abs(a).mean(axis=1) + U * np.abs(mean)
    xh = np.abs(a - mean[:, None]) * rstd[:, None]
    return gamma * ((em * rstd)[:, None] + 44 * U * xh) + U * beta, em


def check_forward(c, got, alpha, scale, residual, eps=EPS):
    y, s, stats = got
    h = half(c["dt"])
    b, r, gate = wide(c["b"]), wide(c["r"]) if residual else None, wide(c["gate"])
    ws, m1, r1 = ref.block_norm(b, r, gate, alpha, scale, c["post"], c["kind"], wide(c["gp"]), wide(c["bp"]), eps)
    sg = np.abs(scale) * (1.0 if gate is None else np.abs(gate))
    part = np.abs(ws - (0 if r is None else alpha * r))
    tol = 4 * U * part + (0 if r is None else 2 * U * np.abs(alpha * r))
    em1 = 0
    if c["post"]:
        tz, em1 = norm_bar(b, m1, r1, mag(c["gp"], 1.0), mag(c["bp"], 0.0))
        tol = tol + sg * tz
    assert (np.abs(to_f64(s) - ws) <= tol + h * (np.abs(ws) + tol)).all(), "s"
    s64 = to_f64(s)
    xh, m2, r2 = ref.row_norm(s64, c["kind"], eps)
    wy = xh * (1.0 if c["ga"] is None else wide(c["ga"])) + (0.0 if c["be"] is None else wide(c["be"]))
    ty, em2 = norm_bar(s64, m2, r2, mag(c["ga"], 1.0), mag(c["be"], 0.0))
    assert (np.abs(to_f64(y) - wy) <= ty + h * (np.abs(wy) + ty)).all(), "y"
    if stats is not None:
        st = to_f64(stats)
        for k, want, off in ((0, m1, em1), (1, r1, 40 * U * r1), (2, m2, em2), (3, r2, 40 * U * r2)):
            assert (np.abs(st[:, k] - want) <= off).all(), f"stats {k}"


def backward_bar(v, xh, rstd, e):
    """Of a norm's backward of v, itself off by e."""
    m = lambda x: x.mean(axis=1, keepdims=True)  # noqa: E731
    return rstd[:, None] * (e + m(e) + xh * m(e * xh) + U * (6 * v + 64 * m(v) + 68 * xh * m(v * xh)))


def check_backward(c, got, s, stats, dy, d_sum, alpha, scale):
    h = half(c["dt"])
    b64, s64, st, dy64, gate = to_f64(c["b"]), to_f64(s), to_f64(stats), to_f64(dy), wide(c["gate"])
    w = ref.block_norm_backward(dy64, b64, s64, st, gate, alpha, scale, c["post"], c["kind"], wide(c["gp"]), wide(c["bp"]), wide(c["ga"]), wide(d_sum))
    shat = np.abs((s64 - st[:, 2:3]) * st[:, 3:4])
    v = np.abs(dy64) * mag(c["ga"], 1.0)
    e = backward_bar(v, shat, st[:, 3], np.zeros_like(v)) + (0 if d_sum is None else U * np.abs(wide(d_sum))) + U * np.abs(w["s"])

    def near(name, off, stored):
        x = to_f64(got[name])
        assert (np.abs(x - w[name]) <= off + (h * (np.abs(w[name]) + off) if stored else 0)).all(), name

    if got["residual"] is not None:
        near("residual", abs(alpha) * e + U * np.abs(w["residual"]), True)
    bhat = np.abs((b64 - st[:, 0:1]) * st[:, 1:2]) if c["post"] else np.abs(b64)
    gp, bp = mag(c["gp"], 1.0), mag(c["bp"], 0.0)
    sg = abs(scale) * (1.0 if gate is None else np.abs(gate))
    ds = np.abs(w["s"])
    v2, e2 = sg * gp * ds, sg * gp * (e + 4 * U * ds)
    near("b", backward_bar(v2, bhat, st[:, 1], e2) if c["post"] else e2 + 2 * U * v2, True)
    if got["gamma"] is None:
        return
    # a thread's rows of a workgroup, its waves, a 16th of the workgroups and 16 sums
    rows = len(b64)
    tpr = 64
    while tpr * 8 < b64.shape[1] and tpr < 512:
        tpr *= 2
    tpr = 1024 if b64.shape[1] > 8192 else tpr
    rpw = 4 if tpr == 64 else 1
    most = 256 if tpr == 1024 else 512 * 256 // max(tpr, 256)
    blocks = max(1, min(most, -(-rows // rpw)))
    depth = -(-rows // (blocks * rpw)) + rpw + -(-blocks // 16) + 16
    col = lambda term, off, by=1.0: by * ((depth + 8) * U * term + off).sum(axis=0)  # noqa: E731
    near("gamma", col(np.abs(dy64) * shat, 0 * shat), False)
    if c["kind"] == "layer":
        near("beta", col(np.abs(dy64), 0 * shat), False)
    if c["post"]:
        near("gamma_post", col(sg * ds * bhat, sg * e * bhat), False)
        if c["kind"] == "layer":
            near("beta_post", col(sg * ds, sg * e), False)
    if gate is not None:
        z = bhat * gp + bp if c["post"] else bhat
        if gate.ndim == 1:
            near("gate", col(abs(scale) * ds * z, abs(scale) * e * z), False)
        else:
            near("gate", abs(scale) * (e + 6 * U * ds) * z, True)


SHAPES = [(1, 1), (3, 2), (1, 64), (5, 8), (7, 130), (33, 512), (4, 520), (129, 1000), (50, 1024), (9, 1032), (66, 2048), (1, 2048), (6, 2056),
          (5, 4096), (3, 4104), (4, 8192), (2, 16384), (2, 8200), (17, 77), (5, 257), (6, 777), (4, 1025), (2, 4097), (2, 8191), (2, 16383),
          (2500, 96), (2301, 33), (3000, 300)]
FORMS = [("layer", "channel", True), ("rms", "rows", True), ("layer", "none", False), ("rms", "channel", False), ("layer", "rows", True),
         ("rms", "none", True)]


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_forward_backward(rows, width, act):
    k = SHAPES.index((rows, width))
    for i, (kind, gate, post) in enumerate(FORMS if rows * width < 30000 else [FORMS[k % 6], FORMS[(k + 1) % 6]]):
        log(f"block norm rows={rows} width={width} {act} {kind} gate={gate} post={post}")
        c = draw(rows, width, act, kind, gate, post, 1000 * rows + width + i)
        kw = dict(gate=c["gate"], alpha=0.9, scale=-1.25, post=post, kind=kind, gamma_post=c["gp"], beta_post=c["bp"], gamma=c["ga"])
        residual = i != 1
        got = bm.block_norm_forward(c["b"], c["r"] if residual else None, beta=c["be"], **kw)
        check_forward(c, got, 0.9, -1.25, residual)
        _, s, stats = got
        for dy in {c["dy"], c["dy"].to(c["dt"])}:
            ds = c["ds"] if i % 2 == 0 else None
            g = bm.block_norm_backward(dy, c["b"], s, stats, d_sum=ds, residual=residual, **kw)
            assert (g["residual"] is None) == (not residual) and (g["gate"] is None) == (gate == "none")
            assert (g["beta"] is None) == (kind == "rms") and (g["gamma_post"] is None) == (not post)
            check_backward(c, g, s, stats, dy, ds, 0.9, -1.25)


@pytest.mark.parametrize("act", ["bf16", "f32"])
@pytest.mark.parametrize("width", [64, 512, 2048, 5000])
def test_unaligned_and_without_weights(width, act):
    c = draw(5, width, act, "layer", "channel", True, width, offset=1)
    kw = dict(gate=c["gate"], alpha=1.0, scale=1.0, gamma_post=c["gp"], beta_post=c["bp"], gamma=c["ga"])
    got = bm.block_norm_forward(c["b"], c["r"], beta=c["be"], **kw)
    check_forward(c, got, 1.0, 1.0, True)
    check_backward(c, bm.block_norm_backward(c["dy"], c["b"], got[1], got[2], d_sum=c["ds"], **kw), got[1], got[2], c["dy"], c["ds"], 1.0, 1.0)
    c.update(gp=None, bp=None, ga=None, be=None, gate=None)
    got = bm.block_norm_forward(c["b"], c["r"])
    check_forward(c, got, 1.0, 1.0, True)
    check_backward(c, bm.block_norm_backward(c["dy"], c["b"], got[1], got[2]), got[1], got[2], c["dy"], None, 1.0, 1.0)


def test_a_first_norm_of_a_model():
    """Without block norm, residual and gate the forward is a plain RMS norm."""
    c = draw(11, 640, "bf16", "rms", "none", False, 3)
    y, s, stats = bm.block_norm_forward(c["b"], post=False, kind="rms", gamma=c["ga"])
    assert (s == c["b"]).all()
    check_forward(c, (y, s, stats), 1.0, 1.0, False)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("width", [200, 3000])
def test_rows_of_any_size(width, kind):
    """Rows whose squares leave fp32 or vanish in it, constant rows, and rows far from 0."""
    import torch
    c = draw(8, width, "f32", kind, "none", True, width)
    r = np.random.default_rng(width)
    size = np.array([1e30, 1e-30, 1e19, 1e-24, 1.0, 1.0, 1e25, 3e-22])[:, None]
    b = (r.standard_normal((8, width)) * size).astype(np.float32)
    b[4] = 7.25
    b[5] = 1000 + 1e-3 * r.standard_normal(width)
    c["b"] = torch.from_numpy(b).cuda()
    for eps in (0.0, 1e-5):
        got = bm.block_norm_forward(c["b"], c["r"], post=True, kind=kind, gamma_post=c["gp"], beta_post=c["bp"], gamma=c["ga"], beta=c["be"], eps=eps)
        keep = [i for i in range(8) if not (kind == "layer" and i == 4 and eps == 0.0)]   # 0 / 0
        sub = dict(c, b=c["b"][keep], r=c["r"][keep])
        check_forward(sub, tuple(x[keep] for x in got), 1.0, 1.0, True, eps)


@pytest.mark.parametrize("width", [20, 200, 500, 777, 1024, 2049])
def test_a_row_does_not_depend_on_its_neighbours(width):
    """Rows of all sizes beside each other, and the same rows in another order."""
    import torch
    c = draw(4500, width, "f32", "layer", "rows", True, width)
    r = np.random.default_rng(width)
    size = np.array([1.0, 1e30, 1.0, 1e-30, 1e19, 1.0, 1e-24])[r.integers(0, 7, 4500)].astype(np.float32)
    c["b"] *= torch.from_numpy(size).cuda()[:, None]
    c["b"][::13] += 1e3
    c["b"][::101, width // 2] = float("nan")
    turn = torch.from_numpy(r.permutation(4500)).cuda()
    for kind in ("layer", "rms"):
        kw = dict(kind=kind, gamma_post=c["gp"], gamma=c["ga"], eps=0.0)
        got = bm.block_norm_forward(c["b"], c["r"], gate=c["gate"], **kw)
        again = bm.block_norm_forward(c["b"][turn], c["r"][turn], gate=c["gate"][turn], **kw)
        one = bm.block_norm_backward(c["dy"], c["b"], got[1], got[2], gate=c["gate"], d_sum=c["ds"], weight_grads=False, **{k: v for k, v in kw.items() if k != "eps"})
        two = bm.block_norm_backward(c["dy"][turn], c["b"][turn], again[1], again[2], gate=c["gate"][turn], d_sum=c["ds"][turn], weight_grads=False,
                                     **{k: v for k, v in kw.items() if k != "eps"})
        for x, y in list(zip(got, again)) + [(one[k], two[k]) for k in ("b", "residual")]:
            assert torch.equal(x[turn].view(torch.int32), y.view(torch.int32)) or torch.equal(x[turn].nan_to_num(7.0), y.nan_to_num(7.0))


def test_bad_rows_stay_alone_and_no_rows():
    import torch
    c = draw(6, 300, "bf16", "layer", "channel", True, 9)
    kw = dict(gate=c["gate"], gamma_post=c["gp"], beta_post=c["bp"], gamma=c["ga"], beta=c["be"])
    want = bm.block_norm_forward(c["b"], c["r"], **kw)
    c["b"][2, 5], c["r"][4, 299] = float("nan"), float("inf")
    got = bm.block_norm_forward(c["b"], c["r"], **kw)
    ok = [0, 1, 3, 5]
    for x, y in zip(got, want):
        assert (x[ok] == y[ok]).all()
    assert torch.isnan(got[0][[2, 4]]).all() and torch.isnan(got[1][2]).all()
    z = torch.zeros(0, 300, device="cuda")
    y, s, st = bm.block_norm_forward(z, z, gamma=c["ga"])
    g = bm.block_norm_backward(z, z, s, st, gamma=c["ga"], gate=c["gate"])
    assert y.shape == (0, 300) and all((g[k] == 0).all() and g[k].shape == (300,) for k in ("gamma", "beta", "gamma_post", "beta_post", "gate"))


def test_in_place_and_without_weight_gradients():
    import torch
    for act in ("bf16", "f32"):
        c = draw(70, 1000, act, "layer", "channel", True, 15)
        kw = dict(gate=c["gate"], alpha=0.5, gamma_post=c["gp"], beta_post=c["bp"], gamma=c["ga"])
        y, s, st = bm.block_norm_forward(c["b"], c["r"], beta=c["be"], **kw)
        b, r = c["b"].clone(), c["r"].clone()
        y2, s2, _ = bm.block_norm_forward(b, r, beta=c["be"], s_out=r, y=b, stats=False, **kw)
        assert y2 is b and s2 is r and (b == y).all() and (r == s).all()
        dy = c["dy"].to(c["dt"])
        want = bm.block_norm_backward(dy, c["b"], s, st, d_sum=c["ds"], **kw)
        b, s2 = c["b"].clone(), s.clone()
        got = bm.block_norm_backward(dy, b, s2, st, d_sum=c["ds"], db=s2, dr=b, weight_grads=False, **kw)
        assert got["gamma"] is None and got["gate"] is None and (s2 == want["b"]).all() and (b == want["residual"]).all()
        d2, e2 = dy.clone(), c["ds"].clone()
        got = bm.block_norm_backward(d2, c["b"], s, st, d_sum=e2, db=d2, dr=e2, **kw)
        assert (d2 == want["b"]).all() and (e2 == want["residual"]).all()
        assert all((got[k] == want[k]).all() for k in ("gate", "gamma", "beta", "gamma_post", "beta_post"))
    torch.cuda.synchronize()


def test_captured_with_its_backward():
    import torch
    c = draw(1500, 512, "bf16", "layer", "rows", True, 20)
    kw = dict(gate=c["gate"], gamma_post=c["gp"], beta_post=c["bp"], gamma=c["ga"])

    def step():
        y, s, st = bm.block_norm_forward(c["b"], c["r"], beta=c["be"], **kw)
        g = bm.block_norm_backward(c["dy"], c["b"], s, st, d_sum=c["ds"], **kw)
        return [y, s, st] + [g[k] for k in ("b", "residual", "gate", "gamma", "beta", "gamma_post", "beta_post")]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        c["b"].mul_(-1.5)
        c["dy"].mul_(0.5)
        graph.replay()
        want = step()
        torch.cuda.synchronize()
        assert all((a == b).all() for a, b in zip(out, want))


def test_binding_refusals():
    import torch
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    b = z(4, 16)
    for kw in (dict(kind="batch"), dict(gate=z(15)), dict(gate=z(4, 16, dtype=torch.bfloat16)), dict(gate=z(16, dtype=torch.bfloat16)), dict(gate=z(1, 16)),
               dict(gamma=z(16, dtype=torch.float64)), dict(gamma_post=torch.ones(16)), dict(residual=z(4, 15)),
               dict(residual=z(4, 16, dtype=torch.bfloat16)), dict(residual=z(16, 4).t()), dict(s_out=z(4, 17)), dict(y=z(2, 16))):
        with pytest.raises(ValueError):
            bm.block_norm_forward(b, **kw)
    for kw in (dict(kind="rms", beta=z(16)), dict(kind="rms", beta_post=z(16)), dict(post=False, gamma_post=z(16)), dict(eps=-1.0), dict(alpha=float("inf")),
               dict(scale=float("nan")), dict(y=b, s_out=b)):
        with pytest.raises(bm.BmoeError):
            bm.block_norm_forward(b, **kw)
    st = z(4, 4)
    for args, kw in (((b, b, b, z(4, 3)), {}), ((b, b, z(4, 15), st), {}), ((b.half(), b, b, st), {}), ((b, z(16), b, st), {}), ((b[0], b, b, st), {}),
                     ((b, b, b, st), dict(d_sum=z(4, 16, dtype=torch.bfloat16))), ((b, b, b, st), dict(residual=False, dr=z(4, 16))),
                     ((b, b.cpu(), b, st), {})):
        with pytest.raises(ValueError):
            bm.block_norm_backward(*args, **kw)
    d = z(4, 16)
    with pytest.raises(bm.BmoeError, match="ALIAS"):
        bm.block_norm_backward(b, z(4, 16), z(4, 16), st, db=d, dr=d)
