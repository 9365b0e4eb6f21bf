"""Layer norm forward and backward (include/bmoe_norm.h) on the GPU against the
fp64 oracle, elementwise.

Bars, with u = 2^-24 and b = finfo(dtype).eps / 2 for the stored outputs: a row
sum adds at most 32 values per thread, then 6 levels over the wave and at most
16 waves, so it is off by at most 54 u sum|.|; every further operation adds u
of its result.  Forward: the mean is off by 54 u mean|s| + u |mean|; a centred
value by the mean's error + u |c|; the variance's first-order dependence on the
mean's error vanishes (centred values sum to 0), so rstd is off by at most
(54 + 3) / 2 + 4 < 40 units u relatively.  Backward, at given mean and rstd:
xhat is off by 2 u |xhat|, each of the two row sums by (54 + 5) u of its sum of
magnitudes.  Column sums add at most rows / 4 values at any one place of the
order (few here), bounded below by their depth.
"""
import numpy as np
import pytest

import compressed_mixture_experts_amd as bm
from oracle import ref
from gpu_helpers import log, to_f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


def draw(rows, width, kind, seed, offset=0.5):
    import torch
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if kind == "bf16" else torch.float32
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (n(rows, width) * torch.exp(0.5 * n(rows, 1)) + offset).to(dt)
    return dict(x=x, r=n(rows, width).to(dt), gamma=1 + 0.3 * n(width), beta=0.3 * n(width), dy=n(rows, width),
                ds=n(rows, width).to(dt), dt=dt)


def half(dt):
    import torch
    return torch.finfo(dt).eps / 2


def check_forward(c, got, gamma, beta, eps, residual):
    y, s, mean, rstd = got
    b = half(c["dt"])
    if residual:
        want = to_f64(c["x"]) + to_f64(c["r"])
        assert (np.abs(to_f64(s) - want) <= (b + 2 * U) * np.abs(want)).all(), "sum"
    s64 = to_f64(s)
    wy, wm, wr = ref.layer_norm(s64, None if gamma is None else to_f64(gamma), None if beta is None else to_f64(beta), eps)
    em = 54 * U * np.abs(s64).mean(axis=1) + U * np.abs(wm)
    if mean is not None:
        assert (np.abs(to_f64(mean) - wm) <= em).all(), "mean"
        assert (np.abs(to_f64(rstd) - wr) <= 40 * U * wr).all(), "rstd"
    ga = 1.0 if gamma is None else np.abs(to_f64(gamma))
    be = 0.0 if beta is None else np.abs(to_f64(beta))
    xh = np.abs(s64 - wm[:, None]) * wr[:, None]
    tol = ga * (em * wr)[:, None] + 44 * U * ga * xh + U * be
    assert (np.abs(to_f64(y) - wy) <= tol + b * (np.abs(wy) + tol)).all(), "y"


def check_backward(c, got, s, dy, gamma, mean, rstd, d_sum):
    dx, dg, db = got
    s64, dy64, m64, r64 = to_f64(s), to_f64(dy), to_f64(mean), to_f64(rstd)
    ga = None if gamma is None else to_f64(gamma)
    ds64 = None if d_sum is None else to_f64(d_sum)
    wx, wg, wb = ref.layer_norm_backward(dy64, s64, ga, m64, r64, ds64)
    xh = np.abs((s64 - m64[:, None]) * r64[:, None])
    v = np.abs(dy64 if ga is None else dy64 * ga)
    mv, mx = v.mean(axis=1, keepdims=True), (v * xh).mean(axis=1, keepdims=True)
    tol = U * r64[:, None] * (6 * v + 64 * mv + 68 * xh * mx) + (0 if ds64 is None else U * np.abs(ds64))
    b = half(c["dt"])
    assert (np.abs(to_f64(dx) - wx) <= tol + b * (np.abs(wx) + tol)).all(), "dx"
    if dg is not None:
        # depth of a column's sum: a wave's rows, the workgroup's waves, the
        # partial rows of one group of the second kernel (64 groups), their sums; or,
        # at up to 1024 rows, a 16th of the rows and 16 sums (a 64th and 64 in a
        # workgroup of 1024)
        rows = dy64.shape[0]
        blocks = max(1, min(512, -(-rows // 4)))
        depth = -(-rows // blocks) + 4 + -(-blocks // 16) + 16
        if rows <= 1024:
            depth = max(depth, -(-rows // 16) + 64)
        assert (np.abs(to_f64(dg) - wg) <= (depth + 4) * U * (np.abs(dy64) * xh).sum(axis=0)).all(), "dgamma"
        assert (np.abs(to_f64(db) - wb) <= (depth + 1) * U * np.abs(dy64).sum(axis=0)).all(), "dbeta"


CASES = [
    # rows, width: every group size and row shape, their edges, odd rows
    (1, 1), (3, 2), (1, 64), (5, 8), (7, 130), (33, 512), (4, 520), (129, 1000), (50, 1024), (9, 1032), (66, 2048),
    (1, 2048), (6, 2056), (5, 4096), (3, 4104), (4, 8192), (2, 16384), (2, 8200),
    (17, 77), (8, 255), (5, 257), (6, 777), (3, 1023), (4, 1025), (2, 4095), (2, 4097), (2, 16383),
    (13, 254), (5, 258), (3, 1022), (3, 1026), (2, 4094), (2, 4098), (2, 16382), (2500, 96), (2301, 33),
    # one launch and two for the columns' sums: at 1024 rows, at 2^21 elements
    (1024, 100), (1025, 100), (1024, 2048), (1000, 2100), (511, 4104), (512, 4098), (128, 16384), (700, 33),
]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,width", CASES)
def test_norm_forward_backward(rows, width, kind):
    log(f"layer norm rows={rows} width={width} {kind}")
    c = draw(rows, width, kind, 1000 * rows + width)
    d = {k: v.cuda() for k, v in c.items() if k != "dt"}
    for residual in (False, True):
        got = bm.layer_norm_forward(d["x"], d["gamma"], d["beta"], eps=1e-5, residual=d["r"] if residual else None)
        check_forward(c, got, d["gamma"], d["beta"], 1e-5, residual)
        y, s, mean, rstd = got
        for dy in {d["dy"], d["dy"].to(c["dt"])}:
            ds = d["ds"] if residual else None
            check_backward(c, bm.layer_norm_backward(dy, s, d["gamma"], mean, rstd, d_sum=ds), s, dy, d["gamma"], mean,
                           rstd, ds)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_norm_without_weights_and_stats(kind):
    c = draw(19, 640, kind, 3)
    x = c["x"].cuda()
    got = bm.layer_norm_forward(x, eps=0.0)
    check_forward(c, got, None, None, 0.0, False)
    y2, s2, m2, r2 = bm.layer_norm_forward(x, eps=0.0, stats=False)
    assert m2 is None and r2 is None and (y2 == got[0]).all() and s2 is x
    dy = c["dy"].cuda()
    dx, dg, db = bm.layer_norm_backward(dy, x, None, got[2], got[3], weight_grads=False)
    assert dg is None and db is None
    check_backward(c, (dx, None, None), x, dy, None, got[2], got[3], None)


@pytest.mark.parametrize("shift", [1, 2, 4])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_norm_unaligned_arrays(kind, shift):
    """Arrays that start `shift` elements past an aligned address give the same
    values as aligned ones up to the order of the sums."""
    import torch
    rows, width = 11, 1024
    c = draw(rows, width, kind, 5)

    def at(t):
        buf = torch.empty(t.numel() + 16, dtype=t.dtype, device="cuda")
        v = buf[shift:shift + t.numel()].view(t.shape)
        v.copy_(t)
        return v
    x, r, ga, be, ds, dy = (at(c[k]) for k in ("x", "r", "gamma", "beta", "ds", "dy"))
    got = bm.layer_norm_forward(x, ga, be, residual=r, y=at(c["x"]), sum_out=at(c["x"]))
    check_forward(c, got, ga, be, 1e-5, True)
    dx = bm.layer_norm_backward(dy, got[1], ga, got[2], got[3], d_sum=ds, dx=at(c["x"]))
    check_backward(c, dx, got[1], dy, ga, got[2], got[3], ds)


def test_norm_in_place():
    c = draw(37, 768, "bf16", 7)
    d = {k: v.cuda() for k, v in c.items() if k != "dt"}
    want = bm.layer_norm_forward(d["x"], d["gamma"], d["beta"], residual=d["r"])
    x, r = d["x"].clone(), d["r"].clone()
    got = bm.layer_norm_forward(x, d["gamma"], d["beta"], residual=r, y=x, sum_out=r)
    assert got[0] is x and got[1] is r
    for a, b in zip(got, want):
        assert (a == b).all()
    dy = d["dy"].bfloat16()
    wdx, wg, wb = bm.layer_norm_backward(dy, want[1], d["gamma"], want[2], want[3], d_sum=d["ds"])
    for name in ("s", "d_sum", "dy"):
        t = {"s": want[1].clone(), "d_sum": d["ds"].clone(), "dy": dy.clone()}
        dx, g, b = bm.layer_norm_backward(t["dy"], t["s"], d["gamma"], want[2], want[3], d_sum=t["d_sum"], dx=t[name])
        assert (dx == wdx).all() and (g == wg).all() and (b == wb).all(), name


@pytest.mark.parametrize("rows,width,kind", [(1024, 2048, "bf16"), (1000, 777, "f32"), (1024, 64, "f32"), (1100, 2048, "bf16"),
                                             (60, 4099, "bf16"), (1200, 1443, "bf16"), (300, 6001, "f32")])
def test_norm_gradient_in_place(rows, width, kind):
    """The columns' sums are those of the inputs, whichever of them dx overwrites."""
    c = draw(rows, width, kind, rows)
    d = {k: v.cuda() for k, v in c.items() if k != "dt"}
    _, s, mean, rstd = bm.layer_norm_forward(d["x"], d["gamma"], d["beta"])
    dy = d["dy"].to(c["dt"])
    want = bm.layer_norm_backward(dy, s, d["gamma"], mean, rstd)
    check_backward(c, want, s, dy, d["gamma"], mean, rstd, None)
    for name in ("s", "dy"):
        for _ in range(4):
            t = {"s": s.clone(), "dy": dy.clone()}
            got = bm.layer_norm_backward(t["dy"], t["s"], d["gamma"], mean, rstd, dx=t[name])
            assert all((a == b).all() for a, b in zip(got, want)), name


@pytest.mark.parametrize("width", [64, 777, 4096])
def test_norm_non_finite_rows_stay_alone(width):
    import torch
    c = draw(12, width, "f32", 8)
    x = c["x"].cuda()
    clean = bm.layer_norm_forward(x)[0].clone()
    x[3, width // 2] = float("nan")
    x[7, 0] = float("inf")
    y, _, mean, rstd = bm.layer_norm_forward(x)
    bad = torch.zeros(12, dtype=torch.bool, device="cuda")
    bad[[3, 7]] = True
    assert torch.isnan(y[bad]).all() and (y[~bad] == clean[~bad]).all()
    dx, dg, db = bm.layer_norm_backward(c["dy"].cuda(), x, None, mean, rstd)
    assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[~bad]).all()
    assert torch.isfinite(db).all() and torch.isnan(dg).any()


def test_norm_constant_row():
    """A constant row has variance 0: y = beta, rstd = eps^-1/2."""
    import torch
    x = torch.full((2, 512), 3.25, device="cuda")
    be = torch.randn(512, device="cuda")
    y, _, mean, rstd = bm.layer_norm_forward(x, None, be, eps=1e-4)
    assert (mean == 3.25).all() and (y == be).all() and torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=40 * U)


def test_norm_no_rows():
    import torch
    x = torch.empty((0, 96), device="cuda")
    y, s, mean, rstd = bm.layer_norm_forward(x)
    assert y.shape == (0, 96) and mean.shape == (0,)
    dx, dg, db = bm.layer_norm_backward(x, x, None, mean, rstd)
    torch.cuda.synchronize()
    assert dx.shape == (0, 96) and (dg == 0).all() and (db == 0).all()


def test_norm_rows_behind_are_left():
    """Nothing past the rows of a call is written."""
    import torch
    c = draw(10, 200, "bf16", 11)
    x = c["x"].cuda()
    y = torch.full((10, 200), 7.0, dtype=torch.bfloat16, device="cuda")
    bm.layer_norm_forward(x[:6], y=y[:6])
    assert (y[6:] == 7.0).all() and (y[:6] == bm.layer_norm_forward(x)[0][:6]).all()


def test_norm_backward_against_differences():
    """A directional derivative of the GPU forward in fp32: L = sum(dy y) along
    (dx', dgamma', dbeta') with step h.  Truncation h^2 |L'''| / 6 and
    cancellation 2 u |L| sqrt(n) / h are both below 1e-3 of the derivative's
    scale at h = 1e-2."""
    import torch
    c = draw(64, 320, "f32", 13)
    d = {k: v.cuda() for k, v in c.items() if k != "dt"}
    y, s, mean, rstd = bm.layer_norm_forward(d["x"], d["gamma"], d["beta"])
    dx, dg, db = bm.layer_norm_backward(d["dy"], s, d["gamma"], mean, rstd)
    g = torch.Generator().manual_seed(14)
    px, pg, pb = (torch.randn(t.shape, generator=g).cuda() for t in (dx, dg, db))
    h = 1e-2

    def loss(k):
        y = bm.layer_norm_forward(d["x"] + k * h * px, d["gamma"] + k * h * pg, d["beta"] + k * h * pb)[0]
        return (d["dy"].double() * y.double()).sum()
    diff = ((loss(1) - loss(-1)) / (2 * h)).item()
    want = ((dx.double() * px).sum() + (dg.double() * pg).sum() + (db.double() * pb).sum()).item()
    scale = max(abs(t) for t in ((dx.double() * px).norm().item(), (dg.double() * pg).norm().item()))
    assert abs(diff - want) <= 1e-2 * scale, (diff, want, scale)


def test_norm_streams_and_graph():
    """Calls on a side stream, and a captured forward and backward replayed on
    new inputs between eager calls."""
    import torch
    c = draw(300, 1024, "bf16", 15)
    d = {k: v.cuda() for k, v in c.items() if k != "dt"}

    def both(x, dy):
        y, s, mean, rstd = bm.layer_norm_forward(x, d["gamma"], d["beta"], residual=d["r"])
        return (y, s, mean, rstd) + tuple(bm.layer_norm_backward(dy, s, d["gamma"], mean, rstd, d_sum=d["ds"]))
    want = both(d["x"], d["dy"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both(d["x"], d["dy"])
        x, dy = d["x"].clone(), d["dy"].clone()
    side.synchronize()
    assert all((a == b).all() for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both(x, dy)
    for k in range(4):
        x.copy_(d["x"] * (k + 1))
        dy.copy_(d["dy"] + k)
        graph.replay()
        torch.cuda.synchronize()
        eager = both(x, dy)
        torch.cuda.synchronize()
        assert all((a == b).all() for a, b in zip(out, eager)), k


def test_norm_many_elements():
    """rows * width past 2^31: the last rows of a 4.3 GB array."""
    import torch
    rows, width = (1 << 31) // 8192 + 3, 8192
    x = torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
    x[:2].normal_()
    x[2:-4] = 0.5
    x[-4:].normal_()
    y, _, mean, rstd = bm.layer_norm_forward(x, y=x.clone())
    tail = bm.layer_norm_forward(x[-4:].clone())
    assert (y[-4:] == tail[0]).all() and (mean[-4:] == tail[2]).all()
    assert (y[5] == 0).all()
    dx, dg, db = bm.layer_norm_backward(y, x, None, mean, rstd, dx=y)
    wx = bm.layer_norm_backward(tail[0], x[-4:].clone(), None, tail[2], tail[3])[0]
    assert (dx[-4:] == wx).all() and torch.isfinite(dg).all()


# widths of every cut and every number of threads per row
WIDTHS = [77, 255, 300, 520, 777, 1000, 1008, 1443, 2000, 2050, 3000, 4099, 6000, 8190, 12000, 12001, 16382]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_constant_rows_are_exact(width, kind):
    """A constant row's centred values are only what its summed mean is off by, at
    most 56 u |value|; centring twice more leaves (57 u)^2 of that, 1e-15 of the
    value, below half a place of it: the mean is the value, y is beta, rstd is
    eps^-1/2 with its own four operations' roundings."""
    import torch
    c = draw(1, width, kind, width)
    values = torch.tensor([96.0, 1000.0, -3000.0, 3.25, 10000.0, 1e-3, 2.0 ** 20]).to(c["dt"])
    x = values[:, None].expand(-1, width).contiguous().cuda()
    y, _, mean, rstd = bm.layer_norm_forward(x, c["gamma"].cuda(), c["beta"].cuda(), eps=1e-5)
    assert (mean.cpu() == values.float()).all(), mean
    assert (np.abs(to_f64(rstd) / float(np.float32(1e-5)) ** -0.5 - 1) <= 4 * U).all(), rstd
    be = to_f64(c["beta"])
    assert (np.abs(to_f64(y) - be) <= 2 * half(c["dt"]) * np.abs(be) + 1e-6).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [30.0, 1e3, 1e5])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_of_rows_far_from_zero(width, offset, kind):
    """Rows that lie `offset` standard deviations from 0.  Centred values are exact
    (both terms of the difference are within a factor 2), what they miss of the true
    mean is known to 57 u of their mean magnitude, which is at most the deviation:
    y is off by 60 u and 46 units of its own, whatever the offset."""
    c = draw(6, width, kind, width, offset=offset)
    d = {k: v.cuda() for k, v in c.items() if k != "dt"}
    for residual in (False, True):
        y, s, mean, rstd = bm.layer_norm_forward(d["x"], d["gamma"], d["beta"], residual=d["r"] if residual else None)
        wy, wm, wr = ref.layer_norm(to_f64(s), to_f64(d["gamma"]), to_f64(d["beta"]), float(np.float32(1e-5)))
        ga, be, b = np.abs(to_f64(d["gamma"])), np.abs(to_f64(d["beta"])), half(c["dt"])
        xh = np.abs((to_f64(s) - wm[:, None]) * wr[:, None])
        tol = ga * U * (60 + 46 * xh) + U * be
        assert (np.abs(to_f64(y) - wy) <= tol + b * (np.abs(wy) + tol)).all(), "y"
        assert (np.abs(to_f64(mean) - wm) <= 1.01 * U * np.abs(wm) + 60 * U / wr).all(), "mean"
        assert (np.abs(to_f64(rstd) - wr) <= 40 * U * wr).all(), "rstd"


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e17, 1e19, 1e25, 1e37])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_of_large_finite_rows(width, size, kind):
    """Rows whose squares, or whose sum, leave fp32: the same bars as for any row,
    powers of two apart nothing is rounded otherwise.  1e37 leaves room for eight
    deviations below 2^127."""
    import torch
    c = draw(5, width, kind, width)
    scale = torch.tensor([1.0, 1.0, 1.0, 1.0, 2.0 ** -60])[:, None]      # the last row is an ordinary one
    z = (torch.randn(5, width, generator=torch.Generator().manual_seed(width)).clamp(-6, 6) + 1.5) * size * scale
    z[2] = c["x"][2].float()
    z[2, width // 2] = size                                              # one entry of a small row
    c = dict(c, x=z.to(c["dt"]), r=c["r"] * size * 0.25)
    d = {k: v.cuda() for k, v in c.items() if k != "dt"}
    for residual in (False, True):
        got = bm.layer_norm_forward(d["x"], d["gamma"], d["beta"], residual=d["r"] if residual else None)
        check_forward(c, got, d["gamma"], d["beta"], 1e-5, residual)
        if size < 1e30:  # gradients that stay above fp32's smallest normal number
            check_backward(c, bm.layer_norm_backward(d["dy"], got[1], d["gamma"], got[2], got[3]), got[1], d["dy"],
                           d["gamma"], got[2], got[3], None)


def test_norm_over_its_input_keeps_no_row():
    """y written over x leaves no s for a backward, so none is returned."""
    import torch
    c = draw(7, 200, "bf16", 17)
    x = c["x"].cuda()
    want = bm.layer_norm_forward(x)
    assert want[1] is x
    z = x.clone()
    got = bm.layer_norm_forward(z, y=z)
    assert got[1] is None and got[0] is z and all((a == b).all() for a, b in zip(got[::2] + got[3:], want[::2] + want[3:]))
    with pytest.raises(ValueError):
        bm.layer_norm_backward(torch.randn(7, 200, device="cuda"), got[1], None, got[2], got[3])
    r = bm.layer_norm_forward(x.clone(), residual=x, y=x)       # a sum of its own is kept
    assert r[1] is not None


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("size,eps", [(1e-15, 0.0), (1e-20, 0.0), (1e-30, 0.0), (1e-20, 1e-40), (1e-20, 1e-5)])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_of_small_rows(width, size, eps, kind):
    """Rows whose squares are below fp32's normal numbers, under an eps that does not
    cover them: the same bars as for any row (entries 1e6 times below the row's
    deviation are still normal numbers)."""
    import torch
    c = draw(5, width, kind, width)
    z = (torch.randn(5, width, generator=torch.Generator().manual_seed(width + 1)) + 0.5) * size
    z[3] = 2.0 * size                                                    # a constant row
    z[4] = c["x"][4].float()                                             # an ordinary one
    x = z.to(c["dt"]).cuda()
    got = bm.layer_norm_forward(x, eps=eps)
    # with eps = 0 a constant row is 0 / 0
    rows = [0, 1, 2, 4] if eps < 1e-30 else [0, 1, 2, 3, 4]
    part = dict(c, x=c["x"][rows])
    e = float(np.float32(eps))
    check_forward(part, [t[rows] for t in got], None, None, e, False)
    dy = c["dy"].cuda()
    grads = bm.layer_norm_backward(dy, x, None, got[2], got[3])
    check_backward(part, (grads[0][rows], None, None), x[rows], dy[rows], None, got[2][rows], got[3][rows], None)
