"""Weight gradients of the norms around a block (include/bmoe_block.h) where the backward's
workgroups go on to further rows, in every number of threads a row, against the fp64
oracle.

Bars as in test_gpu_block_norm.py, but for the column sums, whose depth is that of the
launch (block_norm_plan.py): off by depth + 8 u of their magnitudes (8: a term's own roundings and
the total's factors) and by their terms' e.  A row that is left out or counted twice in a sum of
n rows changes it by some 1 / sqrt(n) of its size or more, 1e-2 here, where the bar is
1e-5 of the magnitudes' sum.
"""
import pytest

import compressed_mixture_experts_amd as bm
from block_norm_plan import column_depth
from oracle import ref
from gpu_helpers import log, to_f64
from test_gpu_block_norm import FORMS, U, backward_bar, check_forward, draw, mag, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


def check_sums(c, got, s, stats, dy, d_sum, alpha, scale):
    b64, s64, st, dy64, gate = to_f64(c["b"]), to_f64(s), to_f64(stats), to_f64(dy), wide(c["gate"])
    w = ref.block_norm_backward(dy64, b64, s64, st, gate, alpha, scale, c["post"], c["kind"], wide(c["gp"]), wide(c["bp"]), wide(c["ga"]), wide(d_sum))
    shat = abs((s64 - st[:, 2:3]) * st[:, 3:4])
    v = abs(dy64) * mag(c["ga"], 1.0)
    e = backward_bar(v, shat, st[:, 3], 0 * v) + (0 if d_sum is None else U * abs(wide(d_sum))) + U * abs(w["s"])
    ds, bhat = abs(w["s"]), abs((b64 - st[:, 0:1]) * st[:, 1:2]) if c["post"] else abs(b64)
    gp, bp = mag(c["gp"], 1.0), mag(c["bp"], 0.0)
    sg = abs(scale) * (1.0 if gate is None else abs(gate))
    depth = column_depth(*b64.shape)

    def near(name, term, off):
        bar = ((depth + 8) * U * term + off).sum(axis=0)
        assert (abs(to_f64(got[name]) - w[name]) <= bar).all(), name

    near("gamma", abs(dy64) * shat, 0 * shat)
    if c["kind"] == "layer":
        near("beta", abs(dy64), 0 * shat)
    if c["post"]:
        near("gamma_post", sg * ds * bhat, sg * e * bhat)
        if c["kind"] == "layer":
            near("beta_post", sg * ds, sg * e)
    if gate is not None and gate.ndim == 1:
        z = bhat * gp + bp if c["post"] else bhat
        near("gate", abs(scale) * ds * z, abs(scale) * e * z)


SHAPES = [
    # several rows of a workgroup at a time: below 8 columns, 16, 32, 64 and 128 threads a row
    (13001, 5), (13003, 33), (25009, 128), (7001, 129), (7003, 256), (4001, 300), (3700, 512), (2000, 520), (1801, 1000),
    # one: 256 and 512 threads, two groups of columns a thread, two of the sums in LDS
    (131, 2048), (515, 1032), (1100, 2048), (3701, 1111), (300, 2056), (131, 4096), (600, 3001), (300, 4104), (301, 8191), (131, 8192),
    (300, 8200), (300, 16384), (529, 9001),
    # as many workgroups as there are, and a row or one more
    (256, 8200), (257, 8200), (12288, 100), (12289, 100), (128, 2048), (129, 2048),
    # few rows of the older tests, at the depth that they have
    (2500, 96), (2301, 33), (1, 64),
]


@pytest.mark.parametrize("rows,width", SHAPES)
def test_weight_gradients(rows, width):
    k = SHAPES.index((rows, width))
    for i in range(2 if rows * width > 1 << 20 else 3):
        (kind, gate, post), act = FORMS[(k + i) % 6], ("bf16", "f32")[(k + i) % 2]
        log(f"block norm rows={rows} width={width} {act} {kind} gate={gate} post={post}")
        c = draw(rows, width, act, kind, gate, post, 7 * rows + width + i)
        kw = dict(gate=c["gate"], alpha=0.9, scale=-1.25, post=post, kind=kind, gamma_post=c["gp"], beta_post=c["bp"], gamma=c["ga"])
        got = bm.block_norm_forward(c["b"], c["r"], beta=c["be"], **kw)
        check_forward(c, got, 0.9, -1.25, True)
        ds = c["ds"] if i % 2 == 0 else None
        for dy in {c["dy"], c["dy"].to(c["dt"])}:
            g = bm.block_norm_backward(dy, c["b"], got[1], got[2], d_sum=ds, **kw)
            check_sums(c, g, got[1], got[2], dy, ds, 0.9, -1.25)
            # rows' gradients do not depend on how many rows a workgroup has
            one = bm.block_norm_backward(dy[-2:].contiguous(), c["b"][-2:].contiguous(), got[1][-2:].contiguous(), got[2][-2:].contiguous(),
                                         d_sum=None if ds is None else ds[-2:].contiguous(),
                                         **dict(kw, gate=c["gate"][-2:].contiguous() if gate == "rows" else c["gate"]))
            for name in ("b", "residual") + (("gate",) if gate == "rows" else ()):
                assert (g[name][-2:] == one[name]).all(), name


def test_every_row_counts_once():
    """One row alone has a gradient that is not 0, wherever it is: the sums are that row's."""
    import torch
    for rows, width in ((1100, 2048), (4001, 300), (300, 8200), (300, 4104)):
        c = draw(rows, width, "f32", "layer", "channel", True, rows)
        kw = dict(gate=c["gate"], gamma_post=c["gp"], beta_post=c["bp"], gamma=c["ga"])
        y, s, st = bm.block_norm_forward(c["b"], c["r"], beta=c["be"], **kw)
        zero = torch.zeros(rows, width, device="cuda")
        for row in (0, 1, rows // 2, rows - 2, rows - 1):
            dy = zero.clone()
            dy[row] = c["dy"][row]
            g = bm.block_norm_backward(dy, c["b"], s, st, **kw)
            sub = bm.block_norm_backward(dy[row:row + 1].contiguous(), c["b"][row:row + 1].contiguous(), s[row:row + 1].contiguous(), st[row:row + 1].contiguous(), **kw)
            for name in ("gamma", "beta", "gamma_post", "beta_post", "gate"):
                assert torch.equal(g[name], sub[name]), (name, row)
