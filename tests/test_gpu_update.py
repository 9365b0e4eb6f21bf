"""Orthogonalised updates and the substrate step (include/bmoe_update.h) on the
GPU against the fp64 oracle, and a whole training step of a normalised layer.

Bars for the orthogonalised update, relative Frobenius norm.  A rounding to
fp16 is off by at most 2^-11, 2^-12 in the mean square.  The map of one step
stretches a change of a settled singular value by at most 4 and what lies
outside the gradient's row space by a = 3.44.  About ten roundings (A, P, T, Q,
X of the five steps) act on settled values: sqrt(10) * 4 * 2^-12 = 3.1e-3 for a
gradient whose row space is full; the rounding of X_3 to one term grows
a^2 = 11.8-fold outside a smaller row space and ||X_3|| / ||X_5|| is at most
1.2 / 0.68: 11.8 * 1.8 * 2^-11 = 1.0e-2 more.  bf16 adds 2^-8 at most.  Bars:
7e-3 (full rank), 1.7e-2 (any).
"""
import numpy as np
import pytest

import compressed_mixture_experts_amd as bm
from compressed_mixture_experts_amd import workloads as wl
from oracle import ref
from gpu_helpers import log, to_dev, to_f64

pytestmark = pytest.mark.gpu
FULL, ANY = 7e-3, 1.7e-2


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


def matrix(kind, rows, cols, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    k = min(rows, cols)
    if kind == "normal":
        return n(rows, cols)
    if kind == "rows":  # a sum over routed rows of unequal size
        return (n(rows, 2 * k) * torch.exp(n(2 * k))) @ n(2 * k, cols) * 1e-3
    if kind == "low":
        return n(rows, max(1, k // 8)) @ n(max(1, k // 8), cols)
    if kind == "one":
        return n(rows, 1) @ n(1, cols)
    if kind == "outliers":
        m = n(rows, cols)
        m[:, ::97] *= 50.0
        return m
    raise ValueError(kind)


def rel(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


ORTHO = [
    # rows, cols: one element, one row and column, ragged, square, wide and tall, several tiles
    (1, 1), (1, 300), (300, 1), (2, 3), (16, 16), (17, 129), (64, 64), (128, 128), (129, 127), (100, 260), (260, 100),
    (256, 256), (255, 513), (512, 512), (384, 640), (640, 384), (300, 777), (1000, 250), (1024, 1024), (512, 2048),
]


@pytest.mark.parametrize("rows,cols", ORTHO)
def test_orthogonalize_matches_oracle(rows, cols):
    log(f"orthogonalize {rows} x {cols}")
    for kind in ("rows", "normal"):
        g = matrix(kind, rows, cols, rows * 7 + cols)
        o, m = bm.orthogonalize(g.cuda())
        assert m is None and o.shape == (rows, cols)
        want, _ = ref.orthogonalize(g.double().numpy())
        e = rel(to_f64(o), want)
        log(f"  {kind}: {e:.2e}")
        assert e <= FULL, (kind, e)


def exact_on_gpu(u):
    """ref.orthogonalize without momentum, the same formula in fp64 on the GPU
    (CPU products of these sizes take seconds)."""
    import torch
    x = u.double()
    x = x / x.norm()
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    a, b, c = ref.NS_COEFFS
    for _ in range(ref.NS_STEPS):
        g = x @ x.T.contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


# every tile size and shared depths: tiles of 32 whole and shared, 64 whole and
# shared, 96, 128, 256, cut tiles of each
LARGE = [(40, 2500), (2500, 40), (63, 8191), (200, 1025), (500, 6000), (6000, 500), (1000, 1024), (1100, 1300), (1900, 2000),
         (2200, 5000), (5000, 2200), (16384, 48), (1, 16384),
         # sides of an odd number of 64: a half step at the end of the second terms' depth
         # and, in tiles of 96, one group's last piece, whole and in shares
         (1590, 1600), (1600, 1590), (890, 8190), (1210, 8190), (8190, 1200), (2235, 2240), (1344, 1340), (700, 704),
         (320, 8190), (330, 1340), (830, 3390), (1980, 1970), (1150, 8100), (1470, 8100), (1470, 3000), (3130, 3136),
         (440, 8100), (1200, 16384), (2170, 2176), (60, 8100), (950, 16384), (2900, 2944), (190, 8100)]


@pytest.mark.parametrize("rows,cols", LARGE)
def test_orthogonalize_large(rows, cols):
    g = matrix("normal", rows, cols, rows + cols).cuda()
    o = bm.orthogonalize(g)[0]
    want = exact_on_gpu(g)
    e = ((o.double() - want).norm() / want.norm()).item()
    log(f"orthogonalize {rows} x {cols}: {e:.2e}")
    assert e <= FULL, e
    for _ in range(3):  # shares are added in order whoever comes last
        assert (bm.orthogonalize(g)[0] == o).all()


def test_orthogonalize_largest():
    """The largest matrix the library takes."""
    import torch
    g = torch.randn(16384, 16384, generator=torch.Generator("cuda").manual_seed(5), device="cuda")
    o = bm.orthogonalize(g)[0]
    want = exact_on_gpu(g)
    assert ((o.double() - want).norm() / want.norm()).item() <= FULL


@pytest.mark.parametrize("kind", ["low", "one", "outliers"])
@pytest.mark.parametrize("rows,cols", [(256, 256), (300, 777), (1000, 250)])
def test_orthogonalize_hard_spectra(rows, cols, kind):
    g = matrix(kind, rows, cols, 21)
    want, _ = ref.orthogonalize(g.double().numpy())
    e = rel(to_f64(bm.orthogonalize(g.cuda())[0]), want)
    log(f"orthogonalize {kind} {rows} x {cols}: {e:.2e}")
    assert e <= (FULL if kind == "outliers" else ANY), e


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("rows,cols", [(200, 328), (129, 67)])
def test_orthogonalize_momentum(rows, cols, nesterov, dtype):
    import torch
    g = matrix("rows", rows, cols, 31)
    if dtype == "bf16":
        g = g.bfloat16()
    m = matrix("normal", rows, cols, 32) * 0.1
    gd, md = g.cuda(), m.cuda()
    o, m1 = bm.orthogonalize(gd, md, mu=0.9, nesterov=nesterov)
    want, wm = ref.orthogonalize(to_f64(g), to_f64(m), mu=float(np.float32(0.9)), nesterov=nesterov)
    # one fused multiply-add
    assert (np.abs(to_f64(m1) - wm) <= 2.0 ** -24 * np.abs(wm)).all() and rel(to_f64(o), want) <= FULL
    # the momentum in place
    o2, m2 = bm.orthogonalize(gd, md, mu=0.9, nesterov=nesterov, momentum_out=md)
    assert m2 is md and (md == m1).all() and (o2 == o).all()


def test_orthogonalize_scale_zero_and_non_finite():
    import torch
    g = matrix("rows", 192, 320, 41).cuda()
    o = bm.orthogonalize(g)[0]
    # a power of two changes only the norm, exactly; far ends of fp32 included
    for k in (40, -60, 100):
        assert (bm.orthogonalize(g * 2.0 ** k)[0] == o).all(), k
    assert (bm.orthogonalize(torch.zeros_like(g))[0] == 0).all()
    for bad in (float("nan"), float("inf")):
        h = g.clone()
        h[5, 7] = bad
        assert torch.isnan(bm.orthogonalize(h)[0]).all()
    # an error in an earlier call does not stay in anything later calls read
    assert (bm.orthogonalize(g)[0] == o).all()


def test_orthogonalize_singular_values():
    import torch
    o = bm.orthogonalize(matrix("normal", 384, 1200, 43).cuda())[0]
    sv = torch.linalg.svdvals(o.double().cpu())
    assert sv.max() < 1.21 and sv.min() > 0.66, (sv.min(), sv.max())


def test_orthogonalize_tall_is_transposed_wide():
    """Both orientations run the same products on the same padded matrices;
    only the order of the norm's fp64 sum differs."""
    g = matrix("rows", 333, 150, 44).cuda()
    a, b = bm.orthogonalize(g)[0], bm.orthogonalize(g.T.contiguous())[0]
    assert rel(to_f64(a), to_f64(b.T)) <= 2.0 ** -8


def test_orthogonalize_unaligned_and_rows_behind():
    import torch
    g = matrix("rows", 70, 136, 45).cuda()
    o = bm.orthogonalize(g)[0]
    buf = torch.empty(g.numel() + 8, device="cuda")
    v = buf[3:3 + g.numel()].view(g.shape)
    v.copy_(g)
    out = torch.full((72, 136), 5.0, dtype=torch.bfloat16, device="cuda")
    off = torch.full((g.numel() + 8,), 5.0, dtype=torch.bfloat16, device="cuda")
    bm.orthogonalize(v, out=off[1:1 + g.numel()].view(g.shape))
    bm.orthogonalize(g, out=out[:70])
    assert (out[70:] == 5.0).all() and (out[:70] == o).all()
    assert (off[0] == 5.0) and (off[1 + g.numel():] == 5.0).all()
    assert rel(to_f64(off[1:1 + g.numel()].view(g.shape)), to_f64(o)) <= 2.0 ** -8


def test_orthogonalize_streams_and_graph():
    """Two streams at once and two captured graphs, replayed in turn with eager
    calls between, all equal to the eager result."""
    import torch
    gs = [matrix("rows", 100, 4096, 51).cuda(), matrix("rows", 384, 256, 52).cuda()]
    ms = [torch.randn_like(g) * 0.01 for g in gs]
    want = [bm.orthogonalize(g, m) for g, m in zip(gs, ms)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(bm.orthogonalize(gs[k], ms[k]))
    torch.cuda.synchronize()
    for k in range(2):
        assert all((o == want[k][0]).all() and (m == want[k][1]).all() for o, m in got[k])
    graphs, outs, ins = [], [], [g.clone() for g in gs]
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(bm.orthogonalize(ins[k], ms[k]))
        graphs.append(graph)
    for rep in range(3):
        for k in range(2):
            ins[k].copy_(gs[k] * (1 + 0.25 * rep) + rep * ms[k])
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in range(2):
            eager = bm.orthogonalize(ins[k], ms[k])
            assert (outs[k][0] == eager[0]).all() and (outs[k][1] == eager[1]).all(), (rep, k)


# ------------------------------------------------------------------ substrate step
STEP = [(1, 16), (3, 16), (5, 48), (64, 64), (256, 64), (257, 64), (1024, 64), (1025, 64), (100, 1040), (512, 512), (1000, 2064), (2048, 1024), (16384, 16)]


@pytest.mark.parametrize("rows,cols", STEP)
@pytest.mark.parametrize("update", [False, True])
def test_substrate_step_is_exact(rows, cols, update):
    """W' is one rounding of an fp64 value, the codes a comparison of fp64 values:
    both equal the oracle's bit for bit; scale is one rounding of a sum whose
    order differs (fp64: below 2^-40 of it)."""
    import torch
    r = np.random.default_rng(rows + cols)
    w = r.standard_normal((rows, cols)).astype(np.float32)
    o = torch.from_numpy(r.standard_normal((rows, cols)).astype(np.float32)).bfloat16()
    w1, packed, scale = bm.substrate_step(torch.from_numpy(w).cuda(), o.cuda() if update else None, step=0.03, decay=0.001)
    ww, codes, ws = ref.substrate_step(w, to_f64(o) if update else None, step=0.03, decay=0.001)
    assert (w1.cpu().numpy() == ww).all()
    assert (packed.cpu().numpy().view(np.uint32) == bm.pack_ternary(codes)).all()
    assert abs(float(scale) - ws) <= (2.0 ** -24 + 2.0 ** -40) * ws


def test_substrate_step_ties_zero_and_non_finite():
    import torch
    tie = torch.tensor([[3.0] * 4 + [-3.0] * 4 + [1.0] * 4 + [-1.0] * 4])
    _, packed, scale = bm.substrate_step(tie.cuda())
    codes = np.array([[1] * 4 + [-1] * 4 + [0] * 8], np.int8)
    assert float(scale) == 2.0 and (packed.cpu().numpy().view(np.uint32) == bm.pack_ternary(codes)).all()
    _, packed, scale = bm.substrate_step(torch.zeros(4, 32, device="cuda"))
    assert (packed == 0).all() and float(scale) == 0.0
    for bad, rows in ((float("nan"), 8), (float("inf"), 8), (float("nan"), 1100), (float("inf"), 1100)):
        w = torch.randn(rows, 64, device="cuda")
        w[2, 5] = bad
        _, packed, scale = bm.substrate_step(w)
        assert (packed == 0).all() and not np.isfinite(float(scale))


@pytest.mark.parametrize("rows", [320, 64, 30])
def test_substrate_step_in_place_and_graph(rows):
    import torch
    g = torch.Generator().manual_seed(61)
    w0 = torch.randn(rows, 256, generator=g).cuda()
    o = torch.randn(rows, 256, generator=g).bfloat16().cuda()
    want = bm.substrate_step(w0, o, step=0.1, decay=0.01)
    w, packed = w0.clone(), torch.empty(rows, 16, dtype=torch.int32, device="cuda")
    got = bm.substrate_step(w, o, step=0.1, decay=0.01, w_out=w, packed=packed)
    assert got[0] is w and got[1] is packed and all((a == b).all() for a, b in zip(got, want))
    w.copy_(w0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = bm.substrate_step(w, o, step=0.1, decay=0.01, w_out=w, packed=packed)
    eager = w0
    for k in range(4):
        graph.replay()
        torch.cuda.synchronize()
        eager, p, s = bm.substrate_step(eager, o, step=0.1, decay=0.01)
        assert (out[0] == eager).all() and (packed == p).all() and (out[2] == s).all(), k


# ------------------------------------------------------------------ a training step
@pytest.mark.parametrize("d_ff", [0, 256])
def test_training_step_of_a_normalised_layer(d_ff):
    """x -> s = x + residual -> norm -> layer -> gradients -> norm's backward ->
    orthogonalised update of every substrate -> new codes in the layer's own
    w_base -> next forward, each link against the oracle at the GPU's inputs."""
    import torch
    cfg = wl.small_config(d_model=128, d_ff=d_ff, n_experts=6, top_k=2, tokens=90, act="bf16", seed_index=700 + d_ff)
    inp = wl.generate(cfg)
    layer = bm.Layer.from_inputs(inp, device="cuda")
    x = to_dev(inp.x, "bf16")
    g = torch.Generator().manual_seed(71)
    res = torch.randn(x.shape, generator=g).bfloat16().cuda()
    gamma, beta = (1 + 0.1 * torch.randn(128, generator=g)).cuda(), (0.1 * torch.randn(128, generator=g)).cuda()
    dy = torch.randn(x.shape, generator=g).bfloat16().cuda()
    n, s, mean, rstd = bm.layer_norm_forward(x, gamma, beta, residual=res)
    y, state = layer.forward_train(n)
    grads = layer.backward(n, dy, state)
    ds, dgamma, dbeta = bm.layer_norm_backward(grads["x"], s, gamma, mean, rstd, d_sum=dy)
    wx, wg, wb = ref.layer_norm_backward(to_f64(grads["x"]), to_f64(s), to_f64(gamma), to_f64(mean), to_f64(rstd), to_f64(dy))
    # bf16's half step per element and fp32 sums
    assert rel(to_f64(ds), wx) <= 2.0 ** -8 and rel(to_f64(dgamma), wg) <= 1e-5 and rel(to_f64(dbeta), wb) <= 1e-5
    codes = []
    for m, latent in enumerate(inp.w_base):
        w = torch.from_numpy(latent.astype(np.float32)).cuda() + 0.1 * torch.randn(latent.shape, generator=g).cuda()
        mom = torch.zeros_like(w)
        o, _ = bm.orthogonalize(grads["w_base"][m], mom, momentum_out=mom)
        assert rel(to_f64(o), ref.orthogonalize(to_f64(grads["w_base"][m]), np.zeros(latent.shape))[0]) <= ANY
        w0 = w.cpu().numpy()
        layer.step_substrate(m, w, o, step=0.5, decay=0.01, w_out=w)
        ww, cc, _ = ref.substrate_step(w0, to_f64(o), step=0.5, decay=0.01)
        assert (w.cpu().numpy() == ww).all()
        codes.append(cc)
    assert any((c != b).any() for c, b in zip(codes, inp.w_base))
    inp.w_base = codes
    want = bm.Layer.from_inputs(inp, device="cuda").forward(n)
    assert (layer.forward(n) == want).all()


def test_step_substrate_prepares_again():
    """A prepared layer forwards with the new codes, not with those it was
    prepared from; misfit substrates are refused."""
    import torch
    inp = wl.generate(wl.small_config(d_model=256, d_ff=0, n_experts=4, top_k=2, tokens=50, act="bf16", seed_index=720))
    layer = bm.Layer.from_inputs(inp, device="cuda").prepare()
    x = to_dev(inp.x, "bf16")
    before = layer.forward(x).clone()
    w = torch.randn(256, 256, generator=torch.Generator().manual_seed(72)).cuda()
    layer.step_substrate(0, w)
    inp.w_base = [ref.substrate_step(w.cpu().numpy())[1]]
    want = bm.Layer.from_inputs(inp, device="cuda").prepare().forward(x)
    got = layer.forward(x)
    assert (got == want).all() and (got != before).any()
    with pytest.raises(ValueError):
        layer.step_substrate(1, w)
    with pytest.raises(ValueError):
        layer.step_substrate(0, w[:128])


@pytest.mark.parametrize("d_ff", [0, 512])
def test_step_substrate_under_captured_forward(d_ff):
    """A forward captured before a substrate step replays with the step's codes:
    the prepared weights stay where the graph reads them, and a step captured
    itself prepares again at every replay."""
    import torch
    inp = wl.generate(wl.small_config(d_model=256, d_ff=d_ff, n_experts=4, top_k=2, tokens=50, act="bf16", seed_index=721))
    layer = bm.Layer.from_inputs(inp, device="cuda").prepare()
    kept = layer.struct.prepared
    x = to_dev(inp.x, "bf16")
    y = torch.empty_like(x)
    layer.forward(x, y)
    torch.cuda.synchronize()
    fwd, upd = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(fwd):
        layer.forward(x, y)
    rows, cols = (d_ff, 256) if d_ff else (256, 256)
    src = torch.zeros(rows, cols, device="cuda")
    with torch.cuda.graph(upd):
        layer.step_substrate(0, src)
    assert layer.struct.prepared == kept
    for k in range(3):
        step = torch.randn(rows, cols, generator=torch.Generator().manual_seed(80 + k)).cuda()
        if k == 1:
            layer.step_substrate(0, step)         # eager, between replays
        else:
            src.copy_(step)
            upd.replay()
        fwd.replay()
        inp.w_base = [ref.substrate_step(step.cpu().numpy())[1]] + list(inp.w_base[1:])
        want = bm.Layer.from_inputs(inp, device="cuda").prepare().forward(x)
        assert (y == want).all(), k


@pytest.mark.parametrize("kw", [dict(d_model=128, d_ff=0, act="f32"), dict(d_model=128, d_ff=256, act="f32"),
                                dict(d_model=256, d_ff=0, act="bf16"), dict(d_model=256, d_ff=512, act="bf16")])
def test_step_substrate_rescales_the_layer(kw):
    """After a step with rescale the layer computes with scale * codes: forward,
    training forward and gradients equal those of a layer built with these scales,
    and the forward is the oracle's with W = scale * codes."""
    import torch
    from gpu_helpers import row_rel_err, tol_for
    inp = wl.generate(wl.small_config(n_experts=4, top_k=2, tokens=60, seed_index=730 + kw["d_model"], **kw))
    layer = bm.Layer.from_inputs(inp, device="cuda").prepare()
    x = to_dev(inp.x, kw["act"])
    g = torch.Generator().manual_seed(73)
    scales, real = [], []
    for m, latent in enumerate(inp.w_base):
        w = (0.3 + m) * torch.randn(latent.shape, generator=g).cuda()
        o = torch.randn(latent.shape, generator=g).bfloat16().cuda()
        w1, scale = layer.step_substrate(m, w, o, step=0.05, decay=0.01, rescale=True)
        _, codes, want = ref.substrate_step(w1.cpu().numpy())
        assert abs(layer.struct.w_scale[m] - want) <= 2.0 ** -23 * want and layer.struct.w_scale[m] == float(scale)
        scales.append(float(scale))
        inp.w_base[m] = codes
        real.append(want * codes)
    fresh = bm.Layer.from_inputs(inp, device="cuda")
    for m, scale in enumerate(scales):
        fresh.struct.w_scale[m] = scale
    y, idx, _ = layer.forward(x, return_routing=True)
    assert (y == fresh.prepare().forward(x)).all()
    (yt, state), (ft, fstate) = layer.forward_train(x), fresh.forward_train(x)
    dy = torch.randn(x.shape, generator=g).to(x.dtype).cuda()
    grads, want = layer.backward(x, dy, state), fresh.backward(x, dy, fstate)
    assert (yt == ft).all() and all((a == b).all() for a, b in zip(grads["w_base"], want["w_base"]))
    inp.w_base = real
    wy = ref.forward(inp, idx_override=idx.cpu().numpy())[0]
    e = row_rel_err(to_f64(y), wy).max()
    log(f"rescaled layer {kw}: {e:.2e}")
    assert e <= tol_for(kw["act"]), e


def test_step_substrate_rescale_refusals():
    """A captured step cannot set a host value; a scale that is not finite is not
    taken over."""
    import torch
    inp = wl.generate(wl.small_config(d_model=128, d_ff=0, n_experts=4, top_k=2, tokens=50, act="bf16", seed_index=740))
    layer = bm.Layer.from_inputs(inp, device="cuda").prepare()
    w = torch.randn(128, 128, generator=torch.Generator().manual_seed(74)).cuda()
    layer.step_substrate(0, w)
    assert layer.struct.w_scale[0] == 1.0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError, match="captured"):
            layer.step_substrate(0, w, rescale=True)
        layer.step_substrate(0, w)
    w[3, 4] = float("nan")
    with pytest.raises(ValueError, match="finite"):
        layer.step_substrate(0, w, rescale=True)
    assert layer.struct.w_scale[0] == 1.0


# Narrower bars, relative Frobenius norm, in the mean square over many entries.  A
# rounding to fp16 is 2^-12.2 (half a place, mantissas spread evenly), to bf16 1.7e-3,
# to e4m3 2^-5.2.
# Full rank: about ten roundings act on settled values, whose map stretches by 2 in
#   the mean square (its slope between -1.5 and 4 over 0.68 .. 1.21): sqrt(10) * 2 *
#   2^-12 = 1.5e-3, with bf16's 2.3e-3.  Diagonals left as stored: 4.8e-3 at 48 x 16384.
# Rank one: noise outside the row space grows 485-fold from X_0, 12-fold from X_3.
#   X_0 has 2^-12.2 2^-5.2 of its own second term's rounding and of P's e4m3 copy as
#   much at most: 2.8e-3 each; X_3, in one term, 2.1e-4 * 11.8 * 1.8 = 4.5e-3 (1.8 for
#   ||X_3|| / ||X_5||); X_4, X_1 and X_2 1e-3 each: 6.3e-3, with bf16's 6.6e-3; half as
#   much again for few rows.  A second term lost at X_2, where it counts least: 1.4e-2.
# Rank S / 8: the signal grows too, 3-fold at the least, and settles before X_3: X_0's
#   1.9e-3, X_3's 2.1e-4 * 11.8 = 2.5e-3, bf16's: 3.6e-3.  Lost at X_2: 6.9e-3.
BARS = dict(normal=3e-3, low=5e-3, one=1e-2)

# every tile of every product, whole and shared, cut and not, with even and odd depths
# where a tile treats them differently, both orientations
TILES = [(64, 64), (48, 16384), (16384, 48), (250, 256), (128, 5500), (5500, 120), (330, 1340), (384, 2620), (2110, 1980),
         (1024, 1024), (4096, 1024), (320, 6592), (8250, 256), (960, 7168), (1300, 3000), (704, 11960), (2048, 8192),
         (8190, 2040), (1275, 15030), (1536, 2750), (2750, 1530), (1020, 12928), (960, 14650), (14650, 950), (1020, 12990),
         (960, 14528), (1020, 12800), (12800, 1000), (1020, 12730), (1150, 7610), (1150, 7800), (1470, 6840), (7030, 1470),
         (2496, 6528)]


@pytest.mark.parametrize("rows,cols", TILES)
def test_orthogonalize_precision_in_every_tile(rows, cols):
    for kind, bar in BARS.items():
        g = matrix(kind, rows, cols, rows + 3 * cols).cuda()
        o, want = bm.orthogonalize(g)[0], exact_on_gpu(g)
        e = ((o.double() - want).norm() / want.norm()).item()
        log(f"orthogonalize {kind} {rows} x {cols}: {e:.2e}")
        assert e <= bar, (kind, e)


@pytest.mark.parametrize("rows,cols", [(4096, 4096), (8192, 8192), (8192, 16384), (16384, 16384)])
def test_orthogonalize_rank_one_of_large_sides(rows, cols):
    """Entries of X_0 shrink with the sides, and their second terms with them: the
    bar is the same at every size.  Rank one is its own solution, u v^T times the
    quintic iterated on 1."""
    import torch
    gen = torch.Generator("cuda").manual_seed(rows + cols)
    u, v = (torch.randn(n, generator=gen, device="cuda") for n in (rows, cols))
    g = u[:, None] * v
    x = 1.0
    for _ in range(ref.NS_STEPS):
        x = ref.NS_COEFFS[0] * x + ref.NS_COEFFS[1] * x ** 3 + ref.NS_COEFFS[2] * x ** 5
    o = bm.orthogonalize(g)[0].double()
    u, v = u.double(), v.double()
    o -= (x / (u.norm() * v.norm()) * u)[:, None] * v
    e = o.norm().item() / x
    log(f"orthogonalize rank one {rows} x {cols}: {e:.2e}")
    assert e <= BARS["one"], e
