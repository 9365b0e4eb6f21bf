"""AdamW over many tensors (include/bmoe_adamw.h) on the GPU against the fp64 oracle.

Bars, with u = 2^-24 (half a step of fp32): beta, 1 - beta, lr, eps and the scalars made of
them are rounded to fp32 once each (u), a product or sum adds u of its result, the hardware's
root and reciprocal 2 u each.  m' = beta1 m + (1 - beta1) g is off by at most
em = 4 u (beta1 |m| + (1 - beta1) |g|), v' by ev = 5 u v'; the divisor by (ev / v' / 2 + 6 u) of
itself, so the step lr m'/.. by 16 u of itself and by em's part of it; p' by 3 u (|p| + |p'|) beside.
A code is one of those that m' or v' within its bar gets by the same fraction (plus 2^-19,
what the sum of a value and its fraction is rounded by).
"""
import numpy as np
import pytest

import compressed_mixture_experts_amd as bm
from oracle import ref
from gpu_helpers import log, to_f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
B1, B2 = 0.9, 0.999


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


def state64(opt, i):
    """(p, m, v) in fp64 and, with codes, the codes and exponents."""
    p = to_f64(opt.params[i]).ravel()
    if opt.bits[i] == 32:
        return p, to_f64(opt.m[i]).ravel(), to_f64(opt.v[i]).ravel(), None
    cm, cv = opt.m[i].cpu().numpy().ravel(), opt.v[i].cpu().numpy().ravel()
    em, ev = opt.m_exp[i].cpu().numpy(), opt.v_exp[i].cpu().numpy()
    m = ref.adamw_values(cm & 127, em, ref.ADAMW_M_TOP) * np.where(cm >= 128, -1.0, 1.0)
    v = ref.adamw_values(cv, ev, ref.ADAMW_V_TOP)
    return p, np.where((cm & 127) == 127, np.nan, m), np.where(cv == 255, np.nan, v), (cm, cv, em, ev)


def check_codes(got, exps, x, off, top, r, floor):
    """The codes of |x|, x known to within off."""
    lo, hi = np.maximum(np.abs(x) - off, 0.0), np.abs(x) + off
    elo, ehi = ref.adamw_exponents(lo), ref.adamw_exponents(hi)
    assert ((elo <= exps) & (exps <= ehi)).all(), "exponents"
    cl, ch = ref.adamw_codes(lo, exps, top, r - 2.0 ** -19), ref.adamw_codes(hi, exps, top, r + 2.0 ** -19)
    if floor:
        cl, ch = np.where(lo > 0, np.maximum(cl, 1), cl), np.where(hi > 0, np.maximum(ch, 1), ch)
    assert ((np.maximum(cl, 0) <= got) & (got <= ch)).all(), "codes"


def check_step(opt, i, before, g, t, lr, decay, seed=0, eps=1e-8):
    p0, m0, v0, _ = before
    p1, m1, v1, codes = state64(opt, i)
    p, m, v = ref.adamw(p0, g, m0, v0, t, lr, (B1, B2), eps, decay)
    em, ev = 4 * U * (B1 * np.abs(m0) + (1 - B1) * np.abs(g)), 5 * U * v
    div = np.sqrt(v / (1 - B2 ** t)) + eps
    by = lr / (1 - B1 ** t) / div
    tol = 16 * U * np.abs(by * m) + by * em + 3 * U * (np.abs(p0) + np.abs(p))
    assert (np.abs(p1 - p) <= tol).all(), f"p of tensor {i}"
    if opt.copies[i] is not None:
        c = to_f64(opt.copies[i]).ravel()
        assert (np.abs(c - p1) <= 2.0 ** -8 * np.abs(p1)).all(), f"copy of tensor {i}"
    if codes is None:
        assert (np.abs(m1 - m) <= em).all() and (np.abs(v1 - v) <= ev).all(), f"moments of tensor {i}"
        return
    cm, cv, xm, xv = codes
    rm, rv = ref.adamw_random(len(g), t, i, seed)
    check_codes(cm & 127, xm, m, em, ref.ADAMW_M_TOP, rm, False)
    check_codes(cv, xv, v, ev, ref.ADAMW_V_TOP, rv, True)
    sure = np.abs(m) > em
    assert ((cm >= 128) == (m < 0))[sure].all(), "signs"


def make(sizes, kinds, bits, inputs, offset=0, **kw):
    """Tensors of the sizes, `offset` values from an aligned place, and gradients."""
    import torch
    gen = torch.Generator().manual_seed(inputs)
    ps, gs = [], []
    for k, n in enumerate(sizes):
        flat = torch.randn(n + offset, generator=gen).cuda()
        ps.append(flat[offset:])
        g = torch.randn(n + offset, generator=gen) * torch.exp(2 * torch.randn(n + offset, generator=gen) - 5)
        gs.append(g.to(torch.bfloat16 if kinds[k % len(kinds)] == "bf16" else torch.float32).cuda()[offset:])
    return bm.AdamW(ps, bits=bits, **kw), gs


SIZES = [1, 2, 3, 4, 5, 63, 255, 256, 257, 511, 1023, 1024, 1025, 4096, 5000, 70001]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_against_the_oracle(bits, offset):
    import torch
    opt, gs = make(SIZES, ["f32", "bf16"], bits, 3 + offset, offset, weight_decay=[0.0, 0.1] * 8, lr_scale=[1.0, 0.5, 2.0, 1.0] * 4,
                   copies=[torch.empty(n + offset, dtype=torch.bfloat16, device="cuda")[offset:] if n % 2 else None for n in SIZES], seed=77)
    for t in range(1, 4):
        log(f"adamw bits={bits} offset={offset} step {t}")
        before = [state64(opt, i) for i in range(len(SIZES))]
        opt.step(gs)
        for i in range(len(SIZES)):
            check_step(opt, i, before[i], to_f64(gs[i]), t, 1e-3 * [1.0, 0.5, 2.0, 1.0][i % 4], [0.0, 0.1][i % 2], 77)
        gs = [(-0.7 * g.flip(0) + 0.1 * g).contiguous() if offset == 0 else g.mul_(-0.6) for g in gs]
    assert opt.steps == 3


def test_more_tensors_than_a_launch_takes_in_both_forms():
    import torch
    sizes = [1 + (37 * k) % 700 for k in range(131)] + [300000]
    opt, gs = make(sizes, ["f32", "f32", "bf16"], [8 if k % 3 else 32 for k in range(132)], 5)
    skipped = {0, 40, 41, 90}
    before = [state64(opt, i) for i in range(132)]
    opt.step([None if i in skipped else g for i, g in enumerate(gs)])
    for i in range(132):
        if i in skipped:
            assert all(np.array_equal(a, b) for a, b in zip(before[i][:3], state64(opt, i)[:3]))
        else:
            check_step(opt, i, before[i], to_f64(gs[i]), 1, 1e-3, 0.01)
    # values over several workgroups of the longer run: 2^21 and more in all
    opt, gs = make([2_500_003, 100], ["bf16", "f32"], [8, 32], 6)
    before = [state64(opt, i) for i in range(2)]
    opt.step(gs)
    for i in range(2):
        check_step(opt, i, before[i], to_f64(gs[i]), 1, 1e-3, 0.01)
    torch.cuda.synchronize()


def test_same_inputs_same_results():
    runs = []
    for _ in range(2):
        opt, gs = make([5000, 257], ["f32"], 8, 9, seed=5)
        for _ in range(3):
            opt.step(gs)
        runs.append([x.clone() for k in (opt.params, opt.m, opt.v, opt.m_exp, opt.v_exp) for x in k])
    assert all((a == b).all() for a, b in zip(*runs))


@pytest.mark.parametrize("size", [1e-30, 1e-18, 1e15, 3e18])
def test_codes_over_the_range(size):
    """Gradients whose squares are near both ends of fp32, blocks of zeros, one value that is
    alone in its block."""
    import torch
    r = np.random.default_rng(2)
    g = (r.standard_normal(1536) * size).astype(np.float32)
    g[256:512] = 0
    g[512:768] = 0
    g[600] = size
    opt = bm.AdamW([torch.zeros(1536, device="cuda")], bits=8, weight_decay=0.0)
    for t in (1, 2):
        p0, m0, v0, _ = state64(opt, 0)
        opt.step([torch.from_numpy(g).cuda()])
        _, m1, v1, (cm, cv, em, ev) = state64(opt, 0)
        g64 = g.astype(np.float64)
        m, v = B1 * m0 + (1 - B1) * g64, B2 * v0 + (1 - B2) * g64 * g64
        # half a unit of fp32's lowest place where values are below its normal range
        sm, sv = 4 * U * (B1 * np.abs(m0) + (1 - B1) * np.abs(g64)) + 2.0 ** -149, 5 * U * v + 3 * 2.0 ** -149
        rm, rv = ref.adamw_random(1536, t, 0, 0)
        check_codes(cm & 127, em, m, sm, ref.ADAMW_M_TOP, rm, False)
        check_codes(cv, ev, v, sv, ref.ADAMW_V_TOP, rv, True)
        assert (cm[256:512] == 0).all() and (cv[256:512] == 0).all() and (em[1] == 1) and (ev[1] == 1)
        live = v > 2.0 ** -140
        assert (cv[live] >= 1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_infinities_and_nans_stay_in_their_value(bits):
    import torch
    opt, gs = make([1000], ["f32"], bits, 12)
    other, _ = make([1000], ["f32"], bits, 12)
    bad = gs[0].clone()
    bad[3], bad[300], bad[301] = float("nan"), float("inf"), float("-inf")
    opt.step([bad])
    # a block's exponent is its largest finite value's: that of the block without these
    good = gs[0].clone()
    good[[3, 300, 301]] = 0.0
    other.step([good])
    hit = torch.zeros(1000, dtype=torch.bool, device="cuda")
    hit[[3, 300, 301]] = True
    assert torch.isnan(opt.params[0][hit]).all() and (opt.params[0][~hit] == other.params[0][~hit]).all()
    (m,), (v,) = opt.moments()
    (m2,), (v2,) = other.moments()
    assert not torch.isfinite(m[hit]).any() and not torch.isfinite(v[hit]).any()
    assert (m[~hit] == m2[~hit]).all() and (v[~hit] == v2[~hit]).all()
    opt.step(gs)
    assert torch.isnan(opt.params[0][hit]).all() and torch.isfinite(opt.params[0][~hit]).all()


def test_v_decays_in_8_bits():
    """Gradients of zero: v falls by 1 - beta2 a step though its codes are 6 to 12 % apart.
    In 2^17 values the mean after 200 steps is 0.999^200 of what it was, to within 6 standard
    deviations: a step's variance is at most p (1 - p) d^2 with d <= v / 8 the distance of codes
    and p d = 0.001 v what is cut off, so <= 0.001 v^2 / 8 a step; v itself only falls."""
    import torch
    n = 1 << 17
    x = torch.rand(n, generator=torch.Generator().manual_seed(1)).cuda() + 0.5
    opt = bm.AdamW([torch.zeros(n, device="cuda")], bits=8, lr=0.0)
    opt.step([x])
    (_,), (v,) = opt.moments()
    start = v.double()
    zero = torch.zeros(n, device="cuda")
    for _ in range(200):
        opt.step([zero])
    (m,), (v,) = opt.moments()
    top = float(start.max())
    assert abs(float(v.double().mean()) - 0.999 ** 200 * float(start.mean())) < 6 * np.sqrt(200 * 0.001 / 8 / n) * top
    # m falls by 0.9 a step, on which the rounding's deviation is 5 % of it a step, 0.7 in its
    # logarithm in 200: 7 of those leave it below 0.9^150
    assert float(m.abs().max()) < 0.9 ** 150 * 0.15


def test_moments_in_both_types():
    import torch
    opt, gs = make([1000, 64, 777], ["f32"], [8, 32, 8], 13)
    opt.step(gs)
    want = [state64(opt, i) for i in range(3)]
    ms, vs = opt.moments()
    assert ms[1] is opt.m[1] and vs[1] is opt.v[1]
    m16 = [torch.empty(1000, dtype=torch.bfloat16, device="cuda"), None, torch.empty(778, dtype=torch.bfloat16, device="cuda")[1:]]
    v16 = [torch.empty(1000, dtype=torch.bfloat16, device="cuda"), None, torch.empty(778, dtype=torch.bfloat16, device="cuda")[1:]]
    opt.moments(m16, v16)
    for i in (0, 2):
        for got in ((ms[i], vs[i]), (m16[i], v16[i])):
            assert np.array_equal(to_f64(got[0]), want[i][1]) and np.array_equal(to_f64(got[1]), want[i][2])


def test_captured_steps_count_on():
    """A captured step replayed with eager work between: every replay equals an eager
    optimiser's step, the rate and the gradients' factor read on the GPU."""
    import torch
    lr, scale = torch.tensor([1e-3], device="cuda"), torch.tensor([0.5], device="cuda")
    sizes = [5000, 300]
    opt, gs = make(sizes, ["f32"], [8, 32], 21, capturable=True, lr=lr, seed=4)
    eager, _ = make(sizes, ["f32"], [8, 32], 21, lr=1e-3, seed=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        opt.step(gs, grad_scale=scale)
    torch.cuda.current_stream().wait_stream(s)
    eager.step([0.5 * g for g in gs])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(gs, grad_scale=scale)
    for k in range(4):
        for g in gs:
            g.mul_(-1.25)
        rate = 1e-3 * (k + 1)
        lr.fill_(rate)
        eager.lr = float(lr.item())
        graph.replay()
        eager.step([0.5 * g for g in gs])
        torch.cuda.synchronize()
        for a, b in zip(opt.params + opt.m + opt.v, eager.params + eager.m + eager.v):
            # the device's bias corrections are the host's to one unit in the last place
            assert (a == b).all() if a.dtype == torch.uint8 else torch.allclose(a, b, rtol=1e-6, atol=1e-7)
    assert opt.steps == eager.steps == 5
    plain, gs = make(sizes, ["f32"], 32, 22)
    refused = torch.cuda.CUDAGraph()
    with pytest.raises(ValueError, match="capturable"):
        with torch.cuda.graph(refused):
            torch.zeros(1, device="cuda")
            plain.step(gs)


def test_another_stream_and_given_moments():
    import torch
    a, gs = make([4097], ["f32"], 32, 30)
    a.step(gs)
    b = bm.AdamW([a.params[0].clone()], m=[a.m[0].clone()], v=[a.v[0].clone()], steps=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.step(gs)
    s.synchronize()
    a.step(gs)
    torch.cuda.synchronize()
    assert (a.params[0] == b.params[0]).all() and (a.m[0] == b.m[0]).all() and a.steps == b.steps == 2


def test_memory_that_moved():
    """A tensor that its owner gives other memory is taken from there, or refused."""
    import torch
    for bits in (32, 8):
        (a, gs), (b, _) = (make([300, 70], ["f32"], bits, 31, copies=[torch.zeros(300, dtype=torch.bfloat16, device="cuda"), None])
                           for _ in range(2))
        for opt in (a, b):
            opt.step(gs)
        old, kept = b.params[0].data, b.params[0].data.clone()
        b.params[0].data = old.clone()
        b.copies[0].data = b.copies[0].data.clone()
        for opt in (a, b):
            opt.step(gs)
        torch.cuda.synchronize()
        assert (old == kept).all() and all((x == y).all() for x, y in zip(a.params, b.params)) and (a.copies[0] == b.copies[0]).all()
        assert all((x == y).all() for p, q in zip(a.moments(), b.moments()) for x, y in zip(p, q))
        b.params[1].data = torch.zeros(70, device="cuda", dtype=torch.bfloat16)
        with pytest.raises(ValueError, match=r"params\[1\]"):
            b.step(gs)
        assert b.steps == 2
    # moments that were given: their memory stays in use
    m = torch.zeros(300, device="cuda")
    opt = bm.AdamW([torch.zeros(300, device="cuda")], m=[m], v=[torch.zeros(300, device="cuda")])
    opt.step([torch.ones(300, device="cuda")])
    assert (m == opt.m[0]).all() and (m > 0).all()
    m.data = torch.ones(300, device="cuda")
    opt.step([torch.zeros(300, device="cuda")])
    assert (m == 1).all() and (opt.m[0] < 0.1).all()


def test_empty_tensors():
    import torch
    z = torch.zeros(0, device="cuda")
    opt = bm.AdamW([z, torch.ones(5, device="cuda")], bits=[8, 32])
    opt.step([z.clone(), torch.ones(5, device="cuda")])
    assert (opt.params[1] < 1).all() and opt.moments()[0][0].shape == (0,)


def test_binding_refusals():
    import torch
    z = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
    u8 = torch.uint8
    for kw in (dict(bits=16), dict(bits=[32]), dict(weight_decay=[0.1]), dict(copies=[None]), dict(copies=[z(8), None]), dict(m=[z(8), None]),
               dict(m=[z(8), z(4)]), dict(m=[z(8), z(4)], v=[z(8), z(5)]), dict(m_exp=[z(1, dtype=u8), None]), dict(seed=-1), dict(steps=-1),
               dict(betas=(0.9,)), dict(bits=8, m=[z(8, dtype=u8), None], v=[z(8, dtype=u8), None])):
        with pytest.raises(ValueError):
            bm.AdamW([z(8), z(4)], **kw)
    for params in ([z(8), z(4, dtype=torch.bfloat16)], [z(8, 4).t()], [z(8), torch.zeros(4)]):
        with pytest.raises(ValueError):
            bm.AdamW(params)
    opt = bm.AdamW([z(8), z(4)])
    for gs in ([z(8)], [z(8), z(5)], [z(8), torch.zeros(4)], [z(8), z(4).half()], [z(8), z(8)[::2]]):
        with pytest.raises(ValueError):
            opt.step(gs)
    with pytest.raises(ValueError):
        opt.step([z(8), z(4)], grad_scale=z(2))
    with pytest.raises(ValueError):
        opt.moments([z(8), None])
    x = z(8)
    with pytest.raises(bm.BmoeError, match="ALIAS"):
        bm.AdamW([x, x]).step([z(8), z(8)])
    with pytest.raises(bm.BmoeError, match="SHAPE"):
        bm.AdamW([x], betas=(1.0, 0.9)).step([z(8)])
    assert opt.steps == 0
