"""AdamW (include/bmoe_adamw.h) at the ends of fp32's range, against the fp64 oracle.

Bars as in test_gpu_adamw.py, and where v' is subnormal two units of fp32's lowest place beside
(its two products and their sum round there): v' is off by ev = 5 u v' + 2^-148, the divisor
by (ev / v' / 2 + 6 u) of itself, the step by that and 10 u of itself and by em's part of it.
"""
import numpy as np
import pytest

import compressed_mixture_experts_amd as bm
from oracle import ref
from gpu_helpers import log
from test_gpu_adamw import B1, B2, U, state64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("bits", [32, 8])
def test_subnormal_v_is_the_divisor(bits, eps):
    """Gradients of 2^-65 to 2^-55, some of them beside larger ones: v' from 2^-140 on."""
    import torch
    r = np.random.default_rng(7)
    g = (np.exp2(r.uniform(-65, -55, 5003)) * r.choice([-1.0, 1.0], 5003)).astype(np.float32)
    g[::97] = 1e-3
    p = torch.from_numpy(r.standard_normal(5003).astype(np.float32)).cuda()
    opt = bm.AdamW([p], bits=bits, lr=1e-2, eps=eps, weight_decay=0.0)
    g64 = g.astype(np.float64)
    for t in (1, 2):
        log(f"adamw subnormal v' bits={bits} eps={eps} step {t}")
        p0, m0, v0, _ = state64(opt, 0)
        opt.step([torch.from_numpy(g).cuda()])
        p1, _, _, _ = state64(opt, 0)
        want, m, v = ref.adamw(p0, g64, m0, v0, t, 1e-2, (B1, B2), eps, 0.0)
        # (in 8 bits a block's lowest v is 2^-33 of its largest from then on)
        assert t == 2 or ((v > 0) & (v < 2.0 ** -126)).sum() > 1000
        em, ev = 4 * U * (B1 * np.abs(m0) + (1 - B1) * np.abs(g64)), 5 * U * v + 2.0 ** -148
        by = 1e-2 / (1 - B1 ** t) / (np.sqrt(v / (1 - B2 ** t)) + eps)
        tol = (16 * U + ev / v / 2) * np.abs(by * m) + by * em + 3 * U * (np.abs(p0) + np.abs(want))
        assert np.isfinite(p1).all() and (np.abs(p1 - want) <= tol).all()


def test_finite_moments_stay_finite_in_8_bits():
    """Moments in fp32's last eighth below 2^128, whose next code up would be that of 2^128:
    with betas of 0 they are the gradient and its square, so all 2000 of them are known."""
    import torch
    r = np.random.default_rng(8)
    for size, which, top, largest in ((2.0 ** 128, 0, ref.ADAMW_M_TOP, 119), (2.0 ** 64, 1, ref.ADAMW_V_TOP, 247)):
        # m, or v's root, from the largest code's value (15/8 of 2^127) on
        lowest = 15 / 16 if which == 0 else np.sqrt(15 / 16)
        g = (size * r.uniform(lowest, 0.999999, 2000)).astype(np.float32) * (r.choice([-1, 1], 2000).astype(np.float32))
        opt = bm.AdamW([torch.zeros(2000, device="cuda")], bits=8, betas=(0.0, 0.0), lr=1e-3)
        opt.step([torch.from_numpy(g).cuda()])
        code = (opt.m if which == 0 else opt.v)[0].cpu().numpy()
        assert ((code & (127 if which == 0 else 255)) == largest).all()
        got = opt.moments()[which][0]
        assert torch.isfinite(got).all() and (got.abs().double() == 2.0 ** 127 * 15 / 8).all()
        if which == 0:
            assert ((got < 0).cpu().numpy() == (g < 0)).all()
        else:
            opt.step([torch.zeros(2000, device="cuda")])
            assert torch.isfinite(opt.params[0]).all()


def test_moments_in_bf16_down_to_its_smallest():
    """The codes' values in fp32 are those of their definition, in bf16 the nearest to them,
    also where bf16's numbers are further apart than codes."""
    import torch
    for size in (1.0, 1e-14, 1e-17, 1e-18):
        r = np.random.default_rng(9)
        g = (r.standard_normal(3000) * size * np.exp(2 * r.standard_normal(3000))).astype(np.float32)
        opt = bm.AdamW([torch.zeros(3000, device="cuda")], bits=8)
        opt.step([torch.from_numpy(g).cuda()])
        _, m, v, _ = state64(opt, 0)
        ms, vs = opt.moments()
        assert np.array_equal(ms[0].cpu().double().numpy(), m) and np.array_equal(vs[0].cpu().double().numpy(), v)
        m16, v16 = opt.moments(m_out=[torch.empty(3000, dtype=torch.bfloat16, device="cuda")])
        assert m16[0].dtype == v16[0].dtype == torch.bfloat16   # the new one is of the given one's type
        for x, y in ((ms[0], m16[0]), (vs[0], v16[0])):
            assert torch.equal(x.cpu().to(torch.bfloat16), y.cpu())
        exact = np.abs(v) >= 2.0 ** -130
        assert np.array_equal(v16[0].cpu().double().numpy()[exact], v[exact])
    assert ((v > 0) & ~exact).any()
