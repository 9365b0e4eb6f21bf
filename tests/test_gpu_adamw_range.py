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
