"""Which kernels the dense gated block takes (bmoe_dbg_gated_ffn_plan).  No GPU needed."""
import ctypes
import math
import random

import pytest

import compressed_mixture_experts_amd as bm
from gated_ffn_cases import SHAPES, kernels


def test_the_tested_sizes_take_every_kernel():
    """Every kernel that one of 20000 sizes of up to 20000 tokens takes is one that a GPU test's
    size takes: a change of the estimate behind the dispatch that leaves one out fails here."""
    from test_gpu_gated_ffn import SHAPES as OLDER
    tested = set().union(*(kernels(*s) for s in SHAPES + OLDER))
    r = random.Random(5)
    seen = {}
    for _ in range(20000):
        size = (int(math.exp(r.uniform(0, math.log(20000)))), 8 * int(math.exp(r.uniform(0, math.log(512)))), 8 * int(math.exp(r.uniform(0, math.log(1024)))))
        for k in kernels(*size):
            seen.setdefault(k, size)
    assert len({k[:2] for k in seen}) == 20   # five products (the two weight gradients are alike) in four tile forms
    assert not {k: s for k, s in seen.items() if k not in tested}


def test_a_plan_is_whole():
    """Shares have a step each, and a product in shares has partial sums."""
    r = random.Random(6)
    for _ in range(5000):
        t, d, ff = r.randint(1, 20000), 8 * r.randint(1, 500), 8 * r.randint(1, 1000)
        p = bm.dbg_gated_ffn_plan(t, d, ff)
        assert p["few"] == (t <= 4)
        for depth, form, shares in zip((ff, 2 * ff, t, t), [p["y"], *p["last"]], [p["y_shares"], *p["last_shares"]]):
            for step in (64, 32):
                steps = -(-depth // step)
                per = -(-steps // shares)
                assert 0 <= form <= 3 and (shares - 1) * per < steps
        assert not p["joint"] or p["joint_parts"] or p["last_shares"] == [1, 1, 1]


def test_plan_refusals():
    D, p = bm.debug_lib(), (ctypes.c_int32 * 13)()
    for size in ((-1, 8, 8), (1, 4, 8), (1, 8, 12), (1, 16392, 8), (1, 8, 65544), (1, 16384, 65536)):
        assert D.bmoe_dbg_gated_ffn_plan(*size, ctypes.byref(p)) == 2
        with pytest.raises(bm.BmoeError, match="SHAPE"):
            bm.dbg_gated_ffn_plan(*size)
    assert D.bmoe_dbg_gated_ffn_plan(1, 8, 8, None) == 1
    assert bm.dbg_gated_ffn_plan(0, 8, 8)["y_shares"] == 0   # no tokens, no kernels
