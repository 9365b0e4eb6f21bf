"""Which activation the gated block's backward (include/bmoe_ffn.h) is the backward of."""
import pytest

import compressed_mixture_experts_amd as bm
from test_gpu_gated_ffn import Want, draw, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


@pytest.mark.parametrize("tokens,d,ff", [(3, 64, 128), (65, 72, 136), (300, 40, 1000), (2049, 264, 1000)])
def test_the_state_s_own(tokens, d, ff):
    import torch
    c = draw(tokens, d, ff, 30)
    states = {act: bm.gated_ffn_forward_train(c["x"], c["w_in"], c["w_down"], act)[1] for act in ("silu", "gelu")}
    got = {(made, named): bm.gated_ffn_backward(c["x"], c["w_in"], c["w_down"], c["dy"], states[made], named) for made in states for named in states}
    for made in states:
        for (want, off), g, h in zip(Want(c, made).backward(c["dy"]), got[made, "silu"], got[made, "gelu"]):
            assert torch.equal(g, h)
            near(f"{made}", g, want, off)
    assert not torch.equal(got["silu", "silu"][0], got["gelu", "gelu"][0])
