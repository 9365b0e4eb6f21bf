"""The dense gated block in every kernel that its dispatch knows (gated_ffn_cases.py; a CPU test
holds the sizes to that), with the bars of test_gpu_gated_ffn.py.  Outputs stand in front
of values that stay as they are."""
import pytest

import compressed_mixture_experts_amd as bm
from gated_ffn_cases import SHAPES
from gpu_helpers import log
from test_gpu_gated_ffn import U, Want, draw, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("tokens,d,ff", SHAPES)
def test_every_kernel(tokens, d, ff, act):
    import torch
    log(f"gated ffn tokens={tokens} d={d} ff={ff} {act}")
    c = draw(tokens, d, ff, tokens + 3 * d + ff)
    w = Want(c, act)

    def room(like):
        """An output, and 1000 values behind it."""
        flat = torch.full((like.numel() + 1000,), 7.0, dtype=torch.bfloat16, device="cuda")
        return flat[:like.numel()].view(like.shape), flat[like.numel():]

    x, wi, wd = c["x"], c["w_in"], c["w_down"]
    y, tail = room(x)
    assert bm.gated_ffn_forward(x, wi, wd, act, y=y) is y
    near("y", y, w.y, w.ey)
    assert (tail == 7.0).all()
    y, tail = room(x)
    _, state = bm.gated_ffn_forward_train(x, wi, wd, act, add=c["add"], y=y)
    near("y + add", y, w.y + c["add"].double(), w.ey + 2 * U * (w.y.abs() + c["add"].double().abs()))
    assert (tail == 7.0).all()
    outs = [room(t) for t in (x, wi, wd)]
    add = c["dx_add"].double()
    dx, dwi, dwd = bm.gated_ffn_backward(x, wi, wd, c["dy"], state, act, dx_add=c["dx_add"], **dict(zip(("dx", "dw_in", "dw_down"), (o[0] for o in outs))))
    (wx, ex), (wwi, ewi), (wwd, ewd) = w.backward(c["dy"])
    near("dx", dx, wx + add, ex + 2 * U * (wx.abs() + add.abs()))
    near("dw_in", dwi, wwi, ewi)
    near("dw_down", dwd, wwd, ewd)
    assert all((o[1] == 7.0).all() for o in outs)
    # each alone and both together give the same
    only = bm.gated_ffn_backward(x, wi, wd, c["dy"], state, act, dx_add=c["dx_add"], weight_grads=False)
    weights = bm.gated_ffn_backward(x, wi, wd, c["dy"], state, act, input_grad=False)
    assert torch.equal(only[0], dx) and torch.equal(weights[1], dwi) and torch.equal(weights[2], dwd)
