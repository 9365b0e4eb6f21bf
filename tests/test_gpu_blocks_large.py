"""Operators around a block on arrays of more than 2^32 values: the last rows (and some in
the middle) equal those of a call on them alone."""
import pytest

import compressed_mixture_experts_amd as bm
from gpu_helpers import log

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of GPU memory")
    yield
    torch.cuda.empty_cache()


def test_adamw_values_past_32_bits():
    import torch
    n, k = 2 ** 32 + 1029, 3000
    log(f"adamw n={n}")
    gen = torch.Generator().manual_seed(1)
    tail, g = torch.randn(k, generator=gen).cuda(), torch.randn(k, generator=gen).to(torch.bfloat16).cuda()
    p, grad = torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-k:], grad[-k:] = tail, g
    opt, small = bm.AdamW([p], bits=8, lr=0.1), bm.AdamW([tail.clone()], lr=0.1)
    opt.step([grad])
    small.step([g])
    assert (p[-k:] == small.params[0]).all() and not (p[-k:] == tail).any()
    assert (p[: 2 ** 20] == 0).all() and (p[2 ** 31 - 2 ** 20: 2 ** 31 + 2 ** 20] == 0).all()
    v = [torch.empty(n, dtype=torch.bfloat16, device="cuda")]
    opt.moments([torch.empty(n, dtype=torch.bfloat16, device="cuda")], v)
    assert ((v[0][-k:] > 0) == (small.v[0] > 0)).all() and (v[0][: 2 ** 20] == 0).all()


def test_block_norm_rows_past_32_bits():
    import torch
    rows, width, k = 2 ** 22 + 1003, 1032, 1500
    log(f"block norm rows={rows} width={width}")
    bf = torch.bfloat16
    gen = torch.Generator().manual_seed(2)
    small = [torch.randn(k, width, generator=gen).to(bf).cuda() for _ in range(4)]
    big = [torch.zeros(rows, width, dtype=bf, device="cuda") for _ in range(4)]
    for a, b in zip(big, small):
        a[-k:] = b
    gamma = torch.randn(width, generator=gen).cuda()
    kw = dict(kind="rms", gamma_post=gamma, gamma=gamma)
    y, s, st = bm.block_norm_forward(big[0], big[1], **kw)
    y1, s1, st1 = bm.block_norm_forward(small[0], small[1], **kw)
    for a, b in ((y, y1), (s, s1), (st, st1)):
        assert (a[-k:] == b).all()
    assert (y[: 2 ** 20] == 0).all()
    got = bm.block_norm_backward(big[2], big[0], s, st, d_sum=big[3], weight_grads=False, db=y, **kw)
    one = bm.block_norm_backward(small[2], small[0], s1, st1, d_sum=small[3], weight_grads=False, **kw)
    for name in ("b", "residual"):
        assert (got[name][-k:] == one[name]).all()


def test_gated_ffn_tokens_past_32_bits():
    """Values of a row do not depend on the tiles but for their last bits (h as bf16 may round
    otherwise at another order of sums): both within the roundings of one another."""
    import torch
    tokens, d, ff, k = 2 ** 20 + 77, 64, 2056, 500
    log(f"gated ffn tokens={tokens} d={d} ff={ff}")
    bf = torch.bfloat16
    gen = torch.Generator().manual_seed(3)
    xs, dys = (torch.randn(k, d, generator=gen).to(bf).cuda() for _ in range(2))
    w_in, w_down = (torch.randn(2 * ff, d, generator=gen) / 8).to(bf).cuda(), (torch.randn(d, ff, generator=gen) / 45).to(bf).cuda()
    x, dy = (torch.zeros(tokens, d, dtype=bf, device="cuda") for _ in range(2))
    x[-k:], dy[-k:] = xs, dys
    y, state = bm.gated_ffn_forward_train(x, w_in, w_down)
    y1, state1 = bm.gated_ffn_forward_train(xs, w_in, w_down)
    got = bm.gated_ffn_backward(x, w_in, w_down, dy, state)
    one = bm.gated_ffn_backward(xs, w_in, w_down, dys, state1)

    def near(a, b):
        # by norm: two roundings to bf16 on either side, 2^-8 of a value at most each
        a, b = a.double(), b.double()
        assert float((a - b).norm() / b.norm()) < 4 * 2.0 ** -8

    near(y[-k:], y1)
    near(got[0][-k:], one[0])
    near(got[1], one[1])
    near(got[2], one[2])
    assert (y[: 2 ** 16] == 0).all() and (got[0][: 2 ** 16] == 0).all() and (y[2 ** 19: 2 ** 19 + 2 ** 16] == 0).all()
