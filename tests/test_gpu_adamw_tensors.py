"""The tensors that an AdamW object holds: what their owner does to them between steps."""
import pytest

import compressed_mixture_experts_amd as bm
from test_gpu_adamw import make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


def test_a_layout_that_changed_at_the_same_address():
    """Parameters and copies that are transposed, cut or read as another type in place."""
    import torch
    for bits in (32, 8):
        for name, change in ((r"params\[1\]", lambda o: o.params[1].data.t()), (r"params\[1\]", lambda o: o.params[1].data[:8]),
                             (r"params\[1\]", lambda o: o.params[1].data.view(8, 32)),
                             (r"params\[1\]", lambda o: o.params[1].data.view(torch.bfloat16)[:, :16]),
                             (r"copies\[1\]", lambda o: o.copies[1].data.t()), (r"copies\[1\]", lambda o: o.copies[1].data.view(torch.float16))):
            ps = [torch.ones(40, device="cuda"), torch.arange(256.0, device="cuda").view(16, 16)]
            opt = bm.AdamW(ps, bits=bits, copies=[None, torch.zeros(16, 16, dtype=torch.bfloat16, device="cuda")])
            gs = [torch.ones(40, device="cuda"), torch.ones(16, 16, device="cuda")]
            opt.step(gs)
            held = opt.params[1] if name.startswith("params") else opt.copies[1]
            whole, memory = held.data, held.data.clone()
            held.data = change(opt)
            assert held.data_ptr() == whole.data_ptr()
            with pytest.raises(ValueError, match=name):
                opt.step(gs)
            torch.cuda.synchronize()
            assert opt.steps == 1 and (whole == memory).all()
            held.data = whole
            opt.step(gs)
            assert opt.steps == 2 and not (whole == memory).all()


def test_autograd_is_told():
    """A step raises the version of what it changes, and of nothing else: a graph that saved a
    parameter or a copy refuses its backward."""
    import torch
    g = torch.ones(8, device="cuda")
    for kind in ("params", "copies"):
        p = [torch.nn.Parameter(torch.ones(8, device="cuda")) for _ in range(3)]
        c = [torch.zeros(8, dtype=torch.bfloat16, device="cuda", requires_grad=True), None, None]
        opt = bm.AdamW(p, copies=c)
        for grads, told in (([g, g, g], True), ([g, None, g], True), ([None, g, g], False), ([None, None, None], False)):
            held = (opt.params if kind == "params" else opt.copies)[0]
            x = torch.ones(8, device="cuda", dtype=held.dtype, requires_grad=True)
            y = (x * held).sum()
            before = [t._version for t in opt.params]
            opt.step(grads)
            assert [t._version > b for t, b in zip(opt.params, before)] == [q is not None for q in grads]
            if told:
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    y.backward()
            else:
                y.backward()
                assert torch.equal(x.grad, held.detach())
    with torch.inference_mode():   # tensors without a version
        p = torch.ones(8, device="cuda")
        opt = bm.AdamW([p])
        opt.step([g])
        assert (p < 1).all()


def test_moments_that_go_together():
    """Some of m, v, m_exp and v_exp without the others: refused, whichever they are."""
    import itertools
    import torch
    z = lambda n, kind=torch.uint8: torch.zeros(n, dtype=kind, device="cuda")  # noqa: E731
    for keep in itertools.product((False, True), repeat=4):
        kw = {k: [x] for k, x, on in zip(("m", "v", "m_exp", "v_exp"), (z(300), z(300), z(2), z(2)), keep) if on}
        if all(keep) or not any(keep):
            bm.AdamW([z(300, torch.float32)], bits=8, **kw).step([z(300, torch.float32)])
        else:
            with pytest.raises(ValueError, match="go together"):
                bm.AdamW([z(300, torch.float32)], bits=8, **kw)
    for kw in (dict(m=[z(300, torch.float32)]), dict(v=[z(300, torch.float32)])):
        with pytest.raises(ValueError, match="m and v of parameter 0 go together"):
            bm.AdamW([z(300, torch.float32)], **kw)


def test_moments_into_what_is_no_tensor():
    import torch
    opt = bm.AdamW([torch.zeros(300, device="cuda")], bits=8)
    for out in ([1.0], ["m"], [torch.zeros(300)], [torch.zeros(300, dtype=torch.float16, device="cuda")]):
        with pytest.raises(ValueError, match=r"m_out\[0\]"):
            opt.moments(m_out=out)
        with pytest.raises(ValueError, match=r"v_out\[0\]"):
            opt.moments(v_out=out)
