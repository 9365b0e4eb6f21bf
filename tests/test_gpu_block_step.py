"""One training step of a model's block as a program runs it: the norms around an expert
layer, the layer with a dense gated block beside it, their backward, AdamW over everything
that is trained, and the layer prepared again; each link against the 64-bit oracle at the
inputs that it gets here, and the whole step captured in a graph."""
import pytest

import compressed_mixture_experts_amd as bm
from compressed_mixture_experts_amd import workloads as wl
from gpu_helpers import log, to_dev, to_f64
from test_gpu_adamw import check_step, state64
from test_gpu_block_norm import check_backward, check_forward
from test_gpu_gated_ffn import U, Want, near

pytestmark = pytest.mark.gpu
D, FF, T = 256, 520, 203


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    bm.lib()
    yield


class Block:
    """A block's weights and one step of them."""

    def __init__(self, capturable=False):
        import torch
        g = torch.Generator().manual_seed(5)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        inp = wl.generate(wl.small_config(d_model=D, d_ff=0, n_experts=6, top_k=2, tokens=T, act="bf16", seed_index=950))
        self.inp = inp
        self.layer = bm.Layer.from_inputs(inp, device="cuda").prepare()
        bf = torch.bfloat16
        self.b0, self.r0 = n(T, D).to(bf).cuda(), (2 * n(T, D)).to(bf).cuda()
        self.dn, self.ds = n(T, D).to(bf).cuda(), n(T, D).to(bf).cuda()
        self.norms = [dict(kind="rms", alpha=1.0, scale=0.9, gate=(0.5 + 0.1 * n(D)).cuda(), gamma_post=(1 + 0.1 * n(D)).cuda(), gamma=(1 + 0.1 * n(D)).cuda())
                      for _ in range(2)]
        self.w_gate = self.layer.w_gate.float()
        self.w_in, self.w_down = (n(2 * FF, D) / D ** 0.5).cuda(), (n(D, FF) / FF ** 0.5).cuda()
        self.in16, self.down16 = self.w_in.to(bf), self.w_down.to(bf)
        small = [k[name] for k in self.norms for name in ("gamma_post", "gate", "gamma")]
        params = [self.layer.theta[0], self.layer.phi[0], self.w_gate, self.w_in, self.w_down] + small
        self.opt = bm.AdamW(params, lr=1e-2, weight_decay=[0.0, 0.0, 0.01, 0.1, 0.1] + [0.0] * 6, bits=[32, 8, 32, 8, 8] + [32] * 6,
                            copies=[None, None, self.layer.w_gate, self.in16, self.down16] + [None] * 6, seed=3, capturable=capturable)

    def step(self, keep=None):
        a, b = self.norms
        n, s, st = bm.block_norm_forward(self.b0, self.r0, **a)
        ye, state = self.layer.forward_train(n)
        y, fst = bm.gated_ffn_forward_train(n, self.in16, self.down16, add=ye)
        n2, s2, st2 = bm.block_norm_forward(y, s, **b)
        g2 = bm.block_norm_backward(self.dn, y, s2, st2, d_sum=self.ds, **b)
        ge = self.layer.backward(n, g2["b"], state)
        dx, dwi, dwd = bm.gated_ffn_backward(n, self.in16, self.down16, g2["b"], fst, dx_add=ge["x"])
        g1 = bm.block_norm_backward(dx, self.b0, s, st, d_sum=g2["residual"], **a)
        grads = [ge["theta"][0], ge["phi"][0], ge["w_gate"], dwi, dwd] + [g[k] for g in (g1, g2) for k in ("gamma_post", "gate", "gamma")]
        if keep is not None:
            keep.update(n=n, s=s, st=st, ye=ye, y=y, n2=n2, s2=s2, st2=st2, g2=g2, ge=ge, dx=dx, dwi=dwi, dwd=dwd, g1=g1, grads=grads,
                        in16=self.in16.clone(), down16=self.down16.clone(), norms=[{k: (v.clone() if hasattr(v, "clone") else v) for k, v in x.items()} for x in self.norms])
        self.opt.step(grads)
        self.layer.refresh()
        return grads, n2, s2


def test_every_link():
    import torch
    m = Block()
    for t in (1, 2):
        log(f"block step {t}")
        k = {}
        before = [state64(m.opt, i) for i in range(len(m.opt.params))]
        m.step(k)
        links = ((m.b0, m.r0, (k["n"], k["s"], k["st"]), k["dx"], k["g2"]["residual"], k["g1"]),
                 (k["y"], k["s"], (k["n2"], k["s2"], k["st2"]), m.dn, m.ds, k["g2"]))
        for (b, r, out, dy, ds, got), norm in zip(links, k["norms"]):
            c = dict(b=b, r=r, dt=torch.bfloat16, kind="rms", post=True, gate=norm["gate"], gp=norm["gamma_post"], bp=None, ga=norm["gamma"], be=None)
            check_forward(c, out, 1.0, 0.9, True)
            check_backward(c, got, out[1], out[2], dy, ds, 1.0, 0.9)
        w = Want(dict(x=k["n"], w_in=k["in16"], w_down=k["down16"]), "silu")
        ye, dxe = k["ye"].double(), k["ge"]["x"].double()
        near("y", k["y"], w.y + ye, w.ey + 2 * U * (w.y.abs() + ye.abs()))
        (dx, ex), (dwi, ewi), (dwd, ewd) = w.backward(k["g2"]["b"])
        near("dx", k["dx"], dx + dxe, ex + 2 * U * (dx.abs() + dxe.abs()))
        near("dw_in", k["dwi"], dwi, ewi)
        near("dw_down", k["dwd"], dwd, ewd)
        for i, g in enumerate(k["grads"]):
            check_step(m.opt, i, before[i], to_f64(g).ravel(), t, 1e-2, m.opt._decay[i], 3)
        # the layer goes on with the new weights, as one built from them does
        x = to_dev(m.inp.x, "bf16")
        fresh = bm.Layer.from_inputs(m.inp, device="cuda")
        for own, new in ((fresh.theta[0], m.layer.theta[0]), (fresh.phi[0], m.layer.phi[0]), (fresh.w_gate, m.layer.w_gate)):
            own.copy_(new)
        assert (m.layer.forward(x) == fresh.prepare().forward(x)).all()
    assert m.opt.steps == 2


def test_captured_step():
    """The whole step as a graph, replayed with eager work between: every replay equals a
    step of a block of its own."""
    import torch
    m, eager = Block(capturable=True), Block()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.step()
    torch.cuda.current_stream().wait_stream(s)
    eager.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads, n2, s2 = m.step()
    for _ in range(3):
        graph.replay()
        want, wn, ws = eager.step()
        torch.cuda.synchronize()
        for a, b in zip(grads + [n2, s2] + m.opt.params, want + [wn, ws] + eager.opt.params):
            # equal to the last bit: the bias corrections too, in fp64 on the GPU and on the host
            assert (a == b).all()
    assert m.opt.steps == eager.opt.steps == 4
