"""The dense operators together, as a layer with routed and shared experts uses
them: router product, top-k, balance losses, the routed layer, the shared
expert (SwiGLU, its input kept in 8 bits) added to the routed output, and the
gradients of all of it -- against torch autograd in 64 bits, and captured in one
graph."""
import numpy as np
import pytest
import torch

from gpu_util import abi, say, synth

pytestmark = pytest.mark.gpu


class Layer:
    """T tokens, hidden size d, E experts (top K) of f, a shared expert of fs"""

    def __init__(self, T, d, E, K, f, fs, dtype, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(dtype)  # noqa: E731
        self.T, self.K, self.E, self.dtype = T, K, E, dtype
        self.x, self.wr, self.br = n(T, d), n(d, E, std=d ** -0.5), n(E, std=0.3)
        self.eg, self.eu, self.ed = (n(E, d, f, std=d ** -0.5), n(E, d, f, std=d ** -0.5),
                                     n(E, f, d, std=f ** -0.5))
        self.wg, self.wu, self.wd = n(d, fs, std=d ** -0.5), n(d, fs, std=d ** -0.5), n(fs, d, std=fs ** -0.5)
        self.bd = n(d, std=0.1)
        self.dy = n(T, d, std=0.2)
        self.dw = torch.randn((T, K), generator=g, device="cuda")
        self.dloss = torch.tensor([0.5 * T, 0.01 * T], device="cuda")
        self.kept = {}

    def step(self):
        """one forward and backward pass; everything it returns is on the GPU"""
        k, ws = self.kept, self.kept.get
        logits, k["a"] = abi.linear(self.x, self.wr, bias=self.br, out_dtype=torch.float32,
                                    workspace=ws("a"))
        ids, w = abi.route(logits, self.K)
        bal, k["b"] = abi.balance_loss(logits, ids, workspace=ws("b"))
        routed, k["c"] = abi.forward(self.x, ids, w, self.eg, self.eu, self.ed, workspace=ws("c"))
        gate, k["d"] = abi.linear(self.x, self.wg, workspace=ws("d"))
        up, k["e"] = abi.linear(self.x, self.wu, workspace=ws("e"))
        h, ck = abi.act_forward(gate, up, act="silu", ckpt=True)
        y, k["f"] = abi.linear(h, self.wd, bias=self.bd, residual=routed, out_dtype=torch.float32,
                               workspace=ws("f"))
        # backward: gate, up and h are gone, the checkpoint stands for them
        back, k["g"] = abi.linear_backward(None, self.wd, self.dy, grads=("dx", "db"),
                                           grad_dtype=torch.float32, workspace=ws("g"))
        act = abi.act_backward(ck, back["dx"], act="silu")
        down, k["h"] = abi.linear_backward(act["h"], None, self.dy, grads=("dw",),
                                           grad_dtype=torch.float32, workspace=ws("h"))
        dg, k["i"] = abi.linear_backward(self.x, self.wg, act["dg"], grads=("dx", "dw"),
                                         grad_dtype=torch.float32, workspace=ws("i"))
        du, k["j"] = abi.linear_backward(self.x, self.wu, act["du"], grads=("dx", "dw"),
                                         grad_dtype=torch.float32, workspace=ws("j"))
        dl = abi.route_backward(logits, ids, w, self.dw, bal["cnt"], self.dloss,
                                out_dtype=self.dtype)
        dr, k["l"] = abi.linear_backward(self.x, self.wr, dl, grad_dtype=torch.float32,
                                         workspace=ws("l"))
        return dict(logits=logits, ids=ids, w=w, routed=routed, y=y, loss=bal["loss"],
                    cnt=bal["cnt"], wd=down["dw"], bd=back["db"], wg=dg["dw"], wu=du["dw"],
                    wr=dr["dw"], br=dr["db"], dl=dl, x_gate=dg["dx"], x_up=du["dx"],
                    x_router=dr["dx"])

    def reference(self, got):
        """the same from torch autograd in 64 bits on the CPU, with the routing and the
        routed experts' output as the GPU gave them"""
        c = lambda t: t.detach().cpu().double()  # noqa: E731
        leaf = {k: c(getattr(self, k)).requires_grad_() for k in ("wr", "br", "wg", "wu", "wd", "bd")}
        xs = {k: c(self.x).requires_grad_() for k in ("x_router", "x_gate", "x_up")}
        ids, dw = got["ids"].cpu().long(), c(self.dw)
        logits = xs["x_router"] @ leaf["wr"] + leaf["br"]
        p = torch.softmax(logits, dim=1)
        f = torch.bincount(ids.reshape(-1), minlength=self.E).double() / ids.numel()
        loss = torch.stack([self.E * (f * p.mean(dim=0)).sum(),
                            torch.logsumexp(logits, dim=1).square().mean()])
        w = torch.softmax(torch.gather(logits, 1, ids), dim=1)
        h = torch.nn.functional.silu(xs["x_gate"] @ leaf["wg"]) * (xs["x_up"] @ leaf["wu"])
        y = h @ leaf["wd"] + leaf["bd"] + c(got["routed"])
        ((y * c(self.dy)).sum() + (w * dw).sum() + (loss * c(self.dloss)).sum()).backward()
        want = {k: v.grad for k, v in {**leaf, **xs}.items()}
        return dict(want, logits=logits.detach(), loss=loss.detach(), y=y.detach(), w=w.detach())


def rel(a, b):
    a, b = a.detach().cpu().double(), b.double()
    return float((a - b).norm() / b.norm())


@pytest.mark.parametrize("T,d,E,K,f,fs", [(96, 128, 8, 2, 256, 192), (300, 320, 30, 4, 64, 200)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_layer_step(T, d, E, K, f, fs, dtype):
    say(f"[dense layer] T={T} d={d} E={E} K={K} f={f} fs={fs} {dtype}")
    layer = Layer(T, d, E, K, f, fs, dtype, seed=T)
    got = layer.step()
    torch.cuda.synchronize()
    want = layer.reference(got)
    half = torch.finfo(dtype).eps / 2
    # 32-bit results of one product: sums of at most 2^9 terms
    assert rel(got["logits"], want["logits"]) < 2.0 ** -14
    assert rel(got["loss"], want["loss"]) < 2.0 ** -14 and rel(got["w"], want["w"]) < 2.0 ** -13
    # y: gate, up and h each rounded to the type (half a step, independent), so at
    # most 3 halves of the shared part; fp32 sums besides
    assert rel(got["y"], want["y"]) < 3 * half + 2.0 ** -14
    # behind the checkpoint every value is off by up to 2^-4 of itself (values far
    # below their block's largest by more, but they weigh less): gate and up in one
    # product, act' with slope up to 1 beside it
    for k in ("wd", "wg", "wu", "x_gate", "x_up"):
        assert rel(got[k], want[k]) < 2.0 ** -3, (k, rel(got[k], want[k]))
    # the router's gradients see dlogits rounded once to the type, x and w not at all
    for k in ("wr", "br", "x_router"):
        assert rel(got[k], want[k]) < 2 * half + 2.0 ** -12, (k, rel(got[k], want[k]))
    assert rel(got["bd"], want["bd"]) < 2.0 ** -14


def test_layer_step_in_a_graph():
    """the whole step captured once (workspaces kept from the eager call) and replayed on
    new inputs between eager steps: the eager bits each time"""
    layer = Layer(160, 256, 16, 2, 64, 128, torch.bfloat16, seed=3)
    layer.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step()
    other = Layer(160, 256, 16, 2, 64, 128, torch.bfloat16, seed=3)
    for rep in range(3):
        new = torch.randn(layer.x.shape, device="cuda").to(torch.bfloat16)
        layer.x.copy_(new)
        other.x.copy_(new)
        for v in layer.kept.values():
            v.fill_(0xA5)
        want = other.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), (rep, k)


def test_decode_step_in_a_graph_with_the_configs_sizes():
    """serving, 4 tokens of the decode workload's sizes: router product to routed layer to
    shared expert, replayed"""
    cfg = synth.CONFIGS["decode_bf16"]
    g = torch.Generator(device="cuda").manual_seed(1)
    n = lambda *s, std: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)  # noqa: E731
    x, wr = n(cfg.T, cfg.d, std=1.0), n(cfg.d, cfg.E, std=cfg.d ** -0.5)
    eg, eu = n(cfg.E, cfg.d, cfg.f, std=0.02), n(cfg.E, cfg.d, cfg.f, std=0.02)
    ed = n(cfg.E, cfg.f, cfg.d, std=0.02)
    wg, wu, wd = n(cfg.d, cfg.f, std=0.02), n(cfg.d, cfg.f, std=0.02), n(cfg.f, cfg.d, std=0.02)
    kept = {}

    def step():
        logits, kept["a"] = abi.linear(x, wr, out_dtype=torch.float32, workspace=kept.get("a"))
        ids, w = abi.route(logits, cfg.K)
        routed, kept["b"] = abi.forward(x, ids, w, eg, eu, ed, workspace=kept.get("b"))
        gate, kept["c"] = abi.linear(x, wg, workspace=kept.get("c"))
        up, kept["d"] = abi.linear(x, wu, workspace=kept.get("d"))
        h, _ = abi.act_forward(gate, up)
        return abi.linear(h, wd, residual=routed, out=routed, workspace=kept.setdefault(
            "e", torch.empty(1 << 22, dtype=torch.uint8, device="cuda")))[0]

    want = step().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        again = step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(again, want)
