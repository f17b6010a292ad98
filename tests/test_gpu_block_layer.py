"""The operators around the block together, as a training step and a decode step use
them: norm, router product, routing by scores, the routed layer with 4-bit weights, the
norm behind it with gate and residual, and the gradients back to the residual stream --
against torch in 64 bits, and captured in graphs; each on other streams, two at once."""
import numpy as np
import pytest
import torch

from gpu_util import abi, say

pytestmark = pytest.mark.gpu
F32 = torch.float32


class Block:
    def __init__(self, T, d, E, K, f, dtype, seed, groups=4):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std  # noqa: E731
        h = lambda *s, std=1.0: n(*s, std=std).to(dtype)  # noqa: E731
        self.E, self.K, self.f, self.dtype = E, K, f, dtype
        self.r = n(T, d)
        self.wr, self.bias = h(d, E, std=d ** -0.5), n(E, std=0.05)
        self.pre, self.post, self.next = (1 + h(d, std=0.1) for _ in range(3))
        self.gate = torch.sigmoid(n(T)).to(dtype)
        ws = n(E, d, f, std=d ** -0.5), n(E, d, f, std=d ** -0.5), n(E, f, d, std=f ** -0.5)
        self.packed = abi.pack_mx4(*ws)
        self.values = [abi.mx4_dequantize(self.packed[k], E, d, f, kind, dtype=dtype)
                       for k, kind in (("gate", "gate"), ("up", "gate"), ("down", "down"))]
        self.dz, self.dh2, self.dw = n(T, d, std=0.3), h(T, d, std=0.3), n(T, K)
        self.dr_add = h(T, E, std=0.01)
        self.how = dict(score="sigmoid", groups=groups, keep=max(1, groups // 2), group_top=2,
                        scale=2.5)
        self.kept = {}

    def step(self, train=True):
        k, ws = self.kept, self.kept.get
        a = abi.norm(self.r, w_pre=self.pre, stats=True)
        logits, k["a"] = abi.linear(a["h"], self.wr, out_dtype=F32, workspace=ws("a"))
        ids, w = abi.route_scored(logits, self.K, bias=self.bias, **self.how)
        y, k["b"] = abi.forward_mx4(a["h"], ids, w, self.packed, self.E, self.f, out_dtype=F32,
                                    workspace=ws("b"))
        c = abi.norm(self.r, y=y, w_post=self.post, gate=self.gate, gate_kind="token",
                     w_pre=self.next, alpha=0.5, stats=True)
        out = dict(h=a["h"], logits=logits, ids=ids, w=w, y=y, z=c["z"], h2=c["h"])
        if not train:
            return out
        back, k["c"] = abi.norm_backward(c["z"], c["stats"], dz=self.dz, dh=self.dh2, y=y,
                                         w_post=self.post, gate=self.gate, gate_kind="token",
                                         w_pre=self.next, alpha=0.5, grad_dtype=F32,
                                         workspace=ws("c"))
        dl = abi.route_scored_backward(logits, ids, self.dw, score="sigmoid", scale=2.5,
                                       add=self.dr_add)
        lin, k["d"] = abi.linear_backward(a["h"], self.wr, dl, grads=("dx", "dw"),
                                          grad_dtype=F32, workspace=ws("d"))
        first, k["e"] = abi.norm_backward(self.r, a["stats"], dz=back["dr"], dh=lin["dx"],
                                          w_pre=self.pre, grad_dtype=F32, workspace=ws("e"))
        return {**out, **{"2" + n: v for n, v in back.items()}, "dl": dl, "dwr": lin["dw"],
                **{"1" + n: v for n, v in first.items()}}


def norm64(v, w):
    return v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + 1e-6) * w


def reference(b, got):
    """The same step in 64 bits; each part takes what the one before it gave (its roundings
    are not followed through the step), gradients by autograd"""
    D = lambda t: t.detach().cpu().double()  # noqa: E731
    ref = {}
    r = D(b.r).requires_grad_()
    pre = D(b.pre).requires_grad_()
    wr = D(b.wr).requires_grad_()
    h = norm64(r, pre)
    ref["h"] = h
    hk = D(got["h"]).requires_grad_()
    logits = hk @ wr
    ref["logits"] = logits
    lk = D(got["logits"]).requires_grad_()
    ids = got["ids"].cpu().long()
    s = torch.sigmoid(lk).gather(1, ids)
    w = 2.5 * s / s.sum(dim=1, keepdim=True)
    ref["w"] = w
    (dl,) = torch.autograd.grad(w, lk, D(b.dw))
    ref["dl"] = dl + D(b.dr_add)
    wg, wu, wd = (D(v) for v in b.values)
    x, wk = D(got["h"]), D(got["w"])
    y = torch.zeros_like(x)
    for e in range(b.E):
        t, k = torch.nonzero(ids == e, as_tuple=True)
        g = x[t] @ wg[e]
        y.index_add_(0, t, wk[t, k][:, None] * ((g * torch.sigmoid(g) * (x[t] @ wu[e])) @ wd[e]))
    ref["y"] = y
    yk, post, nxt, gate = (D(t).requires_grad_() for t in (got["y"], b.post, b.next, b.gate))
    r2 = D(b.r).requires_grad_()
    z = r2 + 0.5 * gate[:, None] * norm64(yk, post)
    h2 = norm64(z, nxt)
    ref["z"], ref["h2"] = z, h2
    grads = torch.autograd.grad([z, h2], [r2, yk, gate, post, nxt], [D(b.dz), D(b.dh2)])
    for name, v in zip(("2dr", "2dy", "2dgate", "2dw_post", "2dw_pre"), grads):
        ref[name] = v
    dlk = D(got["dl"])
    dh, ref["dwr"] = torch.autograd.grad(logits, [hk, wr], dlk)
    dr, ref["1dw_pre"] = torch.autograd.grad(h, [r, pre], dh)
    ref["1dr"] = dr + D(got["2dr"])
    return ref


HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("T", [1, 4, 61, 300])
def test_training_step(T, dtype):
    say(f"[block] training step {T} {dtype}")
    b = Block(T, 328, 16, 3, 200, dtype, seed=T)
    got = b.step()
    ref = reference(b, got)
    for k, want in ref.items():
        want = want.detach()
        off = float((got[k].detach().cpu().double() - want).norm() / want.norm())
        # one rounding of the result; in y one of h besides (and of what it is kept in), in the
        # gradient that reaches the first norm that of dx; fp32 sums of some hundred terms
        half = HALF[got[k].dtype]
        tol = half + 200 * 2.0 ** -24
        if k in ("y", "1dr", "1dw_pre"):
            tol += 3 * HALF[dtype]
        assert off <= tol, (k, off, tol)
    c = torch.sigmoid(got["logits"].double()) + b.bias.double()
    best = torch.topk(c.view(T, 4, 4), 2, dim=2)[0].sum(dim=2)
    open_ = torch.zeros((T, 4), device="cuda").scatter_(1, best.topk(2, dim=1)[1], 1.0).bool()
    c = c.masked_fill(~open_.repeat_interleave(4, dim=1), -9.0)
    assert torch.equal(got["ids"].long(), c.topk(3, dim=1)[1])


@pytest.mark.parametrize("train", [True, False])
@pytest.mark.parametrize("T", [1, 4, 300])
def test_captured_steps(T, train):
    say(f"[block] graph {T} {train}")
    b = Block(T, 264, 16, 3, 136, torch.bfloat16, seed=7 + T)
    inputs = [t.clone() for t in (b.r, b.dz, b.dw)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.step(train)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = b.step(train)
    for turn in range(4):  # the program's own work between the replays
        for t, keep in zip((b.r, b.dz, b.dw), inputs):
            t.copy_(keep * (1 + turn))
        eager = b.step(train)
        for v in got.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(got[k], eager[k]), (turn, k)


def calls():
    b = Block(130, 264, 16, 3, 136, torch.float16, seed=5)
    out = b.step()
    y = out["y"]
    stats = abi.norm(b.r, y=y, w_post=b.post, w_pre=b.next, stats=True)["stats"]
    t = dict(r=b.r, y=y, post=b.post, next=b.next, stats=stats, z=out["z"], dz=b.dz, dh=b.dh2,
             logits=out["logits"], bias=b.bias, ids=out["ids"], w=out["w"], dw=b.dw, h=out["h"],
             wg=b.values[0], **{"p" + k: v for k, v in b.packed.items()})
    pk = lambda q: {k: q["p" + k] for k in ("gate", "up", "down")}  # noqa: E731
    fns = {
        "norm": lambda q, s: abi.norm(q["r"], y=q["y"], w_post=q["post"], w_pre=q["next"],
                                      stats=True, stream=s),
        "norm_backward": lambda q, s: abi.norm_backward(
            q["z"], q["stats"], dz=q["dz"], dh=q["dh"], y=q["y"], w_post=q["post"],
            w_pre=q["next"], grad_dtype=F32, stream=s)[0],
        "route_scored": lambda q, s: abi.route_scored(q["logits"], 3, bias=q["bias"], groups=4,
                                                      keep=2, score="sigmoid", stream=s),
        "route_scored_backward": lambda q, s: abi.route_scored_backward(
            q["logits"], q["ids"], q["dw"], renorm=False, stream=s),
        "mx4_quantize": lambda q, s: abi.mx4_quantize(q["wg"], "gate", stream=s),
        "mx4_dequantize": lambda q, s: abi.mx4_dequantize(q["pgate"], 16, 264, 136, "gate",
                                                          stream=s),
        "forward_mx4": lambda q, s: abi.forward_mx4(q["h"], q["ids"], q["w"], pk(q), 16, 136,
                                                    stream=s)[0],
    }
    return t, fns


def flat(v):
    if torch.is_tensor(v):
        return [v]
    return [t for k in sorted(v) for t in flat(v[k])] if isinstance(v, dict) else \
        [t for q in v for t in flat(q)]


NAMES = ["norm", "norm_backward", "route_scored", "route_scored_backward", "mx4_quantize",
         "mx4_dequantize", "forward_mx4"]


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_another_stream(name, handle):
    """inputs arrive on that stream behind long copies: work on any other would read what
    was there before"""
    say(f"[block] stream {name} {handle}")
    there, fns = calls()
    want = flat(fns[name](there, None))
    here = {k: torch.zeros_like(v) for k, v in there.items()}
    slow = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    slower = torch.zeros_like(slow)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(20):  # about 2 ms
            slower.copy_(slow)
        for k in here:
            here[k].copy_(there[k])
    got = flat(fns[name](here, s.cuda_stream if handle else s))
    s.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_streams_at_once():
    say("[block] two streams")
    there, fns = calls()
    want = {n: flat(fns[n](there, None)) for n in NAMES}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for turn in range(6):
        for s in streams:
            got.append({n: flat(fns[n](there, s)) for n in NAMES})
    torch.cuda.synchronize()
    for one in got:
        for n in NAMES:
            for a, b in zip(one[n], want[n]):
                assert torch.equal(a, b), n
