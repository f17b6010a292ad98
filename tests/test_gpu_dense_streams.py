"""Each dense operator on a stream other than the current one, given as torch's
stream and as its handle: its inputs arrive there behind long copies, so work on
any other stream would read what was there before."""
import pytest
import torch

from gpu_util import abi, say

pytestmark = pytest.mark.gpu
T, D, N, E, K = 700, 264, 520, 60, 4


def inputs():
    g = torch.Generator(device="cuda").manual_seed(21)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    h = lambda *s: r(*s).to(torch.bfloat16)  # noqa: E731
    logits = r(T, E)
    ids, w = abi.route(logits, K)
    _, ckpt = abi.act_forward(h(T, D), h(T, D), ckpt=True)
    return dict(x=h(T, D), w=h(D, N), dz=h(T, N), logits=logits, ids=ids, rw=w, dw=r(T, K),
                cnt=abi.balance_loss(logits, ids)[0]["cnt"],
                dloss=torch.tensor([2.0, 3.0], device="cuda"), g=h(T, D), u=h(T, D), dh=h(T, D),
                **{"ck_" + k: v.view(torch.uint8) for k, v in ckpt.items()})


def ckpt_of(t):
    return {k: t["ck_" + k].view(torch.float8_e4m3fn) if k.endswith("8") else t["ck_" + k]
            for k in ("g8", "gs", "u8", "us")}


def flat(v):
    if torch.is_tensor(v):
        return [v.view(torch.uint8) if v.dtype is torch.float8_e4m3fn else v]
    return [t for k in sorted(v) for t in flat(v[k])] if isinstance(v, dict) else \
        [t for q in v for t in flat(q)]


CALLS = {
    "linear": lambda t, s: abi.linear(t["x"], t["w"], act="silu", stream=s)[0],
    "linear_backward": lambda t, s: abi.linear_backward(t["x"], t["w"], t["dz"], stream=s)[0],
    "balance_loss": lambda t, s: abi.balance_loss(t["logits"], t["ids"], stream=s)[0],
    "route_backward": lambda t, s: abi.route_backward(t["logits"], t["ids"], t["rw"], t["dw"],
                                                      t["cnt"], t["dloss"], stream=s),
    "act_forward": lambda t, s: list(abi.act_forward(t["g"], t["u"], ckpt=True, stream=s)),
    "act_backward": lambda t, s: abi.act_backward(ckpt_of(t), t["dh"], stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("handle", [False, True])
def test_another_stream(name, handle):
    say(f"[stream] {name} handle={handle}")
    call, there = CALLS[name], inputs()
    want = flat(call(there, None))
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
    got = flat(call(here, s.cuda_stream if handle else s))
    s.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once():
    """the same calls on two streams, each with inputs and workspaces of its own"""
    a, b = inputs(), inputs()
    b["x"], b["logits"] = b["x"] * 2, b["logits"] * 2
    want = [[flat(CALLS[n](t, None)) for n in CALLS] for t in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for n in CALLS:
        for i, t in enumerate((a, b)):
            got[i].append(flat(CALLS[n](t, streams[i])))
    for s in streams:
        s.synchronize()
    for i in range(2):
        for p, q in zip(got[i], want[i]):
            assert all(torch.equal(u, v) for u, v in zip(p, q))


def test_the_default_stream_by_its_handle():
    """what a call allocates for the default stream, whose handle is 0, belongs to that
    stream: once freed, it is what the stream's next request of that size gets"""
    x, w = torch.randn(5003, 40, device="cuda"), torch.randn(40, 1900, device="cuda")
    want, _ = abi.linear(x, w)
    for stream in (None, 0, torch.cuda.default_stream()):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        out, _ = abi.linear(x, w, stream=stream)
        assert torch.equal(out, want)
        at = out.data_ptr()
        del out
        assert torch.empty_like(want).data_ptr() == at, stream
