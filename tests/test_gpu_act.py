"""moe_act_forward and moe_act_backward on the GPU: checkpoint codes and scales
bit for bit, activations and gradients within rounding bounds."""
import numpy as np
import pytest
import torch

import dense_ref as ref
from gpu_util import abi, say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CANARY = 320.0


def strided(a, dtype, pad):
    T, f = a.shape
    full = torch.full((T + 2, f + pad), CANARY, dtype=dtype, device="cuda")
    t = full[:T, :f]
    t.copy_(torch.from_numpy(a))
    return full, t


def values(g, T, f, dtype):
    """magnitudes over many powers of two, zero blocks, one large value among small ones"""
    z = g.standard_normal((T, f)) * 2.0 ** g.integers(-8, 4, (T, 1))
    z[::5] = 0
    z[1::7, ::3] *= 1e-4
    return z


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def check(T, f, dtype, kind, gated, pad=0, seed=0):
    say(f"[act] T={T} f={f} {dtype} {kind} gated={gated} pad={pad}")
    g = np.random.default_rng(seed + T * 31 + f)
    D = DT[dtype]
    _, gate = strided(values(g, T, f, dtype), D, pad)
    up = strided(g.standard_normal((T, f)), D, pad)[1] if gated else None
    full_h, h = strided(np.full((T, f), np.nan), D, pad)
    got, ck = abi.act_forward(gate, up, act=kind, ckpt=True, h=h)
    bare, none = abi.act_forward(gate, up, act=kind)  # without a checkpoint
    torch.cuda.synchronize()
    assert got is h and none is None and torch.equal(bare, h)
    assert bool((full_h[T:].float() == CANARY).all()) and bool((full_h[:, f:].float() == CANARY).all())
    G, U = ref.f64(gate), (ref.f64(up) if gated else 1.0)
    want = ref.act(G, kind) * U
    size = np.abs(want)
    tol = (ref.act_rel(G, kind) + 2 * ref.U32) * size
    tol = tol + ref.HALF[D] * (size + tol) + ref.TINY[D] + 2.0 ** -140
    assert np.all(np.abs(ref.f64(h) - want) <= tol)
    for k, z in (("g", gate), ("u", up))[:2 if gated else 1]:
        codes, scales = ref.encode(ref.f64(z))
        assert np.array_equal(bytes_of(ck[k + "s"]), scales), k
        assert np.array_equal(bytes_of(ck[k + "8"]), codes), k
        # what the format promises
        e = np.repeat(scales.astype(int) - 127, 32, axis=1)[:, :f]
        off = np.abs(ref.decode(codes, scales) - ref.f64(z))
        assert np.all(off <= np.maximum(2.0 ** -4 * np.abs(ref.f64(z)), 2.0 ** (e - 10.0)))

    _, dh = strided(g.standard_normal((T, f)), D, pad)
    full_g, dg = strided(np.full((T, f), np.nan), D, pad)
    back = abi.act_backward(ck, dh, act=kind, dg=dg)
    torch.cuda.synchronize()
    assert bool((full_g[T:].float() == CANARY).all()) and bool((full_g[:, f:].float() == CANARY).all())
    Z = ref.decode(bytes_of(ck["g8"]), bytes_of(ck["gs"]))
    V = ref.decode(bytes_of(ck["u8"]), bytes_of(ck["us"])) if gated else 1.0
    dH = ref.f64(dh)
    rel = np.maximum(ref.act_rel(Z, kind), 16 * ref.U32) + 4 * ref.U32
    a = ref.act(Z, kind)
    for k, v, s in (("dg", dH * V * ref.act_slope(Z, kind), np.abs(dH * V) * ref.slope_terms(Z, kind)),
                    ("du", dH * a, np.abs(dH * a)), ("h", a * V, np.abs(a * V))):
        if k == "du" and not gated:
            assert "du" not in back
            continue
        tol = rel * s
        tol = tol + ref.HALF[D] * (np.abs(v) + tol) + ref.TINY[D] + 2.0 ** -140
        err = np.abs(ref.f64(back[k]) - v)
        assert np.all(err <= tol), (k, float((err - tol).max()))
    less = abi.act_backward(ck, dh, act=kind, need_h=False)
    torch.cuda.synchronize()
    assert "h" not in less and torch.equal(less["dg"], back["dg"])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,f", [(1, 1), (1, 8), (3, 31), (2, 32), (5, 33), (7, 40), (64, 704),
                                 (33, 768), (130, 100), (9, 1003), (257, 256), (1000, 72)])
def test_sizes(T, f, dtype):
    check(T, f, dtype, "silu", True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_kinds_and_strides(kind, gated, dtype, pad):
    check(21, 104, dtype, kind, gated, pad)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_every_rounding_border(dtype):
    """each code's value, the midpoints between neighbours (ties), and one step of
    the type beside them, under a maximum that fixes the scale"""
    D = DT[dtype]
    pos = ref.E4M3[:127]
    mids = (pos[1:] + pos[:-1]) / 2
    v = torch.from_numpy(np.concatenate([pos, mids])).to(D)
    step = torch.finfo(D).eps
    v = torch.cat([v, (v.double() * (1 + step)).to(D), (v.double() * (1 - step)).to(D)])
    v = torch.cat([v, -v])
    v = v[v.abs() <= 448]
    n = -(-v.numel() // 31)
    z = torch.zeros(n, 32, dtype=D)
    z[:, 0] = 448.0
    z[:, 1:].reshape(-1)  # (columns 1..31 hold the values)
    flat = torch.zeros(n * 31, dtype=D)
    flat[: v.numel()] = v
    z[:, 1:] = flat.view(n, 31)
    _, ck = abi.act_forward(z.cuda(), act="relu", ckpt=True)
    codes, scales = ref.encode(ref.f64(z))
    assert np.all(scales == 127)
    got = bytes_of(ck["g8"])
    assert np.array_equal(bytes_of(ck["gs"]), scales)
    assert np.array_equal(got, codes)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f16"])
def test_extreme_scales_and_values_that_are_not_finite(dtype):
    """maxima at the border of a power of two, the type's largest and smallest
    values, infinities and NaN (their own code, no part in the scale)"""
    D = DT[dtype]
    fi = torch.finfo(D)
    z = torch.zeros(12, 64, dtype=D)
    g = np.random.default_rng(4)
    z[:, 32:] = torch.from_numpy(g.standard_normal((12, 32))).to(D)
    z[0, 0], z[1, 0], z[2, 0], z[3, 0] = fi.max, -fi.max, fi.tiny, fi.smallest_normal
    z[4, 0] = 448.0
    z[5, 0] = 448.0 * (1 + 2 * fi.eps)
    z[6, 3], z[6, 4] = float("inf"), 2.0
    z[7, 3], z[7, 4] = float("nan"), -3.0
    z[8, :32] = float("-inf")
    z[9, 40] = float("inf")
    z[10, 0] = 2.0 ** -24 if dtype == "f16" else 2.0 ** -126
    h, ck = abi.act_forward(z.cuda(), act="relu", ckpt=True)
    torch.cuda.synchronize()
    codes, scales = ref.encode(ref.f64(z))
    assert np.array_equal(bytes_of(ck["gs"]), scales)
    assert np.array_equal(bytes_of(ck["g8"]), codes)
    assert h[7, 3].isnan() and torch.isinf(h[6, 3]) and h[8, 0] == 0
    back = abi.act_backward(ck, torch.ones(12, 64, dtype=D, device="cuda"), act="relu")
    bad = np.isnan(ref.decode(codes, scales))
    assert np.array_equal(torch.isnan(back["dg"]).cpu().numpy(), bad)


def test_scale_of_one_block_does_not_reach_the_next():
    z = torch.full((4, 96), 1e-3, device="cuda")
    z[:, 33] = 1000.0
    _, ck = abi.act_forward(z, act="silu", ckpt=True)
    s = ck["gs"].cpu().numpy()
    assert (s[:, 0] == s[:, 2]).all() and (s[:, 1] > s[:, 0]).all()


def test_checkpoint_is_reused_and_captured():
    g = np.random.default_rng(6)
    z = [torch.from_numpy(g.standard_normal((200, 136))).to("cuda", torch.bfloat16) for _ in range(3)]
    h, ck = abi.act_forward(z[0], z[1], ckpt=True)
    back = abi.act_backward(ck, z[2])
    out = {k: torch.empty_like(v) for k, v in back.items()}
    h2 = torch.empty_like(h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        abi.act_forward(z[0], z[1], ckpt=ck, h=h2)
        abi.act_backward(ck, z[2], **out)
    for _ in range(3):
        for t in (h2, *out.values()):
            t.zero_()
        for t in ck.values():
            t.view(torch.uint8).zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and all(torch.equal(back[k], out[k]) for k in out)


def test_helper_refuses():
    z = torch.zeros(4, 40, device="cuda")
    _, ck = abi.act_forward(z, z, ckpt=True)
    for call in (lambda: abi.act_forward(z, z.half()), lambda: abi.act_forward(z, act="none"),
                 lambda: abi.act_forward(z, z[:, :39]), lambda: abi.act_forward(z, ckpt=ck),
                 lambda: abi.act_forward(z.t()), lambda: abi.act_forward(z, z, act="swish"),
                 lambda: abi.act_backward(ck, z[:, :32]), lambda: abi.act_backward(ck, z[:2]),
                 lambda: abi.act_backward({k: ck[k] for k in ("g8", "gs")}, z, du=z.clone())):
        with pytest.raises((TypeError, ValueError, KeyError, abi.MoeError)):
            call()


@pytest.mark.parametrize("T,f", [(70, 264), (5, 1003)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_results_in_place_of_an_input(T, f, dtype):
    """h on g or u, and one of dg, du and h on dh, give the bits that they give elsewhere"""
    say(f"[act in place] T={T} f={f} {dtype}")
    r = np.random.default_rng(f)
    g, u, dh = (torch.from_numpy(r.standard_normal((T, f))).to("cuda", DT[dtype]) for _ in range(3))
    want, ck = abi.act_forward(g, u, ckpt=True)
    back = abi.act_backward(ck, dh)
    for on in (0, 1):
        a, b = g.clone(), u.clone()
        h, again = abi.act_forward(a, b, ckpt=True, h=(a, b)[on])
        torch.cuda.synchronize()
        assert torch.equal(h, want)
        assert all(torch.equal(again[k].view(torch.uint8), ck[k].view(torch.uint8)) for k in ck)
    for k in ("dg", "du", "h"):
        a = dh.clone()
        got = abi.act_backward(ck, a, **{k: a})
        torch.cuda.synchronize()
        assert all(torch.equal(got[q], back[q]) for q in back), k
    with pytest.raises(abi.MoeError):
        abi.act_backward(ck, dh, dg=g, du=g)
