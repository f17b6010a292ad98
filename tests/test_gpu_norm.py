"""Norms around a block, with gate, scale and residual, and their gradients, against
the 64-bit forms."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import abi, say

pytestmark = pytest.mark.gpu
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
KINDS = ["none", "token", "channel", "full"]


def rows(g, T, d, dtype, pad=0, std=1.0):
    return (torch.randn((T, d + pad), generator=g, device="cuda") * std).to(dtype)[:, :d]


def make(T, d, D, Y, R, kind, post, pre, pad=0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 13 * d + T)
    a = {"r": rows(g, T, d, R, pad, 2.0), "y": rows(g, T, d, Y, pad, 0.3)}
    if post:
        a["w_post"] = 1 + rows(g, 1, d, D)[0] * 0.1
    if pre:
        a["w_pre"] = 1 + rows(g, 1, d, D)[0] * 0.1
    if kind != "none":
        shape = {"token": (T, 1), "channel": (1, d), "full": (T, d)}[kind]
        a["gate"] = rows(g, *shape, D, pad if kind == "full" else 0)
        if kind != "full":
            a["gate"] = a["gate"].reshape(-1)
    return a, g


def wide(a):
    return {k: ref.f64(v) for k, v in a.items()}


def close(name, got, want, tol):
    got = ref.f64(got)
    tol = tol + 1e-300
    off = np.abs(got - want)
    assert (off <= tol).all(), (name, np.max(off / tol))


def check_forward(a, kind, D, alpha=0.7, eps=1e-6, **out):
    got = abi.norm(a["r"], **{k: v for k, v in a.items() if k != "r"}, gate_kind=kind,
                   alpha=alpha, eps=eps, stats=True, **out)
    w = wide({**a, "r": a["r"].clone()}) if not out else None
    return got, w


def compare_forward(got, w, kind, R, D, alpha=0.7, eps=1e-6):
    alpha = float(np.float32(alpha))
    eps = float(np.float32(eps))
    want = ref.norm(**w, kind=kind, alpha=alpha, eps=eps)
    tol = ref.norm_tolerance(want, w["r"], w.get("gate"), kind, w.get("w_pre"), alpha)
    close("z", got["z"], want["z"], tol["z"] + np.abs(want["z"]) * ref.HALF[R] + ref.TINY[R])
    close("stats", got["stats"], want["stats"], tol["stats"])
    assert ("h" in got) == ("h" in want)
    if "h" in want:
        close("h", got["h"], want["h"], tol["h"] + np.abs(want["h"]) * ref.HALF[D] + ref.TINY[D])
    return want


def check_backward(a, w, got, kind, D, G, g, pad=0, alpha=0.7, **out):
    T, d = w["r"].shape
    z, stats = got["z"], got["stats"]
    dz = rows(g, T, d, z.dtype, pad, 0.5)
    dh = rows(g, T, d, D, pad, 0.5) if "w_pre" in a else None
    back = {k: v for k, v in a.items() if k != "r"}
    if out.pop("dz_in_place", False):
        dz0, out["dr"] = dz.clone(), dz
    else:
        dz0 = dz
    grads, ws = abi.norm_backward(z, stats, dz=dz, dh=dh, **back, gate_kind=kind, alpha=alpha,
                                  grad_dtype=G, **out)
    want, mag = ref.norm_backward(
        ref.f64(z), ref.f64(stats), dz=ref.f64(dz0) if out.get("dr") is None else ref.f64(dz0),
        dh=None if dh is None else ref.f64(dh), **wide(back), kind=kind,
        alpha=float(np.float32(alpha)))
    assert set(grads) == set(want)
    for k in want:
        close(k, grads[k], want[k].reshape(grads[k].shape),
              ref.norm_backward_tolerance(mag[k].reshape(grads[k].shape), T, d, k,
                                          grads[k].dtype, want[k].reshape(grads[k].shape)))
    return grads, dz, dh


TYPES = [(F32, F32, F32), (BF16, BF16, BF16), (BF16, F32, BF16), (BF16, BF16, F32),
         (F16, F32, F32), (F16, F16, F16), (F16, F16, F32)]
#        T    d
SIZES = [(1, 1), (2, 3), (1, 64), (5, 128), (3, 200), (9, 513), (4, 1003), (33, 1024), (6, 2048),
         (7, 2560), (5, 4096), (3, 5000), (2, 8192), (3, 10000), (2, 16384), (2, 32768)]


@pytest.mark.parametrize("D,Y,R", TYPES, ids=str)
@pytest.mark.parametrize("T,d", SIZES)
def test_both_norms_and_gradients(T, d, D, Y, R):
    for kind, pad in (("none", 0), ("token", 8), ("channel", 0), ("full", 0), ("full", 5)):
        say(f"[norm] {T} {d} {D} {Y} {R} {kind} {pad}")
        if pad == 8 and d % 8:
            pad = 3
        a, g = make(T, d, D, Y, R, kind, True, True, pad)
        w = wide(a)
        got, _ = check_forward(a, kind, D)
        compare_forward(got, w, kind, R, D)
        check_backward(a, w, got, kind, D, F32 if pad else D, g, pad)


@pytest.mark.parametrize("post,pre", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,d", [(5, 96), (3, 1001), (40, 2560), (2, 12000)])
def test_parts(T, d, kind, post, pre):
    say(f"[norm] parts {T} {d} {kind} {post} {pre}")
    a, g = make(T, d, BF16, F32, BF16, kind, post, pre)
    if not post and not pre and kind == "none":
        a["y"] = a["y"].to(BF16)  # (the only sign of the type of the weights)
    w = wide(a)
    got, _ = check_forward(a, kind, BF16)
    compare_forward(got, w, kind, BF16, BF16)
    check_backward(a, w, got, kind, BF16, F32, g)


@pytest.mark.parametrize("D,R", [(BF16, F32), (F16, F16), (F32, F32)], ids=str)
@pytest.mark.parametrize("T,d", [(1, 8), (70, 1003), (300, 2816)])
def test_norm_of_the_residual_alone(T, d, D, R):
    say(f"[norm] alone {T} {d} {D} {R}")
    a, g = make(T, d, D, D, R, "none", False, True)
    del a["y"]
    w = wide(a)
    got = abi.norm(a["r"], w_pre=a["w_pre"], stats=True)
    want = ref.norm(**w, eps=float(np.float32(1e-6)))
    tol = ref.norm_tolerance(want, w["r"], None, "none", w["w_pre"], 1.0)
    assert "z" not in got
    close("h", got["h"], want["h"], tol["h"] + np.abs(want["h"]) * ref.HALF[D] + ref.TINY[D])
    assert torch.equal(abi.norm(a["r"], w_pre=a["w_pre"])["h"], got["h"])
    dh = rows(g, T, d, D)
    for dz in (None, rows(g, T, d, R)):
        grads, _ = abi.norm_backward(a["r"], got["stats"], dz=dz, dh=dh, w_pre=a["w_pre"])
        wb, mag = ref.norm_backward(w["r"], ref.f64(got["stats"]), dh=ref.f64(dh), w_pre=w["w_pre"],
                                    dz=None if dz is None else ref.f64(dz))
        assert set(grads) == {"dr", "dw_pre"}
        for k in wb:
            close(k, grads[k], wb[k],
                  ref.norm_backward_tolerance(mag[k], T, d, k, grads[k].dtype, wb[k]))


@pytest.mark.parametrize("d", [96, 1003, 4096, 20000])
def test_in_place(d):
    """z on r, h on y, dr on dz: the bits of the call with outputs of their own"""
    say(f"[norm] in place {d}")
    T = 37
    a, g = make(T, d, BF16, BF16, F32, "full", True, True)
    want = abi.norm(a["r"], **{k: v for k, v in a.items() if k != "r"}, gate_kind="full", stats=True)
    b = {k: v.clone() for k, v in a.items()}
    got = abi.norm(b["r"], **{k: v for k, v in b.items() if k != "r"}, gate_kind="full",
                   stats=True, z=b["r"], h=b["y"])
    for k in want:
        assert torch.equal(want[k], got[k]), k
    assert got["z"] is b["r"] and got["h"] is b["y"]
    dz, dh = rows(g, T, d, F32), rows(g, T, d, BF16)
    back = {k: v for k, v in a.items() if k != "r"}
    one, _ = abi.norm_backward(want["z"], want["stats"], dz=dz, dh=dh, **back, gate_kind="full")
    two, _ = abi.norm_backward(want["z"], want["stats"], dz=dz, dh=dh, **back, gate_kind="full", dr=dz)
    assert two["dr"] is dz
    for k in one:
        assert torch.equal(one[k], two[k]), k


@pytest.mark.parametrize("T", [1, 255, 256, 257, 1000, 3001, 20000])
def test_many_rows_and_column_sums(T):
    say(f"[norm] many rows {T}")
    d = 264
    a, g = make(T, d, F16, F16, F16, "channel", True, True)
    w = wide(a)
    got, _ = check_forward(a, "channel", F16)
    compare_forward(got, w, "channel", F16, F16)
    one, dz, dh = check_backward(a, w, got, "channel", F16, F32, g)
    back = {k: v for k, v in a.items() if k != "r"}
    two, _ = abi.norm_backward(got["z"], got["stats"], dz=dz, dh=dh, **back, gate_kind="channel",
                               alpha=0.7, grad_dtype=F32)
    for k in one:
        assert torch.equal(one[k], two[k]), k  # no sum depends on timing


@pytest.mark.parametrize("asked", [["dy"], ["dgate"], ["dw_post"], ["dw_pre"], []], ids=str)
@pytest.mark.parametrize("kind", ["token", "channel", "full"])
def test_some_gradients(kind, asked):
    say(f"[norm] some gradients {kind} {asked}")
    a, g = make(70, 520, BF16, F32, F32, kind, True, True)
    got, _ = check_forward(a, kind, BF16)
    dz, dh = rows(g, 70, 520, F32), rows(g, 70, 520, BF16)
    back = {k: v for k, v in a.items() if k != "r"}
    kw = dict(dz=dz, dh=dh, **back, gate_kind=kind)
    every, _ = abi.norm_backward(got["z"], got["stats"], **kw)
    some, _ = abi.norm_backward(got["z"], got["stats"], grads=asked, **kw)
    assert set(some) == set(asked) | {"dr"}
    for k in some:
        assert torch.equal(some[k], every[k]), k


def test_rows_next_to_the_ends_of_the_range():
    """squares that overflow and vanish in fp32, zeros, and values that are not finite"""
    say("[norm] range")
    T, d = 8, 1000
    a, _ = make(T, d, F32, F32, F32, "none", True, True)
    for k, scale in ((0, 1e30), (1, 3e38 / 6), (2, 1e-30), (3, 0.0)):
        a["y"][k] *= scale
        a["r"][k] *= scale / 4
    a["y"][4, 7], a["r"][5, 9], a["y"][6, 3] = float("inf"), float("inf"), float("nan")
    w = wide(a)
    got = abi.norm(a["r"], y=a["y"], w_post=a["w_post"], w_pre=a["w_pre"], stats=True)
    with np.errstate(invalid="ignore", over="ignore"):
        want = ref.norm(**w, eps=float(np.float32(1e-6)))
        tol = ref.norm_tolerance(want, w["r"], None, "none", w["w_pre"], 1.0)
    for k in ("z", "h", "stats"):
        x, y = ref.f64(got[k]), want[k]
        fine = np.isfinite(y)
        assert np.array_equal(np.isnan(x), np.isnan(y)), k
        t = tol[k] + np.abs(y) * ref.U32 + 2.0 ** -126
        assert (np.abs(x - y)[fine] <= t[fine]).all(), k


def test_residual_alone_gives_the_type():
    """an fp32 output onto a 16-bit residual stream, nothing else that names a type"""
    say("[norm] no weights, fp32 y")
    a, g = make(9, 264, BF16, F32, BF16, "none", False, False)
    got = abi.norm(a["r"], y=a["y"], alpha=0.5)
    assert set(got) == {"z"}
    want = ref.f64(a["r"]) + 0.5 * ref.f64(a["y"])
    off = np.abs(ref.f64(got["z"]) - want)
    assert (off <= np.abs(want) * ref.HALF[BF16] + 2.0 ** -20).all()
    dz = rows(g, 9, 264, BF16)
    grads, _ = abi.norm_backward(got["z"], torch.zeros((9, 2), device="cuda"), dz=dz, y=a["y"],
                                 alpha=0.5)
    assert set(grads) == {"dr", "dy"} and grads["dy"].dtype is F32
    assert torch.equal(grads["dr"], dz) and torch.equal(grads["dy"], 0.5 * dz.float())


def test_a_given_gradient_is_asked_for():
    say("[norm] given gradients")
    a, g = make(20, 264, BF16, F32, F32, "token", True, True)
    got, _ = check_forward(a, "token", BF16)
    dz, dh = rows(g, 20, 264, F32), rows(g, 20, 264, BF16)
    kw = dict(dz=dz, dh=dh, **{k: v for k, v in a.items() if k != "r"}, gate_kind="token")
    every, _ = abi.norm_backward(got["z"], got["stats"], **kw)
    mine = torch.full((264,), 7.0, dtype=BF16, device="cuda")
    some, _ = abi.norm_backward(got["z"], got["stats"], grads=["dy"], dw_pre=mine, **kw)
    assert set(some) == {"dr", "dy", "dw_pre"} and some["dw_pre"] is mine
    for k in some:
        assert torch.equal(some[k], every[k]), k


@pytest.mark.parametrize("d", [264, 1003, 9000])
def test_offsets_past_32_bits(d):
    """rows 2^20 elements apart, past 2^31 in all, give what rows next to each other give"""
    say(f"[norm] far rows {d}")
    T, ld = 2052, 1 << 20
    a, g = make(T, d, BF16, BF16, BF16, "full", True, True)
    far = torch.empty((T - 1) * ld + d, dtype=BF16, device="cuda").as_strided((T, d), (ld, 1))
    dz, dh = rows(g, T, d, BF16), rows(g, T, d, BF16)
    rest = {k: v for k, v in a.items() if k not in ("r", "y", "gate")}
    near = abi.norm(a["r"], y=a["y"], gate=a["gate"], gate_kind="full", stats=True, **rest)
    back, _ = abi.norm_backward(near["z"], near["stats"], dz=dz, dh=dh, y=a["y"], gate=a["gate"],
                                gate_kind="full", **rest)
    for name in ("r", "y", "gate", "z", "h"):
        t = {**a, **near}[name]
        far.copy_(t)
        kw = dict(a, stats=True, gate_kind="full")
        out = {name: far} if name in ("z", "h") else {}
        kw.update(out or {name: far})
        got = abi.norm(kw.pop("r"), **kw)
        for k in near:
            assert torch.equal(got[k], near[k]), (name, k)
    for name in ("dz", "dh", "z", "y", "gate", "dr", "dy", "dgate"):
        kw = dict(z=near["z"], dz=dz, dh=dh, y=a["y"], gate=a["gate"], **rest)
        if name in kw:
            far.copy_(kw[name])
        kw[name] = far
        got, _ = abi.norm_backward(kw.pop("z"), near["stats"], gate_kind="full", **kw)
        for k in back:
            assert torch.equal(got[k], back[k]), (name, k)
