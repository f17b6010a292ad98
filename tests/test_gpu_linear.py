"""moe_linear and moe_linear_backward on the GPU against the 64-bit forms, at
the sizes, strides and types where tiles, K-steps, splits and padded copies
begin and end. Tolerances are the rounding bounds of tests/dense_ref.py."""
import numpy as np
import pytest
import torch

import dense_ref as ref
from gpu_util import abi, say

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CANARY = 12288.0


def strided(g, rows, cols, std, dtype, pad):
    """[rows, cols] inside rows of cols + pad elements; what lies between is NaN"""
    full = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    t = full[:, :cols]
    t.copy_(torch.from_numpy(g.standard_normal((rows, cols)) * std))
    return t


def out_buffer(rows, cols, dtype, pad):
    """a result inside wider rows, and rows behind it, all marked"""
    full = torch.full((rows + 3, cols + pad), CANARY, dtype=dtype, device="cuda")
    return full, full[:rows, :cols]


def untouched(full, rows, cols):
    t = full.float()
    return bool((t[rows:] == CANARY).all()) and bool((t[:, cols:] == CANARY).all())


def polluted_workspace(nbytes):
    return torch.full((max(nbytes, 1),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type


def check_linear(T, d, n, dtype, out_dtype, kind="none", bias=True, residual=None, pad=0, opad=0,
                 seed=0):
    say(f"[linear] T={T} d={d} n={n} {dtype}->{out_dtype} {kind} bias={bias} res={residual} "
        f"pad={pad} opad={opad}")
    g = np.random.default_rng(seed + 1000 * T + d)
    D, O = DT[dtype], DT[out_dtype]
    x, w = strided(g, T, d, 1.0, D, pad), strided(g, d, n, d ** -0.5, D, pad)
    b = torch.from_numpy(g.standard_normal(n)).to("cuda", D) if bias else None
    r = strided(g, T, n, 1.0, DT[residual], opad) if residual else None
    full, out = out_buffer(T, n, O, opad)
    need = abi.moe_linear_workspace(T, d, n, d + pad if T > 1 else d, n + pad if d > 1 else n,
                                    abi.DTYPE_NAME[dtype])
    got, _ = abi.linear(x, w, bias=b, residual=r, act=kind, out=out,
                        workspace=polluted_workspace(need))
    torch.cuda.synchronize()
    assert got is out
    X, W = ref.f64(x), ref.f64(w)
    B, R = (None if b is None else ref.f64(b)), (None if r is None else ref.f64(r))
    want, z, size = ref.linear(X, W, B, R, kind)
    tol = ref.linear_tol(X, W, B, R, kind, want, z, size, O)
    err = np.abs(ref.f64(out) - want)
    assert np.all(err <= tol), (float((err - tol).max()), np.unravel_index((err - tol).argmax(), err.shape))
    assert untouched(full, T, n)
    again, _ = abi.linear(x, w, bias=b, residual=r, act=kind, out_dtype=O)
    torch.cuda.synchronize()
    assert torch.equal(again, out)  # the same bits, whatever the workspace held


SIZES = [(1, 1, 1), (1, 8, 8), (2, 7, 3), (4, 704, 2816), (5, 64, 40), (15, 65, 17), (16, 128, 64),
         (17, 100, 129), (33, 257, 60), (64, 2560, 512), (65, 40, 128), (100, 1000, 130),
         (127, 512, 127), (128, 64, 128), (129, 72, 136), (300, 1003, 517), (512, 4096, 2048),
         (257, 256, 768), (1000, 136, 264)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,d,n", SIZES)
def test_linear_sizes(T, d, n, dtype):
    check_linear(T, d, n, dtype, "f32")


# the large tile (16-bit types) in the forward product, in dx and in dw, with ragged
# edges; cut along k; and the middle tile, whole and cut
LARGE = [(3900, 400, 3100), (3841, 328, 3329), (3900, 3100, 400), (400, 3900, 3100),
         (333, 3841, 3333), (700, 2600, 700), (20000, 700, 700)]


def test_large_sizes_take_the_tiles_they_stand_for():
    for dt in (abi.MOE_F16, abi.MOE_BF16):
        assert abi.moe_linear_shape(3900, 3100, 400, dt) == (256, 1)
        assert abi.moe_linear_shape(3841, 3329, 328, dt) == (256, 1)
        tile, split = abi.moe_linear_shape(700, 700, 20000, dt)
        assert split > 1 and tile >= 128
        assert abi.moe_linear_shape(333, 3333, 3841, dt)[0] == 128
        assert abi.moe_linear_shape(40, 60, 100, dt) == (64, 1)
        assert abi.moe_linear_shape(64, 512, 2560, dt)[0] == 64
    shapes = {abi.moe_linear_shape(M, N, K, abi.MOE_F32)[0]
              for M, N, K in [(300, 517, 1003), (1900, 1990, 300), (2000, 700, 3001)]}
    assert shapes == {64, 128}


@pytest.mark.parametrize("T,d,n", [(1900, 300, 1990), (2000, 3001, 700)])
def test_linear_large_f32(T, d, n):
    check_linear(T, d, n, "f32", "f32", "silu", residual="f32")
    check_backward(T, d, n, "f32", "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,d,n", LARGE)
def test_linear_large(T, d, n, dtype):
    check_linear(T, d, n, dtype, dtype, "silu", residual="f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,d,n", LARGE)
def test_linear_backward_large(T, d, n, dtype):
    check_backward(T, d, n, dtype, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("out_f32,residual", [(False, None), (False, "own"), (True, "f32"),
                                              (True, "own"), (False, "f32")])
def test_linear_epilogues(dtype, kind, out_f32, residual):
    check_linear(37, 120, 92, dtype, "f32" if out_f32 else dtype, kind,
                 bias=kind != "relu", residual=dtype if residual == "own" else residual)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,opad", [(8, 8), (5, 3), (3, 4), (16, 1)])
@pytest.mark.parametrize("T,d,n", [(1, 33, 5), (3, 64, 64), (70, 130, 71), (130, 256, 200)])
def test_linear_strides(T, d, n, dtype, pad, opad):
    check_linear(T, d, n, dtype, dtype, "silu", residual="f32", pad=pad, opad=opad)


def test_linear_residual_in_place():
    """the residual stream: out is the residual itself, split and not split"""
    for T, d, n in [(4, 704, 2816), (40, 64, 72), (640, 128, 1000)]:
        g = np.random.default_rng(T)
        x, w = strided(g, T, d, 1.0, torch.bfloat16, 0), strided(g, d, n, 0.05, torch.bfloat16, 0)
        y = torch.from_numpy(g.standard_normal((T, n)).astype(np.float32)).cuda()
        want, _ = abi.linear(x, w, residual=y, out_dtype=torch.float32)
        got, _ = abi.linear(x, w, residual=y, out=y)
        torch.cuda.synchronize()
        assert got is y and torch.equal(y, want)


def test_linear_special_values():
    """a NaN or infinity reaches its own rows and columns and no others"""
    T, d, n = 40, 72, 88
    g = np.random.default_rng(3)
    for dtype in (torch.bfloat16, torch.float32):
        x, w = strided(g, T, d, 1.0, dtype, 0), strided(g, d, n, 0.1, dtype, 0)
        clean, _ = abi.linear(x, w, act="gelu")
        x[7, 5] = float("nan")
        x[9, 0] = float("inf")
        w[3, 11] = float("nan")
        got, _ = abi.linear(x, w, act="gelu")
        torch.cuda.synchronize()
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[7], keep[9] = False, False
        keep[:, 11] = False
        assert torch.equal(got[keep], clean[keep])
        assert got[7].isnan().all() and got[:, 11].isnan().all()
        assert not got[9].float()[torch.arange(n) != 11].isfinite().logical_and(
            clean[9].float()[torch.arange(n) != 11].abs() > 1e30).any()


def check_backward(T, d, n, dtype, grad, pad=0, grads=("dx", "dw", "db"), seed=0):
    say(f"[linear backward] T={T} d={d} n={n} {dtype}->{grad} pad={pad} {grads}")
    g = np.random.default_rng(seed + 1000 * T + d)
    D, G = DT[dtype], DT[grad]
    x, w = strided(g, T, d, 1.0, D, pad), strided(g, d, n, d ** -0.5, D, pad)
    dz = strided(g, T, n, 0.3, D, pad)
    bufs = {"dx": out_buffer(T, d, D, pad), "dw": out_buffer(d, n, G, pad)}
    db = torch.full((n + 8,), CANARY, dtype=G, device="cuda")
    kw = {k: bufs[k][1] for k in ("dx", "dw") if k in grads}
    if "db" in grads:
        kw["db"] = db[:n]
    got, _ = abi.linear_backward(x if "dw" in grads or "dx" not in grads else None,
                                 w if "dx" in grads else None, dz, grads=grads, grad_dtype=G, **kw)
    torch.cuda.synchronize()
    assert set(got) == set(grads)
    X, W, Z = ref.f64(x), ref.f64(w), ref.f64(dz)
    want = {"dx": (Z @ W.T, np.abs(Z) @ np.abs(W.T), n, D),
            "dw": (X.T @ Z, np.abs(X.T) @ np.abs(Z), T, G),
            "db": (Z.sum(axis=0), np.abs(Z).sum(axis=0), T, G)}
    for k in grads:
        v, size, terms, R = want[k]
        # `terms` products and additions, each off by one step of the running sum at most
        tol = 2 * terms * 2.0 ** -23 * size
        tol = tol + ref.HALF[R] * (np.abs(v) + tol) + ref.TINY[R]
        err = np.abs(ref.f64(got[k]) - v)
        assert np.all(err <= tol), (k, float((err - tol).max()))
    for k, (full, t) in bufs.items():
        assert untouched(full, t.shape[0], t.shape[1]) if k in grads else bool((full == CANARY).all())
    assert bool((db[n:].float() == CANARY).all())
    again, _ = abi.linear_backward(x, w, dz, grads=grads, grad_dtype=G)
    torch.cuda.synchronize()
    for k in grads:
        assert torch.equal(again[k], got[k]), k


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,d,n", SIZES + [(3000, 72, 40), (4097, 64, 130)])
def test_linear_backward_sizes(T, d, n, dtype):
    check_backward(T, d, n, dtype, "f32")


@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"),
                                        ("f32", "f32")])
@pytest.mark.parametrize("pad", [0, 8, 5])
@pytest.mark.parametrize("T,d,n", [(1, 33, 5), (70, 130, 71), (260, 256, 200)])
def test_linear_backward_strides(T, d, n, dtype, grad, pad):
    check_backward(T, d, n, dtype, grad, pad)


@pytest.mark.parametrize("grads", [("dx",), ("dw",), ("db",), ("dx", "db"), ("dw", "db"),
                                   ("dx", "dw")])
def test_linear_backward_in_part(grads):
    check_backward(50, 96, 61, "bf16", "f32", 0, grads)


@pytest.mark.parametrize("T,n", [(1, 4), (7, 12), (900, 252), (130, 260)])
def test_bias_gradient_of_rows_that_end_in_half_a_piece(T, n):
    """fp32 rows of whole 16-byte chunks that are not whole pieces of 8 columns"""
    check_backward(T, 8, n, "f32", "f32", 0, ("db",))
    check_backward(T, 8, n, "f32", "f32", 4)


def test_results_on_operands_are_refused():
    x = torch.zeros(64, 64, device="cuda")
    w, y = torch.zeros_like(x), torch.zeros_like(x)
    for call in (lambda: abi.linear(x, w, out=x), lambda: abi.linear(x, w, out=w),
                 lambda: abi.linear_backward(x, w, y, dx=y),
                 lambda: abi.linear_backward(x, w, y, dw=x),
                 lambda: abi.linear_backward(x, w, y, dx=w),
                 lambda: abi.route_backward(x, torch.zeros(64, 2, dtype=torch.int32, device="cuda"),
                                            None, None, torch.zeros(66, dtype=torch.int32,
                                                                    device="cuda"),
                                            torch.zeros(2, device="cuda"), out=x)):
        with pytest.raises(abi.MoeError):
            call()
    # the operand that a gradient does not read may be overwritten by it
    got, _ = abi.linear_backward(x, w, y, grads=("dx",), dx=x)
    assert got["dx"] is x


def test_linear_backward_is_the_difference_quotient():
    """<dz, z(x + h v) - z(x - h v)> / 2h = <dx, v>, and so for w: z is linear, so
    what is left is 32-bit rounding of z (2^-24 |z| over h, with h = 1/4)"""
    T, d, n = 33, 64, 48
    g = np.random.default_rng(5)
    x, w, dz = (strided(g, *s, 1.0, torch.float32, 0) for s in ((T, d), (d, n), (T, n)))
    got, _ = abi.linear_backward(x, w, dz)
    h = 0.25
    for name, a in (("dx", x), ("dw", w)):
        v = strided(g, *a.shape, 1.0, torch.float32, 0)
        z = []
        for s in (h, -h):
            args = (x + s * v, w) if name == "dx" else (x, w + s * v)
            z.append(abi.linear(*args)[0].double())
        num = float((dz.double() * (z[0] - z[1])).sum() / (2 * h))
        have = float((got[name].double() * v.double()).sum())
        size = float((dz.abs().double() * (z[0].abs() + z[1].abs())).sum())
        assert abs(num - have) <= 4 * d * 2.0 ** -23 * size / h, (name, num, have)


def test_linear_graph_replays():
    """captured with its workspace and replayed between eager calls: split product,
    padded copies, and the backward pass"""
    g = np.random.default_rng(9)
    for T, d, n in [(4, 704, 2816), (60, 333, 77)]:
        x, w = strided(g, T, d, 1.0, torch.bfloat16, 0), strided(g, d, n, 0.05, torch.bfloat16, 0)
        dz = strided(g, T, n, 1.0, torch.bfloat16, 0)
        want, ws = abi.linear(x, w, act="silu")
        gwant, gws = abi.linear_backward(x, w, dz)
        out = torch.empty_like(want)
        grads = {k: torch.empty_like(v) for k, v in gwant.items()}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            abi.linear(x, w, act="silu", out=out, workspace=ws)
            abi.linear_backward(x, w, dz, workspace=gws, **grads)
        for rep in range(3):
            out.fill_(float("nan"))
            for t in (*grads.values(), ws, gws):
                t.fill_(0 if rep else 77)
            abi.linear(x, w, act="silu")
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want), rep
            for k in grads:
                assert torch.equal(grads[k], gwant[k]), (rep, k)
        del graph


def test_linear_on_another_stream():
    g = np.random.default_rng(11)
    x, w = strided(g, 300, 512, 1.0, torch.float16, 0), strided(g, 512, 77, 0.05, torch.float16, 0)
    want, _ = abi.linear(x, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got, _ = abi.linear(x, w, stream=s)
    raw, _ = abi.linear(x, w, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(raw, want)


def test_linear_helper_refuses():
    x = torch.zeros(4, 8, device="cuda")
    w = torch.zeros(8, 6, device="cuda")
    for bad in (dict(w=torch.zeros(7, 6, device="cuda")), dict(w=w.half()), dict(w=w.t()),
                dict(bias=torch.zeros(5, device="cuda")), dict(bias=torch.zeros(6)),
                dict(residual=torch.zeros(4, 5, device="cuda")), dict(act="tanh"),
                dict(residual=torch.zeros(4, 6, device="cuda", dtype=torch.float16)),
                dict(out=torch.zeros(4, 6, device="cuda", dtype=torch.bfloat16)),
                dict(out=torch.zeros(1, 6, device="cuda").expand(4, 6)),
                dict(x=torch.zeros(0, 8, device="cuda")), dict(x=x[:, ::2], w=w[:4]),
                dict(x=torch.zeros(4, 9, device="cuda")[:, 1:])):
        args = {"x": x, "w": w, **bad}
        with pytest.raises((TypeError, ValueError, KeyError, abi.MoeError)):
            abi.linear(**args)
