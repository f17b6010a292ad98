"""The plain 64-bit forms that the dense operators are checked against: their
gradients against differences, their code format against torch's type."""
import numpy as np
import pytest
import torch

import dense_ref as ref


@pytest.mark.parametrize("kind", ["relu", "silu", "gelu"])
def test_slope_is_the_difference_quotient(kind):
    z = np.linspace(-9, 9, 1801) + 1e-3  # (no point at relu's corner)
    h = 1e-5
    num = (ref.act(z + h, kind) - ref.act(z - h, kind)) / (2 * h)
    # central difference: h^2 / 6 times the third derivative (below 2), and 2^-52 |act| / h
    assert np.max(np.abs(num - ref.act_slope(z, kind))) < 1e-9


def test_e4m3_values_are_torch_codes():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(codes), np.isnan(ref.E4M3))
    ok = ~np.isnan(codes)
    assert np.array_equal(codes[ok], ref.E4M3[ok])


def test_encode_rounds_as_torch_does():
    g = np.random.default_rng(0)
    z = (g.standard_normal((64, 77)) * np.exp(g.uniform(-20, 20, (64, 1)))).astype(np.float32)
    z[3] = 0
    z[4, ::5] = 0
    codes, s = ref.encode(z.astype(np.float64))
    e = np.repeat(s.astype(int) - 127, 32, axis=1)[:, :77]
    want = torch.from_numpy(np.ldexp(z, -e)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(codes, want)
    # the scale is the least that holds the block's maximum
    for r in (0, 1, 2, 5):
        M = np.abs(z[r, :32]).max()
        assert M <= 448 * 2.0 ** (int(s[r, 0]) - 127)
        assert M > 448 * 2.0 ** (int(s[r, 0]) - 128)


def _total(logits, ids, w_of, dw, dl):
    loss, _, _ = ref.balance(logits, ids)
    return float(dl @ loss + (w_of(logits) * dw).sum())


def test_route_gradient_is_the_difference_quotient():
    """dlogits against central differences of dl . loss + sum w dw, w the
    renormalised softmax over each token's picks"""
    g = np.random.default_rng(1)
    T, E, K = 6, 9, 3
    logits = g.standard_normal((T, E))
    ids = np.argsort(-logits, axis=1)[:, :K].astype(np.int32)
    ids[2] = -1
    ids[4, 1] = -1
    dw, dl = g.standard_normal((T, K)), np.array([0.7, -0.3])

    def w_of(l):
        ok = ids >= 0
        v = np.where(ok, np.exp(np.take_along_axis(l, np.where(ok, ids, 0), axis=1)), 0.0)
        s = v.sum(axis=1, keepdims=True)
        return np.where(ok, v / np.where(s == 0, 1, s), 0.0)

    got, _ = ref.route_backward(logits, ids, w_of(logits), dw, ref.counts(ids, E), dl)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            a, b = logits.copy(), logits.copy()
            a[t, e] += h
            b[t, e] -= h
            num = (_total(a, ids, w_of, dw, dl) - _total(b, ids, w_of, dw, dl)) / (2 * h)
            assert abs(num - got[t, e]) < 1e-8  # 2^-52 times about 30, over h; h^2


def test_linear_gradient_is_the_difference_quotient():
    g = np.random.default_rng(2)
    x, w, b = g.standard_normal((3, 4)), g.standard_normal((4, 5)), g.standard_normal(5)
    dz = g.standard_normal((3, 5))
    f = lambda x, w, b: float((ref.linear(x, w, b, None, "none")[0] * dz).sum())  # noqa: E731
    grads = (dz @ w.T, x.T @ dz, dz.sum(axis=0))
    for i, a in enumerate((x, w, b)):
        for at in np.ndindex(a.shape):
            args = [[v.copy() for v in (x, w, b)] for _ in range(2)]
            args[0][i][at] += 1e-5
            args[1][i][at] -= 1e-5
            # f is linear in each of them: only 2^-52 |f| / 1e-5 is left
            assert abs((f(*args[0]) - f(*args[1])) / 2e-5 - grads[i][at]) < 1e-8
