"""The plain forms of the operators around the block, on the CPU: gradients against
differences of the forward forms, 4-bit values against a search over all codes."""
import numpy as np
import pytest

import block_ref as ref


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    logits, dw = rng.normal(size=(5, 12)), rng.normal(size=(5, 3))
    kw = dict(score=score, renorm=renorm, scale=2.5)
    ids, _, gap = ref.route(logits, 3, **kw)
    assert gap > 1e-5  # a step of 1e-6 changes no choice
    got, _ = ref.route_backward(logits, ids, dw, **kw)
    for e in range(12):
        up, down = logits.copy(), logits.copy()
        up[:, e] += 1e-6
        down[:, e] -= 1e-6
        diff = ((ref.route(up, 3, **kw)[1] - ref.route(down, 3, **kw)[1]) * dw).sum(axis=1) / 2e-6
        assert np.allclose(got[:, e], diff, rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("kind", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_norm_gradient_against_differences(kind, post, pre):
    rng = np.random.default_rng(4)
    T, d = 3, 7
    a = {"r": rng.normal(size=(T, d)), "y": rng.normal(size=(T, d))}
    if post:
        a["w_post"] = rng.normal(size=d)
    if pre:
        a["w_pre"] = rng.normal(size=d)
    if kind != "none":
        a["gate"] = rng.normal(size={"token": T, "channel": d, "full": (T, d)}[kind])
    dz, dh = rng.normal(size=(T, d)), rng.normal(size=(T, d)) if pre else None

    def loss(v):
        o = ref.norm(**v, kind=kind, alpha=0.7)
        return (o["z"] * dz).sum() + ((o["h"] * dh).sum() if pre else 0.0)

    out = ref.norm(**a, kind=kind, alpha=0.7)
    back = {k: v for k, v in a.items() if k != "r"}
    got, _ = ref.norm_backward(out["z"], out["stats"], dz=dz, dh=dh, **back, kind=kind, alpha=0.7)
    for name, g in (("r", "dr"), ("y", "dy"), ("w_post", "dw_post"), ("w_pre", "dw_pre"),
                    ("gate", "dgate")):
        if name not in a:
            continue
        want = np.zeros(a[name].shape)
        for i in np.ndindex(a[name].shape):
            up, down = dict(a), dict(a)
            up[name], down[name] = a[name].copy(), a[name].copy()
            up[name][i] += 1e-6
            down[name][i] -= 1e-6
            want[i] = (loss(up) - loss(down)) / 2e-6
        assert np.allclose(got[g], want, rtol=1e-6, atol=1e-7), g


def test_mx4_codes_are_nearest():
    rng = np.random.default_rng(5)
    w = rng.normal(size=(2, 77, 9)) * np.exp(rng.normal(size=(2, 77, 9)) * 4)
    codes, scales = ref.mx4_encode(w)
    v = ref.mx4_values(codes, scales)
    s = np.ldexp(1.0, np.repeat(scales.astype(int), 32, axis=1)[:, :77] - 127)
    near = np.abs(np.abs(w)[..., None] / s[..., None] - ref.VALUES).min(axis=-1) * s
    assert np.allclose(np.abs(v - w), near, rtol=1e-12, atol=0)
    assert (np.abs(w) <= 6 * s).all()
    assert np.array_equal(ref.mx4_values(*ref.mx4_encode(v)), v)  # kept exactly
    big = np.abs(w) >= s
    assert (np.abs(v - w)[big] <= 0.2 * np.abs(w)[big] * (1 + 1e-12)).all()
    assert (np.abs(v - w)[~big] <= 0.25 * s[~big]).all()


def test_mx4_places_are_distinct():
    for Kd, N, down in ((40, 72, False), (72, 520, True), (8, 8, True)):
        code, scale, size = ref.mx4_places(Kd, N, down)
        assert max(code.max(), scale.max()) < size
        pairs = code * 2 + (np.arange(Kd) % 2)[:, None]
        assert len(np.unique(pairs)) == Kd * N
        assert not set(np.unique(code)) & set(np.unique(scale))
        assert len(np.unique(scale)) == -(-Kd // 32) * N
