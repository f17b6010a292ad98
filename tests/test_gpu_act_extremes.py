"""The activation's gradients where the checkpoint stands for +-2^128: the largest
magnitudes of bf16 and fp32 (248 * 2^120 and more) are rounded up to the code of
256 * 2^120, which a value of fp32 does not reach. An entry masked with the
type's lowest value is one of these."""
import numpy as np
import pytest
import torch

import dense_ref as ref
from gpu_util import abi, say
from test_gpu_act import bytes_of

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BIG = 2.0 ** 128


def extremes(dtype):
    """[6, 72]: blocks with the type's largest magnitudes among small values"""
    fi = torch.finfo(DT[dtype])
    g = np.random.default_rng(8)
    z = torch.from_numpy(g.standard_normal((6, 72))).to(DT[dtype])
    z[0, 3], z[0, 4] = fi.min, 1.0
    z[1, 40], z[1, 70] = fi.max, fi.min
    z[2, :32] = fi.min
    z[3, 5], z[3, 6] = 2.0 ** 127 * 1.9375, -(2.0 ** 127) * 1.9375  # 248 * 2^120: a tie, to 256
    z[4, 5] = 2.0 ** 127 * 1.875                                    # 240 * 2^120: itself
    z[5, 1], z[5, 2], z[5, 3] = fi.max, float("nan"), float("inf")
    return z


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["relu", "silu", "gelu"])
@pytest.mark.parametrize("gated,on", [(True, "g"), (True, "u"), (False, "g")])
def test_gradients_of_the_largest_magnitudes(dtype, kind, gated, on):
    say(f"[act extremes] {dtype} {kind} gated={gated} on={on}")
    D, g = DT[dtype], np.random.default_rng(9)
    z = extremes(dtype)
    # (small factors: a product with +-2^128 stays within the type, or infinite in both)
    small = torch.from_numpy(g.uniform(0.25, 0.5, z.shape)).to(D)
    gate, up = (z, small if gated else None) if on == "g" else (small, z)
    _, ck = abi.act_forward(gate.cuda(), None if up is None else up.cuda(), act=kind, ckpt=True)
    dh = torch.from_numpy(g.uniform(2.0 ** -6, 2.0 ** -5, z.shape)).to(D)
    back = abi.act_backward(ck, dh.cuda(), act=kind)
    torch.cuda.synchronize()
    Z = ref.decode(bytes_of(ck["g8"]), bytes_of(ck["gs"]))
    V = ref.decode(bytes_of(ck["u8"]), bytes_of(ck["us"])) if gated else np.ones_like(Z)
    assert (np.abs(Z if on == "g" else V) == BIG).sum() >= 36
    dH, a = ref.f64(dh), ref.act(Z, kind)
    # (beyond 100 the slopes are 0 and 1 with nothing left to add)
    terms = np.where(np.abs(Z) > 100, 1.0, ref.slope_terms(Z, kind))
    # as for ordinary values, and half a step more: in a block with +-2^128 values are read
    # 2^-24 below themselves (the activations and slopes of the others move by no more)
    rel = np.maximum(ref.act_rel(np.clip(np.nan_to_num(Z), -20, 20), kind), 16 * ref.U32) + 6 * ref.U32
    for k, v, s in (("dg", dH * V * ref.act_slope(Z, kind), np.abs(dH * V) * terms),
                    ("du", dH * a, np.abs(dH * a)), ("h", a * V, np.abs(a * V))):
        if k not in back:
            continue
        got = ref.f64(back[k])
        nan = np.isnan(v)
        assert np.array_equal(np.isnan(got), nan), (k, np.argwhere(np.isnan(got) != nan))
        ok = ~nan & (np.abs(v) < torch.finfo(D).max * 0.99)
        # (an h of 2^128 itself is past the type: infinite, or its largest value)
        assert np.all(np.abs(got[~nan & ~ok]) >= torch.finfo(D).max), k
        tol = rel * s
        tol = tol + ref.HALF[D] * (np.abs(v) + tol) + ref.TINY[D] + 2.0 ** -140
        assert np.all(np.abs(got - v)[ok] <= tol[ok]), k
