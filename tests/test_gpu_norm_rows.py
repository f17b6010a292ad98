"""Norms and their gradients over more rows than the launch holds at once, so that every
workgroup takes a second row and more, against the 64-bit forms."""
import numpy as np
import pytest
import torch

import block_ref as ref
from gpu_util import abi, say
from test_gpu_norm import BF16, F16, F32, close, compare_forward, make, rows, wide

pytestmark = pytest.mark.gpu


def partial_rows(T, d):
    """rows of partial column sums that the gradients write: three of d floats each"""
    n, left = divmod(abi.moe_norm_backward_workspace(T, d), 12 * d)
    assert not left
    return n


def column_tolerance(mag, T, d, dtype, want):
    """The terms carry two row sums (d / 64 additions in a lane and a few joins each) and some
    roundings; then a partial row adds its share of the T rows one after another, and the
    join a sixteenth of the partial rows and sixteen sums: so many half-steps of what has
    been added up, at most the sum of magnitudes."""
    n = partial_rows(T, d)
    steps = -(-T // n) + -(-n // 16) + 16
    return mag * (2 * (d / 64 + 48) + steps) * ref.U32 + np.abs(want) * ref.HALF[dtype] \
        + ref.TINY[dtype] + 2.0 ** -120


#         T     d: forward workgroups hold 4,096 rows of up to 1,024 columns at once, 2,560 of
# 1,536, 1,536 of 2,560, 1,024 of 4,096, 768 of 5,000, 512 of 8,192; the gradients' groups
# 512 rows of up to 4,096 columns, 256 of more
MANY = [(4300, 520), (4200, 1003), (2600, 1536), (1700, 2560), (1100, 4096), (900, 5000),
        (600, 8191), (1100, 8192)]
TYPES = [(F32, F32, F32), (BF16, F32, BF16), (F16, F16, F32)]


@pytest.mark.parametrize("D,Y,R", TYPES, ids=str)
@pytest.mark.parametrize("T,d", MANY)
def test_more_rows_than_the_launch_holds(T, d, D, Y, R):
    # whole 16-byte rows with a gate per element, odd strides with one per channel
    for kind, pad in (("full", 0), ("channel", 5)):
        say(f"[norm rows] {T} {d} {D} {Y} {R} {kind} {pad}")
        a, g = make(T, d, D, Y, R, kind, True, True, pad)
        w = wide(a)
        rest = {k: v for k, v in a.items() if k != "r"}
        got = abi.norm(a["r"], **rest, gate_kind=kind, alpha=0.7, stats=True)
        compare_forward(got, w, kind, R, D)
        dz, dh = rows(g, T, d, R, pad, 0.5), rows(g, T, d, D, pad, 0.5)
        grads, ws = abi.norm_backward(got["z"], got["stats"], dz=dz, dh=dh, **rest, gate_kind=kind,
                                      alpha=0.7, grad_dtype=F32)
        del w["r"]
        want, mag = ref.norm_backward(ref.f64(got["z"]), ref.f64(got["stats"]), dz=ref.f64(dz),
                                      dh=ref.f64(dh), **w, kind=kind, alpha=float(np.float32(0.7)))
        assert set(grads) == set(want)
        for k in want:
            shape = tuple(grads[k].shape)
            v, m, t = want[k].reshape(shape), mag[k].reshape(shape), grads[k].dtype
            close(k, grads[k], v, column_tolerance(m, T, d, t, v) if len(shape) == 1 else
                  ref.norm_backward_tolerance(m, T, d, k, t, v))
        ws.fill_(0x7F)  # (bytes of large numbers: nothing of an earlier call's sums counts)
        again, _ = abi.norm_backward(got["z"], got["stats"], dz=dz, dh=dh, **rest, gate_kind=kind,
                                     alpha=0.7, grad_dtype=F32, workspace=ws)
        for k in grads:
            assert torch.equal(grads[k], again[k]), k


@pytest.mark.parametrize("T,d", [(8200, 264), (4100, 9000)])
def test_rows_are_those_of_a_call_of_their_own(T, d):
    """a wavefront's second rows and those of more than 8,192 columns: the last rows of the
    call and some before them, bit for bit"""
    say(f"[norm rows] own {T} {d}")
    a, g = make(T, d, BF16, BF16, F32, "full", True, True)
    every = abi.norm(a["r"], **{k: v for k, v in a.items() if k != "r"}, gate_kind="full",
                     stats=True)
    pick = torch.tensor([0, 1, T // 2, 4095, 4096, 4097, T - 2, T - 1], device="cuda")
    few = {k: (v[pick].contiguous() if v.dim() == 2 else v) for k, v in a.items()}
    some = abi.norm(few.pop("r"), **few, gate_kind="full", stats=True)
    for k in every:
        assert torch.equal(every[k][pick], some[k]), k
