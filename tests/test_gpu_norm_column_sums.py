"""Column sums of the norms' gradients over values that add up exactly: a row or a
partial row that is left out shows as a whole number."""
import pytest
import torch

from gpu_util import abi, say
from test_gpu_norm import BF16, F16, F32

pytestmark = pytest.mark.gpu


def whole(g, T, d, most, dtype):
    """integers from -most to most"""
    return torch.randint(-most, most + 1, (T, d), generator=g, device="cuda").to(dtype)


#        d: a wavefront a row; workgroups of whole and odd rows; a row at a time; longer rows
EXACT = [(264, [1, 1023, 1024, 1025, 1031, 4097, 20000]), (1003, [511, 512, 513, 1025, 4300]),
         (2560, [512, 513, 1700]), (4096, [511, 513, 1100]), (4104, [255, 256, 257, 700]),
         (8191, [256, 257]), (8192, [255, 257, 1100]), (9000, [256, 257, 600])]


@pytest.mark.parametrize("D,Y", [(F32, F32), (BF16, F32), (F16, F16)], ids=str)
@pytest.mark.parametrize("d,Ts", EXACT, ids=lambda v: str(v) if isinstance(v, int) else "")
def test_column_sums_of_whole_numbers(d, Ts, D, Y):
    """Reciprocal norms of 1 and small integers: each term is a multiple of 1/2, each sum
    below 2^24 of those, so fp32 holds every partial sum and the result is exact. Every row
    has a term in every column, so that none can be left out."""
    for T in Ts:
        say(f"[norm rows] exact {T} {d} {D} {Y}")
        g = torch.Generator(device="cuda").manual_seed(T + d)
        one = torch.ones((T, 2), device="cuda")
        z, y = whole(g, T, d, 3, F32), whole(g, T, d, 3, Y)
        z = torch.where(z == 0, 2.0, z)
        y = torch.where(y == 0, torch.ones_like(y), y)
        dh, dz = whole(g, T, d, 2, D), whole(g, T, d, 2, F32)
        dh = torch.where(dh == 0, torch.ones_like(dh), dh)
        dz = torch.where(dz == 0, torch.ones_like(dz), dz)
        pick = torch.randint(1, 3, (3, d), generator=g, device="cuda").to(D)
        w_pre, w_post, gate = pick[0].clone(), pick[1].clone(), pick[2].clone()
        # the weights before the block: sum of dh z
        got, _ = abi.norm_backward(z, one, dz=dz, dh=dh, w_pre=w_pre, grad_dtype=F32)
        assert torch.equal(got["dw_pre"].double(), (dh.double() * z.double()).sum(dim=0))
        # behind it, without the norm before the next: dr = dz
        got, _ = abi.norm_backward(z, one, dz=dz, y=y, w_post=w_post, gate=gate,
                                   gate_kind="channel", alpha=0.5, grad_dtype=F32)
        term = 0.5 * dz.double() * y.double()
        assert torch.equal(got["dr"], dz)
        assert torch.equal(got["dw_post"].double(), (term * gate.double()).sum(dim=0))
        assert torch.equal(got["dgate"].double(), (term * w_post.double()).sum(dim=0))
