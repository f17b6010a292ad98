"""moe_linear and moe_linear_backward on small whole numbers: every product and
every partial sum is a whole number below 2^24, exact in 32 bits in any order,
so a result is equal to the 64-bit product (rounded once where it is written in
a 16-bit type). A dropped, doubled or misplaced K-step, tail or range of k of a
long sum, which lies within a rounding bound of that sum, is seen here. Each
product is made as the forward product, as dx and as dw; its sizes take a known
tile and number of ranges."""
import pytest
import torch

from gpu_util import abi, say

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

# (M, N, K): (tile, ranges of k) of the 16-bit types, and of fp32
PRODUCTS = {
    (2539, 1019, 8201): ((256, 4), (128, 3)),    # the large tile cut, ragged; k ends 9 into a step
    (2552, 1000, 8200): ((256, 4), (128, 3)),    # the same of whole chunks
    (2539, 493, 32011): ((256, 9), (128, 3)),    # nine ranges of unequal length
    (3841, 2027, 8203): ((256, 2), (128, 1)),
    (1000, 2040, 4100): ((128, 2), (128, 2)),    # the middle tile cut
    (700, 700, 20011): ((128, 7), (128, 7)),
    (4001, 2051, 8199): ((256, 1), (64, 1)),     # the large tile whole
    (1090, 1077, 333): ((64, 1), (64, 1)),       # the small tile, one team (more than 256 workgroups)
    (261, 1661, 1003): ((64, 1), (64, 3)),       # fp32: one team, cut
    (264, 1664, 1024): ((64, 1), (64, 3)),
    (517, 130, 4099): ((64, 9), (64, 9)),        # two teams, cut
    (250, 250, 33000): ((64, 16), (64, 16)),
    (40, 60, 100): ((64, 1), (64, 1)),           # two teams, whole
}


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_sizes_take_the_tiles_and_ranges_they_stand_for(M, N, K):
    half, single = PRODUCTS[M, N, K]
    assert abi.moe_linear_shape(M, N, K, abi.MOE_BF16) == half
    assert abi.moe_linear_shape(M, N, K, abi.MOE_F16) == half
    assert abi.moe_linear_shape(M, N, K, abi.MOE_F32) == single


def whole(g, rows, cols, dtype, pad):
    """[rows, cols] of -2 .. 2 inside rows of cols + pad elements; NaN between them"""
    full = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    t = full[:, :cols]
    t.copy_(torch.randint(-2, 3, (rows, cols), generator=g, device="cuda"))
    return t


def same(name, got, want):
    """equal to the whole numbers of `want`, rounded once to got's type"""
    want = want.float().to(got.dtype)
    bad = got != want
    assert not bool(bad.any()), (name, int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 8, 5])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_whole_numbers(M, N, K, pad, dtype):
    assert 4 * K < 2 ** 24
    say(f"[linear exact] {M} x {N} over {K} {dtype} pad={pad}")
    g, D = torch.Generator(device="cuda").manual_seed(M + K), DT[dtype]

    x, w = whole(g, M, K, D, pad), whole(g, K, N, D, pad)
    got, _ = abi.linear(x, w, out_dtype=torch.float32)
    same("out", got, x.double() @ w.double())

    dz, w = whole(g, M, K, D, pad), whole(g, N, K, D, pad)
    got, _ = abi.linear_backward(None, w, dz, grads=("dx",))
    same("dx", got["dx"], dz.double() @ w.double().t())

    x, dz = whole(g, K, M, D, pad), whole(g, K, N, D, pad)
    got, _ = abi.linear_backward(x, None, dz, grads=("dw", "db"), grad_dtype=torch.float32)
    same("dw", got["dw"], x.double().t() @ dz.double())
    same("db", got["db"], dz.double().sum(dim=0))
    # the column sums of the padded copy (above) and of dz where it lies
    alone, _ = abi.linear_backward(x, None, dz, grads=("db",), grad_dtype=torch.float32)
    same("db alone", alone["db"], dz.double().sum(dim=0))
