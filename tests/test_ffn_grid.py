"""The grouped FFN's launches stay below 2^32 threads, past which HIP starts a grid modulo
2^32 without an error: such sizes are refused (host checks, made-up addresses)."""
import pytest
import torch

from mixture_experts_routed_amd import abi

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="made-up addresses: for a machine without a GPU")
N = None
P = [(1 << 20) * (i + 1) for i in range(16)]
BIG = 1 << 60
EINVAL, EHIP = 1, 3


def ffn(call, rows, E, d, f, dtype=1, tm=16):
    #    xs gate up down dtype E d f tm eoff stok sw meta rows h y scratch bytes stream
    return getattr(abi.lib(), call)(P[0], P[1], P[2], P[3], dtype, E, d, f, tm, P[4], P[5], P[6],
                                    P[7], rows, P[8], P[9], P[10], BIG, N)


SIZES = [(1, 8, 8, 1), (1, 8, 512, 2), (1, 1024, 8, 2), (7, 520, 1032, 5)]


@pytest.mark.parametrize("E,d,f,per", SIZES)
def test_row_major_weights(E, d, f, per):
    """cells: max_rows / 64 + 1 + experts, times groups of 256 columns of h and 512 of y; at
    most 2^24 - 9 workgroups of 256 threads"""
    for dtype in (0, 1, 2):
        rows = (((1 << 24) - 16) // per - 1 - E) * 64
        assert ffn("moe_expert_ffn", rows, E, d, f, dtype) == EHIP  # as given it would be launched
        assert ffn("moe_expert_ffn", rows + 64 * 32, E, d, f, dtype) == EINVAL
        assert ffn("moe_expert_ffn", (1 << 31) - 2048, E, d, f, dtype) == EINVAL


@pytest.mark.parametrize("E,d,f,per", SIZES)
def test_packed_weights(E, d, f, per):
    """runs of 4 items besides: max_rows / 193 times 128 columns of h and 256 of y; at most
    2^23 - 1 workgroups of 512 threads"""
    rows = (((1 << 24) - 16) // per - 1 - E) * 64
    assert ffn("moe_expert_ffn_packed", rows, E, d, f, 0) == EHIP  # (fp32 has no such runs)
    runs = max(-(-f // 128), -(-d // 256))
    rows = min(rows, ((1 << 23) - 8) // runs * 193)
    assert ffn("moe_expert_ffn_packed", rows, E, d, f) == EHIP
    assert ffn("moe_expert_ffn_packed", rows + 193 * 32, E, d, f) == EINVAL


def test_layers():
    def status(call, T, K, E, d, f, *more):
        args = [P[0], P[1], P[2], P[3], P[4], P[5], 1, T, K, E, d, f, 16, P[6], BIG, P[7], *more, N]
        return getattr(abi.lib(), call)(*args)

    for call, more in (("moe_forward", ()), ("moe_forward_packed", ()), ("moe_forward_mx4", (0,))):
        assert status(call, 1 << 29, 1, 8, 8, 8, *more) == EHIP
        assert status(call, 1 << 30, 1, 8, 8, 8, *more) == EINVAL
        assert status(call, 1 << 27, 4, 8, 2048, 8, *more) == EINVAL
