"""Outputs that are other arguments of a call (host checks, made-up addresses that
no call here reads or writes: each is refused, or finds no device)."""
import pytest
import torch

from mixture_experts_routed_amd import abi

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="made-up addresses: for a machine without a GPU")
N = None
# distinct, well-aligned
P = [(1 << 20) * (i + 1) for i in range(12)]


def status(call, args, *changes):
    args = list(args)
    for at, value in changes:
        args[at] = value
    return getattr(abi.lib(), call)(*args)


#           logits ids T   E  K  ws   bytes    cnt   prob  loss  stream
BALANCE = [P[0], P[1], 64, 8, 2, P[2], 1 << 20, P[3], P[4], P[5], N]
#                 logits ids   w     dw    cnt   dloss T   E  K  out   dtype stream
ROUTE_BACKWARD = [P[0], P[1], P[2], P[3], P[4], P[5], 64, 8, 2, P[6], 0, N]


def test_router_outputs_apart():
    assert status("moe_balance_loss", BALANCE) == 3
    for out in (7, 8, 9):
        for other in (0, 1, 5, 7, 8, 9):
            if other != out:
                assert status("moe_balance_loss", BALANCE, (out, BALANCE[other])) == 1, (out, other)
    assert status("moe_route_backward", ROUTE_BACKWARD) == 3
    for other in range(6):
        assert status("moe_route_backward", ROUTE_BACKWARD, (9, P[other])) == 1, other
    # w is not read without dw
    assert status("moe_route_backward", ROUTE_BACKWARD, (3, N), (9, P[2])) == 3
