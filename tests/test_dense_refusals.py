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


#              g     ldg u     ldu dt act T  f   h     ldh g8    gs    u8    us    stream
ACT_FORWARD = [P[0], 64, P[1], 64, 2, 2, 8, 64, P[2], 64, P[3], P[4], P[5], P[6], N]
#               g8    gs    u8    us    dh    lddh dt act T f dg    lddg du   lddu h    ldh stream
ACT_BACKWARD = [P[0], P[1], P[2], P[3], P[4], 64, 2, 2, 8, 64, P[5], 64, P[6], 64, P[7], 64, N]


def test_activation_outputs_apart():
    assert status("moe_act_forward", ACT_FORWARD) == 3
    codes = (10, 11, 12, 13)
    for a in codes:
        for b in (0, 2, 8, *codes):
            if a != b:
                assert status("moe_act_forward", ACT_FORWARD, (a, ACT_FORWARD[b])) == 1, (a, b)
    for at in (0, 2):  # h on g or on u is documented
        assert status("moe_act_forward", ACT_FORWARD, (8, ACT_FORWARD[at])) == 3

    assert status("moe_act_backward", ACT_BACKWARD) == 3
    for a in (10, 12, 14):
        for b in (0, 1, 2, 3, 10, 12, 14):
            if a != b:
                assert status("moe_act_backward", ACT_BACKWARD, (a, ACT_BACKWARD[b])) == 1, (a, b)
        # one of them on dh is documented
        assert status("moe_act_backward", ACT_BACKWARD, (a, ACT_BACKWARD[4])) == 3


# (97 columns: operands are copied into padded rows, so a workspace is needed)
#         x     ldx w     ldw bias  res   ldr rdt dt act T   d   n   ws    bytes    out   ldo odt stream
LINEAR = [P[0], 64, P[1], 97, P[2], P[3], 97, 0, 2, 2, 64, 64, 97, P[4], 1 << 30, P[5], 97, 0, N]
#                  x     ldx w     ldw dz    lddz dt T  d   n   ws    bytes    dx    lddx dw lddw db    gdt stream
LINEAR_BACKWARD = [P[0], 64, P[1], 97, P[2], 97, 2, 64, 64, 97, P[3], 1 << 30, P[4], 64, P[5], 97,
                   P[6], 0, N]


def test_product_outputs_apart_from_the_workspace():
    assert status("moe_linear", LINEAR) == 3
    assert status("moe_linear", LINEAR, (15, P[4])) == 1
    assert status("moe_linear_backward", LINEAR_BACKWARD) == 3
    for out in (12, 14, 16):
        assert status("moe_linear_backward", LINEAR_BACKWARD, (out, P[3])) == 1, out
    # a workspace that is not needed is not looked at: whole chunks, many tiles
    whole = [P[0], 64, P[1], 8, N, N, 0, 2, 2, 0, 64, 64, 8, P[5], 0, P[5], 8, 2, N]
    assert status("moe_linear", whole) == 3
