"""What the operators around the block refuse (host checks, made-up addresses that no
call here reads or writes: each is refused, or finds no device)."""
import ctypes

import pytest
import torch

from mixture_experts_routed_amd import abi

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0,
                                reason="made-up addresses: for a machine without a GPU")
N = None
P = [(1 << 20) * (i + 1) for i in range(16)]  # distinct, well-aligned
BIG = 1 << 34
OK, EINVAL, EUNSUPPORTED, EHIP = 0, 1, 2, 3


def status(call, args, *changes):
    args = list(args)
    for at, value in changes:
        args[at] = value
    return getattr(abi.lib(), call)(*args)


def refused(call, args, *cases, rc=EINVAL):
    assert status(call, args) == EHIP  # as given it would be launched
    for c in cases:
        c = c if isinstance(c[0], tuple) else (c,)
        assert status(call, args, *c) == rc, c


#         logits bias sc T   E   K groups keep top renorm scale ids w stream
SCORED = [P[0], P[1], 1, 64, 32, 4, 4, 2, 2, 1, 2.5, P[2], P[3], N]


def test_route_scored():
    refused("moe_route_scored", SCORED, (0, N), (0, P[0] + 2), (1, P[1] + 1), (2, 2), (2, -1),
            (3, 0), (4, 0), (5, 0), (5, 17), (6, 0), (6, 5), (7, 0), (7, 5), (8, 0), (8, 9),
            (10, float("inf")), (10, float("nan")), (11, N), (12, N), (11, P[2] + 1),
            (11, P[0]), (11, P[1]), (11, P[3]), (12, P[0]), (12, P[1]))
    refused("moe_route_scored", SCORED, (4, 1028), (8, 3), ((4, 1024), (6, 128), (8, 1)),
            ((4, 1024), (5, 65)), rc=EUNSUPPORTED)
    # 2 kept groups of 8 hold 16 experts
    assert status("moe_route_scored", SCORED, (5, 16)) == EHIP
    assert status("moe_route_scored", SCORED, (1, N)) == EHIP


#                logits ids  dw    add   sc T   E   K renorm scale out  dtype stream
SCORED_BACKWARD = [P[0], P[1], P[2], P[3], 0, 64, 32, 4, 0, 1.0, P[4], 1, N]


def test_route_scored_backward():
    refused("moe_route_scored_backward", SCORED_BACKWARD, (0, N), (1, N), (2, N), (4, 2), (5, 0),
            (6, 0), (7, 33), (7, 0), (9, float("nan")), (10, N), (10, P[4] + 1), (3, P[3] + 1),
            (11, 3), (10, P[0]), (10, P[1]), (10, P[2]))
    refused("moe_route_scored_backward", SCORED_BACKWARD, (6, 1025), rc=EUNSUPPORTED)
    for change in ((3, N), (10, P[3])):  # nothing to add; in place of it
        assert status("moe_route_scored_backward", SCORED_BACKWARD, change) == EHIP


#       r     ldr rt y     ldy yt post  gate  ldg kind pre  dt T  d   alpha eps   z     ldz h     ldh stats stream
NORM = [P[0], 96, 0, P[1], 96, 2, P[2], P[3], 96, 3, P[4], 2, 7, 96, 1.0, 1e-6, P[5], 96, P[6], 96,
        P[7], N]


def test_norm():
    refused("moe_norm", NORM, (0, N), (0, P[0] + 8), (1, 95), (1, (1 << 20) + 1), (2, 1), (4, 90),
            (5, 1), (5, 3), (6, P[2] + 4), (7, N), (7, P[3] + 2), (8, 95), (9, 0), (9, 4), (9, -1),
            (10, P[4] + 8), (11, 3), (12, 0), (13, 0), (14, float("nan")), (14, float("inf")),
            (15, 0.0), (15, -1.0), (15, 1e-31), (15, float("nan")), (15, float("inf")), (16, N),
            (16, P[5] + 4), (17, 95), (18, N), (18, P[6] + 4), (19, 95), (20, P[7] + 2),
            # what does not go together
            (3, N), ((3, N), (16, N)), ((3, N), (16, N), (6, N)), (10, N),
            ((3, N), (16, N), (6, N), (7, N), (9, 0), (10, N), (18, N)),
            # outputs on other arguments
            (16, P[1]), (16, P[2]), (16, P[3]), (16, P[4]), (16, P[6]), (16, P[7]), (18, P[0]),
            (18, P[2]), (18, P[3]), (18, P[4]), (18, P[7]), (20, P[0]), (20, P[1]), (20, P[2]),
            (20, P[3]), (20, P[4]), ((16, P[0]), (17, 104)), ((18, P[1]), (19, 104)),
            ((18, P[1]), (5, 0)))
    refused("moe_norm", NORM, ((13, 32769), (1, 40000), (4, 40000), (8, 40000), (17, 40000),
                               (19, 40000)), rc=EUNSUPPORTED)
    for change in (((16, P[0]),), ((18, P[1]),), ((20, N),), ((6, N),), ((7, N), (9, 0)),
                   ((10, N), (18, N)), ((9, 1), (8, 0)), ((9, 2), (8, 0)),
                   ((3, N), (16, N), (6, N), (7, N), (9, 0)), ((5, 0),), ((2, 2),)):
        assert status("moe_norm", NORM, *change) == EHIP, change


#          dz    lddz dh  lddh z   ldz rt y   ldy yt post  gate  ldg kind pre  stats dt T  d
BACKWARD = [P[0], 96, P[1], 96, P[2], 96, 0, P[3], 96, 2, P[4], P[5], 96, 3, P[6], P[7], 2, 7, 96,
            # alpha ws bytes dr  lddr dy  lddy  dgate  ld  post    pre   gt stream
            1.0, P[8], BIG, P[9], 96, P[10], 96, P[11], 96, P[12], P[13], 0, N]
DZ, DH, Z, Y, POST, GATE, KIND, PRE, STATS, WS, DR, DY, DGATE, DPOST, DPRE = (
    0, 2, 4, 7, 10, 11, 13, 14, 15, 20, 22, 24, 26, 28, 29)


def test_norm_backward():
    outs = (DR, DY, DGATE, DPOST, DPRE)
    others = (DZ, DH, Z, Y, POST, GATE, PRE, STATS, WS, *outs)
    apart = [(o, BACKWARD[i]) for o in outs for i in others
             if i != o and (o, i) != (DR, DZ)]
    refused("moe_norm_backward", BACKWARD, *apart, ((DR, P[0]), (23, 104)),
            (Z, N), (DR, N), (STATS, N), (STATS, P[7] + 2), (WS, N), (WS, P[8] + 64), (21, 8),
            (1, 95), (3, 95), (5, 95), (8, 95), (12, 95), (23, 95), (25, 95), (27, 95), (6, 1),
            (9, 3), (16, 4), (30, 1), (30, 3), (17, 0), (18, 0), (19, float("nan")), (KIND, 4),
            (KIND, 0), *[(at, BACKWARD[at] + 8) for at in (DZ, DH, Z, Y, POST, GATE, PRE, *outs)],
            (DH, N), (PRE, N), ((PRE, N), (DPRE, N)), (Y, N), (POST, N), (GATE, N),
            ((DZ, N), (DH, N), (PRE, N), (DPRE, N)))
    refused("moe_norm_backward", BACKWARD, ((18, 32769), *[(at, 40000) for at in
                                                          (1, 3, 5, 8, 12, 23, 25, 27)]),
            rc=EUNSUPPORTED)
    for change in (((DR, P[0]),), ((DZ, N),), ((DH, N), (PRE, N), (DPRE, N)), ((DPOST, N),),
                   ((DGATE, N),), ((DY, N),), ((DPRE, N),), ((POST, N), (DPOST, N)),
                   ((GATE, N), (KIND, 0), (DGATE, N)), ((30, 2),),
                   ((Y, N), (POST, N), (GATE, N), (KIND, 0), (DY, N), (DGATE, N), (DPOST, N))):
        assert status("moe_norm_backward", BACKWARD, *change) == EHIP, change


#          w    dt E  d   f   kind packed bytes stream
QUANTIZE = [P[0], 2, 8, 64, 72, 0, P[1], BIG, N]
#             packed bytes E d f  kind w    dt stream
DEQUANTIZE = [P[0], BIG, 8, 64, 72, 1, P[1], 0, N]


def test_mx4():
    refused("moe_mx4_quantize", QUANTIZE, (0, N), (0, P[0] + 8), (1, 3), (2, 0), (3, 60), (3, 0),
            (4, 4), (5, 2), (6, N), (6, P[1] + 8), (7, 8 * 4 * 1088 * 2 - 1), (6, P[0]),
            ((3, 1 << 16), (4, 1 << 16)))
    refused("moe_mx4_dequantize", DEQUANTIZE, (0, N), (1, 100), (2, 0), (3, 60), (4, 4), (5, -1),
            (6, N), (6, P[1] + 4), (6, P[0]), (7, -1))
    for call, args in (("moe_mx4_quantize", QUANTIZE), ("moe_mx4_dequantize", DEQUANTIZE)):
        refused(call, args, (2, 1025), rc=EUNSUPPORTED)
    v = ctypes.c_size_t()
    size = lambda *a: (abi.lib().moe_mx4_weight_bytes(*a, ctypes.byref(v)), v.value)  # noqa: E731
    assert size(8, 64, 72, 0) == (OK, 8 * 2 * 4 * 1088)
    assert size(8, 64, 72, 1) == (OK, 8 * 3 * 8 * 1088)
    assert size(512, 2560, 768, 0) == (OK, 512 * 2560 * 768 * 17 // 32)
    assert abi.lib().moe_mx4_weight_bytes(8, 64, 72, 0, N) == EINVAL


#          x     ids   w     gate  up    down  dt T  K  E  d   f   tm  ws    bytes out   ot stream
FORWARD = [P[0], P[1], P[2], P[3], P[4], P[5], 2, 9, 2, 8, 64, 72, 16, P[6], BIG, P[7], 2, N]


def test_forward_mx4():
    refused("moe_forward_mx4", FORWARD, *[(i, N) for i in range(6)], (13, N), (15, N),
            (0, P[0] + 8), (3, P[3] + 8), (5, P[5] + 4), (13, P[6] + 128), (14, 1000),
            (15, P[7] + 8), (6, 3), (16, 1), (16, 3), (7, 0), (8, 0), (9, 0), (10, 60), (11, 4),
            (12, 0), *[(15, P[i]) for i in range(7)])
    refused("moe_forward_mx4", FORWARD, (6, 0), (9, 1025), rc=EUNSUPPORTED)
    assert status("moe_forward_mx4", FORWARD, (16, 0)) == EHIP


def test_names_of_choices():
    with pytest.raises(TypeError, match="logits"):
        abi.route_scored(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError, match="w: expected a GPU tensor"):
        abi.mx4_quantize(torch.zeros(1, 8, 8), "gate")
    with pytest.raises(ValueError, match="expected one of softmax, sigmoid"):
        abi._named("score", "tanh", abi.SCORES)
    with pytest.raises(ValueError, match="y or w_pre"):
        abi._norm_dtype(None, None)
