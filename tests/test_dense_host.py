"""Host-side checks of the dense operators' C entry points and helpers: sizes,
and every refusal, before any HIP call (made-up addresses, no GPU)."""
import ctypes

import pytest
import torch

from mixture_experts_routed_amd import abi

A = 1 << 20  # a well-aligned address that is never dereferenced
N = None


def L():
    return abi.lib()


def ws(T, d, n, ldx, ldw, dtype):
    v = ctypes.c_size_t()
    return L().moe_linear_workspace(T, d, n, ldx, ldw, dtype, ctypes.byref(v)), v.value


def test_linear_workspace_holds_padded_copies():
    # large, whole 16-byte rows: nothing is copied and nothing is split
    assert ws(32768, 4096, 2048, 4096, 2048, 2) == (0, 0)
    # x rows of 1003 fp32 (padded to 1004), w rows of 517 (520)
    rc, b = ws(32768, 1003, 517, 1003, 517, 0)
    assert rc == 0 and b == 32768 * 1004 * 4 + (1003 * 520 * 4 + 255) // 256 * 256
    # a stride that is no multiple of 8 elements is copied too, at its own width
    rc, b = ws(32768, 1024, 2048, 1029, 2048, 1)
    assert rc == 0 and b == 32768 * 1024 * 2


@pytest.mark.parametrize("T,d,n,ldx,ldw,dtype", [
    (0, 8, 8, 8, 8, 0), (8, 0, 8, 8, 8, 0), (8, 8, 0, 8, 8, 0), (8, 8, 8, 7, 8, 0),
    (8, 8, 8, 8, 7, 0), (8, 8, 8, 8, 8, 3), (8, 8, 8, 8, 8, -1),
    (8, 8, 8, (1 << 20) + 1, 8, 0), (8, 1 << 21, 8, 1 << 21, 8, 0), (-5, 8, 8, 8, 8, 0),
    (2 ** 31 - 1, 8, 8, 8, 8, 0),
])
def test_linear_sizes_refused(T, d, n, ldx, ldw, dtype):
    assert ws(T, d, n, ldx, ldw, dtype)[0] == 1
    v = ctypes.c_size_t()
    assert L().moe_linear_backward_workspace(T, d, n, ldx, ldw, n, dtype, 7, ctypes.byref(v)) == 1


def test_products_of_too_many_tiles_are_refused():
    """2^23 workgroups are one launch: a tall product of one column is served up to there"""
    T = 2 ** 31 - 2048
    tile, split = abi.moe_linear_shape(T, 1, 8, 2)
    rc = ws(T, 8, 1, 8, 1, 2)[0]
    assert rc == (0 if -(-T // tile) * split <= 2 ** 23 - 8 else 1)
    assert ws(T, 8, 4096, 8, 4096, 2)[0] == 1          # 2^23 x 16 tiles
    v = ctypes.c_size_t()
    back = L().moe_linear_backward_workspace
    assert back(T, 4096, 8, 4096, 8, 8, 2, 1, ctypes.byref(v)) == 1   # dx
    assert back(T, 4096, 8, 4096, 8, 8, 2, 2, ctypes.byref(v)) == 0   # dw: few tiles, a long sum


def test_linear_null_size_pointer():
    assert L().moe_linear_workspace(8, 8, 8, 8, 8, 0, None) == 1
    assert L().moe_linear_backward_workspace(8, 8, 8, 8, 8, 8, 0, 7, None) == 1
    v = ctypes.c_size_t()
    for grads in (0, 8, -1):
        assert L().moe_linear_backward_workspace(8, 8, 8, 8, 8, 8, 0, grads, ctypes.byref(v)) == 1


def test_linear_shape():
    a, b = ctypes.c_int(), ctypes.c_int()
    A_, B_ = ctypes.byref(a), ctypes.byref(b)
    for M, N, K, dt in [(0, 8, 8, 0), (8, 0, 8, 0), (8, 8, 0, 0), (8, 8, 8, 3), (8, 8, 2 ** 31 - 1, 0)]:
        assert L().moe_linear_shape(M, N, K, dt, A_, B_) == 1
    assert L().moe_linear_shape(8, 8, 8, 0, None, B_) == 1
    assert L().moe_linear_shape(8, 8, 8, 0, A_, None) == 1
    # few outputs over a long reduction are cut along it; many outputs are not
    assert abi.moe_linear_shape(64, 512, 2560, 2)[1] > 1
    assert abi.moe_linear_shape(32768, 2048, 4096, 2) == (256, 1)
    for dt in (0, 1, 2):  # the workspace holds the partial sums of what the shape says
        for T, d, n in [(1, 8, 8), (64, 2560, 512), (4, 4096, 4096), (512, 4096, 2048)]:
            tile, split = abi.moe_linear_shape(T, n, d, dt)
            want = split * T * n * 4 if split > 1 else 0
            assert ws(T, d, n, d, n, dt) == (0, (want + 255) // 256 * 256)


#          x  ldx w ldw bias res ldr rdt dt act T   d   n  ws bytes   out ldo odt stream
# (97 columns: w's rows are copied into padded ones, so a workspace is needed)
B, C, D, F, H = (A + (i << 20) for i in range(1, 6))  # (never read: refused, or no device)
GOOD = [A, 64, A, 97, A, A, 97, 0, 2, 2, 64, 64, 97, A, 1 << 30, B, 97, 0, N]


@pytest.mark.parametrize("at,value", [
    (0, N), (0, A + 8), (2, N), (2, A + 2), (4, A + 8), (5, A + 4), (15, N), (15, A + 8),
    (1, 63), (3, 96), (6, 96), (16, 96), (1, (1 << 20) + 8), (16, (1 << 20) + 8),
    (7, 1), (7, 5), (8, 3), (9, 4), (9, -1), (17, 1), (17, 7),
    (10, 0), (11, 0), (12, 0), (13, N), (13, A + 128), (14, 0),
])
def test_linear_refuses(at, value):
    args = list(GOOD)
    args[at] = value
    rc, need = ws(64, 64, 97, 64, 97, 2)
    assert rc == 0 and need > 0
    assert L().moe_linear(*args) == 1


#             x ldx w  ldw dz lddz dt T   d   n  ws bytes   dx lddx dw lddw db gdt stream
GOOD_BACK = [A, 64, A, 97, A, 97, 2, 64, 64, 97, A, 1 << 30, B, 64, C, 97, D, 0, N]


@pytest.mark.parametrize("at,value", [
    (0, N), (0, A + 8), (2, N), (2, A + 8), (4, N), (4, A + 8), (12, A + 8), (14, A + 8),
    (16, A + 8), (1, 63), (3, 96), (5, 96), (13, 63), (15, 96), (6, 4), (17, 1), (17, -1),
    (7, 0), (8, 0), (9, 0), (10, A + 16), (11, 0), (13, (1 << 20) + 8), (5, (1 << 20) + 8),
])
def test_linear_backward_refuses(at, value):
    args = list(GOOD_BACK)
    args[at] = value
    assert L().moe_linear_backward(*args) == 1


def test_linear_backward_needs_a_gradient():
    args = list(GOOD_BACK)
    args[12] = args[14] = args[16] = None
    assert L().moe_linear_backward(*args) == 1


def bal(T, E, K):
    v = ctypes.c_size_t()
    return L().moe_balance_workspace(T, E, K, ctypes.byref(v)), v.value


@pytest.mark.parametrize("T,E,K,rc", [(0, 8, 2, 1), (4, 0, 1, 1), (4, 8, 0, 1), (4, 8, 9, 1),
                                      (4, 1025, 2, 2), (4, 512, 65, 2), (2 ** 31 - 1, 8, 2, 1),
                                      (-1, 8, 2, 1)])
def test_balance_sizes_refused(T, E, K, rc):
    assert bal(T, E, K)[0] == rc
    assert L().moe_balance_loss(A, A, T, E, K, A, 1 << 30, A, A, A, N) == rc
    assert L().moe_route_backward(A, A, A, A, A, A, T, E, K, A, 0, N) == rc


def test_balance_refuses():
    rc, need = bal(64, 8, 2)
    assert rc == 0 and need > 0
    assert L().moe_balance_workspace(64, 8, 2, None) == 1
    good = [A, A, 64, 8, 2, A, need, A, A, A, N]
    for at, value in [(0, N), (1, N), (5, N), (7, N), (8, N), (9, N), (0, A + 2), (1, A + 2),
                      (5, A + 128), (6, need - 1), (7, A + 2), (8, A + 1), (9, A + 3)]:
        args = list(good)
        args[at] = value
        assert L().moe_balance_loss(*args) == 1, (at, value)


def test_route_backward_refuses():
    good = [A, A, A, A, A, A, 64, 8, 2, B, 1, N]
    for at, value in [(0, N), (1, N), (2, N), (4, N), (9, N), (0, A + 2), (2, A + 2), (3, A + 1),
                      (5, A + 2), (9, B + 1), (9, A), (10, 3), (10, -1)]:
        args = list(good)
        args[at] = value
        assert L().moe_route_backward(*args) == 1, (at, value)
    args = list(good)
    args[3] = args[5] = None  # no gradient comes in
    assert L().moe_route_backward(*args) == 1


def test_act_forward_refuses():
    #        g ldg u ldu dt act T f h ldh g8 gs u8 us stream
    good = [A, 64, A, 64, 2, 2, 8, 64, A, 64, B, C, D, F, N]
    for at, value in [(0, N), (0, A + 8), (2, A + 8), (8, N), (8, A + 2), (1, 63), (3, 63), (9, 63),
                      (1, (1 << 20) + 1), (4, 3), (5, 0), (5, 4), (6, 0), (7, 0), (10, N), (11, N),
                      (12, N), (13, N), (10, A + 8), (12, A + 8), (2, N)]:
        args = list(good)
        args[at] = value
        assert L().moe_act_forward(*args) == 1, (at, value)


def test_act_backward_refuses():
    #        g8 gs u8 us dh lddh dt act T f dg lddg du lddu h ldh stream
    good = [A, A, A, A, A, 64, 2, 2, 8, 64, A, 64, B, 64, C, 64, N]
    for at, value in [(0, N), (0, A + 8), (1, N), (2, N), (3, N), (2, A + 8), (4, N), (4, A + 2),
                      (5, 63), (6, 3), (7, 0), (7, 4), (8, 0), (9, 0), (10, N), (10, A + 8),
                      (11, 63), (12, N), (12, A + 8), (13, 63), (14, A + 8), (15, 63)]:
        args = list(good)
        args[at] = value
        assert L().moe_act_backward(*args) == 1, (at, value)


def test_outputs_on_other_arguments_are_refused():
    """an output may be an input only where the call names it, element on element"""
    def rc(call, good, *changes):
        args = list(good)
        for at, value in changes:
            args[at] = value
        return getattr(L(), call)(*args)

    fwd = list(GOOD)
    fwd[0], fwd[2], fwd[4], fwd[5] = A, C, D, F
    for at in (0, 2, 4):
        assert rc("moe_linear", fwd, (15, fwd[at])) == 1
    assert rc("moe_linear", fwd, (15, F), (17, 2)) == 1            # residual: fp32, out: not
    assert rc("moe_linear", fwd, (15, F), (16, 98)) == 1           # another stride
    back = list(GOOD_BACK)
    back[0], back[2], back[4] = A, F, H
    for at, value in [(12, F), (12, H), (14, A), (14, H), (16, H), (12, C), (16, C), (16, B)]:
        assert rc("moe_linear_backward", back, (at, value)) == 1, (at, value)
    #        g ldg u ldu dt act T f h ldh g8 gs u8 us stream
    act = [A, 64, B, 64, 2, 2, 8, 64, C, 64, D, F, H, H + 4096, N]
    for changes in [((8, A), (9, 72)), ((8, B), (9, 72)), ((12, D),), ((13, F),)]:
        assert rc("moe_act_forward", act, *changes) == 1, changes
    #         g8 gs u8 us dh lddh dt act T f dg lddg du lddu h ldh stream
    grad = [H, H, H, H, A, 64, 2, 2, 8, 64, B, 64, C, 64, D, 64, N]
    for changes in [((10, A), (11, 72)), ((12, A), (13, 72)), ((14, A), (15, 72)), ((12, B),),
                    ((14, B),), ((14, C),)]:
        assert rc("moe_act_backward", grad, *changes) == 1, changes


def test_helpers_refuse_host_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(8, 8)
    for call in (lambda: abi.linear(x, w), lambda: abi.linear_backward(x, w, x),
                 lambda: abi.balance_loss(x, torch.zeros(4, 2, dtype=torch.int32)),
                 lambda: abi.route_backward(x, torch.zeros(4, 2, dtype=torch.int32), None, None,
                                            torch.zeros(10, dtype=torch.int32), torch.zeros(2)),
                 lambda: abi.act_forward(x), lambda: abi.act_backward({}, x)):
        with pytest.raises(TypeError):
            call()


def _gpu_visible():
    return torch.cuda.device_count() > 0


@pytest.mark.skipif(_gpu_visible(), reason="only meaningful on a machine without a GPU")
def test_no_device_gives_ehip_without_crash():
    assert L().moe_linear(*GOOD) == 3
    assert L().moe_linear_backward(*GOOD_BACK) == 3
    assert L().moe_balance_loss(A, A, 64, 8, 2, A, 1 << 20, A, A, A, N) == 3
    assert L().moe_route_backward(A, A, A, A, A, A, 64, 8, 2, B, 0, N) == 3
    assert L().moe_act_forward(A, 64, A, 64, 2, 2, 8, 64, A, 64, B, C, D, F, N) == 3
    assert L().moe_act_backward(A, A, A, A, A, 64, 2, 2, 8, 64, A, 64, B, 64, C, 64, N) == 3
