"""What the dense operators' Python helpers refuse by name: an activation or a type
that does not exist, a matrix or array that does not start at a 16-byte boundary."""
import pytest
import torch

from gpu_util import abi

pytestmark = pytest.mark.gpu


def z(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def test_unknown_activations():
    x, w = z(4, 8), z(8, 8)
    _, ck = abi.act_forward(x, ckpt=True)
    for call in (lambda: abi.linear(x, w, act="tanh"), lambda: abi.act_forward(x, act="tanh"),
                 lambda: abi.act_backward(ck, x, act="tanh")):
        with pytest.raises(ValueError, match="act: .*tanh"):
            call()


def test_unknown_types():
    d = torch.float64
    x, w, l, i = z(4, 8, dtype=d), z(8, 8, dtype=d), z(4, 8), z(4, 2, dtype=torch.int32)
    _, ck = abi.act_forward(l, ckpt=True)
    for call in (lambda: abi.linear(x, w), lambda: abi.linear_backward(x, w, x),
                 lambda: abi.act_forward(x), lambda: abi.act_backward(ck, x),
                 lambda: abi.route_backward(l, i, None, None, z(10, dtype=torch.int32), z(2),
                                            out_dtype=d)):
        with pytest.raises(TypeError, match="float64"):
            call()


def test_first_elements_that_are_not_at_16_bytes():
    h = torch.bfloat16
    x, w, y = z(4, 8, dtype=h), z(8, 8, dtype=h), z(4, 8, dtype=h)
    odd = z(5, 9, dtype=h)[1:, 1:]  # [4, 8] from byte 20
    bias, column = z(9, dtype=h)[1:], z(8, 9, dtype=h)[:, 1:]
    _, ck = abi.act_forward(x, y, ckpt=True)
    codes = torch.zeros(40, dtype=torch.uint8, device="cuda")[8:].view(torch.float8_e4m3fn).view(4, 8)
    for name, call in (
            ("x", lambda: abi.linear(odd, w)), ("w", lambda: abi.linear(x, column)),
            ("bias", lambda: abi.linear(x, w, bias=bias)),
            ("residual", lambda: abi.linear(x, w, residual=odd)),
            ("out", lambda: abi.linear(x, w, out=odd)),
            ("dz", lambda: abi.linear_backward(x, w, odd)),
            ("dx", lambda: abi.linear_backward(x, w, y, dx=odd)),
            ("dw", lambda: abi.linear_backward(x, w, y, dw=column)),
            ("db", lambda: abi.linear_backward(x, w, y, db=bias)),
            ("g", lambda: abi.act_forward(odd)), ("u", lambda: abi.act_forward(x, odd)),
            ("h", lambda: abi.act_forward(x, h=odd)), ("dh", lambda: abi.act_backward(ck, odd)),
            ("g8", lambda: abi.act_backward({**ck, "g8": codes}, y))):
        with pytest.raises(ValueError, match=f"^{name}: .*16-byte"):
            call()


def test_a_slice_at_16_bytes_is_served():
    x, w = z(9, 16).normal_(), z(16, 12).normal_()
    want, _ = abi.linear(x, w)
    got, _ = abi.linear(x[2:], w)  # two rows of 64 bytes on
    assert torch.equal(got, want[2:])


def test_operands_that_are_not_read_may_start_anywhere():
    x, w, y = z(4, 8).normal_(), z(8, 12).normal_(), z(4, 12).normal_()
    ox, ow = z(5, 9)[1:, 1:], z(8, 13)[:, 1:]
    want, _ = abi.linear_backward(x, w, y)
    assert torch.equal(abi.linear_backward(ox, w, y, grads=("dx",))[0]["dx"], want["dx"])
    assert torch.equal(abi.linear_backward(x, ow, y, grads=("dw",))[0]["dw"], want["dw"])
    assert torch.equal(abi.linear_backward(ox, ow, y, grads=("db",))[0]["db"], want["db"])
