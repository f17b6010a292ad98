"""Device and stream of a dense helper's call, on the CPU with stand-ins: a stream
of another GPU than the tensors' is refused before anything is launched, and the
current device is left as it was."""
import pytest
import torch

from mixture_experts_routed_amd import abi


class OnGpu(torch.Tensor):
    """a tensor that says it is on GPU 1"""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 1


class Stream:
    cuda_stream = 7

    def __init__(self, index):
        self.device_index = index


@pytest.fixture
def devices(monkeypatch):
    """the current device, as torch would keep it"""
    now = [0]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "set_device", lambda i: now.__setitem__(0, i))
    return now


def test_stream_of_another_device_is_refused(devices):
    x = torch.zeros(4, 8).as_subclass(OnGpu)
    with pytest.raises(ValueError, match="stream: on GPU 0, expected GPU 1"):
        abi.linear(x, x, stream=Stream(0))
    with pytest.raises(ValueError, match="stream"):
        abi.act_forward(x, stream=Stream(2))
    assert devices == [0]


def test_the_tensors_device_is_current_within_a_call(devices):
    x = torch.zeros(4, 8).as_subclass(OnGpu)
    for stream, handle in ((Stream(1), 7), (99, 99)):
        with abi._On(x, "x", stream) as at:
            assert devices == [1] and at.handle == handle
        assert devices == [0]
    with pytest.raises(RuntimeError):
        with abi._On(x, "x", Stream(1)):
            raise RuntimeError
    assert devices == [0]
