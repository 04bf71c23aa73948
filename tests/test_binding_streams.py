"""The torch binding without a GPU: a stream of another device than the tensors' is refused before anything is launched."""
import pytest
import torch

import selective_state_space_14_amd as ssd


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the first GPU."""
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", 0))


class Stream:
    cuda_stream = 0x10000

    def __init__(self, index):
        self.device = torch.device("cuda", index)


CALLS = {
    "ssd_delta_scan_fwd": lambda x, **kw: ssd.ssd_delta_scan_fwd(x, x, x, x, x, x, H=1, P=64, N=64, G=1, **kw),
    "ssd_delta_step": lambda x, **kw: ssd.ssd_delta_step(x, x, x, x, x, x, x, H=1, P=64, N=64, G=1, **kw),
    "ssd_delta_scan_bwd": lambda x, **kw: ssd.ssd_delta_scan_bwd(x, x, x, x, x, x, x, H=1, P=64, N=64, G=1, **kw),
    "ssd_norm_fwd": lambda x, **kw: ssd.ssd_norm_fwd(x, **kw),
    "ssd_norm_bwd": lambda x, **kw: ssd.ssd_norm_bwd(x, x, **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name, monkeypatch):
    x = torch.zeros(1, 1, 64).as_subclass(OnGpu)

    def entered(stream, device=None):
        raise AssertionError("the stream was made current")

    monkeypatch.setattr(torch.cuda, "stream", entered)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(device.index))
    with pytest.raises(ValueError, match="stream: on cuda:1, expected cuda:0"):
        CALLS[name](x, stream=Stream(1))
    for mine in (Stream(0), 0x10000):
        with pytest.raises(AssertionError, match="made current"):
            CALLS[name](x, stream=mine)
