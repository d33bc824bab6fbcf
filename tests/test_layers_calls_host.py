"""What the Python classes of the layer operators check before any GPU call."""

import types

import pytest


@pytest.fixture(scope="module")
def tsx():
    import __graft_entry__

    __graft_entry__.build()
    import pipelined_elementwise_streaming_gb300 as m

    return m


class Fake:
    """A tensor on a device that no test has."""

    def __init__(self, device):
        import torch

        self.device, self.is_cuda = torch.device("cuda", device), True

    def get_device(self):
        return self.device.index


def test_a_stream_of_another_device_is_refused(tsx, monkeypatch):
    """Not left aside for the current stream of the tensors' device."""
    import torch

    stream = types.SimpleNamespace(device=torch.device("cuda", 1), device_index=1)
    x = Fake(0)
    norm, glu, pack = tsx.GroupNorm("bf16", 2, 3, 8, 2), tsx.GatedAct("bf16", 4, 8), tsx.Packer("bf16", 4, 8)
    for op in (norm, glu, pack):
        monkeypatch.setattr(op, "_device", lambda: 0)
    for call in (lambda: norm.forward(x, x, x, stream=stream), lambda: norm.backward(x, x, x, x, x, x, stream=stream),
                 lambda: glu.forward(x, x, stream=stream), lambda: glu.backward(x, x, x, stream=stream),
                 lambda: pack.pack(x, stream=stream), lambda: pack.unpack((x, x), stream=stream)):
        with pytest.raises(tsx.TsxError) as e:
            call()
        assert e.value.code == tsx.TSX_ERR_INVALID and "stream" in str(e.value) and "cuda:1" in str(e.value)
