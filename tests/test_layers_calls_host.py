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


def scratch(tsx, backward, n, l, c, groups, dtype=1, aligned=0):
    import ctypes

    d = tsx.tsx_norm_desc(dtype, 2, 1, groups, 0, 128, n, l, c, c, c, 1e-5)
    size = ctypes.c_size_t()
    assert tsx.tsx_group_norm_workspace(ctypes.byref(d), backward, aligned, ctypes.byref(size)) == tsx.TSX_OK
    return size.value


@pytest.mark.parametrize("n,l,c,groups", [
    (8192, 1, 4096, 1), (8192, 1, 4096, 8), (65536, 1, 4096, 1), (8192, 1, 2560, 32), (8192, 1, 1024, 1),
    (8192, 2, 4096, 8), (7088, 3, 352, 11), (7088, 3, 363, 11), (2000, 64, 256, 32), (2000, 1, 6000, 1),
    (300, 1, 65536, 1), (300, 2, 65536, 2), (16384, 1, 8192, 1), (16384, 1, 8191, 1), (1 << 20, 1, 33, 3),
    (1 << 20, 1, 40, 5), (1, 262144, 128, 32), (4, 16384, 512, 32), (256, 256, 512, 32), (100000, 7, 96, 32)])
@pytest.mark.parametrize("dtype,size", [(0, 2), (1, 2), (2, 4)])
def test_scratch_of_the_gradient_does_not_grow_with_the_samples(tsx, n, l, c, groups, dtype, size):
    """Sums for dweight and dbias: 16 MB, or one slice of two floats to a
    channel; beside them a few bytes to a sample's group and range."""
    slices = max(16 << 20, 8 * c)
    pieces = -(-c // groups // 2048)
    parts = 8 * groups * (n + 608) * pieces + 16
    for backward in (0, 1):
        for aligned in (0, 1):
            assert scratch(tsx, backward, n, l, c, groups, dtype, aligned) <= parts + backward * slices
    assert scratch(tsx, 1, n, l, c, groups, dtype) <= n * l * c * size // 2 + (18 << 20)
