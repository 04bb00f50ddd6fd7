"""The binding's scratch buffers and streams."""
import pytest
import torch

from bit_quantization_b200 import ops

pytestmark = pytest.mark.gpu


def test_workspace_of_the_current_device_without_its_index():
    ws = ops.Workspace()
    a = ws.get(1000, "cuda")
    assert a.numel() >= 1000 and a.get_device() == torch.cuda.current_device()
    assert ws.get(10, torch.device("cuda", torch.cuda.current_device())) is a
    with torch.cuda.stream(torch.cuda.Stream()):
        assert ws.get(1000, "cuda") is not a  # another stream, another buffer


def test_streams_are_the_current_ones():
    index = torch.cuda.current_device()
    for stream in [torch.cuda.default_stream()] + [torch.cuda.Stream() for _ in range(3)]:
        with torch.cuda.stream(stream):
            assert ops._raw_stream(index) == torch.cuda.current_stream(index).cuda_stream
            assert ops._raw_stream(index) == stream.cuda_stream
