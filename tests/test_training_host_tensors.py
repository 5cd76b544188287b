"""The binding on the host: versions of tensors that a call wrote, streams of another device."""
from types import SimpleNamespace

import pytest
import torch

from unbiased_nvfp4_gradient_amd import _tensors, training


def test_written_tensors_count_a_version():
    a, b, c = torch.zeros(4), torch.nn.Parameter(torch.zeros(2)), torch.zeros(3)
    view = a[1:]
    _tensors.written([a, b])
    assert a._version == 1 and b._version == 1 and view._version == 1 and c._version == 0
    x = torch.ones(4, requires_grad=True)
    y = 2.0 * x
    z = y.square().sum()
    _tensors.written([y.detach()])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    with torch.inference_mode():
        _tensors.written([torch.zeros(4)])
    for bad in ((a,), [a, None]):
        with pytest.raises(TypeError):
            _tensors.written(bad)


def test_stream_of_another_device_is_refused():
    # kernels would run on the stream's device with the other's addresses
    stream = SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    with pytest.raises(ValueError, match="stream must be one of the tensors' device, cuda:0"):
        training._where(stream, torch.device("cuda:0"))
