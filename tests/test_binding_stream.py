"""The stream handle that the binding hands to the library (no GPU)."""
import types

import pytest
import torch

from tree_verification_jsv_b200 import jsv


def test_given_streams():
    assert jsv._stream(77) == 77
    assert jsv._stream(types.SimpleNamespace(cuda_stream=78)) == 78


@pytest.mark.parametrize("missing", [(), ("_cuda_getCurrentRawStream",), ("_cuda_getDevice",),
                                     ("_cuda_getCurrentRawStream", "_cuda_getDevice")])
@pytest.mark.parametrize("initialised", [False, True])
def test_current_stream_of_the_current_device(monkeypatch, missing, initialised):
    """With and without torch's private shortcuts, which a version may lack."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: initialised)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=103))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    assert jsv._stream(None) == 103
