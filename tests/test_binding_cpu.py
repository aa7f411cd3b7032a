"""The binding's checks that need no GPU."""

import pytest
import torch

from retnet_retention_amd import binding


@pytest.fixture
def no_library(monkeypatch):
    """A library that must not be reached."""

    class Reached:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was reached")

    monkeypatch.setattr(binding, "_lib", Reached())


@pytest.mark.parametrize("call", [binding.chunkwise_error, binding.check_chunkwise])
def test_a_workspace_on_the_host_is_refused(no_library, call):
    """Its address is none of the GPU's."""
    with pytest.raises((ValueError, RuntimeError)) as e:
        call(torch.zeros(64, dtype=torch.uint8))
    assert "reached" not in str(e.value)


def test_the_stream_of_a_host_tensor_is_refused():
    with pytest.raises((ValueError, RuntimeError)):
        binding._stream(torch.zeros(1))


def test_streams_without_the_raw_handle(monkeypatch):
    """A torch that lacks the private name still loads the binding and finds its streams."""
    import importlib.util

    name = "_cuda_getCurrentRawStream"
    if hasattr(torch._C, name):
        monkeypatch.delattr(torch._C, name)
    spec = importlib.util.spec_from_file_location("binding_again", binding.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: Stream)

    class OnGpu:
        def get_device(self):
            return 0

    assert again._stream(OnGpu()) == 77
