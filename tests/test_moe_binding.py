"""The expert-side binding's device check, without a GPU: a library that notes every call instead of making it."""
import types

import pytest
import torch

from weight_only_int4_route_gb300 import moe


@pytest.fixture
def calls(monkeypatch):
    """The library calls made.  GPU 0 is current."""
    made = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: made.append(name) or 0

    monkeypatch.setattr(moe, "lib", Library)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    return made


def test_the_current_gpu_is_taken(calls):
    for dev in ("cuda:0", "cuda"):
        assert moe.device_error(dev) == 0 and moe.check_status(dev) == (0, 0)
    assert len(calls) == 4


def test_another_gpu_is_refused(calls):
    """The library launches on the current GPU: a call for another one's tensors must not reach it."""
    class Fake(torch.Tensor):
        device = torch.device("cuda:1")

    ids = torch.zeros((1, 2, 2), dtype=torch.int32).as_subclass(Fake)
    counts = torch.zeros((1, 4), dtype=torch.int32).as_subclass(Fake)
    layer = types.SimpleNamespace(max_T=4, p=types.SimpleNamespace(w1=counts))
    for call in (lambda: moe.device_error("cuda:1"), lambda: moe.check_status("cuda:1"),
                 lambda: moe.elb_accumulate(ids, 4, counts), lambda: moe.LayerGraph(layer, 1)):
        with pytest.raises(AssertionError):
            call()
    assert not calls
