"""On which device and stream the binding allocates what it returns (no GPU: torch.cuda is replaced)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from paged_variable_length_gb300 import pva


@pytest.fixture
def calls(monkeypatch):
    """The process's current device is 0, whose current stream is 5; device 1's is 7."""
    log = []
    monkeypatch.setattr(pva, "_raw_stream", (lambda dev: {0: 5, 1: 7}[dev], lambda: 0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: ("external", h, str(device)))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", str(device)))

    @contextlib.contextmanager
    def use(stream):
        log.append(stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype, device: log.append((shape, dtype, str(device))))
    return log


@pytest.mark.parametrize("index", [0, 1])
def test_the_tensor_belongs_to_the_stream_on_its_own_device(calls, index):
    like = SimpleNamespace(device=f"cuda:{index}", get_device=lambda: index)
    made = ((4, 2), torch.bfloat16, f"cuda:{index}")
    other = SimpleNamespace(cuda_stream=99)
    current = 7 if index else 5
    for stream, want in ((None, []), (current, []), (SimpleNamespace(cuda_stream=current), []), (other, [other]),
                         (99, [("external", 99, f"cuda:{index}")]), (0, [("default", f"cuda:{index}")])):
        calls.clear()
        pva.PagedAttention._empty((4, 2), like, stream)
        assert calls == want + [made]


def test_the_type_asked_for(calls):
    like = SimpleNamespace(device="cuda:0", get_device=lambda: 0)
    pva.PagedAttention._empty((3,), like, None, torch.float16)
    assert calls == [((3,), torch.float16, "cuda:0")]
