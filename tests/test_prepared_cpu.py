"""Where a prepared call takes its stream from, with torch's calls faked (no
GPU): with torch's raw handles and without either of them."""
from types import SimpleNamespace

import pytest
import torch

import paged_kv_cache_274_gb300 as pkv


@pytest.fixture
def device(monkeypatch):
    """A fake machine: current device 1, stream handles 1000 + device."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: SimpleNamespace(cuda_stream=1000 + (1 if d is None else d)))


@pytest.mark.parametrize("raw", [True, False])
@pytest.mark.parametrize("here", [True, False])
def test_current_handle(device, monkeypatch, raw, here):
    monkeypatch.setattr(pkv, "_raw_stream", (lambda d: 1000 + d) if raw else None)
    monkeypatch.setattr(pkv, "_get_device", (lambda: 1) if here else None)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    assert pkv._current_handle(1) == 1001
    with pytest.raises(pkv.PkvError) as e:
        pkv._current_handle(0)
    assert e.value.status == 1 and "cuda:0" in str(e.value) and "cuda:1" in str(e.value)


def _prepared(kind, device, stream=None):
    call = object.__new__(kind)
    seen = []
    call._fn, call._args = lambda *a: seen.append(a) or 0, (7,)
    call._device = device
    call._stream = stream
    call.out = call.result = "result"
    return call, seen


@pytest.mark.parametrize("kind", [pkv.PreparedDecode, pkv.PreparedCall])
def test_prepared_calls_launch_on_their_tensors_device_only(device, monkeypatch, kind):
    monkeypatch.setattr(pkv, "_raw_stream", None)
    monkeypatch.setattr(pkv, "_get_device", None)
    other = SimpleNamespace(cuda_stream=77)
    call, seen = _prepared(kind, 1)
    assert call() == "result" and call(stream=other) == "result"
    assert seen[0] == (7, 1001) and seen[1][1].value == 77
    call, seen = _prepared(kind, 1, stream=55)
    assert call() == "result" and seen == [(7, 55)]
    for bound in (None, 55):  # whatever the stream: the call would run on another device than its tensors
        call, seen = _prepared(kind, 0, bound)
        for s in (None, other):
            with pytest.raises(pkv.PkvError):
                call(stream=s)
        assert not seen
