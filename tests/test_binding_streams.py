"""Which stream a call runs on, against a stand-in for torch (no GPU): the current stream of the tensors' device, found
with or without torch's raw query; an explicit stream, which has to be on that device."""
import contextlib
import types

import pytest

import sampling_gated_lora_b200 as U


class _Device:
    def __init__(self, kind, index=None):
        self.type, self.index = kind, index

    def __eq__(self, other):
        return (self.type, self.index) == (other.type, other.index)


class _Torch:
    """Device 1 is current; device i's current stream is 100 + i."""

    def __init__(self, raw):
        self.raw_stream = (lambda i: 100 + i) if raw else None
        self.entered = []
        self.device = _Device
        index = lambda d: 1 if d is None else d if isinstance(d, int) else d.index   # noqa: E731
        self.cuda = types.SimpleNamespace(
            current_device=lambda: 1, device=self._enter,
            current_stream=lambda d=None: types.SimpleNamespace(cuda_stream=100 + index(d), device=_Device("cuda", index(d))))

    @contextlib.contextmanager
    def _enter(self, device):
        self.entered.append(device.index)
        yield


@pytest.mark.parametrize("raw", [True, False])
def test_the_current_stream_of_the_device(monkeypatch, raw):
    fake = _Torch(raw)
    monkeypatch.setattr(U, "_torch_module", fake)
    monkeypatch.setattr(U, "_raw_stream", fake.raw_stream)
    calls = []
    fn = lambda *a: calls.append(a) or 0   # noqa: E731
    U._launch_on(1, None, fn, 7)
    U._launch_on(0, None, fn, 8)
    U._launch(_Device("cuda", 1), None, fn, 9)
    U._launch(_Device("cuda", 2), None, fn, 10)
    assert calls == [(7, 101), (8, 100), (9, 101), (10, 102)]
    assert fake.entered == [0, 2]   # only where the tensors' device is not the current one


@pytest.mark.parametrize("raw", [True, False])
def test_an_explicit_stream(monkeypatch, raw):
    fake = _Torch(raw)
    monkeypatch.setattr(U, "_torch_module", fake)
    monkeypatch.setattr(U, "_raw_stream", fake.raw_stream)
    calls = []
    fn = lambda *a: calls.append(a) or 0   # noqa: E731
    s = types.SimpleNamespace(cuda_stream=55, device=_Device("cuda", 1))
    U._launch_on(1, s, fn, 1)
    assert calls == [(1, 55)]
    with pytest.raises(ValueError, match="stream is on"):
        U._launch(_Device("cuda", 0), s, fn, 2)
