"""Which stream a call runs on, for every form that `stream` may take: torch's
stream calls are stand-ins, so nothing reaches a GPU."""

from __future__ import annotations

import contextlib
import types

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv

DEV = torch.device("cuda", 0)


@pytest.fixture
def entered(monkeypatch):
    """The handles of the streams that were made current, one after the other. As torch does, the stand-in of
    ExternalStream takes handle 0 for none given and makes a stream of its own."""
    made = []

    @contextlib.contextmanager
    def stream(s):
        made.append(s.cuda_stream)
        yield

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: types.SimpleNamespace(cuda_stream=0, device=device))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: types.SimpleNamespace(cuda_stream=handle or 0xBAD, device=device))
    return made


@pytest.mark.parametrize("stream,handle", [(0, 0), (0x7000, 0x7000), (types.SimpleNamespace(cuda_stream=0), 0),
                                           (types.SimpleNamespace(cuda_stream=0x7100), 0x7100)])
def test_a_stream_by_its_handle(entered, stream, handle):
    with nv._under(stream, DEV):
        pass
    assert entered == [handle]


@pytest.mark.parametrize("stream,handle", [(0, 0), (0x7000, 0x7000), (types.SimpleNamespace(cuda_stream=0x7100), 0x7100)])
def test_a_workspace_is_cleared_on_the_stream_that_uses_it(entered, monkeypatch, stream, handle):
    monkeypatch.setattr(nv, "_workspaces", {})
    cleared = []
    monkeypatch.setattr(nv, "empty_workspace", lambda device: cleared.append((device, list(entered))) or object())
    ws = nv.stream_workspace(DEV, stream)
    assert cleared == [(DEV, [handle])]
    assert nv.stream_workspace(DEV, handle) is ws and len(cleared) == 1


@pytest.fixture
def current(monkeypatch):
    """Device 0 is the current one, until another is made current; the list holds those that were."""
    seen = [0]

    @contextlib.contextmanager
    def device(d):
        seen.append(d if isinstance(d, int) else d.index)
        yield
        seen.append(0)

    monkeypatch.setattr(nv, "_current_device", lambda: seen[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    return seen


def test_calls_make_their_tensors_device_the_current_one(entered, current):
    assert nv._elsewhere(None, DEV) is None  # it is already
    with nv._elsewhere(None, torch.device("cuda", 1)):
        assert current == [0, 1]
        assert nv._elsewhere(None, torch.device("cuda", 1)) is None
    with nv._elsewhere(0x7000, torch.device("cuda", 1)):
        assert entered == [0x7000]


def test_calls_refuse_a_stream_of_another_device(entered, current):
    with pytest.raises(ValueError, match="cuda:1"):
        nv._elsewhere(types.SimpleNamespace(cuda_stream=0x7000, device=torch.device("cuda", 1)), DEV)


@pytest.mark.parametrize("index,seen", [(0, [0]), (1, [0, 1, 0])])
def test_quantize_calls_make_their_tensors_device_the_current_one(current, index, seen):
    class OnDevice(torch.Tensor):  # a tensor that says it is on a GPU
        def get_device(self):
            return index

    t = torch.zeros(4).as_subclass(OnDevice)
    inside = []
    call = nv._on_its_device(lambda x, n=0: inside.append(list(current)) or n)
    assert call(t, n=3) == 3 and call(nv.Orientation(t, t, t), 4) == 4
    assert current == seen + seen[1:] and inside[0] == seen[:2]
    assert call(torch.zeros(4), 5) == 5  # not on a GPU: the call itself refuses it
    before = len(current)
    assert call(x=t) == 0 and len(current) - before == (2 if index else 0)


def test_every_quantize_call_has_that_guard():
    for name in ("nvfp4_compute_amax", "nvfp4_quantize", "nvfp4_quantize_noalloc", "nvfp4_dequantize", "nvfp4_quantize_grouped",
                 "nvfp4_swizzle_scales", "nvfp4_debug_rht_colwise", "nvfp4_debug_e2m1_pack", "quantize", "quantize_grouped"):
        assert hasattr(getattr(nv, name), "__wrapped__"), name
