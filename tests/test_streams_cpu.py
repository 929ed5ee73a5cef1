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
