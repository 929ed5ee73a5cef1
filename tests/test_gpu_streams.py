"""GPU: the stream handle that each expert-layer call launches on."""

from __future__ import annotations

import types

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


class Recorder:
    """The library, with the last argument (the stream) of each launching call noted."""

    def __init__(self, lib):
        self.lib, self.handles = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)

        def call(*args):
            if f.restype is not None and len(args) >= 9:  # the calls that launch; the size queries have fewer
                self.handles.append(getattr(args[-1], "value", args[-1]) or 0)
            return f(*args)

        return call


def calls():
    """Every call, on operands made on the default stream."""
    ids = torch.randint(0, 3, (40, 2), dtype=torch.int32, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    x = torch.randn((40, 128), device=DEV)
    plan = nv.expert_sort(ids, 3)
    y, w = nv.expert_gather(x, plan), torch.rand((40, 2), device=DEV)
    a, at = nv.fp8_quantize(x, columnwise=True, plan=plan)
    b, _ = nv.fp8_quantize(torch.randn((3, 64, 128), device=DEV), block_2d=True)
    one = nv.Fp8Tensor(b.data[0], b.scales[0], 64, 128, True)
    return {
        "sort": lambda s: nv.expert_sort(ids, 3, stream=s).slot_rows, "gather": lambda s: nv.expert_gather(x, plan, stream=s),
        "combine": lambda s: nv.expert_combine(y, plan, w, stream=s), "gather_grad": lambda s: nv.expert_gather_grad(y, plan, stream=s),
        "combine_grad": lambda s: nv.expert_combine_grad(x, y, plan, w, stream=s)[0],
        "quantize": lambda s: nv.fp8_quantize(x, plan=plan, stream=s)[0].scales, "matmul": lambda s: nv.fp8_matmul(a, one, stream=s),
        "grouped": lambda s: nv.fp8_matmul_grouped(a, b, plan, stream=s), "grouped_k": lambda s: nv.fp8_matmul_grouped_k(at, at, plan, stream=s),
    }


@pytest.mark.parametrize("name", ["sort", "gather", "combine", "gather_grad", "combine_grad", "quantize", "matmul", "grouped", "grouped_k"])
def test_the_stream_that_was_given_is_the_one_launched_on(monkeypatch, name):
    call = calls()[name]
    want = call(None)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    assert torch.cuda.default_stream().cuda_stream == 0
    recorder = Recorder(nv.load())
    monkeypatch.setattr(nv, "load", lambda: recorder)
    with torch.cuda.stream(other):  # so that the current stream is none of those given
        got = []
        for given in (0, types.SimpleNamespace(cuda_stream=0), torch.cuda.default_stream(), side, side.cuda_stream,
                      types.SimpleNamespace(cuda_stream=side.cuda_stream), None):
            got.append(call(given))
    torch.cuda.synchronize()
    assert recorder.handles == [0, 0, 0] + [side.cuda_stream] * 3 + [other.cuda_stream]
    assert all(torch.equal(g, want) for g in got)


def test_a_grouped_call_clears_its_workspace_on_its_stream(monkeypatch):
    x = torch.randn((64, 128), device=DEV)
    want, _ = nv.quantize_grouped(x, [16, 48], columnwise=False)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    cleared_on, real = [], nv.empty_workspace
    monkeypatch.setattr(nv, "empty_workspace", lambda device: cleared_on.append(torch.cuda.current_stream().cuda_stream) or real(device))
    with torch.cuda.stream(other):
        got = [nv.quantize_grouped(x, [16, 48], columnwise=False, stream=s)[0] for s in (0, side, side.cuda_stream, None)]
    torch.cuda.synchronize()
    assert cleared_on == [0, side.cuda_stream, side.cuda_stream, other.cuda_stream]
    for g in got:
        assert torch.equal(g.data, want.data) and torch.equal(g.scales, want.scales) and torch.equal(g.amax, want.amax)


@pytest.mark.parametrize("name", ["sort", "gather", "combine", "gather_grad", "combine_grad", "quantize", "matmul", "grouped", "grouped_k"])
def test_the_tensors_device_is_made_the_current_one(monkeypatch, name):
    call = calls()[name]
    want = call(None)
    entered = []

    class Noted(torch.cuda.device):
        def __enter__(self):
            entered.append(self.idx)
            return super().__enter__()

    monkeypatch.setattr(nv, "_current_device", lambda: 0 if entered else 1)
    monkeypatch.setattr(torch.cuda, "device", Noted)
    assert torch.equal(call(None), want) and entered == [want.device.index]
