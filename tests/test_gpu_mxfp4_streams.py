"""GPU: the stream and the device that each MXFP4 call, and the expert layer for a few tokens, launches on."""

from __future__ import annotations

import types

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

NAMES = ["quantize", "dequantize", "matmul", "grouped", "grouped_k", "mlp_mxfp4", "mlp_fp8"]


class Recorder:
    """The library, with the last argument (the stream) of each launching call noted."""

    def __init__(self, lib):
        self.lib, self.handles = lib, []

    def __getattr__(self, name):
        f = getattr(self.lib, name)

        def call(*args):
            if name.startswith(("nvfp4_mxfp4_", "nvfp4_expert_mlp_")) and not name.endswith("_bytes"):
                self.handles.append(getattr(args[-1], "value", args[-1]) or 0)
            return f(*args)

        return call


def calls():
    """Every call, on operands made on the default stream."""
    g = torch.Generator(DEV).manual_seed(1)
    ids = torch.randint(0, 3, (40, 2), dtype=torch.int32, device=DEV, generator=g)
    x, w = torch.randn((40, 128), device=DEV, generator=g), torch.rand((40, 2), device=DEV, generator=g)
    plan = nv.expert_sort(ids, 3)
    w1, w2 = torch.randn((3, 64, 128), device=DEV, generator=g), torch.randn((3, 128, 32), device=DEV, generator=g)
    a, at = nv.mxfp4_quantize(x, columnwise=True, plan=plan)
    b, b2 = nv.mxfp4_quantize(w1)[0], nv.mxfp4_quantize(w2)[0]
    f, f2 = (nv.fp8_quantize(v, block_2d=True)[0] for v in (w1, w2))
    one = nv.Mxfp4Tensor(b.data[0], b.scales[0], 64, 128)
    return {
        "quantize": lambda s: nv.mxfp4_quantize(x, plan=plan, stream=s)[0].data, "dequantize": lambda s: nv.mxfp4_dequantize(a, stream=s),
        "matmul": lambda s: nv.mxfp4_matmul(a, one, stream=s), "grouped": lambda s: nv.mxfp4_matmul_grouped(a, b, plan, stream=s),
        "grouped_k": lambda s: nv.mxfp4_matmul_grouped_k(at, at, plan, stream=s),
        "mlp_mxfp4": lambda s: nv.expert_mlp(x.bfloat16(), ids, w, b, b2, stream=s), "mlp_fp8": lambda s: nv.expert_mlp(x.bfloat16(), ids, w, f, f2, stream=s),
    }


@pytest.mark.parametrize("name", NAMES)
def test_the_stream_that_was_given_is_the_one_launched_on(monkeypatch, name):
    call = calls()[name]
    want = call(None)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    recorder = Recorder(nv.load())
    monkeypatch.setattr(nv, "load", lambda: recorder)
    with torch.cuda.stream(other):  # so that the current stream is none of those given
        got = []
        for given in (0, types.SimpleNamespace(cuda_stream=0), torch.cuda.default_stream(), side, side.cuda_stream, None):
            got.append(call(given))
            torch.cuda.synchronize()
    assert recorder.handles == [0, 0, 0] + [side.cuda_stream] * 2 + [other.cuda_stream]
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("name", NAMES)
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
