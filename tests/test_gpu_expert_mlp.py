"""GPU: the expert layer for a few tokens, against a plain 64-bit form."""

from __future__ import annotations

import pytest
import torch

import fp8_helpers as F
import mxfp4_helpers as M
import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def layer(kind, experts, cols, hidden, gated, seed):
    g = gen(seed)
    w1 = torch.randn((experts, (1 + gated) * hidden, cols), device=DEV, generator=g) * cols ** -0.5
    w2 = torch.randn((experts, cols, hidden), device=DEV, generator=g) * hidden ** -0.5
    if kind == "fp8":
        return nv.fp8_quantize(w1, block_2d=True)[0], nv.fp8_quantize(w2, block_2d=True)[0]
    return nv.mxfp4_quantize(w1)[0], nv.mxfp4_quantize(w2)[0]


def check(out, x, ids, weights, w1, w2, gated, what=""):
    """out against the definition. h is a BF16 number and another for what the first rounds away: off by 2^-8 2^-8 of itself,
    whose effect on the sum is at most 2^-16 of its terms' magnitudes; binary32's own errors, of n terms each, and of the activation (a few steps of 2^-23 of its value and of
    what its argument is off by, at most 1.1 times that) are below."""
    values = F.values if isinstance(w1, nv.Fp8Tensor) else M.values
    cols, hidden = x.shape[1], w2.k
    want = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(want)
    for e in range(w2.data.shape[0]):
        token, choice = (ids == e).nonzero(as_tuple=True)
        if not token.numel():
            continue
        v1, v2 = values(w1, e)[:, :cols], values(w2, e)[:, :hidden]
        xe, w = x[token].double(), weights[token, choice].double()[:, None]
        h, off = xe @ v1.t(), (xe.abs() @ v1.abs().t()) * 2.0 ** -23 * (cols / 8 + 8)
        gate, up = h[:, :hidden], h[:, hidden:] if gated else torch.ones_like(h)
        act = gate * torch.sigmoid(gate) * up
        off_act = 1.1 * off[:, :hidden] * up.abs() + 2.0 ** -20 * act.abs()
        if gated:
            off_act = off_act + (gate * torch.sigmoid(gate)).abs() * off[:, hidden:] + 1.1 * off[:, :hidden] * off[:, hidden:]
        off_act = off_act * (1 + 2.0 ** -16) + act.abs() * 2.0 ** -16
        mag = (act.abs() + off_act) @ v2.abs().t()
        want.index_add_(0, token, w * (act @ v2.t()))
        bound.index_add_(0, token, w.abs() * (off_act @ v2.abs().t() + mag * 2.0 ** -23 * (hidden / 8 + 16 + ids.shape[1])))
    allowed = bound + 2.0 ** -8 * (want.abs() + bound) + 2.0 ** -126
    miss = (out.double() - want).abs()
    assert bool((miss <= allowed).all()), (what, int((~(miss <= allowed)).sum()), float((miss - allowed).max()))
    norm = float(want.norm())
    assert norm == 0 or float((out.double() - want).norm()) <= 4e-3 * norm, what  # out's rounding to BF16: 2^-8 of an element at most


CASES = [(1, 1, 1, 128, 128), (1, 8, 64, 1024, 512), (1, 2, 4, 1, 1), (2, 3, 7, 130, 200), (5, 2, 8, 64, 96), (16, 4, 32, 1280, 640), (17, 8, 8, 333, 129),
         (33, 2, 3, 515, 1000), (64, 8, 64, 1024, 512), (70, 1, 1, 256, 384), (128, 8, 16, 520, 136), (200, 5, 6, 136, 264), (1024, 1, 256, 128, 64),
         (1, 1, 256, 4100, 2050), (4, 256, 256, 96, 40)]


@pytest.mark.parametrize("tokens,topk,experts,cols,hidden", CASES)
@pytest.mark.parametrize("kind", ["mxfp4", "fp8"])
@pytest.mark.parametrize("gated", [True, False])
def test_layer(tokens, topk, experts, cols, hidden, kind, gated):
    g = gen(tokens + cols)
    x = torch.randn((tokens, cols), device=DEV, generator=g).bfloat16()
    ids = torch.stack([torch.randperm(experts, device=DEV, generator=g)[:topk] for _ in range(tokens)]).to(torch.int32)
    weights = torch.softmax(torch.randn((tokens, topk), device=DEV, generator=g), 1)
    w1, w2 = layer(kind, experts, cols, hidden, gated, hidden)
    out = nv.expert_mlp(x, ids, weights, w1, w2, gated=gated)
    check(out, x, ids, weights, w1, w2, gated)
    assert torch.equal(nv.expert_mlp(x, ids.long(), weights, w1, w2, gated=gated), out)


@pytest.mark.parametrize("kind", ["mxfp4", "fp8"])
def test_dropped_and_repeated_choices(kind):
    g = gen(5)
    x = torch.randn((40, 260), device=DEV, generator=g).bfloat16()
    ids = torch.randint(-3, 9, (40, 6), device=DEV, generator=g)  # 0 .. 5 are experts; a token may name one twice
    ids[3] = -1
    ids[4] = 6
    ids[5] = 2
    ids[6, 0], ids[7, 0] = 1 << 32, -(1 << 40)
    weights = torch.randn((40, 6), device=DEV, generator=g)
    w1, w2 = layer(kind, 6, 260, 300, True, 6)
    out = nv.expert_mlp(x, ids, weights, w1, w2)
    check(out, x, ids, weights, w1, w2, True)
    assert not bool(out[3:5].any())
    none = torch.full_like(ids, -1)
    assert not bool(nv.expert_mlp(x, none, weights, w1, w2).any())
    # a dropped choice's weight does not count, whatever it is
    weights[ids >= 6] = float("nan")
    weights[ids < 0] = float("inf")
    assert torch.equal(nv.expert_mlp(x, ids, weights, w1, w2), out)


def test_no_tokens():
    w1, w2 = layer("mxfp4", 3, 64, 32, True, 7)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    assert nv.expert_mlp(x, torch.empty((0, 2), dtype=torch.int32, device=DEV), torch.empty((0, 2), device=DEV), w1, w2).shape == (0, 64)


def test_experts_that_no_token_chose_are_not_read():
    w1, w2 = layer("mxfp4", 4, 256, 128, True, 8)
    x = torch.randn((3, 256), device=DEV, generator=gen(9)).bfloat16()
    ids = torch.tensor([[0, 2], [2, 0], [0, -1]], dtype=torch.int32, device=DEV)
    weights = torch.rand((3, 2), device=DEV, generator=gen(10))
    want = nv.expert_mlp(x, ids, weights, w1, w2)
    for q in (w1, w2):
        q.scales[1], q.scales[3] = 255, 255
    assert torch.equal(nv.expert_mlp(x, ids, weights, w1, w2), want)


def test_a_token_with_nan_stays_alone():
    w1, w2 = layer("mxfp4", 4, 256, 128, True, 11)
    x = torch.randn((20, 256), device=DEV, generator=gen(12)).bfloat16()
    ids = torch.randint(0, 4, (20, 2), device=DEV, generator=gen(13))
    weights = torch.rand((20, 2), device=DEV, generator=gen(14))
    want = nv.expert_mlp(x, ids, weights, w1, w2)
    x[7, 100] = float("nan")
    out = nv.expert_mlp(x, ids, weights, w1, w2)
    assert bool(torch.isnan(out[7]).all())
    keep = torch.arange(20, device=DEV) != 7
    assert torch.equal(out[keep], want[keep])


def test_every_scale_of_the_weights():
    # w2 as a table: expert 0's row c has one value under scale c
    x = torch.zeros((1, 256), dtype=torch.bfloat16, device=DEV)
    x[0, 0] = 8
    w1 = nv.mxfp4_quantize(torch.eye(32, 256, device=DEV)[None] * 4)[0]
    h = torch.nn.functional.silu(torch.tensor(32.0, dtype=torch.float64)).bfloat16().double().item()
    data = torch.zeros((1, 256, 64), dtype=torch.uint8, device=DEV)
    data[0, :, 0] = 3  # 1.5
    scales = torch.zeros((1, 1, 256, 4), dtype=torch.uint8, device=DEV)
    scales[0, 0, :, 0] = torch.arange(256, device=DEV).to(torch.uint8)
    out = nv.expert_mlp(x, torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones((1, 1), device=DEV), w1,
                        nv.Mxfp4Tensor(data, scales, 256, 32), gated=False)[0]
    want = (h * 1.5 * torch.exp2(torch.arange(256, dtype=torch.float64, device=DEV) - 127)).float().bfloat16()
    assert bool(torch.isnan(out[255])) and torch.equal(out[:255], want[:255])


def test_captured_and_replayed_and_two_at_once():
    tokens, topk, experts, cols, hidden = 24, 4, 16, 512, 256
    w1, w2 = layer("mxfp4", experts, cols, hidden, True, 15)
    g = gen(16)

    def inputs():
        return (torch.randn((tokens, cols), device=DEV, generator=g).bfloat16(), torch.randint(-1, experts, (tokens, topk), device=DEV, generator=g),
                torch.rand((tokens, topk), device=DEV, generator=g))

    static = inputs()
    nv.expert_mlp(*static, w1, w2)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(nv.expert_mlp(*static, w1, w2))
    for i in range(4):
        for s, v in zip(static, inputs()):
            s.copy_(v)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        want = nv.expert_mlp(*static, w1, w2)
        assert all(torch.equal(o, want) for o in outs), i
    one, two = inputs(), inputs()
    want = nv.expert_mlp(*one, w1, w2), nv.expert_mlp(*two, w1, w2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a = nv.expert_mlp(*one, w1, w2)
        b = nv.expert_mlp(*two, w1, w2, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_refusals():
    w1, w2 = layer("mxfp4", 4, 128, 64, True, 17)
    f1, f2 = layer("fp8", 4, 128, 64, True, 17)
    x = torch.zeros((2, 128), dtype=torch.bfloat16, device=DEV)
    ids, weights = torch.zeros((2, 2), dtype=torch.int32, device=DEV), torch.ones((2, 2), device=DEV)
    for args, kw, match in [((x.float(), ids, weights, w1, w2), {}, "bfloat16"), ((x, ids.float(), weights, w1, w2), {}, "ids"),
                            ((x, ids[:1], weights, w1, w2), {}, "ids"), ((x, ids, weights.double(), w1, w2), {}, "weights"),
                            ((x, ids, weights[:, :1], w1, w2), {}, "weights"), ((x, ids, weights, w1, f2), {}, "one format"),
                            ((x, ids, weights, f1, w2), {}, "one format"), ((x, ids, weights, w2, w1), {}, "w1"), ((x, ids, weights, w1, w2), {"gated": False}, "w1"),
                            ((x[:, :64].contiguous(), ids, weights, w1, w2), {}, "w1"), ((x.t().contiguous().t(), ids, weights, w1, w2), {}, "contiguous"),
                            ((x, ids, weights, nv.fp8_quantize(torch.zeros((4, 128, 128), device=DEV))[0], f2), {}, "w1")]:
        with pytest.raises(ValueError, match=match):
            nv.expert_mlp(*args, **kw)
    many = torch.zeros((600, 128), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(nv.NVFP4Error, match="at most 1024"):
        nv.expert_mlp(many, torch.zeros((600, 2), dtype=torch.int32, device=DEV), torch.zeros((600, 2), device=DEV), w1, w2)
