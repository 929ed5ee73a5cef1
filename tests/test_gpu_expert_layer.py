"""GPU: the example expert layer against the same layer in 64 bits, and the
refusals of the expert-layer bindings that need device tensors."""

from __future__ import annotations

import os
import sys

import pytest
import torch

import nvfp4_block_scaled_05_amd as nv
from gpu_helpers import DEV

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer as layer  # noqa: E402

pytestmark = pytest.mark.gpu

# An E4M3 code is off by at most 2^-4 of its value, evenly spread: 2^-4 / sqrt(3) = 0.036 in the mean
# square, 0.051 for a product of two such operands. No result passes through more than three products.
OFF = 3 * 0.051


def exact(x, ids, weights, w1, w2):
    """The layer in binary64, expert by expert, on leaves that autograd follows."""
    leaves = [t.double().requires_grad_() for t in (x, weights, w1, w2)]
    x, weights, w1, w2 = leaves
    out = torch.zeros_like(x)
    for e in range(w1.shape[0]):
        t, j = (ids == e).nonzero(as_tuple=True)
        y = torch.nn.functional.silu(x[t] @ w1[e].t()) @ w2[e].t()
        out = out.index_add(0, t, y * weights[t, j][:, None])
    return out, leaves


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("tokens,topk,experts,c,f", [(300, 3, 5, 256, 384), (70, 2, 16, 200, 136)])
def test_training_step(tokens, topk, experts, c, f):
    x, ids, weights, w1, w2 = layer.make(tokens, topk, experts, c, f, seed=tokens)
    out, saved = layer.forward(x, ids, weights, q1 := layer.Weights.quantize(w1), q2 := layer.Weights.quantize(w2), train=True)
    dout = torch.randn(out.shape, device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(out.dtype)
    grads = layer.backward(dout, weights, q1, q2, saved)
    want, leaves = exact(x, ids, weights, w1, w2)
    want.backward(dout.double())
    assert rel(out, want.detach()) < OFF
    for got, leaf, name in zip(grads, leaves, ("x", "weights", "w1", "w2")):
        assert got.shape == leaf.shape and rel(got, leaf.grad) < OFF, name


@pytest.mark.parametrize("tokens", [1, 16])
def test_decoding_step(tokens):
    x, ids, weights, w1, w2 = layer.make(tokens, 2, 8, 512, 256, seed=tokens)
    out, _ = layer.forward(x, ids, weights, layer.Weights.quantize(w1), layer.Weights.quantize(w2), train=False)
    assert rel(out, exact(x, ids, weights, w1, w2)[0]) < OFF


def test_bindings_refuse_what_does_not_fit():
    ids = torch.zeros((4, 2), dtype=torch.int32, device=DEV)
    plan = nv.expert_sort(ids, 3, align=16)
    x = torch.zeros((4, 64), device=DEV)
    y = torch.zeros((plan.rows, 64), device=DEV)
    w = torch.zeros((4, 2), device=DEV)
    a, _ = nv.fp8_quantize(y)
    b, _ = nv.fp8_quantize(torch.zeros((3, 32, 64), device=DEV), block_2d=True)
    one = nv.Fp8Tensor(b.data[0], b.scales[0], 32, 64, True)
    bad = [
        lambda: nv.expert_sort(ids.float(), 3), lambda: nv.expert_sort(ids[0], 3), lambda: nv.expert_sort(ids[:, :1], 3),
        lambda: nv.expert_gather(x[:3], plan), lambda: nv.expert_gather(x[:, ::2], plan), lambda: nv.expert_gather(x[0], plan),
        lambda: nv.expert_combine(y[1:], plan, w), lambda: nv.expert_combine(y, plan, w[:3]), lambda: nv.expert_combine(y, plan, w.double()),
        lambda: nv.expert_combine_grad(x, y.bfloat16(), plan, w), lambda: nv.expert_combine_grad(x, y, plan, w.t()),
        lambda: nv.fp8_quantize(x[:, ::2]), lambda: nv.fp8_quantize(x[0]), lambda: nv.fp8_quantize(x[:3], plan=plan),
        lambda: nv.fp8_quantize(x[None], plan=plan),
        lambda: nv.fp8_matmul(one, one), lambda: nv.fp8_matmul(a, nv.Fp8Tensor(one.data, one.scales, 32, 63, True)),
        lambda: nv.fp8_matmul(a, nv.Fp8Tensor(one.data, one.scales, 32, 64, False)), lambda: nv.fp8_matmul(a, b),
        lambda: nv.fp8_matmul(nv.Fp8Tensor(a.data[1:], a.scales, a.n, 64), one),
        lambda: nv.fp8_matmul_grouped(a, one, plan), lambda: nv.fp8_matmul_grouped(one, b, plan),
        lambda: nv.fp8_matmul_grouped_k(a, a, plan),  # not aligned to 128
        lambda: nv.expert_gather(x, nv.ExpertPlan(plan.slot_rows.long(), plan.row_slots, plan.offsets, plan.counts, 16)),
        lambda: nv.expert_gather(x, nv.ExpertPlan(plan.slot_rows, plan.row_slots, plan.counts, plan.counts, 16)),
        lambda: nv.expert_gather(x, nv.ExpertPlan(plan.slot_rows, plan.row_slots.cpu(), plan.offsets, plan.counts, 16)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(TypeError):
        nv.expert_gather(x.half(), plan)
    with pytest.raises(TypeError):
        nv.fp8_matmul(a, one, out_dtype=torch.float16)
    for kw, status in ((dict(align=24), nv.NVFP4_ERR_UNSUPPORTED), (dict(rows=5), nv.NVFP4_ERR_SHAPE)):
        with pytest.raises(nv.NVFP4Error) as e:
            nv.expert_sort(ids, 3, **kw)
        assert e.value.status == status
    with pytest.raises(nv.NVFP4Error):
        nv.expert_sort(ids, 257)
