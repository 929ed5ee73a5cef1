"""The expert-layer operators as they are timed: sorting tokens by expert and
back, block-scaled FP8 quantization, and the FP8 matrix products, dense and by
expert, each with its plain form in elementary torch operations.

With ``own`` false, run() computes the plain form (32-bit arithmetic, one
rounding at the end); with ``own`` true it calls the package. exact() is the
definition in 64 bits, written apart from both.

Formats. An FP8 operand is [n][pitch(k)] E4M3 bytes, pitch(k) = k rounded up
to 128 with zero codes in the padding, and float32 decode scales
[ceil(k / 128)][n] (1x128 blocks) or [ceil(k / 128)][ceil(n / 128)] (128x128
blocks), with a leading batch dimension where there is one. A plan has, for
ids [T][k], slot_rows [T][k] (the row of the sorted matrix that a token's
choice went to, -1 if dropped), row_slots [R] (its inverse, -1 for padding),
offsets [E + 1] (each expert's first row, a multiple of `align`) and counts [E].
"""

import math

import torch

own = False

E4M3_MAX = 448.0
FLT_MAX = 3.4028234663852886e38
BLOCK = 128


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # one decoding step of 64 sequences: the latency of routing
        dict(name="route_decode", op="route", tokens=64, topk=8, experts=64, cols=4096, align=16, dtype="bf16", drop=0.0),
        # a long prompt or a training batch, forward
        dict(name="route_prompt", op="route", tokens=8192, topk=8, experts=64, cols=4096, align=128, dtype="bf16", drop=0.0),
        # the same on the way back, with tokens dropped by a capacity limit
        dict(name="route_gradient", op="route_grad", tokens=8192, topk=4, experts=32, cols=5120, align=128, dtype="bf16", drop=0.02),
        # a decoding step's activations before a product
        dict(name="quantize_decode", op="quantize", batch=1, rows=16, cols=5120, dtype="bf16", block_2d=False, rowwise=True, colwise=False),
        # tokens gathered by expert and quantized for the product and for the weight gradient, in one call
        dict(name="quantize_sorted", op="quantize_sorted", tokens=8192, topk=4, experts=32, cols=5120, align=128, dtype="bf16", drop=0.0, colwise=True),
        # the experts' weights after an optimizer step, both orientations
        dict(name="quantize_weights", op="quantize", batch=32, rows=2048, cols=4096, dtype="bf16", block_2d=True, rowwise=True, colwise=True),
        # a decoding step's dense product: bound by reading the weights
        dict(name="matmul_decode", op="matmul", m=16, n=8192, k=5120, b_block_2d=True, out="bf16"),
        # no size a multiple of anything; both operands in 1x128 blocks, as in a weight gradient
        dict(name="matmul_odd", op="matmul", m=777, n=1361, k=1999, b_block_2d=False, out="fp32"),
        # a training batch's dense product
        dict(name="matmul_prompt", op="matmul", m=8192, n=8192, k=5120, b_block_2d=True, out="bf16"),
        # experts' product for one decoding step
        dict(name="experts_decode", op="experts", tokens=64, topk=8, experts=64, align=16, n=4096, k=2048, out="bf16"),
        # experts' product for a prompt or a training batch
        dict(name="experts_prompt", op="experts", tokens=8192, topk=8, experts=64, align=128, n=4096, k=2048, out="bf16"),
        # experts' weight gradients
        dict(name="experts_weight_grad", op="experts_grad", tokens=8192, topk=4, experts=32, align=128, n=4096, k=2048, out="fp32"),
    ]


def _spread(rng, low, high, odd=0.4):
    """A size over [low, high], even over its logarithm; sometimes rounded to a multiple of 128, 16 or 8."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() > odd:
        step = rng.choice([128, 16, 8])
        v = max(step, v // step * step)
    return max(low, min(high, v))


def _draw(rng):
    op = rng.choice(["route", "route_grad", "quantize", "quantize_sorted", "matmul", "matmul", "experts", "experts_grad"])
    dtype = "fp32" if rng.random() < 0.25 else "bf16"
    experts = rng.choice([4, 7, 8, 16, 32, 60, 64, 128, 256])
    topk = min(experts, rng.randint(1, 8))
    drop = rng.choice([0.0, 0.0, 0.02, 0.3])
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("route", "route_grad"):
        return dict(op=op, tokens=_spread(rng, 1, 8192), topk=topk, experts=experts, cols=_spread(rng, 64, 8192),
                    align=rng.choice([1, 16, 128]), dtype=dtype, drop=drop)
    if op == "quantize":
        rowwise = rng.random() < 0.8
        return dict(op=op, batch=rng.choice([1, 1, 1, 3, 16]), rows=_spread(rng, 1, 8192), cols=_spread(rng, 64, 8192), dtype=dtype,
                    block_2d=rng.random() < 0.4, rowwise=rowwise, colwise=not rowwise or rng.random() < 0.5)
    if op == "quantize_sorted":
        return dict(op=op, tokens=_spread(rng, 1, 8192), topk=topk, experts=experts, cols=_spread(rng, 64, 8192), align=128,
                    dtype=dtype, drop=drop, colwise=rng.random() < 0.5)
    if op == "matmul":
        return dict(op=op, m=_spread(rng, 1, 8192), n=_spread(rng, 64, 8192), k=_spread(rng, 64, 8192), b_block_2d=rng.random() < 0.6, out=out)
    experts = min(experts, 64)
    return dict(op=op, tokens=_spread(rng, 1, 8192), topk=min(topk, experts), experts=experts, align=128 if op == "experts_grad" else rng.choice([1, 16, 128]),
                n=_spread(rng, 128, 4096), k=_spread(rng, 128, 4096), out=out)


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        for key in ("bytes", "flops"):
            most[c["op"], key] = max(most.get((c["op"], key), 0), w[key])
    while True:
        c = _draw(rng)
        w = work(c)
        if all(w[key] <= most[c["op"], key] for key in ("bytes", "flops")):
            return c


# ---- inputs -----------------------------------------------------------------

def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _cdiv(a, b):
    return -(-a // b)


def _capacity(tokens, topk, experts, align):
    """Rows that the sorted matrix needs at most, whatever the ids are."""
    slots = tokens * topk
    return (slots + min(experts, slots) * (align - 1)) // align * align


def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, shape, dtype):
    """Normal values with a factor per column, as activations have them, and a row of zeros here and there."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(torch.randn(shape[-1], generator=g, device="cuda"))
    x *= (torch.rand(shape[:-1], generator=g, device="cuda") > 0.01).float().unsqueeze(-1)
    return x.to(dtype)


def _ids(g, c):
    """Distinct experts for each token, some experts more wanted than others; dropped choices are -1."""
    t, e = c["tokens"], c["experts"]
    score = torch.randn((t, e), generator=g, device="cuda") + 0.5 * torch.randn((e,), generator=g, device="cuda")
    score, ids = score.topk(c["topk"], dim=1)
    dropped = torch.rand((t, c["topk"]), generator=g, device="cuda") < c.get("drop", 0.0)
    return torch.where(dropped, -1, ids).to(torch.int32), torch.softmax(score, 1)


def prepare(case, seed):
    c, g = dict(case), _rng(seed)
    op = c["op"]
    s = {"case": c}
    if op in ("route", "route_grad", "quantize_sorted", "experts", "experts_grad"):
        s["ids"], s["weights"] = _ids(g, c)
        s["capacity"] = _capacity(c["tokens"], c["topk"], c["experts"], c["align"])
        plan = _plain_sort(s["ids"], c["experts"], c["align"], s["capacity"])
        if op != "route":
            s["plan"] = plan
    if op == "route":
        s["x"] = _activations(g, (c["tokens"], c["cols"]), _dtype(c["dtype"]))
        s["y"] = torch.randn((s["capacity"], c["cols"]), generator=g, device="cuda").to(_dtype(c["dtype"]))
    elif op == "route_grad":
        dt = _dtype(c["dtype"])
        s["dout"] = torch.randn((c["tokens"], c["cols"]), generator=g, device="cuda").to(dt)
        s["y"] = torch.randn((s["capacity"], c["cols"]), generator=g, device="cuda").to(dt)
        s["dx_sorted"] = torch.randn((s["capacity"], c["cols"]), generator=g, device="cuda").to(dt)
    elif op == "quantize":
        s["x"] = _activations(g, (c["batch"], c["rows"], c["cols"]), _dtype(c["dtype"]))
    elif op == "quantize_sorted":
        s["x"] = _activations(g, (c["tokens"], c["cols"]), _dtype(c["dtype"]))
    elif op == "matmul":
        a = _activations(g, (1, c["m"], c["k"]), torch.float32)
        b = torch.randn((1, c["n"], c["k"]), generator=g, device="cuda")
        s["a"] = tuple(v[0] for v in _plain_quantize(a, False))
        s["b"] = tuple(v[0] for v in _plain_quantize(b, c["b_block_2d"]))
    elif op == "experts":
        x = _activations(g, (c["tokens"], c["k"]), torch.float32)
        s["a"] = tuple(v[0] for v in _plain_quantize(_plain_gather(x, plan, c["topk"])[None], False))
        s["b"] = _plain_quantize(torch.randn((c["experts"], c["n"], c["k"]), generator=g, device="cuda"), True)
    elif op == "experts_grad":
        x = _activations(g, (c["tokens"], c["k"]), torch.float32)
        dy = torch.randn((c["tokens"], c["n"]), generator=g, device="cuda")
        s["a"], s["b"] = (tuple(u[0] for u in _plain_quantize(_plain_gather(v, plan, c["topk"]).t()[None], False)) for v in (dy, x))
    if op in ("experts", "experts_grad"):
        s["longest"] = int((plan["offsets"][1:] - plan["offsets"][:-1]).max())  # rows of the largest expert, known to the plain form's user
    return s


# ---- the plain forms --------------------------------------------------------

def _plain_sort(ids, experts, align, capacity):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    ordered, order = torch.sort(key, stable=True)
    starts = torch.searchsorted(ordered, torch.arange(experts + 1, device=ids.device))
    counts = starts[1:] - starts[:-1]
    ends = torch.cumsum(_cdiv(counts, align) * align, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    place = offsets[ordered] + torch.arange(flat.numel(), device=ids.device) - starts[ordered]
    kept = ordered < experts
    slot_rows = torch.empty_like(flat)
    slot_rows[order] = torch.where(kept, place, -1)
    row_slots = flat.new_full((capacity + 1,), -1)
    row_slots[torch.where(kept, place, capacity)] = order
    i32 = torch.int32
    return {"slot_rows": slot_rows.reshape(ids.shape).to(i32), "row_slots": row_slots[:capacity].to(i32), "offsets": offsets.to(i32), "counts": counts.to(i32)}


def _plain_gather(x, plan, topk):
    slots = plan["row_slots"].long()
    return torch.where((slots >= 0)[:, None], x[slots.clamp(min=0) // topk], x.new_zeros(()))


def _plain_combine(y, plan, weights):
    rows = plan["slot_rows"].long()
    v = torch.where((rows >= 0)[..., None], y[rows.clamp(min=0)].float(), 0.0)
    if weights is not None:
        v = v * weights[..., None]
    return v.sum(1).to(y.dtype)


def _plain_combine_grad(dout, y, plan, weights):
    slots, rows, topk = plan["row_slots"].long(), plan["slot_rows"].long(), weights.shape[1]
    at = slots.clamp(min=0)
    dy = dout[at // topk].float() * weights.reshape(-1)[at][:, None]
    dy = torch.where((slots >= 0)[:, None], dy, 0.0).to(dout.dtype)
    dw = (dout.float()[:, None] * y[rows.clamp(min=0)].float()).sum(-1)
    return dy, torch.where(rows >= 0, dw, 0.0)


def _plain_quantize(x, block_2d):
    """x [B][R][C] -> E4M3 codes [B][R][pitch(C)] and scales [B][ceil(C / 128)][R or ceil(R / 128)]."""
    b, r, c = x.shape
    kb, rb = _cdiv(c, BLOCK), _cdiv(r, BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - c, 0, (rb * BLOCK - r) if block_2d else 0))
    v = v.reshape(b, rb, BLOCK, kb, BLOCK) if block_2d else v.reshape(b, r, 1, kb, BLOCK)
    scale = v.abs().amax((2, 4), keepdim=True)
    scale = scale / scale.new_full((), E4M3_MAX)  # a true division: by a Python number torch multiplies by its reciprocal
    mult = torch.where(scale > 0, (1.0 / scale).clamp(max=FLT_MAX), 0.0)
    q = (v * mult).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.reshape(b, -1, kb * BLOCK)[:, :r].contiguous(), scale[:, :, 0, :, 0].transpose(1, 2).contiguous()


def _plain_values(q, block_2d):
    """The 32-bit values [..][n][pitch] of an FP8 operand."""
    data, scales = q
    s = scales.transpose(-1, -2)  # [..][n or n / 128][k / 128]
    if block_2d:
        s = s.repeat_interleave(BLOCK, -2)[..., :data.shape[-2], :]
    return data.float() * s.repeat_interleave(BLOCK, -1)


def _plain_experts(a, b, offsets, longest, out):
    a, b = _plain_values(a, False), _plain_values(b, True)
    rows = a.shape[0]
    at = offsets[:-1, None].long() + torch.arange(longest, device=a.device)
    inside = at < offsets[1:, None]
    d = torch.bmm(a[at.clamp(max=rows - 1)], b.transpose(1, 2)).to(out)
    result = d.new_zeros((rows + 1, d.shape[2]))
    result[torch.where(inside, at, rows)] = d
    return result[:rows]


def _plain_experts_grad(a, b, offsets, longest, out):
    a, b = _plain_values(a, False), _plain_values(b, False)
    at = offsets[:-1, None].long() + torch.arange(longest, device=a.device)
    inside = (at < offsets[1:, None])[..., None]
    at = at.clamp(max=a.shape[1] - 1)
    a = torch.where(inside, a.t()[at], 0.0)  # [E][longest][m]
    return torch.bmm(a.transpose(1, 2), b.t()[at]).to(out)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        plan = _plain_sort(s["ids"], c["experts"], c["align"], s["capacity"])
        return {**plan, "x_sorted": _plain_gather(s["x"], plan, c["topk"]), "out": _plain_combine(s["y"], plan, s["weights"])}
    if op == "route_grad":
        dy, dw = _plain_combine_grad(s["dout"], s["y"], s["plan"], s["weights"])
        return {"dy": dy, "dweights": dw, "dx": _plain_combine(s["dx_sorted"], s["plan"], None)}
    if op in ("quantize", "quantize_sorted"):
        x = s["x"] if op == "quantize" else _plain_gather(s["x"], s["plan"], c["topk"])[None]
        block_2d = c.get("block_2d", False)
        out = {}
        if c.get("rowwise", True):
            out["row_data"], out["row_scales"] = _plain_quantize(x, block_2d)
        if c["colwise"]:
            out["col_data"], out["col_scales"] = _plain_quantize(x.transpose(1, 2), block_2d)
        return out
    if op == "matmul":
        return _plain_values(s["a"], False).matmul(_plain_values(s["b"], c["b_block_2d"]).t()).to(_dtype(c["out"]))
    f = _plain_experts if op == "experts" else _plain_experts_grad
    return f(s["a"], s["b"], s["plan"]["offsets"], s["longest"], _dtype(c["out"]))


# ---- the package's calls ----------------------------------------------------

def _run_own(s):
    import nvfp4_block_scaled_05_amd as nv

    c = s["case"]
    op = c["op"]

    def fp8(q, k, block_2d=False):
        return nv.Fp8Tensor(q[0], q[1], q[0].shape[-2], k, block_2d)

    def plan():
        return nv.ExpertPlan(**s["plan"], align=c["align"])

    if op == "route":
        p = nv.expert_sort(s["ids"], c["experts"], align=c["align"])
        return {"slot_rows": p.slot_rows, "row_slots": p.row_slots, "offsets": p.offsets, "counts": p.counts,
                "x_sorted": nv.expert_gather(s["x"], p), "out": nv.expert_combine(s["y"], p, s["weights"])}
    if op == "route_grad":
        p = plan()
        dy, dw = nv.expert_combine_grad(s["dout"], s["y"], p, s["weights"])
        return {"dy": dy, "dweights": dw, "dx": nv.expert_gather_grad(s["dx_sorted"], p)}
    if op in ("quantize", "quantize_sorted"):
        row, col = nv.fp8_quantize(s["x"], rowwise=c.get("rowwise", True), columnwise=c["colwise"], block_2d=c.get("block_2d", False),
                                   plan=plan() if op == "quantize_sorted" else None)
        lead = (lambda t: t) if op == "quantize" else (lambda t: t[None])
        out = {}
        if row is not None:
            out["row_data"], out["row_scales"] = lead(row.data), lead(row.scales)
        if col is not None:
            out["col_data"], out["col_scales"] = lead(col.data), lead(col.scales)
        return out
    if op == "matmul":
        return nv.fp8_matmul(fp8(s["a"], c["k"]), fp8(s["b"], c["k"], c["b_block_2d"]), out_dtype=_dtype(c["out"]))
    if op == "experts":
        return nv.fp8_matmul_grouped(fp8(s["a"], c["k"]), fp8(s["b"], c["k"], True), plan(), out_dtype=_dtype(c["out"]))
    return nv.fp8_matmul_grouped_k(fp8(s["a"], s["capacity"]), fp8(s["b"], s["capacity"]), plan(), out_dtype=_dtype(c["out"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    c = dict(case)
    op = c["op"]
    size = {"bf16": 2, "fp32": 4}
    if op in ("matmul",):
        m, n, k = c["m"], c["n"], c["k"]
        kb = _cdiv(k, BLOCK)
        b_scales = _cdiv(n, BLOCK) if c["b_block_2d"] else n
        return {"bytes": (m + n) * k + 4 * kb * (m + b_scales) + size[c["out"]] * m * n, "flops": 2 * m * n * k}
    if op == "quantize":
        n = c["batch"] * c["rows"] * c["cols"]
        sides = int(c["rowwise"]) + int(c["colwise"])
        return {"bytes": n * (size[c["dtype"]] + sides * (1 + (4 / BLOCK ** 2 if c["block_2d"] else 4 / BLOCK))), "flops": 3 * n}
    slots = c["tokens"] * c["topk"]
    used = min(c["experts"], slots)
    kept = slots * (1 - c.get("drop", 0.0))
    capacity = _capacity(c["tokens"], c["topk"], c["experts"], c["align"])
    maps = 4 * (slots + capacity + 2 * c["experts"])
    if op == "route":
        b = size[c["dtype"]]
        return {"bytes": maps + 8 * slots + b * c["cols"] * (2 * c["tokens"] + capacity + kept), "flops": 2 * kept * c["cols"]}
    if op == "route_grad":
        b = size[c["dtype"]]
        return {"bytes": maps + 8 * slots + b * c["cols"] * (2 * c["tokens"] + capacity + 2 * kept), "flops": 4 * kept * c["cols"]}
    if op == "quantize_sorted":
        sides = 1 + int(c["colwise"])
        return {"bytes": 4 * capacity + size[c["dtype"]] * c["tokens"] * c["cols"] + sides * capacity * c["cols"] * (1 + 4 / BLOCK), "flops": 3 * kept * c["cols"]}
    n, k = c["n"], c["k"]
    if op == "experts":
        return {"bytes": slots * (k + 4 * _cdiv(k, BLOCK)) + used * n * k + size[c["out"]] * capacity * n, "flops": 2 * slots * n * k}
    return {"bytes": slots * (n + k) * (1 + 4 / BLOCK) + size[c["out"]] * c["experts"] * n * k, "flops": 2 * slots * n * k}


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_e4m3(v):
    """The nearest E4M3 value (bias 7, three mantissa bits, least step 2^-9), ties to even."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_quantize(x, block_2d):
    """By blocks along the last axis of x [B][R][C] in 64 bits."""
    b, r, c = x.shape
    high = BLOCK if block_2d else 1
    rows, cols = _cdiv(r, high) * high, _cdiv(c, BLOCK) * BLOCK
    v = x.new_zeros((b, rows, cols), dtype=torch.float64)
    v[:, :r, :c] = x.double()
    blocks = v.unfold(1, high, high).unfold(2, BLOCK, BLOCK)  # [B][R / high][C / 128][high][128]
    scale = blocks.abs().amax((3, 4)) / E4M3_MAX
    per_row = scale.repeat_interleave(high, 1).repeat_interleave(BLOCK, 2)
    q = _exact_e4m3(torch.where(per_row > 0, v / per_row, 0.0))
    return q[:, :r], scale.transpose(1, 2).contiguous()


def _exact_operand(q, n_per_scale):
    """[n][k] in 64 bits, block by block."""
    data, scales = q
    v = data.to(torch.float32).double()
    for j in range(scales.shape[-2]):
        s = scales[..., j, :].double()
        at = torch.arange(data.shape[-2], device=data.device) // n_per_scale
        v[..., j * BLOCK:(j + 1) * BLOCK] *= s[..., at].unsqueeze(-1)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op == "matmul":
        return _exact_operand(s["a"], 1) @ _exact_operand(s["b"], BLOCK if c["b_block_2d"] else 1).t()
    if op in ("quantize", "quantize_sorted"):
        x = s["x"]
        if op == "quantize_sorted":
            rows = x.new_zeros((s["capacity"], c["cols"]))
            used = (s["plan"]["row_slots"] >= 0).nonzero()[:, 0]
            rows[used] = x[torch.div(s["plan"]["row_slots"][used].long(), c["topk"], rounding_mode="floor")]
            x = rows[None]
        block_2d, out = c.get("block_2d", False), {}
        if c.get("rowwise", True):
            out["row_data"], out["row_scales"] = _exact_quantize(x, block_2d)
        if c["colwise"]:
            out["col_data"], out["col_scales"] = _exact_quantize(x.transpose(1, 2), block_2d)
        return out
    if op in ("experts", "experts_grad"):
        starts = s["plan"]["offsets"].tolist()
        a = _exact_operand(s["a"], 1)
        if op == "experts":
            d = a.new_zeros((s["capacity"], c["n"]))
            for e in range(c["experts"]):
                w = _exact_operand((s["b"][0][e], s["b"][1][e]), BLOCK)
                d[starts[e]:starts[e + 1]] = a[starts[e]:starts[e + 1]] @ w.t()
            return d
        b = _exact_operand(s["b"], 1)
        return torch.stack([a[:, starts[e]:starts[e + 1]] @ b[:, starts[e]:starts[e + 1]].t() for e in range(c["experts"])])
    # routing: by token, choice after choice
    plan = s.get("plan") or _plain_sort(s["ids"], c["experts"], c["align"], s["capacity"])
    rows = plan["slot_rows"].long()
    total = torch.zeros((c["tokens"], c["cols"]), dtype=torch.float64, device="cuda")
    if op == "route":
        x_sorted = torch.zeros((s["capacity"], c["cols"]), dtype=torch.float64, device="cuda")
        for j in range(c["topk"]):
            kept = (rows[:, j] >= 0).nonzero()[:, 0]
            total[kept] += s["weights"][kept, j].double()[:, None] * s["y"][rows[kept, j]].double()
            x_sorted[rows[kept, j]] = s["x"][kept].double()
        return {"slot_rows": None, "row_slots": None, "offsets": None, "counts": None, "x_sorted": x_sorted, "out": total}
    dy = torch.zeros((s["capacity"], c["cols"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((c["tokens"], c["topk"]), dtype=torch.float64, device="cuda")
    for j in range(c["topk"]):
        kept = (rows[:, j] >= 0).nonzero()[:, 0]
        at, d = rows[kept, j], s["dout"][kept].double()
        dy[at] = s["weights"][kept, j].double()[:, None] * d
        dw[kept, j] = (d * s["y"][at].double()).sum(-1)
        total[kept] += s["dx_sorted"][at].double()
    return {"dy": dy, "dweights": dw, "dx": total}
