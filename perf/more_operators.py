"""The MXFP4 operators as they are timed: quantization and reading back, the
products, dense and by expert, and the expert layer for a few tokens, each with
its plain form in elementary torch operations.

With ``own`` false, run() computes the plain form (32-bit arithmetic, one
rounding at the end); with ``own`` true it calls the package. exact() is the
definition in 64 bits, written apart from both.

Formats. An MXFP4 operand is [n][pitch(k) / 2] bytes of two E2M1 codes each (the
even element in the low half), pitch(k) = k rounded up to 128 with zero codes in
the padding, and E8M0 scales [ceil(k / 128)][n][4], one byte for each 32 values
of a row, with a leading batch dimension where there is one. An FP8 operand and
a plan are those of operators.py.
"""

import math

import torch

own = False

BLOCK = 128  # values that a row is padded to a multiple of
MX = 32      # values that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3_MAX = 448.0


# ---- cases ------------------------------------------------------------------

def listed():
    return [
        # a decoding step's activations, quantized and read back
        dict(name="quantize_decode", op="quantize", batch=1, rows=16, cols=5120, dtype="bf16", block_2d=False, rowwise=True, colwise=False),
        # tokens gathered by expert and quantized for the product and for the weight gradient, in one call; both read back
        dict(name="quantize_sorted", op="quantize_sorted", tokens=8192, topk=4, experts=32, cols=5120, align=128, dtype="bf16", drop=0.0, colwise=True),
        # the experts' weights after an optimizer step, both orientations, and the values that training continues with
        dict(name="quantize_weights", op="quantize", batch=32, rows=2048, cols=4096, dtype="bf16", block_2d=True, rowwise=True, colwise=True),
        # a decoding step's dense product: bound by reading the weights
        dict(name="matmul_decode", op="matmul", m=16, n=8192, k=5120, out="bf16"),
        # no size a multiple of anything, as in a weight gradient
        dict(name="matmul_odd", op="matmul", m=777, n=1361, k=1999, out="fp32"),
        # a training batch's dense product
        dict(name="matmul_prompt", op="matmul", m=8192, n=8192, k=5120, out="bf16"),
        # experts' product for one decoding step
        dict(name="experts_decode", op="experts", tokens=64, topk=8, experts=64, align=16, n=4096, k=2048, out="bf16"),
        # experts' product for a prompt or a training batch
        dict(name="experts_prompt", op="experts", tokens=8192, topk=8, experts=64, align=128, n=4096, k=2048, out="bf16"),
        # experts' weight gradients
        dict(name="experts_weight_grad", op="experts_grad", tokens=8192, topk=4, experts=32, align=128, n=4096, k=2048, out="fp32"),
        # one sequence's next token through a gated expert layer
        dict(name="layer_one_token", op="layer", tokens=1, topk=8, experts=64, cols=4096, hidden=2048, gated=True, weights="mxfp4", drop=0.0),
        # a decoding step of 64 sequences
        dict(name="layer_decode", op="layer", tokens=64, topk=8, experts=64, cols=4096, hidden=2048, gated=True, weights="mxfp4", drop=0.0),
        # a decoding step of 16 sequences with FP8 weights and a plain activation
        dict(name="layer_fp8", op="layer", tokens=16, topk=4, experts=32, cols=5120, hidden=2048, gated=False, weights="fp8", drop=0.0),
    ]


def _spread(rng, low, high, odd=0.4):
    """A size over [low, high], even over its logarithm; sometimes rounded to a multiple of 128, 16 or 8."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() > odd:
        step = rng.choice([128, 16, 8])
        v = max(step, v // step * step)
    return max(low, min(high, v))


def _draw(rng):
    op = rng.choice(["quantize", "quantize_sorted", "matmul", "matmul", "experts", "experts_grad", "layer", "layer"])
    dtype = "fp32" if rng.random() < 0.25 else "bf16"
    experts = rng.choice([4, 7, 8, 16, 32, 60, 64, 128, 256])
    topk = min(experts, rng.randint(1, 8))
    drop = rng.choice([0.0, 0.0, 0.02, 0.3])
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op == "quantize":
        rowwise = rng.random() < 0.8
        return dict(op=op, batch=rng.choice([1, 1, 1, 3, 16]), rows=_spread(rng, 1, 8192), cols=_spread(rng, 64, 8192), dtype=dtype,
                    block_2d=rng.random() < 0.4, rowwise=rowwise, colwise=not rowwise or rng.random() < 0.5)
    if op == "quantize_sorted":
        return dict(op=op, tokens=_spread(rng, 1, 8192), topk=topk, experts=experts, cols=_spread(rng, 64, 8192), align=128,
                    dtype=dtype, drop=drop, colwise=rng.random() < 0.5)
    if op == "matmul":
        return dict(op=op, m=_spread(rng, 1, 8192), n=_spread(rng, 64, 8192), k=_spread(rng, 64, 8192), out=out)
    experts = min(experts, 64)
    topk = min(topk, experts)
    if op == "layer":
        return dict(op=op, tokens=_spread(rng, 1, 1024 // topk), topk=topk, experts=experts, cols=_spread(rng, 128, 8192), hidden=_spread(rng, 128, 4096),
                    gated=rng.random() < 0.7, weights=rng.choice(["mxfp4", "mxfp4", "fp8"]), drop=drop)
    return dict(op=op, tokens=_spread(rng, 1, 8192), topk=topk, experts=experts, align=128 if op == "experts_grad" else rng.choice([1, 16, 128]),
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


def _weights(g, kind, experts, n, k):
    """Normal weights [experts][n][k] as a program keeps them for the layer."""
    w = torch.randn((experts, n, k), generator=g, device="cuda") * k ** -0.5
    return _fp8_pack(w) if kind == "fp8" else _pack(*_plain_codes(w, False))


def prepare(case, seed):
    c, g = dict(case), _rng(seed)
    op = c["op"]
    s = {"case": c}
    if op in ("quantize_sorted", "experts", "experts_grad", "layer"):
        s["ids"], s["weights"] = _ids(g, c)
        align = c.get("align", 1)
        s["capacity"] = _capacity(c["tokens"], c["topk"], c["experts"], align)
        plan = _plain_sort(s["ids"], c["experts"], align, s["capacity"])
        if op != "layer":
            s["plan"] = plan
    if op == "quantize":
        s["x"] = _activations(g, (c["batch"], c["rows"], c["cols"]), _dtype(c["dtype"]))
    elif op == "quantize_sorted":
        s["x"] = _activations(g, (c["tokens"], c["cols"]), _dtype(c["dtype"]))
    elif op == "matmul":
        s["a"] = _pack(*_plain_codes(_activations(g, (c["m"], c["k"]), torch.float32), False))
        s["b"] = _pack(*_plain_codes(torch.randn((c["n"], c["k"]), generator=g, device="cuda"), False))
    elif op == "experts":
        x = _activations(g, (c["tokens"], c["k"]), torch.float32)
        s["a"] = _pack(*_plain_codes(_plain_gather(x, plan, c["topk"]), False))
        s["b"] = _pack(*_plain_codes(torch.randn((c["experts"], c["n"], c["k"]), generator=g, device="cuda"), True))
    elif op == "experts_grad":
        x = _activations(g, (c["tokens"], c["k"]), torch.float32)
        dy = torch.randn((c["tokens"], c["n"]), generator=g, device="cuda")
        s["a"], s["b"] = (_pack(*_plain_codes(_plain_gather(v, plan, c["topk"]).t(), False)) for v in (dy, x))
    elif op == "layer":
        s["x"] = _activations(g, (c["tokens"], c["cols"]), torch.bfloat16)
        s["w1"] = _weights(g, c["weights"], c["experts"], (1 + c["gated"]) * c["hidden"], c["cols"])
        s["w2"] = _weights(g, c["weights"], c["experts"], c["cols"], c["hidden"])
    if op in ("experts", "experts_grad", "layer"):
        s["longest"] = max(1, int((plan["offsets"][1:] - plan["offsets"][:-1]).max()))  # rows of the largest expert, known to the plain form's user
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


def _plain_codes(x, block_2d):
    """x [..][R][C] -> signed E2M1 values [..][R][pitch(C)] in 32 bits and the exponents of the scales [..][R][pitch(C) / 32]."""
    r, c = x.shape[-2:]
    high = MX if block_2d else 1
    v = torch.nn.functional.pad(x.float(), (0, -c % BLOCK, 0, -r % high))
    v = v.reshape(*x.shape[:-2], -1, high, v.shape[-1] // MX, MX)
    power = (torch.frexp(v.abs().amax((-3, -1), keepdim=True))[1] - 3).clamp(min=-127)
    power = torch.where(v.abs().amax((-3, -1), keepdim=True) > 0, power, -127)
    y = torch.ldexp(v, -power)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    q = (torch.round(y / step) * step).clamp(-6.0, 6.0)
    q = q.reshape(*x.shape[:-2], -1, v.shape[-2] * MX)[..., :r, :]
    power = power[..., 0].expand(v.shape[:-1]).reshape(*x.shape[:-2], -1, v.shape[-2])[..., :r, :]
    return q, power


def _pack(q, power):
    """The bytes of an operand: codes two by two, scales block by block of 128."""
    m = q.abs()
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8) + 8 * (q < 0).to(torch.uint8)
    scales = (power + 127).to(torch.uint8)
    scales = scales.reshape(*scales.shape[:-1], -1, BLOCK // MX).transpose(-3, -2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).contiguous(), scales.contiguous()


def _plain_values(q):
    """The 32-bit values [..][n][pitch] of an operand."""
    data, scales = q
    code = torch.stack([data & 15, data >> 4], -1).reshape(*data.shape[:-1], -1)
    m = (code & 7).float()
    m = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8)) * (1.0 - 2.0 * (code >= 8).float())
    power = scales.transpose(-3, -2).reshape(*data.shape[:-1], -1).int() - 127
    return torch.ldexp(m.reshape(*power.shape, MX), power[..., None]).reshape(m.shape)


def _fp8_pack(w):
    """E4M3 codes and FP32 scales of 128x128 blocks of w [E][n][k]."""
    e, n, k = w.shape
    v = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK)).reshape(e, _cdiv(n, BLOCK), BLOCK, _cdiv(k, BLOCK), BLOCK)
    scale = v.abs().amax((2, 4), keepdim=True) / E4M3_MAX
    q = (v / scale.clamp(min=1e-30)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.reshape(e, -1, _cdiv(k, BLOCK) * BLOCK)[:, :n].contiguous(), scale[:, :, 0, :, 0].transpose(1, 2).contiguous()


def _fp8_values(q):
    data, scales = q
    s = scales.transpose(-1, -2).repeat_interleave(BLOCK, -2)[..., :data.shape[-2], :]
    return data.float() * s.repeat_interleave(BLOCK, -1)


def _plain_experts(a, b, offsets, longest):
    """Each expert's rows of a times its matrix of b."""
    rows = a.shape[0]
    at = offsets[:-1, None].long() + torch.arange(longest, device=a.device)
    inside = at < offsets[1:, None]
    d = torch.bmm(a[at.clamp(max=rows - 1)], b.transpose(1, 2))
    result = d.new_zeros((rows + 1, d.shape[2]))
    result[torch.where(inside, at, rows)] = d
    return result[:rows]


def _plain_experts_grad(a, b, offsets, longest):
    at = offsets[:-1, None].long() + torch.arange(longest, device=a.device)
    inside = (at < offsets[1:, None])[..., None]
    at = at.clamp(max=a.shape[1] - 1)
    a = torch.where(inside, a.t()[at], 0.0)  # [E][longest][m]
    return torch.bmm(a.transpose(1, 2), b.t()[at])


def _plain_layer(s):
    c = s["case"]
    ids, experts, hidden = s["ids"], c["experts"], c["hidden"]
    values = _fp8_values if c["weights"] == "fp8" else _plain_values
    kept = (ids >= 0) & (ids < experts)
    x = s["x"].float()

    def act(h):
        g = h[..., :hidden]
        a = g / (1.0 + torch.exp(-g))
        return a * h[..., hidden:] if c["gated"] else a

    def product(v, weights, use):
        # few slots: each with its own expert's weights; else expert by expert
        w = values(tuple(t[use] for t in weights) if use is not None else weights)[..., :v.shape[-1]]
        if use is not None:
            return torch.bmm(w, v[..., None])[..., 0]
        return _plain_experts(v, w, plan["offsets"], s["longest"])

    if ids.numel() <= experts:
        use = ids.reshape(-1).long().clamp(0, experts - 1)
        y = product(act(product(x.repeat_interleave(c["topk"], 0), s["w1"], use)), s["w2"], use)
        y = y.reshape(*ids.shape, -1)
    else:
        plan = _plain_sort(ids, experts, 1, s["capacity"])
        y = product(act(product(_plain_gather(x, plan, c["topk"]), s["w1"], None)), s["w2"], None)
        y = y[plan["slot_rows"].long().clamp(min=0)]
    return (torch.where(kept[..., None], y, 0.0) * s["weights"][..., None]).sum(1).to(torch.bfloat16)


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("quantize", "quantize_sorted"):
        x = s["x"] if op == "quantize" else _plain_gather(s["x"], s["plan"], c["topk"])[None]

        def read_back(x):
            q, power = _plain_codes(x, c.get("block_2d", False))
            v = torch.ldexp(q.reshape(*power.shape, MX), power[..., None]).reshape(q.shape)
            return v[..., :x.shape[-1]].to(x.dtype)

        out = {}
        if c.get("rowwise", True):
            out["row"] = read_back(x)
        if c["colwise"]:
            out["col"] = read_back(x.transpose(-1, -2))
        return out
    if op == "layer":
        return _plain_layer(s)
    a, b = _plain_values(s["a"]), _plain_values(s["b"])
    if op == "matmul":
        d = a.matmul(b.t())
    elif op == "experts":
        d = _plain_experts(a, b, s["plan"]["offsets"], s["longest"])
    else:
        d = _plain_experts_grad(a, b, s["plan"]["offsets"], s["longest"])
    return d.to(_dtype(c["out"]))


# ---- the package's calls ----------------------------------------------------

def _run_own(s):
    import nvfp4_block_scaled_05_amd as nv

    c = s["case"]
    op = c["op"]

    def mx(q, k):
        return nv.Mxfp4Tensor(q[0], q[1], q[0].shape[-2], k)

    def plan():
        return nv.ExpertPlan(**s["plan"], align=c["align"])

    if op in ("quantize", "quantize_sorted"):
        row, col = nv.mxfp4_quantize(s["x"], rowwise=c.get("rowwise", True), columnwise=c["colwise"], block_2d=c.get("block_2d", False),
                                     plan=plan() if op == "quantize_sorted" else None)
        out = {}
        for name, q in (("row", row), ("col", col)):
            if q is not None:
                v = nv.mxfp4_dequantize(q, out_dtype=_dtype(c["dtype"]))
                out[name] = v if op == "quantize" else v[None]
        return out
    if op == "matmul":
        return nv.mxfp4_matmul(mx(s["a"], c["k"]), mx(s["b"], c["k"]), out_dtype=_dtype(c["out"]))
    if op == "experts":
        return nv.mxfp4_matmul_grouped(mx(s["a"], c["k"]), mx(s["b"], c["k"]), plan(), out_dtype=_dtype(c["out"]))
    if op == "experts_grad":
        return nv.mxfp4_matmul_grouped_k(mx(s["a"], s["capacity"]), mx(s["b"], s["capacity"]), plan(), out_dtype=_dtype(c["out"]))

    def weights(q, k):
        return nv.Fp8Tensor(q[0], q[1], q[0].shape[-2], k, True) if c["weights"] == "fp8" else mx(q, k)

    return nv.expert_mlp(s["x"], s["ids"], s["weights"], weights(s["w1"], c["cols"]), weights(s["w2"], c["hidden"]), gated=c["gated"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ------------------------------------------

def work(case):
    c = dict(case)
    op = c["op"]
    size = {"bf16": 2, "fp32": 4}
    mx = 1 / 2 + 1 / MX  # bytes of a value
    if op == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * k * mx + size[c["out"]] * m * n, "flops": 2 * m * n * k}
    if op == "quantize":  # the codes are written and read back
        n = c["batch"] * c["rows"] * c["cols"]
        b, sides = size[c["dtype"]], int(c["rowwise"]) + int(c["colwise"])
        return {"bytes": n * (b + sides * (2 * mx + b)), "flops": 4 * n * sides}
    slots = c["tokens"] * c["topk"]
    used = min(c["experts"], slots)
    kept = slots * (1 - c.get("drop", 0.0))
    if op == "layer":
        n1, k, f = (1 + c["gated"]) * c["hidden"], c["cols"], c["hidden"]
        each = (n1 * k + k * f) * (1 if c["weights"] == "fp8" else mx)
        return {"bytes": used * each + 4 * c["tokens"] * k + 8 * slots, "flops": 2 * kept * (n1 * k + k * f)}
    capacity = _capacity(c["tokens"], c["topk"], c["experts"], c["align"])
    if op == "quantize_sorted":
        b, sides = size[c["dtype"]], 1 + int(c["colwise"])
        return {"bytes": 4 * capacity + b * c["tokens"] * c["cols"] + sides * capacity * c["cols"] * (2 * mx + b), "flops": 4 * kept * c["cols"] * sides}
    n, k = c["n"], c["k"]
    if op == "experts":
        return {"bytes": slots * k * mx + used * n * k * mx + size[c["out"]] * capacity * n, "flops": 2 * slots * n * k}
    return {"bytes": slots * (n + k) * mx + size[c["out"]] * c["experts"] * n * k, "flops": 2 * slots * n * k}


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_values(x, block_2d):
    """What the rows of x [R][C] are after quantization, in 64 bits: the nearest E2M1 value by the middles between
    neighbours, a middle going to the even code, of each value over its block's power of two."""
    r, c = x.shape
    high = MX if block_2d else 1
    v = x.new_zeros((_cdiv(r, high) * high, _cdiv(c, MX) * MX), dtype=torch.float64)
    v[:r, :c] = x.double()
    amax = v.unfold(0, high, high).unfold(1, MX, MX).abs().amax((2, 3))
    scale = torch.exp2(torch.floor(torch.log2(amax)).clamp(min=-125) - 2)
    scale = scale.repeat_interleave(high, 0).repeat_interleave(MX, 1)
    y = v.abs() / scale
    code = torch.zeros_like(y, dtype=torch.long)
    for i in range(7):
        middle = (E2M1[i] + E2M1[i + 1]) / 2
        code += (y > middle) | ((y == middle) & (i % 2 == 1))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    return (grid[code] * torch.sign(v) * scale)[:r, :c]


def _exact_operand(q):
    """[n][pitch] in 64 bits, from the bytes."""
    data, scales = q
    table = torch.tensor([s * v for s in (1.0, -1.0) for v in E2M1], dtype=torch.float64, device=data.device)
    v = torch.empty((data.shape[0], 2 * data.shape[1]), dtype=torch.float64, device=data.device)
    v[:, 0::2] = table[(data & 15).long()]
    v[:, 1::2] = table[(data >> 4).long()]
    for j in range(v.shape[1] // MX):
        v[:, j * MX:(j + 1) * MX] *= torch.exp2(scales[j // 4, :, j % 4].double() - 127)[:, None]
    return v


def _exact_fp8(q):
    data, scales = q
    v = data.to(torch.float32).double()
    at = torch.arange(data.shape[0], device=data.device) // BLOCK
    for j in range(scales.shape[0]):
        v[:, j * BLOCK:(j + 1) * BLOCK] *= scales[j].double()[at][:, None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    op = c["op"]
    if op in ("quantize", "quantize_sorted"):
        x = s["x"]
        if op == "quantize_sorted":
            rows = x.new_zeros((s["capacity"], c["cols"]))
            used = (s["plan"]["row_slots"] >= 0).nonzero()[:, 0]
            rows[used] = x[torch.div(s["plan"]["row_slots"][used].long(), c["topk"], rounding_mode="floor")]
            x = rows[None]
        block_2d, out = c.get("block_2d", False), {}
        if c.get("rowwise", True):
            out["row"] = torch.stack([_exact_values(m, block_2d) for m in x])
        if c["colwise"]:
            out["col"] = torch.stack([_exact_values(m.t(), block_2d) for m in x])
        return out
    if op == "matmul":
        return _exact_operand(s["a"]) @ _exact_operand(s["b"]).t()
    if op in ("experts", "experts_grad"):
        starts = s["plan"]["offsets"].tolist()
        a = _exact_operand(s["a"])
        if op == "experts":
            d = a.new_zeros((s["capacity"], c["n"]))
            for e in range(c["experts"]):
                w = _exact_operand((s["b"][0][e], s["b"][1][e]))
                d[starts[e]:starts[e + 1]] = a[starts[e]:starts[e + 1]] @ w.t()
            return d
        b = _exact_operand(s["b"])
        return torch.stack([a[:, starts[e]:starts[e + 1]] @ b[:, starts[e]:starts[e + 1]].t() for e in range(c["experts"])])
    # the layer: expert by expert, its tokens one after the other
    operand = _exact_fp8 if c["weights"] == "fp8" else _exact_operand
    out = torch.zeros((c["tokens"], c["cols"]), dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        token, choice = (s["ids"] == e).nonzero(as_tuple=True)
        if not token.numel():
            continue
        w1, w2 = (operand((w[0][e], w[1][e])) for w in (s["w1"], s["w2"]))
        h = s["x"][token].double() @ w1[:, :c["cols"]].t()
        gate = h[:, :c["hidden"]]
        a = gate * torch.sigmoid(gate)
        if c["gated"]:
            a = a * h[:, c["hidden"]:]
        out.index_add_(0, token, s["weights"][token, choice].double()[:, None] * (a @ w2[:, :c["hidden"]].t()))
    return out
