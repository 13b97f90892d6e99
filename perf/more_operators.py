"""The operators around the experts: what is measured, and their plain forms.

Four groups of operators, each with its plain torch form (32-bit arithmetic, rounded once at the
end), its 64-bit definition (``exact``) and the calls a user makes of the package:

* ``sort``: tokens laid out by the experts that were chosen for them (with their scales and weights),
  and the gradient of it;
* ``combine``: the experts' rows back to their tokens, weighted and summed, and the gradient of it;
* ``norm``: a residual's addition and the root-mean-square norm of the sum, with the result also in 8
  bits or MXFP4, and the gradient of it;
* ``gate_grad``: the gradient of the routing decision (scores, top-k, scaled weights).
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "i8": torch.int8}
BYTES = {"f16": 2, "bf16": 2, "f32": 4, "i8": 1}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one token's row in 8 bits, laid out for its 8 experts (decode)
        {"name": "sort_1x7168_top8of256_i8", "op": "sort", "grad": False, "T": 1, "H": 7168, "k": 8, "E": 256,
         "first": 0, "held": 256, "padded": 0, "dtype": "i8", "skew": 0.0},
        # a prefill or training batch, every expert held
        {"name": "sort_16384x7168_top8of256_bf16", "op": "sort", "grad": False, "T": 16384, "H": 7168, "k": 8, "E": 256,
         "first": 0, "held": 256, "padded": 0, "dtype": "bf16", "skew": 0.5},
        # a rank that holds a third of the experts, a padded batch, rows of an odd size
        {"name": "sort_4099x2050_top6of60_f16", "op": "sort", "grad": False, "T": 4099, "H": 2050, "k": 6, "E": 60,
         "first": 20, "held": 20, "padded": 131, "dtype": "f16", "skew": 0.5},
        # a training step's gradient of the sort
        {"name": "sort_grad_8191x4096_top4of64_bf16", "op": "sort", "grad": True, "T": 8191, "H": 4096, "k": 4, "E": 64,
         "first": 0, "held": 64, "padded": 0, "dtype": "bf16", "skew": 0.5},
        # a decode step's rows back to three tokens
        {"name": "combine_3x5120_top8of128_bf16", "op": "combine", "grad": False, "T": 3, "H": 5120, "k": 8, "E": 128,
         "first": 0, "held": 128, "padded": 0, "dtype": "bf16", "skew": 0.0},
        # a prefill batch's rows back
        {"name": "combine_16384x7168_top8of256_bf16", "op": "combine", "grad": False, "T": 16384, "H": 7168, "k": 8,
         "E": 256, "first": 0, "held": 256, "padded": 0, "dtype": "bf16", "skew": 0.5},
        # a training step's gradient of the weighted sum: of the rows and of the weights
        {"name": "combine_grad_4095x7168_top8of256_bf16", "op": "combine", "grad": True, "T": 4095, "H": 7168, "k": 8,
         "E": 256, "first": 0, "held": 256, "padded": 0, "dtype": "bf16", "skew": 0.5},
        # the norm in front of a decode step's experts, in MXFP8
        {"name": "norm_1x7168_bf16_mxfp8", "op": "norm", "grad": False, "T": 1, "H": 7168, "dtype": "bf16",
         "residual": True, "quant": "mxfp8"},
        # the same for a prefill batch, in int8 with a scale for each row
        {"name": "norm_16384x7168_bf16_int8", "op": "norm", "grad": False, "T": 16384, "H": 7168, "dtype": "bf16",
         "residual": True, "quant": "int8"},
        # a training step's gradient of the norm, rows that are no multiple of 16 bytes
        {"name": "norm_grad_8191x4100_bf16", "op": "norm", "grad": True, "T": 8191, "H": 4100, "dtype": "bf16",
         "residual": True, "quant": ""},
        # the router's gradient on a small batch, softmax scores in float32
        {"name": "gate_grad_61x60_top6_f32", "op": "gate_grad", "T": 61, "E": 60, "k": 6, "dtype": "f32", "norm": 0,
         "bias": False, "out": False},
        # the router's gradient on a training batch, biased sigmoid scores
        {"name": "gate_grad_16384x256_top8_bf16", "op": "gate_grad", "T": 16384, "E": 256, "k": 8, "dtype": "bf16",
         "norm": 1, "bias": True, "out": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sort", "sort", "combine", "combine", "norm", "norm", "gate_grad"])
    if op == "gate_grad":
        E = _log(rng, 4, 1024)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, E)),
                "dtype": rng.choice(["f16", "bf16", "f32"]), "norm": rng.choice([0, 1, 2]), "bias": rng.random() < 0.5,
                "out": rng.random() < 0.3}
    H = _log(rng, 64, 8192)
    if rng.random() < 0.5:
        H = 64 * max(1, H // 64)
    if op == "norm":
        grad = rng.random() < 0.4
        if not grad:
            H = 2 * ((H + 1) // 2)
        dtype = rng.choice(["f16", "bf16", "f32"])
        return {"op": op, "grad": grad, "T": _log(rng, 1, min(16384, 16384 * 7168 * 2 // (H * BYTES[dtype]))), "H": H,
                "dtype": dtype, "residual": rng.random() < 0.7,
                "quant": "" if grad else rng.choice(["", "int8", "e4m3", "e4m3_128", "mxfp8", "mxfp4"])}
    grad = rng.random() < 0.4
    dtype = rng.choice(["f16", "bf16", "f32"] + ["i8"] * (op == "sort" and not grad))
    E = _log(rng, 2, 512)
    k = rng.randint(1, min(8, E))
    passes = 2 * k + 1 if grad and op == "combine" else k + 1     # over a token's row
    T = _log(rng, 1, max(1, min(16384, 16384 * 7168 * 9 * 2 // (H * BYTES[dtype] * passes))))
    held = rng.choice([E, E, max(1, E // rng.choice([2, 4, 8]))])
    return {"op": op, "grad": grad, "T": T, "H": H, "k": k, "E": E, "first": rng.randint(0, E - held), "held": held,
            "padded": rng.choice([0, 0, T // rng.randint(2, 20)]), "dtype": dtype, "skew": rng.choice([0.0, 0.3, 0.5])}


# --------------------------------------------------------------------------- inputs

def _hidden(gen, rows, K):
    """Hidden states: normal, rows of different sizes, a few channels much larger than the others."""
    x = torch.randn(rows, K, generator=gen, device="cuda")
    x = x * torch.exp(0.5 * torch.randn(rows, 1, generator=gen, device="cuda"))
    loud = torch.rand(K, generator=gen, device="cuda") < 0.005
    return torch.where(loud, 8 * x, x)


def _choice(gen, T, E, k, skew):
    """k different experts for each token, expert j drawn with a weight of (j+1)^-skew in a shuffled order."""
    p = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -skew
    p = p[torch.randperm(E, generator=gen, device="cuda")]
    u = torch.rand(T, E, generator=gen, device="cuda").clamp_(1e-20, 1 - 1e-7)
    return torch.topk(p.log() - torch.log(-torch.log(u)), k, dim=1)[1].int()


def _maps(experts, first, held):
    """(row of each slot or -1 [T, k], flat slot of each row or -1 [T k]) of a layout by expert."""
    T, k = experts.shape
    key = experts.flatten().long() - first
    key = torch.where((key >= 0) & (key < held), key, torch.full_like(key, held))
    order = torch.argsort(key, stable=True)
    row = torch.empty_like(order)
    row[order] = torch.arange(T * k, device=order.device)
    row = torch.where(key < held, row, torch.full_like(row, -1))
    slot = torch.where(key[order] < held, order, torch.full_like(order, -1))
    return row.view(T, k).int(), slot.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    T = case["T"]
    if case["op"] == "gate_grad":
        E, k, dtype = case["E"], case["k"], DTYPES[case["dtype"]]
        s["x"] = torch.randn(T, E, generator=gen, device="cuda").to(dtype)
        s["b"] = (0.1 * torch.rand(E, generator=gen, device="cuda")).to(dtype) if case["bias"] else None
        score = _score(s["x"].float(), case["norm"])
        s["experts"] = torch.topk(score if s["b"] is None else score + s["b"].float(), k, dim=1)[1].int()
        s["dy"] = torch.randn(T, k, generator=gen, device="cuda").to(dtype)
        s["dout"] = 0.1 * torch.randn(T, E, generator=gen, device="cuda") if case["out"] else None
        return s
    H, dtype = case["H"], DTYPES[case["dtype"]]
    if case["op"] == "norm":
        s["x"] = _hidden(gen, T, H).to(dtype)
        s["res"] = _hidden(gen, T, H).to(dtype) if case["residual"] else None
        s["w"] = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(dtype)
        if case["grad"]:
            s["dy"] = torch.randn(T, H, generator=gen, device="cuda").to(dtype)
            s["dh"] = torch.randn(T, H, generator=gen, device="cuda").to(dtype) if case["residual"] else None
        return s
    k = case["k"]
    experts = _choice(gen, T, case["E"], k, case["skew"])
    if case["padded"]:
        experts[T - case["padded"]:] = -1
    weight = torch.rand(T, k, generator=gen, device="cuda") + 0.05
    weight = weight / weight.sum(1, keepdim=True)
    if case["op"] == "sort" and not case["grad"]:
        x = _hidden(gen, T, H)
        s["experts"], s["weight"], s["scales"] = experts, weight, None
        if case["dtype"] == "i8":
            s["scales"] = x.abs().amax(1) / 127
            x = torch.round(x / s["scales"][:, None])
        s["x"] = x.to(dtype)
        return s
    s["row"], s["slot"] = _maps(experts, case["first"], case["held"])
    s["rows"] = torch.randn(T * k, H, generator=gen, device="cuda").to(dtype)
    if case["op"] == "combine":
        s["weight"] = weight.to(dtype)
        if case["grad"]:
            s["dy"] = torch.randn(T, H, generator=gen, device="cuda").to(dtype)
    return s


# --------------------------------------------------------------------------- plain forms

def _score(x, norm):
    return torch.softmax(x, -1) if norm == 0 else torch.sigmoid(x) if norm == 1 else torch.nn.functional.softplus(x)


def _plain_sort(s):
    T, k, held = s["T"], s["k"], s["held"]
    row, slot = _maps(s["experts"], s["first"], held)
    key = s["experts"].flatten().long() - s["first"]
    here = ((key >= 0) & (key < held)).int()
    num = torch.zeros(held, dtype=torch.int32, device=key.device).index_add_(0, key.clamp(0, held - 1), here)
    used = slot >= 0
    at = slot.clamp(min=0).long()
    rows = torch.where(used[:, None], s["x"][at // k], torch.zeros((), dtype=s["x"].dtype, device=key.device))
    weight = torch.where(used, s["weight"].flatten()[at], 0.0)
    scales = None if s["scales"] is None else torch.where(used, s["scales"][at // k], 0.0)
    return {"rows": rows, "scales": scales, "slot": slot, "row": row, "num": num, "weight": weight}


def _picked(rows, row):
    """[T, k, H] float32: each slot's row, zeros where it has none."""
    x = rows[row.clamp(min=0).long()].float()
    return torch.where((row >= 0)[..., None], x, torch.zeros((), device=x.device))


def _plain_combine(s):
    x = _picked(s["rows"], s["row"])
    if s["op"] == "sort":
        return x.sum(1).to(s["rows"].dtype)
    return (x * s["weight"].float()[..., None]).sum(1).to(s["rows"].dtype)


def _plain_combine_grad(s):
    dy, T, k = s["dy"].float(), s["T"], s["k"]
    dw = (_picked(s["rows"], s["row"]) * dy[:, None]).sum(2)
    at = s["slot"].clamp(min=0).long()
    drows = dy[at // k] * s["weight"].float().flatten()[at][:, None]
    drows = torch.where((s["slot"] >= 0)[:, None], drows, torch.zeros((), device=dy.device))
    return {"rows": drows.to(s["rows"].dtype), "weight": dw.to(s["weight"].dtype)}


def _e2m1(v):
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.sign(v) * torch.clamp(torch.round(a / step) * step, max=6.0)


def _e4m3(v):
    """The nearest e4m3 value: 4 bits of significand down to 2^-6, steps of 2^-9 below, held to 448."""
    exponent = (torch.frexp(v)[1] - 1).clamp(min=-6)
    q = torch.ldexp(torch.round(torch.ldexp(v, 3 - exponent)), exponent - 3)
    return q.clamp(-448, 448)


def _plain_quant(y, quant):
    """The float32 values that y's rows stand for in 8 or 4 bits."""
    T, H = y.shape
    if quant in ("int8", "e4m3"):
        top = 127.0 if quant == "int8" else 448.0
        scale = (y.abs().amax(1, keepdim=True) / top).clamp(min=2.0 ** -126)
        v = y / scale
        return (torch.round(v) if quant == "int8" else _e4m3(v)) * scale
    block = 128 if quant == "e4m3_128" else 32
    b = torch.nn.functional.pad(y, (0, -H % block)).reshape(T, -1, block)
    amax = b.abs().amax(-1, keepdim=True)
    if quant == "e4m3_128":
        scale = (amax / 448).clamp(min=2.0 ** -126)
        out = _e4m3(b / scale) * scale
    else:
        shared = torch.frexp(amax)[1] - 1 - (8 if quant == "mxfp8" else 2)
        shared = torch.where(amax == 0, torch.full_like(shared, -127), shared.clamp(min=-127))
        v = torch.ldexp(b, -shared)
        out = torch.ldexp(_e4m3(v) if quant == "mxfp8" else _e2m1(v), shared)
    return out.reshape(T, -1)[:, :H]


def _plain_norm(s):
    h = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6) * s["w"].float()
    dtype = s["x"].dtype
    return {"y": y.to(dtype), "h": None if s["res"] is None else h.to(dtype),
            "q": _plain_quant(y, s["quant"]).to(dtype) if s["quant"] else None}


def _plain_norm_grad(s):
    h, dy = s["x"].float(), s["dy"].float()
    r = torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-6)
    g, unit = dy * s["w"].float(), h * r
    dx = r * (g - unit * (g * unit).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"x": dx.to(s["x"].dtype), "w": (dy * unit).sum(0).to(s["w"].dtype)}


def _plain_gate_grad(s):
    x, at, dy = s["x"].float(), s["experts"].long(), s["dy"].float()
    score = _score(x, s["norm"])
    p = (score if s["b"] is None else score + s["b"].float()).gather(1, at)
    total = p.sum(1, keepdim=True) + 1e-20
    dp = 2.5 / total * (dy - (dy * p).sum(1, keepdim=True) / total)
    ds = (torch.zeros_like(x) if s["dout"] is None else s["dout"]).scatter_add(1, at, dp)
    if s["norm"] == 0:
        dx = score * (ds - (ds * score).sum(1, keepdim=True))
    else:
        dx = ds * (score * (1 - score) if s["norm"] == 1 else torch.sigmoid(x))
    return {"x": dx.to(s["x"].dtype), "bias": None if s["b"] is None else ds.sum(0).to(s["x"].dtype)}


# --------------------------------------------------------------------------- one pass

def run(state):
    s = state
    op = s["op"]
    if not own:
        if op == "gate_grad":
            return _plain_gate_grad(s)
        if op == "norm":
            return _plain_norm_grad(s) if s["grad"] else _plain_norm(s)
        if op == "sort" and not s["grad"]:
            return _plain_sort(s)
        return _plain_combine_grad(s) if op == "combine" and s["grad"] else _plain_combine(s)
    elif op == "sort" and not s["grad"] and "as_called" not in s:
        # the package gives the sorted weights as [T k, 1], as the grouped product takes them, the plain form as [T k]
        out = run({**s, "as_called": True})
        return {**out, "weight": out["weight"].view(-1)}
    import moe_expert_token_gb300 as moe

    if op == "gate_grad":
        dx, dbias, _ = moe.moe_gating_top_k_grad(s["dy"], s["x"], s["experts"], bias=s["b"], grad_out=s["dout"],
                                                 routed_scaling_factor=2.5, norm_type=s["norm"])
        return {"x": dx, "bias": dbias}
    if op == "norm":
        if s["grad"]:
            dx, dw = moe.moe_add_rms_norm_grad(s["dy"], s["x"], s["w"], grad_h=s["dh"], eps=1e-6)
            return {"x": dx, "w": dw}
        y, h, q, scales = moe.moe_add_rms_norm(s["x"], s["w"], s["res"], eps=1e-6, quant=s["quant"] or None)
        if s["quant"] == "mxfp4":
            q = moe.moe_mx_dequantize(q, scales, s["x"].dtype)
        elif s["quant"]:
            q = moe.moe_dequantize_rows(q, scales, s["x"].dtype)
        return {"y": y, "h": None if s["res"] is None else h, "q": q}
    if op == "sort":
        if s["grad"]:
            return moe.moe_sort_tokens_grad(s["rows"], s["row"])
        rows, scales, slot, row, num, weight = moe.moe_sort_tokens(
            s["x"], s["experts"], s["held"], first_expert=s["first"], per_token_scales=s["scales"],
            expert_topk_weight=s["weight"])
        return {"rows": rows, "scales": scales, "slot": slot, "row": row, "num": num, "weight": weight}
    if s["grad"]:
        drows, dw = moe.moe_combine_tokens_grad(s["dy"], s["rows"], s["row"], s["slot"], s["weight"])
        return {"rows": drows, "weight": dw}
    return moe.moe_combine_tokens(s["rows"], s["row"], s["weight"])


def work(case):
    """Each input read once, each output written once. Rows of experts that are not held here are not read, and the
    rows in their place are written as zeros; a padded token has no rows."""
    T = case["T"]
    if case["op"] == "gate_grad":
        E, k, b = case["E"], case["k"], BYTES[case["dtype"]]
        return {"bytes": 2 * T * E * b + T * k * (4 + b) + (4 * T * E if case["out"] else 0), "flops": 10 * T * E}
    H, b = case["H"], BYTES[case["dtype"]]
    if case["op"] == "norm":
        n = T * H * b
        if case["grad"]:
            return {"bytes": n * (4 if case["residual"] else 3) + 2 * H * b, "flops": 10 * T * H}
        # the 8-bit rows are written, read again and their values written
        q = {"": 0, "int8": 2 * T * H + n, "e4m3": 2 * T * H + n, "e4m3_128": 2 * T * H + n, "mxfp8": 2 * T * H + n,
             "mxfp4": T * H + n}[case["quant"]]
        return {"bytes": n * (4 if case["residual"] else 2) + H * b + q, "flops": 8 * T * H}
    k = case["k"]
    used = (T - case["padded"]) * k * case["held"] / case["E"]
    if case["op"] == "sort" and not case["grad"]:
        n = (T - case["padded"]) * H * b + T * k * H * b + T * k * (4 + 4 + 4 + 8)
        return {"bytes": n + (4 * T + 4 * T * k if case["dtype"] == "i8" else 0), "flops": T * k}
    if case["grad"] and case["op"] == "combine":
        return {"bytes": (T * H + used * H + T * k * H) * b + T * k * (4 + 4 + 2 * b), "flops": 3 * used * H}
    return {"bytes": (used * H + T * H) * b + T * k * (4 + b), "flops": 2 * used * H}


# --------------------------------------------------------------------------- 64 bits

def _exact_sort(s):
    k = s["k"]
    flat = s["experts"].flatten()
    slots = torch.cat([torch.nonzero(flat == e).flatten() for e in range(s["first"], s["first"] + s["held"])])
    n = slots.numel()
    rows = torch.zeros(flat.numel(), s["H"], dtype=s["x"].dtype, device="cuda")
    weight = torch.zeros(flat.numel(), dtype=torch.float64, device="cuda")
    rows[:n] = s["x"][torch.div(slots, k, rounding_mode="floor")]
    weight[:n] = s["weight"].double().flatten()[slots]
    scales = None
    if s["scales"] is not None:
        scales = torch.zeros(flat.numel(), dtype=torch.float64, device="cuda")
        scales[:n] = s["scales"].double()[torch.div(slots, k, rounding_mode="floor")]
    floating = s["x"].is_floating_point()
    return {"rows": rows if floating else None, "scales": scales, "slot": None, "row": None, "num": None, "weight": weight}


def _exact_combine(s):
    y = torch.zeros(s["T"], s["H"], dtype=torch.float64, device="cuda")
    for j in range(s["k"]):
        t = torch.nonzero(s["row"][:, j] >= 0).flatten()
        for part in t.split(2048):
            x = s["rows"][s["row"][part, j].long()].double()
            y[part] += x if s["op"] == "sort" else x * s["weight"][part, j].double()[:, None]
    return y


def _exact_combine_grad(s):
    k = s["k"]
    drows = torch.zeros(s["T"] * k, s["H"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["T"], k, dtype=torch.float64, device="cuda")
    for j in range(k):
        t = torch.nonzero(s["row"][:, j] >= 0).flatten()
        for part in t.split(2048):
            at, dy = s["row"][part, j].long(), s["dy"][part].double()
            drows[at] = dy * s["weight"][part, j].double()[:, None]
            dw[part, j] = torch.einsum("th,th->t", dy, s["rows"][at].double())
    return {"rows": drows, "weight": dw}


def _nearest(v, values):
    """v's magnitudes rounded to the nearest of `values` (ascending; ties to the even index), with v's signs."""
    a = v.abs()
    middle = (values[1:] + values[:-1]) / 2
    i = torch.bucketize(a, middle)                       # ties go down
    last = len(values) - 1
    tie = (i < last) & (a == middle[i.clamp(max=last - 1)]) & (i % 2 == 1)
    return torch.sign(v) * values[i + tie.long()]


def _exact_quant(y, quant):
    H = y.shape[1]
    if quant == "mxfp4":
        values = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    elif quant == "int8":
        values = [float(i) for i in range(128)]
    else:
        values = [i * 2.0 ** -9 for i in range(8)] + [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)]
        values = [v for v in values if v <= 448]
    values = torch.tensor(values, dtype=torch.float64, device=y.device)
    step = {"int8": H, "e4m3": H, "e4m3_128": 128}.get(quant, 32)
    out = torch.empty_like(y)
    for lo in range(0, H, step):
        b = y[:, lo:lo + step]
        m = b.abs().amax(1, keepdim=True)
        if quant.startswith("mx"):
            e = torch.floor(torch.log2(m))
            e = e + (torch.exp2(e + 1) <= m).double() - (torch.exp2(e) > m).double()
            scale = torch.exp2(torch.clamp(e - (8 if quant == "mxfp8" else 2), -127, 127))
        else:
            scale = torch.clamp(m / values[-1], min=2.0 ** -126)
        out[:, lo:lo + step] = _nearest(b / scale, values) * scale
    return out


def _exact_norm(s):
    h = s["x"].double()
    if s["res"] is not None:
        h = h + s["res"].double()
    y = torch.empty_like(h)
    for part in torch.arange(s["T"], device="cuda").split(4096):
        z = h[part]
        y[part] = z / torch.sqrt(torch.einsum("th,th->t", z, z) / s["H"] + 1e-6)[:, None] * s["w"].double()
    return {"y": y, "h": None if s["res"] is None else h, "q": _exact_quant(y, s["quant"]) if s["quant"] else None}


def _exact_norm_grad(s):
    """d/dh of sum(dy * w * h / root), root = sqrt(mean(h^2) + eps): dy w / root - h (sum dy w h) / (H root^3)."""
    dw = torch.zeros(s["H"], dtype=torch.float64, device="cuda")
    dx = torch.empty(s["T"], s["H"], dtype=torch.float64, device="cuda")
    for part in torch.arange(s["T"], device="cuda").split(4096):
        h, g = s["x"][part].double(), s["dy"][part].double()
        root = torch.sqrt(torch.einsum("th,th->t", h, h) / s["H"] + 1e-6)[:, None]
        inner = torch.einsum("th,th,h->t", g, h, s["w"].double())[:, None]
        dx[part] = g * s["w"].double() / root - h * inner / (s["H"] * root ** 3)
        dw += torch.einsum("th,th->h", g, h / root)
    if s["dh"] is not None:
        dx += s["dh"].double()
    return {"x": dx, "w": dw}


def _exact_gate_grad(s):
    """By the chain of the definition's steps, one Jacobian after the other."""
    T, E, k = s["T"], s["E"], s["k"]
    x = s["x"].double()
    if s["norm"] == 0:
        z = torch.exp(x - x.max(1, keepdim=True)[0])
        score = z / z.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x)) if s["norm"] == 1 else torch.log1p(torch.exp(x))
    at = s["experts"].long()
    tokens = torch.arange(T, device="cuda")
    b = torch.zeros(E, dtype=torch.float64, device="cuda") if s["b"] is None else s["b"].double()
    p = score[tokens[:, None], at] + b[at]
    total = p.sum(1) + 1e-20
    ds = torch.zeros_like(x) if s["dout"] is None else s["dout"].double().clone()
    dy = s["dy"].double()
    for j in range(k):                                   # dy_i / dp_j = 2.5 (delta_ij / total - p_i / total^2)
        dp = sum(dy[:, i] * 2.5 * ((i == j) / total - p[:, i] / total ** 2) for i in range(k))
        ds[tokens, at[:, j]] += dp
    if s["norm"] == 0:                                   # dscore_i / dx_j = score_i (delta_ij - score_j)
        dx = score * ds - score * torch.einsum("te,te->t", score, ds)[:, None]
    elif s["norm"] == 1:
        dx = ds * torch.exp(-x) / (1 + torch.exp(-x)) ** 2
    else:
        dx = ds / (1 + torch.exp(-x))
    return {"x": dx, "bias": None if s["b"] is None else ds.sum(0)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gate_grad":
        return _exact_gate_grad(s)
    if case["op"] == "norm":
        return _exact_norm_grad(s) if case["grad"] else _exact_norm(s)
    if case["op"] == "sort" and not case["grad"]:
        return _exact_sort(s)
    return _exact_combine_grad(s) if case["op"] == "combine" and case["grad"] else _exact_combine(s)
