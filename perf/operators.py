"""The cases that the matrix operators are measured on, their plain forms and their 64-bit definitions.

The operators: orthogonalising a stack of matrices by Newton-Schulz products; the optimizer step built on it
(momentum, orthogonalised update, fp32 master weights, 16-bit slot); MXFP4 quantisation along rows and columns;
the product of MXFP4 operands; the linear layer whose forward and backward products take MXFP4 operands.
"""
import math

import torch

own = False

COEFFS = (3.4445, -4.7750, 2.0315)
NS_STEPS = 5
NS_EPS = 1e-7
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the latency end: one small projection of a head, fp32 momentum in, bf16 update out
        {"name": "ortho one 96x65", "op": "ortho", "count": 1, "rows": 96, "cols": 65, "src": "f32", "dst": "bf16"},
        # a wide matrix of odd sizes, fp16 both ways
        {"name": "ortho odd 1500x4099", "op": "ortho", "count": 1, "rows": 1500, "cols": 4099, "src": "f16", "dst": "f16"},
        # many small matrices in one call, as a stack of per-head blocks gives
        {"name": "muon 32 of 128x128", "op": "muon", "count": 32, "rows": 128, "cols": 128, "slot": "bf16", "lr": 3e-4,
         "wd": 0.01, "nesterov": True},
        # the attention input projections of eight layers of a GPT-2-sized shard
        {"name": "muon 8 of 2304x768", "op": "muon", "count": 8, "rows": 2304, "cols": 768, "slot": "f16", "lr": 3e-4,
         "wd": 0.01, "nesterov": True},
        # one large feed-forward matrix of a 7B-sized buffer, tall
        {"name": "muon 11008x4096", "op": "muon", "count": 1, "rows": 11008, "cols": 4096, "slot": "bf16", "lr": 1e-4,
         "wd": 0.0, "nesterov": False},
        # the payload of a large weight in both directions, sent and rebuilt
        {"name": "quantize 8192x8192 both", "op": "quant", "rows": 8192, "cols": 8192, "src": "bf16", "way": "both"},
        # fp32 rows of odd length, blocks along the columns
        {"name": "quantize 1537x5001 cols", "op": "quant", "rows": 1537, "cols": 5001, "src": "f32", "way": "cols"},
        # serving: one token's activations against a quantised weight
        {"name": "matmul one token", "op": "matmul", "m": 1, "n": 11008, "k": 4096, "a": "bf16", "out": "bf16"},
        # a ragged batch of quantised rows, fp32 result
        {"name": "matmul 333x4099x2080", "op": "matmul", "m": 333, "n": 4099, "k": 2080, "a": "mx4", "out": "f32"},
        # a large product, both operands quantised before
        {"name": "matmul 8192x8192x4096", "op": "matmul", "m": 8192, "n": 8192, "k": 4096, "a": "mx4", "out": "bf16"},
        # training: forward and both gradients, a short ragged batch and a full one
        {"name": "linear 500x1024x768", "op": "linear", "tokens": 500, "n": 1024, "k": 768, "dtype": "f16"},
        {"name": "linear 4096x11008x4096", "op": "linear", "tokens": 4096, "n": 11008, "k": 4096, "dtype": "bf16"},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; odd ones as often as multiples of 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["ortho", "muon", "quant", "matmul", "linear"])
    if op in ("ortho", "muon"):
        rows, cols = _size(rng, 1, 5000), _size(rng, 1, 5000)
        room = max(1, (24 << 20) // (rows * cols))
        case = {"op": op, "count": _size(rng, 1, min(room, 48)), "rows": rows, "cols": cols}
        if op == "ortho":
            return {**case, "src": rng.choice(["f32", "f16", "bf16"]), "dst": rng.choice(["f16", "bf16"])}
        return {**case, "slot": rng.choice(["f16", "bf16"]), "lr": rng.choice([1e-4, 3e-4]),
                "wd": rng.choice([0.0, 0.01]), "nesterov": rng.random() < 0.5}
    if op == "quant":
        return {"op": op, "rows": _size(rng, 1, 8000), "cols": _size(rng, 1, 8000),
                "src": rng.choice(["f32", "f16", "bf16"]), "way": rng.choice(["rows", "cols", "both"])}
    if op == "matmul":
        a = rng.choice(["mx4", "bf16", "f16", "f32"])
        return {"op": op, "m": _size(rng, 1, 8000 if a == "mx4" else 64), "n": _size(rng, 1, 8000),
                "k": _size(rng, 1, 12000), "a": a, "out": rng.choice(["f32", "f16", "bf16"])}
    return {"op": op, "tokens": _size(rng, 1, 6000), "n": _size(rng, 16, 8000), "k": _size(rng, 16, 6000),
            "dtype": rng.choice(["f16", "bf16"])}


# ------------------------------------------------------------------------------------------------ inputs
def _gradient(gen, count, rows, cols, sigma):
    """Gradients of a matrix: a few strong directions over noise, columns of unlike scale."""
    r = max(1, min(rows, cols) // 16)
    u = torch.randn(count, rows, r, device="cuda", generator=gen)
    v = torch.randn(count, r, cols, device="cuda", generator=gen)
    g = torch.bmm(u, v).div_(math.sqrt(r))
    g.add_(torch.randn(count, rows, cols, device="cuda", generator=gen), alpha=0.3)
    g.mul_(torch.exp(0.5 * torch.randn(count, 1, cols, device="cuda", generator=gen)))
    return g.mul_(sigma)


def _activations(gen, rows, cols):
    """Activations: normal, with some columns of much larger values."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    return x.mul_(1.0 + 15.0 * (torch.rand(cols, device="cuda", generator=gen) < 0.01))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, state = case["op"], {"case": case}
    if op == "ortho":
        state["x"] = _gradient(gen, case["count"], case["rows"], case["cols"], 1e-3).to(DTYPES[case["src"]])
    elif op == "muon":
        shape = (case["count"], case["rows"], case["cols"])
        state["g"] = _gradient(gen, *shape, 1e-3)
        state["mom"] = _gradient(gen, *shape, 5e-4)
        state["master"] = torch.randn(shape, device="cuda", generator=gen).mul_(0.02)
        state["slot"] = state["master"].to(DTYPES[case["slot"]])
    elif op == "quant":
        state["x"] = _activations(gen, case["rows"], case["cols"]).to(DTYPES[case["src"]])
    elif op == "matmul":
        a = _activations(gen, case["m"], case["k"])
        b = torch.randn(case["n"], case["k"], device="cuda", generator=gen).mul_(0.02)
        state["b"] = _packed(b)
        state["a"] = _packed(a) if case["a"] == "mx4" else a.to(DTYPES[case["a"]])
    else:
        dt = DTYPES[case["dtype"]]
        state["x"] = _activations(gen, case["tokens"], case["k"]).to(dt).requires_grad_()
        state["w"] = torch.randn(case["n"], case["k"], device="cuda", generator=gen).mul_(0.02).to(dt).requires_grad_()
        state["dy"] = torch.randn(case["tokens"], case["n"], device="cuda", generator=gen).mul_(0.1).to(dt)
    return state


# ------------------------------------------------------------------------------------------------ plain forms
def _newton_schulz(x):
    """The iteration on a stack of matrices in the type of x."""
    a, b, c = COEFFS
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    x = (x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)).contiguous()
    for _ in range(NS_STEPS):
        s = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
    return x.transpose(1, 2).contiguous() if tall else x


MOMENTUM = 0.95


def _update_scale(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))


def _power_of_two(e):
    """2^e exactly, fp64, for a tensor of integers."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _mx4_parts(x):
    """(codes, exponents) of rows in blocks of 32, zero-filled to a multiple of 128 columns: codes 0..15 as
    integers [rows, padded], exponents [rows, padded / 32] with 2^(exponent - 127) the block's scale."""
    rows, cols = x.shape
    padded = -(-cols // 128) * 128
    x = torch.nn.functional.pad(x.float(), (0, padded - cols)).view(rows, padded // 32, 32)
    amax = x.abs().amax(2)
    power = ((amax.view(torch.int32) >> 23) - 127 - 2).clamp(-127, 127)  # floor(log2(amax)) - 2
    y = x.abs() * _power_of_two(-power).unsqueeze(2)  # 64 bits: exact next to the borders
    code = ((y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code += 8 * torch.signbit(x)
    return code.view(rows, padded), power + 127


def _packed(x):
    """MXFP4 rows as a program keeps them: {codes, scales, rows, cols}, the even element in the low four bits."""
    code, exponent = _mx4_parts(x)
    return {"codes": (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8), "scales": exponent.to(torch.uint8),
            "rows": x.shape[0], "cols": x.shape[1]}


def _values(code, exponent, cols):
    """The values that codes and exponents stand for, fp32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    v = table[code & 7] * (1 - 2 * (code >> 3))
    v = v.view(code.shape[0], -1, 32) * _power_of_two(exponent - 127).unsqueeze(2)
    return v.float().view(code.shape)[:, :cols]


def _rounded(x):
    """The MXFP4 values of rows, fp32."""
    return _values(*_mx4_parts(x), x.shape[1])


def _unpacked(q):
    c = q["codes"].int()
    return _values(torch.stack((c & 15, c >> 4), 2).view(c.shape[0], -1), q["scales"].int(), q["cols"])


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "ortho":
        return _newton_schulz(state["x"].float()).to(DTYPES[case["dst"]])
    if op == "muon":
        g, mom, master = state["g"], state["mom"], state["master"]
        mom.mul_(MOMENTUM).add_(g * (1 - MOMENTUM))
        u = g * (1 - MOMENTUM) + mom * MOMENTUM if case["nesterov"] else mom
        o = _newton_schulz(u) * (case["lr"] * _update_scale(case["rows"], case["cols"]))
        master.sub_(master * (case["lr"] * case["wd"])).sub_(o)
        state["slot"].copy_(master)
        return master, mom, state["slot"]
    if op == "quant":
        x = state["x"].float()
        out = [_rounded(x)] if case["way"] != "cols" else []
        if case["way"] != "rows":
            out.append(_rounded(x.t()))
        return [v.to(torch.bfloat16) for v in out]
    if op == "matmul":
        a = _unpacked(state["a"]) if case["a"] == "mx4" else _rounded(state["a"])
        return (a @ _unpacked(state["b"]).t()).to(DTYPES[case["out"]])
    x, w, dy = (state[k].detach().float() for k in ("x", "w", "dy"))
    dt = DTYPES[case["dtype"]]
    y = _rounded(x) @ _rounded(w).t()
    dx = _rounded(dy) @ _rounded(w.t()).t()
    dw = _rounded(dy.t()) @ _rounded(x.t()).t()
    return y.to(dt), dx.to(dt), dw.to(dt)


# ------------------------------------------------------------------------------------------------ the framework's calls
def _own(state):
    import zero_partitioned_mixed_amd as Z

    case = state["case"]
    op = case["op"]
    if op == "ortho":
        return Z.orthogonalize(state["x"], DTYPES[case["dst"]], coeffs=COEFFS, steps=NS_STEPS, eps=NS_EPS)
    if op == "muon":
        if "hp" not in state:
            state["hp"] = Z.muon_hparams(lr=case["lr"], momentum=MOMENTUM, weight_decay=case["wd"],
                                         nesterov=case["nesterov"], scale=Z.MUON_SCALE_RMS, coeffs=COEFFS,
                                         steps=NS_STEPS, eps=NS_EPS)
        Z.muon_step(state["master"], state["mom"], state["g"], state["hp"], slot=state["slot"])
        return state["master"], state["mom"], state["slot"]
    if op == "quant":
        way = case["way"]
        q = Z.mx4_quantize(state["x"], rows=way != "cols", cols=way != "rows")
        return [Z.mx4_dequantize(p, torch.bfloat16) for p in (q if way == "both" else (q,))]
    if op == "matmul":
        b = Z.MX4(**state["b"])
        a = Z.MX4(**state["a"]) if case["a"] == "mx4" else state["a"]
        return Z.mx4_matmul(a, b, DTYPES[case["out"]])
    y = Z.mx4_linear(state["x"], state["w"])
    dx, dw = torch.autograd.grad(y, (state["x"], state["w"]), state["dy"])
    return y.detach(), dx, dw


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _plain(state)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    op, size = case["op"], {"f32": 4, "f16": 2, "bf16": 2, "mx4": 0.53125}
    if op in ("ortho", "muon"):
        count, lo, hi = case["count"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # per step X X^T and A^2 are symmetric (half the products), M X is whole
        flops = count * NS_STEPS * (3.0 * lo * lo * hi + 1.0 * lo ** 3)
        per = size[case["src"]] + size[case["dst"]] if op == "ortho" else 4 * 3 + 4 * 2 + 2
        return {"bytes": per * count * lo * hi, "flops": flops}
    if op == "quant":
        n, ways = case["rows"] * case["cols"], 2 if case["way"] == "both" else 1
        return {"bytes": n * (size[case["src"]] + ways * (size["mx4"] + 2)), "flops": 0}
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * size[case["a"]] + n * k * size["mx4"] + m * n * size[case["out"]],
                "flops": 2.0 * m * n * k}
    t, n, k = case["tokens"], case["n"], case["k"]
    return {"bytes": 2 * 2 * (t * k + n * k) + 2 * 2 * t * n, "flops": 6.0 * t * n * k}


# ------------------------------------------------------------------------------------------------ 64 bits
def _polar_steps(g):
    """The iteration in 64 bits, one matrix at a time, on the side given: X (a I + b S + c S^2) with S = X^T X,
    or with S = X X^T from the left, whichever S is smaller."""
    a, b, c = COEFFS
    out = []
    for m in g.double():
        x = m / (torch.linalg.vector_norm(m) + NS_EPS)
        eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
        for _ in range(NS_STEPS):
            if x.shape[0] > x.shape[1]:
                s = x.t() @ x
                x = x @ (a * eye + s @ (b * eye + c * s))
            else:
                s = x @ x.t()
                x = (a * eye + s @ (b * eye + c * s)) @ x
        out.append(x)
    return torch.stack(out)


def _nearest(x):
    """MXFP4 values in 64 bits from the definition: the block's scale by its largest value's power of two, each
    value to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 times it, halfway cases to the even neighbour."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    rows, cols = x.shape
    full = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    full[:, :cols] = x.double()
    blocks = full.view(rows, -1, 32)
    top = blocks.abs().max(2, keepdim=True).values
    scale = top.clone().view(torch.int64).bitwise_and_(0x7FF << 52).view(torch.float64) / 4  # 2^floor(log2(top)) / 4
    scale = torch.where(top > 0, scale, torch.ones_like(top))
    t = (blocks.abs() / scale).clamp(max=6.0)
    hi = torch.searchsorted(grid, t.contiguous()).clamp(1, 7)
    below, above = t - grid[hi - 1], grid[hi] - t
    pick = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)
    v = torch.where(top > 0, grid[pick] * scale * torch.sign(blocks), torch.zeros_like(blocks))
    return v.view(rows, -1)[:, :cols]


def exact(case, seed):
    state, op = prepare(case, seed), case["op"]
    with torch.no_grad():
        if op == "ortho":
            return _polar_steps(state["x"])
        if op == "muon":
            g, mom, p = (state[k].double() for k in ("g", "mom", "master"))
            mom = MOMENTUM * mom + (1 - MOMENTUM) * g
            u = (1 - MOMENTUM) * g + MOMENTUM * mom if case["nesterov"] else mom
            p = p * (1 - case["lr"] * case["wd"]) - case["lr"] * _update_scale(case["rows"], case["cols"]) * _polar_steps(u)
            return p, mom, p
        if op == "quant":
            x = state["x"]
            return [_nearest(v) for v in ([x] if case["way"] != "cols" else []) + ([x.t()] if case["way"] != "rows" else [])]
        if op == "matmul":
            a = _unpacked(state["a"]).double() if case["a"] == "mx4" else _nearest(state["a"])
            return a @ _unpacked(state["b"]).double().t()
        x, w, dy = (state[k].detach() for k in ("x", "w", "dy"))
        return (_nearest(x) @ _nearest(w).t(), _nearest(dy) @ _nearest(w.t()).t(), _nearest(dy.t()) @ _nearest(x.t()).t())
