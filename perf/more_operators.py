"""The cases that the operators on rows of tokens are measured on, their plain forms and their 64-bit definitions.

The operators: the root-mean-square norm with the residual's addition, its gradients, and its output as MXFP8; the
product of MXFP8 rows with MXFP4 weights; dropout from a counter-based generator; the embedding lookup and its
gradient by sorted tokens; tokens sorted by expert and back, with weights and gradients.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "mx8": 1.03125, "mx4": 0.53125}
EPS = 1e-6


def listed():
    return [
        # serving, the latency end: one token's row on its way into a product with 4-bit weights
        {"name": "norm one token to 8 bits", "op": "norm", "way": "mx8", "tokens": 1, "cols": 4096, "dtype": "bf16", "residual": "same"},
        # a prompt's rows on the same way
        {"name": "norm 4000x8192 to 8 bits", "op": "norm", "way": "mx8", "tokens": 4000, "cols": 8192, "dtype": "bf16", "residual": "same"},
        # training: forward and gradients in the middle of a residual stream
        {"name": "norm train 8192x4096", "op": "norm", "way": "train", "tokens": 8192, "cols": 4096, "dtype": "bf16", "residual": "same"},
        # a ragged batch of odd rows, fp16 into an fp32 residual stream
        {"name": "norm train 1537x5001", "op": "norm", "way": "train", "tokens": 1537, "cols": 5001, "dtype": "f16", "residual": "f32"},
        # serving: one token's values against a quantised weight
        {"name": "product one token", "op": "product", "m": 1, "n": 11008, "k": 4096, "a": "bf16", "out": "bf16"},
        # a prompt's 8-bit rows against the same weight
        {"name": "product 4096x11008x4096", "op": "product", "m": 4096, "n": 11008, "k": 4096, "a": "mx8", "out": "bf16"},
        # training, a short batch of odd rows: forward and gradient
        {"name": "dropout 500x1001", "op": "dropout", "rows": 500, "cols": 1001, "dtype": "f16", "p": 0.1, "residual": False},
        # a full batch's hidden rows, added to the residual stream
        {"name": "dropout 16384x8192", "op": "dropout", "rows": 16384, "cols": 8192, "dtype": "bf16", "p": 0.1, "residual": True},
        # a GPT-2-sized table and one sequence
        {"name": "embedding 50257x768", "op": "embedding", "vocab": 50257, "cols": 768, "tokens": 1024, "dtype": "f16", "scale": 1.0, "ids": "i64"},
        # a large table and a full batch, scaled, with rows that are padding
        {"name": "embedding 131072x4096", "op": "embedding", "vocab": 131072, "cols": 4096, "tokens": 32768, "dtype": "bf16", "scale": 64.0, "ids": "i32"},
        # a short ragged batch, two experts a token, some of them dropped
        {"name": "experts 333 to 8", "op": "experts", "tokens": 333, "experts": 8, "k": 2, "cols": 1000, "dtype": "f16", "weights": "f32", "dropped": 0.05},
        # a full batch over many experts
        {"name": "experts 16384 to 64", "op": "experts", "tokens": 16384, "experts": 64, "k": 8, "cols": 4096, "dtype": "bf16", "weights": "f32", "dropped": 0.0},
    ]


def _size(rng, lo, hi):
    """A size between lo and hi, even over the logarithm; odd ones as often as multiples of 64."""
    hi = max(lo, hi)
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "product", "dropout", "embedding", "experts"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        cols = _size(rng, 1, 16000)
        return {"op": op, "way": rng.choice(["train", "mx8"]), "tokens": _size(rng, 1, min(20000, (1 << 25) // cols)),
                "cols": cols, "dtype": dtype, "residual": rng.choice(["none", "same", "f32"])}
    if op == "product":
        n, k = _size(rng, 1, 11000), _size(rng, 1, 11000)
        return {"op": op, "m": _size(rng, 1, min(8000, 4096 * 11008 * 4096 // (n * k))), "n": n, "k": k,
                "a": rng.choice(["mx8", "mx8", "f32", "f16", "bf16"]), "out": rng.choice(["f32", "f16", "bf16"])}
    if op == "dropout":
        cols = _size(rng, 1, 16000)
        return {"op": op, "rows": _size(rng, 1, min(20000, (1 << 26) // cols)), "cols": cols, "dtype": dtype,
                "p": rng.choice([0.05, 0.1, 0.3, 0.5]), "residual": rng.random() < 0.5}
    if op == "embedding":
        cols = _size(rng, 1, 8000)
        return {"op": op, "vocab": _size(rng, 1, min(150000, (1 << 28) // cols)), "cols": cols,
                "tokens": _size(rng, 1, min(65000, (1 << 26) // cols)), "dtype": dtype,
                "scale": rng.choice([1.0, 0.5, 12.3]), "ids": rng.choice(["i32", "i64"])}
    cols, experts = _size(rng, 1, 8000), _size(rng, 1, 256)
    k = rng.randint(1, min(8, experts))
    return {"op": op, "tokens": _size(rng, 1, min(16000, (1 << 28) // (cols * k))), "experts": experts, "k": k, "cols": cols,
            "dtype": dtype, "weights": rng.choice(["f32", dtype]), "dropped": rng.choice([0.0, 0.05, 0.5])}


# ------------------------------------------------------------------------------------------------ inputs
def _activations(gen, rows, cols):
    """Activations: normal, with some columns of much larger values."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    return x.mul_(1.0 + 15.0 * (torch.rand(cols, device="cuda", generator=gen) < 0.01))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, state = case["op"], {"case": case}

    def normal(*shape, scale=1.0, dtype=None):
        return torch.randn(*shape, device="cuda", generator=gen).mul_(scale).to(dtype or DTYPES[case["dtype"]])

    if op == "norm":
        t, c, dt = case["tokens"], case["cols"], DTYPES[case["dtype"]]
        stream = torch.float32 if case["residual"] == "f32" else dt
        train = case["way"] == "train"
        state["x"] = _activations(gen, t, c).to(dt).requires_grad_(train)
        state["w"] = normal(c, scale=0.2).add_(1.0).requires_grad_(train)
        state["residual"] = None
        if case["residual"] != "none":
            state["residual"] = (_activations(gen, t, c) * 4.0).to(stream).requires_grad_(train)
            state["dh"] = normal(t, c, scale=0.1, dtype=stream) if train else None
        state["dy"] = normal(t, c, scale=0.1) if train else None
    elif op == "product":
        a = _activations(gen, case["m"], case["k"])
        b = torch.randn(case["n"], case["k"], device="cuda", generator=gen).mul_(0.02)
        state["b"] = _packed4(b)
        state["a"] = _packed8(a) if case["a"] == "mx8" else a.to(DTYPES[case["a"]])
    elif op == "dropout":
        state["x"] = _activations(gen, case["rows"], case["cols"]).to(DTYPES[case["dtype"]]).requires_grad_()
        state["residual"] = normal(case["rows"], case["cols"], scale=4.0).requires_grad_() if case["residual"] else None
        state["dy"] = normal(case["rows"], case["cols"], scale=0.1)
        state["seed"], state["offset"] = 0x9E3779B97F4A7C15 ^ seed, 12345 + seed
    elif op == "embedding":
        state["table"] = normal(case["vocab"], case["cols"], scale=0.02).requires_grad_()
        # the frequencies of words: the n-th most frequent one about 1 / n as often as the first
        u = torch.rand(case["tokens"], device="cuda", generator=gen, dtype=torch.float64)
        ids = (torch.exp(u * math.log(case["vocab"] + 1.0)) - 1.0).long().clamp_(0, case["vocab"] - 1)
        ids[torch.rand(case["tokens"], device="cuda", generator=gen) < 0.02] = -1
        state["tokens"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
        state["dy"] = normal(case["tokens"], case["cols"], scale=0.1)
    else:
        t, e, k, c = case["tokens"], case["experts"], case["k"], case["cols"]
        # a router's logits with some experts liked more than others
        logits = torch.randn(t, e, device="cuda", generator=gen) + 0.5 * torch.randn(e, device="cuda", generator=gen)
        top, ids = torch.softmax(logits, 1).topk(k, 1)
        ids[torch.rand(t, k, device="cuda", generator=gen) < case["dropped"]] = -1
        state["ids"] = ids
        state["weights"] = (top / top.sum(1, keepdim=True)).to(DTYPES[case["weights"]]).requires_grad_()
        state["x"] = _activations(gen, t, c).to(DTYPES[case["dtype"]]).requires_grad_()
        state["z"] = normal(t * k, c).requires_grad_()  # what the experts made of the sorted rows
        state["dz"] = normal(t * k, c, scale=0.1)  # and the gradient that comes back from them
        state["dy"] = normal(t, c, scale=0.1)
    return state


# ------------------------------------------------------------------------------------------------ plain forms
def _power_of_two(e):
    """2^e exactly, fp64, for a tensor of integers."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _blocks(x):
    """Rows in blocks of 32, zero-filled to a multiple of 128 columns, fp32."""
    rows, cols = x.shape
    padded = -(-cols // 128) * 128
    return torch.nn.functional.pad(x.float(), (0, padded - cols)).view(rows, padded // 32, 32)


def _mx8_parts(x):
    """(codes, exponents) of rows in blocks of 32: codes as E4M3 numbers [rows, padded], 2^(exponent - 127) the
    block's scale, the smallest one that leaves its largest value at 448 or below."""
    x = _blocks(x)
    bits = x.abs().amax(2).view(torch.int32)
    power = (((bits + 0x1FFFFF) >> 23) - 127 - 8).clamp(-127, 127)
    y = (x.double() * _power_of_two(-power).unsqueeze(2)).float()  # exact: 64 bits hold the product
    return y.to(torch.float8_e4m3fn).view(x.shape[0], -1), power + 127


def _mx4_parts(x):
    """The same for MXFP4: codes 0..15 as integers."""
    x = _blocks(x)
    power = ((x.abs().amax(2).view(torch.int32) >> 23) - 127 - 2).clamp(-127, 127)  # floor(log2(amax)) - 2
    y = x.abs() * _power_of_two(-power).unsqueeze(2)  # 64 bits: exact next to the borders
    code = ((y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code += 8 * torch.signbit(x)
    return code.view(x.shape[0], -1), power + 127


def _packed8(x):
    """MXFP8 rows as a program keeps them."""
    code, exponent = _mx8_parts(x)
    return {"codes": code.view(torch.uint8), "scales": exponent.to(torch.uint8), "rows": x.shape[0], "cols": x.shape[1]}


def _packed4(x):
    """MXFP4 rows as a program keeps them: the even element in the low four bits."""
    code, exponent = _mx4_parts(x)
    return {"codes": (code[:, 0::2] | code[:, 1::2] << 4).to(torch.uint8), "scales": exponent.to(torch.uint8),
            "rows": x.shape[0], "cols": x.shape[1]}


def _scaled(values, scales, cols):
    v = values.view(values.shape[0], -1, 32) * _power_of_two(scales.int() - 127).unsqueeze(2)
    return v.float().view(values.shape)[:, :cols]


def _unpacked8(q):
    return _scaled(q["codes"].view(torch.float8_e4m3fn).float(), q["scales"], q["cols"])


def _unpacked4(q):
    c = q["codes"].int()
    code = torch.stack((c & 15, c >> 4), 2).view(c.shape[0], -1)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=code.device)
    return _scaled(table[code & 7] * (1 - 2 * (code >> 3)), q["scales"], q["cols"])


def _rounded8(x):
    """The MXFP8 values of rows, fp32."""
    code, exponent = _mx8_parts(x)
    return _scaled(code.float(), exponent, x.shape[1])


def _norm(state):
    x, w, r = state["x"], state["w"].float(), state["residual"]
    h = x if r is None else (x.float() + r.float()).to(r.dtype)  # the norm is that of the sum as it is kept
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1, keepdim=True) + EPS)
    unit = hf * rstd
    y = unit * w
    if state["case"]["way"] == "mx8":
        out = [_rounded8(y).to(torch.bfloat16)]
        return out if r is None else out + [h]
    dy = state["dy"].float()
    g = dy * w
    dh = (g - unit * (g * unit).mean(1, keepdim=True)) * rstd
    dw = (dy * unit).sum(0)
    if r is None:
        return y.to(x.dtype), dh.to(x.dtype), dw.to(x.dtype)
    dh = dh + state["dh"].float()
    return y.to(x.dtype), h, dh.to(x.dtype), dw.to(x.dtype), dh.to(r.dtype)


def _generator(counter, key):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; 2011) on int64
    tensors that hold 32-bit words."""
    low = 0xFFFFFFFF
    c0, c1, c2, c3 = counter
    k0, k1 = key & low, key >> 32 & low
    for _ in range(10):
        p, q = c0 * 0xD2511F53, c2 * 0xCD9E8D57  # modulo 2^64
        c0, c1, c2, c3 = (q >> 32 & low) ^ c1 ^ k0, q & low, (p >> 32 & low) ^ c3 ^ k1, p & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return c0, c1, c2, c3


def _kept(rows, cols, p, seed, offset):
    """Which elements stay: element c of row r takes 16 bits of the words at the counter (c / 8, r, offset)."""
    group = torch.arange(-(-cols // 8), device="cuda")
    row = torch.arange(rows, device="cuda").unsqueeze(1)
    group, row = torch.broadcast_tensors(group, row)
    offset = torch.full_like(row, offset)
    words = _generator((group, row, offset & 0xFFFFFFFF, offset >> 32), seed)
    halves = torch.stack([v for w in words for v in (w & 0xFFFF, w >> 16)], 2)
    return halves.view(rows, -1)[:, :cols] >= round(p * 65536)


def _dropout(state):
    case, x, r = state["case"], state["x"], state["residual"]
    limit = round(case["p"] * 65536)
    scale = 65536 / (65536 - limit)
    keep = _kept(case["rows"], case["cols"], case["p"], state["seed"], state["offset"])
    y = torch.where(keep, x.float() * scale, 0.0)
    dx = torch.where(keep, state["dy"].float() * scale, 0.0).to(x.dtype)
    if r is None:
        return y.to(x.dtype), dx
    return (y + r.float()).to(x.dtype), dx, state["dy"]


def _embedding(state):
    case, table, ids, dy = state["case"], state["table"], state["tokens"].long(), state["dy"]
    there = (ids >= 0) & (ids < case["vocab"])
    rows = table[ids.clamp(0, case["vocab"] - 1)].float() * case["scale"]
    y = torch.where(there.unsqueeze(1), rows, 0.0).to(table.dtype)
    grad = torch.zeros(case["vocab"] + 1, case["cols"], device="cuda")
    grad.index_add_(0, torch.where(there, ids, case["vocab"]), dy.float())
    return y, (grad[:-1] * case["scale"]).to(table.dtype)


def _expert_order(ids, experts):
    """(order, place, offsets): the slots sorted by expert, those of no expert last; where each slot went, -1 for
    none; where each expert's rows start."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order), device="cuda")
    place = torch.where(key < experts, place, -1)
    offsets = (key.unsqueeze(0) < torch.arange(experts + 1, device="cuda").unsqueeze(1)).sum(1)
    return order.int(), place.int().view(ids.shape), offsets.int()


def _experts(state):
    case = state["case"]
    t, k, c = case["tokens"], case["k"], case["cols"]
    x, z, w, dz, dy = (state[n].detach().float() for n in ("x", "z", "weights", "dz", "dy"))
    order, place, offsets = _expert_order(state["ids"], case["experts"])
    at, there = place.long().clamp(min=0), (place >= 0).unsqueeze(2)
    used = (torch.arange(t * k, device="cuda") < offsets[-1]).unsqueeze(1)
    rows = torch.where(used, x[order.long() // k], 0.0)
    mine = torch.where(there, z[at.view(-1)].view(t, k, c), 0.0)
    y = (mine * w.unsqueeze(2)).sum(1)
    dw = (mine * dy.unsqueeze(1)).sum(2)
    dback = torch.where(used, dy[order.long() // k] * w.reshape(-1)[order.long()].unsqueeze(1), 0.0)
    dx = torch.where(there, dz[at.view(-1)].view(t, k, c), 0.0).sum(1)
    dt = state["x"].dtype
    return order, offsets, rows.to(dt), y.to(dt), dback.to(dt), dw.to(state["weights"].dtype), dx.to(dt)


def _plain(state):
    case = state["case"]
    op = case["op"]
    if op == "product":
        a = _unpacked8(state["a"]) if case["a"] == "mx8" else _rounded8(state["a"])
        return (a @ _unpacked4(state["b"]).t()).to(DTYPES[case["out"]])
    return {"norm": _norm, "dropout": _dropout, "embedding": _embedding, "experts": _experts}[op](state)


# ------------------------------------------------------------------------------------------------ the framework's calls
def _own(state):
    import zero_partitioned_mixed_amd as Z

    case = state["case"]
    op = case["op"]
    grad = torch.autograd.grad
    if op == "norm":
        x, w, r = state["x"], state["w"], state["residual"]
        if case["way"] == "mx8":
            out = Z.rms_norm_mx8(x, w, r, eps=EPS)
            q, h = (out, []) if r is None else (out[0], [out[1]])
            return [Z.mx8_dequantize(q, torch.bfloat16)] + h
        if r is None:
            y = Z.rms_norm(x, w, eps=EPS)
            return (y.detach(), *grad(y, (x, w), state["dy"]))
        y, h = Z.rms_norm(x, w, r, eps=EPS)
        return (y.detach(), h.detach(), *grad((y, h), (x, w, r), (state["dy"], state["dh"])))
    if op == "product":
        a = Z.MX8(**state["a"]) if case["a"] == "mx8" else state["a"]
        return Z.mx8_matmul(a, Z.MX4(**state["b"]), DTYPES[case["out"]])
    if op == "dropout":
        x, r = state["x"], state["residual"]
        y = Z.dropout(x, case["p"], state["seed"], state["offset"], residual=r)
        return (y.detach(), *grad(y, (x,) if r is None else (x, r), state["dy"]))
    if op == "embedding":
        y = Z.embedding(state["tokens"], state["table"], scale=case["scale"])
        return (y.detach(), *grad(y, (state["table"],), state["dy"]))
    plan = Z.expert_sort(state["ids"], case["experts"])
    rows = Z.expert_rows(state["x"], plan)
    y = Z.expert_combine(state["z"], state["weights"], plan)
    dback, dw = grad(y, (state["z"], state["weights"]), state["dy"])
    dx, = grad(rows, (state["x"],), state["dz"])
    return plan.order, plan.offsets, rows.detach(), y.detach(), dback, dw, dx


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _plain(state)


# ------------------------------------------------------------------------------------------------ what a pass needs
def work(case):
    op, size = case["op"], SIZES
    if op == "norm":
        n, each = case["tokens"] * case["cols"], size[case["dtype"]]
        stream = {"none": 0, "same": each, "f32": 4}[case["residual"]]
        if case["way"] == "mx8":  # x and the residual in; the sum, codes and scales, and their values out
            return {"bytes": n * (each + 2 * stream + size["mx8"] + 2), "flops": 0}
        # forward: x, residual, sum, y; backward: dy, sum, its gradient, dx and the residual's where its type differs
        back = each + (stream or each) + stream + each + (stream if case["residual"] == "f32" and each != 4 else 0)
        return {"bytes": n * (2 * each + 2 * stream + back), "flops": 0}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k * size[case["a"]] + n * k * size["mx4"] + m * n * size[case["out"]], "flops": 2.0 * m * n * k}
    if op == "dropout":
        return {"bytes": case["rows"] * case["cols"] * size[case["dtype"]] * (4 + case["residual"]), "flops": 0}
    if op == "embedding":
        t, v, c, each = case["tokens"], case["vocab"], case["cols"], size[case["dtype"]]
        return {"bytes": 3 * t * c * each + v * c * each + t * (4 if case["ids"] == "i32" else 8), "flops": 0}
    t, k, c, each = case["tokens"], case["k"], case["cols"], size[case["dtype"]]
    # rows: x once, the rows; combine: the rows, y; its gradient: dy once, the rows, their gradients; dx: rows, dx
    return {"bytes": c * each * (t + t * k + t * k + t + t + 2 * t * k + t * k + t) + t * k * (8 + 2 * size[case["weights"]] + 8), "flops": 0}


# ------------------------------------------------------------------------------------------------ 64 bits
def _nearest8(x):
    """MXFP8 values in 64 bits from the definition: the smallest power of two that brings the block's largest value
    to 448 or below, each value to the nearest multiple of its step, halfway cases to the even one."""
    rows, cols = x.shape
    full = torch.zeros(rows, -(-cols // 32) * 32, dtype=torch.float64, device=x.device)
    full[:, :cols] = x.double()
    b = full.view(rows, -1, 32)
    top = b.abs().max(2, keepdim=True).values
    part, power = torch.frexp(torch.where(top > 0, top, 1.0))  # top = part 2^power, part in [.5, 1); 448 = .875 2^9
    power = power - 9 + (part > 0.875)
    scale = _power_of_two(power.clamp(min=-127))
    t = b / scale
    step = _power_of_two((torch.frexp(t).exponent - 1).clamp(min=-6) - 3)
    return (torch.round(t / step) * step * scale).view(rows, -1)[:, :cols]


def _nearest4(x):
    """MXFP4 values in 64 bits, as above from 0, .5, 1, 1.5, 2, 3, 4, 6 times the block's scale."""
    return _unpacked4(x).double()


def _mixed(counter, key):
    """Philox4x32-10 on numpy's unsigned 64-bit integers."""
    import numpy as np
    low, c = np.uint64(0xFFFFFFFF), [np.asarray(v, dtype=np.uint64) for v in counter]
    for i in range(10):
        k0, k1 = (np.uint64((k + i * w) & 0xFFFFFFFF) for k, w in ((key & 0xFFFFFFFF, 0x9E3779B9), (key >> 32, 0xBB67AE85)))
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ k0, b & low, (a >> np.uint64(32)) ^ c[3] ^ k1, a & low]
    return c


def _kept_exact(case, state):
    import numpy as np
    rows, cols = case["rows"], case["cols"]
    r, g = np.meshgrid(np.arange(rows), np.arange((cols + 7) // 8), indexing="ij")
    words = np.stack(_mixed((g, r, np.full_like(r, state["offset"] & 0xFFFFFFFF), np.full_like(r, state["offset"] >> 32)), state["seed"]), 2)
    halves = words.astype("<u4").reshape(rows, -1).view("<u2")[:, :cols]
    return torch.from_numpy(np.ascontiguousarray(halves.astype(np.int32))).cuda() >= round(case["p"] * 65536)


def exact(case, seed):
    op = case["op"]
    if op == "dropout" and case["rows"] * case["cols"] > 1 << 26:
        return None  # the generator on the host takes too long
    state = prepare(case, seed)
    with torch.no_grad():
        if op == "norm":
            x, w, r = state["x"], state["w"].double(), state["residual"]
            total = x.double() if r is None else x.double() + r.double()
            h = total.to(x.dtype if r is None else r.dtype).double()
            root = torch.sqrt((h * h).sum(1) / case["cols"] + EPS).unsqueeze(1)
            y = h / root * w
            more = [] if r is None else [total]
            if case["way"] == "mx8":
                return [_nearest8(y)] + more
            dy = state["dy"].double()
            g = dy * w
            dx = g / root - h * ((g * h).sum(1, keepdim=True) / case["cols"]) / root ** 3
            dw = (dy * h / root).sum(0)
            if r is not None:
                dx = dx + state["dh"].double()
            return [y] + more + [dx, dw] + ([] if r is None else [dx])
        if op == "product":
            a = _unpacked8(state["a"]).double() if case["a"] == "mx8" else _nearest8(state["a"])
            return a @ _nearest4(state["b"]).t()
        if op == "dropout":
            keep = _kept_exact(case, state).double()
            keep = keep * (65536 / (65536 - round(case["p"] * 65536)))
            y, dx = state["x"].double() * keep, state["dy"].double() * keep
            return (y, dx) if state["residual"] is None else (y + state["residual"].double(), dx, state["dy"].double())
        if op == "embedding":
            ids, table = state["tokens"].long(), state["table"].double()
            pad = (ids < 0) | (ids >= case["vocab"])
            y = table[ids.masked_fill(pad, 0)].mul_(case["scale"]).masked_fill_(pad.unsqueeze(1), 0.0)
            grad = torch.zeros_like(table)
            grad.index_add_(0, ids[~pad], state["dy"].double()[~pad])
            return y, grad.mul_(case["scale"])
        t, k, c = case["tokens"], case["k"], case["cols"]
        ids = state["ids"].reshape(-1).cpu().tolist()
        lists = [[] for _ in range(case["experts"] + 1)]
        for slot, e in enumerate(ids):
            lists[e if 0 <= e < case["experts"] else -1].append(slot)
        used = torch.tensor([s for part in lists[:-1] for s in part], dtype=torch.int64, device="cuda")
        token = used // k
        x, z, dz, dy = (state[n].double() for n in ("x", "z", "dz", "dy"))
        w = state["weights"].double().reshape(-1)
        rows, dback = torch.zeros_like(z), torch.zeros_like(z)
        n = len(used)
        rows[:n] = x[token]
        dback[:n] = dy[token] * w[used].unsqueeze(1)
        y, dx = torch.zeros_like(x), torch.zeros_like(x)
        y.index_add_(0, token, z[:n] * w[used].unsqueeze(1))
        dx.index_add_(0, token, dz[:n])
        dw = torch.zeros_like(w)
        for i in range(0, n, 1 << 16):
            dw[used[i:i + (1 << 16)]] = (z[i:min(n, i + (1 << 16))] * dy[token[i:i + (1 << 16)]]).sum(1)
        return None, None, rows, y, dback, dw.view(t, k), dx
