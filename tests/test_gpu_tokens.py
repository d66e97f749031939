"""The operators on rows of tokens on the GPU against plain computations in 64 bits: MXFP8
rows and their product with MXFP4 operands, the root-mean-square norm and its gradients,
dropout, the embedding lookup and its gradient, tokens sorted by expert and back.

Tolerances.  Codes, scales, masks, orders and copied rows are exact.  A sum of n terms in fp32
is off by at most d 2^-24 times the sum of their magnitudes, d the additions that a term goes
through; a result rounds once to its type, by at most half a step, or half of the smallest
number below the normal ones.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TYPES = [F32, F16, BF16]
U = 2.0 ** -24  # half a step of fp32
EPS = 1e-6


@pytest.fixture(scope="module")
def Z():
    import zero_partitioned_mixed_amd as Z
    return Z


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def last(dtype):
    """Half of the type's smallest number."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, dtype=F32, seed=0):
    return torch.randn(*shape, device="cuda", generator=gen(seed)).to(dtype)


def near(got, want, slack):
    """got (its type) against want (64 bits), beside the type's own rounding within slack (64 bits)."""
    err = (got.double() - want).abs()
    tol = slack + half_step(got.dtype) * (want.abs() + slack) + last(got.dtype)
    past = torch.isinf(got) & (got.double() * want > 0) & (want.abs() + slack >= torch.finfo(got.dtype).max)  # rounds to inf
    bad = ~((err <= tol) | past)
    assert not bad.any(), (int(bad.sum()), float(err[bad].max()), float((err / tol)[bad].max()))


def same(a, b):
    """Equal values, NaN in the same places."""
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(a.nan_to_num(0.0, math.inf, -math.inf), b.nan_to_num(0.0, math.inf, -math.inf))


def strided(x, extra=5, at=3):
    """x's values in rows of a wider buffer that start at an odd offset, and the buffer."""
    wide = torch.full((x.shape[0], x.shape[1] + extra), 7.0, dtype=x.dtype, device=x.device)
    wide[:, at:at + x.shape[1]] = x
    return wide[:, at:at + x.shape[1]], wide


# ----------------------------------------------------------------------------- MXFP8
def power(e):
    return torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e)  # on the CPU: exact


E4M3 = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
GRID = torch.sort(E4M3[:127]).values  # 0 .. 448


def mx8_reference(x):
    """(values in units of the scale, scale bytes) of the rows of x, on the CPU, by search over the codes in 64 bits."""
    x = x.double().cpu()
    rows, cols = x.shape
    p = -(-cols // 128) * 128
    full = torch.zeros(rows, p, dtype=torch.float64)
    full[:, :cols] = x
    blk = full.view(rows, p // 32, 32)
    bad = ~torch.isfinite(blk).all(2)
    blk = torch.where(bad.unsqueeze(2), 0.0, blk)
    top = blk.abs().amax(2)
    part, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (part > 0.875), -127).clamp(min=-127)
    t = (blk.abs() / power(e).unsqueeze(2)).contiguous()
    hi = torch.searchsorted(GRID, t).clamp(1, 126)
    below, above = t - GRID[hi - 1], GRID[hi] - t
    code = torch.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, hi - 1)
    code = torch.where(bad.unsqueeze(2), 0, code + 128 * torch.signbit(blk))
    return code.view(rows, p).to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def values8(q):
    """The matrix that an MX8 stands for, in 64 bits, on the CPU."""
    s = q.scales.cpu()
    scale = torch.where(s == 255, float("nan"), power(s.int() - 127))
    v = E4M3[q.codes.cpu().long()].view(q.rows, -1, 32) * scale.unsqueeze(2)
    return v.view(q.rows, -1)[:, :q.cols]


def values4(q):
    """The same of an MX4."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    c, s = q.codes.cpu(), q.scales.cpu()
    code = torch.stack((c & 15, c >> 4), 2).view(q.rows, -1)
    v = grid[(code & 7).long()] * torch.where(code >= 8, -1.0, 1.0)
    scale = torch.where(s == 255, float("nan"), power(s.int() - 127))
    return (v.view(q.rows, -1, 32) * scale.unsqueeze(2)).view(q.rows, -1)[:, :q.cols]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (3, 33), (5, 127), (7, 128), (2, 129), (65, 300), (130, 1001), (64, 4099)])
def test_mx8_quantize_exact(Z, rows, cols, dtype):
    x = (randn(rows, cols, seed=rows * 7 + cols) * torch.exp(3 * randn(rows, cols, seed=1))).to(dtype)
    for v in (x, strided(x)[0], x.t().contiguous().t()):
        q = Z.mx8_quantize(v)
        code, s = mx8_reference(v)
        assert torch.equal(q.scales.cpu(), s)
        assert torch.equal(q.codes.cpu(), code)
    for out in TYPES:
        same(Z.mx8_dequantize(q, out).cpu(), values8(q).to(out))


@pytest.mark.parametrize("dtype", TYPES)
def test_mx8_borders(Z, dtype):
    """Every halfway point between codes and its neighbours at several scales, both signs; largest values on both
    sides of 448 times a power of two; zeros, the type's smallest and largest numbers, infinities and NaN."""
    info = torch.finfo(dtype)
    mid = (GRID[1:] + GRID[:-1]) / 2
    near_ = torch.cat([mid, mid * (1 + info.eps), mid * (1 - info.eps / 2), GRID])
    rows = []
    for scale in (1.0, 2.0 ** -6, 2.0 ** 3):
        for sign in (1.0, -1.0):
            for part in (near_ * scale * sign).split(31):
                row = torch.zeros(32, dtype=torch.float64)
                row[:len(part)] = part
                row[31] = 448.0 * scale
                rows.append(row)
    tops = [1.75, 1.75 * (1 + info.eps), 1.75 * (1 - info.eps), 1.99, 1.0, 1.5]
    odd = [[t] + [t / 3] * 31 for t in tops] + [
        [0.0] * 32, [-0.0] * 32, [info.tiny] * 32, [info.smallest_normal / 4] * 32, [info.max] * 32, [-info.max] * 32,
        [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("nan")], [info.max] + [info.tiny] * 31]
    x = torch.cat([torch.stack(rows), torch.tensor(odd, dtype=torch.float64)]).to(dtype).cuda()
    q = Z.mx8_quantize(x)
    code, s = mx8_reference(x)
    assert torch.equal(q.scales.cpu(), s)
    assert torch.equal(q.codes.cpu(), code)


@pytest.mark.parametrize("dtype", TYPES)
def test_mx8_range(Z, dtype):
    """Every exponent of the type as a block's largest, its numbers below the normal ones among them."""
    info = torch.finfo(dtype)
    low, high = math.floor(math.log2(info.smallest_normal)) - (10 if dtype == F16 else 7), math.floor(math.log2(info.max))
    e = torch.arange(low, high, dtype=torch.float64).repeat_interleave(3)
    g = torch.Generator().manual_seed(4)
    x = torch.rand(len(e), 64, generator=g, dtype=torch.float64) + 0.5
    x = x * torch.pow(2.0, e[:, None] - torch.randint(0, 12, x.shape, generator=g)) * torch.sign(torch.randn(x.shape, generator=g))
    x = x.to(dtype).cuda()
    q = Z.mx8_quantize(x)
    code, s = mx8_reference(x)
    assert torch.equal(q.scales.cpu(), s)
    assert torch.equal(q.codes.cpu(), code)


def test_mx8_every_code_and_scale(Z):
    """All codes but NaN's under every scale byte: fp32 values equal 64 bits rounded once."""
    q = Z.MX8.alloc(256, 256, "cuda")
    q.codes.copy_(torch.arange(256, dtype=torch.int32).to(torch.uint8).cuda().expand(256, 256))
    q.scales.copy_(torch.arange(256, dtype=torch.int32).to(torch.uint8).cuda()[:, None].expand(256, 8))
    for dtype in TYPES:
        same(Z.mx8_dequantize(q, dtype).cpu(), values8(q).to(dtype))


def nominal(v, least, scale):
    """2^e of values v scale with codes v, e their exponents, not below `least`'s; of eight neighbours the largest."""
    e = power(torch.frexp(torch.maximum(v.abs(), torch.tensor(least))).exponent - 1) * scale
    p = -(-v.shape[1] // 8) * 8
    return torch.nn.functional.pad(e, (0, p - v.shape[1])).view(len(v), -1, 8).amax(2)


def scales_of(q):
    return power(q.scales.cpu().int() - 127).repeat_interleave(32, 1)[:, :q.cols]


def check_product(got, qa, qb, extra=None, rows=slice(None)):
    """fp32 results: sums in fp32.  16-bit ones: the matrix instruction also cuts what lies below 2^-13 of the largest
    of eight neighbouring products' exponents, seven of the eight by less than that."""
    a64, b64 = values8(qa)[rows], values4(qb)
    want, size = a64 @ b64.t(), a64.abs() @ b64.abs().t()
    slack = (qa.cols + 1) * U * size
    if extra is not None:
        want, slack = want + extra, slack + (qa.cols + 1) * U * extra.abs()
    if got.dtype != F32:
        sa, sb = scales_of(qa)[rows], scales_of(qb)
        slack = slack + 7 * 2.0 ** -13 * (nominal(a64 / sa, 2.0 ** -6, sa) @ nominal(b64 / sb, 1.0, sb).t())
    near(got.cpu(), want, slack)


PRODUCTS = [(1, 1, 1), (1, 1, 128), (2, 3, 129), (1, 300, 256), (17, 65, 300), (32, 33, 384), (33, 32, 128), (64, 64, 512),
            (65, 63, 640), (130, 200, 257), (300, 260, 1024), (257, 513, 384), (3, 4099, 2080), (333, 129, 96)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_mx8_product(Z, m, n, k):
    qa = Z.mx8_quantize(randn(m, k, seed=1) * torch.exp(2 * randn(m, k, seed=3)))
    qb = Z.mx4_quantize(randn(n, k, seed=2) * torch.exp(randn(n, k, seed=5)))
    for dtype in TYPES:
        check_product(Z.mx8_matmul(qa, qb, dtype), qa, qb)
    out, wide = strided(randn(m, n, seed=4), 3, 1)
    before = out.double().cpu()
    Z.mx8_matmul(qa, qb, out=out, accumulate=True)
    check_product(out, qa, qb, extra=before)
    assert (wide[:, :1] == 7).all() and (wide[:, n + 1:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 40, 128), (8, 70, 384), (32, 300, 512), (33, 70, 640), (300, 500, 1024), (3900, 4000, 384),
                                   (1286, 5928, 384), (4096, 4096, 512)])
def test_mx8_product_large_values_against_zeros(Z, m, n, k, dtype):
    """A column of large values that meets a weight of zero, as 4-bit weights have many, takes nothing from its
    neighbours: seven small products of eight, the smallest normal codes, the smallest below them, and ones."""
    a = torch.empty(m, k, device="cuda")
    b = torch.ones(n, k, device="cuda")
    b[:, ::8] = 0.0
    qb = Z.mx4_quantize(b)
    for small in (2.0 ** -6, 2.0 ** -9, 1.0):
        a.fill_(small)
        a[:, ::8] = 448.0
        want = float((k - -(-k // 8)) * small)
        assert float(torch.tensor(want).to(dtype)) == want  # seven eighths of k: few bits
        for x in (Z.mx8_quantize(a), a):
            assert (Z.mx8_matmul(x, qb, dtype) == want).all(), (small, want)


@pytest.mark.parametrize("m,n,k", PRODUCTS + [(4096, 4096, 512), (3900, 4000, 384), (1286, 5928, 384), (1000, 1100, 1024)])
def test_mx8_product_sums(Z, m, n, k):
    """Results of every type are fp32 sums, rounded once: rows with columns of much larger values, against 64 bits."""
    a = randn(m, k, seed=1) * (1 + 60 * (torch.rand(k, device="cuda", generator=gen(3)) < 0.05))
    qa, qb = Z.mx8_quantize(a), Z.mx4_quantize(randn(n, k, seed=2))
    rows = torch.arange(0, m, max(1, m // 61))
    a64, b64 = values8(qa)[rows], values4(qb)
    want, slack = a64 @ b64.t(), (k + 1) * U * (a64.abs() @ b64.abs().t())
    for dtype in TYPES:
        near(Z.mx8_matmul(qa, qb, dtype)[rows.cuda()].cpu(), want, slack)


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 512), (2048, 5000, 640), (1000, 1100, 384), (8192, 130, 256), (1286, 5928, 384),
                                   (657, 5969, 256), (657, 5395, 320), (400, 700, 4096),
                                   (3000, 4000, 1536), (1000, 1100, 1024), (300, 500, 2560), (1020, 4090, 512)])
def test_mx8_product_large_tiles(Z, m, n, k):
    """Sizes that take the larger tiles; a sample of rows in 64 bits."""
    qa, qb = Z.mx8_quantize(randn(m, k, seed=1)), Z.mx4_quantize(randn(n, k, seed=2))
    rows = torch.cat([torch.arange(0, m, max(1, m // 61)), torch.tensor([m - 1])])
    for dtype in TYPES:
        check_product(Z.mx8_matmul(qa, qb, dtype)[rows.cuda()], qa, qb, rows=rows)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("m", [1, 2, 7, 16, 32, 33, 64, 100])
def test_mx8_product_of_values(Z, m, dtype):
    for n, k in ((33, 100), (1000, 640), (300, 1700), (2000, 4096)):
        x = (randn(m, k, seed=m) * torch.exp(randn(m, k, seed=5))).to(dtype)
        qb = Z.mx4_quantize(randn(n, k, seed=6))
        for out in TYPES:
            check_product(Z.mx8_matmul(x, qb, out), Z.mx8_quantize(x), qb)
    wide = randn(m, 700, seed=9).to(dtype)
    qb = Z.mx4_quantize(randn(50, 129, seed=6))
    qa = Z.mx8_quantize(wide[:, 5:134])
    check_product(Z.mx8_matmul(wide[:, 5:134], qb, F32), qa, qb)
    out = randn(m, 50, seed=10)
    before = out.double().cpu()
    Z.mx8_matmul(wide[:, 5:134], qb, out=out, accumulate=True)
    check_product(out, qa, qb, extra=before)


@pytest.mark.parametrize("m,n,k", [(1, 40, 128), (20, 70, 384), (50, 70, 640), (300, 500, 1024)])
def test_mx8_product_range(Z, m, n, k):
    """Rows of every size against weights of the opposite one, the types' smallest and largest scales among them."""
    e = torch.linspace(-140, 119, m, device="cuda").round()[:, None]
    a = (randn(m, k, seed=1).double() * torch.pow(2.0, e.double())).float()
    for f in (-118.0, -60.0, 0.0, 60.0, 124.0):
        b = (randn(n, k, seed=2).double().clamp(-3, 3) * 2.0 ** f).float()
        qa, qb = Z.mx8_quantize(a), Z.mx4_quantize(b)
        a64, b64 = values8(qa), values4(qb)
        want = a64 @ b64.t()
        rows = (want.abs().amax(1) < 2.0 ** 120)
        # the smallest results: products and sums below the normal numbers, each off by half of the smallest one
        slack = (k + 1) * U * (a64.abs() @ b64.abs().t()) + 2 * k * last(F32)
        for x in (qa, a):
            got = Z.mx8_matmul(x, qb, F32).cpu()
            near(got[rows], want[rows], slack[rows])


def test_mx8_product_places(Z):
    """Every place of a block in k and every row meet their own scale: one element at a time against ones whose
    blocks' scales differ."""
    k = 512
    for m in (5, 70):
        b = torch.ones(40, k, device="cuda")
        b *= torch.pow(2.0, (torch.arange(k, device="cuda") // 32 % 7).float())[None] * torch.pow(2.0, (torch.arange(40, device="cuda") % 5).float())[:, None]
        qb = Z.mx4_quantize(b)
        a = torch.zeros(m, k, device="cuda")
        at = torch.arange(m, device="cuda") * 37 % k
        for shift in range(0, k, 11 if m == 5 else 29):
            a.zero_()
            a[torch.arange(m, device="cuda"), (at + shift) % k] = torch.pow(2.0, (torch.arange(m, device="cuda") % 9).float())
            assert torch.equal(Z.mx8_matmul(Z.mx8_quantize(a), qb, F32).double(), (a.double() @ b.double().t().contiguous()))


def test_mx8_product_nan_block_and_empty(Z):
    for m, n, k in ((20, 70, 256), (40, 70, 256), (300, 300, 1024)):
        a, b = randn(m, k), randn(n, k, seed=1)
        a[3, 40] = float("inf")
        b[5, k - 1] = float("nan")
        for x in (Z.mx8_quantize(a), a):
            c = Z.mx8_matmul(x, Z.mx4_quantize(b), F32)
            nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
            nan[3] = True
            nan[:, 5] = True
            assert torch.equal(torch.isnan(c), nan)
    for m in (1, 40, 300):
        assert (Z.mx8_matmul(Z.MX8.alloc(m, 0, "cuda"), Z.MX4.alloc(7, 0, "cuda"), F32) == 0).all()
        assert (Z.mx8_matmul(torch.empty(m, 0, device="cuda"), Z.MX4.alloc(7, 0, "cuda"), F32) == 0).all()
    assert Z.mx8_matmul(Z.MX8.alloc(0, 64, "cuda"), Z.mx4_quantize(randn(3, 64))).shape == (0, 3)


# ----------------------------------------------------------------------------- root-mean-square norm
def depth(cols):
    """Additions that a square goes through: eight at a time in a lane, then between lanes and waves, at most."""
    return 8 * max(4, math.ceil(cols / 8192)) + 6 + 16


def norm64(h, w, eps=EPS):
    root = torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h / root * w, root


def check_norm_gradients(h, w, dy, dh, dx, dr, dw, eps=EPS):
    """h and its type's gradient in 64 bits; dr and dx against it, dw."""
    tokens, cols = h.shape
    y, root = norm64(h, 1.0, eps)
    u, g = y, dy * w
    m, am = (g * u).mean(1, keepdim=True), (g * u).abs().mean(1, keepdim=True)
    want = (g - u * m) / root + (0.0 if dh is None else dh)
    # the mean of g u is off by its sum's depth, u and 1 / root by half of the squares' sum's, and a few roundings each
    slack = (2 * depth(cols) + 12) * U * (g.abs() + 2 * u.abs() * am) / root + 2 * U * want.abs()
    for got in (dx, dr):
        if got is not None:
            near(got, want, slack)
    if dw is not None:
        # rows of a group one after the other, at most 2048 groups in sixteen runs
        terms = dy * u
        near(dw, terms.sum(0), (math.ceil(tokens / 256) + 128 + 16 + depth(cols)) * U * terms.abs().sum(0))


NORM_SIZES = [(1, 1), (3, 7), (1, 8), (5, 100), (2, 1023), (4, 1024), (9, 1025), (3, 4096), (2, 4097), (7, 5001), (1, 8192),
              (3, 8193), (2, 16384), (2, 32768), (2, 32771), (1, 70001), (700, 96), (1300, 33)]


@pytest.mark.parametrize("stream", ["none", "same", "f32"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,cols", NORM_SIZES)
def test_norm_and_gradients(Z, tokens, cols, dtype, stream):
    x = (randn(tokens, cols, seed=1) * torch.exp(randn(tokens, 1, seed=2))).to(dtype).requires_grad_()
    w = (1 + 0.3 * randn(cols, seed=3)).to(dtype).requires_grad_()
    dy = randn(tokens, cols, seed=4).to(dtype)
    u = (depth(cols) / 2 + 8) * U
    if stream == "none":
        y = Z.rms_norm(x, w, eps=EPS)
        want, _ = norm64(x.double(), w.double())
        near(y.detach(), want.detach(), u * want.detach().abs())
        dx, dw = torch.autograd.grad(y, (x, w), dy)
        check_norm_gradients(x.detach().double(), w.detach().double(), dy.double(), None, dx, None, dw)
        return
    kind = dtype if stream == "same" else F32
    r = (2 * randn(tokens, cols, seed=5)).to(kind).requires_grad_()
    dh = randn(tokens, cols, seed=6).to(kind)
    y, h = Z.rms_norm(x, w, r, eps=EPS)
    assert torch.equal(h, (x.float() + r.float()).to(kind))
    want, _ = norm64(h.detach().double(), w.detach().double())
    near(y.detach(), want, u * want.abs())
    dx, dw, dr = torch.autograd.grad((y, h), (x, w, r), (dy, dh))
    assert dx.dtype == dtype and dr.dtype == kind and dw.dtype == dtype
    check_norm_gradients(h.detach().double(), w.detach().double(), dy.double(), dh.double(), dx, dr, dw)
    # the norm's result alone, one gradient at a time
    for leaf in (x, w, r):
        y, h = Z.rms_norm(x, w, r, eps=EPS)
        got, = torch.autograd.grad(y, leaf, dy)
        check_norm_gradients(h.detach().double(), w.detach().double(), dy.double(), None, got if leaf is x else None,
                             got if leaf is r else None, got if leaf is w else None)
    # the sum alone
    y, h = Z.rms_norm(x, w, r, eps=EPS)
    dx, dw, dr = torch.autograd.grad(h, (x, w, r), dh, allow_unused=True)
    assert torch.equal(dx, dh.to(dtype)) and torch.equal(dr, dh) and (dw is None or not dw.any())


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_strides(Z, dtype):
    tokens, cols = 11, 333
    x, r = randn(tokens, cols, dtype=dtype), randn(tokens, cols, seed=1, dtype=dtype)
    w, dy, dh = randn(cols, seed=2, dtype=dtype), randn(tokens, cols, seed=3, dtype=dtype), randn(tokens, cols, seed=4, dtype=dtype)

    def run(x, r, w, dy, dh):
        x, r, w = (t.detach().requires_grad_() for t in (x, r, w))
        y, h = Z.rms_norm(x, w, r)
        return (y.detach(), h.detach(), *torch.autograd.grad((y, h), (x, r, w), (dy, dh)))

    want = run(x, r, w, dy, dh)
    turned = lambda t: t.t().contiguous().t()  # noqa: E731
    for f in (lambda t: strided(t)[0], turned):
        got = run(f(x), f(r), torch.stack((w, w), 1)[:, 0], f(dy), f(dh))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    one = dy[:1].expand(tokens, cols)  # a broadcast gradient
    assert all(torch.equal(a, b) for a, b in zip(run(x, r, w, one, dh), run(x, r, w, one.contiguous(), dh)))


def test_norm_gradient_by_differences(Z):
    x, w, r = randn(3, 40, seed=1), 1 + 0.2 * randn(40, seed=2), randn(3, 40, seed=3)
    dy, dh = randn(3, 40, seed=4), randn(3, 40, seed=5)
    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    grads = torch.autograd.grad(Z.rms_norm(leaves[0], leaves[1], leaves[2]), leaves, (dy, dh))

    def f(x, w, r):
        h = x.double() + r.double()
        return float((norm64(h, w.double())[0] * dy + h * dh).sum())

    for i, (t, g) in enumerate(zip((x, w, r), grads)):
        step = randn(*t.shape, seed=9 + i).double()
        a, b = [v.double() for v in (x, w, r)], [v.double() for v in (x, w, r)]
        a[i], b[i] = a[i] + 1e-5 * step, b[i] - 1e-5 * step
        slope = (f(*a) - f(*b)) / 2e-5
        assert abs(slope - float((g.double() * step).sum())) < 1e-5 * float((g.double() * step).abs().sum())


@pytest.mark.parametrize("tokens,cols,groups", [(9000, 96, 2048), (5000, 1500, 1024), (2500, 3000, 512), (2500, 9000, 256), (300, 20000, 256)])
def test_norm_weight_gradient_sums(Z, tokens, cols, groups):
    """The weights' gradient against the additions that a term goes through: a group's rows one after the other, at most
    32 groups a run, 64 runs."""
    x, w, dy = randn(tokens, cols, seed=1), randn(cols, seed=2).requires_grad_(), randn(tokens, cols, seed=3)
    dw, = torch.autograd.grad(Z.rms_norm(x, w), w, dy)
    terms = dy.double() * norm64(x.double(), 1.0)[0]
    near(dw, terms.sum(0), (math.ceil(tokens / groups) + 32 + 64 + depth(cols)) * U * terms.abs().sum(0))


@pytest.mark.parametrize("cols", [40, 2000, 5000, 20000, 40000])
def test_norm_range(Z, cols):
    """Rows whose squares leave fp32's range or fall below it; zeros; infinities and NaN in one row alone."""
    base = randn(10, cols, seed=1)
    scale = torch.tensor([1e37, 1e30, 1e19, 1.0, 1e-18, 1e-24, 1e-30, 1.0, 1.0, 0.0], device="cuda")[:, None]
    for dtype in (F32, BF16):
        x = (base * scale).to(dtype)
        x[7, cols // 2], x[8, 3] = float("inf"), float("nan")
        w, dy = randn(cols, seed=2).to(dtype), randn(10, cols, seed=3).to(dtype)
        for eps in (1e-6, 1e-30, 0.0):
            leaf, lw = x.clone().requires_grad_(), w.clone().requires_grad_()
            y = Z.rms_norm(leaf, lw, eps=eps)
            dx, = torch.autograd.grad(y, leaf, dy)
            n = 7
            want, root = norm64(x[:n].double(), w.double(), float(torch.tensor(eps)))
            near(y.detach()[:n], want, (depth(cols) / 2 + 8) * U * want.abs())
            # beside rounding: products with 1 / root may fall below the normal numbers of fp32
            g = dy.double() * w.double()
            u, _ = norm64(x[:n].double(), 1.0, float(torch.tensor(eps)))
            slack = (2 * depth(cols) + 12) * U * (g[:n].abs() + 2 * u.abs() * (g[:n] * u).abs().mean(1, keepdim=True)) / root
            grad = (g[:n] - u * (g[:n] * u).mean(1, keepdim=True)) / root
            near(dx[:n].double().clamp(-3e38, 3e38).to(F32), grad.clamp(-3e38, 3e38), slack + 8 * 2.0 ** -126 + half_step(dtype) * grad.abs())
            assert torch.isnan(y[8]).all() and torch.isnan(y[7, cols // 2])
            rest = torch.ones(cols, dtype=torch.bool, device="cuda")
            rest[cols // 2] = False
            assert (y[7][rest] == 0).all()
            assert torch.isnan(y[9]).all() if eps == 0.0 else (y[9] == 0).all()


@pytest.mark.parametrize("cols", [40, 2000, 20000])
def test_norm_weights_range(Z, cols):
    """Weights whose products with the rows alone would leave fp32's range on either side; infinite ones and NaN."""
    x = randn(4, cols, seed=1) * torch.tensor([1e15, 1e-15, 1.0, 3e37], device="cuda")[:, None]
    x[:, 7] = 0.0
    w = torch.ones(cols, device="cuda")
    w[:5] = torch.tensor([1e30, 1e-30, 3e37, 1e-37, -1e33], device="cuda")
    w[5:9] = torch.tensor([math.inf, -math.inf, math.inf, math.nan], device="cuda")
    y = Z.rms_norm(x, w, eps=1e-36)
    want = norm64(x.double(), w.double(), float(torch.tensor(1e-36)))[0]
    fine = torch.isfinite(want)
    near(y[fine], want[fine], (depth(cols) / 2 + 8) * U * want[fine].abs())
    same(y[~fine], want[~fine].float())


@pytest.mark.parametrize("cols", [40, 2000, 5000, 20000, 40000])
def test_norm_smallest_rows(Z, cols):
    """Rows of numbers below the normal ones, without an eps: elements of about one, not infinities."""
    for dtype in (F32, BF16):
        least = float(2 * last(dtype))
        x = torch.randint(-3, 4, (6, cols), device="cuda", generator=gen(1)).double() * least
        x[1] *= 100.0
        x[2], x[3] = 0.0, 0.0
        x[2, cols // 2], x[3, cols - 1] = least, -2.0 * least
        x[4, 0] = 2.0 ** -60  # and beside a much larger one
        x[:, 1] = least
        x, w = x.to(dtype), randn(cols, seed=2).to(dtype)
        y = Z.rms_norm(x, w, eps=0.0)
        want = norm64(x.double(), w.double(), 0.0)[0]
        near(y, want, (depth(cols) / 2 + 8) * U * want.abs())


@pytest.mark.parametrize("cols", [40, 2000, 5000, 20000, 40000])
def test_norm_small_elements_of_large_rows(Z, cols):
    """Where a row's squares leave fp32's range, each of its elements still has all its bits."""
    x = randn(3, cols, seed=1) * torch.tensor([2.0 ** -45, 2.0 ** -30, 1.0], device="cuda")[:, None]
    x[:, 3] = torch.tensor([2.0 ** 66, 2.0 ** 90, -2.0 ** 127], device="cuda")
    w = randn(cols, seed=2)
    y = Z.rms_norm(x, w)
    want = norm64(x.double(), w.double())[0]
    # h / root is kept in two parts; the lower one of a result near the smallest numbers is itself below the normal ones:
    # rounded when it is made, by half of the smallest number, then times w, and so is their product
    near(y, want, (depth(cols) / 2 + 8) * U * want.abs() + (1 + w.double().abs()) * last(F32))


@pytest.mark.parametrize("stream", ["none", "f32"])
@pytest.mark.parametrize("cols", [40, 2000, 5000, 20000, 40000])
def test_norm_gradient_range(Z, cols, stream):
    """Gradients of rows and weights whose products, or sums of products, leave fp32's range on either side."""
    scale = torch.tensor([1e37, 1e30, 1e15, 1.0, 1e-15, 1e-30, 1e-40], device="cuda")[:, None]
    for dtype in (F32, BF16):
        kind = dtype if stream == "none" else F32
        h = (randn(7, cols, seed=1) * scale).to(kind)
        dy = randn(7, cols, seed=3).to(dtype)
        for weights in ([3e37, 1e30, 1e-30, 1e-37, -1e33], [1.0] * 5, [1e-37] * 5):
            w = randn(cols, seed=2) if weights[0] > 1e-3 else randn(cols, seed=2) * 1e-30
            w[:5] = torch.tensor(weights)
            w = w.to(dtype)
            for eps in (1e-6, 0.0):
                e64, lw = float(torch.tensor(eps)), w.clone().requires_grad_()
                if stream == "none":
                    leaf = h.clone().requires_grad_()
                    dx, dw = torch.autograd.grad(Z.rms_norm(leaf, lw, eps=eps), (leaf, lw), dy)
                    check_norm_gradients(h.double(), w.double(), dy.double(), None, dx, None, dw, eps=e64)
                    continue
                zero, leaf, dh = torch.zeros(7, cols, dtype=dtype, device="cuda").requires_grad_(), h.clone().requires_grad_(), randn(7, cols, seed=5)
                dx, dw, dr = torch.autograd.grad(Z.rms_norm(zero, lw, leaf, eps=eps), (zero, lw, leaf), (dy, dh))
                check_norm_gradients(h.double(), w.double(), dy.double(), dh.double(), dx, dr, dw, eps=e64)


@pytest.mark.parametrize("tokens,cols", [(9000, 96), (5000, 1500), (2500, 3000), (1500, 5000), (1500, 12000), (700, 20000)])
def test_norm_gradient_rows_of_all_sizes(Z, tokens, cols):
    """Ordinary rows and others among those of a group, of which there are several for each."""
    power = torch.randint(0, 5, (tokens, 1), device="cuda", generator=gen(4))
    scale = torch.tensor([1.0, 1.0, 1e30, 1e-30, 1e-12], device="cuda")[power]
    x, w, dy = randn(tokens, cols, seed=1) * scale, randn(cols, seed=2), randn(tokens, cols, seed=3)
    for eps in (1e-6, 0.0):
        leaf, lw = x.clone().requires_grad_(), w.clone().requires_grad_()
        dx, dw = torch.autograd.grad(Z.rms_norm(leaf, lw, eps=eps), (leaf, lw), dy)
        check_norm_gradients(x.double(), w.double(), dy.double(), None, dx, None, dw, eps=float(torch.tensor(eps)))
        again, = torch.autograd.grad(Z.rms_norm(leaf, lw, eps=eps), lw, dy)
        assert torch.equal(again, dw)


@pytest.mark.parametrize("cols", [40, 2000, 20000, 40000])
def test_norm_gradient_infinities(Z, cols):
    """Infinities and NaN in one row's gradient or values leave the other rows' gradients alone."""
    x, w, dy = randn(6, cols, seed=1), randn(cols, seed=2), randn(6, cols, seed=3)
    dy[1, 5], dy[2, cols - 1], x[4, 7] = math.inf, math.nan, -math.inf
    leaf, lw = x.clone().requires_grad_(), w.clone().requires_grad_()
    dx, dw = torch.autograd.grad(Z.rms_norm(leaf, lw), (leaf, lw), dy)
    fine = [0, 3, 5]
    check_norm_gradients(x.double()[fine], w.double(), dy.double()[fine], None, dx[fine], None, None)
    # (g - u m) / root with m infinite: NaN in the infinity's own place, infinities of -u's sign (times m's) elsewhere
    u = norm64(x[1:2].double(), 1.0)[0][0]
    want = -u * torch.sign(w[5].double() * u[5]) * math.inf
    want[5] = math.nan
    same(dx[1], want.float())
    assert torch.isnan(dx[2]).all() and torch.isnan(dx[4]).all()
    assert torch.isinf(dw[5]) and torch.isnan(dw[cols - 1]) and torch.isnan(dw[7])


@pytest.mark.parametrize("stream", ["none", "same", "f32"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,cols", [(1, 1), (3, 33), (2, 127), (5, 1024), (3, 1025), (1, 4096), (4, 5001), (2, 8191), (2, 9000),
                                         (1, 33000), (300, 200)])
def test_norm_mx8(Z, tokens, cols, dtype, stream):
    """Against the quantised 64-bit norm: the same scale but where the block's largest value is within fp32's error of a
    border, each value within half a step of its code."""
    x, w = randn(tokens, cols, seed=1).to(dtype), (1 + 0.3 * randn(cols, seed=2)).to(dtype)
    r = None if stream == "none" else randn(tokens, cols, seed=3).to(dtype if stream == "same" else F32)
    out = Z.rms_norm_mx8(x, w, r, eps=EPS)
    q, h = out if r is not None else (out, x)
    if r is not None:
        assert torch.equal(h, (x.float() + r.float()).to(r.dtype))
    want = norm64(h.double(), w.double())[0].cpu()
    u = (depth(cols) / 2 + 8) * U
    low, high = mx8_reference(want * (1 - u))[1], mx8_reference(want * (1 + u))[1]
    s = q.scales.cpu()
    assert ((s == low) | (s == high)).all()
    scale = power(s.int() - 127).repeat_interleave(32, 1)[:, :cols]
    step = torch.maximum(want.abs() * 2.0 ** -4, scale * 2.0 ** -10)
    assert ((values8(q) - want).abs() <= step * (1 + 2.0 ** -10) + 2 * u * want.abs()).all()
    pad = q.codes.cpu()[:, cols:]
    assert not pad.any() and not s[:, -(-cols // 32):].any()
    # and its product is that of its values
    qb = Z.mx4_quantize(randn(9, cols, seed=7))
    check_product(Z.mx8_matmul(q, qb, F32), q, qb)


# ----------------------------------------------------------------------------- dropout
def philox(counter, key):
    """Philox4x32-10 in numpy's 64-bit integers: four arrays of words."""
    low = np.uint64(0xFFFFFFFF)
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k = [key & 0xFFFFFFFF, key >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def kept(rows, cols, p, seed, offset):
    r, g = np.meshgrid(np.arange(rows), np.arange((cols + 7) // 8), indexing="ij")
    one = np.ones_like(r)
    w = np.stack(philox((g, r, one * (offset & 0xFFFFFFFF), one * (offset >> 32)), seed), 2).astype("<u4")
    return torch.from_numpy(w.reshape(rows, -1).view("<u2")[:, :cols].astype(np.int32)).cuda() >= round(p * 65536)


def test_generator_is_the_published_one():
    """The known answers of Philox4x32-10: counter and key zero, all ones, and digits of pi."""
    assert [int(v) for v in philox((0, 0, 0, 0), 0)] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert [int(v) for v in philox((0xFFFFFFFF,) * 4, 0xFFFFFFFFFFFFFFFF)] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    got = philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), 0x299F31D0A4093822)
    assert [int(v) for v in got] == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1,), (7,), (1, 8), (3, 33), (500, 1001), (2, 3, 40), (1000, 1), (1, 70000), (64, 4096)])
def test_dropout(Z, shape, dtype):
    x, r, dy = (randn(*shape, seed=s, dtype=dtype) for s in (1, 2, 3))
    rows, cols = (1, shape[0]) if len(shape) == 1 else (math.prod(shape[:-1]), shape[-1])
    for p, seed, offset in ((0.1, 1234567890123456789, 0), (0.5, 0xFFFFFFFFFFFFFFFF, 0x123456789ABCDEF), (0.0, 3, 1), (1.0, 3, 1),
                            (0.99999, 1, 2), (1e-9, 1, 2)):
        keep = kept(rows, cols, p, seed, offset).view(shape)
        limit = round(p * 65536)
        scale = 65536 / (65536 - limit) if limit < 65536 else 0.0
        want = torch.where(keep, x.double() * scale, 0.0)
        y = Z.dropout(x, p, seed, offset)
        near(y, want, 2 * U * want.abs())
        assert not y[~keep].any()
        lx, lr = x.clone().requires_grad_(), r.clone().requires_grad_()
        y = Z.dropout(lx, p, seed, offset, residual=lr)
        near(y.detach(), want + r.double(), 3 * U * (want.abs() + r.double().abs()))
        dx, dr = torch.autograd.grad(y, (lx, lr), dy)
        assert torch.equal(dr, dy) and torch.equal(dx, Z.dropout(dy, p, seed, offset))
    dev = torch.tensor([0x123456789ABCDEF], device="cuda")
    assert torch.equal(Z.dropout(x, 0.5, 5, dev), Z.dropout(x, 0.5, 5, 0x123456789ABCDEF))
    assert torch.equal(Z.dropout(x, 0.5, -1, -2), Z.dropout(x, 0.5, (1 << 64) - 1, (1 << 64) - 2))


def test_dropout_values_and_strides(Z):
    """Infinities and NaN in dropped places leave nothing; other layouts take the same mask."""
    x = randn(40, 77)
    keep = kept(40, 77, 0.5, 9, 8)
    x[~keep] = float("nan")
    x[0, ~keep[0]] = float("inf")
    y = Z.dropout(x, 0.5, 9, 8)
    assert torch.isfinite(y).all() and not y[~keep].any()
    for v in (strided(x)[0], x.t().contiguous().t(), torch.stack((x, x))[0]):
        assert torch.equal(Z.dropout(v, 0.5, 9, 8, residual=v.nan_to_num(0, 0)), Z.dropout(x, 0.5, 9, 8, residual=x.nan_to_num(0, 0)))
    # rows do not depend on how many there are
    assert torch.equal(Z.dropout(x[:10], 0.5, 9, 8), y[:10])
    share = float((Z.dropout(torch.ones(4096, 4096, device="cuda", dtype=BF16), 0.1, 42) == 0).float().mean())
    assert abs(share - 0.1) < 5 * math.sqrt(0.09) / 4096 + 1e-5  # five standard deviations, and p's own rounding
    a, b = (Z.dropout(torch.ones(1000, 1000, device="cuda"), 0.5, 42, i) != 0 for i in (0, 1))
    assert abs(float((a == b).float().mean()) - 0.5) < 5 * 0.5 / 1000


def test_dropout_offset_is_guarded(Z):
    """The offset tensor may not move between a forward pass and its backward pass."""
    x, offset = randn(4, 8).requires_grad_(), torch.zeros(1, dtype=torch.int64, device="cuda")
    y = Z.dropout(x, 0.5, 1, offset)
    offset.add_(1)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, x, torch.ones_like(y))


# ----------------------------------------------------------------------------- embedding
def ids_of(tokens, vocab, seed, dtype=torch.int64):
    """Ids of unlike frequency, some of them outside the table on either side."""
    u = torch.rand(tokens, device="cuda", generator=gen(seed), dtype=torch.float64)
    ids = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
    pick = torch.rand(tokens, device="cuda", generator=gen(seed + 1))
    ids[pick < 0.05] = -1
    ids[(pick >= 0.05) & (pick < 0.08)] = vocab
    ids[(pick >= 0.08) & (pick < 0.1)] = torch.iinfo(dtype).max
    ids[(pick >= 0.1) & (pick < 0.12)] = torch.iinfo(dtype).min
    return ids.to(dtype)


def check_embedding(Z, ids, table, scale, dy, got_y, got_d):
    vocab, cols = table.shape
    flat = ids.reshape(-1).long()
    there = (flat >= 0) & (flat < vocab)
    want = torch.where(there[:, None], table.double()[flat.clamp(0, vocab - 1)] * float(np.float32(scale)), 0.0)
    near(got_y.reshape(-1, cols), want, U * want.abs())
    sums, sizes = (torch.zeros(vocab + 1, cols, dtype=torch.float64, device="cuda") for _ in range(2))
    at, d = torch.where(there, flat, vocab), dy.reshape(-1, cols).double()
    sums.index_add_(0, at, d)
    sizes.index_add_(0, at, d.abs())
    many = int(torch.bincount(at[there], minlength=1).max()) if there.any() else 0
    near(got_d, sums[:-1] * scale, abs(scale) * (min(many, 128 + math.ceil(many / 128) + 2) + 2) * U * sizes[:-1])
    assert not got_d[sizes[:-1] == 0].any()


EMBED_SIZES = [(1, 1, 1), (5, 3, 8), (40, 100, 7), (300, 50, 33), (1000, 5000, 64), (129, 1, 16), (3000, 20, 40), (5000, 1000, 100),
               (2049, 131072, 9), (20000, 300, 130), (1, 50000, 300), (513, 511, 2500), (70, 512, 9000), (33, 2, 40000)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,vocab,cols", EMBED_SIZES)
def test_embedding_and_gradient(Z, tokens, vocab, cols, dtype):
    for idt, scale in ((torch.int64, 1.0), (torch.int32, 12.3)):
        ids = ids_of(tokens, vocab, tokens, idt)
        table, dy = randn(vocab, cols, seed=1, dtype=dtype).requires_grad_(), randn(tokens, cols, seed=2, dtype=dtype)
        y = Z.embedding(ids, table, scale=scale)
        d, = torch.autograd.grad(y, table, dy)
        check_embedding(Z, ids, table.detach(), scale, dy, y.detach(), d)
        again, = torch.autograd.grad(Z.embedding(ids, table, scale=scale), table, dy)
        assert torch.equal(d, again)


@pytest.mark.parametrize("runs", [[128], [129], [127, 129, 128], [256, 1, 300], [1, 127, 1, 255, 1], [1000], [3, 5000, 7], [130] * 9])
def test_embedding_runs(Z, runs):
    """Runs of equal ids that end before, at and past the places where long ones are cut; shuffled in the batch."""
    vocab, cols = len(runs) + 2, 72
    ids = torch.cat([torch.full((n,), i + 1) for i, n in enumerate(runs)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].cuda()
    table, dy = randn(vocab, cols).requires_grad_(), randn(len(ids), cols, seed=1)
    y = Z.embedding(ids, table)
    check_embedding(Z, ids, table.detach(), 1.0, dy, y.detach(), torch.autograd.grad(y, table, dy)[0])


def piece_of(n):
    """Tokens of the sorted order that are summed together: 8 to 32, more where there are more than 4096 pieces."""
    return -(-max(min(max(n // 1024, 8), 32), math.ceil(n / 4096)) // 8) * 8


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [3000, 17000, 25000, 33000, 140000, 270001])
def test_embedding_gradient_at_the_cuts(Z, n, dtype):
    """Runs that end one before, at and one past the cuts of the sorted order, within a piece, over exactly two and
    three, and over many, for pieces of 8, 16, 24, 32 and more; the bound from the additions that a term goes through."""
    piece, cols = piece_of(n), 40
    ends = sorted({piece * a + d for a in (1, 2, 3, 5, 8, 9, 20, 150) for d in (-1, 0, 1)} | {piece * 30 + piece // 2, piece * 32, n})
    runs = torch.tensor(ends).diff(prepend=torch.tensor([0]))
    ids = torch.repeat_interleave(torch.arange(1, len(ends) + 1), runs)
    ids = ids[torch.randperm(n, generator=torch.Generator().manual_seed(1))].cuda()
    table, dy = randn(len(ends) + 2, cols, dtype=dtype).requires_grad_(), randn(n, cols, seed=1, dtype=dtype)
    d, = torch.autograd.grad(Z.embedding(ids, table, scale=0.5), table, dy)
    sums, sizes = (torch.zeros(table.shape, dtype=torch.float64) for _ in range(2))
    sums.index_add_(0, ids.cpu(), dy.double().cpu())
    sizes.index_add_(0, ids.cpu(), dy.double().abs().cpu())
    many = torch.nn.functional.pad(runs, (1, 1)).double()
    # in a piece one after the other; of the pieces an eighth each, and eight of these
    adds = many.clamp(max=piece) + torch.where(many > piece, torch.ceil((many / piece + 2) / 8) + 8, 2.0) + 1
    near(d.cpu(), sums * 0.5, 0.5 * adds[:, None] * U * sizes)
    assert not d[0].any() and not d[-1].any()


def test_embedding_order_and_shapes(Z):
    """The sum is in the tokens' order: large terms that cancel leave what comes after them; ids of any shape; other
    layouts; no ids; all of them padding."""
    table = randn(10, 8).requires_grad_()
    dy = torch.zeros(6, 8, device="cuda")
    dy[0], dy[2], dy[4] = 2.0 ** 30, -2.0 ** 30, 1.0
    ids = torch.tensor([4, 1, 4, 2, 4, 1], device="cuda")
    d, = torch.autograd.grad(Z.embedding(ids, table), table, dy)
    assert (d[4] == 1.0).all()
    y = Z.embedding(ids.view(2, 3), table)
    assert y.shape == (2, 3, 8)
    assert torch.equal(torch.autograd.grad(y, table, dy.view(2, 3, 8))[0], d)
    wide, _ = strided(table.detach())
    leaf = wide.requires_grad_()
    y = Z.embedding(torch.stack((ids, ids), 1)[:, 0], leaf)
    assert torch.equal(y, table[ids]) and torch.equal(torch.autograd.grad(y, leaf, strided(dy)[0])[0], d)
    for none in (ids[:0], ids * 0 - 1, ids + 100):
        y = Z.embedding(none, table)
        assert not y.any() and y.shape == (len(none), 8)
        assert not torch.autograd.grad(y, table, dy[:len(none)])[0].any()
    nan = torch.full((6, 8), float("nan"), device="cuda")  # of padding: no part of any row
    assert not torch.autograd.grad(Z.embedding(ids * 0 - 1, table), table, nan)[0].any()


def test_embedding_many_tokens(Z):
    """More tokens than one workgroup sorts, ids of three passes, long runs; against a sum in 64 bits."""
    tokens, vocab, cols = 300_000, 1 << 19, 8
    ids = ids_of(tokens, vocab, 5)
    table, dy = randn(vocab, cols, seed=1, dtype=BF16).requires_grad_(), randn(tokens, cols, seed=2, dtype=BF16)
    y = Z.embedding(ids, table)
    check_embedding(Z, ids, table.detach(), 1.0, dy, y.detach(), torch.autograd.grad(y, table, dy)[0])


# ----------------------------------------------------------------------------- tokens by expert
def plan_reference(ids, experts):
    flat = ids.reshape(-1).long().cpu()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(len(order))
    offsets = torch.tensor([int((key < e).sum()) for e in range(experts + 1)])
    return order.int(), place.int().view(ids.shape), offsets.int()


def choices(tokens, k, experts, seed, drop=0.1, dtype=torch.int64):
    ids = torch.randint(0, experts, (tokens, k), device="cuda", generator=gen(seed))
    ids[torch.rand(tokens, k, device="cuda", generator=gen(seed + 1)) < drop] = -1
    ids[torch.rand(tokens, k, device="cuda", generator=gen(seed + 2)) < drop / 2] = experts
    return ids.to(dtype)


SORTS = [(1, 1, 1), (3, 2, 4), (100, 2, 8), (333, 3, 5), (2048, 1, 64), (2049, 1, 64), (1500, 8, 256), (5000, 4, 511), (700, 2, 512),
         (5000, 3, 1000), (40000, 8, 16), (9000, 2, 300000), (512, 1, 64), (513, 1, 600), (4096, 1, 64), (4097, 1, 600),
         (1365, 3, 700), (2000, 2, 300000)]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,k,experts", SORTS)
def test_expert_sort(Z, tokens, k, experts, dtype):
    for ids in (choices(tokens, k, experts, 1, dtype=dtype), choices(tokens, k, experts, 1, 0.0, dtype),
                torch.full((tokens, k), experts - 1, dtype=dtype, device="cuda"), torch.full((tokens, k), -5, dtype=dtype, device="cuda")):
        plan = Z.expert_sort(ids, experts)
        want = plan_reference(ids, experts) if experts < 10000 else None
        if want is None:
            key = torch.where((ids >= 0) & (ids < experts), ids, experts).reshape(-1).long()
            assert torch.equal(plan.offsets.long(), torch.searchsorted(key.sort().values, torch.arange(experts + 1, device="cuda")))
            order = torch.sort(key, stable=True).indices
            assert torch.equal(plan.order.long(), order)
            assert torch.equal(plan.place.view(-1)[order].long(), torch.arange(tokens * k, device="cuda"))
            continue
        for got, ref in zip((plan.order, plan.place, plan.offsets), want):
            assert got.dtype == torch.int32 and torch.equal(got.cpu(), ref)


EXPERTS = [(1, 1, 1, 1), (3, 2, 4, 7), (100, 2, 8, 33), (333, 3, 5, 1000), (64, 8, 40, 2048), (65, 9, 7, 2049), (20, 17, 30, 4100),
           (2000, 1, 100, 16)]


@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,k,experts,cols", EXPERTS)
def test_expert_rows_and_back(Z, tokens, k, experts, cols, dtype, drop):
    ids = choices(tokens, k, experts, 3, drop)
    if tokens > 2:
        ids[1] = -1  # a token without an expert
    plan = Z.expert_sort(ids, experts)
    order, place, offsets = plan_reference(ids, experts)
    used, slots = int(offsets[-1]), tokens * k
    order, place = order.long().cuda(), place.long().cuda()
    x, dz = randn(tokens, cols, seed=1, dtype=dtype).requires_grad_(), randn(slots, cols, seed=2, dtype=dtype)
    rows = Z.expert_rows(x, plan)
    want = x.detach()[order // k]
    want[used:] = 0
    assert torch.equal(rows, want)
    there = (place < used)[:, :, None]
    dz[used:] = float("nan")  # takes no part
    mine = torch.where(there, dz.double()[place.view(-1)].view(tokens, k, cols), 0.0)
    near(torch.autograd.grad(rows, x, dz)[0], mine.sum(1), k * U * mine.abs().sum(1))
    for wt in {dtype, F32}:
        z, w = randn(slots, cols, seed=4, dtype=dtype), torch.rand(tokens, k, device="cuda", generator=gen(5)).to(wt)
        z[used:] = float("nan")
        w[place >= used] = float("nan")
        z.requires_grad_()
        w.requires_grad_()
        dy = randn(tokens, cols, seed=6, dtype=dtype)
        y = Z.expert_combine(z, w, plan)
        z64, w64, dy64 = z.detach().double(), torch.where(place < used, w.detach().double(), 0.0), dy.double()
        mine = torch.where(there, z64[place.view(-1)].view(tokens, k, cols), 0.0)
        near(y.detach(), (mine * w64[:, :, None]).sum(1), (k + 1) * U * (mine * w64[:, :, None]).abs().sum(1))
        dzz, dw = torch.autograd.grad(y, (z, w), dy)
        want = dy64[order // k] * w64.view(-1)[order][:, None]
        want[used:] = 0
        near(dzz, want, U * want.abs())
        dots = mine * dy64[:, None]
        assert dw.dtype == wt
        near(dw, dots.sum(2), (cols / 64 + 12) * U * dots.abs().sum(2))
        # one gradient at a time
        assert torch.equal(torch.autograd.grad(Z.expert_combine(z, w.detach(), plan), z, dy)[0], dzz)
        assert torch.equal(torch.autograd.grad(Z.expert_combine(z.detach(), w, plan), w, dy)[0], dw)


@pytest.mark.parametrize("tokens,cols", [((1 << 23) + 5, 2056), (1 << 24, 1032)])
def test_expert_calls_on_many_tokens(Z, tokens, cols):
    """As many tokens as expert_rows takes, there, back and backward: more than one launch of a workgroup a token."""
    if torch.cuda.mem_get_info()[0] < 190 << 30:
        pytest.skip("needs 190 GB of free GPU memory")
    slots = torch.arange(tokens, device="cuda")
    x = (slots % 13).to(BF16)[:, None].expand(tokens, cols).contiguous().requires_grad_()
    plan = Z.expert_sort((slots % 3)[:, None], 3)
    rows = Z.expert_rows(x, plan)
    assert torch.equal(rows[:, 0].float(), (plan.order % 13).float())
    dx, = torch.autograd.grad(rows, x, rows.detach())
    assert torch.equal(dx, x)
    del dx
    rows, w = rows.detach().requires_grad_(), torch.ones(tokens, 1, device="cuda").requires_grad_()
    y = Z.expert_combine(rows, w, plan)
    assert torch.equal(y, x)
    drows, dw = torch.autograd.grad(y, (rows, w), x.detach())
    assert torch.equal(drows, rows)
    assert torch.equal(dw[:, 0], (slots % 13).float() ** 2 * cols)  # whole numbers below 2^24
    del x, rows, y, drows
    torch.cuda.empty_cache()


def test_expert_strides(Z):
    tokens, k, experts, cols = 50, 3, 6, 77
    plan = Z.expert_sort(choices(tokens, k, experts, 1).t().contiguous().t(), experts)
    x, z, w, dy = randn(tokens, cols), randn(tokens * k, cols, seed=1), torch.rand(tokens, k, device="cuda"), randn(tokens, cols, seed=2)

    def run(x, z, w, dy):
        x, z, w = (t.detach().requires_grad_() for t in (x, z, w))
        rows, y = Z.expert_rows(x, plan), Z.expert_combine(z, w, plan)
        return (rows.detach(), y.detach(), *torch.autograd.grad(y, (z, w), dy), *torch.autograd.grad(rows, x, z.detach()))

    want = run(x, z, w, dy)
    for f in (lambda t: strided(t)[0], lambda t: t.t().contiguous().t()):
        assert all(torch.equal(a, b) for a, b in zip(run(f(x), f(z), f(w), f(dy)), want))
    none = Z.expert_sort(torch.empty(0, 4, dtype=torch.int64, device="cuda"), 9)
    assert not none.offsets.any() and Z.expert_rows(x[:0], none).shape == (0, cols)
    assert Z.expert_combine(x[:0], torch.empty(0, 4, device="cuda"), none).shape == (0, cols)


# ----------------------------------------------------------------------------- together
def block(Z, ids, table, norm, up, down, router, seed, offset, mx8=False):
    """A small network's block as a program writes it: lookup, norm, a layer of experts, dropout into the stream."""
    h = Z.embedding(ids, table, scale=8.0)
    y, h = Z.rms_norm(h, norm, h)
    weights, chosen = torch.softmax(y.float() @ router, 1).topk(2, 1)
    plan = Z.expert_sort(chosen, len(up))
    rows = Z.expert_rows(y, plan)
    ends = plan.offsets.tolist()
    out = [Z.mx4_linear(torch.relu(Z.mx4_linear(rows[a:b], up[e])), down[e]) if b > a else rows[a:b]
           for e, (a, b) in enumerate(zip(ends, ends[1:]))] + [rows[ends[-1]:]]
    return Z.dropout(Z.expert_combine(torch.cat(out), weights, plan), 0.25, seed, offset, residual=h), plan


def test_a_block_of_them(Z):
    """Lookup, norm, experts and dropout in a row, forward and gradients, against the same steps in 64 bits with the
    products' operands as they were quantised; and the block's norm on the serving path."""
    vocab, cols, wide, experts, tokens = 90, 64, 96, 4, 50
    ids = ids_of(tokens, vocab, 3)
    make = lambda *s, seed, scale: (randn(*s, seed=seed) * scale).requires_grad_()  # noqa: E731
    table, norm = make(vocab, cols, seed=1, scale=0.1), (1 + 0.1 * randn(cols, seed=2)).requires_grad_()
    up = [make(wide, cols, seed=10 + e, scale=0.2) for e in range(experts)]
    down = [make(cols, wide, seed=20 + e, scale=0.2) for e in range(experts)]
    router = make(cols, experts, seed=3, scale=0.3)
    out, plan = block(Z, ids, table, norm, up, down, router, 77, 5)
    dy = randn(tokens, cols, seed=4)
    leaves = [table, norm, router, *up, *down]
    grads = torch.autograd.grad(out, leaves, dy)
    assert all(torch.isfinite(g).all() for g in grads)

    # forward in 64 bits
    flat = ids.clamp(0, vocab - 1)
    h = torch.where(((ids >= 0) & (ids < vocab))[:, None], table.double()[flat] * 8.0, 0.0)
    h = h + h
    y = norm64(h, norm.double())[0]
    weights, chosen = torch.softmax(y @ router.double(), 1).topk(2, 1)
    order, place, offsets = plan_reference(chosen, experts)
    assert torch.equal(plan.place.cpu(), place)
    rows = y[(order // 2).long().cuda()]
    q = lambda v: values4(Z.mx4_quantize(v.detach().float())).cuda()  # noqa: E731
    parts = [torch.relu(q(rows[a:b]) @ q(up[e]).t().contiguous()) for e, (a, b) in enumerate(zip(offsets, offsets[1:]))]
    parts = [q(v) @ q(down[e]).t().contiguous() if len(v) else rows[:0] for e, v in enumerate(parts)]
    mine = torch.cat(parts)[place.view(-1).long().cuda()].view(tokens, 2, cols)
    mixed = (mine * weights[:, :, None]).sum(1)
    want = torch.where(kept(tokens, cols, 0.25, 77, 5), mixed / 0.75, 0.0) + h
    # values next to a border of the 4-bit codes may take the neighbour: few, and each a step of one operand
    err = (out.detach().double() - want.detach()).norm() / want.detach().norm()
    assert float(err) < 0.02, float(err)
    # the serving path: the same norm as 8-bit rows against 4-bit weights
    with torch.no_grad():
        h = Z.embedding(ids, table, scale=8.0)
        rows8, _ = Z.rms_norm_mx8(h, norm, h)
        qb = Z.mx4_quantize(up[0])
        check_product(Z.mx8_matmul(rows8, qb, F32), rows8, qb)


def load_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "experts_mx8.py")
    spec = importlib.util.spec_from_file_location("experts_mx8", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_example_runs(Z):
    m = load_example()
    losses, p, ctrl = m.train(steps=3, ranks=2, width=128, tokens=100)
    assert ctrl["t"] == 3 and all(math.isfinite(v) for v in losses)
    ids, _ = m.batch(torch.Generator().manual_seed(1), 50)
    served = m.serve(p, ids)
    assert served.shape == (50, m.VOCAB) and torch.isfinite(served).all()


class Plain:
    """The calls that the example makes, from torch operations in the inputs' type, but for the products."""

    def __init__(self, Z):
        self.mx4_linear = Z.mx4_linear

    def embedding(self, ids, table):
        return table[ids]

    def rms_norm(self, x, w, r=None):
        h = x if r is None else x + r
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * w
        return y if r is None else (y, h)

    def dropout(self, x, p, seed, offset):
        return torch.where(kept(*x.shape, p, seed, offset), x * (65536 / (65536 - round(p * 65536))), 0.0)

    def expert_sort(self, chosen, experts):
        class Plan:
            pass
        plan = Plan()
        order, place, plan.offsets = plan_reference(chosen, experts)
        plan.order, plan.place = order.long().cuda(), place.long().cuda()
        return plan

    def expert_rows(self, x, plan):
        return x[plan.order // plan.place.shape[1]]

    def expert_combine(self, rows, weights, plan):
        return (rows[plan.place.view(-1)].view(*plan.place.shape, -1) * weights[:, :, None]).sum(1)


def test_example_gradients(Z):
    """The example's loss and gradients in fp32 against the same program on torch operations: equal but for fp32's
    rounding, and for 4-bit codes next to a border that it moves to the neighbour."""
    m = load_example()
    places, psi = m.layout(64)
    flat = randn(psi, seed=1) * 0.2
    m.views(flat, places)["norms"].fill_(1.0)
    ids, following = m.batch(torch.Generator().manual_seed(2), 80)
    got = []
    for calls in (Z, Plain(Z)):
        m.Z = calls
        leaf = flat.clone().requires_grad_()
        loss = torch.nn.functional.cross_entropy(m.forward(ids, m.views(leaf, places), 0.3, 5, 6), following)
        got.append((loss.detach(), torch.autograd.grad(loss, leaf)[0]))
    (loss, grad), (want_loss, want) = got
    assert abs(float(loss - want_loss)) <= 0.02 * float(want_loss)
    for name in places:
        a, b = m.views(grad, places)[name], m.views(want, places)[name]
        assert float((a - b).norm()) <= 0.02 * float(b.norm()) and float(b.norm()) > 0, name


def test_other_stream_and_graph(Z):
    """All calls on a side stream and in replayed graphs, with new values each time, equal the eager results."""
    tokens, cols, vocab, experts = 300, 200, 70, 5
    dtype = BF16
    x, r, w = randn(tokens, cols, dtype=dtype), randn(tokens, cols, seed=1, dtype=dtype), randn(cols, seed=2, dtype=dtype)
    table, dy = randn(vocab, cols, seed=3, dtype=dtype), randn(tokens, cols, seed=4, dtype=dtype)
    z, gates = randn(tokens * 2, cols, seed=5, dtype=dtype), torch.rand(tokens, 2, device="cuda", generator=gen(6))
    ids, chosen = ids_of(tokens, vocab, 7), choices(tokens, 2, experts, 8)
    offset = torch.zeros(1, dtype=torch.int64, device="cuda")
    qb = Z.mx4_quantize(randn(90, cols, seed=9))
    inputs = [x, r, w, table, dy, z, gates]

    def leaves():
        return [t.clone().requires_grad_() for t in (x, r, w, table, z, gates)]

    def work(x, r, w, table, z, gates):
        grad = torch.autograd.grad
        y, h = Z.rms_norm(x, w, r)
        got = [y, h, *grad((y, h), (x, w, r), (dy, dy))]
        d = Z.dropout(x, 0.3, 11, offset, residual=r)
        got += [d, *grad(d, (x, r), dy)]
        e = Z.embedding(ids, table)
        got += [e, *grad(e, table, dy)]
        plan = Z.expert_sort(chosen, experts)
        rows, c = Z.expert_rows(x, plan), Z.expert_combine(z, gates, plan)
        got += [plan.order, plan.place, plan.offsets, rows, c, *grad(c, (z, gates), dy), *grad(rows, x, z.detach())]
        with torch.no_grad():
            q = Z.rms_norm_mx8(x, w)
            got += [Z.mx8_dequantize(q), Z.mx8_matmul(q, qb), Z.mx8_matmul(x[:7], qb), Z.mx8_matmul(x, qb)]
        return [t.detach() for t in got]

    eager = work(*leaves())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = work(*leaves())
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    mine = leaves()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work(*mine)
    for i in range(4):
        with torch.no_grad():
            for j, t in enumerate(inputs):
                t.copy_(randn(*t.shape, seed=100 * i + j, dtype=t.dtype))
            for leaf, t in zip(mine, (x, r, w, table, z, gates)):
                leaf.copy_(t)
            ids.copy_(ids_of(tokens, vocab, 50 + i))
            chosen.copy_(choices(tokens, 2, experts, 60 + i))
            offset.fill_(i)
            for t in held:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(got, work(*leaves())))


def test_two_streams_at_once(Z):
    """Two streams with their own calls at the same time, as two layers' passes may be."""
    jobs = []
    for i in range(2):
        ids = ids_of(5000, 900, 20 + i)
        table, dy = randn(900, 300, seed=i).requires_grad_(), randn(5000, 300, seed=i + 5)
        chosen = choices(5000, 2, 40, 30 + i)
        jobs.append((ids, table, dy, chosen))

    def work(ids, table, dy, chosen):
        plan = Z.expert_sort(chosen, 40)
        return torch.autograd.grad(Z.embedding(ids, table), table, dy)[0], plan.order, Z.expert_rows(dy, plan)

    want = [work(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, j in zip(streams, jobs):
            with torch.cuda.stream(s):
                got.append(work(*j))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 2]))


CODES = {F16: 1, BF16: 2, F32: 3}


def c_call(Z, name, *args):
    """A C call on the current stream: tensors by their pointers."""
    args = [a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args]
    rc = getattr(Z._lib, name)(*args, torch.cuda.current_stream().cuda_stream)
    assert rc == 0, Z.zero_last_error()


def wide_like(x):
    """Room for x's values in rows of a wider buffer, which holds 7 everywhere."""
    return strided(torch.full_like(x, 7.0))


def gaps_untouched(wide, cols, at=3):
    assert (wide[:, :at] == 7).all() and (wide[:, at + cols:] == 7).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,cols", [(5, 3), (40, 77), (33, 1024), (7, 5001), (2, 20001)])
def test_strided_results_and_results_in_place(Z, tokens, cols, dtype):
    """Results in rows of wider buffers, whose gaps stay as they were; results in their inputs' place."""
    code, big = CODES[dtype], cols + 5
    x, r, w = randn(tokens, cols, seed=1, dtype=dtype), randn(tokens, cols, seed=2), randn(cols, seed=3, dtype=dtype)
    dy, dh = randn(tokens, cols, seed=4, dtype=dtype), randn(tokens, cols, seed=5)
    y, h = Z.rms_norm(x, w, r)
    eps = 1e-6
    (yw, yb), (hw, hb) = wide_like(x), wide_like(r)
    c_call(Z, "zero_rms_norm", x, code, cols, r, 3, cols, w, tokens, cols, eps, yw, big, hw, big)
    assert torch.equal(yw, y) and torch.equal(hw, h)
    gaps_untouched(yb, cols)
    gaps_untouched(hb, cols)
    xp, rp = x.clone(), r.clone()
    c_call(Z, "zero_rms_norm", xp, code, cols, rp, 3, cols, w, tokens, cols, eps, xp, cols, rp, cols)
    assert torch.equal(xp, y) and torch.equal(rp, h)
    rp = r.clone()
    q, qp = Z.rms_norm_mx8(x, w, r)[0], Z.MX8.alloc(tokens, cols, "cuda")
    c_call(Z, "zero_rms_norm_mx8", x, code, cols, rp, 3, cols, w, tokens, cols, eps, *qp._places, rp, cols)
    assert torch.equal(rp, h) and torch.equal(qp.codes, q.codes) and torch.equal(qp.scales, q.scales)

    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    dx, dw, dr = torch.autograd.grad(Z.rms_norm(*leaves), leaves, (dy, dh))
    (xw, xb), (rw, rb), dwp = wide_like(x), wide_like(r), torch.empty_like(w)
    size = Z._lib.zero_rms_norm_grad_workspace_bytes(tokens, cols)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    c_call(Z, "zero_rms_norm_grad", dy, cols, h, 3, cols, w, code, dh, cols, tokens, cols, eps, xw, big, rw, big, dwp, ws, size)
    assert torch.equal(xw, dx) and torch.equal(rw, dr) and torch.equal(dwp, dw)
    gaps_untouched(xb, cols)
    gaps_untouched(rb, cols)

    s = randn(tokens, cols, seed=6, dtype=dtype)
    want = Z.dropout(x, 0.3, 5, 6, residual=s)
    yw, yb = wide_like(x)
    c_call(Z, "zero_dropout", x, code, cols, s, cols, tokens, cols, 0.3, 5, 6, None, yw, big)
    assert torch.equal(yw, want)
    gaps_untouched(yb, cols)
    for place in (x.clone(), s.clone()):
        a, b = (place, s) if torch.equal(place, x) else (x, place)
        c_call(Z, "zero_dropout", a, code, cols, b, cols, tokens, cols, 0.3, 5, 6, None, place, cols)
        assert torch.equal(place, want)

    ids = torch.arange(tokens, device="cuda") * 3 % 7 - 1
    table = randn(6, cols, seed=7, dtype=dtype).requires_grad_()
    e = Z.embedding(ids, table, scale=3.0)
    de, = torch.autograd.grad(e, table, dy)
    (ew, eb), (gw, gb) = wide_like(x), wide_like(table.detach())
    c_call(Z, "zero_embedding", ids, 8, tokens, table.detach(), code, cols, 6, cols, 3.0, ew, big)
    size = Z._lib.zero_embedding_grad_workspace_bytes(tokens, 6, cols)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    c_call(Z, "zero_embedding_grad", ids, 8, tokens, dy, code, cols, 6, cols, 3.0, gw, big, ws, size)
    assert torch.equal(ew, e) and torch.equal(gw, de)
    gaps_untouched(eb, cols)
    gaps_untouched(gb, cols)

    plan = Z.expert_sort(choices(tokens, 2, 3, 8, 0.2), 3)
    used = plan.offsets.data_ptr() + 12
    rows = Z.expert_rows(x, plan)
    g = torch.rand(tokens, 2, device="cuda", generator=gen(9)).requires_grad_()
    z = randn(tokens * 2, cols, seed=10, dtype=dtype).requires_grad_()
    c = Z.expert_combine(z, g, plan)
    dz, dg = torch.autograd.grad(c, (z, g), dy)
    (rw, rb), (cw, cb), (zw, zb), dgp = wide_like(rows), wide_like(x), wide_like(rows), torch.empty_like(dg)
    c_call(Z, "zero_expert_rows", x, code, cols, plan.place, used, tokens, 2, cols, rw, big)
    c_call(Z, "zero_expert_combine", z.detach(), code, cols, plan.place, used, g.detach(), 3, tokens, 2, cols, cw, big)
    c_call(Z, "zero_expert_combine_grad", dy, cols, z.detach(), code, cols, plan.place, used, g.detach(), 3, tokens, 2, cols, zw, big, dgp)
    assert torch.equal(rw, rows) and torch.equal(cw, c) and torch.equal(zw, dz) and torch.equal(dgp, dg)
    for b in (rb, cb, zb):
        gaps_untouched(b, cols)


def test_expert_places_out_of_range(Z):
    """A plan whose memory holds anything: places outside the rows are left out, and no more rows are used than there are."""
    tokens, k, cols = 6, 2, 40
    place = torch.tensor([[0, -1], [1, 99], [2, -(1 << 31)], [3, (1 << 31) - 1], [4, 12], [5, 6]], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([0, (1 << 31) - 1], dtype=torch.int32, device="cuda")
    plan = Z.ExpertPlan(torch.zeros(12, dtype=torch.int32, device="cuda"), place, offsets, tokens, k, 1)
    x, z, w, dy = randn(tokens, cols), randn(12, cols, seed=1), torch.rand(tokens, k, device="cuda") + 0.5, randn(tokens, cols, seed=2)
    there = ((place >= 0) & (place < 12)).double()
    at = place.clamp(0, 11).long()
    want = (z.double()[at.view(-1)].view(tokens, k, cols) * (w.double() * there)[:, :, None]).sum(1)
    z.requires_grad_()
    w.requires_grad_()
    y = Z.expert_combine(z, w, plan)
    near(y.detach(), want, 4 * U * want.abs() + 4 * U)
    dw, = torch.autograd.grad(y, w, dy)
    assert not dw[there == 0].any() and dw[there == 1].all()
    c_rows = torch.full((12, cols), 7.0, device="cuda")
    c_call(Z, "zero_expert_rows", x, 3, cols, place, offsets.data_ptr() + 4, tokens, k, cols, c_rows, cols)
    assert torch.equal(c_rows[:6], x) and torch.equal(c_rows[6], x[5]) and (c_rows[7:] == 7).all()


def test_far_rows(Z):
    """Rows more than 2^31 elements apart."""
    far, rows, cols = (1 << 31) + 8, 3, 1001
    base = torch.empty((rows - 1) * far + cols, dtype=F16, device="cuda")
    x = base.as_strided((rows, cols), (far, 1))
    x.copy_(randn(rows, cols))
    near_x, w = x.contiguous(), randn(cols, seed=1, dtype=F16)
    dy = randn(rows, cols, seed=2, dtype=F16)

    def work(x):
        leaf = x.detach().requires_grad_()
        y = Z.rms_norm(leaf, w)
        ids = torch.tensor([2, 0, 2, 1], device="cuda")
        e = Z.embedding(ids, leaf)
        plan = Z.expert_sort(torch.tensor([[1], [0], [1]], device="cuda"), 2)
        gates = torch.ones(rows, 1, device="cuda").requires_grad_()
        c = Z.expert_combine(leaf, gates, plan)
        grad = torch.autograd.grad
        with torch.no_grad():
            q = Z.mx8_quantize(x)
            more = [q.codes, q.scales, Z.mx8_matmul(x, Z.mx4_quantize(x)), Z.expert_rows(x, plan)]
        return [y.detach(), grad(y, leaf, dy)[0], Z.dropout(x, 0.5, 1, residual=x), e.detach(), c.detach(), grad(c, gates, x)[0], *more]

    assert all(torch.equal(a, b) for a, b in zip(work(x), work(near_x)))


def test_without_gradients(Z):
    """Where torch records nothing, nothing is kept."""
    x, w = randn(4, 64).requires_grad_(), randn(64, seed=1)
    with torch.no_grad():
        assert not Z.rms_norm(x, w).requires_grad and not Z.dropout(x, 0.5, 1).requires_grad
        assert not Z.embedding(torch.tensor([1], device="cuda"), x).requires_grad
    assert not Z.rms_norm(x.detach(), w).requires_grad
    y = Z.dropout(x, 0.5, 1)
    d, = torch.autograd.grad(y, x, torch.ones_like(y), create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(d.sum(), x)


def test_empty(Z):
    x, w = torch.empty(0, 40, device="cuda").requires_grad_(), randn(40).requires_grad_()
    y, h = Z.rms_norm(x, w, x)
    dx, dw = torch.autograd.grad((y, h), (x, w), (y.detach(), h.detach()))
    assert dx.shape == (0, 40) and not dw.any()
    assert Z.rms_norm_mx8(x, w).rows == 0 and Z.dropout(x, 0.5, 1).shape == (0, 40)
    for shape in ((3, 0), (0,), (2, 3, 0), (0, 4, 5)):
        assert Z.dropout(torch.empty(shape, device="cuda"), 0.5, 1).shape == shape
    assert Z.mx8_quantize(x).rows == 0 and Z.mx8_dequantize(Z.MX8.alloc(3, 0, "cuda")).shape == (3, 0)


def test_refusals_of_tensors(Z):
    x, w = randn(8, 64), randn(64)
    b = Z.mx4_quantize(randn(4, 64))
    plan = Z.expert_sort(torch.zeros(8, 2, dtype=torch.int64, device="cuda"), 3)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    for error, call in [
            (TypeError, lambda: Z.mx8_quantize(x.double())), (ValueError, lambda: Z.mx8_quantize(x[0])),
            (ValueError, lambda: Z.mx8_matmul(x[:, :63], b)), (TypeError, lambda: Z.mx8_matmul(b, b)),
            (TypeError, lambda: Z.mx8_matmul(x, Z.mx8_quantize(x))), (ValueError, lambda: Z.mx8_matmul(x, b, accumulate=True)),
            (ValueError, lambda: Z.mx8_matmul(x, b, out=torch.empty(8, 5, device="cuda"))),
            (ValueError, lambda: Z.mx8_matmul(x.cpu(), b)), (TypeError, lambda: Z.mx8_matmul(x, b, torch.float64)),
            (ValueError, lambda: Z.rms_norm(x, w[:63])), (TypeError, lambda: Z.rms_norm(x, w.half())),
            (ValueError, lambda: Z.rms_norm(x, w, x[:7])), (TypeError, lambda: Z.rms_norm(x, w, x.half())),
            (ValueError, lambda: Z.rms_norm(x, w, eps=-1.0)), (ValueError, lambda: Z.rms_norm(x, w, eps=float("nan"))),
            (ValueError, lambda: Z.rms_norm(x.view(2, 4, 64), w)), (ValueError, lambda: Z.rms_norm(x, w.cpu())),
            (ValueError, lambda: Z.dropout(x, 1.1, 0)), (ValueError, lambda: Z.dropout(x, -0.1, 0)),
            (ValueError, lambda: Z.dropout(x, 0.1, 0, residual=x[:7])), (ValueError, lambda: Z.dropout(x, 0.1, 0, residual=x.half())),
            (ValueError, lambda: Z.dropout(x, 0.1, 0, torch.zeros(2, dtype=torch.int64, device="cuda"))),
            (ValueError, lambda: Z.dropout(x, 0.1, 0, torch.zeros(1, dtype=torch.int64))), (TypeError, lambda: Z.dropout(x.double(), 0.1, 0)),
            (TypeError, lambda: Z.embedding(x, x)), (ValueError, lambda: Z.embedding(ids, x[0])),
            (ValueError, lambda: Z.embedding(ids, x[:0])), (ValueError, lambda: Z.embedding(ids.cpu(), x)),
            (ValueError, lambda: Z.embedding(ids, x, scale=float("inf"))),
            (ValueError, lambda: Z.expert_sort(ids, 3)), (TypeError, lambda: Z.expert_sort(x, 3)),
            (ValueError, lambda: Z.expert_sort(plan.place, 0)), (ValueError, lambda: Z.expert_rows(x[:7], plan)),
            (ValueError, lambda: Z.expert_combine(x, torch.ones(8, 2, device="cuda"), plan)),
            (ValueError, lambda: Z.expert_combine(randn(16, 5), torch.ones(8, 3, device="cuda"), plan)),
            (TypeError, lambda: Z.expert_combine(randn(16, 5), torch.ones(8, 2, device="cuda").half(), plan))]:
        with pytest.raises(error):
            call()


def test_calls_without_gradients_refuse_them(Z):
    """Calls that are not differentiable and return a tensor say so instead of returning it without its graph."""
    import torch.autograd.forward_ad as forward_ad
    x, r, w, b = randn(4, 64), randn(4, 64, seed=1), randn(64, seed=2), Z.mx4_quantize(randn(8, 64))
    leaf = x.clone().requires_grad_()
    for call in (lambda t: Z.rms_norm_mx8(t, w, r), lambda t: Z.rms_norm_mx8(x, w, t), lambda t: Z.mx8_matmul(t, b)):
        with pytest.raises(RuntimeError, match="not differentiable"):
            call(leaf)
        with forward_ad.dual_level():
            with pytest.raises(RuntimeError, match="not differentiable"):
                call(forward_ad.make_dual(x, torch.ones_like(x)))
            call(x)
        with torch.no_grad():
            call(leaf)
        call(leaf.detach())
