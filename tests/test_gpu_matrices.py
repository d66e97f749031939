"""The matrix operators on the GPU against plain computations in 64 bits:
orthogonalised updates, the optimizer step built on them, MXFP4 quantisation,
its values, and products of MXFP4 operands.

Tolerances.  MXFP4 codes, scales and fp32 values are exact.  A product of
given operands sums k terms in fp32: each addition is off by at most 2^-24 of
the sum of magnitudes, and the result rounds once to its type.  The
orthogonalisation of large matrices rounds three operands a step to 11 bits;
with five steps and independent errors of at most 2^-12 root mean square each
that is sqrt(15) 2^-12 = 1e-3, doubled for the errors' growth between steps, and
4 x that where all elements round alike.  Where the smaller side is at most 128
the operands have 22 bits, and a thousandth of it holds plus what fp32 adds:
singular values far below the largest grow 500-fold over five steps, and a fp32
rounding (2^-24) of the largest with them.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
COEFFS = (3.4445, -4.7750, 2.0315)
NS_TOL = 2 * math.sqrt(15) * 2.0 ** -12


@pytest.fixture(scope="module")
def Z():
    import zero_partitioned_mixed_amd as Z
    return Z


def ns_tol(rows, cols):
    return NS_TOL if min(rows, cols) > 128 else NS_TOL / 1000 + 500 * 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ----------------------------------------------------------------------------- oracles
def ns64(x, steps=5, eps=1e-7, coeffs=COEFFS):
    a, b, c = coeffs
    x = x.double().cpu()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    norm = x.square().sum((-2, -1), keepdim=True).sqrt() + eps
    x = x / torch.where(norm > 0, norm, torch.ones_like(norm))
    for _ in range(steps):
        s = x @ x.mT
        x = a * x + (b * s + c * s @ s) @ x
    return x.mT if tall else x


def ns64_gpu(x):
    """ns64 of one matrix in 64 bits on the GPU, for sizes that take the CPU long."""
    a, b, c = COEFFS
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = (x.t() if tall else x).contiguous()
    x = x / (x.square().sum().sqrt() + 1e-7)
    for _ in range(5):
        s = torch.mm(x, x.t())
        x = a * x + torch.mm(b * s + c * torch.mm(s, s), x)
    return (x.t() if tall else x).cpu()


GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def mx4_reference(x):
    """(codes per element, scale bytes) of the rows of x, on the CPU, by search over the grid in 64 bits."""
    x = x.double().cpu()
    rows, cols = x.shape
    p = -(-cols // 128) * 128
    full = torch.zeros(rows, p, dtype=torch.float64)
    full[:, :cols] = x
    blk = full.view(rows, p // 32, 32)
    top = blk.abs().amax(2)
    bad = ~torch.isfinite(blk).all(2)
    e = torch.where((top > 0) & ~bad, torch.frexp(torch.where(bad, 1.0, top)).exponent - 1 - 2, -127)
    e = e.clamp(-127, 127)
    t = torch.where(bad.unsqueeze(2), 0.0, blk.abs() * torch.pow(2.0, -e.double()).unsqueeze(2)).clamp(max=6.0)
    d = (t.unsqueeze(-1) - GRID).abs()
    near = d == d.amin(-1, keepdim=True)
    # of two equally near codes the even one
    order = torch.tensor([0, 8, 1, 9, 2, 10, 3, 11])
    code = torch.where(near, order, 99).argmin(-1)
    code = code + 8 * torch.signbit(blk)
    code = torch.where(bad.unsqueeze(2), 0, code)
    return code.view(rows, p).to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def unpack(q):
    c = q.codes.cpu()
    return torch.stack((c & 15, c >> 4), 2).view(c.shape[0], -1)


def values64(q):
    """The matrix that an MX4 stands for, in 64 bits, on the CPU."""
    code, s = unpack(q), q.scales.cpu()
    v = GRID[(code & 7).long()] * torch.where(code >= 8, -1.0, 1.0)
    scale = torch.where(s == 255, float("nan"), torch.pow(2.0, s.double() - 127))
    v = v.view(code.shape[0], -1, 32) * scale.unsqueeze(2)
    return v.view(code.shape)[:, :q.cols]


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(*shape, dtype=F32, seed=0):
    return torch.randn(*shape, device="cuda", generator=gen(seed)).to(dtype)


# ----------------------------------------------------------------------------- MXFP4: quantisation
QUANT_SIZES = [(1, 1), (1, 31), (1, 32), (3, 33), (1, 4096), (5, 127), (7, 128), (2, 129), (33, 1), (128, 128),
               (129, 257), (257, 129), (300, 500), (64, 4099)]


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", QUANT_SIZES)
def test_quantize_exact(Z, rows, cols, dtype):
    x = randn(rows, cols, seed=rows * 7 + cols)
    x = (x * torch.exp(2 * randn(rows, cols, seed=1))).to(dtype)
    r = Z.mx4_quantize(x)
    both = Z.mx4_quantize(x, cols=True)
    c = Z.mx4_quantize(x, rows=False, cols=True)
    for q, want in ((r, x), (both[0], x), (c, x.t()), (both[1], x.t())):
        code, s = mx4_reference(want)
        assert torch.equal(unpack(q), code)
        assert torch.equal(q.scales.cpu(), s)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_quantize_large(Z, dtype):
    """A matrix of many patches, in both directions; a sample of rows and columns."""
    rows, cols = 2900, 3001
    x = (randn(rows, cols, seed=8) * torch.exp(randn(rows, 1, seed=9))).to(dtype)
    r, c = Z.mx4_quantize(x, cols=True)
    for q, want, n in ((r, x, rows), (c, x.t(), cols)):
        pick = torch.cat([torch.arange(0, n, 97), torch.arange(n - 3, n)])
        code, s = mx4_reference(want[pick.cuda()])
        part = Z.MX4(q.codes[pick.cuda()], q.scales[pick.cuda()], len(pick), q.cols)
        assert torch.equal(unpack(part), code) and torch.equal(part.scales.cpu(), s)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_quantize_borders(Z, dtype):
    """Every halfway point and its neighbours, both signs, at several scales; zeros, the smallest and the largest
    numbers of the type, infinities and NaN."""
    info = torch.finfo(dtype)
    mid = torch.tensor([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 6.5, 7.0, 7.9])
    near = torch.cat([mid, mid * (1 + info.eps), mid * (1 - info.eps / 2)])
    rows = []
    for scale in (1.0, 2.0 ** -9, 2.0 ** 9):
        for sign in (1.0, -1.0):
            v = near * scale * sign
            for i in range(0, len(v), 31):
                row = torch.zeros(32)
                part = v[i:i + 31]
                row[:len(part)] = part
                row[31] = 4.0 * scale  # fixes the block's scale
                rows.append(row)
    odd = [[0.0] * 32, [-0.0] * 32, [info.tiny] * 32, [info.smallest_normal / 4] * 32, [info.max] * 32, [-info.max] * 32,
           [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("nan")], [1.0] * 16 + [-float("inf")] + [2.0] * 15,
           [info.max] + [info.tiny] * 31, [7.999] * 32]
    x = torch.cat([torch.stack(rows), torch.tensor(odd)]).to(dtype).cuda()
    for q, want in ((Z.mx4_quantize(x), x), (Z.mx4_quantize(x.t().contiguous(), rows=False, cols=True), x)):
        code, s = mx4_reference(want)
        assert torch.equal(q.scales.cpu(), s)
        assert torch.equal(unpack(q), code)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_quantize_range(Z, dtype):
    """Random values over the whole range of the type, its numbers below the normal ones among them: every exponent
    as a block's largest, spread below it."""
    info = torch.finfo(dtype)
    low, high = math.floor(math.log2(info.smallest_normal)) - (10 if dtype == F16 else 7), math.floor(math.log2(info.max))
    e = torch.arange(low, high, dtype=torch.float64).repeat_interleave(3)
    g = torch.Generator().manual_seed(4)
    x = torch.rand(len(e), 64, generator=g, dtype=torch.float64) + 0.5
    x = x * torch.pow(2.0, e[:, None] - torch.randint(0, 5, x.shape, generator=g)) * torch.sign(torch.randn(x.shape, generator=g))
    x = x.to(dtype).cuda()
    q, t = Z.mx4_quantize(x, cols=True)
    for got, want in ((q, x), (t, x.t()), (Z.mx4_quantize(x.t().contiguous(), rows=False, cols=True), x)):
        code, s = mx4_reference(want)
        assert torch.equal(got.scales.cpu(), s)
        assert torch.equal(unpack(got), code)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_quantize_strides(Z, dtype):
    """Rows of a wider buffer, at an odd offset too; a transposed view."""
    base = randn(40, 517, dtype=dtype)
    for x in (base[:, 3:200], base[5:, 8:136], base.t(), base[::2]):
        code, s = mx4_reference(x)
        q, t = Z.mx4_quantize(x, cols=True)
        assert torch.equal(unpack(q), code) and torch.equal(q.scales.cpu(), s)
        code, s = mx4_reference(x.t())
        assert torch.equal(unpack(t), code) and torch.equal(t.scales.cpu(), s)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 33), (5, 128), (65, 300)])
def test_dequantize(Z, rows, cols, dtype):
    x = randn(rows, cols) * torch.exp(3 * randn(rows, 1, seed=2))
    q = Z.mx4_quantize(x)
    want = values64(q)
    got = Z.mx4_dequantize(q, dtype).cpu()
    assert torch.equal(got, want.to(dtype))
    wide = torch.full((rows, cols + 5), 7.0, dtype=dtype, device="cuda")
    Z.mx4_dequantize(q, out=wide[:, 2:cols + 2])
    assert torch.equal(wide[:, 2:cols + 2].cpu(), want.to(dtype))
    assert (wide[:, :2] == 7).all() and (wide[:, cols + 2:] == 7).all()


def test_every_code_and_scale(Z):
    """All 16 codes under every scale byte, as bytes that a receiver gets: fp32 values equal 64 bits rounded once."""
    q = Z.MX4.alloc(256, 32, "cuda")
    q.codes.zero_()
    q.codes[:, :16] = torch.arange(256, dtype=torch.int32).view(16, 16)[:, :].sum(1).remainder(256).to(torch.uint8).cuda()
    q.codes[:, :8] = torch.tensor([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE], dtype=torch.uint8, device="cuda")
    q.scales.zero_()
    q.scales[:, 0] = torch.arange(256, dtype=torch.int32).to(torch.uint8).cuda()
    for dtype in (F32, F16, BF16):
        want = values64(q).to(dtype)
        got = Z.mx4_dequantize(q, dtype).cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)])


# ----------------------------------------------------------------------------- MXFP4: products
def check_product(got, a64, b64, k, extra=None):
    want = a64 @ b64.t()
    size = a64.abs() @ b64.abs().t()
    if extra is not None:
        want, size = want + extra, size + extra.abs()
    tol = (k + 1) * 2.0 ** -24 * size + half_step(got.dtype) * want.abs() + torch.finfo(got.dtype).smallest_normal
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err - tol).max())


PRODUCTS = [(1, 1, 1), (1, 1, 128), (2, 3, 129), (1, 300, 256), (17, 65, 300), (64, 64, 512), (65, 63, 640), (130, 200, 257),
            (300, 260, 1024), (257, 513, 384), (3, 4099, 2080), (333, 129, 96)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(Z, m, n, k):
    a, b = randn(m, k, seed=1), randn(n, k, seed=2)
    a = a * torch.exp(randn(m, k, seed=3))
    qa, qb = Z.mx4_quantize(a), Z.mx4_quantize(b)
    a64, b64 = values64(qa), values64(qb)
    for dtype in (F32, F16, BF16):
        check_product(Z.mx4_matmul(qa, qb, dtype), a64, b64, k)
    base = randn(m, n + 3, seed=4)
    out = base[:, 1:n + 1]
    before = out.double().cpu()
    Z.mx4_matmul(qa, qb, out=out, accumulate=True)
    check_product(out, a64, b64, k, extra=before)


@pytest.mark.parametrize("m,n,k", [(4096, 4096, 512), (2048, 5000, 640), (1000, 1100, 384), (8192, 130, 256), (1286, 5928, 384),
                                   (657, 5969, 256), (657, 5395, 320)])
def test_product_large_tiles(Z, m, n, k):
    """Sizes that take the larger tiles; a sample of rows in 64 bits."""
    qa, qb = Z.mx4_quantize(randn(m, k, seed=1)), Z.mx4_quantize(randn(n, k, seed=2))
    rows = torch.cat([torch.arange(0, m, max(1, m // 61)), torch.tensor([m - 1])])
    b64, a64 = values64(qb), values64(qa)[rows]
    for dtype in (F32, BF16, F16):
        check_product(Z.mx4_matmul(qa, qb, dtype)[rows.cuda()], a64, b64, k)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("m", [1, 2, 7, 16, 33, 64, 65])
def test_product_of_values(Z, m, dtype):
    """Rows given as values equal their own quantisation's product, bit for bit up to the order of the sums."""
    for n, k in ((33, 100), (1000, 640), (4096, 4096)):
        x = (randn(m, k, seed=m) * torch.exp(randn(m, k, seed=5))).to(dtype)
        qb = Z.mx4_quantize(randn(n, k, seed=6))
        a64 = values64(Z.mx4_quantize(x))
        for out in (F32, BF16, F16):
            check_product(Z.mx4_matmul(x, qb, out), a64, values64(qb), k)
    wide = randn(m, 700, seed=9).to(dtype)
    qb = Z.mx4_quantize(randn(50, 129, seed=6))
    check_product(Z.mx4_matmul(wide[:, 5:134], qb, F32), values64(Z.mx4_quantize(wide[:, 5:134])), values64(qb), 129)


def test_product_nan_block(Z):
    """A block holding inf makes its row's results NaN, and only those; empty sums are zero."""
    for m, n, k in ((40, 70, 256), (300, 300, 1024)):
        a, b = randn(m, k), randn(n, k, seed=1)
        a[3, 40] = float("inf")
        b[5, k - 1] = float("nan")
        for x in (Z.mx4_quantize(a), a):
            c = Z.mx4_matmul(x, Z.mx4_quantize(b), F32)
            nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
            nan[3] = True
            nan[:, 5] = True
            assert torch.equal(torch.isnan(c), nan)
    q = Z.MX4.alloc(5, 0, "cuda")
    assert (Z.mx4_matmul(q, Z.MX4.alloc(7, 0, "cuda"), F32) == 0).all()
    assert Z.mx4_matmul(Z.MX4.alloc(0, 64, "cuda"), Z.mx4_quantize(randn(3, 64))).shape == (0, 3)


# ----------------------------------------------------------------------------- the linear layer
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("t,n,k", [(1, 1, 1), (3, 40, 130), (64, 128, 256), (200, 300, 100), (513, 257, 129)])
def test_linear_and_gradients(Z, t, n, k, dtype):
    x, w = randn(t, k, seed=1).to(dtype).requires_grad_(), randn(n, k, seed=2).to(dtype).requires_grad_()
    dy = randn(t, n, seed=3).to(dtype)
    y = Z.mx4_linear(x, w)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    q = lambda v: values64(Z.mx4_quantize(v.detach().contiguous()))  # noqa: E731
    check_product(y.detach(), q(x), q(w), k)
    check_product(dx, q(dy), q(w.t()), n)
    check_product(dw, q(dy.t()), q(x.t()), t)
    # one gradient wanted; dy of odd strides
    dy2 = randn(n, t, seed=4).to(dtype).t()
    y = Z.mx4_linear(x, w.detach())
    check_product(torch.autograd.grad(y, x, dy2)[0], q(dy2), q(w.t()), n)
    y = Z.mx4_linear(x.detach(), w)
    check_product(torch.autograd.grad(y, w, dy2)[0], q(dy2.t()), q(x.t()), t)


def test_linear_gradient_by_differences(Z):
    """Inputs on the 4-bit grid of one scale: the quantised map is then exact, and linear between grid points."""
    g = torch.tensor([-4.0, -2.0, -1.0, 0.0, 1.0, 2.0, 4.0], device="cuda")
    pick = lambda r, c, s: g[torch.randint(0, 7, (r, c), device="cuda", generator=gen(s))]  # noqa: E731
    x, w, dy = pick(64, 96, 1), pick(32, 96, 2), pick(64, 32, 3)
    for v in (x, w, dy):  # every block of 32, along either dimension, holds a 4
        v[::16, :] = 4.0
        v[:, ::16] = 4.0
    x.requires_grad_()
    w.requires_grad_()
    dx, dw = torch.autograd.grad(Z.mx4_linear(x, w), (x, w), dy)
    f = lambda a, b: (Z.mx4_linear(a, b).double() * dy.double()).sum()  # noqa: E731
    with torch.no_grad():
        for i, j in ((1, 1), (17, 50), (63, 95)):
            step = torch.zeros_like(x)
            step[i, j] = -x[i, j] + 2.0
            assert abs(float(f(x + step, w) - f(x, w)) - float(dx[i, j] * step[i, j])) < 1e-6
        for i, j in ((1, 1), (30, 77)):
            step = torch.zeros_like(w)
            step[i, j] = -w[i, j] - 1.0
            assert abs(float(f(x, w + step) - f(x, w)) - float(dw[i, j] * step[i, j])) < 1e-6


# ----------------------------------------------------------------------------- orthogonalisation
def rel(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


NS_SIZES = [(1, 1, 1), (1, 1, 77), (1, 300, 1), (3, 2, 3), (2, 32, 32), (1, 33, 20), (2, 64, 64), (1, 65, 96), (3, 128, 128),
            (1, 128, 129), (2, 129, 128), (1, 5, 200), (1, 200, 130), (2, 256, 700), (1, 700, 257), (1, 1000, 64), (1, 520, 1030), (2, 20, 3000), (1, 3001, 128), (2, 100, 700)]


@pytest.mark.parametrize("count,rows,cols", NS_SIZES)
def test_orthogonalize(Z, count, rows, cols):
    for src, dst in ((F32, BF16), (F16, F16), (BF16, BF16), (F32, F16), (BF16, F16), (F16, BF16)):
        x = randn(count, rows, cols, seed=rows + cols).to(src)
        out = Z.orthogonalize(x, dst)
        assert out.dtype == dst and out.shape == x.shape
        for i in range(count):
            assert rel(out[i], ns64(x[i])) <= ns_tol(rows, cols) + half_step(dst)


# one size for every tile shape of the symmetric products, then of the product with X, and strips past the
# count that makes M in each of them
NS_SHAPES = [(16, 1160, 1160), (16, 900, 900), (16, 650, 650), (16, 450, 450), (8, 900, 900), (16, 330, 330),
             (16, 390, 1560), (16, 330, 1320), (16, 1040, 260), (16, 170, 680), (8, 330, 1320), (16, 430, 130),
             (1, 20, 33000), (1, 40, 17000), (2, 8500, 100), (130, 60, 500), (130, 1000, 20)]


@pytest.mark.parametrize("count,rows,cols", NS_SHAPES)
def test_orthogonalize_every_tile_shape(Z, count, rows, cols):
    x = randn(count, rows, cols, seed=rows)
    out = Z.orthogonalize(x, F16)
    for i in {0, count // 2, count - 1}:
        assert rel(out[i], ns64_gpu(x[i])) <= ns_tol(rows, cols) + half_step(F16)


@pytest.mark.parametrize("rows,cols", [(5, 200), (64, 64), (96, 65), (128, 100), (130, 200), (700, 256)])
def test_orthogonalize_spectra(Z, rows, cols):
    m = min(rows, cols)
    torch.manual_seed(rows)
    u = torch.linalg.qr(torch.randn(rows, m, dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(cols, m, dtype=torch.float64))[0]
    power = (u * torch.arange(1, m + 1, dtype=torch.float64) ** -1.0) @ v.t()
    rank1 = torch.randn(rows, 1) @ torch.randn(1, cols)
    scaled = torch.randn(rows, cols) * torch.exp(torch.randn(1, cols)) * torch.exp(torch.randn(rows, 1))
    tol = ns_tol(rows, cols)
    for name, x, tol in (("power", power, tol), ("rank one", rank1, 2 * tol), ("scaled", scaled, tol),
                         ("constant", torch.ones(rows, cols), 4 * tol), ("identity", torch.eye(rows, cols), 4 * tol),
                         ("huge", power * 1e30, tol), ("tiny", power * 1e-4, tol)):
        x = x.float().cuda()
        assert rel(Z.orthogonalize(x, F16), ns64(x)) <= tol + half_step(F16), name


def test_orthogonalize_settings(Z):
    for shape in ((60, 40), (150, 200)):
        x = randn(*shape)
        for steps in (0, 1, 2, 9):
            assert rel(Z.orthogonalize(x, F16, steps=steps), ns64(x, steps)) <= 2 * ns_tol(*shape) + half_step(F16)
        cubic = (1.5, -0.5, 0.0)
        assert rel(Z.orthogonalize(x, F16, steps=6, coeffs=cubic), ns64(x, 6, coeffs=cubic)) <= 2 * ns_tol(*shape) + half_step(F16)
        small = x * 1e-9
        assert rel(Z.orthogonalize(small, F16, eps=1e-3), ns64(small, eps=1e-3)) <= NS_TOL + half_step(F16) + 2.0 ** -6


def test_orthogonalize_zero_and_not_finite(Z):
    for shape in ((2, 50, 60), (2, 200, 130)):
        x = randn(*shape)
        x[0] = 0
        for eps in (1e-7, 0.0):
            o = Z.orthogonalize(x, BF16, eps=eps)
            assert (o[0] == 0).all() and torch.isfinite(o[1].float()).all()
        for bad in (float("inf"), float("nan")):
            y = x.clone()
            y[0, 3, 7] = bad
            o = Z.orthogonalize(y, BF16)
            assert torch.isnan(o[0].float()).all() and torch.isfinite(o[1].float()).all()
    assert Z.orthogonalize(torch.empty(0, 5, 5, device="cuda")).shape == (0, 5, 5)
    assert Z.orthogonalize(torch.empty(3, 0, 5, device="cuda")).shape == (3, 0, 5)


def test_orthogonalize_strides_and_in_place(Z):
    base = randn(3, 140, 300)
    for x in (base[:, :130, 5:205], base[:, :60, 3:90], base.mT, base[:2, ::2, :100], base[1, :, ::2]):
        o = Z.orthogonalize(x, F16)
        want = x.reshape(-1, *x.shape[-2:])
        got = o.reshape(-1, *x.shape[-2:])
        for i in range(want.shape[0]):
            assert rel(got[i], ns64(want[i])) <= ns_tol(*x.shape[-2:]) + half_step(F16)
    h = base.to(BF16)
    keep = h.clone()
    want = Z.orthogonalize(h[:, :, :200])
    Z.orthogonalize(h[:, :, :200], out=h[:, :, :200])
    assert torch.equal(h[:, :, :200], want) and torch.equal(h[:, :, 200:], keep[:, :, 200:])


def test_orthogonalize_is_reproducible(Z):
    for shape in ((4, 100, 128), (2, 300, 700)):
        x = randn(*shape)
        a, b = Z.orthogonalize(x, F16), Z.orthogonalize(x, F16)
        assert torch.equal(a, b)
        # a matrix of a stack is computed as it is alone
        assert torch.equal(Z.orthogonalize(x[1], F16), a[1])


# ----------------------------------------------------------------------------- the optimizer step
def muon64(p, m, g, clip, lr, mu, wd, nesterov, scale, rows, cols):
    p, m, g = p.double().cpu(), m.double().cpu(), g.double().cpu() * clip
    m = mu * m + (1 - mu) * g
    u = (1 - mu) * g + mu * m if nesterov else m
    s = 0.2 * math.sqrt(max(rows, cols)) if scale else math.sqrt(max(1.0, rows / cols))
    o = ns64(u)
    return p - lr * wd * p - lr * s * o, m, lr * s * o


@pytest.mark.parametrize("count,rows,cols", [(1, 1, 1), (3, 40, 33), (2, 128, 128), (2, 200, 130), (1, 130, 300), (1, 700, 257),
                                             (1, 20, 2000), (2, 1000, 60), (1, 128, 700)])
@pytest.mark.parametrize("nesterov,scale,wd", [(True, 1, 0.01), (False, 0, 0.0)])
def test_muon_step(Z, count, rows, cols, nesterov, scale, wd):
    lr, mu = 1e-2, 0.95
    for slot_dtype in (BF16, F16):
        p, m, g = (randn(count, rows, cols, seed=i) * f for i, f in ((1, 0.02), (2, 1e-3), (3, 1e-3)))
        slot = p.to(slot_dtype)
        hp = Z.muon_hparams(lr=lr, momentum=mu, weight_decay=wd, nesterov=nesterov, scale=scale)
        old_p, old_m = p.clone(), m.clone()
        for step in range(2):
            Z.muon_step(p, m, g, hp, slot=slot)
            for i in range(count):
                wp, wm, up = muon64(old_p[i], old_m[i], g[i], 1.0, lr, mu, wd, nesterov, scale, rows, cols)
                # the coefficients mu, 1 - mu, lr are fp32: half a step each, and one per operation
                assert ((m[i].double().cpu() - wm).abs() <= 5 * 2.0 ** -24 * (wm.abs() + g[i].abs().double().cpu()
                                                                             + old_m[i].abs().double().cpu())).all()
                err = (p[i].double().cpu() - wp).norm()
                assert err <= ns_tol(rows, cols) * up.norm() + 4 * 2.0 ** -24 * wp.norm()
            assert torch.equal(slot, p.to(slot_dtype))
            old_p, old_m = p.clone(), m.clone()


def test_muon_step_in_a_shard(Z):
    """Matrices of a flat shard at a stride, into the gather buffer's slot; what lies between them is left alone;
    clip and skip come from the control block."""
    for rows, cols, count, stride in ((24, 40, 3, 1000), (150, 130, 2, 20003)):
        total = count * stride + 7
        flat = [randn(total, seed=i) * f for i, f in ((1, 0.02), (2, 1e-3), (3, 1e-3))]
        gather = torch.full((total + 11,), 5.0, dtype=F16, device="cuda")
        view = lambda t, o=0: t[7 + o:].as_strided((count, rows, cols), (stride, cols, 1), 7 + o)  # noqa: E731
        p, m, g = (view(t) for t in flat)
        slot = gather.as_strided((count, rows, cols), (stride, cols, 1), 11)
        inside = torch.zeros(total, dtype=torch.bool, device="cuda")
        view(inside).fill_(True)
        before = [t.clone() for t in flat]
        hp = Z.muon_hparams(lr=1e-2)
        ctrl = torch.empty(Z.zero_ctrl_bytes(), dtype=torch.uint8, device="cuda")
        Z.zero_ctrl_init(ctrl, 1.0)
        offset = Z.Ctrl.skip.offset
        ctrl[offset:offset + 4] = torch.tensor([1], dtype=torch.int32).view(torch.uint8).cuda()
        Z.muon_step(p, m, g, hp, slot=slot, ctrl=ctrl)
        assert all(torch.equal(a, b) for a, b in zip(flat, before)) and (gather == 5).all()
        ctrl[offset:offset + 4] = 0
        offset = Z.Ctrl.clip.offset
        ctrl[offset:offset + 4] = torch.tensor([0.25]).view(torch.uint8).cuda()
        Z.muon_step(p, m, g, hp, slot=slot, ctrl=ctrl)
        for a, b in zip(flat, before):
            assert torch.equal(a[~inside], b[~inside])
        assert torch.equal(flat[2], before[2])
        for i in range(count):
            wp, wm, up = muon64(view(before[0])[i], view(before[1])[i], view(before[2])[i], 0.25, 1e-2, 0.95, 0.0, True, 1,
                                rows, cols)
            assert rel(m[i], wm) <= 5 * 2.0 ** -24
            assert (p[i].double().cpu() - wp).norm() <= ns_tol(rows, cols) * up.norm() + 4 * 2.0 ** -24 * wp.norm()
        assert torch.equal(slot, p.to(F16))
        outside = torch.ones(total + 11, dtype=torch.bool, device="cuda")
        outside.as_strided((count, rows, cols), (stride, cols, 1), 11).fill_(False)
        assert (gather[outside] == 5).all()


# ----------------------------------------------------------------------------- together
def test_shard_step_with_matrices(Z):
    """MuonShardStep equals its parts: reduce, decision, AdamW between the matrices, the matrix step on them; a step
    with an overflow leaves everything."""
    matrices = [(8, 2, 40, 33), (3000, 1, 150, 200)]
    n, psi, offset = 3, 34000, 24
    stride = 34048
    hp, muon = Z.hparams(lr=1e-2, weight_decay=0.01, max_grad_norm=0.5), Z.muon_hparams(lr=1e-2)
    state = tuple(randn(psi, seed=i) * f for i, f in ((1, 0.02), (2, 1e-3)))
    state = (*state, (randn(psi, seed=3) * 1e-3).square())
    other = tuple(t.clone() for t in state)
    g, g2 = torch.empty(psi, device="cuda"), torch.empty(psi, device="cuda")
    gather, gather2 = (torch.zeros(psi + offset, dtype=BF16, device="cuda") for _ in range(2))
    step = Z.MuonShardStep(n, stride, psi, offset, Z.BF16, Z.BF16, hp, muon, matrices, state, g)
    ctrl = torch.empty(Z.zero_ctrl_bytes(), dtype=torch.uint8, device="cuda")
    ws = torch.empty(Z.zero_workspace_bytes(psi), dtype=torch.uint8, device="cuda")
    Z.zero_ctrl_init(ctrl, 1.0)
    for k in range(3):
        c = randn(n, stride, seed=10 + k).to(BF16) * 1e-2
        if k == 1:
            c[1, 5000] = float("inf")
            before = [t.clone() for t in (*state, gather)]
        step.step(c, gather)
        Z.zero_reduce_grads(c, Z.BF16, n, stride, psi, ctrl, g2, ws)
        Z.zero_grad_norm_overflow([ws], [psi], [ctrl], hp, False)
        for a, b in ((0, 8), (8 + 2 * 40 * 33, 3000), (3000 + 150 * 200, psi)):
            Z.zero_adam_step(tuple(t[a:] for t in other), g2[a:], b - a, hp, ctrl, gather2, Z.BF16, offset + a)
        for a, count, rows, cols in matrices:
            b = a + count * rows * cols
            part = [t[a:b].view(count, rows, cols) for t in (other[0], other[1], g2)]
            Z.muon_step(*part, muon, slot=gather2[offset + a:offset + b].view(count, rows, cols), ctrl=ctrl)
        for a, b in zip((*state, gather), (*other, gather2)):
            assert torch.equal(a, b)
        assert step.ctrl_dict()["skip"] == (k == 1)
        if k == 1:
            assert all(torch.equal(a, b) for a, b in zip((*state, gather), before))
    assert step.ctrl_dict()["t"] == 2 and step.ctrl_dict()["clip"] < 1
    for bad in ([(0, 1, 10, 10), (50, 1, 4, 4)], [(0, 1, 300, 300)], [(0, 1, 3, 3)]):
        with pytest.raises(ValueError):
            Z.MuonShardStep(n, stride, psi, 0, Z.BF16, Z.BF16, hp, muon, bad, state, g)


def test_example_learns(Z):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "muon_mx4.py")
    spec = importlib.util.spec_from_file_location("muon_mx4", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, (weights, bias), ctrl = m.train(steps=40, ranks=2, width=128)
    assert ctrl["t"] == 40
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5])
    rows = randn(4, 64)
    one = m.serve(weights, bias, rows)
    x = rows.bfloat16()
    for i, (w, b) in enumerate(zip(weights, bias)):
        x = Z.mx4_linear(x, w) + b
        x = torch.nn.functional.gelu(x) if i < len(weights) - 1 else x
    # the same codes and fp32 sums in another order: a rounding of a layer's bf16 result now and then
    assert (one.float() - x.detach().float()).norm() <= 0.02 * x.detach().float().norm()


# ----------------------------------------------------------------------------- streams, graphs, refusals
def test_other_stream_and_graph(Z):
    """Work on a side stream and in a replayed graph equals the eager result each time."""
    x, w = randn(70, 200, dtype=BF16), randn(90, 200, seed=1, dtype=BF16)
    g = randn(150, 140, seed=2)
    ws = torch.empty(Z._lib.zero_ns_workspace_bytes(1, 150, 140), dtype=torch.uint8, device="cuda")
    out = torch.empty(150, 140, dtype=BF16, device="cuda")

    def work():
        Z.orthogonalize(g, out=out, ws=ws)
        xr, xc = Z.mx4_quantize(x, cols=True)
        wr = Z.mx4_quantize(w)
        return Z.mx4_matmul(xr, wr), Z.mx4_matmul(x[:9], wr), Z.mx4_dequantize(xc)

    eager = [t.clone() for t in work()] + [out.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = work()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip([*got, out], eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work()
    for i in range(4):
        for t in (*held, out):
            t.zero_()
        graph.replay()
        randn(64, 64, seed=i).sum().item()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([*held, out], eager))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_and_gradients_in_graph(Z, dtype):
    """Forward and backward replayed with new values equal the eager ones each time.

    The leaves are the capture's own, so that no eager graph holds them."""
    tokens, n, k = 70, 90, 200
    x, w, dy = randn(tokens, k, dtype=dtype), randn(n, k, seed=1, dtype=dtype), randn(tokens, n, seed=2, dtype=dtype)

    def work(x, w):
        y = Z.mx4_linear(x, w)
        return (y.detach(), *torch.autograd.grad(y, (x, w), dy))

    work(x.clone().requires_grad_(), w.clone().requires_grad_())  # loads the kernels
    xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = work(xs, ws)
    for i in range(4):
        with torch.no_grad():
            xs.copy_(randn(tokens, k, seed=10 + i, dtype=dtype))
            ws.copy_(randn(n, k, seed=20 + i, dtype=dtype))
            dy.copy_(randn(tokens, n, seed=30 + i, dtype=dtype))
            for t in held:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        eager = work(xs.detach().clone().requires_grad_(), ws.detach().clone().requires_grad_())
        assert all(torch.equal(a, b) for a, b in zip(got, eager))


def test_refusals_of_tensors(Z):
    x = randn(8, 64)
    with pytest.raises(TypeError):
        Z.orthogonalize(x, F32)
    with pytest.raises(TypeError):
        Z.mx4_quantize(x.double())
    with pytest.raises(ValueError):
        Z.mx4_quantize(x, rows=False)
    with pytest.raises(ValueError):
        Z.mx4_matmul(x, Z.mx4_quantize(randn(8, 65)))
    with pytest.raises(ValueError):
        Z.mx4_matmul(x, Z.mx4_quantize(x), out=torch.empty(8, 9, device="cuda"))
    with pytest.raises(ValueError):
        Z.mx4_matmul(x, Z.mx4_quantize(x), accumulate=True)
    with pytest.raises(ValueError):
        Z.muon_step(x, x[:, :32], x, Z.muon_hparams())
    with pytest.raises(ValueError):
        Z.muon_step(x.t(), x.t(), x.t(), Z.muon_hparams())
    with pytest.raises(Z.ZeroError):
        Z.orthogonalize(x, F16, steps=65)
    with pytest.raises(Z.ZeroError) as e:
        Z.orthogonalize(randn(200, 200), F16, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -4


# ----------------------------------------------------------------------------- rows whose elements round alike
# One element a row: S is diagonal then, and its diagonal is fp32, so nothing is rounded to 11 bits but the result.
# The tolerance is the narrow matrices' share for fp32, and half a step of the result, whose elements all round alike.
@pytest.mark.parametrize("rows,cols", [(412, 412), (482, 482), (493, 700), (900, 482), (520, 520), (1100, 1040)])
def test_orthogonalize_one_element_a_row(Z, rows, cols):
    m = min(rows, cols)
    torch.manual_seed(rows)
    spread = torch.zeros(rows, cols)
    spread[torch.randperm(rows)[:m], torch.randperm(cols)[:m]] = 1.0
    for x in (torch.eye(rows, cols), spread):
        assert rel(Z.orthogonalize(x.cuda(), F16), ns64(x)) <= 500 * 2.0 ** -24 + half_step(F16)


# Elements of one or two values would round alike; independent roundings of rows make the tolerance of other matrices
# hold for them.
@pytest.mark.parametrize("rows,cols", [(177, 790), (372, 2000), (817, 1200), (1190, 1500), (6328, 1939), (1393, 21020)])
def test_orthogonalize_equal_elements(Z, rows, cols):
    torch.manual_seed(rows)
    two = 1.0 + (torch.randn(1, cols) > 0).float().expand(rows, cols)
    for x in (torch.ones(rows, cols), two, two.flip(1) * (1.0 + (torch.randn(rows, 1) > 0).float())):
        x = x.cuda()
        assert rel(Z.orthogonalize(x, F16), ns64_gpu(x)) <= NS_TOL + half_step(F16)


# ----------------------------------------------------------------------------- few rows, few slabs
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("k", [100, 256, 300, 640, 1024, 1700, 1920, 2047])
def test_product_of_few_rows_and_slabs(Z, k, dtype):
    """Up to seven slabs of 256: some of the eight waves have none.  Rows as values and as operands take the same sums."""
    for m, n in ((1, 4096), (5, 1000), (8, 33)):
        x = randn(m, k, seed=k).to(dtype)
        qx, qb = Z.mx4_quantize(x), Z.mx4_quantize(randn(n, k, seed=6))
        want = Z.mx4_matmul(qx, qb, F32)
        check_product(want, values64(qx), values64(qb), k)
        for _ in range(20):
            assert torch.equal(Z.mx4_matmul(x, qb, F32), want)


# ----------------------------------------------------------------------------- several ranks with matrices
def test_several_ranks_with_matrices(Z):
    """Two ranks on one decision equal their own calls around the same decision, eager and from a replayed graph."""
    n, psi, stride = 2, 4000, 4032
    matrices = [(0, 2, 20, 33), (1400, 1, 40, 60)]
    hp, muon = Z.hparams(lr=1e-2, max_grad_norm=0.5), Z.muon_hparams(lr=1e-2)

    def ranks():
        out = []
        for r in range(2):
            state = (randn(psi, seed=r) * 0.02, randn(psi, seed=r + 5) * 1e-3, (randn(psi, seed=r + 9) * 1e-3).square())
            out.append(Z.MuonShardStep(n, stride, psi, r * psi, Z.BF16, Z.BF16, hp, muon, matrices, state,
                                       torch.empty(psi, device="cuda")))
        return out

    contribs = [torch.zeros(n, stride, dtype=BF16, device="cuda") for _ in range(2)]
    gathers = [torch.zeros(2 * psi, dtype=BF16, device="cuda") for _ in range(3)]
    a, b, c = ranks(), ranks(), ranks()
    multi, graphed = Z.MultiShardStep(a), Z.MultiShardStep(c)
    graph = graphed.capture(contribs, gathers[2])
    for k in range(3):
        for r in range(2):
            contribs[r].copy_(randn(n, stride, seed=20 + 2 * k + r) * 1e-2)
        multi.step(contribs, gathers[0])
        for s, t in zip(b, contribs):
            s.run_pieces(t, gathers[1])
        Z.zero_grad_norm_overflow([s.ws for s in b], [psi] * 2, [s.ctrl for s in b], hp, False)
        for s in b:
            s.complete(gathers[1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, gathers[0]) for g in gathers[1:])
        for other in (b, c):
            for s, t in zip(a, other):
                assert all(torch.equal(x, y) for x, y in zip(s.state, t.state))


@pytest.mark.parametrize("m", [1, 32, 33, 64, 65])
def test_product_of_empty_rows(Z, m):
    """k = 0, as values and as operands: zeros, or what was there."""
    b = Z.MX4.alloc(70, 0, "cuda")
    for dtype in (F32, BF16):
        for a in (torch.empty(m, 0, dtype=dtype, device="cuda"), Z.MX4.alloc(m, 0, "cuda")):
            out = torch.full((m, 70), 3.0, device="cuda")
            assert (Z.mx4_matmul(a, b, out=out) == 0).all()
            out.fill_(3.0)
            assert (Z.mx4_matmul(a, b, out=out, accumulate=True) == 3).all()


def test_results_beside_what_is_read(Z):
    """A result may take columns or rows of the operand's own buffer, not its elements."""
    base = randn(40, 200, dtype=BF16)
    x, q = base[:, :64], Z.mx4_quantize(randn(64, 64, seed=1))
    for rows in (1, 16, 40):
        want = Z.mx4_matmul(x[:rows].clone(), q)
        Z.mx4_matmul(x[:rows], q, out=base[:rows, 64:128])
        assert torch.equal(base[:rows, 64:128], want)
        for over in (x[:rows], base[:rows, 63:127]):
            with pytest.raises(Z.ZeroError):
                Z.mx4_matmul(x[:rows], q, out=over)
    h = randn(4, 70, 90, dtype=BF16)
    want = Z.orthogonalize(h[::2, :, :40].clone())
    for out in (h[1::2, :, :40], h[::2, :, 41:81], h[::2, :, :40]):  # the last one in place
        Z.orthogonalize(h[::2, :, :40], out=out)
        assert torch.equal(out, want)
    with pytest.raises(Z.ZeroError):
        Z.orthogonalize(h[::2, :, :40], out=h[::2, :, 1:41])
    space = torch.zeros(4, 256, dtype=BF16, device="cuda")
    held = Z.MX4(space.view(torch.uint8)[0, :256].view(4, 64), torch.zeros(4, 4, dtype=torch.uint8, device="cuda"), 4, 128)
    with pytest.raises(Z.ZeroError):
        Z.mx4_dequantize(held, out=space[:, :128])
    Z.mx4_dequantize(held, out=space[:, 128:])


def test_linear_without_gradients(Z):
    """The same values where torch does not record; a checkpointed block's gradients are those of a recorded one."""
    from torch.utils.checkpoint import checkpoint
    x, w, dy = randn(70, 200, dtype=BF16), randn(90, 200, seed=1, dtype=BF16), randn(70, 90, seed=2, dtype=BF16)
    xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()
    y = Z.mx4_linear(xs, ws)
    grads = torch.autograd.grad(y, (xs, ws), dy)
    for mode in (torch.no_grad(), torch.inference_mode()):
        with mode:
            assert torch.equal(Z.mx4_linear(xs, ws), y)
    for reentrant in (False, True):
        xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()
        again = checkpoint(Z.mx4_linear, xs, ws, use_reentrant=reentrant)
        again.backward(dy)
        assert torch.equal(again, y) and torch.equal(xs.grad, grads[0]) and torch.equal(ws.grad, grads[1])


@pytest.mark.parametrize("rows,cols", [(60, 40), (20, 3000), (150, 200), (600, 530)])
def test_orthogonalize_coefficients_up_to_the_range(Z, rows, cols):
    """Singular values that reach 3 between two steps, S 9 and M 90: the products' operands stay in fp16's range.  The
    second step magnifies the first one's relative error by s f'(s) / f(s) = 4.8 there, and adds its own."""
    x = torch.randn(rows, 1, generator=torch.Generator().manual_seed(rows)) * torch.ones(1, cols)
    tol = NS_TOL if min(rows, cols) > 128 else ns_tol(rows, cols)
    for coeffs in ((1.0, 1.0, 1.0), (-1.0, -1.0, -1.0), (0.0, 3.0, 0.0)):
        got = Z.orthogonalize(x.cuda(), BF16, coeffs=coeffs, steps=2)
        assert rel(got, ns64(x, 2, coeffs=coeffs)) <= 5.8 * tol + half_step(BF16)


@pytest.mark.parametrize("m,n,k", [(16, 9000, 1024), (9, 8200, 1792), (32, 8193, 500)])
def test_product_of_values_and_of_operands(Z, m, n, k):
    """Where the two forms add their sums in different orders, both keep to the same bound."""
    x = randn(m, k, seed=1) * torch.exp(4 * randn(m, k, seed=2))
    qx, qb = Z.mx4_quantize(x), Z.mx4_quantize(randn(n, k, seed=3) * torch.exp(4 * randn(n, k, seed=4)))
    for a in (x, qx):
        check_product(Z.mx4_matmul(a, qb, F32), values64(qx), values64(qb), k)


# ----------------------------------------------------------------------------- large matrices and strips, all that is special
# Above a smaller side of 512 X^T has one fp16 part.  Tolerances: NS_TOL, twice it where the rank is low, as for
# rank-one matrices above: the roundings then put noise into directions that X lacks.
@pytest.mark.parametrize("rows,cols", [(513, 513), (520, 1030), (2304, 768), (1041, 1166)])
def test_orthogonalize_spectra_large(Z, rows, cols):
    m = min(rows, cols)
    torch.manual_seed(rows)
    r = lambda *shape: torch.randn(*shape, dtype=torch.float64)  # noqa: E731
    u, v = torch.linalg.qr(r(rows, m))[0], torch.linalg.qr(r(cols, m))[0]
    k = torch.arange(1, m + 1, dtype=torch.float64)
    hot = torch.zeros(rows, cols, dtype=torch.float64)
    hot[torch.arange(rows), torch.randint(0, cols, (rows,))] = 1.0
    for name, x, tol in (("1/k", (u / k) @ v.t(), 1), ("1/sqrt k", (u / k.sqrt()) @ v.t(), 1), ("flat", u @ v.t(), 1),
                         ("rank one", r(rows, 1) @ r(1, cols), 2), ("quarter rank", r(rows, m // 4) @ r(m // 4, cols), 2),
                         ("one-hot rows", hot, 1), ("signs", torch.sign(r(rows, cols)), 1), ("constant", torch.ones(rows, cols), 1),
                         ("scaled", r(rows, cols) * torch.exp(r(1, cols)) * torch.exp(r(rows, 1)), 1)):
        x = x.float().cuda()
        assert rel(Z.orthogonalize(x, F16), ns64_gpu(x)) <= tol * NS_TOL + half_step(F16), name


STRIPS = [(2, 20, 3000), (2, 20, 33000), (2, 3000, 60), (2, 17000, 40), (2, 100, 700), (2, 8500, 100)]


@pytest.mark.parametrize("count,rows,cols", STRIPS)
def test_strips_zero_and_not_finite(Z, count, rows, cols):
    x = randn(count, rows, cols)
    x[0] = 0
    for eps in (1e-7, 0.0):
        o = Z.orthogonalize(x, BF16, eps=eps)
        assert (o[0] == 0).all() and torch.isfinite(o[1].float()).all()
    for bad in (float("inf"), float("nan")):
        y = x.clone()
        y[0, rows - 1, cols - 1] = bad
        o = Z.orthogonalize(y, BF16)
        assert torch.isnan(o[0].float()).all() and torch.isfinite(o[1].float()).all()


@pytest.mark.parametrize("count,rows,cols", [*STRIPS, (2, 30, 20), (2, 130, 200)])
def test_muon_step_skipped_and_clipped(Z, count, rows, cols):
    """A skipped step leaves master, momentum and slot as they are, whatever the gradient holds; a clipped one is the
    step of the clipped gradient."""
    ctrl = torch.empty(Z.zero_ctrl_bytes(), dtype=torch.uint8, device="cuda")
    Z.zero_ctrl_init(ctrl, 1.0)
    skip, clip = Z.Ctrl.skip.offset, Z.Ctrl.clip.offset
    p, m, g = (randn(count, rows, cols, seed=i) * f for i, f in ((1, 0.02), (2, 1e-3), (3, 1e-3)))
    slot = torch.full((count, rows, cols), 5.0, dtype=BF16, device="cuda")
    hp = Z.muon_hparams(lr=1e-2, weight_decay=0.01)
    before = [t.clone() for t in (p, m)]
    bad = g.clone()
    bad[0, 0, 0] = float("inf")
    ctrl[skip:skip + 4] = torch.tensor([1], dtype=torch.int32).view(torch.uint8).cuda()
    Z.muon_step(p, m, bad, hp, slot=slot, ctrl=ctrl)
    assert torch.equal(p, before[0]) and torch.equal(m, before[1]) and (slot == 5).all()
    ctrl[skip:skip + 4] = 0
    ctrl[clip:clip + 4] = torch.tensor([0.25]).view(torch.uint8).cuda()
    Z.muon_step(p, m, g, hp, slot=slot, ctrl=ctrl)
    q, n = before[0].clone(), before[1].clone()
    Z.muon_step(q, n, g * 0.25, hp)  # a power of two: the same numbers
    assert torch.equal(p, q) and torch.equal(m, n) and torch.equal(slot, p.to(BF16))
    for i in range(count):
        step = before[0][i].double() * (1 - 1e-4) - p[i].double()
        u = 0.95 * (0.95 * before[1][i].double() + 0.05 * 0.25 * g[i].double()) + 0.05 * 0.25 * g[i].double()
        want = 1e-2 * 0.2 * math.sqrt(max(rows, cols)) * ns64_gpu(u)
        err = float((step.cpu() - want).norm())
        # NS, and what fp32 leaves of the momentum and of master
        assert err <= ns_tol(rows, cols) * float(want.norm()) + 4 * 2.0 ** -24 * float(before[0][i].double().norm())


def test_orthogonalize_large_is_reproducible(Z):
    for shape in ((1500, 4099), (700, 2304)):
        x = randn(*shape, dtype=F16)
        first = Z.orthogonalize(x, F16)
        for _ in range(3):
            assert torch.equal(Z.orthogonalize(x, F16), first)


@pytest.mark.parametrize("count,rows,cols", [(1, 700, 900), (2, 1100, 600), (1, 1200, 2500)])
def test_muon_step_large(Z, count, rows, cols):
    lr, wd = 1e-2, 0.01
    p, m, g = (randn(count, rows, cols, seed=i) * f for i, f in ((1, 0.02), (2, 1e-3), (3, 1e-3)))
    slot, before = torch.empty_like(p, dtype=BF16), [t.double() for t in (p, m)]
    Z.muon_step(p, m, g, Z.muon_hparams(lr=lr, weight_decay=wd), slot=slot)
    for i in range(count):
        mom = 0.95 * before[1][i] + 0.05 * g[i].double()
        assert ((m[i].double() - mom).abs() <= 5 * 2.0 ** -24 * (mom.abs() + g[i].double().abs() + before[1][i].abs())).all()
        step = (before[0][i] * (1 - lr * wd) - p[i].double()).cpu()
        want = lr * 0.2 * math.sqrt(max(rows, cols)) * ns64_gpu(0.05 * g[i].double() + 0.95 * mom)
        assert float((step - want).norm()) <= NS_TOL * float(want.norm()) + 4 * 2.0 ** -24 * float(before[0][i].norm())
    assert torch.equal(slot, p.to(BF16))


# ----------------------------------------------------------------------------- operands of two parts, and of one
# An fp16 result leaves nothing but its own rounding: the operands have 22 bits, a thousandth of NS_TOL and what fp32
# adds, as for narrow matrices.  Sums over m equal terms (the products with M and M's own, of matrices of rank one) round
# alike at each of their m / 4 steps, 2^-24 of the sum, and the first cancels to a quarter: 10 m 2^-24 over five steps.
def spectra(rows, cols):
    m = min(rows, cols)
    torch.manual_seed(rows)
    r = lambda *shape: torch.randn(*shape, dtype=torch.float64)  # noqa: E731
    u, v = torch.linalg.qr(r(rows, m))[0], torch.linalg.qr(r(cols, m))[0]
    k = torch.arange(1, m + 1, dtype=torch.float64)
    hot = torch.zeros(rows, cols, dtype=torch.float64)
    hot[torch.arange(rows), torch.randint(0, cols, (rows,))] = 1.0
    return {"normal": r(rows, cols), "1/k": (u / k) @ v.t(), "1/sqrt k": (u / k.sqrt()) @ v.t(), "flat": u @ v.t(),
            "quarter rank": r(rows, m // 4) @ r(m // 4, cols), "one-hot rows": hot, "signs": torch.sign(r(rows, cols)),
            "scaled": r(rows, cols) * torch.exp(r(1, cols)) * torch.exp(r(rows, 1)), "rank one": r(rows, 1) @ r(1, cols),
            "constant": torch.ones(rows, cols, dtype=torch.float64)}


@pytest.mark.parametrize("rows,cols", [(130, 200), (300, 700), (513, 513), (1100, 1600), (2304, 768)])
def test_orthogonalize_fp16_leaves_its_rounding(Z, rows, cols):
    for name, x in spectra(rows, cols).items():
        x = x.float().cuda()
        want = ns64_gpu(x)
        if name in ("rank one", "constant", "one-hot rows"):  # equal elements round to the next one alike
            tol = half_step(F16) + 10 * min(rows, cols) * 2.0 ** -24
        else:
            tol = 1.02 * rel(want.half(), want) + NS_TOL / 1000 + 500 * 2.0 ** -24
        assert rel(Z.orthogonalize(x, F16), want) <= tol, name


def update(Z, x):
    """The optimizer's update of one matrix in fp32: no 16-bit rounding hides what its products leave."""
    hp = Z.muon_hparams(lr=1.0, momentum=0.0, nesterov=False, scale=Z.MUON_SCALE_SHAPE)
    p, m = torch.zeros_like(x), torch.zeros_like(x)
    Z.muon_step(p, m, x, hp)
    return -p.double() / math.sqrt(max(1.0, x.shape[0] / x.shape[1]))


@pytest.mark.parametrize("rows,cols", [(130, 200), (300, 700), (513, 513), (1100, 1600), (2304, 768)])
def test_update_of_spectra(Z, rows, cols):
    for name, x in spectra(rows, cols).items():
        x = x.float().cuda()
        tol = 2 * NS_TOL if name in ("quarter rank", "rank one") else NS_TOL
        assert rel(update(Z, x), ns64_gpu(x)) <= tol, name


@pytest.mark.parametrize("rows,cols", [(412, 412), (482, 482), (900, 482), (520, 520), (1100, 1040)])
def test_update_of_one_element_a_row(Z, rows, cols):
    x = torch.eye(rows, cols, device="cuda")
    assert rel(update(Z, x), ns64_gpu(x)) <= 500 * 2.0 ** -24


@pytest.mark.parametrize("rows,cols", [(177, 790), (817, 1200), (6328, 1939), (1393, 21020)])
def test_update_of_equal_elements(Z, rows, cols):
    x = torch.ones(rows, cols, device="cuda")
    assert rel(update(Z, x), ns64_gpu(x)) <= NS_TOL


def test_workspaces_of_results(Z):
    """A bf16 result and the optimizer step take the smaller workspace to the byte, an fp16 result the larger."""
    x = randn(200, 300)
    large, small = (f(1, 200, 300) for f in (Z._lib.zero_ns_workspace_bytes, Z._lib.zero_muon_workspace_bytes))
    space = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    assert torch.equal(Z.orthogonalize(x, BF16, ws=space(small)), Z.orthogonalize(x, BF16))
    assert torch.equal(Z.orthogonalize(x, F16, ws=space(large)), Z.orthogonalize(x, F16))
    Z.muon_step(x.clone(), x.clone(), x.clone(), Z.muon_hparams(), ws=space(small))
    for dtype, n in ((BF16, small - 1), (F16, large - 1), (F16, small)):
        with pytest.raises(Z.ZeroError) as e:
            Z.orthogonalize(x, dtype, ws=space(n))
        assert e.value.code == -4


@pytest.mark.parametrize("count,rows,cols", [shape for shape in NS_SHAPES if min(shape[1:]) > 128])
def test_update_every_tile_shape(Z, count, rows, cols):
    x = randn(count, rows, cols, seed=rows)
    hp = Z.muon_hparams(lr=1.0, momentum=0.0, nesterov=False, scale=Z.MUON_SCALE_SHAPE)
    p, m = torch.zeros_like(x), torch.zeros_like(x)
    Z.muon_step(p, m, x, hp)
    for i in {0, count // 2, count - 1}:
        assert rel(-p[i].double() / math.sqrt(max(1.0, rows / cols)), ns64_gpu(x[i])) <= NS_TOL


@pytest.mark.parametrize("count,rows,cols", [(2, 60, 40), (1, 20, 3000), (2, 130, 200), (1, 1100, 600), (2, 513, 700)])
def test_exact_update(Z, count, rows, cols):
    """In fp32, with nothing but fp32's own roundings; in a shard step too."""
    x = randn(count, rows, cols, seed=rows)
    hp = Z.muon_hparams(lr=1.0, momentum=0.0, nesterov=False, scale=Z.MUON_SCALE_SHAPE)
    p, m = torch.zeros_like(x), torch.zeros_like(x)
    slot = torch.empty_like(x, dtype=F16)
    ws = torch.empty(Z._lib.zero_ns_workspace_bytes(count, rows, cols), dtype=torch.uint8, device="cuda")
    Z.muon_step(p, m, x, hp, slot=slot, ws=ws, exact=True)
    for i in range(count):
        got = -p[i].double() / math.sqrt(max(1.0, rows / cols))
        assert rel(got, ns64_gpu(x[i])) <= NS_TOL / 1000 + 500 * 2.0 ** -24
    assert torch.equal(slot, p.to(F16))
    size = count * rows * cols
    state = [torch.zeros(size, device="cuda") for _ in range(3)]
    contrib, gather = x.view(1, -1).to(BF16), torch.empty(size, dtype=BF16, device="cuda")
    step = Z.MuonShardStep(1, size, size, 0, Z.BF16, Z.BF16, Z.hparams(max_grad_norm=1e9), hp, [(0, count, rows, cols)], state,
                           torch.empty(size, device="cuda"), exact=True)
    step.step(contrib, gather)
    want, mom = torch.zeros_like(x), torch.zeros_like(x)
    Z.muon_step(want, mom, contrib.float().view_as(x), hp, exact=True)
    assert torch.equal(state[0].view_as(x), want) and torch.equal(gather.view_as(x), want.to(BF16))
