"""The sizes and refusals of the calls on rows of tokens, on the host: every argument error is
returned before anything is enqueued, so no GPU is needed."""
import ctypes

import pytest

EINVAL, EALIGN, ERANGE, ESPACE = -1, -2, -3, -4
F16, BF16, F32 = 1, 2, 3
# aligned addresses far apart that no refused call touches
A, B, C, D, E, W = (0x100000000000 + (i << 42) for i in range(6))
BIG = (1 << 24) + 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def Z():
    import zero_partitioned_mixed_amd as Z
    return Z


def call(Z, name, defaults, **kw):
    assert set(kw) <= set(defaults), kw
    rc = getattr(Z._lib, name)(*{**defaults, **kw}.values(), None)
    if rc != 0:
        assert name in Z.zero_last_error()
    return rc


def test_sizes(Z):
    lib = Z._lib
    assert lib.zero_mx8_code_bytes(3, 129) == 3 * 256 and lib.zero_mx8_code_bytes(0, 5) == 0 == lib.zero_mx8_code_bytes(4, 0)
    rows = lib.zero_mx8_matmul_rows_workspace_bytes
    assert rows(1, 9, 8192) == 0 and rows(32, 9, 256) == 0 and rows(0, 9, 9) == 0 and rows(9, BIG, 9) == 0
    assert rows(33, 9, 128) == 33 * 128 + 128 + 256  # codes and scales, each to 256 bytes
    assert rows(2, 9, 16384) == 2 * 16384 + 1024
    norm = lib.zero_rms_norm_grad_workspace_bytes
    assert norm(0, 9) == 0 and norm(9, 0) == 0 and norm(BIG, 4) == 0 and norm(1, 9) == 36
    embed = lib.zero_embedding_grad_workspace_bytes
    assert embed(0, 9, 9) == 0 and embed(9, 9, 0) == 0 and embed(9, BIG, 9) == 0
    assert embed(1, 9, 9) == 4 * 64 and embed(8, 9, 9) == 4 * 64  # ids and where they came from
    assert embed(33, 9, 9) == 4 * (128 + 5 * 2 * 9)  # and two parts for each piece of the order
    sort = lib.zero_expert_sort_workspace_bytes
    assert sort(0, 9) == 0 and sort(4096, 511) == 0 and sort(4097, 8) == 4 * 3 * 512 and sort(9, BIG) == 0


QUANT = dict(src=A, dt=BF16, rows=4, cols=64, ld=64, codes=B, scales=C)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(dt=4), EINVAL), (dict(src=None), EINVAL), (dict(codes=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(src=A + 1), EALIGN), (dict(codes=B + 8), EALIGN), (dict(scales=C + 4), EALIGN), (dict(rows=-1), ERANGE),
    (dict(cols=BIG, ld=BIG), ERANGE), (dict(ld=63), ERANGE), (dict(codes=A + 256), EINVAL), (dict(scales=A), EINVAL)])
def test_quantize_refuses(Z, kw, code):
    assert call(Z, "zero_mx8_quantize", QUANT, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(codes=None), EINVAL), (dict(dst=None), EINVAL), (dict(codes=A + 1), EALIGN), (dict(dst=C + 1), EALIGN),
    (dict(rows=-2), ERANGE), (dict(ld=10), ERANGE), (dict(dst=A + 128), EINVAL)])
def test_dequantize_refuses(Z, kw, code):
    assert call(Z, "zero_mx8_dequantize", dict(codes=A, scales=B, rows=4, cols=64, dst=C, dt=F16, ld=64), **kw) == code


MATMUL = dict(a=A, sa=A + (1 << 30), b=B, sb=B + (1 << 30), m=8, n=8, k=64, c=C, cdt=BF16, ldc=8, acc=0)


@pytest.mark.parametrize("kw,code", [
    (dict(cdt=9), EINVAL), (dict(acc=2, cdt=F32), EINVAL), (dict(acc=1, cdt=F16), EINVAL), (dict(a=None), EINVAL), (dict(sa=None), EINVAL),
    (dict(sb=None), EINVAL), (dict(c=None), EINVAL), (dict(a=A + 8), EALIGN), (dict(b=B + 1), EALIGN), (dict(c=C + 1), EALIGN),
    (dict(ldc=7), ERANGE), (dict(m=-1), ERANGE), (dict(n=BIG), ERANGE), (dict(k=1 << 25), ERANGE), (dict(c=A + 1000), EINVAL),
    (dict(c=B), EINVAL)])
def test_matmul_refuses(Z, kw, code):
    assert call(Z, "zero_mx8_matmul", MATMUL, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(adt=0), EINVAL), (dict(a=None), EINVAL), (dict(b=None), EINVAL), (dict(ws=None), EINVAL), (dict(a=A + 1), EALIGN),
    (dict(ws=W + 4), EALIGN), (dict(lda=4095), ERANGE), (dict(wsb=1), ESPACE), (dict(acc=1), EINVAL), (dict(c=A + 2), EINVAL)])
def test_matmul_rows_refuses(Z, kw, code):
    a = dict(a=A, adt=BF16, lda=4096, b=B, sb=C, m=8, n=8, k=4096, c=D, cdt=BF16, ldc=8, acc=0, ws=W, wsb=1 << 40)
    assert call(Z, "zero_mx8_matmul_rows", a, **kw) == code


NORM = dict(x=A, dt=BF16, ldx=64, r=B, rdt=F32, ldr=64, w=C, tokens=4, cols=64, eps=1e-6)
OUT = dict(y=D, ldy=64, h=E, ldh=64)
OUT8 = dict(codes=D, scales=W, h=E, ldh=64)
REFUSED = [(dict(dt=0), EINVAL), (dict(rdt=F16), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(h=None), EINVAL),
           (dict(r=None), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=NAN), EINVAL), (dict(eps=INF), EINVAL), (dict(x=A + 1), EALIGN),
           (dict(r=B + 2), EALIGN), (dict(w=C + 1), EALIGN), (dict(h=E + 2), EALIGN), (dict(ldx=63), ERANGE), (dict(ldr=63), ERANGE),
           (dict(ldh=63), ERANGE), (dict(tokens=-1), ERANGE), (dict(cols=BIG, ldx=BIG, ldr=BIG, ldh=BIG), ERANGE),
           (dict(h=A + 64), EINVAL), (dict(h=B + 4), EINVAL), (dict(h=C), EINVAL)]


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(y=None), EINVAL), (dict(y=D + 1), EALIGN), (dict(ldy=63), ERANGE), (dict(y=A + 2), EINVAL), (dict(y=A, ldy=65), EINVAL),
    (dict(y=B), EINVAL), (dict(y=C), EINVAL), (dict(y=E), EINVAL)])
def test_norm_refuses(Z, kw, code):
    assert call(Z, "zero_rms_norm", {**NORM, **OUT}, **kw) == code


@pytest.mark.parametrize("kw,code", REFUSED + [
    (dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(codes=D + 8), EALIGN), (dict(scales=W + 1), EALIGN),
    (dict(codes=A + 16), EINVAL), (dict(scales=B), EINVAL), (dict(codes=E), EINVAL)])
def test_norm_mx8_refuses(Z, kw, code):
    assert call(Z, "zero_rms_norm_mx8", {**NORM, **OUT8}, **kw) == code


GRAD = dict(dy=A, lddy=64, h=B, hdt=F32, ldh=64, w=C, dt=BF16, dh=D, lddh=64, tokens=4, cols=64, eps=1e-6, dx=E, lddx=64,
            dr=E + (1 << 40), lddr=64, dw=E + (1 << 41), ws=W, wsb=1 << 40)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(hdt=F16), EINVAL), (dict(dy=None), EINVAL), (dict(h=None), EINVAL), (dict(w=None), EINVAL),
    (dict(eps=-0.5), EINVAL), (dict(dy=A + 1), EALIGN), (dict(h=B + 2), EALIGN), (dict(dh=D + 1), EALIGN), (dict(dx=E + 1), EALIGN),
    (dict(lddy=63), ERANGE), (dict(ldh=63), ERANGE), (dict(lddh=63), ERANGE), (dict(lddx=63), ERANGE), (dict(lddr=63), ERANGE),
    (dict(tokens=BIG), ERANGE), (dict(ws=None), EINVAL), (dict(ws=W + 8), EALIGN), (dict(wsb=1023), ESPACE), (dict(dx=A), EINVAL),
    (dict(dr=B), EINVAL), (dict(dr=D), EINVAL), (dict(dw=C), EINVAL)])
def test_norm_grad_refuses(Z, kw, code):
    assert call(Z, "zero_rms_norm_grad", GRAD, **kw) == code


DROP = dict(x=A, dt=BF16, ldx=64, r=B, ldr=64, rows=4, cols=64, p=0.5, seed=1, offset=2, dev=C, y=D, ldy=64)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), EINVAL), (dict(p=-0.1), EINVAL), (dict(p=1.0001), EINVAL), (dict(p=NAN), EINVAL), (dict(x=None), EINVAL),
    (dict(y=None), EINVAL), (dict(x=A + 1), EALIGN), (dict(r=B + 1), EALIGN), (dict(y=D + 1), EALIGN), (dict(dev=C + 4), EALIGN),
    (dict(ldx=63), ERANGE), (dict(ldr=63), ERANGE), (dict(ldy=63), ERANGE), (dict(rows=-1), ERANGE), (dict(rows=(1 << 32) + 1), ERANGE),
    (dict(rows=1 << 32, cols=1 << 9, ldx=512, ldy=512, ldr=512), ERANGE), (dict(y=A + 2), EINVAL), (dict(y=A, ldy=65), EINVAL),
    (dict(y=B + 2), EINVAL), (dict(y=C), EINVAL)])
def test_dropout_refuses(Z, kw, code):
    assert call(Z, "zero_dropout", DROP, **kw) == code


LOOKUP = dict(ids=A, size=8, tokens=5, table=B, dt=F32, ldt=64, vocab=10, cols=64, scale=1.0, out=C, ldo=64)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(size=2), EINVAL), (dict(ids=None), EINVAL), (dict(table=None), EINVAL), (dict(out=None), EINVAL),
    (dict(ids=A + 4), EALIGN), (dict(table=B + 2), EALIGN), (dict(out=C + 1), EALIGN), (dict(tokens=-1), ERANGE), (dict(tokens=BIG), ERANGE),
    (dict(vocab=0), ERANGE), (dict(vocab=BIG), ERANGE), (dict(ldt=63), ERANGE), (dict(ldo=63), ERANGE), (dict(out=B + 64), EINVAL),
    (dict(out=A), EINVAL)])
def test_embedding_refuses(Z, kw, code):
    assert call(Z, "zero_embedding", LOOKUP, **kw) == code


LOOKUP_GRAD = dict(ids=A, size=4, tokens=5, dy=B, dt=F32, lddy=64, vocab=10, cols=64, scale=1.0, out=C, ldo=64, ws=W, wsb=1 << 40)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(size=1), EINVAL), (dict(ids=None), EINVAL), (dict(dy=None), EINVAL), (dict(out=None), EINVAL),
    (dict(ids=A + 2), EALIGN), (dict(dy=B + 2), EALIGN), (dict(out=C + 2), EALIGN), (dict(vocab=0), ERANGE), (dict(lddy=1), ERANGE),
    (dict(ldo=63), ERANGE), (dict(ws=None), EINVAL), (dict(ws=W + 4), EALIGN), (dict(wsb=255), ESPACE), (dict(out=B), EINVAL),
    (dict(out=A), EINVAL)])
def test_embedding_grad_refuses(Z, kw, code):
    assert call(Z, "zero_embedding_grad", LOOKUP_GRAD, **kw) == code


SORT = dict(ids=A, size=8, slots=5000, experts=8, order=B, place=C, offsets=D, ws=W, wsb=1 << 40)


@pytest.mark.parametrize("kw,code", [
    (dict(size=3), EINVAL), (dict(ids=None), EINVAL), (dict(order=None), EINVAL), (dict(place=None), EINVAL), (dict(offsets=None), EINVAL),
    (dict(ids=A + 4), EALIGN), (dict(order=B + 2), EALIGN), (dict(slots=-1), ERANGE), (dict(slots=BIG), ERANGE), (dict(experts=0), ERANGE),
    (dict(experts=BIG), ERANGE), (dict(ws=None), EINVAL), (dict(ws=W + 8), EALIGN), (dict(wsb=4095), ESPACE), (dict(order=A + 8), EINVAL),
    (dict(offsets=A), EINVAL)])
def test_expert_sort_refuses(Z, kw, code):
    assert call(Z, "zero_expert_sort", SORT, **kw) == code


ROWS = dict(x=A, dt=F32, ldx=64, place=B, used=C, tokens=5, k=2, cols=64, rows=D, ldr=64)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(x=None), EINVAL), (dict(place=None), EINVAL), (dict(used=None), EINVAL), (dict(rows=None), EINVAL),
    (dict(x=A + 2), EALIGN), (dict(place=B + 2), EALIGN), (dict(rows=D + 2), EALIGN), (dict(k=0), ERANGE), (dict(k=1 << 23), ERANGE),
    (dict(tokens=-1), ERANGE), (dict(ldx=63), ERANGE), (dict(ldr=63), ERANGE), (dict(rows=A), EINVAL), (dict(rows=B), EINVAL)])
def test_expert_rows_refuses(Z, kw, code):
    assert call(Z, "zero_expert_rows", ROWS, **kw) == code


COMBINE = dict(rows=A, dt=BF16, ldr=64, place=B, used=C, w=E, wdt=F32, tokens=5, k=2, cols=64, y=D, ldy=64)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(wdt=F16), EINVAL), (dict(rows=None), EINVAL), (dict(y=None), EINVAL), (dict(place=None), EINVAL),
    (dict(w=E + 2), EALIGN), (dict(y=D + 1), EALIGN), (dict(ldr=1), ERANGE), (dict(ldy=1), ERANGE), (dict(k=0), ERANGE),
    (dict(y=A), EINVAL), (dict(y=E), EINVAL), (dict(y=B), EINVAL)])
def test_expert_combine_refuses(Z, kw, code):
    assert call(Z, "zero_expert_combine", COMBINE, **kw) == code


COMBINE_GRAD = dict(dy=A, lddy=64, rows=B, dt=BF16, ldr=64, place=C, used=C + (1 << 40), w=D, wdt=F32, tokens=5, k=2, cols=64, drows=E,
                    lddr=64, dw=W)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(wdt=F16), EINVAL), (dict(dy=None), EINVAL), (dict(rows=None), EINVAL), (dict(w=None), EINVAL),
    (dict(place=None), EINVAL), (dict(dw=W + 2), EALIGN), (dict(drows=E + 1), EALIGN), (dict(lddr=63), ERANGE), (dict(lddy=63), ERANGE),
    (dict(ldr=63), ERANGE), (dict(drows=A), EINVAL), (dict(drows=B), EINVAL), (dict(dw=D), EINVAL), (dict(dw=A), EINVAL)])
def test_expert_combine_grad_refuses(Z, kw, code):
    assert call(Z, "zero_expert_combine_grad", COMBINE_GRAD, **kw) == code


def test_nothing_to_do(Z):
    for name, a, kws in [
            ("zero_mx8_quantize", QUANT, [dict(rows=0), dict(cols=0)]), ("zero_mx8_matmul", MATMUL, [dict(m=0), dict(n=0)]),
            ("zero_rms_norm", {**NORM, **OUT}, [dict(tokens=0), dict(cols=0)]),
            ("zero_rms_norm_grad", GRAD, [dict(cols=0), dict(dx=None, dr=None, dw=None), dict(tokens=0, dw=None)]),
            ("zero_dropout", DROP, [dict(rows=0), dict(cols=0)]), ("zero_embedding", LOOKUP, [dict(tokens=0), dict(cols=0)]),
            ("zero_embedding_grad", LOOKUP_GRAD, [dict(cols=0)]), ("zero_expert_rows", ROWS, [dict(tokens=0), dict(cols=0)]),
            ("zero_expert_combine", COMBINE, [dict(tokens=0), dict(cols=0)]),
            ("zero_expert_combine_grad", COMBINE_GRAD, [dict(tokens=0), dict(drows=None, dw=None)])]:
        for kw in kws:
            assert call(Z, name, a, **kw) == 0, (name, kw)
    assert Z.zero_last_error() == ""


def test_cpu_tensors_refused(Z):
    import torch
    x, w, ids = torch.zeros(4, 64), torch.zeros(64), torch.zeros(4, 2, dtype=torch.int64)
    numbers = torch.zeros(8, dtype=torch.int32)
    plan = Z.ExpertPlan(numbers, numbers.view(4, 2), numbers[:4], 4, 2, 3)
    for call_ in (lambda: Z.mx8_quantize(x), lambda: Z.mx8_dequantize(Z.MX8.alloc(4, 64, "cpu")), lambda: Z.rms_norm(x, w),
                  lambda: Z.mx8_matmul(x, Z.MX4.alloc(4, 64, "cpu")), lambda: Z.rms_norm(x, w, x), lambda: Z.rms_norm_mx8(x, w),
                  lambda: Z.dropout(x, 0.5, 1), lambda: Z.embedding(ids, x), lambda: Z.expert_sort(ids, 3),
                  lambda: Z.expert_rows(x, plan), lambda: Z.expert_combine(x[:1].expand(8, 64), ids.float(), plan)):
        with pytest.raises(ValueError):
            call_()
    with pytest.raises(ValueError):
        Z.MX8(torch.zeros(4, 127, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64)
    q = Z.MX8(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64)
    assert q.codes.shape == (4, 128) and ctypes.sizeof(ctypes.c_void_p) == 8


def test_plans_refused(Z):
    import torch
    n = torch.zeros(8, dtype=torch.int32)
    Z.ExpertPlan(n, n.view(4, 2), n[:4], 4, 2, 3)
    for order, place, offsets in ((n[:7], n, n[:4]), (n, n[:6], n[:4]), (n, n, n[:3]), (n.long(), n, n[:4]), (n, n.long(), n[:4]),
                                  (n, n, n[:4].float()), (n, n.expand(2, 8)[:, :4], n[:4]), (n, n, n[::2])):
        with pytest.raises(ValueError):
            Z.ExpertPlan(order, place, offsets, 4, 2, 3)


def test_launches_past_32_bits_refused(Z):
    # 2^24 rows of 256 threads; the addresses are far enough apart for rows of 4096 bytes
    n, cols = 1 << 24, 2048
    rows = dict(tokens=n, cols=cols)
    assert call(Z, "zero_rms_norm", {**NORM, **OUT}, rdt=BF16, ldx=cols, ldr=cols, ldy=cols, ldh=cols, **rows) == ERANGE
    assert call(Z, "zero_rms_norm_mx8", {**NORM, **OUT8}, rdt=BF16, ldx=cols, ldr=cols, ldh=cols, **rows) == ERANGE
    assert call(Z, "zero_embedding", LOOKUP, ldt=cols, ldo=cols, **rows) == ERANGE


def test_tangents_are_not_lost(Z, monkeypatch):
    """In forward mode, where no input requires a gradient, the calls raise as torch's own do without a formula,
    rather than return a result without its tangent.  The C calls stubbed out."""
    import torch
    import torch.autograd.forward_ad as forward_ad
    from zero_partitioned_mixed_amd import tokens as M
    monkeypatch.setattr(M, "_gpu", lambda *t: 0)
    monkeypatch.setattr(M, "_call", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    x, w, numbers = torch.ones(8, 64), torch.ones(64), torch.zeros(8, dtype=torch.int32)
    plan, ids, gates = Z.ExpertPlan(numbers, numbers.view(8, 1), numbers[:4], 8, 1, 3), torch.zeros(5, dtype=torch.int64), torch.ones(8, 1)
    calls = [(lambda t: Z.rms_norm(t, w), x), (lambda t: Z.rms_norm(x, t), w), (lambda t: Z.rms_norm(x, w, t), x),
             (lambda t: Z.dropout(t, 0.5, 1), x), (lambda t: Z.dropout(x, 0.5, 1, residual=t), x), (lambda t: Z.embedding(ids, t), x),
             (lambda t: Z.expert_rows(t, plan), x), (lambda t: Z.expert_combine(t, gates, plan), x),
             (lambda t: Z.expert_combine(x, t, plan), gates)]
    for call_, t in calls:
        with forward_ad.dual_level():
            call_(t)  # without a tangent as ever
            for recorded in (torch.enable_grad, torch.no_grad):
                with recorded(), pytest.raises(RuntimeError, match="jvp"):
                    call_(forward_ad.make_dual(t, torch.ones_like(t)))
        call_(t)


@pytest.mark.parametrize("name,defaults,kw", [
    ("zero_mx8_quantize", QUANT, dict(scales=B)), ("zero_mx8_quantize", QUANT, dict(codes=C - 496)),
    ("zero_rms_norm_mx8", {**NORM, **OUT8}, dict(scales=D + 496)),
    ("zero_rms_norm_grad", GRAD, dict(dr=E)), ("zero_rms_norm_grad", GRAD, dict(dw=E + 256)),
    ("zero_rms_norm_grad", GRAD, dict(dw=E + (1 << 40) + 64)), ("zero_rms_norm_grad", GRAD, dict(dx=W)),
    ("zero_rms_norm_grad", GRAD, dict(dr=W + 1020)), ("zero_rms_norm_grad", GRAD, dict(dw=W + 16)),
    ("zero_rms_norm_grad", GRAD, dict(ws=A)), ("zero_rms_norm_grad", GRAD, dict(ws=B + 16)), ("zero_rms_norm_grad", GRAD, dict(ws=C)),
    ("zero_rms_norm_grad", GRAD, dict(ws=D - 1008)),
    ("zero_mx8_matmul_rows", dict(a=A, adt=BF16, lda=4096, b=B, sb=C, m=8, n=8, k=4096, c=D, cdt=BF16, ldc=8, acc=0, ws=D, wsb=1 << 40), {}),
    ("zero_mx8_matmul_rows", dict(a=A, adt=BF16, lda=4096, b=B, sb=C, m=8, n=8, k=4096, c=D, cdt=BF16, ldc=8, acc=0, ws=A + 16, wsb=1 << 40), {}),
    ("zero_mx8_matmul_rows", dict(a=A, adt=BF16, lda=4096, b=B, sb=C, m=8, n=8, k=4096, c=D, cdt=BF16, ldc=8, acc=0, ws=B, wsb=1 << 40), {}),
    ("zero_mx8_matmul_rows", dict(a=A, adt=BF16, lda=4096, b=B, sb=C, m=8, n=8, k=4096, c=D, cdt=BF16, ldc=8, acc=0, ws=C, wsb=1 << 40), {}),
    ("zero_embedding_grad", LOOKUP_GRAD, dict(ws=A)), ("zero_embedding_grad", LOOKUP_GRAD, dict(ws=B)),
    ("zero_embedding_grad", LOOKUP_GRAD, dict(ws=C + 2544)),
    ("zero_expert_sort", SORT, dict(order=C)), ("zero_expert_sort", SORT, dict(place=D + 4)), ("zero_expert_sort", SORT, dict(offsets=B + 400)),
    ("zero_expert_sort", SORT, dict(ws=A)), ("zero_expert_sort", SORT, dict(ws=B)), ("zero_expert_sort", SORT, dict(ws=C + 19984)),
    ("zero_expert_sort", SORT, dict(offsets=W + 4)),
    ("zero_expert_combine_grad", COMBINE_GRAD, dict(dw=E)), ("zero_expert_combine_grad", COMBINE_GRAD, dict(dw=E + 1276))])
def test_results_and_workspaces_share_nothing(Z, name, defaults, kw):
    """Two results of a call, or its workspace and anything else of its, in the same memory."""
    assert call(Z, name, defaults, **kw) == EINVAL


def test_plans_are_guarded(Z, monkeypatch):
    """A plan's memory may not be written between a forward pass and its backward pass.  The C calls stubbed out."""
    import torch
    from zero_partitioned_mixed_amd import tokens as M
    monkeypatch.setattr(M, "_gpu", lambda *t: 0)
    monkeypatch.setattr(M, "_call", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    x, gates = torch.ones(8, 64).requires_grad_(), torch.ones(8, 1).requires_grad_()
    for call_ in (lambda p: Z.expert_rows(x, p), lambda p: Z.expert_combine(x, gates, p)):
        for touched in (None, "place", "offsets"):
            n = torch.zeros(8, dtype=torch.int32)
            plan = Z.ExpertPlan(n, n.clone().view(8, 1), n[:4].clone(), 8, 1, 3)
            y = call_(plan)
            if touched is None:
                torch.autograd.grad(y, x, torch.ones_like(y))
                continue
            getattr(plan, touched).add_(1)
            with pytest.raises(RuntimeError, match="inplace"):
                torch.autograd.grad(y, x, torch.ones_like(y))
