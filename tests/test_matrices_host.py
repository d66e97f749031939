"""The matrix calls' sizes and refusals, on the host: every argument error is
returned before anything is enqueued, so no GPU is needed."""
import ctypes
import os
import random
import subprocess
import sys

import pytest

EINVAL, EALIGN, ERANGE, ESPACE = -1, -2, -3, -4
F16, BF16, F32 = 1, 2, 3
P = 0x10000  # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def Z():
    import zero_partitioned_mixed_amd as Z
    return Z


def ns(Z, **kw):
    return ctypes.byref(Z.newton_schulz(**kw))


def test_struct_sizes(Z):
    assert ctypes.sizeof(Z.NewtonSchulz) == 20 and ctypes.sizeof(Z.MuonHparams) == 40


def test_sizes(Z):
    assert [Z._lib.zero_mx4_padded(c) for c in (-1, 0, 1, 128, 129)] == [0, 0, 128, 128, 256]
    assert Z._lib.zero_mx4_code_bytes(3, 129) == 3 * 128 and Z._lib.zero_mx4_scale_bytes(3, 129) == 3 * 8
    assert Z._lib.zero_mx4_code_bytes(0, 5) == 0 == Z._lib.zero_mx4_scale_bytes(5, 0)
    ws = Z._lib.zero_ns_workspace_bytes
    assert ws(5, 128, 128) == 0 and ws(0, 500, 500) == 0 and ws(1, 0, 9) == 0 and ws(1, 70000, 9) == 0
    one = ws(1, 129, 400)
    assert one > 129 * 400 * 4 and ws(7, 129, 400) == 7 * one and ws(1, 400, 129) == one
    assert ws(1, 65536, 65536) > 0


def ortho(Z, src=P, sdt=F32, count=1, rows=200, cols=300, sld=300, sst=60000, dst=P, ddt=BF16, dld=300, dst_st=60000,
          s=None, ws=P, ws_bytes=1 << 40):
    return Z._lib.zero_orthogonalize(src, sdt, count, rows, cols, sld, sst, dst, ddt, dld, dst_st,
                                     s if s is not None else ns(Z), ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(sdt=0), EINVAL), (dict(sdt=4), EINVAL), (dict(ddt=F32), EINVAL), (dict(src=None), EINVAL), (dict(dst=None), EINVAL),
    (dict(src=P + 2), EALIGN), (dict(dst=P + 1), EALIGN), (dict(sdt=F16, src=P + 1), EALIGN), (dict(count=-1), ERANGE),
    (dict(count=65536), ERANGE), (dict(rows=-1), ERANGE), (dict(cols=65537, sld=70000, dld=70000), ERANGE),
    (dict(sld=299), ERANGE), (dict(dld=299), ERANGE), (dict(count=2, sst=59999), ERANGE), (dict(count=2, dst_st=100), ERANGE),
    (dict(ws=None), EINVAL), (dict(ws=P + 8), EALIGN), (dict(ws_bytes=1000), ESPACE)])
def test_orthogonalize_refuses(Z, kw, code):
    assert ortho(Z, **kw) == code
    assert "zero_orthogonalize" in Z.zero_last_error()


@pytest.mark.parametrize("kw", [dict(steps=-1), dict(steps=65), dict(eps=-1.0), dict(eps=float("nan")),
                                dict(coeffs=(float("inf"), 0, 0)), dict(coeffs=(1, float("nan"), 0))])
def test_settings_refused(Z, kw):
    assert ortho(Z, s=ns(Z, **kw)) == EINVAL


def test_nothing_to_do(Z):
    for kw in (dict(count=0), dict(rows=0), dict(cols=0, sld=0, dld=0)):
        assert ortho(Z, src=None, dst=None, ws=None, **kw) == 0
    assert Z.zero_last_error() == ""


def muon(Z, master=P, mom=P, g=P, count=1, rows=200, cols=300, stride=60000, ctrl=None, gather=P, gdt=F16, offset=0, ws=P,
         ws_bytes=1 << 40, **hp):
    h = Z.muon_hparams(**hp)
    return Z._lib.zero_muon_step(master, mom, g, count, rows, cols, stride, ctypes.byref(h), ctrl, gather, gdt, offset, ws,
                                 ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(momentum=1.0), EINVAL), (dict(momentum=-0.1), EINVAL), (dict(momentum=float("nan")), EINVAL),
    (dict(lr=float("inf")), EINVAL), (dict(weight_decay=float("nan")), EINVAL), (dict(scale=2), EINVAL), (dict(steps=100), EINVAL),
    (dict(gdt=F32), EINVAL), (dict(master=None), EINVAL), (dict(mom=None), EINVAL), (dict(g=None), EINVAL),
    (dict(master=P + 2), EALIGN), (dict(gather=P + 1), EALIGN), (dict(ctrl=P + 4), EALIGN), (dict(offset=-1), ERANGE),
    (dict(count=2, stride=59999), ERANGE), (dict(rows=70000), ERANGE), (dict(ws_bytes=16), ESPACE)])
def test_muon_refuses(Z, kw, code):
    assert muon(Z, **kw) == code
    assert "zero_muon_step" in Z.zero_last_error()


def quant(Z, src=P, dt=BF16, rows=4, cols=64, ld=64, c=P, s=P, ct=P, st=P):
    return Z._lib.zero_mx4_quantize(src, dt, rows, cols, ld, c, s, ct, st, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), EINVAL), (dict(c=None), EINVAL), (dict(st=None), EINVAL), (dict(c=None, s=None, ct=None, st=None), EINVAL),
    (dict(src=None), EINVAL), (dict(src=P + 1), EALIGN), (dict(c=P + 8), EALIGN), (dict(st=P + 4), EALIGN), (dict(rows=-1), ERANGE),
    (dict(cols=(1 << 24) + 1, ld=1 << 25), ERANGE), (dict(ld=63), ERANGE)])
def test_quantize_refuses(Z, kw, code):
    assert quant(Z, **kw) == code
    assert "zero_mx4_quantize" in Z.zero_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(c=None), EINVAL), (dict(d=None), EINVAL), (dict(c=P + 1), EALIGN), (dict(d=P + 1), EALIGN),
    (dict(rows=-2), ERANGE), (dict(ld=10), ERANGE)])
def test_dequantize_refuses(Z, kw, code):
    a = dict(c=P, s=P, rows=4, cols=64, d=P, dt=F16, ld=64)
    a.update(kw)
    assert Z._lib.zero_mx4_dequantize(a["c"], a["s"], a["rows"], a["cols"], a["d"], a["dt"], a["ld"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(cdt=9), EINVAL), (dict(acc=2, cdt=F32), EINVAL), (dict(acc=1, cdt=F16), EINVAL), (dict(a=None), EINVAL),
    (dict(sb=None), EINVAL), (dict(c=None), EINVAL), (dict(a=P + 8), EALIGN), (dict(b=P + 1), EALIGN), (dict(c=P + 1), EALIGN),
    (dict(ldc=7), ERANGE), (dict(m=-1), ERANGE), (dict(k=1 << 25), ERANGE)])
def test_matmul_refuses(Z, kw, code):
    a = dict(a=P, sa=P, b=P, sb=P, m=8, n=8, k=64, c=P, cdt=BF16, ldc=8, acc=0)
    a.update(kw)
    assert Z._lib.zero_mx4_matmul(a["a"], a["sa"], a["b"], a["sb"], a["m"], a["n"], a["k"], a["c"], a["cdt"], a["ldc"],
                                  a["acc"], P, 1 << 40, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(adt=0), EINVAL), (dict(a=None), EINVAL), (dict(b=None), EINVAL), (dict(ws=None), EINVAL), (dict(a=P + 1), EALIGN),
    (dict(ws=P + 4), EALIGN), (dict(m=65), ERANGE), (dict(lda=63), ERANGE), (dict(wsb=1), ESPACE)])
def test_matmul_rows_refuses(Z, kw, code):
    a = dict(a=P, adt=BF16, lda=4096, b=P, sb=P, m=8, n=8, k=4096, c=P, cdt=BF16, ldc=8, ws=P, wsb=1 << 40)
    a.update(kw)
    assert Z._lib.zero_mx4_matmul_rows(a["a"], a["adt"], a["lda"], a["b"], a["sb"], a["m"], a["n"], a["k"], a["c"], a["cdt"],
                                       a["ldc"], a["ws"], a["wsb"], None) == code


def test_cpu_tensors_refused(Z):
    import torch
    x = torch.zeros(4, 64)
    for call in (lambda: Z.orthogonalize(x, torch.float16), lambda: Z.mx4_quantize(x),
                 lambda: Z.muon_step(x, x, x, Z.muon_hparams()), lambda: Z.mx4_linear(x, x),
                 lambda: Z.mx4_matmul(x, Z.MX4.alloc(4, 64, "cpu"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        Z.MX4(torch.zeros(4, 31, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64)


def linear(Z, x=P, ldx=64, w=P, ldw=64, dt=BF16, t=8, n=16, k=64, y=P, ldy=16, xt=P, wt=P, ws=P, wsb=1 << 40):
    return Z._lib.zero_mx4_linear(x, ldx, w, ldw, dt, t, n, k, y, ldy, xt, wt, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=0), EINVAL), (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(x=P + 1), EALIGN), (dict(y=P + 1), EALIGN), (dict(xt=P + 8), EALIGN), (dict(ws=P + 8), EALIGN), (dict(ldx=63), ERANGE),
    (dict(ldw=63), ERANGE), (dict(ldy=15), ERANGE), (dict(t=0), ERANGE), (dict(k=0), ERANGE), (dict(n=-1), ERANGE),
    (dict(wsb=100), ESPACE)])
def test_linear_refuses(Z, kw, code):
    assert linear(Z, **kw) == code
    assert "zero_mx4_linear" in Z.zero_last_error()


def grad(Z, dy=P, ld=16, dt=BF16, t=8, n=16, k=64, xt=P, wt=P, dx=P, ldx=64, dw=P, ldw=64, ws=P, wsb=1 << 40):
    return Z._lib.zero_mx4_linear_grad(dy, ld, dt, t, n, k, xt, wt, dx, ldx, dw, ldw, ws, wsb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=5), EINVAL), (dict(dy=None), EINVAL), (dict(xt=None), EINVAL), (dict(wt=None), EINVAL), (dict(ws=None), EINVAL),
    (dict(dy=P + 1), EALIGN), (dict(dw=P + 1), EALIGN), (dict(wt=P + 4), EALIGN), (dict(ld=15), ERANGE), (dict(ldx=63), ERANGE),
    (dict(ldw=1), ERANGE), (dict(t=0), ERANGE), (dict(wsb=8), ESPACE)])
def test_linear_grad_refuses(Z, kw, code):
    assert grad(Z, **kw) == code
    assert "zero_mx4_linear_grad" in Z.zero_last_error()


def test_linear_grad_of_nothing(Z):
    assert grad(Z, dx=None, dw=None, xt=None, wt=None, ws=None, wsb=0) == 0


def test_operand_sizes(Z):
    assert Z._lib.zero_mx4_operand_bytes(3, 129) == 512 + 256
    assert Z._lib.zero_mx4_operand_bytes(0, 129) == 0 == Z._lib.zero_mx4_operand_bytes(1, 1 << 25)
    assert Z._lib.zero_mx4_matmul_rows_workspace_bytes(1, 100, 4096) == 0
    assert Z._lib.zero_mx4_matmul_rows_workspace_bytes(64, 100, 4096) > 64 * 2048


# ----------------------------------------------------------------------------- several ranks with matrices
class Rows:
    """Stands in for a contribution tensor, and for any buffer that is only sliced."""

    def data_ptr(self):
        return id(self)

    def __getitem__(self, _):
        return self

    def view(self, *_):
        return self


def fake_rank(Z, cls, two_pass=True):
    st = object.__new__(cls)
    st.bucket, st.nranks, st.stride, st.valid_len, st.offset = 0, 2, 4096, 4096, 0
    st.dtype = st.gather_dtype = Z.F16
    st.hp, st.fused = Z.hparams(), not two_pass
    st.state, st.g, st.ctrl, st.ws, st.pair = (Rows(), Rows(), Rows()), Rows(), "ctrl", "ws", None
    st.muon, st.matrices, st.between, st.matrix_ws = "muon", [(0, 2, 8, 16)], [(256, 3840)], None
    st.exact = False
    return st


def test_several_ranks_with_matrices(Z, monkeypatch):
    """The batched calls know nothing of matrices: ranks that hold some take their own calls, the matrix step among
    them, also beside ranks that hold none."""
    from zero_partitioned_mixed_amd import matrices
    calls = []
    names = ("zero_reduce_grads", "zero_reduce_grads_shards", "zero_adam_step", "zero_adam_step_shards",
             "zero_grad_norm_overflow")
    for name in names:
        monkeypatch.setattr(Z, name, lambda *a, _n=name, **k: calls.append(_n))
    monkeypatch.setattr(Z, "shard_table", lambda shards: list(shards))
    for name in ("zero_adam_step", "muon_step"):
        monkeypatch.setattr(matrices, name, lambda *a, _n=name, **k: calls.append(_n))
    for other, last in ((Z.MuonShardStep, ["zero_adam_step", "muon_step"]), (Z.ShardStep, ["zero_adam_step"])):
        calls.clear()
        multi = Z.MultiShardStep([fake_rank(Z, Z.MuonShardStep), fake_rank(Z, other)])
        rows = [Rows(), Rows()]
        assert not multi.takes_batched(rows, Rows())
        multi.step(rows, Rows())
        assert calls == ["zero_reduce_grads"] * 2 + ["zero_grad_norm_overflow", "zero_adam_step", "muon_step"] + last
    with pytest.raises(ValueError):  # the fused path's decision is not the two-pass path's
        Z.MultiShardStep([fake_rank(Z, Z.MuonShardStep), fake_rank(Z, Z.ShardStep, two_pass=False)])


# ----------------------------------------------------------------------------- results over what is read
@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    """The library's own predicate of two places, built for the host alone."""
    folder = tmp_path_factory.mktemp("overlap")
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "zero_partitioned_mixed_amd", "csrc")
    (folder / "o.cpp").write_text("""#include "zero_internal.h"
        extern "C" int meet(const int64_t* p) {
            auto place = [](const int64_t* q) { return Place((const void*)q[0], q[1], q[2], q[3], q[4], q[5]); };
            return overlap(place(p), place(p + 6)); }""")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-shared", "-fPIC", "-I", csrc, "-o", "o.so", "o.cpp"],
                   cwd=folder, check=True)
    meet = ctypes.CDLL(str(folder / "o.so")).meet
    return lambda *p: bool(meet((ctypes.c_int64 * 12)(*p)))


def test_overlap_by_comparing_bytes(overlap):
    """Random stacks of strided runs against their bytes: runs that lie between each other are apart."""
    rng = random.Random(3)
    seen = [0, 0]

    def place(like):
        rows, width, count = rng.choice([1, 2, 5]), rng.randint(1, 9), rng.choice([1, 1, 3])
        ld = like[3] if like and rng.random() < 0.6 and like[3] >= width else rng.randint(width, width + 12)
        span = (rows - 1) * ld + width
        stride = like[5] if like and rng.random() < 0.6 and like[5] >= span else span + rng.randint(0, 20)
        return [1000 + rng.randint(-150, 150), rows, width, ld, count, stride]

    def taken(p):
        at, rows, width, ld, count, stride = p
        return {at + c * stride + r * ld + b for c in range(count) for r in range(rows) for b in range(width)}

    for _ in range(20000):
        p = place(None)
        q = place(p)
        meet = not taken(p).isdisjoint(taken(q))
        assert overlap(*p, *q) == meet == overlap(*q, *p), (p, q)
        seen[meet] += 1
    assert min(seen) > 3000
    assert not overlap(0, 1, 8, 8, 1, 8, 0, 1, 8, 8, 1, 8)  # null
    assert not overlap(1000, 0, 8, 8, 1, 8, 1000, 1, 8, 8, 1, 8)
    far = 1 << 40  # large matrices, far apart and not, at once
    assert not overlap(far, 1 << 24, 100, 400, 1, 0, far + 100, 1 << 24, 300, 400, 1, 0)
    assert not overlap(far, 1 << 20, 1, 64, 1, 0, far + 32, 1 << 20, 1, 128, 1, 0)
    assert overlap(far, 1 << 20, 1, 64, 1, 0, far + 32, 1 << 20, 33, 128, 1, 0)
    for at, meet in ((65535 << 34, False), ((65535 << 34) - 1, True), (0, True), (-1, False)):
        assert overlap(far, 65536, 1 << 18, 1 << 18, 65535, 1 << 34, far + at, 1, 1, 1, 1, 1) == meet


def test_overlaps_refused(Z):
    big = 1 << 30
    over = dict(ws=8 * big, ws_bytes=1 << 40)
    for kw in (dict(sdt=F32), dict(sdt=BF16, dld=301), dict(sdt=BF16, dst=P + 600), dict(sdt=BF16, dst=P - 2)):
        assert ortho(Z, src=P, **{"dst": P, **kw}, **over) == EINVAL
    for kw in (dict(mom=P), dict(g=P + 4 * 59999), dict(gather=P + 4), dict(g=big + 16)):
        kw = {**dict(master=P, mom=big, g=2 * big, gather=None, gdt=BF16), **kw}
        assert muon(Z, **kw, **over) == EINVAL
    # matrices of one buffer, into the others' of it
    assert muon(Z, count=3, stride=180000, master=big, mom=big + 4 * 60000, g=big + 4 * 119999, gather=None, **over) == EINVAL
    assert quant(Z, src=P, c=P, s=big, ct=None, st=None) == EINVAL
    assert quant(Z, src=P, c=big, s=2 * big, ct=3 * big, st=P + 512 - 16) == EINVAL
    assert Z._lib.zero_mx4_dequantize(P, big, 4, 64, P + 16, F16, 64, None) == EINVAL
    assert Z._lib.zero_mx4_matmul(P, big, 2 * big, 3 * big, 8, 8, 64, P + 48, F16, 8, 0, None, 0, None) == EINVAL
    assert Z._lib.zero_mx4_matmul(P, big, 2 * big, 3 * big, 8, 8, 64, 3 * big, F16, 8, 0, None, 0, None) == EINVAL
    for m, k in ((1, 64), (32, 64), (33, 64), (8, 5000)):
        rows = lambda c, ldc=64: Z._lib.zero_mx4_matmul_rows(P, BF16, k, big, 2 * big, m, 64, k, c, BF16, ldc, 3 * big,  # noqa: E731
                                                             1 << 40, None)
        assert rows(P) == rows(P + 2 * m * k - 2) == rows(P - 2, 6400) == rows(big) == rows(2 * big) == EINVAL
    assert grad(Z, dy=P, xt=big, wt=2 * big, dx=big, dw=3 * big, ws=4 * big) == EINVAL
    assert linear(Z, x=P, w=big, y=2 * big, xt=P, wt=3 * big, ws=4 * big) == EINVAL
    assert "overlap" in Z.zero_last_error()


def test_workspace_of_scattered_bytes_refused(Z, monkeypatch):
    """A strided tensor holds fewer bytes from its address on than it has elements."""
    import torch
    from zero_partitioned_mixed_amd import matrices
    monkeypatch.setattr(matrices, "_gpu", lambda *t: 0)
    space = torch.zeros(64, dtype=torch.float32)
    pointer, size, _ = matrices._space(100, space[8:40], space)
    assert (pointer, size) == (space.data_ptr() + 32, 128)
    for ws in (space[::2], space.view(8, 8).t(), space.view(8, 8)[:, :4]):
        with pytest.raises(ValueError, match="contiguous"):
            matrices._space(16, ws, space)


def test_linear_without_gradients_keeps_nothing(Z, monkeypatch):
    """Where torch does not record, the forward call is asked for no operands of the gradients, whatever its inputs
    require; where it does, for those of the gradients that are wanted."""
    import torch
    from zero_partitioned_mixed_amd import matrices
    calls, kept = [], []
    monkeypatch.setattr(matrices, "_gpu", lambda *t: 0)
    monkeypatch.setattr(matrices, "_call", lambda index, name, *a: calls.append((name, a[10], a[11])))
    monkeypatch.setattr(matrices, "_empty", lambda *a, **k: kept.append(torch.empty(*a, **k)) or kept[-1])
    x, w = torch.randn(8, 64, requires_grad=True), torch.randn(16, 64, requires_grad=True)

    def wanted(x, w):
        calls.clear(), kept.clear()
        Z.mx4_linear(x, w)
        (name, x_t, w_t), = calls
        assert name == "zero_mx4_linear"
        size = Z._lib.zero_mx4_operand_bytes(64, 8) * (x_t is not None) + Z._lib.zero_mx4_operand_bytes(64, 16) * (w_t is not None)
        # the result and the call's workspace, and what is kept for the gradients
        assert [t.numel() for t in kept] == [8 * 16] + [size] * (size > 0) + [Z._lib.zero_mx4_linear_workspace_bytes(8, 16, 64)]
        return x_t is not None, w_t is not None

    assert wanted(x, w) == (True, True)
    assert wanted(x, w.detach()) == (False, True) and wanted(x.detach(), w) == (True, False)
    assert wanted(x.detach(), w.detach()) == (False, False)
    for mode in (torch.no_grad(), torch.inference_mode()):
        with mode:
            assert wanted(x, w) == (False, False)
            assert wanted(x.detach(), w) == (False, False)


def test_coefficients_that_leave_the_range_refused(Z):
    """Against the largest value on a fine grid, step by step; too small a workspace ends what is taken."""
    import numpy as np

    def reach(a, b, c, steps):
        r = top = 1.0
        for _ in range(steps - 1):
            s = np.linspace(0.0, r, 2001)
            r = float(np.abs(a * s + b * s ** 3 + c * s ** 5).max())
            top = max(top, r)
            if top > 100:
                break
        return top

    rng = random.Random(6)
    seen = [0, 0]
    for _ in range(1000):
        coeffs = rng.uniform(-4, 4), rng.choice([0.0, rng.uniform(-6, 6)]), rng.choice([0.0, rng.uniform(-4, 4)])
        steps = rng.randint(0, 6)
        top = reach(*coeffs, steps)
        if abs(top - 3.5) < 0.01:
            continue
        taken = top < 3.5
        assert ortho(Z, s=ns(Z, coeffs=coeffs, steps=steps), ws_bytes=0) == (ESPACE if taken else EINVAL), (coeffs, steps, top)
        assert muon(Z, coeffs=coeffs, steps=steps, ws_bytes=0) == (ESPACE if taken else EINVAL)
        seen[taken] += 1
    assert min(seen) > 200
    for usual in ((3.4445, -4.7750, 2.0315), (1.5, -0.5, 0.0), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)):
        assert ortho(Z, s=ns(Z, coeffs=usual, steps=64), ws_bytes=0) == ESPACE


def test_import_without_torch_internals():
    """The package needs no private name of torch."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'): del torch._C._cuda_getCurrentRawStream\n"
            "import zero_partitioned_mixed_amd as Z\n"
            "class Stream: cuda_stream = 77\n"
            "torch.cuda.current_stream = lambda index=None: Stream\n"
            "from zero_partitioned_mixed_amd import matrices\n"
            "assert matrices._raw_stream(0) == 77")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_payload_with_matrices_refused_before_the_step(Z, monkeypatch):
    """Nothing is enqueued: a decision made before the refusal would have counted the step."""
    calls = []
    for name in ("zero_reduce_grads", "zero_grad_norm_overflow"):
        monkeypatch.setattr(Z, name, lambda *a, _n=name, **k: calls.append(_n))
    payload = Z.QGather(1 << 24, 1 << 25, 8, 4096)
    with pytest.raises(ValueError, match="payload"):
        fake_rank(Z, Z.MuonShardStep).step(Rows(), Rows(), payload)
    with pytest.raises(ValueError, match="payload"):
        Z.MultiShardStep([fake_rank(Z, Z.MuonShardStep)]).step([Rows()], Rows(), [payload])
    assert calls == []


def test_workspace_of_the_step(Z):
    """Never more than an orthogonalisation's, and the same where every operand has two parts anyway."""
    ns_bytes, muon_bytes = Z._lib.zero_ns_workspace_bytes, Z._lib.zero_muon_workspace_bytes
    for size in ((1, 129, 400), (3, 700, 300), (2, 5000, 5000)):
        assert 0 < muon_bytes(*size) < ns_bytes(*size)
    for size in ((5, 128, 128), (1, 20, 33000), (2, 3000, 60)):
        assert muon_bytes(*size) == ns_bytes(*size)
    for size in ((0, 500, 500), (1, 0, 9), (1, 70000, 9), (-1, 5, 5), (65536, 5, 5)):
        assert muon_bytes(*size) == 0
    size = muon_bytes(1, 200, 300)
    assert muon(Z, ws_bytes=size - 1) == ESPACE
    hp = Z.muon_hparams()
    assert Z._lib.zero_muon_step_exact(P, P, P, 1, 200, 300, 60000, ctypes.byref(hp), None, P, F16, 0, P, size, None) == ESPACE
    assert "zero_muon_step_exact" in Z.zero_last_error()
    assert ortho(Z, dst=1 << 40, ddt=BF16, ws_bytes=size - 1) == ESPACE == ortho(Z, dst=1 << 40, ddt=F16, ws_bytes=size)


def test_ranks_of_another_pass_take_their_own_calls(Z, monkeypatch):
    """A class that replaces either part of the step is not what the batched calls stand for."""
    monkeypatch.setattr(Z, "shard_table", lambda shards: list(shards))

    class Pass(Z.ShardStep):
        def run_pieces(self, *a, **k):
            pass

    class Named(Z.ShardStep):
        name = "a rank"

    for cls, batched in ((Pass, False), (Named, True), (Z.ShardStep, True)):
        assert Z.MultiShardStep([fake_rank(Z, cls), fake_rank(Z, Z.ShardStep)]).takes_batched([Rows(), Rows()], Rows()) == batched
