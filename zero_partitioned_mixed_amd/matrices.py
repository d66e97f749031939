"""The matrix calls on torch tensors: orthogonalised updates (Newton-Schulz) and
MXFP4 operands with their products.

Argument marshalling only, as in the package's other calls: every function
checks its tensors, passes their pointers to the C calls of the same name
(include/zero_shard.h) and enqueues on torch's current stream of the tensors'
device.  Outputs and workspaces that are not passed in come from torch's
allocator, which keeps memory by stream.
"""
from __future__ import annotations

import ctypes

import torch

from . import (BF16, F16, F32, MUON_SCALE_RMS, MUON_SCALE_SHAPE, MX4_ROWS_MAX,  # noqa: F401
               MuonHparams, NewtonSchulz, _check, _lib, _vp)

_DTYPES = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
COEFFS = (3.4445, -4.7750, 2.0315)  # the usual quintic's


def _code(dtype, allowed=_DTYPES) -> int:
    if dtype not in allowed:
        raise TypeError(f"dtype {dtype} is not one of {', '.join(str(d) for d in allowed)}")
    return _DTYPES[dtype]


_HALVES = (torch.float16, torch.bfloat16)


def _gpu(*tensors) -> None:
    dev = tensors[0].device
    for t in tensors:
        if not t.is_cuda:
            raise ValueError("expected a GPU tensor")
        if t.device != dev:
            raise ValueError("tensors on different GPUs")


def _stream(t) -> ctypes.c_void_p:
    return _vp(torch.cuda.current_stream(t.device).cuda_stream)


class _on:
    """The tensor's device as the current one (launches go to it)."""

    def __init__(self, t):
        self.dev = t.device
        self.swap = None

    def __enter__(self):
        if torch.cuda.current_device() != self.dev.index:
            self.swap = torch.cuda.device(self.dev)
            self.swap.__enter__()

    def __exit__(self, *exc):
        if self.swap is not None:
            self.swap.__exit__(*exc)


def _space(nbytes: int, ws, like):
    """(pointer, bytes, tensor) of a workspace: ws, or a new tensor."""
    if ws is None:
        if nbytes == 0:
            return _vp(None), 0, None
        ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    else:
        _gpu(like, ws)
    return _vp(ws.data_ptr()), ws.numel() * ws.element_size(), ws


# ----------------------------------------------------------------------------- orthogonalised updates
def newton_schulz(coeffs=COEFFS, steps: int = 5, eps: float = 1e-7) -> NewtonSchulz:
    a, b, c = coeffs
    return NewtonSchulz(a, b, c, eps, steps)


def muon_hparams(lr=3e-4, momentum=0.95, weight_decay=0.0, nesterov=True, scale=MUON_SCALE_RMS,
                 coeffs=COEFFS, steps=5, eps=1e-7) -> MuonHparams:
    return MuonHparams(lr, momentum, weight_decay, int(bool(nesterov)), scale,
                       newton_schulz(coeffs, steps, eps))


def _stack(x):
    """(count, rows, cols, row stride, matrix stride) of [rows, cols] or [count, rows, cols]."""
    if x.dim() not in (2, 3):
        raise ValueError("expected [rows, cols] or [count, rows, cols]")
    count = x.shape[0] if x.dim() == 3 else 1
    rows, cols = x.shape[-2:]
    ld = x.stride(-2) if rows > 1 else max(x.stride(-2), cols)
    stride = x.stride(0) if x.dim() == 3 and count > 1 else rows * ld
    return count, rows, cols, ld, stride


def _laid_out(x) -> bool:
    """Rows of unit stride that do not overlap, matrices that do not overlap."""
    if x.numel() == 0:
        return True
    _, rows, cols, ld, stride = _stack(x)
    return (cols == 1 or x.stride(-1) == 1) and ld >= cols and stride >= (rows - 1) * ld + cols


def orthogonalize(x, out_dtype=None, *, coeffs=COEFFS, steps: int = 5, eps: float = 1e-7, out=None,
                  ws=None):
    """The Newton-Schulz orthogonalisation of every matrix of x ([rows, cols] or
    [count, rows, cols]; fp16, bf16 or fp32, any strides: other layouts than
    unit-stride rows are copied).  Returns fp16 or bf16 (out_dtype; by default x's
    type, bf16 for fp32), in ``out`` when given (it may be x).  Not differentiable."""
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = torch.bfloat16 if x.dtype == torch.float32 else x.dtype
    src_code, dst_code = _code(x.dtype), _code(out_dtype, _HALVES)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    _gpu(x, out)
    if out.shape != x.shape or not _laid_out(out):
        raise ValueError("out: another shape, or rows without unit stride")
    if not _laid_out(x):
        x = x.contiguous()
    count, rows, cols, ld, stride = _stack(x)
    _, _, _, out_ld, out_stride = _stack(out)
    ns = newton_schulz(coeffs, steps, eps)
    with _on(x):
        p, n, _keep = _space(_lib.zero_ns_workspace_bytes(count, rows, cols), ws, x)
        _check("zero_orthogonalize", _lib.zero_orthogonalize(
            x.data_ptr(), src_code, count, rows, cols, ld, stride, out.data_ptr(), dst_code,
            out_ld, out_stride, ctypes.byref(ns), p, n, _stream(x)))
    return out


def muon_step(master, mom, g, hp: MuonHparams, *, slot=None, ctrl=None, ws=None) -> None:
    """One optimizer step, in place, for the matrices of master ([rows, cols] or
    [count, rows, cols] fp32, matrices contiguous; mom and g alike, usually
    views of a shard's flat buffers).  slot: the fp16 or bf16 parameters laid
    out like master (a view of the gather buffer).  ctrl: the rank's control
    block, whose clip and skip then apply."""
    for t in (master, mom, g):
        _code(t.dtype, (torch.float32,))
    tensors = [master, mom, g] + [t for t in (slot, ctrl) if t is not None]
    _gpu(*tensors)
    for t in [master, mom, g] + ([slot] if slot is not None else []):
        if t.shape != master.shape or not _laid_out(t):
            raise ValueError("master, mom, g and slot take one shape and layout")
    count, rows, cols, ld, stride = _stack(master)
    if master.numel() and (ld != cols or any(_stack(t)[3:] != (ld, stride)
                                             for t in tensors[1:3] + ([slot] if slot is not None else []))):
        raise ValueError("master, mom, g and slot: contiguous matrices at one stride")
    with _on(master):
        p, n, _keep = _space(_lib.zero_ns_workspace_bytes(count, rows, cols), ws, master)
        _check("zero_muon_step", _lib.zero_muon_step(
            master.data_ptr(), mom.data_ptr(), g.data_ptr(), count, rows, cols, stride,
            ctypes.byref(hp), None if ctrl is None else ctrl.data_ptr(),
            None if slot is None else slot.data_ptr(),
            F16 if slot is None else _code(slot.dtype, _HALVES), 0, p, n, _stream(master)))


# ----------------------------------------------------------------------------- MXFP4
class MX4:
    """A rows x cols matrix in MXFP4, blocks of 32 along its rows: codes
    [rows, P / 2] and scales [rows, P / 32] bytes, P = mx4 padded cols (a multiple of
    128, the padding zero)."""

    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes, scales, rows: int, cols: int):
        p = (cols + 127) // 128 * 128
        for t, width, what in ((codes, p // 2, "codes"), (scales, p // 32, "scales")):
            if t.dtype != torch.uint8 or t.numel() != rows * width or not t.is_contiguous():
                raise ValueError(f"{what}: {rows * width} contiguous bytes for {rows} x {cols}")
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, cols

    @staticmethod
    def alloc(rows: int, cols: int, device) -> "MX4":
        p = (cols + 127) // 128 * 128
        return MX4(torch.empty((rows, p // 2), dtype=torch.uint8, device=device),
                   torch.empty((rows, p // 32), dtype=torch.uint8, device=device), rows, cols)


def _matrix(x):
    """x as unit-stride rows, and its row stride."""
    if x.dim() != 2:
        raise ValueError("expected a matrix")
    if not _laid_out(x):
        x = x.contiguous()
    return x, _stack(x)[3]


def mx4_quantize(x, rows: bool = True, cols: bool = False):
    """x (fp16, bf16 or fp32 matrix) as MX4 along its rows, along its columns (the
    quantisation of x's transpose), or both from one read: MX4, or (along
    rows, along columns)."""
    code = _code(x.dtype)
    if not rows and not cols:
        raise ValueError("neither rows nor columns")
    _gpu(x)
    x, ld = _matrix(x)
    m, n = x.shape
    r = MX4.alloc(m, n, x.device) if rows else None
    c = MX4.alloc(n, m, x.device) if cols else None
    if x.numel():
        with _on(x):
            _check("zero_mx4_quantize", _lib.zero_mx4_quantize(
                x.data_ptr(), code, m, n, ld, r and r.codes.data_ptr(), r and r.scales.data_ptr(),
                c and c.codes.data_ptr(), c and c.scales.data_ptr(), _stream(x)))
    return (r, c) if rows and cols else r or c


def mx4_dequantize(q: MX4, dtype=torch.bfloat16, out=None):
    """The matrix that q stands for."""
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=dtype, device=q.codes.device)
    if tuple(out.shape) != (q.rows, q.cols) or not _laid_out(out):
        raise ValueError("out: another shape, or rows without unit stride")
    _gpu(q.codes, q.scales, out)
    code = _code(out.dtype)
    if out.numel():
        with _on(out):
            _check("zero_mx4_dequantize", _lib.zero_mx4_dequantize(
                q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, out.data_ptr(), code,
                _stack(out)[3], _stream(out)))
    return out


def mx4_matmul(a, b: MX4, out_dtype=torch.bfloat16, *, out=None, accumulate: bool = False, ws=None):
    """a b^T: a an MX4, or a matrix of values that is quantised along its rows (in
    the product's own call for up to MX4_ROWS_MAX rows); b an MX4 over the
    same columns.  accumulate adds into ``out`` (fp32)."""
    values = not isinstance(a, MX4)
    m, k = a.shape if values else (a.rows, a.cols)
    if k != b.cols:
        raise ValueError(f"a has {k} columns and b {b.cols}")
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate needs an fp32 out")
    if out is None:
        out = torch.empty((m, b.rows), dtype=out_dtype, device=b.codes.device)
    elif tuple(out.shape) != (m, b.rows) or not _laid_out(out):
        raise ValueError("out: another shape, or rows without unit stride")
    c_code, n = _code(out.dtype), b.rows
    if values and (m > MX4_ROWS_MAX or accumulate):
        a, values = mx4_quantize(a), False
    _gpu(b.codes, b.scales, out, *((a,) if values else (a.codes, a.scales)))
    if not out.numel():
        return out
    with _on(out):
        if values:
            a_code = _code(a.dtype)
            a, lda = _matrix(a)
            p, size, _keep = _space(_lib.zero_mx4_matmul_rows_workspace_bytes(m, n, k), ws, out)
            _check("zero_mx4_matmul_rows", _lib.zero_mx4_matmul_rows(
                a.data_ptr(), a_code, lda, b.codes.data_ptr(), b.scales.data_ptr(), m, n, k,
                out.data_ptr(), c_code, _stack(out)[3], p, size, _stream(out)))
        else:
            p, size, _keep = _space(_lib.zero_mx4_matmul_workspace_bytes(m, n, k), ws, out)
            _check("zero_mx4_matmul", _lib.zero_mx4_matmul(
                a.codes.data_ptr(), a.scales.data_ptr(), b.codes.data_ptr(), b.scales.data_ptr(),
                m, n, k, out.data_ptr(), c_code, _stack(out)[3], int(accumulate), p, size,
                _stream(out)))
    return out


class _Mx4Linear(torch.autograd.Function):
    """y = x w^T and its gradients dx = dy w, dw = dy^T x, every product over MXFP4
    operands whose blocks lie along the dimension that it sums over."""

    @staticmethod
    def forward(ctx, x, w):
        need_x, need_w = ctx.needs_input_grad
        xr, xc = mx4_quantize(x, cols=True) if need_w else (mx4_quantize(x), None)
        wr, wc = mx4_quantize(w, cols=True) if need_x else (mx4_quantize(w), None)
        keep = [t for q in (xc, wc) if q is not None for t in (q.codes, q.scales)]
        ctx.save_for_backward(*keep)
        ctx.sizes = (x.shape[0], w.shape[0], w.shape[1], x.dtype, w.dtype)
        return mx4_matmul(xr, wr, x.dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        tokens, n, k, x_dtype, w_dtype = ctx.sizes
        need_x, need_w = ctx.needs_input_grad
        saved = list(ctx.saved_tensors)
        dx = dw = None
        dy, _ = _matrix(dy)
        q = mx4_quantize(dy, rows=need_x, cols=need_w)
        dr, dc = q if need_x and need_w else (q, q)
        if need_w:
            dw = mx4_matmul(dc, MX4(saved[0], saved[1], k, tokens), w_dtype)
            saved = saved[2:]
        if need_x:
            dx = mx4_matmul(dr, MX4(saved[0], saved[1], k, n), x_dtype)
        return dx, dw


def mx4_linear(x, w):
    """x w^T for x [tokens, k] and w [n, k] (fp16, bf16 or fp32), both quantised to
    MXFP4; differentiable: the gradients are the products of quantised operands
    too (the rounding itself is passed through)."""
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("expected x [tokens, k] and w [n, k]")
    return _Mx4Linear.apply(x, w)
