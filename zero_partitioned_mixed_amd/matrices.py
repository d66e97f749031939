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
               MuonHparams, NewtonSchulz, ShardStep, _check, _lib, zero_adam_step)

_DTYPES = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
COEFFS = (3.4445, -4.7750, 2.0315)  # the usual quintic's


def _code(dtype, allowed=_DTYPES) -> int:
    if dtype not in allowed:
        raise TypeError(f"dtype {dtype} is not one of {', '.join(str(d) for d in allowed)}")
    return _DTYPES[dtype]


_HALVES = (torch.float16, torch.bfloat16)
# torch.cuda.current_stream(index).cuda_stream, without the object where this torch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch.cuda.current_device
_empty, _bytes = torch.empty, torch.uint8


def _gpu(first, *others) -> int:
    """The index of the GPU that all the tensors are on."""
    index = first.get_device()  # -1 on the CPU
    if index < 0:
        raise ValueError("expected GPU tensors")
    for t in others:
        if t.get_device() != index:
            raise ValueError("expected GPU tensors" if not t.is_cuda else "tensors on different GPUs")
    return index


def _call(index: int, name: str, *args) -> None:
    """The C call on the GPU's current stream."""
    if _current_device() == index:
        rc = getattr(_lib, name)(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = getattr(_lib, name)(*args, _raw_stream(index))
    if rc != 0:
        _check(name, rc)


def _space(nbytes: int, ws, like):
    """(pointer, bytes, tensor) of a workspace: ws, or a new tensor."""
    if ws is None:
        if nbytes == 0:
            return None, 0, None
        ws = _empty(nbytes, dtype=_bytes, device=like.device)
        return ws.data_ptr(), nbytes, ws
    _gpu(like, ws)
    if not ws.is_contiguous():
        raise ValueError("ws: its bytes are not contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


# ----------------------------------------------------------------------------- orthogonalised updates
def newton_schulz(coeffs=COEFFS, steps: int = 5, eps: float = 1e-7) -> NewtonSchulz:
    """The settings of an orthogonalisation.  The coefficients may not let singular values,
    which start in [0, 1], grow above 3.5 between the steps (the calls refuse them)."""
    a, b, c = coeffs
    return NewtonSchulz(a, b, c, eps, steps)


def muon_hparams(lr=3e-4, momentum=0.95, weight_decay=0.0, nesterov=True, scale=MUON_SCALE_RMS,
                 coeffs=COEFFS, steps=5, eps=1e-7) -> MuonHparams:
    return MuonHparams(lr, momentum, weight_decay, int(bool(nesterov)), scale,
                       newton_schulz(coeffs, steps, eps))


def _stack(x):
    """(count, rows, cols, row stride, matrix stride) of [rows, cols] or [count, rows, cols]."""
    shape = x.shape
    if len(shape) == 2:
        (rows, cols), count = shape, 1
    elif len(shape) == 3:
        count, rows, cols = shape
    else:
        raise ValueError("expected [rows, cols] or [count, rows, cols]")
    if x.is_contiguous():
        return count, rows, cols, cols, rows * cols
    ld = x.stride(-2) if rows > 1 else max(x.stride(-2), cols)
    stride = x.stride(0) if x.dim() == 3 and count > 1 else rows * ld
    return count, rows, cols, ld, stride


def _laid_out(x) -> bool:
    """Rows of unit stride that do not overlap, matrices that do not overlap."""
    if x.is_contiguous() or x.numel() == 0:
        return True
    _, rows, cols, ld, stride = _stack(x)
    return (cols == 1 or x.stride(-1) == 1) and ld >= cols and stride >= (rows - 1) * ld + cols


def orthogonalize(x, out_dtype=None, *, coeffs=COEFFS, steps: int = 5, eps: float = 1e-7, out=None,
                  ws=None):
    """The Newton-Schulz orthogonalisation of every matrix of x ([rows, cols] or
    [count, rows, cols]; fp16, bf16 or fp32, any strides: other layouts than
    unit-stride rows are copied).  Returns fp16 or bf16 (out_dtype; by default x's
    type, bf16 for fp32), in ``out`` when given (it may be x, or share no element with
    it).  A result in fp16 is exact but for its own rounding (1e-5); one in bf16, for a
    smaller side above 128, to 1.8e-3 in 0.4 of the time.  coeffs: as newton_schulz
    takes them.  Not differentiable."""
    if out is not None:
        out_dtype = out.dtype
    elif out_dtype is None:
        out_dtype = torch.bfloat16 if x.dtype == torch.float32 else x.dtype
    src_code, dst_code = _code(x.dtype), _code(out_dtype, _HALVES)
    if out is None:
        out = _empty(x.shape, dtype=out_dtype, device=x.device)
    elif out.shape != x.shape or not _laid_out(out):
        raise ValueError("out: another shape, or rows without unit stride")
    index = _gpu(x, out)
    if not _laid_out(x):
        x = x.contiguous()
    count, rows, cols, ld, stride = _stack(x)
    _, _, _, out_ld, out_stride = _stack(out)
    # a bf16 result needs no more than the optimizer step
    size = _lib.zero_ns_workspace_bytes if dst_code == F16 else _lib.zero_muon_workspace_bytes
    p, n, _keep = _space(size(count, rows, cols), ws, x)
    _call(index, "zero_orthogonalize", x.data_ptr(), src_code, count, rows, cols, ld, stride,
          out.data_ptr(), dst_code, out_ld, out_stride,
          ctypes.byref(newton_schulz(coeffs, steps, eps)), p, n)
    return out


def _muon_space(exact: bool):
    return _lib.zero_ns_workspace_bytes if exact else _lib.zero_muon_workspace_bytes


def muon_step(master, mom, g, hp: MuonHparams, *, slot=None, ctrl=None, ws=None, exact: bool = False) -> None:
    """One optimizer step, in place, for the matrices of master ([rows, cols] or
    [count, rows, cols] fp32, matrices contiguous; mom and g alike, usually
    views of a shard's flat buffers).  slot: the fp16 or bf16 parameters laid
    out like master (a view of the gather buffer).  ctrl: the rank's control
    block, whose clip and skip then apply.  exact: the update to 1e-5 where the smaller
    side is above 128 too (else to 1.8e-3), in 2.4 times the time."""
    matrices = (master, mom, g) if slot is None else (master, mom, g, slot)
    index = _gpu(*matrices) if ctrl is None else _gpu(*matrices, ctrl)
    for t in (master, mom, g):
        _code(t.dtype, (torch.float32,))
    slot_code = F16 if slot is None else _code(slot.dtype, _HALVES)
    place = _stack(master)
    count, rows, cols, ld, stride = place
    for t in matrices:
        if t.shape != master.shape or not _laid_out(t) or (t.numel() and (ld != cols or _stack(t) != place)):
            raise ValueError("master, mom, g and slot: one shape, contiguous matrices at one stride")
    p, n, _keep = _space(_muon_space(exact)(count, rows, cols), ws, master)
    _call(index, "zero_muon_step_exact" if exact else "zero_muon_step", master.data_ptr(), mom.data_ptr(), g.data_ptr(), count, rows, cols,
          stride, ctypes.byref(hp), None if ctrl is None else ctrl.data_ptr(),
          None if slot is None else slot.data_ptr(), slot_code, 0, p, n)


class MuonShardStep(ShardStep):
    """One rank's shard step with whole matrices in it: the two-pass path's reduce and
    decision over all of the shard, then muon_step for the matrices and zero_adam_step
    for what lies between them.

    matrices: (first element in the shard, count, rows, cols) of each stack of
    contiguous matrices, in order and apart; whatever lies between two stacks starts at a
    multiple of four elements.  A matrix that a shard's border cuts is none of them: its
    parts take AdamW, or the border is placed elsewhere.  The momentum of a matrix is its
    part of the state's m; its part of v is not used.  No quantised payload is written.
    exact: as muon_step takes it."""

    def __init__(self, nranks, stride, valid_len, offset, dtype, gather_dtype, hp, muon: MuonHparams,
                 matrices, state, g, loss_scale=1.0, bucket: int = 0, exact: bool = False):
        super().__init__(nranks, stride, valid_len, offset, dtype, gather_dtype, hp, state, g, loss_scale,
                         bucket, two_pass=True)
        self.muon, self.matrices, self.between, self.exact = muon, list(matrices), [], exact
        at = space = 0
        for start, count, rows, cols in self.matrices + [(valid_len, 0, 0, 0)]:
            if start < at or start + count * rows * cols > valid_len:
                raise ValueError("matrices overlap or leave the shard")
            if start > at:
                if at % 4:
                    raise ValueError("what follows a stack of matrices starts at a multiple of 4 elements")
                self.between.append((at, start - at))
            at = start + count * rows * cols
            space = max(space, _muon_space(exact)(count, rows, cols))
        self.matrix_ws = _empty(space, dtype=_bytes, device=state[0].device) if space else None

    @staticmethod
    def _no_payload(qgather) -> None:
        if qgather is not None:
            raise ValueError("no INT8 or INT4 payload with matrices: quantise the slot")

    def run_pieces(self, contrib, gather, qgather=None) -> None:
        self._no_payload(qgather)  # before the step has begun
        super().run_pieces(contrib, gather)

    def complete(self, gather, qgather=None) -> None:
        self._no_payload(qgather)
        master, m, v = self.state
        for start, length in self.between:
            zero_adam_step(tuple(t[start:] for t in self.state), self.g[start:], length, self.hp, self.ctrl,
                           gather, self.gather_dtype, self.offset + start)
        for start, count, rows, cols in self.matrices:
            end = start + count * rows * cols
            part = [t[start:end].view(count, rows, cols) for t in (master, m, self.g)]
            slot = None if gather is None else \
                gather[self.offset + start:self.offset + end].view(count, rows, cols)
            muon_step(*part, self.muon, slot=slot, ctrl=self.ctrl, ws=self.matrix_ws, exact=self.exact)


# ----------------------------------------------------------------------------- MXFP4
class MX4:
    """A rows x cols matrix in MXFP4, blocks of 32 along its rows: codes
    [rows, P / 2] and scales [rows, P / 32] bytes, P = cols rounded up to a multiple
    of 128 (the padding zero)."""

    __slots__ = ("rows", "cols", "_codes", "_scales", "_both", "_places")

    def __init__(self, codes, scales, rows: int, cols: int):
        p = (cols + 127) // 128 * 128
        for t, width in ((codes, p // 2), (scales, p // 32)):
            if t.dtype != _bytes or t.numel() != rows * width or not t.is_contiguous():
                raise ValueError(f"{rows} x {cols} takes {rows * p // 2} contiguous bytes of codes and "
                                 f"{rows * p // 32} of scales")
        self._codes, self._scales, self.rows, self.cols = codes, scales, rows, cols
        self._both, self._places = None, (codes.data_ptr(), scales.data_ptr())

    @staticmethod
    def alloc(rows: int, cols: int, device) -> "MX4":
        """Codes and scales in one new buffer."""
        blocks = rows * ((cols + 127) // 128)
        q = MX4.__new__(MX4)
        q.rows, q.cols, q._codes = rows, cols, None
        q._both = both = _empty(68 * blocks, dtype=_bytes, device=device)
        at = both.data_ptr()
        q._places = (at, at + 64 * blocks)
        return q

    def _split(self):
        n = self.rows * ((self.cols + 127) // 128)
        self._codes = self._both[:64 * n].view(self.rows, -1) if n else self._both.view(self.rows, 0)
        self._scales = self._both[64 * n:].view(self.rows, -1) if n else self._codes

    @property
    def codes(self):
        if self._codes is None:
            self._split()
        return self._codes

    @property
    def scales(self):
        if self._codes is None:
            self._split()
        return self._scales

    @property
    def device(self):
        return (self._codes if self._both is None else self._both).device

    def _index(self) -> int:
        return _gpu(self._codes, self._scales) if self._both is None else _gpu(self._both)


def _matrix(x):
    """x as unit-stride rows, and its row stride."""
    if x.dim() != 2:
        raise ValueError("expected a matrix")
    if x.is_contiguous():
        return x, x.shape[1]
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
    index = _gpu(x)
    x, ld = _matrix(x)
    m, n = x.shape
    device = x.device
    r = MX4.alloc(m, n, device) if rows else None
    c = MX4.alloc(n, m, device) if cols else None
    if m and n:
        _call(index, "zero_mx4_quantize", x.data_ptr(), code, m, n, ld,
              *(r._places if rows else _NOWHERE), *(c._places if cols else _NOWHERE))
    return (r, c) if rows and cols else r if rows else c


_NOWHERE = (None, None)


def mx4_dequantize(q: MX4, dtype=torch.bfloat16, out=None):
    """The matrix that q stands for."""
    index = q._index()
    if out is None:
        out = _empty((q.rows, q.cols), dtype=dtype, device=q.device)
        ld = q.cols
    elif tuple(out.shape) != (q.rows, q.cols) or not _laid_out(out):
        raise ValueError("out: another shape, or rows without unit stride")
    else:
        ld = _stack(out)[3]
    code = _code(out.dtype)
    if out.get_device() != index:
        raise ValueError("out is elsewhere")
    if q.rows and q.cols:
        _call(index, "zero_mx4_dequantize", *q._places, q.rows, q.cols, out.data_ptr(), code, ld)
    return out


def mx4_matmul(a, b: MX4, out_dtype=torch.bfloat16, *, out=None, accumulate: bool = False, ws=None):
    """a b^T: a an MX4, or a matrix of values that is quantised along its rows (in
    the product's own call for up to MX4_ROWS_MAX rows); b an MX4 over the
    same columns.  accumulate adds into ``out`` (fp32).  out shares no element with a or b."""
    values = not isinstance(a, MX4)
    m, k = a.shape if values else (a.rows, a.cols)
    n = b.rows
    if k != b.cols:
        raise ValueError(f"a has {k} columns and b {b.cols}")
    if accumulate and (out is None or out.dtype != torch.float32):
        raise ValueError("accumulate needs an fp32 out")
    index = b._index()
    if out is None:
        out = _empty((m, n), dtype=out_dtype, device=b.device)
        ldc = n
    elif tuple(out.shape) != (m, n) or not _laid_out(out):
        raise ValueError("out: another shape, or rows without unit stride")
    else:
        ldc = _stack(out)[3]
    c_code = _code(out.dtype)
    if values and (m > MX4_ROWS_MAX or accumulate):
        a, values = mx4_quantize(a), False
    if out.get_device() != index or (a.get_device() if values else a._index()) != index:
        raise ValueError("operands and result on one GPU")
    if not (m and n):
        return out
    if values:
        a_code = _code(a.dtype)
        a, lda = _matrix(a)
        p, size, _keep = _space(_lib.zero_mx4_matmul_rows_workspace_bytes(m, n, k), ws, out)
        _call(index, "zero_mx4_matmul_rows", a.data_ptr(), a_code, lda, *b._places, m, n, k,
              out.data_ptr(), c_code, ldc, p, size)
    else:
        p, size, _keep = _space(_lib.zero_mx4_matmul_workspace_bytes(m, n, k), ws, out)
        _call(index, "zero_mx4_matmul", *a._places, *b._places, m, n, k, out.data_ptr(), c_code, ldc,
              int(accumulate), p, size)
    return out


class _Mx4Linear(torch.autograd.Function):
    """y = x w^T and its gradients dx = dy w, dw = dy^T x, every product over MXFP4
    operands whose blocks lie along the dimension that it sums over."""

    @staticmethod
    def forward(ctx, x, w, grad):
        # grad: whether torch records (here it never does); needs_input_grad is set all the same
        need_x, need_w = (grad and need for need in ctx.needs_input_grad[:2])
        x, ldx = _matrix(x)
        w, ldw = _matrix(w)
        tokens, k = x.shape
        n = w.shape[0]
        code, index, dev = _DTYPES[x.dtype], x.get_device(), x.device
        y = _empty((tokens, n), dtype=x.dtype, device=dev)
        size_x = _lib.zero_mx4_operand_bytes(k, tokens) if need_w else 0
        size_w = _lib.zero_mx4_operand_bytes(k, n) if need_x else 0
        # what the gradients need
        kept = _empty(size_x + size_w, dtype=_bytes, device=dev) if need_x or need_w else None
        size = _lib.zero_mx4_linear_workspace_bytes(tokens, n, k)
        ws = _empty(size, dtype=_bytes, device=dev)
        at = kept.data_ptr() if need_x or need_w else None
        _call(index, "zero_mx4_linear", x.data_ptr(), ldx, w.data_ptr(), ldw, code, tokens, n, k,
              y.data_ptr(), n, at if need_w else None, at + size_x if need_x else None,
              ws.data_ptr(), size)
        if kept is not None:
            ctx.save_for_backward(kept)
            ctx.sizes = (tokens, n, k, code, size_x)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        tokens, n, k, code, size_x = ctx.sizes
        need_x, need_w, _ = ctx.needs_input_grad
        kept, = ctx.saved_tensors
        dy, ld = _matrix(dy)
        dev = dy.device
        dx = _empty((tokens, k), dtype=dy.dtype, device=dev) if need_x else None
        dw = _empty((n, k), dtype=dy.dtype, device=dev) if need_w else None
        size = _lib.zero_mx4_linear_grad_workspace_bytes(tokens, n)
        ws = _empty(size, dtype=_bytes, device=dev)
        at = kept.data_ptr()
        _call(dy.get_device(), "zero_mx4_linear_grad", dy.data_ptr(), ld, code, tokens, n, k,
              at if need_w else None, at + size_x if need_x else None,
              dx.data_ptr() if need_x else None, k, dw.data_ptr() if need_w else None, k,
              ws.data_ptr(), size)
        return dx, dw, None


def mx4_linear(x, w):
    """x w^T for x [tokens, k] and w [n, k] of one type (fp16, bf16 or fp32), both
    quantised to MXFP4; differentiable: the gradients are the products of quantised
    operands too (the rounding itself is passed through).  Where torch does not record,
    nothing is made or kept for them.

    Forward and backward can be captured into a HIP graph.  As with every autograd
    function, no eager result of the same leaves may be alive then: torch would
    accumulate their gradients on that result's stream, inside the capture."""
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1] or not x.numel() or not w.numel():
        raise ValueError("expected x [tokens, k] and w [n, k], not empty")
    if x.dtype != w.dtype:
        raise TypeError(f"x is {x.dtype} and w {w.dtype}")
    _code(x.dtype)
    _gpu(x, w)
    return _Mx4Linear.apply(x, w, torch.is_grad_enabled())
