"""The calls on rows of tokens: MXFP8 rows and their product with MXFP4 operands, the
root-mean-square norm with the residual's addition, dropout, the embedding lookup, and
tokens sorted by expert and back; the last four with their gradients.

Argument marshalling only, as in matrices.py: the functions check their tensors, pass their
pointers to the C calls (include/zero_shard.h) and enqueue on torch's current stream
of the tensors' device.  Rows of unit stride are taken where they are, others are copied.

Forward and backward can be captured into a HIP graph.  As with every autograd function, no
eager result of the same leaves may be alive then: torch would accumulate their gradients on
that result's stream, inside the capture.  Gradients are those of backward passes: tensors with a
tangent of forward mode are refused.
"""
from __future__ import annotations

import torch
import torch.autograd.forward_ad as _forward

from . import F32, _lib
from .matrices import (MX4, _Blocks, _bytes, _call, _code, _DTYPES, _empty, _gpu, _laid_out,
                       _matrix, _space, _stack)

_f32 = torch.float32
_IDS = (torch.int32, torch.int64)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _constant(what: str, *tensors) -> None:
    """Refuses tensors whose derivative a call that has none would drop."""
    for t in tensors:
        if t is not None and (_grads() and t.requires_grad or _dual() and _forward.unpack_dual(t).tangent is not None):
            raise RuntimeError(f"{what} is not differentiable: detach its inputs, or call it under torch.no_grad()")


_rows_like, _flat = torch.empty_like, torch.contiguous_format


def _like(x):
    """A new contiguous tensor of x's shape and type."""
    return _rows_like(x, memory_format=_flat)


_grads = torch.is_grad_enabled


def _dual() -> bool:
    """Whether a level of forward mode is open: a tensor may have a tangent then without requiring a gradient, which
    the autograd functions, that have no formula for it, refuse."""
    return getattr(_forward, "_current_level", 0) >= 0


def _once(backward):
    """once_differentiable, without its own guard where torch records nothing, as in most backward passes."""
    guarded = torch.autograd.function.once_differentiable(backward)
    return staticmethod(lambda ctx, *g: guarded(ctx, *g) if _grads() else backward(ctx, *g))


# ----------------------------------------------------------------------------- MXFP8
class MX8(_Blocks):
    """A rows x cols matrix in MXFP8 (E4M3), blocks of 32 along its rows: codes [rows, P]
    and scales [rows, P / 32] bytes, P = cols rounded up to a multiple of 128 (the padding
    zero)."""

    __slots__ = ()
    CODE = 128


def mx8_quantize(x) -> MX8:
    """x (fp16, bf16 or fp32 matrix) as MX8."""
    code, index = _code(x.dtype), _gpu(x)
    x, ld = _matrix(x)
    m, n = x.shape
    q = MX8.alloc(m, n, x.device)
    if m and n:
        _call(index, "zero_mx8_quantize", x.data_ptr(), code, m, n, ld, *q._places)
    return q


def mx8_dequantize(q: MX8, dtype=torch.bfloat16, out=None):
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
        _call(index, "zero_mx8_dequantize", *q._places, q.rows, q.cols, out.data_ptr(), code, ld)
    return out


def mx8_matmul(a, b: MX4, out_dtype=torch.bfloat16, *, out=None, accumulate: bool = False, ws=None):
    """a b^T: a an MX8 (rms_norm_mx8 and mx8_quantize make them), or a matrix of values that is
    quantised along its rows (in the product's own kernel for few rows); b an MX4 over the same
    columns.  accumulate adds into ``out`` (fp32).  out shares no element with a or b.  Results are sums in
    fp32, rounded once to their type.  Not differentiable: values that require a gradient are refused."""
    values = not isinstance(a, MX8)
    if values:
        if isinstance(a, _Blocks):
            raise TypeError("a is neither an MX8 nor a matrix of values")
        _constant("mx8_matmul", a)
    if not isinstance(b, MX4):
        raise TypeError("b is not an MX4")
    m, k = a.shape if values else (a.rows, a.cols)
    n = b.rows
    if k != b.cols:
        raise ValueError(f"a has {k} columns and b {b.cols}")
    if accumulate and (out is None or out.dtype != _f32):
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
    if out.get_device() != index or (a.get_device() if values else a._index()) != index:
        raise ValueError("operands and result on one GPU")
    if not (m and n):
        return out
    if values:
        a_code = _code(a.dtype)
        a, lda = _matrix(a)
        p, size, _keep = _space(_lib.zero_mx8_matmul_rows_workspace_bytes(m, n, k), ws, out)
        _call(index, "zero_mx8_matmul_rows", a.data_ptr(), a_code, lda, *b._places, m, n, k,
              out.data_ptr(), c_code, ldc, int(accumulate), p, size)
    else:
        _call(index, "zero_mx8_matmul", *a._places, *b._places, m, n, k, out.data_ptr(), c_code, ldc,
              int(accumulate))
    return out


# ----------------------------------------------------------------------------- root-mean-square norm
def _norm_inputs(x, weight, residual, eps):
    """(index, x, ldx, residual, ldr, weight, code, code of the residual)"""
    code = _code(x.dtype)
    if x.dim() != 2 or weight.dim() != 1 or weight.shape[0] != x.shape[1]:
        raise ValueError("expected x [tokens, cols] and weight [cols]")
    if weight.dtype != x.dtype:
        raise TypeError(f"x is {x.dtype} and weight {weight.dtype}")
    if not 0.0 <= eps < float("inf"):
        raise ValueError("eps is finite and not negative")
    if residual is None:
        index, ldr, code_r = _gpu(x, weight), 0, code
    else:
        if residual.shape != x.shape:
            raise ValueError("residual: another shape than x")
        if residual.dtype not in (x.dtype, _f32):
            raise TypeError(f"x is {x.dtype} and residual {residual.dtype}: the same or fp32")
        index = _gpu(x, weight, residual)
        code_r = _DTYPES[residual.dtype]
        residual, ldr = _matrix(residual)
    x, ldx = _matrix(x)
    return index, x, ldx, residual, ldr, weight.contiguous(), code, code_r


def _norm(x, weight, residual, eps, packed):
    index, x, ldx, residual, ldr, weight, code, code_r = _norm_inputs(x, weight, residual, eps)
    tokens, cols = x.shape
    h = None if residual is None else _like(residual)
    inputs = (x.data_ptr(), code, ldx, _ptr(residual), code_r, ldr, weight.data_ptr(), tokens, cols, eps)
    if packed:
        y = MX8.alloc(tokens, cols, x.device)
        _call(index, "zero_rms_norm_mx8", *inputs, *y._places, _ptr(h), cols)
    else:
        y = _like(x)
        _call(index, "zero_rms_norm", *inputs, y.data_ptr(), cols, _ptr(h), cols)
    return y, h


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        y, h = _norm(x, weight, residual, eps, False)
        ctx.save_for_backward(x if h is None else h, weight)
        ctx.eps, ctx.dtype = eps, x.dtype
        ctx.set_materialize_grads(False)
        return y if h is None else (y, h)

    @_once
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        if dy is None:  # y was not used: the sum's gradient alone
            dw = torch.zeros_like(weight) if need_w else None
            return (None if dh is None or not need_x else dh.to(ctx.dtype)), dw, dh if need_r else None, None
        (h, ldh), (dy, lddy) = _matrix(h), _matrix(dy)
        weight = weight.contiguous()
        dh, lddh = (None, 0) if dh is None else _matrix(dh)
        tokens, cols = h.shape
        one = h.dtype == ctx.dtype  # one: x's gradient is the residual's
        dr = _like(h) if need_r and not one else None
        dx = _like(dy) if need_x or (need_r and one) else None
        dw = None if not need_w else _like(weight) if tokens else torch.zeros_like(weight)
        if tokens and cols:
            size = _lib.zero_rms_norm_grad_workspace_bytes(tokens, cols) if need_w else 0
            ws = _empty(size, dtype=_bytes, device=h.device) if size else None
            _call(h.get_device(), "zero_rms_norm_grad", dy.data_ptr(), lddy, h.data_ptr(), _DTYPES[h.dtype], ldh,
                  weight.data_ptr(), _DTYPES[ctx.dtype], _ptr(dh), lddh, tokens, cols, ctx.eps, _ptr(dx), cols,
                  _ptr(dr), cols, _ptr(dw), _ptr(ws), size)
        if one:
            dr = dx
        return dx if need_x else None, dw, dr if need_r else None, None


def rms_norm(x, weight, residual=None, *, eps: float = 1e-6):
    """The root-mean-square norm of every row of x [tokens, cols] times weight [cols] (one type: fp16,
    bf16 or fp32).  With a residual (x's type or fp32) it is the norm of h = x + residual, rounded
    to the residual's type, and (y, h) is returned.  Differentiable in all three; nothing but h (x
    without a residual) is kept for the gradients."""
    if _dual() or _grads() and (x.requires_grad or weight.requires_grad or residual is not None and residual.requires_grad):
        return _RmsNorm.apply(x, weight, residual, eps)
    y, h = _norm(x, weight, residual, eps, False)
    return y if h is None else (y, h)


def rms_norm_mx8(x, weight, residual=None, *, eps: float = 1e-6):
    """rms_norm whose result is left as MX8 rows, from its fp32 values, for mx8_matmul: MX8, or
    (MX8, h) with a residual.  Not differentiable: with a residual, x and residual that require
    a gradient are refused, since h, a tensor that goes on, would come back without its graph."""
    if residual is not None:
        _constant("rms_norm_mx8", x, residual)
    y, h = _norm(x, weight, residual, eps, True)
    return y if h is None else (y, h)


# ----------------------------------------------------------------------------- dropout
def _rows_of(x):
    """x as [rows, cols] with unit-stride rows, and its row stride."""
    return _matrix(x if x.dim() == 2 else x.reshape(-1, x.shape[-1]) if x.dim() > 2 else x.reshape(1, -1))


def _drop(x, residual, p, seed, offset, offset_dev):
    y = _like(x)
    if not x.numel():
        return y
    x, ldx = _rows_of(x)
    rows, cols = x.shape
    at, ldr = None, 0
    if residual is not None:
        residual, ldr = _rows_of(residual)
        at = residual.data_ptr()
    _call(x.get_device(), "zero_dropout", x.data_ptr(), _DTYPES[x.dtype], ldx, at, ldr, rows, cols, p, seed & _WORD, offset & _WORD,
          None if offset_dev is None else offset_dev.data_ptr(), y.data_ptr(), cols)
    return y


_WORD = (1 << 64) - 1


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, how, offset_dev):
        ctx.how = how
        if offset_dev is not None:
            ctx.save_for_backward(offset_dev)
        return _drop(x, residual, *how, offset_dev)

    @_once
    def backward(ctx, dy):
        need_x, need_r = ctx.needs_input_grad[:2]
        dx = _drop(dy, None, *ctx.how, *(ctx.saved_tensors or (None,))) if need_x else None
        return dx, dy if need_r else None, None, None


def dropout(x, p: float, seed: int, offset=0, *, residual=None):
    """x (fp16, bf16 or fp32) with elements dropped with probability p (a multiple of 1 / 65536, the
    nearest) and the others divided by 1 - p; plus residual (x's shape and type).  Differentiable in
    both.  Which elements stay is a function of (seed, offset), of the element's place in its row
    (the last dimension) and of the row's number; no mask is stored, the backward pass computes it again.

    seed and offset: 64-bit integers; different offsets of a seed (a layer's number, a step's)
    are different masks.  offset may be an int64 GPU tensor of one element, read when the kernels run:
    a captured graph then draws anew after the program has moved it.  It may not be moved between a
    forward pass and its backward pass."""
    _code(x.dtype)
    if not 0.0 <= p <= 1.0:
        raise ValueError("p is not in [0, 1]")
    offset_dev = None
    if isinstance(offset, torch.Tensor):
        if offset.dtype != torch.int64 or offset.numel() != 1:
            raise ValueError("offset: an integer, or an int64 GPU tensor of one element")
        offset, offset_dev = 0, offset
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError("residual: another shape or type than x")
    if residual is None and offset_dev is None:
        _gpu(x)
    else:
        _gpu(x, *(t for t in (residual, offset_dev) if t is not None))
    if _dual() or _grads() and (x.requires_grad or residual is not None and residual.requires_grad):
        return _Dropout.apply(x, residual, (p, seed, offset), offset_dev)
    return _drop(x, residual, p, seed, offset, offset_dev)


# ----------------------------------------------------------------------------- embedding
def _lookup(ids, table, scale):
    index = table.get_device()
    table, ldt = _matrix(table)
    vocab, cols = table.shape
    out = _empty((*ids.shape, cols), dtype=table.dtype, device=table.device)
    _call(index, "zero_embedding", ids.data_ptr(), ids.element_size(), ids.numel(), table.data_ptr(),
          _DTYPES[table.dtype], ldt, vocab, cols, scale, out.data_ptr(), cols)
    return out


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.how = (*table.shape, scale)
        return _lookup(ids, table, scale)

    @_once
    def backward(ctx, dy):
        ids, = ctx.saved_tensors
        vocab, cols, scale = ctx.how
        dy, ld = _matrix(dy.reshape(-1, cols))
        out = _empty((vocab, cols), dtype=dy.dtype, device=dy.device)
        tokens = ids.numel()
        size = _lib.zero_embedding_grad_workspace_bytes(tokens, vocab, cols)
        ws = _empty(size, dtype=_bytes, device=dy.device) if size else None
        _call(dy.get_device(), "zero_embedding_grad", ids.data_ptr(), ids.element_size(), tokens, dy.data_ptr(),
              _DTYPES[dy.dtype], ld, vocab, cols, scale, out.data_ptr(), cols, _ptr(ws), size)
        return None, out, None


def embedding(tokens, table, *, scale: float = 1.0):
    """table[tokens] * scale for a table [vocab, cols] (fp16, bf16 or fp32) and int32 or int64 tokens of
    any shape: [*tokens.shape, cols].  A token outside [0, vocab) gives zeros and takes no part in the
    gradient (padding; the other ranks' part of a table that is split by rows: subtract the first).

    Differentiable in the table: the gradient is dense, of the table's type, each row the sum over its
    tokens in their order (fp32, rounded once), found by sorting the tokens: the same bits every time."""
    if table.dim() != 2 or not table.numel():
        raise ValueError("expected a table [vocab, cols], not empty")
    _code(table.dtype)
    if tokens.dtype not in _IDS:
        raise TypeError("tokens are int32 or int64")
    if not -3.4e38 < scale < 3.4e38:
        raise ValueError("scale is not finite")
    _gpu(table, tokens)
    tokens = tokens.contiguous()
    if _dual() or _grads() and table.requires_grad:
        return _Embedding.apply(tokens, table, scale)
    return _lookup(tokens, table, scale)


# ----------------------------------------------------------------------------- tokens by expert
class ExpertPlan:
    """Where each of a batch's assignments goes in the order of experts.  Slot t k + j is token t's
    j-th assignment.  order [tokens k]: the slot at each place; place [tokens, k]: its inverse;
    offsets [experts + 1]: where each expert's rows start, the last entry the number of slots that
    have an expert (all int32, on the GPU: nothing waits for the host)."""

    __slots__ = ("order", "place", "offsets", "tokens", "k", "experts")

    def __init__(self, order, place, offsets, tokens: int, k: int, experts: int):
        for t, n in ((order, tokens * k), (place, tokens * k), (offsets, experts + 1)):
            if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous():
                raise ValueError("order and place: tokens k contiguous int32 numbers, offsets: experts + 1")
        self.order, self.place, self.offsets = order, place, offsets
        self.tokens, self.k, self.experts = tokens, k, experts

    def _check(self, t, rows: int, what: str) -> int:
        _code(t.dtype)
        if t.dim() != 2 or t.shape[0] != rows:
            raise ValueError(f"{what}: expected [{rows}, cols]")
        return _gpu(t, self.place, self.offsets)

    def _versions(self):
        """How often torch has written the memory that the calls read; forward and backward passes read the same."""
        return tuple(None if t.is_inference() else t._version for t in (self.place, self.offsets))

    def _again(self, versions) -> None:
        if versions != self._versions():
            raise RuntimeError("the plan was modified by an inplace operation between a forward pass and its backward pass")

    def _places(self):
        return self.place.data_ptr(), self.offsets.data_ptr() + 4 * self.experts


def expert_sort(experts, n_experts: int) -> ExpertPlan:
    """The plan of a batch: experts [tokens, k] (int32 or int64) are each token's choices.  A choice
    outside [0, n_experts) is dropped: its place is behind all others.  The order is stable."""
    if experts.dim() != 2 or not experts.shape[1]:
        raise ValueError("expected experts [tokens, k]")
    if experts.dtype not in _IDS:
        raise TypeError("experts are int32 or int64")
    index = _gpu(experts)
    tokens, k = experts.shape
    n = tokens * k
    experts = experts.contiguous()
    dev = experts.device
    order = _empty(n, dtype=torch.int32, device=dev)
    place = _empty((tokens, k), dtype=torch.int32, device=dev)
    if n_experts < 1:
        raise ValueError("no experts")
    offsets = _empty(n_experts + 1, dtype=torch.int32, device=dev)
    p, size, _keep = _space(_lib.zero_expert_sort_workspace_bytes(n, n_experts), None, experts)
    _call(index, "zero_expert_sort", experts.data_ptr(), experts.element_size(), n, n_experts, order.data_ptr(),
          place.data_ptr(), offsets.data_ptr(), p, size)
    return ExpertPlan(order, place, offsets, tokens, k, n_experts)


def _to_rows(x, plan):
    x, ld = _matrix(x)
    cols = x.shape[1]
    rows = _empty((plan.tokens * plan.k, cols), dtype=x.dtype, device=x.device)
    _call(x.get_device(), "zero_expert_rows", x.data_ptr(), _DTYPES[x.dtype], ld, *plan._places(), plan.tokens, plan.k,
          cols, rows.data_ptr(), cols)
    return rows


def _to_tokens(rows, weights, plan):
    rows, ld = _matrix(rows)
    cols = rows.shape[1]
    y = _empty((plan.tokens, cols), dtype=rows.dtype, device=rows.device)
    _call(rows.get_device(), "zero_expert_combine", rows.data_ptr(), _DTYPES[rows.dtype], ld, *plan._places(),
          _ptr(weights), F32 if weights is None else _DTYPES[weights.dtype], plan.tokens, plan.k, cols, y.data_ptr(), cols)
    return y


class _ExpertRows(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan, ctx.versions = plan, plan._versions()
        return _to_rows(x, plan)

    @_once
    def backward(ctx, drows):
        ctx.plan._again(ctx.versions)
        return _to_tokens(drows, None, ctx.plan), None


def expert_rows(x, plan: ExpertPlan):
    """The rows of x [tokens, cols] in the plan's order, [tokens k, cols]: expert e's are rows
    offsets[e] .. offsets[e + 1]; the rows behind the last are zeros.  Differentiable."""
    plan._check(x, plan.tokens, "x")
    if _dual() or _grads() and x.requires_grad:
        return _ExpertRows.apply(x, plan)
    return _to_rows(x, plan)


class _ExpertCombine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, plan):
        ctx.plan, ctx.versions = plan, plan._versions()
        ctx.save_for_backward(rows if ctx.needs_input_grad[1] else None, weights)
        return _to_tokens(rows, weights, plan)

    @_once
    def backward(ctx, dy):
        rows, weights = ctx.saved_tensors
        plan, (need_rows, need_weights) = ctx.plan, ctx.needs_input_grad[:2]
        plan._again(ctx.versions)
        dy, lddy = _matrix(dy)
        cols, dev = dy.shape[1], dy.device
        rows, ldr = (None, 0) if rows is None else _matrix(rows)
        drows = _empty((plan.tokens * plan.k, cols), dtype=dy.dtype, device=dev) if need_rows else None
        dweights = None
        if need_weights:
            dweights = _like(weights) if cols else torch.zeros_like(weights)
        _call(dy.get_device(), "zero_expert_combine_grad", dy.data_ptr(), lddy, _ptr(rows), _DTYPES[dy.dtype], ldr,
              *plan._places(), weights.data_ptr(), _DTYPES[weights.dtype], plan.tokens, plan.k, cols, _ptr(drows), cols,
              _ptr(dweights))
        return drows, dweights, None


def expert_combine(rows, weights, plan: ExpertPlan):
    """The tokens' results from the experts' rows [tokens k, cols]: the sum over a token's slots of
    weights [tokens, k] (rows' type or fp32) times the slot's row, in fp32, rounded once;
    dropped slots left out, whatever their weights and rows hold.  Differentiable in rows and weights."""
    index = plan._check(rows, plan.tokens * plan.k, "rows")
    if tuple(weights.shape) != (plan.tokens, plan.k):
        raise ValueError(f"weights: expected [{plan.tokens}, {plan.k}]")
    if weights.dtype not in (rows.dtype, _f32):
        raise TypeError(f"rows are {rows.dtype} and weights {weights.dtype}: the same or fp32")
    if weights.get_device() != index:
        raise ValueError("rows and weights on one GPU")
    weights = weights.contiguous()
    if _dual() or _grads() and (rows.requires_grad or weights.requires_grad):
        return _ExpertCombine.apply(rows, weights, plan)
    return _to_tokens(rows, weights, plan)
