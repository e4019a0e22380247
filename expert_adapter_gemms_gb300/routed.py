"""Around the experts' products: rows by expert and back, and projections with the adapters of
many requests beside them, for training and serving.

Thin like :mod:`.api`: tensors are checked, outputs allocated, and the C entry points of the
same names called on the current stream; nothing here computes. Tensors are contiguous and on
the current device; a given `out` shares no memory with the call's other tensors, and counts as
changed in place for autograd. The order of the rows is that of an align buffer (moe_lora_align):
autograd's backward passes refuse one that was aligned anew after the forward pass (by a call; that a
replayed graph aligned into it they cannot see).

Capturing a backward pass into a CUDA graph has PyTorch's own condition: no eager autograd graph of
the same leaves may be alive meanwhile. The *_backward functions are plain calls and have none.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib as L_
from ._lib import check, lib, ptr, stream_handle
from .api import Align, _need, _no_tangents, forward_ad
from .ffn import DTYPES, _16


def _rows(t, name: str, dtypes, rows: int, cols: Optional[int] = None) -> torch.Tensor:
    """A contiguous [rows, cols] tensor of one of these types."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == 2 and t.is_contiguous():
        n, c = t.shape
        if n == rows and c >= 1 and (cols is None or c == cols):
            return t
    if isinstance(t, torch.Tensor) and t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    _need(t, name, t.dtype if isinstance(t, torch.Tensor) else None, 2)
    if t.shape[0] != rows or (cols is not None and t.shape[1] != cols) or t.shape[1] < 1:
        raise ValueError(f"{name} must have shape ({rows}, {cols if cols is not None else 'H >= 1'}), got {tuple(t.shape)}")
    return t


def _fits(t, dtype, shape) -> bool:
    """Whether t is a contiguous tensor of this type and shape: one look, no message (a call on few
    rows takes the GPU less time than the checks one by one)."""
    return isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _here(what: str, *tensors: Optional[torch.Tensor]) -> int:
    """The current stream; refuses tensors that are not on the current device, whose stream it is."""
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != device or device < 0):
            raise ValueError(f"{what}: every tensor must be on one CUDA device (there is no CPU path), got "
                             f"{tensors[0].device} and {t.device}")
    if device != torch.cuda.current_device():
        raise ValueError(f"{what}: the tensors are on cuda:{device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(device)


def _apart(what: str, out: torch.Tensor, *tensors: Optional[torch.Tensor]) -> None:
    """Refuses a given `out` that shares memory with what the call reads (or works in) meanwhile."""
    first = out.data_ptr()
    end = first + out.nbytes
    for t in tensors:
        if t is not None:
            at = t.data_ptr()
            if first < at + t.nbytes and at < end:
                raise ValueError(f"{what}: out shares memory with another of the call's tensors")


def _written(out: torch.Tensor) -> None:
    """Lets autograd see that a given `out` changes, should it have saved that memory for a backward pass."""
    if not out.is_inference():
        torch.autograd.graph.increment_version(out)


def _wants(*tensors: Optional[torch.Tensor]) -> bool:
    return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)


def _grad_rows(g: torch.Tensor, align: int) -> torch.Tensor:
    """A gradient as the kernels take it: autograd chooses its strides and where it starts."""
    g = g.contiguous()
    return g.clone() if g.data_ptr() % align else g


def _order(ctx, buf: torch.Tensor) -> Align:
    """The order of the forward pass, over the buffer as autograd saved it (reading that raised if it
    was aligned anew). Saved-tensor hooks may have put it elsewhere."""
    if ctx.al.buf is not buf:
        ctx.al.buf = buf
    return ctx.al


_ANY = tuple(DTYPES)


# ---------------------------------------------------------------------------
# rows by expert and back
# ---------------------------------------------------------------------------
def _permute(x, al, out, stream):
    H = x.shape[1]
    flags = 0
    if out is None:
        out = torch.empty((al.S, H), dtype=x.dtype, device=x.device)
        flags = L_.ROWS_ZERO_DROPPED
    else:
        _written(out)
    st = lib().moe_permute(x.data_ptr(), DTYPES[x.dtype], al.ref(), H, flags, out.data_ptr(), stream)
    if st:
        check(st, "moe_permute")
    return out


def _unpermute(o, al, w, out, stream):
    H = o.shape[1]
    if out is None:
        out = torch.empty((al.T, H), dtype=o.dtype, device=o.device)
    else:
        _written(out)
    st = lib().moe_unpermute(o.data_ptr(), DTYPES[o.dtype], al.ref(), 0 if w is None else w.data_ptr(), H,
                             out.data_ptr(), stream)
    if st:
        check(st, "moe_unpermute")
    return out


class _Permute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, al):
        ctx.save_for_backward(al.buf)
        ctx.al = al.kept()
        return _permute(x, al, None, stream_handle())

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dxs):
        buf, = ctx.saved_tensors
        return _unpermute(_grad_rows(dxs, dxs.element_size()), _order(ctx, buf), None, None, stream_handle()), None


class _Unpermute(torch.autograd.Function):
    @staticmethod
    def forward(ctx, o, w, al):
        ctx.save_for_backward(al.buf, w, o if ctx.needs_input_grad[1] else None)
        ctx.al = al.kept()
        return _unpermute(o, al, w, None, stream_handle())

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        buf, w, o = ctx.saved_tensors
        do, dw = moe_unpermute_backward(_grad_rows(dy, dy.element_size()), o, _order(ctx, buf), w,
                                        need_do=ctx.needs_input_grad[0], need_dw=ctx.needs_input_grad[1])
        return do, dw, None


def moe_permute(x: torch.Tensor, al: Align, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """xs[row] = x[token(row)], [T k, H]: the tokens' rows x [T, H] (bf16, fp16 or fp32) in the align
    buffer's sorted order, by expert and adapter. Rows past the last kept one are zero, or left as
    they are in a given `out`. Differentiable (without `out`): the gradient is moe_unpermute without
    weights."""
    _rows(x, "x", _ANY, al.T)
    if out is not None:
        _rows(out, "out", (x.dtype,), al.S, x.shape[1])
        _apart("moe_permute", out, x, al.buf)
    stream = _here("moe_permute", x, al.buf, out)
    if out is None and _wants(x):
        return _Permute.apply(x, al)
    if forward_ad._current_level >= 0:
        _no_tangents("moe_permute", x)
    return _permute(x, al, out, stream)


def moe_unpermute(o: torch.Tensor, al: Align, w: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y[t] = sum over j of w[t, j] o[row(t, j)], [T, H]: the sorted rows o [T k, H] (bf16, fp16 or
    fp32) back at their tokens, summed with the routing weights w [T, k] (fp32; None: ones) in fp32 and
    rounded once. Dropped slots add nothing. Differentiable in o and w (without `out`)."""
    _rows(o, "o", _ANY, al.S)
    if w is not None and not _fits(w, torch.float32, (al.T, al.k)):
        _need(w, "w", torch.float32, 2, (al.T, al.k))
    if out is not None:
        _rows(out, "out", (o.dtype,), al.T, o.shape[1])
        _apart("moe_unpermute", out, o, al.buf, w)
    stream = _here("moe_unpermute", o, al.buf, w, out)
    if out is None and _wants(o, w):
        return _Unpermute.apply(o, w, al)
    if forward_ad._current_level >= 0:
        _no_tangents("moe_unpermute", *((o,) if w is None else (o, w)))
    return _unpermute(o, al, w, out, stream)


def moe_unpermute_backward(dy: torch.Tensor, o: Optional[torch.Tensor], al: Align, w: Optional[torch.Tensor] = None,
                           need_do: bool = True, need_dw: bool = True):
    """(do, dw) of moe_unpermute for dy [T, H]: do[row(t, j)] = w[t, j] dy[t] (zero in rows past the
    last kept one) and dw[t, j] = <o[row(t, j)], dy[t]> (fp32; zero for a dropped slot). None for one that
    is not wanted; o may be None where dw is not."""
    _rows(dy, "dy", _ANY, al.T)
    H, dtype = dy.shape[1], dy.dtype
    if need_dw and o is None:
        raise ValueError("dw needs o")
    if o is not None:
        _rows(o, "o", (dtype,), al.S, H)
    if w is not None and not _fits(w, torch.float32, (al.T, al.k)):
        _need(w, "w", torch.float32, 2, (al.T, al.k))
    stream = _here("moe_unpermute_backward", dy, o, al.buf, w)
    if forward_ad._current_level >= 0:
        _no_tangents("moe_unpermute_backward", *(t for t in (dy, o, w) if t is not None))
    do = torch.empty((al.S, H), dtype=dtype, device=dy.device) if need_do else None
    dw = torch.empty((al.T, al.k), dtype=torch.float32, device=dy.device) if need_dw else None
    st = lib().moe_unpermute_backward(dy.data_ptr(), ptr(o), DTYPES[dtype], al.ref(), ptr(w), H, L_.ROWS_ZERO_DROPPED,
                                      ptr(do), ptr(dw), stream)
    if st:
        check(st, "moe_unpermute_backward")
    return do, dw


# ---------------------------------------------------------------------------
# a projection with adapters
# ---------------------------------------------------------------------------
def _linear_shapes(x, W, A, B, al, rows_sorted):
    """(R, N, K, r) of valid operands: rows, output columns, input columns, rank."""
    R, E, L = al.T * al.k, al.E, al.L
    if isinstance(x, torch.Tensor) and isinstance(W, torch.Tensor) and isinstance(A, torch.Tensor):
        dtype, ws, dims = x.dtype, W.shape, W.dim()
        if (dtype in _16 and A.dim() == dims + 1 and (dims == 3 or (dims == 2 and E == 1))
                and (rows_sorted or al.k == 1) and L >= 1):
            N, K, r = ws[-2], ws[-1], A.shape[-2]
            lead = (E,) if dims == 3 else ()
            if (_fits(x, dtype, (R, K)) and _fits(W, dtype, (*lead, N, K)) and _fits(A, dtype, (L, *lead, r, K))
                    and _fits(B, dtype, (L, *lead, N, r))):
                return R, N, K, r
    # one by one, for the message
    for t, name in ((x, "x"), (W, "W"), (A, "A"), (B, "B")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype not in _16:
        raise ValueError(f"x must be torch.bfloat16 or torch.float16, got {x.dtype}")
    if not rows_sorted and al.k != 1:
        raise ValueError(f"rows in the tokens' order need k = 1, the align buffer has k = {al.k}: "
                         "lay them out with moe_permute and pass rows_sorted=True")
    if L < 1:
        raise ValueError("the align buffer has no adapters")
    if W.dim() == 2 and E != 1:
        raise ValueError(f"W must have shape ({E}, N, K), got {tuple(W.shape)}")
    lead, dims = ((), 2) if W.dim() == 2 else ((E,), 3)
    _need(W, "W", x.dtype, dims)
    N, K = W.shape[-2:]
    if A.dim() != dims + 1:
        raise ValueError(f"A must have {dims + 1} dims, got {tuple(A.shape)}")
    r = A.shape[-2]
    _need(x, "x", x.dtype, 2, (R, K))
    _need(W, "W", x.dtype, dims, (*lead, N, K))
    _need(A, "A", x.dtype, dims + 1, (L, *lead, r, K))
    _need(B, "B", x.dtype, dims + 1, (L, *lead, N, r))
    return R, N, K, r


def moe_lora_linear_workspace_size(al: Align, N: int, K: int, r: int, rows_sorted: bool = False,
                                   backward: bool = False) -> int:
    return al.linear_workspace_size(N, K, r, L_.ROWS_SORTED if rows_sorted else 0, int(backward))


def _workspace(workspace, al, N, K, r, flags, backward, like):
    if workspace is not None:
        return _need(workspace, "workspace", torch.uint8, 1), workspace.numel()
    n = al.linear_workspace_size(N, K, r, flags, backward)
    if n == 0:
        raise L_.MoeLoraError(L_.ERR_UNSUPPORTED, "moe_lora_linear_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=like.device), n


def _linear(x, W, A, B, al, rows_sorted, out, workspace, shapes, stream):
    R, N, K, r = shapes
    flags = L_.ROWS_SORTED if rows_sorted else 0
    if out is None:
        out = torch.empty((R, N), dtype=x.dtype, device=x.device)
        flags |= L_.ROWS_ZERO_DROPPED
    else:
        _written(out)
    workspace, n = _workspace(workspace, al, N, K, r, flags, 0, x)
    st = lib().moe_lora_linear(x.data_ptr(), W.data_ptr(), A.data_ptr(), B.data_ptr(), DTYPES[x.dtype], al.ref(), N, K,
                               r, flags, out.data_ptr(), workspace.data_ptr(), n, stream)
    if st:
        check(st, "moe_lora_linear")
    return out


class _LoraLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, A, B, al, rows_sorted, shapes):
        ctx.save_for_backward(x, W, A, B, al.buf)
        ctx.al, ctx.rows_sorted = al.kept(), rows_sorted
        return _linear(x, W, A, B, al, rows_sorted, None, None, shapes, stream_handle())

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, W, A, B, buf = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx, dA, dB = moe_lora_linear_backward(_grad_rows(dy, 16), x, W, A, B, _order(ctx, buf),
                                              rows_sorted=ctx.rows_sorted, need_dx=need[0], need_dA=need[2], need_dB=need[3])
        return dx, None, dA, dB, None, None, None


def moe_lora_linear(x: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, al: Align, *,
                    rows_sorted: bool = False, out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x W^T + (x A^T) B^T with each row's own adapter: one projection W [N, K] shared by every row
    with A [L, r, K] and B [L, N, r], or one per expert, W [E, N, K], A [L, E, r, K], B [L, E, N, r];
    bf16 or fp16. `al` is the align buffer of the rows' experts (zeros for one projection) and adapters
    (-1: W alone); one serves every projection that the rows go through. Rows are in the tokens' order
    (k = 1) or, rows_sorted, in its sorted order, as moe_permute lays them out. Dropped rows are zero, or
    left as they are in a given `out`. N, K and r are multiples of 8, r at most 128.

    Differentiable in x, A and B (without `out`); W is frozen, and one that requires a gradient is
    refused."""
    shapes = _linear_shapes(x, W, A, B, al, rows_sorted)
    if out is not None:
        if not _fits(out, x.dtype, shapes[:2]):
            _need(out, "out", x.dtype, 2, shapes[:2])
        _apart("moe_lora_linear", out, x, W, A, B, al.buf, workspace)
    stream = _here("moe_lora_linear", x, W, A, B, al.buf, out, workspace)
    if W.requires_grad and torch.is_grad_enabled():
        raise ValueError("W is frozen and has no gradient here: pass W.detach()")
    if out is None and _wants(x, A, B):
        if workspace is not None:
            raise ValueError("a differentiable call takes no workspace")
        return _LoraLinear.apply(x, W, A, B, al, rows_sorted, shapes)
    if forward_ad._current_level >= 0:
        _no_tangents("moe_lora_linear", x, W, A, B)
    return _linear(x, W, A, B, al, rows_sorted, out, workspace, shapes, stream)


def moe_lora_linear_backward(dy: torch.Tensor, x: torch.Tensor, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                             al: Align, *, rows_sorted: bool = False, need_dx: bool = True, need_dA: bool = True,
                             need_dB: bool = True, workspace: Optional[torch.Tensor] = None):
    """(dx, dA, dB) of moe_lora_linear for dy [rows, N]; None for one that is not wanted. x A^T is
    computed again: nothing is kept from the forward pass. Rows of dx that were dropped are zero, and
    so are the gradients of adapters without a row."""
    R, N, K, r = _linear_shapes(x, W, A, B, al, rows_sorted)
    if not _fits(dy, x.dtype, (R, N)):
        _need(dy, "dy", x.dtype, 2, (R, N))
    stream = _here("moe_lora_linear_backward", dy, x, W, A, B, al.buf, workspace)
    if forward_ad._current_level >= 0:
        _no_tangents("moe_lora_linear_backward", dy, x, W, A, B)
    dtype, device = x.dtype, x.device
    dx = torch.empty((R, K), dtype=dtype, device=device) if need_dx else None
    dA = torch.empty(A.shape, dtype=dtype, device=device) if need_dA else None
    dB = torch.empty(B.shape, dtype=dtype, device=device) if need_dB else None
    flags = L_.ROWS_ZERO_DROPPED | (L_.ROWS_SORTED if rows_sorted else 0)
    workspace, n = _workspace(workspace, al, N, K, r, flags, 1, x)
    st = lib().moe_lora_linear_backward(dy.data_ptr(), x.data_ptr(), W.data_ptr(), A.data_ptr(), B.data_ptr(),
                                        DTYPES[x.dtype], al.ref(), N, K, r, flags, ptr(dx), ptr(dA), ptr(dB),
                                        workspace.data_ptr(), n, stream)
    if st:
        check(st, "moe_lora_linear_backward")
    return dx, dA, dB
