"""The feed-forward block by itself: training, gradient clipping and 4-bit serving.

Thin like :mod:`.api`: tensors are checked, outputs allocated, and the C entry points of the
same names called on the current stream; nothing here computes. Tensors are contiguous and
on one GPU.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from operator import attrgetter
from typing import Optional, Sequence

import torch

from . import _lib as L_
from ._lib import check, lib, ptr, stream_handle
from .api import Align, _need, _no_tangents

try:  # a compiled look at the type, sizes and strides of many tensors at once
    from torch._C._dynamo.guards import TensorGuards as _TensorGuards
except ImportError:
    _TensorGuards = None

ACTS = {None: L_.ACT_NONE, "silu": L_.ACT_SILU, "gelu": L_.ACT_GELU}
_16 = (torch.bfloat16, torch.float16)
DTYPES = {torch.bfloat16: L_.DTYPE_BF16, torch.float16: L_.DTYPE_FP16, torch.float32: L_.DTYPE_FP32}


def _need16(t: torch.Tensor, name: str, ndim: int, shape=None):
    """A contiguous bf16 or fp16 CUDA tensor."""
    if isinstance(t, torch.Tensor) and t.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    return _need(t, name, t.dtype if isinstance(t, torch.Tensor) else None, ndim, shape)


def _same(t, dtype, shape) -> bool:
    """Whether t is a contiguous CUDA tensor of this type and shape: one look, no message (the
    checks of _need one by one cost microseconds that a small product does not take)."""
    return (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.shape == shape
            and t.is_contiguous())


def _act(act: Optional[str], gated: bool = True) -> int:
    if act not in ACTS or (gated and act is None):
        raise ValueError(f"act must be 'silu' or 'gelu'{'' if gated else ' or None'}, got {act!r}")
    return ACTS[act]


def ffn_get_error() -> int:
    """The sticky device error word of the gated block's kernels (0: no error)."""
    v = ctypes.c_uint32(0)
    st = lib().moe_ffn_get_error(stream_handle(), ctypes.byref(v))
    if st not in (L_.OK, L_.ERR_TIMEOUT):
        check(st, "moe_ffn_get_error")
    return int(v.value)


def ffn_clear_error() -> None:
    check(lib().moe_ffn_clear_error(stream_handle()), "moe_ffn_clear_error")


def ffn_set_wait_limit(ns: int) -> None:
    """The limit of the gated block's device waits in this thread's later calls (tests of the
    give-up path): 0 the default of 4 s, < 0 give up at once."""
    check(lib().moe_ffn_set_wait_limit(int(ns)), "moe_ffn_set_wait_limit")


# ---------------------------------------------------------------------------
# the gated block
# ---------------------------------------------------------------------------
def _gated_shapes(x, W1):
    """(T, H, I) of valid x and W1."""
    if isinstance(x, torch.Tensor) and isinstance(W1, torch.Tensor):
        dtype, xs, ws = x.dtype, x.shape, W1.shape
        if (dtype in _16 and W1.dtype is dtype and len(xs) == 2 and len(ws) == 2 and ws[1] == xs[1] and ws[0] % 2 == 0
                and x.is_cuda and W1.is_cuda and x.is_contiguous() and W1.is_contiguous()):
            return xs[0], xs[1], ws[0] // 2
    _need16(x, "x", 2)
    _need(W1, "W1", x.dtype, 2)
    raise ValueError(f"W1 must have shape (2I, {x.shape[1]}), got {tuple(W1.shape)}")


def _gated_forward(x, W1, act, out, shapes):
    T, H, I = shapes
    dtype = x.dtype
    if out is None:
        out = torch.empty((T, I), dtype=dtype, device=x.device)
    else:
        _need(out, "out", dtype, 2, (T, I))
    st = lib().moe_gated_ffn(x.data_ptr(), W1.data_ptr(), DTYPES[dtype], _act(act), T, H, I, out.data_ptr(),
                             stream_handle())
    if st:
        check(st, "moe_gated_ffn")
    return out


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W1, act):
        ctx.save_for_backward(x, W1)
        ctx.act = act
        return _gated_forward(x, W1, act, None, (*x.shape, W1.shape[0] // 2))

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        x, W1 = ctx.saved_tensors
        dh = dh.contiguous()
        if dh.data_ptr() % 16:  # a slice of a larger gradient: autograd chose where it starts
            dh = dh.clone()
        dx, dW1 = moe_gated_ffn_backward(dh, x, W1, act=ctx.act,
                                         need_dx=ctx.needs_input_grad[0],
                                         need_dW1=ctx.needs_input_grad[1])
        return dx, dW1, None


def moe_gated_ffn(x: torch.Tensor, W1: torch.Tensor, act: str = "silu",
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """h = act(x Wg^T) * (x Wu^T), [T, I], for x [T, H] and W1 [2I, H] (gate rows first), bf16
    or fp16. Differentiable: where x or W1 require a gradient (and no `out` is given) the
    backward pass is moe_gated_ffn_backward, which keeps nothing but x and W1. Neither has a
    forward-mode derivative: tensors with a tangent are refused."""
    shapes = _gated_shapes(x, W1)
    if out is None and (x.requires_grad or W1.requires_grad) and torch.is_grad_enabled():
        return _GatedFFN.apply(x, W1, act)  # which refuses forward-mode inputs itself
    _no_tangents("moe_gated_ffn", x, W1)
    return _gated_forward(x, W1, act, out, shapes)


def moe_gated_ffn_backward_workspace_size(T: int, H: int, I: int) -> int:
    return int(lib().moe_gated_ffn_backward_workspace_size(T, H, I))


def moe_gated_ffn_backward(dh: torch.Tensor, x: torch.Tensor, W1: torch.Tensor, act: str = "silu",
                           need_dx: bool = True, need_dW1: bool = True,
                           workspace: Optional[torch.Tensor] = None):
    """(dx, dW1) of moe_gated_ffn for dh [T, I]; None for one that is not wanted."""
    T, H, I = _gated_shapes(x, W1)
    dtype, device = x.dtype, x.device
    if not _same(dh, dtype, (T, I)):
        _need(dh, "dh", dtype, 2, (T, I))
    _no_tangents("moe_gated_ffn_backward", dh, x, W1)
    a = _act(act)
    dx = torch.empty((T, H), dtype=dtype, device=device) if need_dx else None
    dW1 = torch.empty((2 * I, H), dtype=dtype, device=device) if need_dW1 else None
    if workspace is None:
        n = moe_gated_ffn_backward_workspace_size(T, H, I)
        if n == 0:
            raise L_.MoeLoraError(L_.ERR_UNSUPPORTED, "moe_gated_ffn_backward_workspace_size")
        workspace = torch.empty(n, dtype=torch.uint8, device=device)
    else:
        _need(workspace, "workspace", torch.uint8, 1)
        n = workspace.numel()
    st = lib().moe_gated_ffn_backward(dh.data_ptr(), x.data_ptr(), W1.data_ptr(), DTYPES[dtype], a, T, H, I, ptr(dx),
                                      ptr(dW1), workspace.data_ptr(), n, stream_handle())
    if st:
        check(st, "moe_gated_ffn_backward")
    return dx, dW1


# ---------------------------------------------------------------------------
# gradient clipping
# ---------------------------------------------------------------------------
class GradClip:
    """The table of a program's gradient tensors, kept so that a clip costs two launches and
    no per-tensor work in Python: ``norm = GradClip(grads, out=...)(max_norm)``.

    grads: contiguous bf16, fp16 or fp32 CUDA tensors of any shapes, empty ones among them;
    out: tensors of the same shapes and types that receive the clipped gradients (default: in
    place). norm_only: no gradient is written. Each call looks at the tensors as they are then:
    one whose storage moved is followed, one whose size, type, layout or device changed is
    refused."""

    def __init__(self, grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None,
                 norm_only: bool = False):
        self.grads = list(grads)
        self.outs = None if norm_only else (self.grads if out is None else list(out))
        n = len(self.grads)
        if norm_only and out is not None:
            raise ValueError("norm_only takes no out")
        if self.outs is not None and len(self.outs) != n:
            raise ValueError("out must have one tensor per gradient")
        for i, g in enumerate(self.grads):
            if isinstance(g, torch.Tensor) and g.dtype not in DTYPES:
                raise ValueError(f"grads[{i}] must be bfloat16, float16 or float32, got {g.dtype}")
            _need(g, f"grads[{i}]", g.dtype if isinstance(g, torch.Tensor) else None)
            if self.outs is not None and out is not None:
                _need(self.outs[i], f"out[{i}]", g.dtype, None, g.shape)
        separate = self.outs is not None and self.outs is not self.grads
        self._all = self.grads + self.outs if separate else self.grads
        numels = [g.numel() for g in self.grads]
        self._numels = [t.numel() for t in self._all]
        self._dtypes = [t.dtype for t in self._all]
        self._guards, self._called = None, False
        self._c_numels = (ctypes.c_int64 * n)(*numels)
        self._c_dtypes = (ctypes.c_int32 * n)(*[DTYPES[g.dtype] for g in self.grads])
        self._in_ptrs = self._out_ptrs = None
        self._device = self.grads[0].device if n else torch.device("cuda")
        self._workspaces = {}
        self._workspace_bytes = int(lib().moe_grad_clip_workspace_size(n, self._c_numels))

    def __call__(self, max_norm: float) -> torch.Tensor:
        """Clips, and returns the norm before it (a 0-d fp32 tensor on the device)."""
        self._check_bound(max_norm)
        self._look()
        return self._clip(max_norm)

    @staticmethod
    def _check_bound(max_norm: float) -> None:
        if not max_norm >= 0:
            raise ValueError(f"max_norm must be at least 0, got {max_norm}")

    def _look(self) -> None:
        """Sees that every tensor has the size, type and layout that the table was made of: by
        guards that compare a tensor's at once where this torch has them, else one after the
        other (1500 gradients and outputs: 0.17 against 0.58 ms a call)."""
        if self._guards is not None and self._guards.check(*self._all):
            return
        every = self._all
        if (list(map(torch.Tensor.numel, every)) != self._numels or list(map(attrgetter("dtype"), every)) != self._dtypes
                or not all(map(attrgetter("is_cuda"), every)) or not all(map(torch.Tensor.is_contiguous, every))):
            raise ValueError("a tensor's size, type, layout or device changed: build a new GradClip")
        if not self._called:  # the guards take longer to make than one look: a second call needs them
            self._called = True
        elif _TensorGuards is not None:
            self._guards = _TensorGuards(*every, dynamic_dims_sizes=[list(t.shape) for t in every],
                                         dynamic_dims_strides=[list(t.stride()) for t in every])

    def _clip(self, max_norm: float) -> torch.Tensor:
        n = len(self.grads)
        ins = list(map(torch.Tensor.data_ptr, self.grads))
        if ins != self._in_ptrs:
            self._in_ptrs, self._c_in = ins, (ctypes.c_void_p * n)(*ins)
        if self.outs is not None and self.outs is not self.grads:
            outs = list(map(torch.Tensor.data_ptr, self.outs))
            if outs != self._out_ptrs:
                self._out_ptrs, self._c_out = outs, (ctypes.c_void_p * n)(*outs)
        # a workspace per stream, so that calls on several streams do not share one, and one of
        # its own for a call that a graph records: graphs recorded on one stream replay on others
        stream = stream_handle()
        workspace = None if torch.cuda.is_current_stream_capturing() else self._workspaces.get(stream)
        if workspace is None:
            workspace = torch.empty(self._workspace_bytes, dtype=torch.uint8, device=self._device)
            if not torch.cuda.is_current_stream_capturing():
                self._workspaces[stream] = workspace
        norm = torch.empty((), dtype=torch.float32, device=self._device)
        c_outs = None if self.outs is None else self._c_in if self.outs is self.grads else self._c_out
        st = lib().moe_grad_clip(self._c_in, c_outs, self._c_numels, self._c_dtypes, n, max_norm, norm.data_ptr(),
                                 workspace.data_ptr(), self._workspace_bytes, stream)
        if st:
            check(st, "moe_grad_clip")
        return norm


def moe_grad_clip(grads: Sequence[torch.Tensor], max_norm: float = math.inf,
                  out: Optional[Sequence[torch.Tensor]] = None, norm_only: bool = False) -> torch.Tensor:
    """The global norm of grads, and grads * min(1, max_norm / (norm + 1e-6)) in place or into
    `out`; an infinite max_norm scales nothing. For gradients that stay where they are, keep a
    GradClip."""
    plan = GradClip(grads, out, norm_only)  # whose tensors have just been looked at
    plan._check_bound(max_norm)
    return plan._clip(max_norm)


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
def moe_w4_quantize(W: torch.Tensor, group: int = 32):
    """(codes, scales) of W [E, N, K] or [N, K], bf16 or fp16: symmetric, zeros 8. Any K here;
    moe_w4_pack and the product take multiples of 8."""
    _need16(W, "W", W.dim() if isinstance(W, torch.Tensor) else None)
    if W.dim() not in (2, 3):
        raise ValueError(f"W must have 2 or 3 dims, got {tuple(W.shape)}")
    E = W.shape[0] if W.dim() == 3 else 1
    N, K = W.shape[-2:]
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    codes = torch.empty((E, N, (K + 1) // 2), dtype=torch.uint8, device=W.device)
    scales = torch.empty((E, N, -(-K // group)), dtype=W.dtype, device=W.device)
    check(lib().moe_w4_quantize(ptr(W), DTYPES[W.dtype], E, N, K, group, ptr(codes), ptr(scales),
                                stream_handle()), "moe_w4_quantize")
    return codes, scales


@dataclass
class W4Weight:
    """Weights [E, N, K] at 4 bits in moe_w4_matvec's layout."""
    packed: torch.Tensor
    dtype: torch.dtype
    E: int
    N: int
    K: int
    group: int
    has_zeros: bool
    gated: bool


def moe_w4_pack(codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None, *,
                group: int, gated: bool = False, K: Optional[int] = None) -> W4Weight:
    """Lays codes [E, N, ceil(K/2)], scales and zeros [E, N, ceil(K/group)] out for
    moe_w4_matvec. K: the columns (default: two per byte), a multiple of 8 up to 16384. gated:
    the rows are a gate and an up half, as the gated form needs."""
    _need(codes, "codes", torch.uint8, 3)
    E, N, kb = codes.shape
    K = 2 * kb if K is None else K
    if (K + 1) // 2 != kb:
        raise ValueError(f"codes hold {2 * kb} columns, not {K}")
    if group not in (32, 64, 128):
        raise ValueError(f"group must be 32, 64 or 128, got {group}")
    shape = (E, N, -(-K // group))
    _need16(scales, "scales", 3, shape)
    if zeros is not None:
        _need(zeros, "zeros", torch.uint8, 3, shape)
    n = int(lib().moe_w4_packed_size(E, N, K, group, int(zeros is not None), int(gated)))
    if n == 0:
        raise L_.MoeLoraError(L_.ERR_UNSUPPORTED, "moe_w4_packed_size")
    packed = torch.empty(n, dtype=torch.uint8, device=codes.device)
    check(lib().moe_w4_pack(ptr(codes), ptr(scales), ptr(zeros), E, N, K, group, int(gated), ptr(packed),
                            stream_handle()), "moe_w4_pack")
    return W4Weight(packed, scales.dtype, E, N, K, group, zeros is not None, gated)


def moe_w4_matvec(x: torch.Tensor, w: W4Weight, *, al: Optional[Align] = None, rows_sorted: bool = False,
                  act: Optional[str] = None, out_fp32: bool = False,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x W^T for a few rows of x, or with `act` the gated act(gate) * up of its two halves.

    Without `al`: w holds one matrix; x [T, K] gives [T, N]. With the align buffer of a
    routing: every row of its sorted order times its expert's matrix, [T k, N]; x [T, K]
    holds the tokens, or with rows_sorted [T k, K] rows in that order. out_fp32: fp32 sums,
    the base that lora_expand_add adds to. Rows of dropped slots are left as they are in
    `out`, zero in an output allocated here."""
    if not (isinstance(x, torch.Tensor) and x.dim() == 2 and _same(x, w.dtype, x.shape)):
        _need(x, "x", w.dtype, 2)
    T = R = x.shape[0]
    if al is not None:
        T, R = al.T, al.S
        if al.E != w.E:
            raise ValueError(f"the align buffer has {al.E} experts, the weights {w.E}")
        if x.shape[0] != (R if rows_sorted else T):
            raise ValueError(f"x must have {R if rows_sorted else T} rows, got {tuple(x.shape)}")
    elif w.E != 1:
        raise ValueError("weights of several experts need an align buffer")
    if x.shape[1] != w.K:
        raise ValueError(f"x must have {w.K} columns, got {tuple(x.shape)}")
    a = _act(act, gated=False)
    if act is not None and (not w.gated or out_fp32):
        raise ValueError("the gated form needs weights packed with gated=True, and has no fp32 output")
    shape = (R, w.N // 2 if act is not None else w.N)
    dtype = torch.float32 if out_fp32 else w.dtype
    flags = L_.W4_ROWS_SORTED if rows_sorted else 0
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
        flags |= L_.W4_ZERO_DROPPED
    else:
        _need(out, "out", dtype, 2, shape)
    d = ctypes.byref(al.desc()) if al is not None else None
    st = lib().moe_w4_matvec(x.data_ptr(), DTYPES[w.dtype], w.packed.data_ptr(), w.E, w.N, w.K, w.group, w.has_zeros,
                             w.gated, a, T, d, flags, out.data_ptr(), out_fp32, stream_handle())
    if st:
        check(st, "moe_w4_matvec")
    return out
