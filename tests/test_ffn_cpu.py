"""Refusals of the feed-forward entry points: on the host, before anything is launched."""
import ctypes
import math
import os

import pytest
import torch

import expert_adapter_gemms_gb300 as m

OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 4
P = 1 << 20  # a non-null, aligned address that no refused call may touch


@pytest.fixture(scope="session")
def L():
    from expert_adapter_gemms_gb300 import build as b
    if not os.path.exists(b.LIB_PATH):
        b.build()
    return m.lib()


def test_gated_refusals(L):
    def call(x=P, W1=P, dtype=0, act=1, T=4, H=64, I=32, h=P):
        return L.moe_gated_ffn(x, W1, dtype, act, T, H, I, h, 0)

    for bad in (dict(dtype=2), dict(dtype=-1), dict(act=0), dict(act=3), dict(T=-1), dict(H=0), dict(I=0),
                dict(x=0), dict(W1=0), dict(h=0), dict(x=P + 2), dict(W1=P + 8), dict(h=P + 4)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=63), dict(H=4), dict(I=12), dict(T=(1 << 22) + 1), dict(H=1 << 22), dict(I=1 << 21)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(T=0, x=0, W1=0, h=0) == OK


def test_gated_backward_refusals(L):
    size = L.moe_gated_ffn_backward_workspace_size

    def call(dh=P, x=P, W1=P, dtype=0, act=1, T=4, H=64, I=32, dx=P, dW1=P, ws=P, n=None):
        return L.moe_gated_ffn_backward(dh, x, W1, dtype, act, T, H, I, dx, dW1, ws,
                                        size(4, 64, 32) if n is None else n, 0)

    for bad in (dict(dtype=2), dict(act=0), dict(T=-1), dict(dh=0), dict(x=0), dict(W1=0), dict(dh=P + 2),
                dict(dx=P + 2), dict(dW1=P + 8), dict(ws=0), dict(ws=P + 16)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(H=60), dict(I=33)):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(n=size(4, 64, 32) - 1) == SMALL
    assert call(dx=0, dW1=0) == OK
    assert size(4, 60, 32) == 0 and size(-1, 64, 32) == 0
    assert size(4, 64, 32) >= 4 * 64 * 2 and size(0, 64, 32) > 0


def test_clip_refusals(L):
    def call(n=2, numels=(5, 7), dtypes=(0, 2), grads=(P, P), outs=(P, P), max_norm=1.0, norm=P, ws=P,
             ws_bytes=None):
        c64, c32, cp = ctypes.c_int64 * 2, ctypes.c_int32 * 2, ctypes.c_void_p * 2
        c = c64(*numels) if numels else None
        need = L.moe_grad_clip_workspace_size(max(n, 0), c) if ws_bytes is None else ws_bytes
        return L.moe_grad_clip(cp(*grads) if grads else None, cp(*outs) if outs else None, c,
                               c32(*dtypes) if dtypes else None, n, max_norm, norm, ws, need, 0)

    for bad in (dict(n=-1), dict(numels=(5, -1), ws_bytes=1 << 20), dict(dtypes=(0, 3)), dict(dtypes=(-1, 0)),
                dict(grads=(P, 0)), dict(grads=(P + 1, P)), dict(grads=(P, P + 2)), dict(outs=(P, 0)),
                dict(outs=(P + 1, P)), dict(max_norm=-1.0), dict(max_norm=math.nan), dict(norm=0),
                dict(ws=0), dict(ws=P + 4), dict(grads=None), dict(numels=None, ws_bytes=1 << 20),
                dict(dtypes=None)):
        assert call(**bad) == INVALID, bad
    assert call(numels=(1 << 41, 1)) == UNSUPPORTED
    assert call(ws_bytes=8) == SMALL
    assert L.moe_grad_clip_workspace_size(-1, None) == 0
    assert L.moe_grad_clip_workspace_size(2, None) == 0


def test_w4_refusals(L):
    size = L.moe_w4_packed_size
    assert size(1, 16, 128, 32, 0, 0) == 1024 + 128 and size(1, 16, 128, 32, 1, 0) == 1024 + 128 + 64
    assert size(2, 17, 129, 128, 0, 0) == 2 * 2 * 2 * (1024 + 32)
    assert size(1, 18, 128, 32, 0, 1) == 2 * (1024 + 128)
    for bad in ((0, 16, 128, 32, 0, 0), (1, 0, 128, 32, 0, 0), (1, 16, 0, 32, 0, 0), (1, 16, 128, 16, 0, 0),
                (1, 17, 128, 32, 0, 1)):
        assert size(*bad) == 0, bad

    def pack(codes=P, scales=P, zeros=0, E=1, N=16, K=128, group=32, gated=0, packed=P):
        return L.moe_w4_pack(codes, scales, zeros, E, N, K, group, gated, packed, 0)

    for bad in (dict(codes=0), dict(scales=0), dict(packed=0), dict(packed=P + 8)):
        assert pack(**bad) == INVALID, bad
    for bad in (dict(group=48), dict(N=15, gated=1), dict(E=0)):
        assert pack(**bad) == UNSUPPORTED, bad

    def quant(W=P, dtype=0, E=1, N=16, K=128, group=32, codes=P, scales=P):
        return L.moe_w4_quantize(W, dtype, E, N, K, group, codes, scales, 0)

    for bad in (dict(W=0), dict(dtype=2), dict(codes=0), dict(scales=0)):
        assert quant(**bad) == INVALID, bad
    assert quant(group=33) == UNSUPPORTED

    def mul(x=P, dtype=0, packed=P, E=1, N=16, K=128, group=32, zeros=0, gated=1, act=0, T=4, al=None,
            rows_sorted=0, out=P, out_fp32=0):
        return L.moe_w4_matvec(x, dtype, packed, E, N, K, group, zeros, gated, act, T, al, rows_sorted, out,
                               out_fp32, 0)

    for bad in (dict(dtype=2), dict(act=3), dict(act=-1), dict(act=1, gated=0), dict(act=1, out_fp32=1),
                dict(T=-1), dict(E=2), dict(x=0), dict(packed=0), dict(out=0), dict(x=P + 8),
                dict(packed=P + 8), dict(out=P + 1), dict(out=P + 2, out_fp32=1)):
        assert mul(**bad) == INVALID, bad
    for bad in (dict(K=12), dict(group=31), dict(N=7)):
        assert mul(**bad) == UNSUPPORTED, bad
    assert mul(T=0, x=0, packed=0, out=0) == OK


def test_w4_row_flags(L):
    def mul(flags, x=P):
        return L.moe_w4_matvec(x, 0, P, 1, 16, 128, 32, 0, 1, 0, 0, None, flags, P, 0, 0)

    assert [mul(f) for f in (0, 1, 2, 3)] == [OK] * 4  # T = 0
    assert mul(4) == INVALID and mul(-1) == INVALID


def test_python_refusals_on_the_host():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    W1 = torch.zeros((32, 64), dtype=torch.bfloat16)
    for f in (lambda: m.moe_gated_ffn(x, W1), lambda: m.moe_gated_ffn_backward(x, x, W1),
              lambda: m.moe_grad_clip([x], 1.0), lambda: m.moe_w4_quantize(W1),
              lambda: m.moe_gated_ffn(x.float(), W1), lambda: m.moe_grad_clip([x.int()], 1.0)):
        with pytest.raises(ValueError):  # on the CPU, or of another type
            f()
    with pytest.raises(TypeError):
        m.moe_gated_ffn(None, W1)
