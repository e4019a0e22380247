"""Refusals of the entry points around the experts' products: on the host, before anything is
launched."""
import ctypes
import os

import pytest
import torch

import expert_adapter_gemms_gb300 as m
from expert_adapter_gemms_gb300._lib import AlignDesc

OK, INVALID, UNSUPPORTED, SMALL = 0, 1, 2, 4
P = 1 << 20  # a non-null, aligned address that no refused call may touch


@pytest.fixture(scope="session")
def L():
    from expert_adapter_gemms_gb300 import build as b
    if not os.path.exists(b.LIB_PATH):
        b.build()
    return m.lib()


def desc(buf=P, T=4, k=2, E=4, L=0, bm_base=256, bm_lora=16, ranks=None):
    return ctypes.byref(AlignDesc(buf, T, k, E, L, bm_base, bm_lora, ranks))


BAD_ALIGN = (dict(buf=0), dict(buf=P + 64))
BAD_SHAPE = (dict(T=-1), dict(k=0), dict(E=0), dict(bm_base=8), dict(bm_lora=0), dict(T=1 << 22, k=2))


def test_rows_refusals(L):
    def permute(x=P, dtype=0, al=None, H=64, flags=2, xs=P):
        return L.moe_permute(x, dtype, desc() if al is None else al, H, flags, xs, 0)

    def back(o=P, dtype=0, al=None, w=P, H=64, y=P):
        return L.moe_unpermute(o, dtype, desc() if al is None else al, w, H, y, 0)

    def grads(dy=P, o=P, dtype=0, al=None, w=P, H=64, flags=2, do=P, dw=P):
        return L.moe_unpermute_backward(dy, o, dtype, desc() if al is None else al, w, H, flags, do, dw, 0)

    for call in (permute, back, grads):
        for bad in (dict(dtype=3), dict(dtype=-1), dict(H=0), dict(H=-8)):
            assert call(**bad) == INVALID, (call, bad)
        assert call(H=(1 << 24) + 1) == UNSUPPORTED
        for bad in BAD_ALIGN:
            assert call(al=desc(**bad)) == INVALID, bad
        for bad in BAD_SHAPE:
            assert call(al=desc(**bad)) == UNSUPPORTED, bad
    for call, bad in ((permute, dict(x=0)), (permute, dict(xs=0)), (permute, dict(x=P + 1)), (permute, dict(xs=P + 2, dtype=2)),
                      (permute, dict(flags=1)), (permute, dict(flags=4)),
                      (back, dict(o=0)), (back, dict(y=0)), (back, dict(w=P + 2)), (back, dict(o=P + 2, dtype=2)),
                      (grads, dict(dy=0)), (grads, dict(o=0)), (grads, dict(dw=P + 2)), (grads, dict(do=P + 1)),
                      (grads, dict(w=P + 1)), (grads, dict(flags=1))):
        assert call(**bad) == INVALID, (call, bad)
    empty = desc(T=0)
    assert permute(al=empty, x=0, xs=0) == OK and back(al=empty, o=0, y=0) == OK
    assert grads(al=empty, dy=0, o=0, do=0, dw=0) == OK
    assert grads(do=0, dw=0) == OK


def test_router_gradient_refusals(L):
    def call(dw=P, ids=P, w=P, T=4, E=8, k=2, dl=P):
        return L.moe_topk_softmax_backward(dw, ids, w, T, E, k, dl, 0)

    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(dw=0), dict(ids=0), dict(w=0), dict(dl=0),
                dict(E=64, k=33)):
        assert call(**bad) == INVALID, bad
    assert call(E=1025) == UNSUPPORTED
    assert call(T=0, dw=0, ids=0, w=0, dl=0) == OK


def linear_desc(**kw):
    return desc(**{**dict(T=40, k=1, E=2, L=3), **kw})


def test_linear_refusals(L):
    size = L.moe_lora_linear_workspace_size
    big = 1 << 40

    def forward(x=P, W=P, A=P, B=P, dtype=0, al=None, N=64, K=128, r=16, flags=2, y=P, ws=P, n=big):
        return L.moe_lora_linear(x, W, A, B, dtype, linear_desc() if al is None else al, N, K, r, flags, y, ws, n, 0)

    def backward(x=P, W=P, A=P, B=P, dtype=0, al=None, N=64, K=128, r=16, flags=2, y=P, ws=P, n=big, dx=P, dA=P, dB=P):
        return L.moe_lora_linear_backward(y, x, W, A, B, dtype, linear_desc() if al is None else al, N, K, r, flags, dx,
                                          dA, dB, ws, n, 0)

    for call in (forward, backward):
        for bad in (dict(dtype=2), dict(dtype=-1), dict(N=0), dict(K=-8), dict(r=0), dict(flags=4), dict(x=0), dict(W=0),
                    dict(A=0), dict(B=0), dict(y=0), dict(ws=0), dict(x=P + 8), dict(W=P + 2), dict(A=P + 4), dict(B=P + 8),
                    dict(y=P + 8), dict(ws=P + 16), dict(al=linear_desc(L=0)),
                    dict(al=linear_desc(k=2))):  # slots are no tokens
            assert call(**bad) == INVALID, bad
        for bad in (dict(N=60), dict(K=4), dict(r=12), dict(r=136), dict(N=1 << 21), dict(K=1 << 21),
                    dict(N=1 << 20, K=1 << 20), dict(al=linear_desc(E=2048, L=1024)), dict(al=linear_desc(ranks=P))):
            assert call(**bad) == UNSUPPORTED, bad
        for bad in BAD_ALIGN:
            assert call(al=linear_desc(**bad)) == INVALID, bad
        for bad in BAD_SHAPE:
            assert call(al=linear_desc(**bad)) == UNSUPPORTED, bad
        n = size(linear_desc(), 64, 128, 16, 2, int(call is backward))
        assert n > 0 and call(n=n - 1) == SMALL
    for bad in (dict(dx=P + 8), dict(dA=P + 8), dict(dB=P + 2)):
        assert backward(**bad) == INVALID, bad
    assert backward(dx=0, dA=0, dB=0) == OK
    assert forward(al=linear_desc(T=0), x=0, W=0, A=0, B=0, y=0, ws=0) == OK
    # tiles of either direction counted in 30 bits: 2^18 + 1 of 16 rows by 2^14 of 64 columns
    many = dict(al=linear_desc(T=1 << 22, E=1, bm_base=16))
    assert forward(N=1 << 18, **many) == UNSUPPORTED and backward(K=1 << 18, **many) == UNSUPPORTED


def test_linear_workspace(L):
    size = L.moe_lora_linear_workspace_size
    al = linear_desc(T=1000, E=1, L=3)
    z, copies = 1000 * 16 * 4, 1000 * 128 * 2
    assert z <= size(al, 64, 128, 16, 1, 0) < z + 1024        # sorted rows: z alone
    assert z + copies <= size(al, 64, 128, 16, 0, 0) < z + copies + 1024
    assert 2 * z + 1000 * 64 * 2 <= size(al, 64, 128, 16, 0, 1) < 2 * z + 1000 * 64 * 2 + 2048
    assert size(linear_desc(T=100, E=1, L=3), 64, 128, 16, 0, 0) < 100 * 16 * 4 + 1024  # few rows: no copies
    assert size(al, 64, 128, 12, 0, 0) == 0 and size(al, 60, 128, 16, 0, 0) == 0 and size(None, 64, 128, 16, 0, 0) == 0
    assert size(linear_desc(k=2), 64, 128, 16, 0, 0) == 0 and size(linear_desc(k=2), 64, 128, 16, 1, 0) > 0
    assert size(linear_desc(T=0), 64, 128, 16, 0, 1) > 0


def fake_align(T=4, k=2, E=4, L=0):
    return m.Align(torch.zeros(1 << 12, dtype=torch.uint8), T, k, E, L, 256, 16)


def test_python_refuses_cpu_tensors_and_shapes(L):
    al = fake_align()
    x, o, w = torch.zeros(4, 16), torch.zeros(8, 16), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_permute(x, al)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_unpermute(o, al)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_unpermute_backward(x, o, al)
    for call in (lambda: m.moe_permute(torch.zeros(5, 16), al), lambda: m.moe_permute(torch.zeros(4, 16, 1), al),
                 lambda: m.moe_permute(torch.zeros(4, 32)[:, ::2], al), lambda: m.moe_permute(x.double(), al),
                 lambda: m.moe_permute(torch.zeros(4, 0), al), lambda: m.moe_permute(x, al, out=torch.zeros(8, 15)),
                 lambda: m.moe_unpermute(x, al), lambda: m.moe_unpermute(o, al, torch.zeros(4, 3)),
                 lambda: m.moe_unpermute(o, al, w.half()), lambda: m.moe_unpermute(o, al, out=torch.zeros(8, 16)),
                 lambda: m.moe_unpermute_backward(x, o.half(), al), lambda: m.moe_unpermute_backward(x, None, al),
                 lambda: m.moe_unpermute_backward(o, o, al)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        m.moe_permute([1.0], al)


def test_python_refuses_linear_operands(L):
    bf = torch.bfloat16
    one = fake_align(T=4, k=1, E=1, L=2)
    x, W, A, B = torch.zeros(4, 64, dtype=bf), torch.zeros(32, 64, dtype=bf), torch.zeros(2, 8, 64, dtype=bf), \
        torch.zeros(2, 32, 8, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_lora_linear(x, W, A, B, one)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_lora_linear_backward(torch.zeros(4, 32, dtype=bf), x, W, A, B, one)
    for args in ((x.float(), W, A, B), (x[:3], W, A, B), (x, W.half(), A, B), (x, W[:, :56], A, B), (x, W, A[:1], B),
                 (x, W, A, B[:, :, :4]), (x, W, A[0], B), (x, W[None], A, B), (x.t(), W, A, B)):
        with pytest.raises(ValueError):
            m.moe_lora_linear(*args, one)
    with pytest.raises(TypeError):
        m.moe_lora_linear(x, None, A, B, one)
    with pytest.raises(ValueError, match="rows_sorted"):
        m.moe_lora_linear(x, W, A, B, fake_align(T=2, k=2, E=1, L=2))
    with pytest.raises(ValueError, match="no adapters"):
        m.moe_lora_linear(x, W, A, B, fake_align(T=4, k=1, E=1, L=0))
    with pytest.raises(ValueError, match="shape"):
        m.moe_lora_linear(x, W, A, B, fake_align(T=4, k=1, E=2, L=2))


def test_align_reference_follows_the_buffer(L):
    """The kept description is made anew when a field or the buffer changes."""
    al = fake_align(T=4, k=1, E=1, L=2)
    first = al.ref()
    assert al.ref() is first and first._obj.T == 4
    n = al.linear_workspace_size(64, 64, 8, 0, 0)
    al.T = 300
    assert al.ref() is not first and al.ref()._obj.T == 300 and al.linear_workspace_size(64, 64, 8, 0, 0) > n
    kept = al.ref()
    al.buf = torch.zeros(1 << 13, dtype=torch.uint8)
    assert al.ref() is not kept and al.ref()._obj.buf == al.buf.data_ptr()
    kept = al.ref()
    al.buf.set_(torch.zeros(1 << 14, dtype=torch.uint8))
    assert al.ref()._obj.buf == al.buf.data_ptr() and kept._obj.buf != al.buf.data_ptr()


def test_python_refuses_out_over_its_inputs(L):
    """Rows are written while others are still read: an `out` over an input's memory is refused, and one
    that only touches it is not (it goes on to the refusal of tensors that are not on the GPU)."""
    bf = torch.bfloat16
    al = fake_align(T=4, k=1, E=1, L=2)
    mem = torch.zeros(12, 64, dtype=bf)
    x, w = mem[4:8], torch.zeros(4, 1)
    W, A, B = torch.zeros(64, 64, dtype=bf), torch.zeros(2, 8, 64, dtype=bf), torch.zeros(2, 64, 8, dtype=bf)
    ws = torch.zeros(1 << 12, dtype=torch.uint8)
    calls = (lambda out: m.moe_permute(x, al, out=out), lambda out: m.moe_unpermute(x, al, w, out=out),
             lambda out: m.moe_lora_linear(x, W, A, B, al, out=out, workspace=ws))
    for call in calls:
        for first in (4, 1, 7):
            with pytest.raises(ValueError, match="shares memory"):
                call(mem[first:first + 4])
        for first in (0, 8):
            with pytest.raises(ValueError, match="CUDA"):
                call(mem[first:first + 4])
    for t in (W, A.view(16, 64), B.view(16, 64), ws.view(bf).view(-1, 64)):
        with pytest.raises(ValueError, match="shares memory"):
            calls[2](t[:4])
    wide = torch.zeros(4, 1)
    with pytest.raises(ValueError, match="shares memory"):
        m.moe_unpermute(torch.zeros(4, 1), al, wide, out=wide)
    with pytest.raises(ValueError, match="shares memory"):
        m.moe_permute(x, al, out=al.buf.view(bf)[:256].view(4, 64))
    empty = fake_align(T=0, k=1, E=1, L=2)
    none = torch.zeros(0, 64)
    with pytest.raises(ValueError, match="CUDA"):
        m.moe_permute(none, empty, out=none)
