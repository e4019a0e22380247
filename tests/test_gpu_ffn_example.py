"""The operators as they are used together: the example, and a routed layer on 4-bit weights
with adapters through the library's own building blocks."""
import math
import os
import sys

import pytest
import torch

import gpu_util as gu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_train_clip_serve_example():
    gu.need_gpu()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_clip_serve
    finally:
        sys.path.pop(0)
    losses, off = train_clip_serve.main(steps=60, hidden=128, intermediate=256, tokens=512, quiet=True)
    assert losses[-1] < 0.7 * losses[0]
    # a 15-level code is off by 1/14 of its group's largest weight at most, evenly spread: about
    # 0.041 of 2.2 standard deviations, 9 % of a weight's, in three matrices (sqrt(3) of it)
    assert 0.01 < off < 0.35


def test_routed_layer_on_4bit_weights_with_adapters():
    """align -> 4-bit gate_up product -> shrink -> expand + SwiGLU -> 4-bit down product ->
    shrink -> expand + combine, against the same chain on the dequantised weights in fp64."""
    m = gu.need_gpu()
    T, E, k, H, I, L, r, G = 24, 6, 2, 128, 192, 3, 8, 32
    g = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    x = normal(T, H).to(bf)
    W1, W2 = (normal(E, 2 * I, H) / math.sqrt(H)).to(bf), (normal(E, H, I) / math.sqrt(I)).to(bf)
    A1, B1 = (normal(L, E, r, H) / math.sqrt(H)).to(bf), (normal(L, E, 2 * I, r) / math.sqrt(r)).to(bf)
    A2, B2 = (normal(L, E, r, I) / math.sqrt(I)).to(bf), (normal(L, E, H, r) / math.sqrt(r)).to(bf)
    ad = torch.randint(-1, L, (T,), generator=g, device="cuda", dtype=torch.int32)
    ids, w = m.moe_topk_softmax(normal(T, E), k)
    al = m.moe_lora_align(ids, ad, E, L, 16, 16)
    c1, c2 = m.moe_w4_quantize(W1, group=G), m.moe_w4_quantize(W2, group=G)
    w1, w2 = m.moe_w4_pack(*c1, group=G), m.moe_w4_pack(*c2, group=G)
    base = m.moe_w4_matvec(x, w1, al=al, out_fp32=True)
    h = m.lora_expand_add(m.lora_shrink(x, False, A1, al), B1, al, 1, base)
    base2 = m.moe_w4_matvec(h, w2, al=al, rows_sorted=True, out_fp32=True)
    # the second shrink reads h in sorted order
    y = m.lora_expand_add(m.lora_shrink(h, True, A2, al), B2, al, 2, base2, out_fp32=True, topk_w=w)

    def dense(codes, scales, K):
        col = torch.arange(K, device="cuda")
        q = (codes[..., col // 2] >> (4 * (col % 2)).to(torch.uint8)) & 15
        return (q.double() - 8) * scales[..., col // G].double()

    d1, d2 = dense(*c1, H), dense(*c2, I)
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for t in range(T):
        a = int(ad[t])
        for j in range(k):
            e = int(ids[t, j])
            z = d1[e] @ x[t].double()
            if a >= 0:
                z = z + B1[a, e].double() @ (A1[a, e].double() @ x[t].double())
            s = (z[:I] * torch.sigmoid(z[:I]) * z[I:]).to(bf).double()
            o = d2[e] @ s
            if a >= 0:
                o = o + B2[a, e].double() @ (A2[a, e].double() @ s)
            ref[t] += float(w[t, j]) * o
    # h may round to the neighbouring bf16 value; the rest is fp32 (the layer's own bound)
    gu.assert_close(y, gu.f64(ref), gu.LAYER_RTOL, "y")
