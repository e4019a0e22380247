"""The feed-forward operators read what earlier launches of the stream write, however early
those let the next launch start."""
import pytest
import torch

import gpu_util as gu

pytestmark = pytest.mark.gpu


def normal(seed, shape, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("between", [False, True], ids=["directly", "behind_a_routing"])
@pytest.mark.parametrize("T", [1, 4, 128, 200])
def test_gated_weights_written_by_earlier_launches(T, between):
    """W1 is the output of a long kernel that triggers its dependents at its start, directly
    before the product or with a launch in between that triggers before its own wait."""
    m = gu.need_gpu()
    H, I = 2048, 8192
    x, dh, new = normal(1, (T, H)), normal(2, (T, I), std=0.1), normal(3, (2 * I, H), std=0.04)
    logits = torch.randn((1, 8), device="cuda")
    m.moe_topk_softmax(logits, 2)
    # the writer: new doubled at first, and scaled back to half by the clip
    twice = new * 2
    norm = float(m.moe_grad_clip([twice], norm_only=True))
    W1 = torch.zeros_like(new)
    plan = m.GradClip([twice], out=[W1])
    plan(norm / 2)
    torch.cuda.synchronize()
    assert float((W1.float() - new.float()).abs().max()) <= 2.0 ** -7 * float(new.abs().max())
    want_h, want_dx = m.moe_gated_ffn(x, W1), m.moe_gated_ffn_backward(dh, x, W1, need_dW1=False)[0]
    for _ in range(3):
        for call, want in ((lambda: m.moe_gated_ffn(x, W1), want_h),
                           (lambda: m.moe_gated_ffn_backward(dh, x, W1, need_dW1=False)[0], want_dx)):
            W1.zero_()
            torch.cuda.synchronize()
            plan(norm / 2)
            if between:
                m.moe_topk_softmax(logits, 2)
            got = call()
            torch.cuda.synchronize()
            assert torch.equal(got, want)


@pytest.mark.parametrize("between", [False, True], ids=["directly", "behind_a_routing"])
@pytest.mark.parametrize("T,act", [(1, None), (6, "silu")])
def test_w4_weights_written_by_earlier_launches(T, act, between):
    """The packed weights arrive by a row gather, which triggers its dependents early."""
    m = gu.need_gpu()
    N, K, E = 16384, 4096, 1
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = normal(2, (E, N, K // 32), std=0.01)
    x, logits = normal(3, (T, K)), torch.randn((1, 8), device="cuda")
    w = m.moe_w4_pack(codes, scales, group=32, gated=act is not None)
    want = m.moe_w4_matvec(x, w, act=act)
    # one expert, a slot per row: the sorted order is the order itself
    cols = 512
    rows = w.packed.numel() // (2 * cols)
    assert rows * 2 * cols == w.packed.numel()
    src = w.packed.view(torch.bfloat16).view(rows, cols).clone()
    al = m.moe_lora_align(torch.zeros((rows, 1), dtype=torch.int32, device="cuda"), None, 1, 0, 16, 16)
    m.moe_topk_softmax(logits, 2)
    for _ in range(3):
        w.packed.zero_()
        torch.cuda.synchronize()
        m.moe_gather_rows(src, al, out=w.packed.view(torch.bfloat16).view(rows, cols))
        if between:
            m.moe_topk_softmax(logits, 2)
        got = m.moe_w4_matvec(x, w, act=act)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_clip_gradients_written_by_earlier_launches():
    """Odd slices, whose ends are read element by element, of rows that a gather (which triggers
    its dependents early) has just written, other values every time."""
    m = gu.need_gpu()
    rows, cols = 4096, 512
    src = [normal(i, (rows, cols), std=1.0 + i) for i in range(2)]
    al = m.moe_lora_align(torch.zeros((rows, 1), dtype=torch.int32, device="cuda"), None, 1, 0, 16, 16)
    buf = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    for views in ([buf.view(-1)[1 + 5 * i:4 + 5 * i] for i in range(40)],
                  [buf.view(-1)[1 + 5 * i:4 + 5 * i] for i in range(4000)], [buf.view(-1)[3:-1]]):
        outs = [torch.zeros_like(v) for v in views]
        plan = m.GradClip(views, out=outs)
        want = []
        for s in src:
            buf.copy_(s)
            torch.cuda.synchronize()
            want.append((float(plan(1.0)), torch.cat(outs)))
        for i in range(10):
            m.moe_gather_rows(src[i % 2], al, out=buf)
            norm = plan(1.0)
            got = torch.cat(outs)
            assert float(norm) == want[i % 2][0] and torch.equal(got, want[i % 2][1])
