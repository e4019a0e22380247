"""The operators around the experts' products at values, states and sizes that the other tests leave
out: infinite sums, the bits that the low parts keep, tangents, outputs over saved tensors, changed
descriptions, the smallest widths, enough tiles that every CTA pair takes several, and offsets past 32 bits."""
import math

import pytest
import torch
from torch.autograd import forward_ad

import gpu_util as gu
from test_gpu_routed import ADD, check, linear_inputs, linear_reference, normal, rounding, routing, run_linear

pytestmark = pytest.mark.gpu


def dense(m, of, L):
    return m.moe_lora_align(torch.zeros((len(of), 1), dtype=torch.int32, device="cuda"), of, 1, L, 256, 16)


def test_router_refuses_forward_mode_derivatives():
    """A tangent is refused, not dropped."""
    m = gu.need_gpu()
    logits, dw = normal(1, (5, 8), torch.float32), normal(2, (5, 2), torch.float32)
    ids, w = m.moe_topk_softmax(logits, 2)
    with forward_ad.dual_level():
        dual, dual_dw, dual_w = (forward_ad.make_dual(t, torch.ones_like(t)) for t in (logits, dw, w))
        for call in (lambda: m.moe_topk_softmax(dual, 2),
                     lambda: m.moe_topk_softmax(forward_ad.make_dual(logits.clone().requires_grad_(), logits), 2),
                     lambda: m.moe_topk_softmax_backward(dual_dw, ids, w, 8),
                     lambda: m.moe_topk_softmax_backward(dw, ids, dual_w, 8)):
            with pytest.raises(NotImplementedError, match="forward"):
                call()
        ids2, w2 = m.moe_topk_softmax(logits, 2)  # no tangent: as ever
        assert torch.equal(ids2, ids) and torch.equal(w2, w)
        m.moe_topk_softmax_backward(dw, ids, w, 8)


@pytest.mark.parametrize("T", [30, 400], ids=["few", "pairs"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_an_infinite_z_is_infinite(T, dtype):
    """z = x A^T (or v = dy B) of one adapter's first rank is infinite -- in fp16 past 65504, where it is
    as infinite as an fp16 z would be -- and every other factor has a sign and is finite: the sums that
    take it are infinite, not NaN, and nothing else changes."""
    m = gu.need_gpu()
    L, r, K, N = 3, 24, 72, 136
    _, _, of = routing(T, T, 1, 1, L)
    al = dense(m, of, L)
    x, W, A, B, dy = (t.abs() + 0.125 for t in linear_inputs(T, T, 1, L, r, K, N, dtype))
    mine = of == 1
    sign = torch.where(torch.arange(T, device="cuda") % 2 == 0, 1.0, -1.0)
    x = x * sign[:, None].to(dtype)
    y = m.moe_lora_linear(x, W, A, B, al)
    dx, dA, dB = m.moe_lora_linear_backward(dy, x, W, A, B, al)
    # infinite in bf16; some 72 (or 136) x 0.125 x 60000 and more in fp16
    big = A.clone()
    if dtype == torch.bfloat16:
        big[1, 0, 0, 0] = math.inf
    else:
        big[1, 0, 0] = 60000
    got = m.moe_lora_linear(x, W, big, B, al)
    assert torch.equal(got[~mine], y[~mine])
    assert torch.equal(got[mine].float(), (sign[mine, None] * math.inf).expand(-1, N))
    x = x.abs()
    _, dA, dB = m.moe_lora_linear_backward(dy, x, W, A, B, al)
    _, dA2, dB2 = m.moe_lora_linear_backward(dy, x, W, big, B, al)
    want = dB.clone()
    want[1, 0, :, 0] = math.inf
    assert torch.equal(dB2, want) and torch.equal(dA2, dA)
    big = B.clone()
    if dtype == torch.bfloat16:
        big[1, 0, 0, 0] = math.inf
    else:
        big[1, 0, :, 0] = 60000
    dx, dA, dB = m.moe_lora_linear_backward(dy, x, W, A, B, al)
    dx2, dA2, dB2 = m.moe_lora_linear_backward(dy, x, W, A, big, al)
    assert torch.equal(dx2[~mine], dx[~mine]) and bool((dx2[mine] == math.inf).all())
    want = dA.clone()
    want[1, 0, 0] = math.inf
    assert torch.equal(dA2, want) and torch.equal(dB2, dB)
    # NaN stays NaN
    big = A.clone()
    big[1, 0, 0, 0] = math.nan
    got = m.moe_lora_linear(x, W, big, B, al)
    assert bool(torch.isnan(got[mine]).all()) and not bool(torch.isnan(got[~mine]).any())


@pytest.mark.parametrize("T", [30, 400], ids=["few", "pairs"])
def test_z_is_rounded_twice(T):
    """z enters as two bf16 values, its rounding and the remainder's: off by 2^-17 of it (each half a step:
    the remainder is 2^-8 of z's power of two at most, and lies below a step's power of two). z = a + b
    2^-10 with 8-bit a, b is exact in fp32, and the base adds -z to 17 bits to it: y is the error itself."""
    m = gu.need_gpu()
    L, r, K, N = 2, 128, 64, 128
    g = torch.Generator(device="cuda").manual_seed(T)
    of = torch.randint(0, L, (T,), generator=g, device="cuda", dtype=torch.int32)
    al = dense(m, of, L)
    for seed in range(4):
        g.manual_seed(seed)
        a, b = (1 + torch.randint(0, 128, (r,), generator=g, device="cuda").double() / 128 for _ in range(2))
        a = a * torch.where(torch.rand((r,), generator=g, device="cuda") < 0.5, -1.0, 1.0)
        z = a + b * 2.0 ** -10
        hi = z.bfloat16()
        lo = (z - hi.double()).bfloat16()
        x, W, A, B = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((T, K), (N, K), (L, r, K), (L, N, r)))
        x[:, 0], x[:, 1], x[:, 2:4] = 1, 2.0 ** -10, -1
        A[:, :, 0], A[:, :, 1] = a.bfloat16(), b.bfloat16()
        W[:, 2], W[:, 3] = hi, lo
        B[:] = torch.eye(N, dtype=torch.bfloat16, device="cuda")
        y = m.moe_lora_linear(x, W, A, B, al)
        want = (z - hi.double() - lo.double()).expand(T, N)
        # six values other than zero in a sum
        check(y, want, ((2.0 ** -17 + 6 * ADD) * z.abs()).expand(T, N), "y")


def test_an_out_over_a_saved_tensor_is_seen():
    """A given `out` that a differentiable call saved: its backward pass is refused, as after any change
    in place."""
    m = gu.need_gpu()
    T, L, r, H = 20, 2, 8, 64
    _, _, of = routing(1, T, 1, 1, L)
    al = dense(m, of, L)
    x, W, A, B, _ = linear_inputs(1, T, 1, L, r, H, H, torch.bfloat16)
    w = torch.ones((T, 1), device="cuda")
    for write in (lambda out: m.moe_permute(x, al, out=out), lambda out: m.moe_unpermute(x, al, w, out=out),
                  lambda out: m.moe_lora_linear(x, W, A, B, al, out=out)):
        saved = x.clone()
        y = m.moe_unpermute(saved, al, w.clone().requires_grad_(True))
        write(torch.empty_like(saved))
        y.sum().backward(retain_graph=True)  # another tensor: fine
        write(saved)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
    with torch.inference_mode():  # has no versions
        m.moe_permute(x, al, out=torch.empty_like(x))


def test_one_description_for_batch_after_batch():
    """A program that gives its Align the next batch's sizes and buffer before it goes back through this
    one gets this one's gradients."""
    m = gu.need_gpu()
    T, k, E, L, r, K, N = 40, 2, 4, 3, 16, 64, 72
    ids, w, of = routing(1, T, k, E, L)
    al = m.moe_lora_align(ids, of, E, L, 256, 16)
    x, W, A, B, _ = linear_inputs(1, T, E, L, r, K, N, torch.bfloat16)
    dy = normal(9, (T, N), torch.bfloat16)

    def step(change):
        leaves = [t.clone().requires_grad_(True) for t in (x, A, B, w)]
        xs = m.moe_permute(leaves[0], al)
        y = m.moe_unpermute(m.moe_lora_linear(xs, W, leaves[1], leaves[2], al, rows_sorted=True), al, leaves[3])
        if change:
            other = m.moe_lora_align(*(t.cuda() for t in (ids[:8], of[:8])), E, L, 256, 16)
            al.T, al.buf = other.T, other.buf
        y.backward(dy)
        return [y] + [t.grad for t in leaves]

    want = step(False)
    assert all(torch.equal(a, b) for a, b in zip(step(True), want))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 130])
@pytest.mark.parametrize("E", [1, 2])
def test_smallest_widths(T, E, dtype):
    """Eight columns, eight summed, eight ranks: less than a TMA box, a tile's half and a step."""
    m = gu.need_gpu()
    ids, _, of = routing(T, T, 1, E, 2)
    al = m.moe_lora_align(ids, of, E, 2, 256, 16)
    dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
    for r, K, N in ((8, 8, 8), (8, 8, 136), (24, 136, 8)):
        run_linear(m, al, False, E, 2, r, K, N, dt, T)
        run_linear(m, al, True, E, 2, r, K, N, dt, T)


def every_pair_has_several(m, al, N, K):
    """Whether y and dx have at least four tiles for each CTA pair that the card holds (tiles are 256
    columns at most)."""
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    return al.header()["n_tiles"] * min(-(-N // 256), -(-K // 256)) >= 4 * pairs


# Both stage counts (r up to 32, and more), one or two rank steps, adapters mixed (rows copied in sorted
# order) or one request after the other (rows in boxes where they are neighbours).
@pytest.mark.parametrize("r,dtype,mixed", [(16, "bf16", True), (104, "fp16", False), (72, "bf16", True)])
def test_several_tiles_to_a_pair_shared(r, dtype, mixed):
    """One projection with so many tiles that each CTA pair goes round its two accumulators more than
    once, and looks tiles and adapters up again and again."""
    m = gu.need_gpu()
    T, L, K, N = 5003, 9, 4096, 4104
    _, _, of = routing(r, T, 1, 1, L, mixed=mixed)
    al = dense(m, of, L)
    assert every_pair_has_several(m, al, N, K)
    run_linear(m, al, False, 1, L, r, K, N, {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype], r)


@pytest.mark.parametrize("T,k,rows_sorted,drop", [(2400, 4, True, False), (3000, 4, True, True), (9600, 1, False, False)],
                         ids=["sorted", "dropped", "tokens"])
@pytest.mark.parametrize("r,dtype", [(16, "fp16"), (72, "bf16")])
def test_several_tiles_to_a_pair_experts(T, k, rows_sorted, drop, r, dtype):
    m = gu.need_gpu()
    E, L, K, N = 32, 5, 1288, 1544
    ids, _, of = routing(T, T, k, E, L, drop=drop)
    al = m.moe_lora_align(ids, of, E, L, 256, 16)
    assert every_pair_has_several(m, al, N, K)
    run_linear(m, al, rows_sorted, E, L, r, K, N, {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype], r)


def test_offsets_past_32_bits():
    """Rows whose elements are numbered past 2^31, through every operator: the last ones against fp64, and
    others that are far apart."""
    m = gu.need_gpu()
    T, k, E, L, r, K, N = 140000, 2, 8, 4, 16, 8192, 64
    ids, w, of = routing(1, T, k, E, L)
    al = m.moe_lora_align(ids, of, E, L, 256, 16)
    S = T * k
    assert S * K > 2 ** 31 and al.header()["n_valid"] == S
    slots, expert, adapter = al.sorted_slots().long(), al.row_expert().long(), al.row_adapter().long()
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, K), generator=g, device="cuda", dtype=torch.bfloat16)
    _, W, A, B, _ = linear_inputs(2, 1, E, L, r, K, N, torch.bfloat16)
    dy = normal(7, (S, N), torch.bfloat16, 0.1)
    xs = m.moe_permute(x, al)
    at = torch.cat([torch.arange(0, S, S // 97, device="cuda"), torch.arange(S - 300, S, device="cuda")])
    assert torch.equal(xs[at], x[slots[at] // k])
    y = m.moe_lora_linear(xs, W, A, B, al, rows_sorted=True)
    value, bound = linear_reference(xs[at], W, A, B, expert[at], adapter[at])
    check(y[at], value, bound, "y")
    dx, dA, dB = m.moe_lora_linear_backward(dy, xs, W, A, B, al, rows_sorted=True)
    value, bound = linear_reference(xs[at], W, A, B, expert[at], adapter[at], dy[at])["dx"]
    check(dx[at], value, bound, "dx")
    # gradients of the last expert's adapters, whose rows are the far ones
    mine = (expert == E - 1).nonzero()[:, 0]
    ref = linear_reference(xs[mine], W[-1:], A[:, -1:], B[:, -1:], expert[mine] - (E - 1), adapter[mine], dy[mine])
    check(dA[:, -1:], *ref["dA"], "dA")
    check(dB[:, -1:], *ref["dB"], "dB")
    # rows back, over the 2^31 elements of xs, and their gradients
    t = torch.cat([torch.arange(0, T, T // 97, device="cuda"), torch.arange(T - 100, T, device="cuda")])
    rows = al.slot_row().long().view(T, k)
    parts = xs[rows[t]].double() * w[t].double()[:, :, None]
    back = m.moe_unpermute(xs, al, w)
    check(back[t], parts.sum(1), rounding(torch.bfloat16, parts.sum(1)) + (k + 1) * ADD * parts.abs().sum(1), "unpermute")
    do, dw = m.moe_unpermute_backward(x, xs, al, w)
    ref = x[t].double()[:, None] * w[t].double()[:, :, None]
    check(do[rows[t]], ref, rounding(torch.bfloat16, ref) + 2 * ADD * ref.abs(), "do")
    prod = xs[rows[t]].double() * x[t].double()[:, None]
    check(dw[t], prod.sum(2), K * ADD * prod.abs().sum(2), "dw")
