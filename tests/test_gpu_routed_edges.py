"""The operators around the experts' products where calls can go wrong: adapters and rows that are
not finite, adapters without rows, orders that changed, streams, graphs, early launches, limits of
the waits; and a run of them together as a layer's training step."""
import ctypes
import math

import pytest
import torch

import gpu_util as gu
from test_gpu_routed import ADD, check, linear_inputs, linear_reference, normal, rounding, routing, row_owners, run_linear

pytestmark = pytest.mark.gpu

ERR_TIMEOUT, DEVERR_TIMEOUT = 5, 0x4


def dense(m, of, L, **kw):
    ids = torch.zeros((len(of), 1), dtype=torch.int32, device="cuda")
    return m.moe_lora_align(ids, of, 1, L, 256, 16, **kw)


@pytest.mark.parametrize("T,r,K,N", [(150, 72, 200, 136), (140, 104, 264, 264), (200, 56, 72, 200), (70, 112, 136, 72),
                                     (513, 48, 1024, 64), (1200, 8, 64, 1048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_other_ranks(T, r, K, N, dtype):
    m = gu.need_gpu()
    _, _, of = routing(T, T, 1, 1, 6)
    run_linear(m, dense(m, of, 6), False, 1, 6, r, K, N, dtype, T)


@pytest.mark.parametrize("T,L", [(40, 3), (300, 3), (3000, 2)])
def test_no_token_has_an_adapter(T, L):
    m = gu.need_gpu()
    of = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    *_, grads = run_linear(m, dense(m, of, L), False, 1, L, 16, 128, 136, torch.bfloat16, T)
    assert not bool(grads["dA"].any()) and not bool(grads["dB"].any())


@pytest.mark.parametrize("T,mixed", [(9, True), (100, True), (290, True), (700, False), (5000, False)])
def test_one_adapter_many_rows_and_many_adapters_few(T, mixed):
    """A sum shared by a cluster (one adapter), and as many adapters as rows."""
    m = gu.need_gpu()
    one = torch.zeros(T, dtype=torch.int32, device="cuda")
    run_linear(m, dense(m, one, 1), False, 1, 1, 24, 136, 200, torch.float16, T)
    if T <= 300:
        each = torch.randperm(T, generator=torch.Generator().manual_seed(T)).to(torch.int32).cuda()
        run_linear(m, dense(m, each, T), False, 1, T, 8, 136, 72, torch.bfloat16, T)


@pytest.mark.parametrize("T", [20, 100, 500])
@pytest.mark.parametrize("rows_sorted", [False, True], ids=["tokens", "sorted"])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_what_is_not_finite_stays_with_its_own(T, rows_sorted, value):
    """An adapter's weights touch its own rows only, a row its own outputs and its own adapter's
    gradients only, in the bits."""
    m = gu.need_gpu()
    L, r, K, N = 5, 16, 136, 264
    _, _, of = routing(T, T, 1, 1, L)
    al = dense(m, of, L)
    x, W, A, B, dy = linear_inputs(T, T, 1, L, r, K, N, torch.bfloat16)
    _, owner = row_owners(al, rows_sorted)
    y = m.moe_lora_linear(x, W, A, B, al, rows_sorted=rows_sorted)
    dx, dA, dB = m.moe_lora_linear_backward(dy, x, W, A, B, al, rows_sorted=rows_sorted)
    A2, B2 = A.clone(), B.clone()
    A2[2], B2[3] = value, value
    y2 = m.moe_lora_linear(x, W, A2, B2, al, rows_sorted=rows_sorted)
    dx2, dA2, dB2 = m.moe_lora_linear_backward(dy, x, W, A2, B2, al, rows_sorted=rows_sorted)
    clean = (owner != 2) & (owner != 3)
    assert torch.equal(y2[clean], y[clean]) and torch.equal(dx2[clean], dx[clean])
    assert bool((~torch.isfinite(y2[~clean])).all()) and bool((~torch.isfinite(dx2[~clean])).all())
    for l in (0, 1, 4):
        assert torch.equal(dA2[l], dA[l]) and torch.equal(dB2[l], dB[l])
    # rows: all of adapter 1's, and one of the base model's
    x3, dy3 = x.clone(), dy.clone()
    bad = owner == 1
    bad[(owner == -1).nonzero()[0]] = True
    x3[bad], dy3[bad] = value, value
    y3 = m.moe_lora_linear(x3, W, A, B, al, rows_sorted=rows_sorted)
    dx3, dA3, dB3 = m.moe_lora_linear_backward(dy3, x3, W, A, B, al, rows_sorted=rows_sorted)
    assert torch.equal(y3[~bad], y[~bad]) and torch.equal(dx3[~bad], dx[~bad])
    for l in (0, 2, 3, 4):
        assert torch.equal(dA3[l], dA[l]) and torch.equal(dB3[l], dB[l])
    assert not bool(torch.isfinite(dA3[1]).any()) and not bool(torch.isfinite(dB3[1]).any())


@pytest.mark.parametrize("T", [30, 400])
def test_small_gradients_in_fp16_keep_their_bits(T):
    """v far below fp16's steps: dA takes it in steps of 2^-36 (dx in 2^-25)."""
    m = gu.need_gpu()
    L, r, K, N = 2, 16, 128, 64
    _, _, of = routing(T, T, 1, 1, L)
    al = dense(m, of, L)
    x, W, A, B, dy = linear_inputs(T, T, 1, L, r, K, N, torch.float16)
    x, dy, B = x * 1000, dy * 1e-3, B * 1e-2
    expert, owner = row_owners(al, False)
    ref = linear_reference(x, W, A, B, expert, owner, dy)
    got = dict(zip(("dx", "dA", "dB"), m.moe_lora_linear_backward(dy, x, W, A, B, al)))
    for name, (value, bound) in ref.items():
        check(got[name], value, bound, name)


@pytest.mark.parametrize("T,E,k", [(50, 1, 1), (200, 1, 1), (300, 4, 2)])
def test_only_what_is_wanted(T, E, k):
    m = gu.need_gpu()
    L, r, K, N = 3, 16, 72, 136
    ids, _, of = routing(T, T, k, E, L)
    al = m.moe_lora_align(ids, of, E, L, 256, 16)
    x, W, A, B, dy = linear_inputs(T, T * k, E, L, r, K, N, torch.bfloat16)
    kw = dict(rows_sorted=E > 1)
    want = m.moe_lora_linear_backward(dy, x, W, A, B, al, **kw)
    for mask in range(8):
        need = dict(need_dx=bool(mask & 1), need_dA=bool(mask & 2), need_dB=bool(mask & 4))
        got = m.moe_lora_linear_backward(dy, x, W, A, B, al, **kw, **need)
        for g, w, n in zip(got, want, need.values()):
            assert torch.equal(g, w) if n else g is None
    # a caller's workspace, dirty and larger than asked for
    n = m.moe_lora_linear_workspace_size(al, N, K, r, rows_sorted=E > 1, backward=True)
    ws = torch.full((n + 1000,), 255, dtype=torch.uint8, device="cuda")
    got = m.moe_lora_linear_backward(dy, x, W, A, B, al, workspace=ws, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(m.MoeLoraError):
        m.moe_lora_linear_backward(dy, x, W, A, B, al, workspace=ws[:n - 256], **kw)
    with pytest.raises(m.MoeLoraError):  # rows off a 16-byte boundary
        flat = torch.zeros(x.numel() + 1, dtype=x.dtype, device="cuda")
        m.moe_lora_linear(flat[1:].view(x.shape), W, A, B, al, **kw)


def test_empty_batches():
    m = gu.need_gpu()
    al = m.new_align(0, 2, 4, 3, 256, 16)
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    assert m.moe_permute(x, al).shape == (0, 64) and m.moe_unpermute(x, al).shape == (0, 64)
    do, dw = m.moe_unpermute_backward(x, x, al, torch.zeros((0, 2), device="cuda"))
    assert do.shape == (0, 64) and dw.shape == (0, 2)
    assert m.moe_topk_softmax_backward(dw, dw.int(), dw, 4).shape == (0, 4)
    W, A, B = (normal(i, s, torch.bfloat16) for i, s in enumerate(((4, 32, 64), (3, 4, 8, 64), (3, 4, 32, 8))))
    assert m.moe_lora_linear(x, W, A, B, al, rows_sorted=True).shape == (0, 32)
    dx, dA, dB = m.moe_lora_linear_backward(x[:, :32].contiguous(), x, W, A, B, al, rows_sorted=True)
    assert dx.shape == (0, 64) and not bool(dA.any()) and not bool(dB.any())


@pytest.mark.parametrize("offset", [0, 1, 2, 4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_rows_at_any_alignment(offset, dtype):
    """Rows that start off a 16-byte boundary, of a width that is a multiple of 16 bytes."""
    m = gu.need_gpu()
    T, k, E, H = 37, 3, 8, 64
    ids, w, _ = routing(1, T, k, E)
    al = m.moe_lora_align(ids, None, E, 0, 256, 16)

    def at(t):
        flat = torch.empty(t.numel() + offset, dtype=dtype, device="cuda")
        flat[offset:] = t.reshape(-1)
        return flat[offset:].view(t.shape)

    x, o, dy = normal(1, (T, H), dtype), normal(2, (T * k, H), dtype), normal(3, (T, H), dtype)
    assert torch.equal(m.moe_permute(at(x), al), m.moe_permute(x, al))
    assert torch.equal(m.moe_unpermute(at(o), al, w), m.moe_unpermute(o, al, w))
    a, b = m.moe_unpermute_backward(at(dy), at(o), al, w), m.moe_unpermute_backward(dy, o, al, w)
    assert torch.equal(a[0], b[0])
    mag = o.double().abs().sum(1).max() * dy.double().abs().max()
    assert float((a[1] - b[1]).abs().max()) <= 2 * H * ADD * float(mag)  # another order of the sum


def test_an_order_that_changed_is_refused():
    """A backward pass whose align buffer was aligned anew after the forward pass."""
    m = gu.need_gpu()
    T, k, E, L = 24, 2, 4, 2
    ids, w, of = routing(1, T, k, E, L)
    al = m.moe_lora_align(ids, of, E, L, 256, 16)
    x, W, A, B, _ = linear_inputs(1, T, E, L, 8, 64, 64, torch.bfloat16)

    def outputs():
        xs = m.moe_permute(x.requires_grad_(True), al)
        y = m.moe_lora_linear(xs, W, A, B, al, rows_sorted=True)
        return xs, m.moe_lora_linear(xs.detach().requires_grad_(True), W, A, B, al, rows_sorted=True), \
            m.moe_unpermute(y.detach().requires_grad_(True), al, w)

    for out in outputs():
        out.sum().backward()  # as it was: fine
    for out in outputs():
        m.moe_lora_align(ids, of, E, L, al=al)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()


def test_differentiable_calls_and_their_refusals():
    m = gu.need_gpu()
    T, L, r, K, N = 70, 3, 16, 64, 96
    _, _, of = routing(2, T, 1, 1, L)
    al = dense(m, of, L)
    x, W, A, B, dy = linear_inputs(3, T, 1, L, r, K, N, torch.bfloat16)
    W, A, B = W[0], A[:, 0].contiguous(), B[:, 0].contiguous()  # one projection: without the experts' dimension
    leaves = [t.clone().requires_grad_(True) for t in (x, A, B)]
    y = m.moe_lora_linear(leaves[0], W, leaves[1], leaves[2], al)
    assert torch.equal(y, m.moe_lora_linear(x, W, A, B, al))
    wide = torch.zeros((T, 2 * N), dtype=y.dtype, device="cuda")
    wide[:, N:] = dy
    y.backward(wide[:, N:])  # a strided gradient
    want = m.moe_lora_linear_backward(dy, x, W, A, B, al)
    assert all(torch.equal(t.grad, g) and t.grad.shape == t.shape for t, g in zip(leaves, want))
    # only one of them
    b = B.clone().requires_grad_(True)
    m.moe_lora_linear(x, W, A, b, al).backward(dy)
    assert torch.equal(b.grad, want[2])
    with pytest.raises(ValueError, match="frozen"):
        m.moe_lora_linear(x, W.clone().requires_grad_(True), A, B, al)
    with torch.no_grad():
        m.moe_lora_linear(x, W.clone().requires_grad_(True), A, B, al)
    with pytest.raises(ValueError, match="workspace"):
        m.moe_lora_linear(leaves[0], W, A, B, al, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        for call in (lambda: m.moe_lora_linear(dual, W, A, B, al), lambda: m.moe_permute(dual, al),
                     lambda: m.moe_unpermute(dual, al), lambda: m.moe_unpermute_backward(dual, None, al, need_dw=False)):
            with pytest.raises(NotImplementedError):
                call()


def test_gradients_against_differences():
    """The gradients of a scalar of the outputs along a direction, against fp64 differences of the
    definition at the same values."""
    m = gu.need_gpu()
    T, k, E, L, r, K, N = 40, 2, 3, 2, 8, 64, 72
    ids, w, of = routing(5, T, k, E, L)
    al = m.moe_lora_align(ids, of, E, L, 256, 16)
    slots = al.sorted_slots().long()
    e, l = al.row_expert().long(), al.row_adapter().long()
    x, W, A, B, _ = linear_inputs(6, T, E, L, r, K, N, torch.float16)
    c = normal(7, (T, N), torch.float64, 0.1)

    def f(x, A, B, w, W=W.double(), c=c):
        xs = x[slots // k]
        rows = []
        for i in range(T * k):
            y = W[e[i]] @ xs[i]
            if l[i] >= 0:
                y = y + B[l[i], e[i]] @ (A[l[i], e[i]] @ xs[i])
            rows.append(w.reshape(-1)[slots[i]] * y)
        return (torch.zeros((T, N), dtype=torch.float64, device="cuda").index_add(0, slots // k, torch.stack(rows)) * c).sum()

    leaves = [t.clone().requires_grad_(True) for t in (x, A, B, w)]
    xs = m.moe_permute(leaves[0], al)
    y = m.moe_unpermute(m.moe_lora_linear(xs, W, leaves[1], leaves[2], al, rows_sorted=True), al, leaves[3])
    (y.double() * c).sum().backward()
    wide = [t.double() for t in (x, A, B, w)]
    # the same with every magnitude: along v it bounds what roundings on the way move. Four at most
    # meet a gradient (c and the rows' gradient to fp16, y's rounding for dw, its own), each 2^-11
    mags = [t.abs().requires_grad_(True) for t in wide]
    f(*mags, W=W.double().abs(), c=c.abs()).backward()
    for i, leaf in enumerate(leaves):
        v = normal(20 + i, leaf.shape, torch.float64)
        h = 1e-4
        there, back = list(wide), list(wide)
        there[i], back[i] = wide[i] + h * v, wide[i] - h * v
        slope = float((f(*there) - f(*back)) / (2 * h))  # f is linear in each argument: exact but for rounding
        got = float((leaf.grad.double() * v).sum())
        bound = float((mags[i].grad * v.abs()).sum())
        assert abs(got - slope) <= (4 * 2.0 ** -11 + 1e-9) * bound


def layer_reference(x, logits, W1, A1, B1, W2, A2, B2, ids, of):
    """A layer of experts with adapters in fp64, differentiable."""
    T, k = ids.shape
    w = torch.softmax(torch.gather(logits, 1, ids.long()), 1)
    out = torch.zeros_like(x)
    for e in range(W1.shape[0]):
        for l in range(-1, A1.shape[0]):
            t, j = ((ids == e) & (of[:, None] == l)).nonzero(as_tuple=True)
            if not len(t):
                continue
            h = x[t]
            u = h @ W1[e].t() + ((h @ A1[l, e].t()) @ B1[l, e].t() if l >= 0 else 0)
            I = u.shape[1] // 2
            a = torch.nn.functional.silu(u[:, :I]) * u[:, I:]
            y = a @ W2[e].t() + ((a @ A2[l, e].t()) @ B2[l, e].t() if l >= 0 else 0)
            out = out.index_add(0, t, w[t, j][:, None] * y)
    return out


@pytest.mark.parametrize("T", [24, 400])
def test_a_layer_trains_through_them(T):
    """Router, rows by expert, adapted gate and up, activation, adapted down, rows back: values and all
    gradients, against fp64. Each of some eight values on the way rounds to bf16 by 2^-9 at most: the
    relative error of a whole tensor stays below 8 2^-9 (weights of the routing in fp32)."""
    m = gu.need_gpu()
    E, k, L, r, H, I = 4, 2, 3, 16, 128, 192
    dt = torch.bfloat16
    x, logits, dy = normal(1, (T, H), dt), normal(2, (T, E), torch.float32), normal(3, (T, H), dt)
    W1, A1, B1 = normal(4, (E, 2 * I, H), dt, H ** -0.5), normal(5, (L, E, r, H), dt, H ** -0.5), \
        normal(6, (L, E, 2 * I, r), dt, 0.5 * r ** -0.5)
    W2, A2, B2 = normal(7, (E, H, I), dt, I ** -0.5), normal(8, (L, E, r, I), dt, I ** -0.5), \
        normal(9, (L, E, H, r), dt, 0.5 * r ** -0.5)
    of = torch.randint(-1, L, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int32).cuda()
    leaves = [t.clone().requires_grad_(True) for t in (x, logits, A1, B1, A2, B2)]

    def step(x, logits, A1, B1, A2, B2):
        ids, w = m.moe_topk_softmax(logits, k)
        al = m.moe_lora_align(ids, of, E, L, 256, 16)
        u = m.moe_lora_linear(m.moe_permute(x, al), W1, A1, B1, al, rows_sorted=True)
        a = torch.nn.functional.silu(u[:, :I]) * u[:, I:]
        return ids, m.moe_unpermute(m.moe_lora_linear(a, W2, A2, B2, al, rows_sorted=True), al, w)

    ids, y = step(*leaves)
    y.backward(dy)
    wide = [t.double().requires_grad_(True) for t in (x, logits, A1, B1, A2, B2)]
    ref = layer_reference(wide[0], wide[1], W1.double(), wide[2], wide[3], W2.double(), wide[4], wide[5], ids, of)
    ref.backward(dy.double())
    for got, want in [(y, ref)] + [(a.grad, b.grad) for a, b in zip(leaves, wide)]:
        err = float((got.detach().double() - want.detach()).norm() / want.detach().norm())
        assert err <= 8 * 2 ** -9, err
    # the same bits again
    again = [t.clone().requires_grad_(True) for t in (x, logits, A1, B1, A2, B2)]
    ids2, y2 = step(*again)
    y2.backward(dy)
    assert torch.equal(y2, y) and all(torch.equal(a.grad, b.grad) for a, b in zip(again, leaves))


@pytest.mark.parametrize("T,E,k", [(9, 1, 1), (300, 1, 1), (200, 4, 2)])
def test_graphs_and_streams(T, E, k):
    """Two graphs captured with other inputs and replayed at once on two streams, and calls on a side
    stream: the results of eager calls, in the bits."""
    m = gu.need_gpu()
    L, r, K, N = 4, 16, 128, 264
    ids, w, of = routing(T, T, k, E, L)
    kw = dict(rows_sorted=E > 1)
    sets = [linear_inputs(s, T * k, E, L, r, K, N, torch.bfloat16) for s in (1, 50)]
    buffers = [m.new_align(T, k, E, L, 256, 16) for _ in sets]

    def run(al, x, W, A, B, dy):
        m.moe_lora_align(ids, of, E, L, al=al)
        y = m.moe_lora_linear(x, W, A, B, al, **kw)
        back = m.moe_lora_linear_backward(dy, x, W, A, B, al, **kw)
        t = m.moe_unpermute(y, al, w)
        return (y, *back, t, m.moe_permute(t, al), *m.moe_unpermute_backward(t, y, al, w))

    want = [run(al, *s) for al, s in zip(buffers, sets)]
    side = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for al, s, st, ref in zip(buffers, sets, side, want):
        with torch.cuda.stream(st):
            got = run(al, *s)
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    graphs, outs = [], []
    for al, s in zip(buffers, sets):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(al, *s))
        graphs.append(g)
    for out in outs:
        for t in out:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, side):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for out, ref in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert m.ffn_get_error() == 0


@pytest.mark.parametrize("between", [False, True], ids=["directly", "behind_a_routing"])
@pytest.mark.parametrize("T", [1, 100, 300])
def test_operands_written_by_earlier_launches(T, between):
    """Each operand is the output of a long kernel that triggers its dependents at its start, directly
    before the call or with a launch in between that triggers before its own wait."""
    m = gu.need_gpu()
    L, r, K, N = 4, 32, 1024, 4096
    _, _, of = routing(T, T, 1, 1, L)
    al = dense(m, of, L)
    x, W, A, B, dy = linear_inputs(1, T, 1, L, r, K, N, torch.bfloat16)
    logits = torch.randn((1, 8), device="cuda")
    m.moe_topk_softmax(logits, 2)
    ballast = normal(9, (1 << 24,), torch.bfloat16)  # keeps the writer at work for a while
    operands = dict(x=x, W=W, A=A, B=B, dy=dy)
    source = [ballast] + [t * 2 for t in operands.values()]
    norm = float(m.moe_grad_clip(source, norm_only=True))
    outs = [torch.empty_like(ballast)] + [torch.zeros_like(t) for t in operands.values()]
    plan = m.GradClip(source, out=outs)
    plan(norm / 2)
    torch.cuda.synchronize()
    x, W, A, B, dy = outs[1:]
    calls = (lambda: (m.moe_lora_linear(x, W, A, B, al),), lambda: m.moe_lora_linear_backward(dy, x, W, A, B, al),
             lambda: (m.moe_permute(x, al),), lambda: (m.moe_unpermute(x, al),),
             lambda: m.moe_unpermute_backward(x, x, al))
    for call in calls:
        want = call()
        for _ in range(3):
            for t in outs:
                t.zero_()
            torch.cuda.synchronize()
            plan(norm / 2)
            if between:
                m.moe_topk_softmax(logits, 2)
            got = call()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,E,N,K", [(3, 1, 2048, 2048), (100, 1, 1024, 1024), (300, 1, 8192, 8192), (2057, 3, 5120, 5120)],
                         ids=["few", "few_128", "pairs", "several_tiles"])
def test_bounded_waits_give_up_and_recover(T, E, N, K):
    """With the waits' limit below zero each gives up at its first unsuccessful poll: the word is set,
    and later calls give the usual results. (A pair's poll itself waits for a while: a tile's products
    take longer.)"""
    m = gu.need_gpu()
    L, r = 3, 16
    ids, _, of = routing(T, T, 1, E, L)
    al = m.moe_lora_align(ids, of, E, L, 256, 16)
    x, W, A, B, dy = linear_inputs(1, T, E, L, r, K, N, torch.bfloat16)
    calls = (lambda: (m.moe_lora_linear(x, W, A, B, al),),
             lambda: m.moe_lora_linear_backward(dy, x, W, A, B, al, need_dA=False, need_dB=False)[:1])
    m.ffn_clear_error()
    for call in calls:
        want = call()
        torch.cuda.synchronize()
        m.ffn_set_wait_limit(-1)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            m.ffn_set_wait_limit(0)
        word = ctypes.c_uint32(0)
        st = m.lib().moe_ffn_get_error(torch.cuda.current_stream().cuda_stream, ctypes.byref(word))
        assert st == ERR_TIMEOUT and word.value == DEVERR_TIMEOUT
        m.ffn_clear_error()
        assert m.ffn_get_error() == 0
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(call(), want))
        assert m.ffn_get_error() == 0
