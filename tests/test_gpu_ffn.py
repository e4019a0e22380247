"""The feed-forward operators against their definitions in fp64, element by element.

Bounds are worst cases of the arithmetic: an output rounds by half a step (eps / 2 of its
type), a sum of n fp32 products is off by at most n 2^-23 of the sum of magnitudes (adds that
may truncate), the activation by 2^-18 of its value, and dg and du round once to 16 bits.
"""
import math
import threading

import pytest
import torch

import gpu_util as gu

pytestmark = pytest.mark.gpu

ADD = 2.0 ** -23   # one fp32 addition, relative to the sum of magnitudes
ACT = 2.0 ** -18   # the activation and its derivative, relative
SUB16 = 2.0 ** -25  # half of fp16's subnormal step
DTYPES = [torch.bfloat16, torch.float16]
IDS = ["bf16", "fp16"]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(dtype, v):
    return half_step(dtype) * v.abs() + (SUB16 if dtype == torch.float16 else 0.0)


def act64(g, act):
    """a(g) and a'(g) in fp64."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    # (1 + tanh z) / 2 as the logistic function of 2z: 1 + tanh loses the left tail, even in fp64
    s = torch.sigmoid(2 * c * (g + 0.044715 * g ** 3))
    return g * s, s + 2 * g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def normal(seed, shape, dtype, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def check(got, ref, bound, what):
    got, ref = got.double(), ref
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bool(bad.any()):
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} out of bounds, first at {i}: "
                             f"{got[i].item()!r} for {ref[i].item()!r}, bound {bound[i].item():.3g}")


def gated_ref(x, W1, act):
    """g, u, a, a', and the bounds on g and u."""
    I = W1.shape[0] // 2
    xd, wd = x.double(), W1.double()
    y = xd @ wd.t()
    off = x.shape[1] * ADD * (xd.abs() @ wd.abs().t())
    a, d = act64(y[:, :I], act)
    return y[:, :I], y[:, I:], a, d, off[:, :I], off[:, I:]


def gated_bounds(x, W1, act):
    g, u, a, d, og, ou = gated_ref(x, W1, act)
    h = a * u
    slope = d.abs() + og  # |a''| is below 1
    return h, rounding(x.dtype, h) + (slope * og) * (u.abs() + ou) + a.abs() * ou + ACT * h.abs()


def backward_bounds(dh, x, W1, act):
    I = W1.shape[0] // 2
    g, u, a, d, og, ou = gated_ref(x, W1, act)
    e = dh.double()
    dg, du = e * u * d, e * a
    odg = e.abs() * (ou * (d.abs() + og) + u.abs() * og) + ACT * (dg.abs() + (e * u).abs())
    odu = e.abs() * (d.abs() + og) * og + ACT * du.abs()
    dy = torch.cat([dg, du], 1)
    ody = torch.cat([odg, odu], 1)
    ody = ody + rounding(x.dtype, dy.abs() + ody)
    wd, xd = W1.double(), x.double()
    mag = dy.abs() + ody
    dx, dw = dy @ wd, dy.t() @ xd
    odx = ody @ wd.abs() + 2 * I * ADD * (mag @ wd.abs())
    odw = ody.t() @ xd.abs() + x.shape[0] * ADD * (mag.t() @ xd.abs())
    return (dx, odx + rounding(x.dtype, dx.abs() + odx)), (dw, odw + rounding(x.dtype, dw.abs() + odw))


# (T, H, I): one token, tiles that end inside, one element past a tile, K of 8, long K
GATED = [(1, 8, 8), (1, 256, 512), (2, 2880, 264), (7, 72, 1000), (8, 4096, 136), (15, 248, 248),
         (16, 256, 512), (17, 264, 40), (33, 520, 776), (64, 256, 512), (127, 136, 8), (128, 64, 128),
         (129, 1032, 264), (255, 72, 264), (257, 256, 256), (300, 2048, 768), (513, 392, 1288),
         (1021, 64, 72)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,H,I", GATED)
def test_gated(T, H, I, dtype, act):
    m = gu.need_gpu()
    x = normal(1, (T, H), dtype)
    W1 = normal(2, (2 * I, H), dtype, 1.5 / math.sqrt(H))
    out = gu.Guarded((T, I), dtype)
    m.moe_gated_ffn(x, W1, act=act, out=out.t)
    out.check()
    h, bound = gated_bounds(x, W1, act)
    check(out.t, h, bound, "h")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,H,I", GATED)
def test_gated_backward(T, H, I, dtype, act):
    m = gu.need_gpu()
    x = normal(1, (T, H), dtype)
    W1 = normal(2, (2 * I, H), dtype, 1.5 / math.sqrt(H))
    dh = normal(3, (T, I), dtype, 0.25)
    dx, dW1 = m.moe_gated_ffn_backward(dh, x, W1, act=act)
    rx, rw = backward_bounds(dh, x, W1, act)
    check(dx, *rx, "dx")
    check(dW1, *rw, "dW1")
    # either one by itself is the same
    only, none = m.moe_gated_ffn_backward(dh, x, W1, act=act, need_dW1=False)
    assert none is None and torch.equal(only, dx)
    none, only = m.moe_gated_ffn_backward(dh, x, W1, act=act, need_dx=False)
    assert none is None and torch.equal(only, dW1)


def test_gated_backward_writes_nothing_else():
    m = gu.need_gpu()
    T, H, I, dt = 77, 136, 264, torch.bfloat16
    x, W1, dh = normal(1, (T, H), dt), normal(2, (2 * I, H), dt, 0.1), normal(3, (T, I), dt)
    dx, dW1 = gu.Guarded((T, H), dt), gu.Guarded((2 * I, H), dt)
    n = m.moe_gated_ffn_backward_workspace_size(T, H, I)
    raw = torch.full((n + 2048,), 0xA5, dtype=torch.uint8, device="cuda")
    at = 1024 + -(raw.data_ptr() + 1024) % 256
    lib = m.lib()
    st = lib.moe_gated_ffn_backward(dh.data_ptr(), x.data_ptr(), W1.data_ptr(), 0, 1, T, H, I,
                                    dx.t.data_ptr(), dW1.t.data_ptr(), raw.data_ptr() + at, n,
                                    torch.cuda.current_stream().cuda_stream)
    assert st == 0
    dx.check()
    dW1.check()
    assert bool((raw[:at] == 0xA5).all()) and bool((raw[at + n:] == 0xA5).all())
    want = m.moe_gated_ffn_backward(dh, x, W1)
    assert torch.equal(dx.t, want[0]) and torch.equal(dW1.t, want[1])


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_gradient_against_differences(act):
    """The loss sum(dh * h) along a direction, by central differences of the definition."""
    m = gu.need_gpu()
    T, H, I, dt = 19, 64, 48, torch.float16
    x, W1, dh = normal(1, (T, H), dt), normal(2, (2 * I, H), dt, 0.15), normal(3, (T, I), dt, 0.25)
    dx, dW1 = m.moe_gated_ffn_backward(dh, x, W1, act=act)
    (_, bx), (_, bw) = backward_bounds(dh, x, W1, act)
    (rx, _), (rw, _) = backward_bounds(dh, x, W1, act)

    def loss(step, vx, vw):
        y = (x.double() + step * vx) @ (W1.double() + step * vw).t()
        return (dh.double() * act64(y[:, :I], act)[0] * y[:, I:]).sum()

    e = 1e-4
    # a direction of no relation to the gradient, and the gradient's own: there the
    # derivative stands far above the roundings' bound
    for vx, vw in [(normal(4, (T, H), torch.float64), normal(5, (2 * I, H), torch.float64, 0.1)),
                   (rx / rx.norm(), rw / rw.norm())]:
        diff = (loss(e, vx, vw) - loss(-e, vx, vw)) / (2 * e)
        wide = (loss(2 * e, vx, vw) - loss(-2 * e, vx, vw)) / (4 * e)
        got = (dx.double() * vx).sum() + (dW1.double() * vw).sum()
        # the roundings' bound, and the differences' own: e^2 terms (from two steps), 1e-11 / e
        bound = (bx * vx.abs()).sum() + (bw * vw.abs()).sum() + (wide - diff).abs() + 1e-7 * diff.abs() + 1e-7
        assert abs(got - diff) <= bound
    assert float(diff.abs()) > 3 * float(bound)


def test_gated_autograd_shared_leaves_and_graph():
    m = gu.need_gpu()
    T, H, I, dt = 40, 64, 32, torch.bfloat16
    x = normal(1, (T, H), dt).requires_grad_()
    W1 = normal(2, (2 * I, H), dt, 0.2).requires_grad_()
    dh = normal(3, (T, I), dt)
    h = m.moe_gated_ffn(x, W1, "gelu")
    assert torch.equal(h, m.moe_gated_ffn(x.detach(), W1.detach(), "gelu"))
    h.backward(dh)
    dx, dW1 = m.moe_gated_ffn_backward(dh, x.detach(), W1.detach(), act="gelu")
    assert torch.equal(x.grad, dx) and torch.equal(W1.grad, dW1)
    # a non-contiguous gradient, and a frozen weight
    x.grad = None
    h = m.moe_gated_ffn(x, W1.detach(), "gelu")
    h.t().backward(dh.t())
    assert torch.equal(x.grad, dx)


def test_gated_autograd_unaligned_gradient():
    """Autograd hands over the slice of a larger gradient, wherever that starts."""
    m = gu.need_gpu()
    T, H, I, dt = 5, 64, 32, torch.bfloat16
    x = normal(1, (T, H), dt).requires_grad_()
    W1 = normal(2, (2 * I, H), dt, 0.2).requires_grad_()
    flat = normal(3, (T * I + 3,), dt)
    torch.cat([normal(4, (3,), dt), m.moe_gated_ffn(x, W1).flatten()]).backward(flat)
    dx, dW1 = m.moe_gated_ffn_backward(flat[3:].view(T, I).clone(), x.detach(), W1.detach())
    assert torch.equal(x.grad, dx) and torch.equal(W1.grad, dW1)


def test_gated_no_tokens():
    m = gu.need_gpu()
    x, W1 = normal(1, (0, 64), torch.bfloat16), normal(2, (32, 64), torch.bfloat16)
    assert m.moe_gated_ffn(x, W1).shape == (0, 16)
    dx, dW1 = m.moe_gated_ffn_backward(x.new_empty((0, 16)), x, W1)
    assert dx.shape == (0, 64) and bool((dW1 == 0).all()) and dW1.shape == W1.shape


def test_gated_nan_and_infinity_stay_in_their_rows():
    m = gu.need_gpu()
    x, W1 = normal(1, (300, 64), torch.bfloat16), normal(2, (96, 64), torch.bfloat16)
    clean = m.moe_gated_ffn(x, W1)
    x[5, 3], x[299, 7] = float("nan"), float("inf")
    h = m.moe_gated_ffn(x, W1)
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[5] = keep[299] = False
    assert torch.equal(h[keep], clean[keep])
    assert bool(h[5].isnan().all()) and not bool(h[299].isfinite().any())


def test_gated_large_arguments():
    """Gates far from zero: the activation saturates without overflowing."""
    m = gu.need_gpu()
    for act in ("silu", "gelu"):
        for T in (3, 40):
            x = torch.zeros((T, 16), dtype=torch.bfloat16, device="cuda")
            x[:, 0] = torch.linspace(-300, 300, T)
            x[:, 1] = 1
            W1 = torch.zeros((16, 16), dtype=torch.bfloat16, device="cuda")
            W1[:8, 0] = 1  # g = x0
            W1[8:, 1] = 1  # u = 1
            g = x[:, :1].double().expand(T, 8)
            a, d = act64(g, act)
            check(m.moe_gated_ffn(x, W1, act=act), a, rounding(x.dtype, a) + ACT * a.abs() + 1e-30, act)
            dx, _ = m.moe_gated_ffn_backward(torch.ones((T, 8), dtype=x.dtype, device="cuda"), x, W1, act=act)
            assert bool(dx.isfinite().all())
            want = 8 * d[:, 0]
            assert float((dx[:, 0].double() - want).abs().max()) <= 8 * (2 * half_step(x.dtype) * 1.2 + ACT)


# ---------------------------------------------------------------------------
# gradient clipping
# ---------------------------------------------------------------------------
def clip_ref(grads, bound):
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in grads))
    return norm, min(1.0, bound / (norm + 1e-6))


CLIP = [[1], [0, 5, 0], [8192], [8191, 8193], [3, 70000, 1, 16384, 0, 31], [250_001] * 3, [11] * 1500,
        list(range(0, 2100))]


@pytest.mark.parametrize("kinds", [["bf16"], ["fp16"], ["fp32"], ["bf16", "fp32", "fp16"]],
                         ids=["bf16", "fp16", "fp32", "mixed"])
@pytest.mark.parametrize("sizes", CLIP, ids=[f"{len(s)}x{max(s)}" for s in CLIP])
def test_grad_clip(sizes, kinds):
    m = gu.need_gpu()
    types = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)
    grads = [normal(i, (n,), types[kinds[i % len(kinds)]], 0.5) for i, n in enumerate(sizes)]
    norm, _ = clip_ref(grads, 1.0)
    for bound in (0.5 * norm, 10 * norm + 1, math.inf, 0.0):
        _, scale = clip_ref(grads, bound)
        outs = [torch.full_like(t, 7) for t in grads]
        got = m.moe_grad_clip(grads, bound, out=outs)
        assert got.shape == () and got.dtype == torch.float32
        assert abs(float(got) - norm) <= 2.0 ** -19 * norm
        for t, o in zip(grads, outs):
            ref = t.double() * scale
            check(o, ref, rounding(t.dtype, ref) + 2.0 ** -18 * ref.abs(), "out")
        # in place: the same bits
        mine = [t.clone() for t in grads]
        assert float(m.moe_grad_clip(mine, bound)) == float(got)
        assert all(torch.equal(a, b) for a, b in zip(mine, outs))
    before = [t.clone() for t in grads]
    assert float(m.moe_grad_clip(grads, 0.1, norm_only=True)) == float(got)
    assert all(torch.equal(a, b) for a, b in zip(before, grads))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lead_in,lead_out", [(0, 0), (1, 1), (3, 3), (0, 1), (2, 5)])
@pytest.mark.parametrize("n", [1, 7, 8, 9, 8190, 20000])
def test_grad_clip_unaligned_views(n, lead_in, lead_out, dtype):
    m = gu.need_gpu()
    flat = normal(1, (n + 64,), dtype)
    into = torch.full((n + 64,), 3.0, dtype=dtype, device="cuda")
    g, o = flat[lead_in:lead_in + n], into[lead_out:lead_out + n]
    norm, scale = clip_ref([g], 0.25)
    got = m.moe_grad_clip([g], 0.25, out=[o])
    assert abs(float(got) - norm) <= 2.0 ** -19 * norm
    ref = g.double() * scale
    check(o, ref, rounding(dtype, ref) + 2.0 ** -18 * ref.abs(), "out")
    assert bool((into[:lead_out] == 3).all()) and bool((into[lead_out + n:] == 3).all())


def test_grad_clip_not_finite():
    m = gu.need_gpu()
    a, b = normal(1, (100,), torch.float32), normal(2, (50,), torch.bfloat16)
    a[3] = float("inf")
    outs = [torch.empty_like(a), torch.empty_like(b)]
    assert math.isinf(float(m.moe_grad_clip([a, b], 1.0, out=outs)))
    assert bool(outs[0][3].isnan()) and bool((outs[0][4:] == 0).all()) and bool((outs[1] == 0).all())
    a[3] = float("nan")
    assert math.isnan(float(m.moe_grad_clip([a, b], 1.0, out=outs)))
    assert bool(outs[0].isnan().all()) and bool(outs[1].isnan().all())


def test_grad_clip_nothing():
    m = gu.need_gpu()
    assert float(m.moe_grad_clip([], 1.0)) == 0
    z = torch.zeros(10, device="cuda")
    assert float(m.moe_grad_clip([z, z.new_empty(0)], 1.0)) == 0 and bool((z == 0).all())


def test_grad_clip_plan_follows_moved_storage():
    m = gu.need_gpu()
    a, b = normal(1, (1000,), torch.float32), normal(2, (77,), torch.float32)
    t = a.clone()
    plan = m.GradClip([t, b], out=[torch.empty_like(t), torch.empty_like(b)])
    assert float(plan(1.0)) == float(m.moe_grad_clip([a, b], 1.0, norm_only=True))
    keep, t.data = t.data, 2 * a
    assert float(plan(1.0)) == float(m.moe_grad_clip([2 * a, b], 1.0, norm_only=True))
    t.data = a[:10].clone()
    with pytest.raises(ValueError):
        plan(1.0)
    del keep


def test_grad_clip_plan_refuses_changed_tensors():
    m = gu.need_gpu()
    a = normal(1, (1000,), torch.float32)
    for change in (lambda t: t.resize_(10), lambda t: setattr(t, "data", t.data[:10]),
                   lambda t: setattr(t, "data", t.data.bfloat16())):
        for t, o in ((a.clone(), a.clone()), (a.clone(), None)):
            plan = m.GradClip([t], out=None if o is None else [o])
            plan(1.0)
            change(t if o is None else o)
            with pytest.raises(ValueError):
                plan(1.0)


def test_grad_clip_graphs_share_no_workspace():
    """Two recorded calls of one plan, replayed at the same time on two streams."""
    m = gu.need_gpu()
    a = normal(1, (3_000_000,), torch.float32)
    plan, outs = m.GradClip([a], norm_only=True), []
    plan(1.0)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    kept = dict(plan._workspaces)
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(plan(1.0))
    assert plan._workspaces == kept  # a recorded call's workspace belongs to its graph
    streams = [torch.cuda.Stream() for _ in range(2)]
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert float(outs[0]) == float(outs[1]) == float(plan(1.0))


# ---------------------------------------------------------------------------
# 4-bit weights
# ---------------------------------------------------------------------------
def w4_case(seed, E, N, K, group, zeros, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    groups = -(-K // group)
    codes = torch.randint(0, 256, (E, N, (K + 1) // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand((E, N, groups), generator=g, device="cuda")) * 0.3 / math.sqrt(K)).to(dtype)
    z = torch.randint(0, 16, (E, N, groups), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales, z


def w4_dense(codes, scales, zeros, K, group):
    """The weights in fp64."""
    col = torch.arange(K, device="cuda")
    q = (codes[..., col // 2] >> (4 * (col % 2)).to(torch.uint8)) & 15
    z = zeros[..., col // group].double() if zeros is not None else 8.0
    return (q.double() - z) * scales[..., col // group].double()


def w4_bound(x, W, dtype, out_fp32):
    """x W^T over rows of x [R, K] and W [N, K] or [R, N, K], and its bound."""
    if W.dim() == 2:
        y, mag = x.double() @ W.t(), x.double().abs() @ W.abs().t()
    else:
        y = torch.bmm(W, x.double().unsqueeze(2)).squeeze(2)
        mag = torch.bmm(W.abs(), x.double().abs().unsqueeze(2)).squeeze(2)
    off = (x.shape[1] + 16) * ADD * mag
    return y, off + (0 if out_fp32 else rounding(dtype, y.abs() + off)), off


def w4_gated(y, off, act, dtype):
    n = y.shape[1] // 2
    a, d = act64(y[:, :n], act)
    u, og, ou = y[:, n:], off[:, :n], off[:, n:]
    h = a * u
    return h, rounding(dtype, h) + (d.abs() + og) * og * (u.abs() + ou) + a.abs() * ou + ACT * h.abs()


W4 = [(1, 1, 8, 32), (1, 16, 128, 32), (1, 17, 136, 64), (2, 100, 2880, 32), (5, 33, 64, 128),
      (8, 48, 264, 128), (9, 31, 520, 64), (16, 16, 4096, 128), (17, 250, 72, 32), (33, 64, 384, 64),
      (64, 40, 1000, 32), (100, 18, 248, 32)]


@pytest.mark.parametrize("zeros", [False, True], ids=["mid", "zeros"])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,N,K,group", W4)
def test_w4_matvec(T, N, K, group, dtype, zeros):
    m = gu.need_gpu()
    c = w4_case(N + K, 1, N, K, group, zeros, dtype)
    W = w4_dense(*c, K, group)[0]
    x = normal(5, (T, K), dtype)
    for gated in ([False, True] if N % 2 == 0 else [False]):
        w = m.moe_w4_pack(*c, group=group, gated=gated)
        for out_fp32 in (True, False):
            out = gu.Guarded((T, N), torch.float32 if out_fp32 else dtype)
            m.moe_w4_matvec(x, w, out=out.t, out_fp32=out_fp32)
            out.check()
            y, bound, off = w4_bound(x, W, dtype, out_fp32)
            check(out.t, y, bound, "y")
        for act in (["silu", "gelu"] if gated else []):
            out = gu.Guarded((T, N // 2), dtype)
            m.moe_w4_matvec(x, w, act=act, out=out.t)
            out.check()
            check(out.t, *w4_gated(y, off, act, dtype), act)


@pytest.mark.parametrize("zeros", [False, True], ids=["mid", "zeros"])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,E,k,N,K,group", [(1, 4, 2, 32, 256, 32), (8, 4, 2, 50, 136, 64),
                                             (64, 32, 4, 40, 264, 32), (64, 2, 1, 24, 128, 128),
                                             (130, 3, 2, 16, 96, 32), (5, 200, 3, 18, 64, 64)])
def test_w4_routed(T, E, k, N, K, group, dtype, zeros):
    m = gu.need_gpu()
    c = w4_case(E + K, E, N, K, group, zeros, dtype)
    W = w4_dense(*c, K, group)
    x = normal(5, (T, K), dtype)
    g = torch.Generator().manual_seed(T)
    ids = torch.rand((T, E), generator=g).topk(k, dim=1).indices.to(torch.int32)
    if T > 4:
        ids[1, 0], ids[3, k - 1] = E, -1  # out of range: these slots are dropped
    al = m.moe_lora_align(ids.cuda(), None, E, 0, 16, 16)
    slots = [s for s in range(T * k) if 0 <= ids.view(-1)[s] < E]
    slots.sort(key=lambda s: (int(ids.view(-1)[s]), s))
    rows = torch.tensor(slots, device="cuda")
    experts = ids.view(-1)[slots].long().cuda()
    n = len(slots)
    w = m.moe_w4_pack(*c, group=group, gated=N % 2 == 0)
    R = T * k
    for rows_sorted in (False, True):
        xs = x[rows // k]
        xin = x if not rows_sorted else torch.cat([xs, normal(9, (R - n, K), dtype)])
        for out_fp32 in (True, False):
            out = gu.Guarded((R, N), torch.float32 if out_fp32 else dtype, fill=3.0)
            m.moe_w4_matvec(xin, w, al=al, rows_sorted=rows_sorted, out=out.t, out_fp32=out_fp32)
            out.check()
            y, bound, off = w4_bound(xs, W[experts], dtype, out_fp32)
            check(out.t[:n], y, bound, "y")
            assert bool((out.t[n:] == 3).all())  # dropped slots' rows
        h = m.moe_w4_matvec(xin, w, al=al, rows_sorted=rows_sorted, act="silu")
        check(h[:n], *w4_gated(y, off, "silu", dtype), "h")
        assert bool((h[n:] == 0).all())


@pytest.mark.parametrize("every", [False, True], ids=["some", "all"])
def test_w4_routed_zeroes_dropped_rows(every, monkeypatch):
    """An output that the call allocates, in memory that held something else before."""
    m = gu.need_gpu()
    T, E, k, N, K, dt = 37, 5, 2, 18, 64, torch.bfloat16
    codes, scales, _ = w4_case(3, E, N, K, 32, False, dt)
    w = m.moe_w4_pack(codes, scales, group=32, gated=True)
    x = normal(5, (T, K), dt)
    ids = (torch.arange(T * k, device="cuda", dtype=torch.int32).view(T, k) * 3) % (E + 2)  # E, E + 1: dropped
    if every:
        ids.fill_(E)
    al = m.moe_lora_align(ids, None, E, 0, 16, 16)
    n = int((ids < E).sum())
    for act, fp32, cols in ((None, True, N), (None, False, N), ("gelu", False, N // 2)):
        want = torch.full((T * k, cols), 3.0, dtype=torch.float32 if fp32 else dt, device="cuda")
        m.moe_w4_matvec(x, w, al=al, act=act, out_fp32=fp32, out=want)
        with monkeypatch.context() as patch:
            patch.setattr(torch, "empty", lambda shape, **kw: torch.full(shape, 3.0, **kw))
            got = m.moe_w4_matvec(x, w, al=al, act=act, out_fp32=fp32)
        assert torch.equal(got[:n], want[:n]) and bool((got[n:] == 0).all()) and bool((want[n:] == 3).all())


def test_w4_skewed_routing():
    """Experts with many, few and no rows: tiles are shared out by the experts' cost."""
    m = gu.need_gpu()
    T, E, N, K, dt = 150, 70, 400, 136, torch.float16
    codes, scales, _ = w4_case(4, E, N, K, 64, False, dt)
    W = w4_dense(codes, scales, None, K, 64)
    w = m.moe_w4_pack(codes, scales, group=64)
    x = normal(6, (T, K), dt)
    ids = torch.where(torch.arange(T) < 90, 41, torch.arange(T) % 35 * 2).to(torch.int32).view(T, 1)
    al = m.moe_lora_align(ids.cuda(), None, E, 0, 16, 16)
    order = ids.view(-1).sort(stable=True).indices.cuda()
    y, bound, _ = w4_bound(x[order], W[ids.view(-1).cuda()[order].long()], dt, True)
    check(m.moe_w4_matvec(x, w, al=al, out_fp32=True), y, bound, "y")


def test_w4_zero_scale_and_not_finite_rows():
    m = gu.need_gpu()
    codes, scales, _ = w4_case(1, 1, 32, 256, 32, False, torch.bfloat16)
    scales[0, :, 2] = 0  # a group that says nothing
    x = normal(2, (5, 256), torch.bfloat16)
    w = m.moe_w4_pack(codes, scales, group=32)
    y = m.moe_w4_matvec(x, w, out_fp32=True)
    x2 = x.clone()
    x2[:, 64:96] = 100.0
    assert torch.equal(y, m.moe_w4_matvec(x2, w, out_fp32=True))
    x2 = x.clone()
    x2[1, 9], x2[4, 255] = float("nan"), float("inf")
    z = m.moe_w4_matvec(x2, w, out_fp32=True)
    assert torch.equal(z[[0, 2, 3]], y[[0, 2, 3]])
    assert bool(z[1].isnan().all()) and not bool(z[4].isfinite().any())


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("E,N,K,group", [(1, 1, 1, 32), (1, 3, 31, 32), (2, 5, 129, 64), (3, 7, 300, 128)])
def test_w4_quantize(E, N, K, group, dtype):
    m = gu.need_gpu()
    W = normal(3, (E, N, K), dtype)
    W[0, 0, :] = 0
    codes, scales = m.moe_w4_quantize(W, group=group)
    w = W.float().cpu()
    for grp in range(-(-K // group)):
        part = w[..., grp * group:(grp + 1) * group]
        s = (part.abs().amax(-1) / 7).to(dtype)
        assert torch.equal(scales[..., grp].cpu(), s)
        q = torch.where(s.unsqueeze(-1) > 0, part / s.float().unsqueeze(-1), torch.zeros(()))
        q = q.round().clamp(-7, 7).to(torch.int64) + 8
        col = torch.arange(grp * group, grp * group + part.shape[-1])
        got = (codes.cpu()[..., col // 2].long() >> (4 * (col % 2))) & 15
        assert torch.equal(got, q)
    if K % 2:
        assert bool((codes[..., -1] >> 4 == 8).all())


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------
def operators(m):
    """One call of each operator on fixed inputs, as functions of no arguments."""
    dt = torch.bfloat16
    x, W1, dh = normal(1, (70, 128), dt), normal(2, (96, 128), dt, 0.1), normal(3, (70, 48), dt)
    one = x[:2].contiguous()
    grads = [normal(4 + i, (n,), dt) for i, n in enumerate((5000, 33, 9000))]
    outs = [torch.empty_like(t) for t in grads]
    plan = m.GradClip(grads, out=outs)
    c = w4_case(1, 4, 64, 128, 32, False, dt)
    w = m.moe_w4_pack(*c, group=32)
    ids = torch.arange(140, device="cuda", dtype=torch.int32).view(70, 2) % 4
    al = m.moe_lora_align(ids, None, 4, 0, 16, 16)
    torch.cuda.synchronize()
    return [lambda: [m.moe_gated_ffn(x, W1)], lambda: [m.moe_gated_ffn(one, W1)],
            lambda: list(m.moe_gated_ffn_backward(dh, x, W1)),
            lambda: [plan(0.5)] + [o.clone() for o in outs],
            lambda: [m.moe_w4_matvec(x, w, al=al, out_fp32=True)]]


def test_on_another_stream_and_in_a_graph():
    m = gu.need_gpu()
    for f in operators(m):
        want = f()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got = f()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = f()
        for t in got:
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_from_a_new_thread():
    """A thread whose first CUDA call is the operator's (an autograd worker's often is)."""
    m = gu.need_gpu()
    for f in operators(m):
        want, got = f(), []
        torch.cuda.synchronize()
        s = torch.cuda.current_stream()

        def work():
            with torch.cuda.stream(s):
                got.extend(f())

        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(want, got))


def test_same_bits_every_time():
    m = gu.need_gpu()
    for f in operators(m):
        want = f()
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(want, f()))
