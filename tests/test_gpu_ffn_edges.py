"""The feed-forward operators at values and sizes where they could go wrong: far outliers and
infinities, changed tensors, derivatives that do not exist, and enough work that every CTA
takes several tiles. Bounds are those of test_gpu_ffn."""
import math

import pytest
import torch
from torch.autograd import forward_ad

import gpu_util as gu
from test_gpu_ffn import (ACT, DTYPES, IDS, act64, backward_bounds, check, gated_bounds, half_step, normal, rounding,
                          w4_bound, w4_case, w4_dense, w4_gated)

pytestmark = pytest.mark.gpu


def test_gated_refuses_forward_mode_derivatives():
    """A tangent is refused, not dropped."""
    m = gu.need_gpu()
    x, W1, dh = normal(1, (4, 64), torch.bfloat16), normal(2, (32, 64), torch.bfloat16), normal(3, (4, 16), torch.bfloat16)
    with forward_ad.dual_level():
        dual = [forward_ad.make_dual(t, torch.ones_like(t)) for t in (x, W1, dh)]
        for call in (lambda: m.moe_gated_ffn(dual[0], W1), lambda: m.moe_gated_ffn(x, dual[1]),
                     lambda: m.moe_gated_ffn(dual[0], W1, out=torch.empty_like(dh)),
                     lambda: m.moe_gated_ffn(dual[0], W1.clone().requires_grad_()),
                     lambda: m.moe_gated_ffn_backward(dual[2], x, W1),
                     lambda: m.moe_gated_ffn_backward(dh, dual[0], W1),
                     lambda: m.moe_gated_ffn_backward(dh, x, dual[1])):
            with pytest.raises(RuntimeError, match="forward"):
                call()
        m.moe_gated_ffn(x, W1)  # no tangent: as ever
        m.moe_gated_ffn_backward(dh, x, W1)


def test_grad_clip_plan_refuses_another_type_or_layout_in_place():
    """The same address and number of elements, but other values there."""
    m = gu.need_gpu()
    for into in (False, True):
        for change in (lambda t, buf: t.view(torch.float16), lambda t, buf: buf[::2],
                       lambda t, buf: buf[:1].expand(1000), lambda t, buf: t.cpu()):
            buf = normal(1, (2000,), torch.bfloat16)
            t = buf[:1000]
            plan = m.GradClip([t.clone() if into else t], out=[t] if into else None)
            for _ in range(3):  # the first calls look the tensors over, later ones compare
                plan(1e9)
            t.data = change(t.data, buf)
            with pytest.raises(ValueError):
                plan(1e9)
            with pytest.raises(ValueError):  # and stays refused
                plan(1e9)
            t.data = buf[:1000]
            plan(1e9)


def test_grad_clip_plan_takes_another_view_of_the_same_elements():
    m = gu.need_gpu()
    t = normal(1, (1000,), torch.float32)
    plan = m.GradClip([t], norm_only=True)
    want = float(plan(1.0))
    t.data = t.data.view(10, 100)
    assert float(plan(1.0)) == want
    t.requires_grad_()
    assert float(plan(1.0)) == want
    with torch.inference_mode():
        assert float(plan(1.0)) == want
    t.data = t.data.view(10, 100).t()
    with pytest.raises(ValueError):
        plan(1.0)


@pytest.mark.parametrize("zeros", [False, True], ids=["mid", "zeros"])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,group", [(1, 32), (5, 64), (12, 128), (30, 32)])
def test_w4_columns_of_weight_zero_say_nothing(T, group, dtype, zeros):
    """Outliers in x a million times its usual size (or up to fp16's largest), in columns whose
    codes are the zero point: the result's error does not grow with them."""
    m = gu.need_gpu()
    N, K = 48, 256
    codes, scales, z = w4_case(7, 1, N, K, group, zeros, dtype)
    loud = [3, 40, 41, 100, 255]
    for c in loud:
        q = z[..., c // group] if zeros else torch.full((1, N), 8, dtype=torch.uint8, device="cuda")
        half = codes[..., c // 2]
        codes[..., c // 2] = (half & 15) | (q << 4) if c % 2 else (half & 240) | q
    W = w4_dense(codes, scales, z, K, group)[0]
    assert bool((W[:, loud] == 0).all())
    x = normal(5, (T, K), dtype)
    x[:, loud] = 1e6 if dtype == torch.bfloat16 else 6e4
    for gated in (False, True):
        w = m.moe_w4_pack(codes, scales, z, group=group, gated=gated)
        y, bound, off = w4_bound(x, W, dtype, True)
        check(m.moe_w4_matvec(x, w, out_fp32=True), y, bound, "y")
        if gated:
            check(m.moe_w4_matvec(x, w, act="gelu"), *w4_gated(y, off, "gelu", dtype), "h")


@pytest.mark.parametrize("zeros", [False, True], ids=["mid", "zeros"])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_w4_weights_of_zero_give_zero(dtype, zeros):
    m = gu.need_gpu()
    N, K = 33, 520
    for group in (32, 64, 128):
        z = torch.randint(0, 16, (1, N, -(-K // group)), device="cuda", dtype=torch.uint8) if zeros else None
        q = z.repeat_interleave(group, -1)[..., :K] if zeros else torch.full((1, N, K), 8, dtype=torch.uint8, device="cuda")
        codes = q[..., 0::2] | (q[..., 1::2] << 4)
        scales = torch.full((1, N, -(-K // group)), 0.75, dtype=dtype, device="cuda")
        w = m.moe_w4_pack(codes, scales, z, group=group)
        for T in (1, 9, 20):
            assert bool((m.moe_w4_matvec(normal(3, (T, K), dtype, 1e4), w, out_fp32=True) == 0).all())


@pytest.mark.parametrize("zeros", [False, True], ids=["mid", "zeros"])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_w4_infinities_as_the_definition_has_them(dtype, zeros):
    m = gu.need_gpu()
    N, K = 64, 256
    c = w4_case(9, 1, N, K, 64, zeros, dtype)
    W = w4_dense(*c, K, 64)[0]
    x = normal(2, (6, K), dtype)
    clean = m.moe_w4_matvec(x, m.moe_w4_pack(*c, group=64), out_fp32=True)
    x[1, 9], x[2, 77], x[4, 255] = math.inf, -math.inf, math.inf
    x[4, 8] = math.nan
    x[5, 0], x[5, 200] = math.inf, -math.inf
    y = m.moe_w4_matvec(x, m.moe_w4_pack(*c, group=64), out_fp32=True)
    # inf (q - z) s: an infinity of its sign, NaN where q = z; infinities of two signs: NaN
    want = (x.double().unsqueeze(1) * W).sum(-1)
    assert torch.equal(y[[0, 3]], clean[[0, 3]])
    bad = [1, 2, 4, 5]
    assert torch.equal(y[bad].isnan(), want[bad].isnan())
    assert torch.equal(y[bad].nan_to_num(0, 1, -1), want[bad].nan_to_num(0, 1, -1).float())


@pytest.mark.parametrize("size", [2e37, 1e-30])
@pytest.mark.parametrize("zeros", [False, True], ids=["mid", "zeros"])
@pytest.mark.parametrize("T", [2, 11])
def test_w4_rows_near_the_ends_of_bf16(T, zeros, size):
    """No sum on the way leaves fp32's range where the result does not."""
    m = gu.need_gpu()
    dt = torch.bfloat16
    N, K = 40, 256
    for group in (32, 128):
        c = w4_case(11, 1, N, K, group, zeros, dt)
        x = (normal(4, (T, K), torch.float32).clamp(-3, 3) * size).to(dt)
        y, bound, _ = w4_bound(x, w4_dense(*c, K, group)[0], dt, True)
        check(m.moe_w4_matvec(x, m.moe_w4_pack(*c, group=group), out_fp32=True), y, bound, "y")


@pytest.mark.parametrize("n", [1000, 2_000_000], ids=["one_launch", "two_launches"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 1e25])
def test_grad_clip_infinite_bound_scales_nothing(n, value):
    """Whatever the norm: of an infinity, a NaN, squares past fp32's range."""
    m = gu.need_gpu()
    a, b = normal(1, (n,), torch.float32), normal(2, (77,), torch.bfloat16)
    a[5] = value
    bits = lambda t: t.view(torch.int32 if t.dtype == torch.float32 else torch.int16).clone()  # noqa: E731
    before = [bits(a), bits(b)]
    got = m.moe_grad_clip([a, b])
    assert math.isnan(float(got)) if math.isnan(value) else math.isinf(float(got))
    assert torch.equal(bits(a), before[0]) and torch.equal(bits(b), before[1])
    outs = [torch.zeros_like(a), torch.zeros_like(b)]
    m.moe_grad_clip([a, b], math.inf, out=outs)
    keep = ~a.isnan()
    assert torch.equal(outs[0][keep], a[keep]) and torch.equal(outs[0].isnan(), a.isnan())
    assert torch.equal(outs[1], b)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T", [9, 180])
def test_gated_gates_as_far_as_bf16_goes(T, act):
    """The derivative tends to 0 and 1; its terms on the way there do not overflow into NaN."""
    m = gu.need_gpu()
    dt = torch.bfloat16
    x = torch.zeros((T, 16), dtype=dt, device="cuda")
    far = [-3e38, -1e25, -1e20, -1e15, 0.0, 1e15, 1e20, 1e25, 3e38]
    x[:, 0] = torch.tensor(far * (T // 9), dtype=dt)
    x[:, 1] = 1
    W1 = torch.zeros((16, 16), dtype=dt, device="cuda")
    W1[:8, 0] = 1  # g = x0
    W1[8:, 1] = 1  # u = 1
    g = x[:, :1].double().expand(T, 8)
    a, d = (torch.where(g > 0, g, 0.0), torch.where(g > 0, 1.0, torch.where(g < 0, 0.0, 0.5)))  # the limits
    check(m.moe_gated_ffn(x, W1, act=act), a, rounding(dt, a) + ACT * a.abs(), act)
    dx, _ = m.moe_gated_ffn_backward(torch.ones((T, 8), dtype=dt, device="cuda"), x, W1, act=act)
    want = 8 * d[:, 0]
    check(dx[:, 0], want, 8 * (2 * half_step(dt) * d[:, 0] + ACT), "dx")


def test_grad_clip_graphs_of_other_gradients_do_not_meet():
    """Two recorded calls of one plan, replayed at the same time on two streams, the second with
    other values in the plan's tensors' place: each norm is its own call's."""
    m = gu.need_gpu()
    a = normal(1, (3_000_000,), torch.float32)
    plan = m.GradClip([a], norm_only=True)
    want = [float(plan(1.0))]
    graphs, norms = [torch.cuda.CUDAGraph() for _ in range(2)], []
    with torch.cuda.graph(graphs[0]):
        norms.append(plan(1.0))
    first, other = a.data, 3 * normal(2, (3_000_000,), torch.float32)
    a.data = other  # followed: the second graph reads the other memory
    want.append(float(plan(1.0)))
    with torch.cuda.graph(graphs[1]):
        norms.append(plan(1.0))
    assert abs(want[1] / want[0] - 3) < 0.1
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert [float(v) for v in norms] == want
    del first


# Tiles of 256 rows by 128 features, (rows x features of them), on 76 CTA pairs: 17 x 12 = 204, no
# last wave worth cutting; 14 x 13 = 182, its last 30 cut in halves; 9 x 26 = 234, its last 6 in
# quarters; 5 x 61 = 305, the last one; 2 x 76, two to every pair. Ragged in every direction.
MANY = [(4099, 72, 1416), (3484, 64, 1624), (2057, 136, 3304), (1030, 64, 7720), (512, 72, 9728)]


@pytest.mark.parametrize("act,dtype", [("silu", torch.bfloat16), ("gelu", torch.float16)], ids=["silu-bf16", "gelu-fp16"])
@pytest.mark.parametrize("T,H,I", MANY)
def test_gated_several_tiles_to_a_pair(T, H, I, dtype, act):
    m = gu.need_gpu()
    x = normal(1, (T, H), dtype)
    W1 = normal(2, (2 * I, H), dtype, 1.5 / math.sqrt(H))
    out = gu.Guarded((T, I), dtype)
    m.moe_gated_ffn(x, W1, act=act, out=out.t)
    out.check()
    check(out.t, *gated_bounds(x, W1, act), "h")


@pytest.mark.parametrize("act,dtype", [("gelu", torch.bfloat16), ("silu", torch.float16)], ids=["gelu-bf16", "silu-fp16"])
@pytest.mark.parametrize("T,H,I", MANY + [(1500, 2824, 1032)])
def test_gated_backward_several_tiles_to_a_pair(T, H, I, dtype, act):
    """dg and du of several tiles a pair, dh staged a tile ahead; (1500, 2824, 1032): several
    tiles of dx and dW1 to a pair."""
    m = gu.need_gpu()
    x = normal(1, (T, H), dtype)
    W1 = normal(2, (2 * I, H), dtype, 1.5 / math.sqrt(H))
    dh = normal(3, (T, I), dtype, 0.25)
    dx, dW1 = m.moe_gated_ffn_backward(dh, x, W1, act=act)
    rx, rw = backward_bounds(dh, x, W1, act)
    check(dx, *rx, "dx")
    check(dW1, *rw, "dW1")
    again = m.moe_gated_ffn_backward(dh, x, W1, act=act)
    assert torch.equal(dx, again[0]) and torch.equal(dW1, again[1])


# rows in tiles of 16 on 152 CTAs of 16 warps: several tiles to a warp where N is large, K long
# enough that shared memory holds fewer than 8 rows of x
W4_LARGE = [(3, 40_001, 72, 32), (7, 40_010, 136, 64), (20, 30_007, 264, 128), (40, 24_998, 136, 32),
            (8, 70, 11008, 32), (9, 34, 14336, 64), (33, 18, 16384, 128), (5, 2600, 14336, 32)]


@pytest.mark.parametrize("zeros,dtype", [(False, torch.bfloat16), (True, torch.float16)], ids=["mid-bf16", "zeros-fp16"])
@pytest.mark.parametrize("T,N,K,group", W4_LARGE)
def test_w4_several_tiles_to_a_warp_and_long_rows(T, N, K, group, dtype, zeros):
    m = gu.need_gpu()
    c = w4_case(N + K, 1, N, K, group, zeros, dtype)
    W = w4_dense(*c, K, group)[0]
    x = normal(5, (T, K), dtype)
    y, bound, off = w4_bound(x, W, dtype, True)
    for gated in ([False, True] if N % 2 == 0 else [False]):
        w = m.moe_w4_pack(*c, group=group, gated=gated)
        out = gu.Guarded((T, N), torch.float32)
        m.moe_w4_matvec(x, w, out=out.t, out_fp32=True)
        out.check()
        check(out.t, y, bound, "y")
        if gated:
            out = gu.Guarded((T, N // 2), dtype)
            m.moe_w4_matvec(x, w, act="silu", out=out.t)
            out.check()
            check(out.t, *w4_gated(y, off, "silu", dtype), "h")


# many units of an expert to a CTA; more experts than the shared list holds; long rows whose
# experts take several passes
@pytest.mark.parametrize("T,E,k,N,K,group", [(60, 3, 2, 40_002, 64, 32), (90, 1500, 3, 34, 64, 64),
                                             (150, 5, 1, 66, 14336, 32), (64, 40, 2, 2000, 72, 128)])
def test_w4_routed_several_units_and_many_experts(T, E, k, N, K, group):
    m = gu.need_gpu()
    dtype = torch.bfloat16
    c = w4_case(E + K, E, N, K, group, False, dtype)
    x = normal(5, (T, K), dtype)
    g = torch.Generator().manual_seed(T)
    # some experts get many rows, some none
    weight = torch.rand(E, generator=g).square() + 1e-3
    ids = torch.multinomial(weight.expand(T, E), k, generator=g).to(torch.int32)
    al = m.moe_lora_align(ids.cuda(), None, E, 0, 16, 16)
    flat = ids.view(-1)
    slots = flat.sort(stable=True).indices
    w = m.moe_w4_pack(*c, group=group, gated=True)
    got = m.moe_w4_matvec(x, w, al=al, out_fp32=True)
    h = m.moe_w4_matvec(x, w, al=al, act="gelu")
    at = 0
    for e in range(E):
        n = int((flat == e).sum())
        if n == 0:
            continue
        W = w4_dense(c[0][e:e + 1], c[1][e:e + 1], None, K, group)[0]
        y, bound, off = w4_bound(x[(slots[at:at + n] // k).cuda()], W, dtype, True)
        check(got[at:at + n], y, bound, f"y of expert {e}")
        check(h[at:at + n], *w4_gated(y, off, "gelu", dtype), f"h of expert {e}")
        at += n
    assert at == T * k
