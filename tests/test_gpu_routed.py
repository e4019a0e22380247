"""Rows by expert and back, the router's gradient and the projection with adapters, against their
definitions in fp64, element by element.

Bounds are worst cases of the arithmetic: an output rounds by half a step (eps / 2 of its type), a
sum of n fp32 products is off by at most n 2^-23 of the sum of magnitudes (adds that may truncate),
z and v enter a product as two 16-bit values (2^-16 of them in bf16: two roundings of 2^-9 relative, the
second of the first's remainder; 2^-22 and fp16's smallest half step in fp16, where the adapters'
gradients take the remainder times 2^11: a half step of 2^-36).
"""
import math

import pytest
import torch

import gpu_util as gu

pytestmark = pytest.mark.gpu

ADD = 2.0 ** -23   # one fp32 addition, relative to the sum of magnitudes
SUB16 = 2.0 ** -25  # half of fp16's subnormal step
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(dtype, v):
    return half_step(dtype) * v.abs() + (SUB16 if dtype == torch.float16 else 0.0)


def normal(seed, shape, dtype, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def check(got, ref, bound, what):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= bound)
    if bool(bad.any()):
        i = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.numel()} out of bounds, first at {i}: "
                             f"{got[i].item()!r} for {ref[i].item()!r}, bound {bound[i].item():.3g}")


def routing(seed, T, k, E, L=0, drop=False, mixed=True):
    """(ids, w, token_adapter): distinct experts per token; with `drop` some ids out of range."""
    g = torch.Generator()
    g.manual_seed(seed)
    ids = torch.rand((T, E), generator=g).topk(k, dim=1).indices.to(torch.int32)
    w = torch.rand((T, k), generator=g)
    of = None
    if L:
        of = torch.randint(-1, L, (T,), generator=g, dtype=torch.int32)
        if not mixed:
            of = of.sort().values
    if drop and T:
        ids[torch.rand((T, k), generator=g) < 0.2] = E + 5
        ids[0] = -7  # a token without any kept slot
        if of is not None:
            of[-1] = L + 3
    return ids.cuda(), w.cuda(), None if of is None else of.cuda()


def order_of(al):
    """The kept slots in sorted order, and each slot's row."""
    n = al.header()["n_valid"]
    return al.sorted_slots()[:n].long(), al.slot_row().long()


ROWS = [  # T, k, E, H
    (1, 1, 1, 8), (1, 4, 32, 2880), (7, 3, 5, 1), (5, 2, 4, 3), (33, 8, 16, 264), (64, 4, 32, 2880), (129, 2, 3, 100),
    (700, 4, 8, 4099), (3000, 2, 64, 128), (2, 32, 40, 520),
]


@pytest.mark.parametrize("drop", [False, True], ids=["kept", "dropped"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,k,E,H", ROWS)
def test_rows_and_back(T, k, E, H, dtype, drop):
    m = gu.need_gpu()
    dt = TYPES[dtype]
    ids, w, _ = routing(T + H, T, k, E, drop=drop)
    al = m.moe_lora_align(ids, None, E, 0, 256, 16)
    slots, rows = order_of(al)
    n, S = len(slots), T * k
    x, o, dy = normal(1, (T, H), dt), normal(2, (S, H), dt), normal(3, (T, H), dt)
    o[n:] = math.nan  # rows that hold nothing are not read
    if drop:
        w[rows.view(T, k) < 0] = math.nan  # nor the weights of dropped slots

    xs = m.moe_permute(x, al)
    assert torch.equal(xs[:n], x[slots // k]) and not bool(xs[n:].any())
    out = gu.Guarded((S, H), dt, fill=7.0)
    m.moe_permute(x, al, out=out.t)
    out.check()
    assert torch.equal(out.t[:n], xs[:n]) and bool((out.t[n:] == 7).all())

    wide, ww = o[:n].double(), w.reshape(-1)[slots].double()
    zero = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for weights, scaled in ((w, wide * ww[:, None]), (None, wide)):
        ref = zero.index_add(0, slots // k, scaled)
        mag = zero.index_add(0, slots // k, scaled.abs())
        y = gu.Guarded((T, H), dt)
        m.moe_unpermute(o, al, weights, out=y.t)
        y.check()
        check(y.t, ref, rounding(dt, ref) + (k + 1) * ADD * mag, "unpermute")
        assert torch.equal(m.moe_unpermute(o, al, weights), y.t)

        do, dw = m.moe_unpermute_backward(dy, o, al, weights)
        ref = dy.double()[slots // k] * (1 if weights is None else ww[:, None])
        check(do[:n], ref, rounding(dt, ref) + 2 * ADD * ref.abs(), "do")
        assert not bool(do[n:].any())
        prod = wide * dy.double()[slots // k]
        refw, magw = (torch.zeros(S, dtype=torch.float64, device="cuda") for _ in range(2))
        refw[slots], magw[slots] = prod.sum(1), prod.abs().sum(1)
        check(dw.view(-1), refw, H * ADD * magw, "dw")
        only, none = m.moe_unpermute_backward(dy, None, al, weights, need_dw=False)
        assert torch.equal(only, do) and none is None
        none, only = m.moe_unpermute_backward(dy, o, al, weights, need_do=False)
        assert torch.equal(only, dw) and none is None


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 4, 2), (64, 32, 4), (33, 128, 8), (9, 1024, 32), (300, 40, 3)])
def test_router_gradient(T, E, k):
    m = gu.need_gpu()
    logits = normal(T, (T, E), torch.float32)
    dw = normal(T + 1, (T, k), torch.float32)
    ids, w = m.moe_topk_softmax(logits, k)
    got = m.moe_topk_softmax_backward(dw, ids, w, E)
    p, d = w.double(), dw.double()
    dl = p * (d - (p * d).sum(1, keepdim=True))
    ref = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, ids.long(), dl)
    mag = torch.zeros_like(ref).scatter_(1, ids.long(), p * (d.abs() + (p * d.abs()).sum(1, keepdim=True)))
    check(got, ref, (k + 4) * ADD * mag, "dlogits")
    # against differences of the softmax over the same choice, in fp64
    h = 1e-6
    v = normal(T + 2, (T, E), torch.float64)

    def f(s):
        return (torch.softmax(torch.gather(logits.double() + s * v, 1, ids.long()), 1) * d).sum()

    slope = (f(h) - f(-h)) / (2 * h)
    # the weights are fp32 values of an exponential, off by a few 2^-22; differences leave 1e-8
    tol = 1e-5 * float((mag * v.abs()).sum()) + 1e-8 * T
    assert abs(float((got.double() * v).sum()) - float(slope)) <= tol
    # through autograd
    leaf = logits.clone().requires_grad_(True)
    ids2, w2 = m.moe_topk_softmax(leaf, k)
    assert torch.equal(ids2, ids) and torch.equal(w2, w) and not ids2.requires_grad
    w2.backward(dw)
    assert torch.equal(leaf.grad, got)


def test_router_gradient_of_odd_ids():
    """Ids out of range take no part; the same id twice adds up."""
    m = gu.need_gpu()
    ids = torch.tensor([[0, 9, 2], [1, 1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, math.nan, 0.5], [0.25, 0.75, math.nan]], device="cuda")
    dw = torch.tensor([[1.0, math.nan, 3.0], [1.0, 2.0, math.nan]], device="cuda")
    got = m.moe_topk_softmax_backward(dw, ids, w, 3)
    assert got.tolist() == [[-0.5, 0.0, 0.5], [0.0, 0.0, 0.0]]


# ---------------------------------------------------------------------------
# the projection with adapters
# ---------------------------------------------------------------------------
def linear_reference(x, W, A, B, expert, adapter, dy=None):
    """Values and bounds in fp64: y, or dx, dA, dB. expert, adapter: per row; expert -1: no row."""
    dt = x.dtype
    split = 2.0 ** -16 if dt == torch.bfloat16 else 2.0 ** -22
    floor = 2 * SUB16 if dt == torch.float16 else 0.0
    f64 = dict(dtype=torch.float64, device="cuda")
    R, K, N, r = x.shape[0], x.shape[1], W.shape[1], A.shape[2]
    xd, Wd, Ad, Bd = x.double(), W.double(), A.double(), B.double()
    out = {}
    if dy is None:
        y, by = torch.zeros((R, N), **f64), torch.zeros((R, N), **f64)
    else:
        dyd = dy.double()
        dx, bx = torch.zeros((R, K), **f64), torch.zeros((R, K), **f64)
        dA, bA = torch.zeros(A.shape, **f64), torch.zeros(A.shape, **f64)
        dB, bB = torch.zeros(B.shape, **f64), torch.zeros(B.shape, **f64)
    for e in range(W.shape[0]):
        rows = (expert == e).nonzero()[:, 0]
        if not len(rows):
            continue
        if dy is None:
            y[rows] = xd[rows] @ Wd[e].t()
            by[rows] = (K + 2 * r) * ADD * (xd[rows].abs() @ Wd[e].abs().t())
        else:
            dx[rows] = dyd[rows] @ Wd[e]
            bx[rows] = (N + 2 * r) * ADD * (dyd[rows].abs() @ Wd[e].abs())
        for l in range(A.shape[0]):
            mine = ((expert == e) & (adapter == l)).nonzero()[:, 0]
            if not len(mine):
                continue
            a, b, xr = Ad[l, e], Bd[l, e], xd[mine]
            z = xr @ a.t()
            ez = K * ADD * (xr.abs() @ a.abs().t())
            if dy is None:
                y[mine] += z @ b.t()
                by[mine] += (ez + split * z.abs() + floor + (K + 2 * r) * ADD * z.abs()) @ b.abs().t()
                continue
            g, n = dyd[mine], len(mine)
            v = g @ b
            ev = N * ADD * (g.abs() @ b.abs())
            dx[mine] += v @ a
            bx[mine] += (ev + split * v.abs() + floor + (N + 2 * r) * ADD * v.abs()) @ a.abs()
            dA[l, e], dB[l, e] = v.t() @ xr, g.t() @ z
            bA[l, e] = (ev + (split + 2 * n * ADD) * v.abs() + floor / 2048).t() @ xr.abs()
            bB[l, e] = g.abs().t() @ (ez + (split + 2 * n * ADD) * z.abs() + floor / 2048)
    if dy is None:
        return y, by + rounding(dt, y)
    return {"dx": (dx, bx + rounding(dt, dx)), "dA": (dA, bA + rounding(dt, dA)), "dB": (dB, bB + rounding(dt, dB))}


def linear_inputs(seed, R, E, L, r, K, N, dt):
    return (normal(seed, (R, K), dt), normal(seed + 1, (E, N, K), dt, 1 / math.sqrt(K)),
            normal(seed + 2, (L, E, r, K), dt, 1 / math.sqrt(K)), normal(seed + 3, (L, E, N, r), dt, 0.5 / math.sqrt(r)),
            normal(seed + 4, (R, N), dt, 0.1))


def row_owners(al, rows_sorted):
    """Each row's expert and adapter (-1: a dropped row's expert)."""
    n = al.header()["n_valid"]
    e = torch.full((al.S,), -1, dtype=torch.long, device="cuda")
    l = torch.full((al.S,), -1, dtype=torch.long, device="cuda")
    at = torch.arange(n, device="cuda") if rows_sorted else al.sorted_slots()[:n].long()
    e[at], l[at] = al.row_expert()[:n].long(), al.row_adapter()[:n].long()
    return e, l


def run_linear(m, al, rows_sorted, E, L, r, K, N, dt, seed):
    R = al.S
    x, W, A, B, dy = linear_inputs(seed, R, E, L, r, K, N, dt)
    expert, adapter = row_owners(al, rows_sorted)
    gone = expert < 0
    x[gone] = math.nan  # dropped rows are not read into anything
    dy[gone] = math.nan
    y, by = linear_reference(x, W, A, B, expert, adapter)
    y[gone], by[gone] = 0, 0
    m.ffn_clear_error()
    out = gu.Guarded((R, N), dt, fill=7.0)
    m.moe_lora_linear(x, W, A, B, al, rows_sorted=rows_sorted, out=out.t)
    out.check()
    assert m.ffn_get_error() == 0
    assert bool((out.t[gone] == 7).all())
    got = m.moe_lora_linear(x, W, A, B, al, rows_sorted=rows_sorted)
    assert torch.equal(got[~gone], out.t[~gone])
    check(got, y, by, "y")
    ref = linear_reference(x, W, A, B, expert, adapter, dy)
    grads = dict(zip(("dx", "dA", "dB"), m.moe_lora_linear_backward(dy, x, W, A, B, al, rows_sorted=rows_sorted)))
    assert m.ffn_get_error() == 0
    ref["dx"][0][gone], ref["dx"][1][gone] = 0, 0
    for name, (value, bound) in ref.items():
        check(grads[name], value, bound, name)
    return x, W, A, B, dy, got, grads


DENSE = [  # T, L, r, K, N
    (1, 1, 8, 64, 64), (1, 8, 16, 512, 256), (5, 3, 24, 72, 136), (31, 7, 64, 256, 200), (33, 2, 32, 1000, 120),
    (64, 64, 16, 512, 640), (65, 5, 128, 264, 128), (128, 40, 72, 320, 264), (129, 4, 16, 256, 256), (257, 3, 8, 136, 72),
    (300, 70, 64, 192, 520), (600, 5, 128, 520, 328), (1021, 32, 40, 64, 768), (2500, 2, 32, 128, 1032),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,L,r,K,N", DENSE)
def test_linear_shared(T, L, r, K, N, dtype):
    """One projection, tokens as they come, adapters mixed among them."""
    m = gu.need_gpu()
    _, _, of = routing(T + L, T, 1, 1, L)
    al = m.moe_lora_align(torch.zeros((T, 1), dtype=torch.int32, device="cuda"), of, 1, L, 256, 16)
    run_linear(m, al, False, 1, L, r, K, N, TYPES[dtype], 10 * T)


EXPERTS = [  # T, k, E, L, r, K, N, bm_base, bm_lora
    (3, 2, 4, 2, 8, 64, 72, 256, 16), (64, 2, 4, 2, 8, 256, 1024, 256, 16), (200, 4, 8, 5, 16, 136, 256, 64, 7),
    (500, 3, 5, 1, 32, 200, 520, 256, 16), (1500, 1, 3, 20, 64, 128, 264, 128, 16), (90, 8, 128, 3, 16, 64, 128, 16, 1),
]


@pytest.mark.parametrize("drop", [False, True], ids=["kept", "dropped"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,k,E,L,r,K,N,bm_base,bm_lora", EXPERTS)
def test_linear_experts(T, k, E, L, r, K, N, bm_base, bm_lora, dtype, drop):
    """A projection per expert, rows in sorted order; some slots dropped."""
    m = gu.need_gpu()
    ids, _, of = routing(T + L, T, k, E, L, drop=drop)
    al = m.moe_lora_align(ids, of, E, L, bm_base, bm_lora)
    run_linear(m, al, True, E, L, r, K, N, TYPES[dtype], 10 * T)


@pytest.mark.parametrize("T", [20, 100, 400])
@pytest.mark.parametrize("rows_sorted", [False, True], ids=["tokens", "sorted"])
def test_linear_dropped_tokens(T, rows_sorted):
    """Tokens of adapters out of range, and experts with k = 1 in the tokens' order."""
    m = gu.need_gpu()
    for E in (1, 3):
        ids, _, of = routing(T, T, 1, E, 4, drop=True)
        al = m.moe_lora_align(ids, of, E, 4, 256, 16)
        run_linear(m, al, rows_sorted, E, 4, 16, 128, 136, torch.bfloat16, T)
