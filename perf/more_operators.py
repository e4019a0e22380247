"""The operators of training and serving around the experts' products, as they are measured.

* ``permute``: tokens' rows laid out by expert, and the gradient (each token's rows added up);
* ``unpermute``: the experts' rows brought back and summed with the routing weights, and the
  gradient: of the rows, and through the weights' softmax of the router's logits;
* ``linear``: a projection shared by all rows (or one per expert) with the low-rank adapters of
  many requests beside it, y = x W^T + (x A^T) B^T, and the gradients of x, A and B.

Every case is a dict of plain values. ``own`` chooses between the plain form (elementary
torch operations in fp32) and the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # a decode batch of 64 tokens on its way to 4 of 32 experts each: latency
        dict(name="permute_64", op="permute", back=False, T=64, k=4, E=32, H=2880, dtype="bf16"),
        # the gradient of a prefill-sized training batch coming back to its tokens
        dict(name="permute_back_4096", op="permute", back=True, T=4096, k=4, E=32, H=2880, dtype="bf16"),
        # one decode token's four expert rows: the smallest call
        dict(name="unpermute_1", op="unpermute", back=False, T=1, k=4, E=32, H=2880, dtype="bf16"),
        # a long ragged prefill over many narrow experts, the other 16-bit type
        dict(name="unpermute_4099", op="unpermute", back=False, T=4099, k=8, E=128, H=2048, dtype="fp16"),
        # a small training step over many experts
        dict(name="unpermute_back_256", op="unpermute", back=True, T=256, k=8, E=128, H=2048, dtype="bf16"),
        # a full training step's gradient of fp32 rows and of the router
        dict(name="unpermute_back_4096", op="unpermute", back=True, T=4096, k=2, E=8, H=4096, dtype="fp32"),
        # one decode token with its adapter through a dense projection: the weights' stream
        dict(name="linear_1", op="linear", back=False, T=1, k=1, E=1, L=8, r=16, K=4096, N=4096,
             mixed=True, dtype="bf16"),
        # 64 requests' tokens, their adapters mixed, through the dense 4096/14336 gate and up
        dict(name="linear_64", op="linear", back=False, T=64, k=1, E=1, L=8, r=16, K=4096, N=28672,
             mixed=True, dtype="fp16"),
        # a prefill of 16 requests, one adapter each, through 32 experts' gate and up
        dict(name="linear_experts", op="linear", back=False, T=4096, k=4, E=32, L=16, r=16, K=2880,
             N=5760, mixed=False, dtype="bf16"),
        # the smallest training step, narrow experts and ranks: launches count
        dict(name="linear_back_64", op="linear", back=True, T=64, k=2, E=4, L=2, r=8, K=256, N=1024,
             mixed=True, dtype="fp16"),
        # an odd number of tokens of many adapters at once, wide ranks
        dict(name="linear_back_1021", op="linear", back=True, T=1021, k=1, E=1, L=32, r=64, K=2048,
             N=768, mixed=True, dtype="fp16"),
        # a full training step of 16 adapters beside the 4096/11008 example's projection
        dict(name="linear_back_4096", op="linear", back=True, T=4096, k=1, E=1, L=16, r=32, K=4096,
             N=11008, mixed=False, dtype="bf16"),
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, in steps of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["permute", "unpermute", "linear", "linear"])
    back = rng.random() < 0.5
    if op != "linear":
        while True:
            E = _spread(rng, 2, 256)
            k = rng.randint(1, min(E, 8))
            T, H = _spread(rng, 1, 16384), _spread(rng, 1, 8192)
            if rng.random() < 0.8:
                H = -(-H // 8) * 8  # most models' widths
            dtype = rng.choice(["bf16", "fp16", "fp32"])
            if T * k * H * (4 if dtype == "fp32" else 2) <= 8192 * 4096 * 4:
                return dict(op=op, back=back, T=T, k=k, E=E, H=H, dtype=dtype)
    while True:
        E = rng.choice([1, 1, _spread(rng, 2, 128)])
        k = 1 if E == 1 else rng.randint(1, min(E, 8))
        T, L, r = _spread(rng, 1, 8192), _spread(rng, 1, 128), rng.choice([8, 16, 24, 32, 64, 128])
        K, N = _spread(rng, 64, 14336, 8), _spread(rng, 64, 14336, 8)
        if (T * k * K * N <= 4096 * 4096 * 11008 and E * N * K <= 32 * 5760 * 2880
                and E * L * r * (K + N) <= 1 << 27 and T * k * (K + N) <= 1 << 28 and min(E * L, T * k) <= 1024):
            return dict(op=op, back=back, T=T, k=k, E=E, L=L, r=r, K=K, N=N,
                        mixed=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp16"]))


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DTYPES[dtype])


def _adapters(case, g):
    """Each token's adapter, -1 for the base model alone: requests of uneven lengths, their
    tokens one after the other (a prefill) or mixed (a decode batch)."""
    T, L = case["T"], case["L"]
    if case["mixed"]:
        of = torch.randint(0, L, (T,), generator=g, device="cuda")
    else:
        # as many requests as adapters; where one request ends and the next begins
        ends = torch.randint(0, T + 1, (L - 1,), generator=g, device="cuda").sort().values
        of = torch.searchsorted(ends, torch.arange(T, device="cuda"), right=True)
    off = torch.rand((L,), generator=g, device="cuda") < 0.1  # requests without an adapter
    of = torch.where(off[of], -1, of)
    return of.to(torch.int32)


def _inputs(case, seed):
    """The case's data, from the seed alone."""
    g = _generator(seed)
    T, k, E, dt = case["T"], case["k"], case["E"], case["dtype"]
    s = {}
    logits = torch.randn((T, E), generator=g, device="cuda")
    top = logits.topk(k, dim=1)
    s["ids"] = top.indices.to(torch.int32)
    s["w"] = torch.softmax(top.values, dim=1)
    if case["op"] == "permute":
        s["rows" if case["back"] else "x"] = _normal(g, (T * k if case["back"] else T, case["H"]), dt)
    elif case["op"] == "unpermute":
        s["o"] = _normal(g, (T * k, case["H"]), dt)
        if case["back"]:
            s["dy"] = _normal(g, (T, case["H"]), dt, 0.1)
    else:
        L, r, K, N = (case[v] for v in ("L", "r", "K", "N"))
        s["token_adapter"] = _adapters(case, g)
        s["x"] = _normal(g, (T * k, K), dt)
        s["W"] = _normal(g, (E, N, K), dt, 1 / math.sqrt(K))
        s["A"] = _normal(g, (L, E, r, K), dt, 1 / math.sqrt(K))
        s["B"] = _normal(g, (L, E, N, r), dt, 0.5 / math.sqrt(r))
        if case["back"]:
            s["dy"] = _normal(g, (T * k, N), dt, 0.1)
    return s


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    E, k, L = case["E"], case["k"], case.get("L", 0)
    # the order of the rows, by expert, adapter and place: a program has it in hand, from its
    # routing (or its batch's adapters), for every operator of the block and both directions
    if own:
        import expert_adapter_gemms_gb300 as m
        s["al"] = m.moe_lora_align(s["ids"], s.get("token_adapter"), E, L, 256, 16)
        return s
    key = s["ids"].reshape(-1).long() * (L + 1)
    if L:
        key += s["token_adapter"].long().repeat_interleave(k) + 1
    s["order"] = torch.sort(key, stable=True).indices
    s["row"] = torch.empty_like(s["order"])
    s["row"][s["order"]] = torch.arange(len(s["order"]), device="cuda")
    if case["op"] == "linear":
        counts = torch.bincount(key, minlength=E * (L + 1)).tolist()
        s["segments"], at = [], 0  # (expert, adapter, first row, behind the last)
        for i, n in enumerate(counts):
            if n:
                s["segments"].append((i // (L + 1), i % (L + 1) - 1, at, at + n))
            at += n
        s["experts"] = {}
        for e, _, a, b in s["segments"]:
            s["experts"][e] = (s["experts"].get(e, (a, b))[0], b)
    return s


def _plain_linear(s, case):
    x, dtype, tokens = s["x"].float(), s["x"].dtype, case["E"] == 1
    A, B = s["A"].float(), s["B"].float()
    if tokens:
        x = x[s["order"]]
    if not case["back"]:
        y = torch.empty((x.shape[0], case["N"]), device="cuda")
        for e, (a, b) in s["experts"].items():
            y[a:b] = x[a:b] @ s["W"][e].float().t()
        for e, l, a, b in s["segments"]:
            if l >= 0:
                y[a:b] += (x[a:b] @ A[l, e].t()) @ B[l, e].t()
        return (y[s["row"]] if tokens else y).to(dtype)
    dy = s["dy"].float()
    if tokens:
        dy = dy[s["order"]]
    dx, dA, dB = torch.empty_like(x), torch.zeros_like(A), torch.zeros_like(B)
    for e, (a, b) in s["experts"].items():
        dx[a:b] = dy[a:b] @ s["W"][e].float()
    for e, l, a, b in s["segments"]:
        if l >= 0:
            z, v = x[a:b] @ A[l, e].t(), dy[a:b] @ B[l, e]
            dx[a:b] += v @ A[l, e]
            dA[l, e] = v.t() @ x[a:b]
            dB[l, e] = dy[a:b].t() @ z
    dx = dx[s["row"]] if tokens else dx
    return {"dx": dx.to(dtype), "dA": dA.to(dtype), "dB": dB.to(dtype)}


def run(s):
    case = s["case"]
    op, back = case["op"], case["back"]
    T, k = case["T"], case["k"]
    if own:
        import expert_adapter_gemms_gb300 as m
        al = s["al"]
        if op == "permute":
            # the gradient of the rows' layout is their unweighted sum, token by token
            return m.moe_unpermute(s["rows"], al) if back else m.moe_permute(s["x"], al)
        if op == "unpermute":
            if not back:
                return m.moe_unpermute(s["o"], al, s["w"])
            do, dw = m.moe_unpermute_backward(s["dy"], s["o"], al, s["w"])
            return {"do": do, "dlogits": m.moe_topk_softmax_backward(dw, s["ids"], s["w"], case["E"])}
        # dense: rows in the tokens' order; experts: in the order that moe_permute made
        rows_sorted = case["E"] > 1
        if not back:
            return m.moe_lora_linear(s["x"], s["W"], s["A"], s["B"], al, rows_sorted=rows_sorted)
        dx, dA, dB = m.moe_lora_linear_backward(s["dy"], s["x"], s["W"], s["A"], s["B"], al,
                                                rows_sorted=rows_sorted)
        return {"dx": dx, "dA": dA, "dB": dB}
    if op == "linear":
        return _plain_linear(s, case)
    if op == "permute":
        if not back:
            return s["x"][s["order"] // k]
        return s["rows"].float()[s["row"]].view(T, k, -1).sum(dim=1).to(s["rows"].dtype)
    o, w = s["o"].float(), s["w"]
    mine = o[s["row"]].view(T, k, -1)
    if not back:
        return (mine * w[:, :, None]).sum(dim=1).to(s["o"].dtype)
    dy = s["dy"].float()
    do = ((dy[:, None, :] * w[:, :, None]).reshape(T * k, -1)[s["order"]]).to(s["o"].dtype)
    dw = (mine * dy[:, None, :]).sum(dim=2)
    dl = w * (dw - (w * dw).sum(dim=1, keepdim=True))
    dlogits = torch.zeros((T, case["E"]), device="cuda")
    dlogits[torch.arange(T, device="cuda")[:, None], s["ids"].long()] = dl
    return {"do": do, "dlogits": dlogits}


def work(case):
    T, k, E = case["T"], case["k"], case["E"]
    S = T * k
    size = 4 if case["dtype"] == "fp32" else 2
    if case["op"] != "linear":
        H = case["H"]
        if case["op"] == "permute":
            return {"bytes": size * H * (T + S) + 4 * S, "flops": S * H}
        if not case["back"]:
            return {"bytes": size * H * (T + S) + 8 * S, "flops": 2 * S * H}
        # dy and the rows in, the rows' gradient out; weights, ids and places in, logits' gradient out
        return {"bytes": size * H * (T + 2 * S) + 12 * S + 4 * T * E, "flops": 3 * S * H}
    L, r, K, N = (case[v] for v in ("L", "r", "K", "N"))
    met = E * (1 - (1 - k / E) ** T)  # experts that some token goes to
    if case["mixed"]:  # (expert, adapter) pairs that some row has
        pairs = E * L * (1 - (1 - k / (E * L)) ** T)
    else:
        pairs = L * E * (1 - (1 - k / E) ** (T / L))
    adapters = 0.9 * pairs * r * (K + N)
    one = 2 * S * (K * N + 0.9 * r * (K + N))
    if not case["back"]:
        return {"bytes": 2 * (met * N * K + S * (K + N) + adapters), "flops": one}
    # x, dy, W, A and B in; dx out, and dA and dB of every adapter
    return {"bytes": 2 * (met * N * K + S * (2 * K + N) + adapters + E * L * r * (K + N)),
            "flops": one + 2 * S * 0.9 * 2 * r * (K + N)}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits: token by token choices as matrices of
    ones, or expert by expert and adapter by adapter with masks."""
    s = _inputs(case, seed)
    T, k, E = case["T"], case["k"], case["E"]
    S, L = T * k, case.get("L", 0)
    wide = lambda t: t.to(torch.float64)  # noqa: E731
    ids = s["ids"].reshape(-1).tolist()
    of = s["token_adapter"].tolist() if L else [-1] * T
    # the slots by (expert, adapter, slot)
    order = sorted(range(S), key=lambda i: (ids[i], of[i // k], i))
    at = torch.tensor(order, device="cuda")
    if case["op"] == "permute" and not case["back"]:
        return wide(s["x"]).index_select(0, at // k)
    if case["op"] != "linear":
        rows = wide(s["rows" if case["op"] == "permute" else "o"])
        w = wide(s["w"]).reshape(-1)[at] if case["op"] == "unpermute" else None
        if not case["back"] or case["op"] == "permute":
            if w is not None:
                rows = rows * w[:, None]
            return torch.zeros((T, rows.shape[1]), dtype=torch.float64, device="cuda").index_add_(0, at // k, rows)
        dy = wide(s["dy"]).index_select(0, at // k)
        dw = torch.empty(S, dtype=torch.float64, device="cuda")
        dw[at] = torch.einsum("sh,sh->s", rows, dy)
        # the softmax of the chosen logits: its Jacobian, token by token
        p = wide(s["w"])
        jac = torch.diag_embed(p) - p[:, :, None] * p[:, None, :]
        dl = torch.bmm(jac, dw.view(T, k, 1)).view(T, k)
        return {"do": dy * w[:, None],
                "dlogits": torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_add_(1, s["ids"].long(), dl)}
    if 2 * S * case["K"] * case["N"] * (2 if case["back"] else 1) > 8e12:
        return None  # minutes in 64 bits
    expert = torch.tensor([ids[i] for i in order], device="cuda")
    adapter = torch.tensor([of[i // k] for i in order], device="cuda")
    if E == 1:  # the rows are the tokens, as they come
        expert, adapter = torch.zeros(S, dtype=torch.long, device="cuda"), torch.tensor(of, device="cuda")
    x = wide(s["x"])
    pairs = sorted(set(zip(expert.tolist(), adapter.tolist())))
    if not case["back"]:
        y = torch.zeros((S, case["N"]), dtype=torch.float64, device="cuda")
        for e in sorted({e for e, _ in pairs}):
            m = (expert == e).nonzero()[:, 0]
            y[m] = torch.einsum("sk,nk->sn", x[m], wide(s["W"][e]))
        for e, l in pairs:
            if l >= 0:
                m = ((expert == e) & (adapter == l)).nonzero()[:, 0]
                y[m] += torch.einsum("sk,rk,nr->sn", x[m], wide(s["A"][l, e]), wide(s["B"][l, e]))
        return y
    dy = wide(s["dy"])
    out = {"dx": torch.zeros_like(x),
           "dA": torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda"),
           "dB": torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")}
    for e in sorted({e for e, _ in pairs}):
        m = (expert == e).nonzero()[:, 0]
        out["dx"][m] = torch.einsum("sn,nk->sk", dy[m], wide(s["W"][e]))
    for e, l in pairs:
        if l < 0:
            continue
        m = ((expert == e) & (adapter == l)).nonzero()[:, 0]
        a, b = wide(s["A"][l, e]), wide(s["B"][l, e])
        out["dx"][m] += (dy[m] @ b) @ a
        out["dA"][l, e] = (b.t() @ dy[m].t()) @ x[m]
        out["dB"][l, e] = dy[m].t() @ (x[m] @ a.t())
    return out
