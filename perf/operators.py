"""The feed-forward operators beside the MoE-LoRA layer, as they are measured.

Four operators of one feed-forward block, from its training to its serving:

* ``gated``: h = act(x Wg^T) * (x Wu^T), gate rows first in W1 [2I, H], from one token on;
* ``backward``: its gradients dx and dW1 from dh, x and W1 (nothing else is kept);
* ``clip``: the global norm of many gradient tensors, and the gradients scaled to a bound;
* ``w4``: products with 4-bit weights under group scales for a few tokens, dense or with a
  weight matrix per routed expert, plain or with the gated activation.

Every case is a dict of plain values. ``own`` chooses between the plain form (elementary
torch operations in fp32) and the library's kernels.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-6  # added to the norm before the division, so that a zero norm divides


def listed():
    return [
        # one decode token through a small expert's block: latency
        dict(name="gated_1", op="gated", T=1, H=2880, I=2880, dtype="bf16", act="silu"),
        # a ragged decode batch of a dense 4096/14336 block: the weights' stream
        dict(name="gated_13", op="gated", T=13, H=4096, I=14336, dtype="bf16", act="silu"),
        # a prefill chunk at the 4096/11008 example's size
        dict(name="gated_512", op="gated", T=512, H=4096, I=11008, dtype="bf16", act="silu"),
        # a long prefill, an odd number of tokens, the other type and activation
        dict(name="gated_4099", op="gated", T=4099, H=2880, I=2880, dtype="fp16", act="gelu"),
        # the smallest training step: launches count
        dict(name="backward_64", op="backward", T=64, H=256, I=512, dtype="bf16", act="silu"),
        # narrow experts, an odd number of tokens, fp16
        dict(name="backward_1021", op="backward", T=1021, H=2048, I=768, dtype="fp16", act="gelu"),
        # a full training step of the 4096/11008 example: the largest
        dict(name="backward_4096", op="backward", T=4096, H=4096, I=11008, dtype="bf16", act="silu"),
        # one token against one 4-bit matrix: latency
        dict(name="w4_1", op="w4", T=1, E=1, k=1, N=5760, K=2880, group=32, zeros=False, act="",
             dtype="bf16", out="bf16"),
        # a few tokens through the gated half of a dense 4096/14336 block, zero points
        dict(name="w4_6_gated", op="w4", T=6, E=1, k=1, N=28672, K=4096, group=128, zeros=True,
             act="silu", dtype="fp16", out="fp16"),
        # decode over 32 routed experts: the base product that the adapters are added to
        dict(name="w4_64_routed", op="w4", T=64, E=32, k=4, N=5760, K=2880, group=32, zeros=False,
             act="", dtype="bf16", out="fp32"),
        # one layer's adapters: few small tensors
        dict(name="clip_4", op="clip", count=4, total=196608, dtype="bf16", bound=0.5),
        # the adapters of many layers at full size, fp32 gradients among them
        dict(name="clip_1500", op="clip", count=1500, total=300_000_001, dtype="mixed", bound=0.25),
    ]


def _spread(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, in steps of `step`."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["gated", "backward", "w4", "clip"])
    dtype = rng.choice(["bf16", "fp16"])
    act = rng.choice(["silu", "gelu"])
    if op in ("gated", "backward"):
        while True:
            T = _spread(rng, 1, 8192)
            H, I = _spread(rng, 64, 4096, 8), _spread(rng, 64, 14336, 8)
            if T * H * I <= 4096 * 4096 * 11008:
                return dict(op=op, T=T, H=H, I=I, dtype=dtype, act=act)
    if op == "clip":
        return dict(op=op, count=_spread(rng, 1, 1500), total=_spread(rng, 20_000, 300_000_000),
                    dtype=rng.choice(["bf16", "fp16", "fp32", "mixed"]), bound=rng.choice([0.05, 0.5, 1e9]))
    while True:
        E = rng.choice([1, 1, _spread(rng, 2, 128)])
        k = 1 if E == 1 else rng.randint(1, min(E, 8))
        T, K = _spread(rng, 1, 64), _spread(rng, 64, 14336, 8)
        gated = rng.random() < 0.4
        N = _spread(rng, 16, 28672, 2 if gated else 1)
        if E * N * K <= 32 * 5760 * 2880 and E * T * (N + K) <= 1 << 27:
            return dict(op=op, T=T, E=E, k=k, N=N, K=K, group=rng.choice([32, 64, 128]),
                        zeros=rng.random() < 0.5, act=act if gated else "", dtype=dtype,
                        out=dtype if gated else rng.choice([dtype, "fp32"]))


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(DTYPES[dtype])


def _sizes(case):
    """Uneven tensor sizes that add up to the total: a model's, the same for every seed."""
    g = torch.Generator()
    n, total = case["count"], case["total"]
    g.manual_seed(total)
    cuts = torch.randint(1, total, (n - 1,), generator=g).sort().values.tolist()
    ends = cuts + [total]
    return [b - a for a, b in zip([0] + cuts, ends)]


def _inputs(case, seed):
    """The case's data, from the seed alone."""
    g = _generator(seed)
    op = case["op"]
    if op in ("gated", "backward"):
        T, H, I, dt = case["T"], case["H"], case["I"], case["dtype"]
        s = dict(x=_normal(g, (T, H), dt), W1=_normal(g, (2 * I, H), dt, 1.2 / math.sqrt(H)))
        if op == "backward":
            s["dh"] = _normal(g, (T, I), dt, 0.1)
        return s
    if op == "clip":
        # gradients of uneven sizes and magnitudes, each a tensor of its own; their clipped
        # form goes to buffers that the optimiser reads
        sizes = _sizes(case)
        kinds = ["bf16", "fp32", "fp16"] if case["dtype"] == "mixed" else [case["dtype"]]
        flat = {}
        for i, kind in enumerate(kinds):
            # every tensor starts on its own 16-byte boundary, as allocations do
            room = sum(-(-n // 8) * 8 for n in sizes[i::len(kinds)])
            flat[kind] = _normal(g, (room,), kind, 2.0 / math.sqrt(case["total"]))
        out = {kind: torch.zeros_like(v) for kind, v in flat.items()}
        at = dict.fromkeys(kinds, 0)
        grads, outs = [], []
        for i, n in enumerate(sizes):
            kind = kinds[i % len(kinds)]
            grads.append(flat[kind][at[kind]:at[kind] + n])
            outs.append(out[kind][at[kind]:at[kind] + n])
            at[kind] += -(-n // 8) * 8
        return dict(grads=grads, outs=outs, out=out)
    T, E, k, N, K, G = (case[v] for v in ("T", "E", "k", "N", "K", "group"))
    groups = -(-K // G)
    s = dict(x=_normal(g, (T, K), case["dtype"]))
    s["codes"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s["scales"] = ((0.5 + torch.rand((E, N, groups), generator=g, device="cuda"))
                   * (0.25 / math.sqrt(K))).to(DTYPES[case["dtype"]])
    s["zeros"] = (torch.randint(4, 12, (E, N, groups), generator=g, device="cuda", dtype=torch.uint8)
                  if case["zeros"] else None)
    # each token's k distinct experts
    s["ids"] = (torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
                if E > 1 else None)
    return s


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if own and case["op"] == "clip":
        # a training program keeps its gradient buffers, and the table of them
        import expert_adapter_gemms_gb300 as m
        s["clip"] = m.GradClip(s["grads"], out=s["outs"])
    if own and case["op"] == "w4":
        # a serving program lays its weights out once, when it loads them, and keeps the
        # buffer that its routing is sorted into
        import expert_adapter_gemms_gb300 as m
        s["w4"] = m.moe_w4_pack(s["codes"], s["scales"], s["zeros"], group=case["group"],
                                gated=bool(case["act"]))
        if case["E"] > 1:
            s["al"] = m.new_align(case["T"], case["k"], case["E"], 0, 16, 16)
    return s


def _activation(g, act):
    """The activation and its derivative."""
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return g * p, p * (1 + g * (1 - p))
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1 + th),
            0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g))


def _halves(y):
    n = y.shape[-1] // 2
    return y[..., :n], y[..., n:]


def _plain_clip(s, case):
    squares = [torch.sum(t.float() * t.float()) for t in s["grads"]]
    norm = torch.sqrt(torch.sum(torch.stack(squares)))
    scale = torch.clamp(case["bound"] / (norm + EPS), max=1.0)
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * scale)
    return {"norm": norm, **s["out"]}


def _plain_w4(s, case):
    E, N, K, G, T, k = (case[v] for v in ("E", "N", "K", "group", "T", "k"))
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=-1).view(E, N, K).float()
    zeros = s["zeros"].float() if s["zeros"] is not None else torch.full((), 8.0, device="cuda")
    spread = lambda v: v.repeat_interleave(G, dim=-1)[..., :K] if v.dim() else v  # noqa: E731
    W = (codes - spread(zeros)) * spread(s["scales"].float())
    x = s["x"].float()
    if E == 1:
        y = x @ W[0].t()
    else:
        # slots in the order (expert, slot); each expert's tokens in rows of their own
        expert, order = torch.sort(s["ids"].reshape(-1).long(), stable=True)
        place = torch.arange(T * k, device="cuda") - torch.searchsorted(expert, expert)
        rows = torch.zeros((E, T, K), device="cuda")
        rows[expert, place] = x[order // k]
        y = torch.bmm(rows, W.transpose(1, 2))[expert, place]
    if case["act"]:
        gate, up = _halves(y)
        y = _activation(gate, case["act"])[0] * up
    return y.to(DTYPES[case["out"]])


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import expert_adapter_gemms_gb300 as m
        if op == "gated":
            return m.moe_gated_ffn(s["x"], s["W1"], act=case["act"])
        if op == "backward":
            dx, dW1 = m.moe_gated_ffn_backward(s["dh"], s["x"], s["W1"], act=case["act"])
            return {"dx": dx, "dW1": dW1}
        if op == "clip":
            return {"norm": s["clip"](case["bound"]), **s["out"]}
        al = m.moe_lora_align(s["ids"], None, case["E"], 0, 16, 16, al=s["al"]) if case["E"] > 1 else None
        return m.moe_w4_matvec(s["x"], s["w4"], al=al, act=case["act"] or None,
                               out_fp32=case["out"] == "fp32")
    if op == "clip":
        return _plain_clip(s, case)
    if op == "w4":
        return _plain_w4(s, case)
    x, W1 = s["x"].float(), s["W1"].float()
    gate, up = _halves(x @ W1.t())
    a, da = _activation(gate, case["act"])
    if op == "gated":
        return (a * up).to(s["x"].dtype)
    dh = s["dh"].float()
    dy = torch.cat([dh * up * da, dh * a], dim=1)
    return {"dx": (dy @ W1).to(s["x"].dtype), "dW1": (dy.t() @ x).to(s["x"].dtype)}


def work(case):
    op = case["op"]
    if op in ("gated", "backward"):
        T, H, I = case["T"], case["H"], case["I"]
        one = 4 * T * H * I  # the two projections
        if op == "gated":
            return {"bytes": 2 * (T * H + 2 * I * H + T * I), "flops": one}
        # the projections again, dx and dW1; x, dh and W1 in, dx and dW1 out
        return {"bytes": 2 * (2 * T * H + T * I + 4 * I * H), "flops": 3 * one}
    if op == "clip":
        size = {"bf16": 2, "fp16": 2, "fp32": 4, "mixed": 8 / 3}[case["dtype"]]
        return {"bytes": 2 * size * case["total"], "flops": 3 * case["total"]}
    T, E, k, N, K = (case[v] for v in ("T", "E", "k", "N", "K"))
    met = E * (1 - (1 - k / E) ** T)  # experts that some token goes to
    weights = met * N * (K / 2 + -(-K // case["group"]) * (3 if case["zeros"] else 2))
    outs = T * k * (N // 2 if case["act"] else N) * (4 if case["out"] == "fp32" else 2)
    return {"bytes": weights + 2 * T * K + outs, "flops": 2 * T * k * N * K}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = _inputs(case, seed)
    op = case["op"]
    wide = lambda t: t.to(torch.float64)  # noqa: E731

    def gelu(v):
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))

    f = torch.nn.functional.silu if case.get("act") == "silu" else gelu
    if op == "clip":
        norm = math.sqrt(sum(float(wide(t).square().sum()) for t in s["grads"]))
        scale = min(1.0, case["bound"] / (norm + EPS))
        out = {kind: torch.zeros_like(v, dtype=torch.float64) for kind, v in s["out"].items()}
        # the outputs' places within their buffers, as the views have them
        for t, o in zip(s["grads"], s["outs"]):
            kind = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}[t.dtype]
            at = o.storage_offset()
            out[kind][at:at + t.numel()] = wide(t) * scale
        return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"), **out}
    if op == "w4":
        K, G = case["K"], case["group"]
        column = torch.arange(K, device="cuda")
        q = torch.where(column % 2 == 0, s["codes"][..., column // 2] % 16, s["codes"][..., column // 2] // 16)
        at = column // G
        z = wide(s["zeros"])[..., at] if s["zeros"] is not None else 8.0
        W = ((wide(q) - z) * wide(s["scales"])[..., at])
        del q
        if case["E"] == 1:
            y = wide(s["x"]) @ W[0].t()
        else:
            slots = sorted(range(case["T"] * case["k"]), key=s["ids"].reshape(-1).tolist().__getitem__)
            ids = s["ids"].reshape(-1).tolist()
            y = torch.stack([W[ids[i]] @ wide(s["x"][i // case["k"]]) for i in slots])
        if case["act"]:
            n = y.shape[1] // 2
            y = f(y[:, :n]) * y[:, n:]
        return y
    I = case["I"]
    x, Wg, Wu = wide(s["x"]), wide(s["W1"][:I]), wide(s["W1"][I:])
    g, u = x @ Wg.t(), x @ Wu.t()
    if op == "gated":
        return f(g) * u
    dh = wide(s["dh"])
    with torch.enable_grad():  # the derivative by the chain rule's own record
        v = g.clone().requires_grad_(True)
        a = f(v)
        slope, = torch.autograd.grad(a.sum(), v)
    dg, du = dh * u * slope, dh * a.detach()
    return {"dx": dg @ Wg + du @ Wu, "dW1": torch.cat([dg.t() @ x, du.t() @ x])}
