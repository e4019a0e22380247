"""One feed-forward block from training to 4-bit serving.

A gated block y = (silu(x Wg^T) * (x Wu^T)) Wd^T is fitted to a teacher's outputs with plain
gradient descent: moe_gated_ffn and its backward pass through autograd, the gradients clipped
to a global norm by GradClip, which reads them as they are and hands the optimiser clipped
copies. Then both matrices are quantised to 4 bits with group scales and serve: the gated half
with its activation in one product, the down projection as a plain one. At the end the served
outputs are compared with the 16-bit block's.

    python examples/train_clip_serve.py [--steps 200] [--hidden 256] [--intermediate 512]
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import expert_adapter_gemms_gb300 as m  # noqa: E402


def block(x, W1, Wd):
    return m.moe_gated_ffn(x, W1) @ Wd.t()


def main(steps=200, hidden=256, intermediate=512, tokens=1024, serve_tokens=4, group=32, quiet=False):
    torch.manual_seed(0)
    dt, dev = torch.bfloat16, "cuda"
    H, I = hidden, intermediate
    normal = lambda *s: torch.randn(*s, device=dev)  # noqa: E731
    teacher = [(normal(2 * I, H) / math.sqrt(H)).to(dt), (normal(H, I) / math.sqrt(I)).to(dt)]
    # fp32 master weights, and the 16-bit copies that the kernels read
    master = [t.float() + 0.02 * normal(*t.shape) for t in teacher]
    weights = [t.to(dt).requires_grad_() for t in master]
    for w in weights:
        w.grad = torch.zeros_like(w)
    clipped = [torch.empty_like(w) for w in weights]
    clip = m.GradClip([w.grad for w in weights], out=clipped)
    losses, norms = [], []
    for step in range(steps):
        x = normal(tokens, H).to(dt)
        with torch.no_grad():
            want = block(x, *teacher)
        for w in weights:
            w.grad.zero_()
        loss = (block(x, *weights).float() - want.float()).square().mean()
        loss.backward()
        norms.append(clip(0.05))
        losses.append(loss.detach())
        with torch.no_grad():
            for w, f, g in zip(weights, master, clipped):
                f -= 2.0 * g.float()
                w.copy_(f)
    assert m.ffn_get_error() == 0
    # serving: 4-bit weights, laid out once
    W1, Wd = (w.detach() for w in weights)
    gate_up = m.moe_w4_pack(*m.moe_w4_quantize(W1, group=group), group=group, gated=True)
    down = m.moe_w4_pack(*m.moe_w4_quantize(Wd.contiguous(), group=group), group=group)
    x = normal(serve_tokens, H).to(dt)
    y16 = block(x, W1, Wd).float()
    y4 = m.moe_w4_matvec(m.moe_w4_matvec(x, gate_up, act="silu"), down).float()
    off = float((y4 - y16).norm() / y16.norm())
    losses = [float(v) for v in losses]
    if not quiet:
        print(f"loss {losses[0]:.4g} -> {losses[-1]:.4g} in {steps} steps; gradient norm "
              f"{float(norms[0]):.3g} -> {float(norms[-1]):.3g}")
        print(f"4-bit outputs of {serve_tokens} tokens: {100 * off:.1f} % off the 16-bit block's; weights "
              f"{(gate_up.packed.numel() + down.packed.numel()) / 2**20:.2f} MiB against "
              f"{2 * (W1.numel() + Wd.numel()) / 2**20:.2f} MiB")
    return losses, off


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--intermediate", type=int, default=512)
    a = ap.parse_args()
    main(a.steps, a.hidden, a.intermediate)
