"""Training a router over frozen 8-bit experts.

The experts of one layer are converted to 8 bits once and frozen; the router
(logits = x R^T) learns to keep the layer's output near a target while the
balance loss spreads the tokens over the experts.  One step:

    route -> balance loss and counts -> route lists -> 8-bit experts -> combine
    -> gradient of the gates -> gradient of the logits (gates and balance loss)
    -> gradient of R

Run from the repository's root:  python examples/router_on_fp8_experts.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import routed_expert_ffn_02_gb300 as moe   # noqa: E402


def run(T=2048, E=32, k=4, H=512, I=512, steps=60, coef=0.1, lr=0.2, seed=0, verbose=True):
    """Trains; returns per-step (output error, balance loss / coef, share of the busiest expert)."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=dev) * scale

    shape = moe.Shape(T, E, k, H, I)
    experts = moe.quantize_experts(*(randn(*s, scale=0.04).to(torch.bfloat16)
                                     for s in ((E, I, H), (E, I, H), (E, H, I))))
    x = randn(T, H).to(torch.bfloat16)
    target = randn(T, H, scale=0.05)
    R = randn(E, H, scale=H ** -0.5)
    R[: E // 8] += 4.0 * x.float().mean(0) + randn(1, H, scale=0.08)   # a router that has collapsed
    # packed sequences of different lengths, the last tokens are padding
    offsets = torch.tensor([0, T // 4, T // 4 + 7, T - 100], dtype=torch.int32, device=dev)
    real = torch.zeros(T, 1, device=dev)
    real[: T - 100] = 1

    ffn_ws = moe.Workspace(moe.expert_ffn_fp8_workspace_size(shape))
    bal_ws = moe.Workspace(moe.balance_workspace_size(T, E, len(offsets) - 1))
    seen = []
    for step in range(steps):
        logits = x.float() @ R.t()
        idx, gates = moe.moe_route(logits, k)
        loss, counts, stats = moe.moe_balance(logits, idx, offsets, coef, ws=bal_ws)
        _, row_offsets, perm, inv = moe.moe_permute(idx, E)
        y = moe.moe_expert_ffn_fp8(shape, x, perm, row_offsets, experts, ws=ffn_ws)
        out = moe.moe_combine(y, inv, gates, T, k, H)
        err = (out.float() - target) * real
        # d(mean square error) / d gate of slot (t, j) = d_out[t] . y of the slot
        d_out = err * (2.0 / err.numel())
        d_gates = torch.bmm(y[inv.long()].view(T, k, H).float(), d_out[:, :, None]).squeeze(2)
        d_logits = moe.moe_balance_backward(logits, stats, counts, k, offsets, coef,
                                            topk_idx=idx, gates=gates, d_gates=d_gates.contiguous())
        R -= lr * (d_logits.t() @ x.float())
        # the layer in one call gives the same output
        if step == 0:
            same = moe.moe_forward_fp8(shape, logits, x, experts)
            assert torch.equal(same, out), "moe_forward_fp8 differs from its parts"
        per_expert = counts.sum(0).float()
        seen.append((err.square().mean().item(), loss.item() / coef,
                     (per_expert.max() / per_expert.sum()).item()))
        if verbose and step % 10 == 0:
            print(f"step {step:3d}  output error {seen[-1][0]:.5f}  balance {seen[-1][1]:.3f}  "
                  f"busiest expert {seen[-1][2]:.3f} of the slots (even: {1 / E:.3f})")
    assert ffn_ws.status() == 0 and bal_ws.status() == 0
    return seen


if __name__ == "__main__":
    run()
