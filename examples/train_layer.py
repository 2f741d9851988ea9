"""One training step of a routed expert layer on one GPU.

    python examples/train_layer.py [--tokens 4096 --hidden 2048 --inner 1024
                                    --experts 64 --topk 8 --steps 20]

Forward: dispatch, the experts' two products with a SiLU between them, combine.
Backward: the combine's gradient, both products' gradients, the dispatch's
gradient; then the gradients are clipped to a global norm and the weights
updated.  The router's own products stay in torch.  Every packed row, map and
bucket size stays on the device: the host reads nothing back.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_moe_plan_02_gb300 as moe  # noqa: E402

F32 = torch.float32


def forward(x, topk_idx, topk_w, w_up, w_down, capacity=0):
    """The layer's output and what the backward pass needs.  x bf16 [S, D],
    topk_idx int32 [S, K], topk_w f32 [S, K], w_up bf16 [E, F, D], w_down bf16
    [E, D, F]."""
    E = w_up.shape[0]
    if capacity:
        plan = moe.moe_plan_capacity(topk_idx, E, capacity)
        packed = torch.empty(E * capacity, x.shape[1], dtype=x.dtype, device=x.device)
        moe.moe_dispatch(x, plan.tok_map, packed_x=packed)
    else:
        plan, packed, _ = moe.moe_plan_dispatch(topk_idx, x, E)
    up = moe.moe_expert_gemm(packed, w_up, plan)
    act = torch.nn.functional.silu(up)
    y = moe.moe_expert_gemm(act, w_down, plan)
    out = moe.moe_combine(y, topk_w, plan.tok_map)
    return out, (plan, packed, up, act, y)


def backward(dout, topk_w, w_up, w_down, saved):
    """Gradients of forward for (x, topk_w, w_up, w_down); those of the weights
    in f32."""
    plan, packed, up, act, y = saved
    dy, dtopk_w = moe.moe_combine_backward(dout, y, topk_w, plan)
    dw_down = moe.moe_expert_gemm_wgrad(dy, act, plan)
    dact = moe.moe_expert_gemm_dgrad(dy, w_down, plan)
    s = torch.sigmoid(up.float())
    dup = (dact.float() * s * (1 + up.float() * (1 - s))).to(up.dtype)
    dw_up = moe.moe_expert_gemm_wgrad(dup, packed, plan)
    dpacked = moe.moe_expert_gemm_dgrad(dup, w_up, plan)
    dx = moe.moe_dispatch_backward(dpacked, plan, out_dtype=F32)
    return dx, dtopk_w, dw_up, dw_down


def train_step(x, target, topk_idx, topk_w, weights, lr, max_norm):
    """One step of gradient descent on mean((layer(x) - target)^2).  `weights`
    are the f32 masters [w_up, w_down], updated in place.  Returns the loss and
    the gradient norm, both on the device."""
    w_up, w_down = (w.to(torch.bfloat16) for w in weights)
    out, saved = forward(x, topk_idx, topk_w, w_up, w_down)
    diff = out.float() - target
    loss = diff.square().mean()
    dout = diff * (2.0 / diff.numel())
    _, _, *grads = backward(dout, topk_w, w_up, w_down, saved)
    norm = moe.moe_clip_grad_norm(grads, max_norm)
    for w, g in zip(weights, grads):
        w.add_(g, alpha=-lr)
    return loss, norm


def main():
    p = argparse.ArgumentParser()
    for name, value in (("tokens", 4096), ("hidden", 2048), ("inner", 1024), ("experts", 64),
                        ("topk", 8), ("steps", 20)):
        p.add_argument(f"--{name}", type=int, default=value)
    a = p.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rand(a.tokens, a.hidden).to(torch.bfloat16)
    target = rand(a.tokens, a.hidden)
    scores, topk_idx = rand(a.tokens, a.experts).topk(a.topk)
    topk_idx, topk_w = topk_idx.to(torch.int32), scores.softmax(-1)
    weights = [rand(a.experts, a.inner, a.hidden) * a.hidden ** -0.5,
               rand(a.experts, a.hidden, a.inner) * a.inner ** -0.5]
    events = [torch.cuda.Event(enable_timing=True) for _ in range(a.steps + 1)]
    losses = []
    events[0].record()
    for i in range(a.steps):
        losses.append(train_step(x, target, topk_idx, topk_w, weights, lr=200.0, max_norm=0.009))
        events[i + 1].record()
    torch.cuda.synchronize()
    for i, (loss, norm) in enumerate(losses):
        print(f"step {i}: loss {float(loss):.5f}  gradient norm {float(norm):.4f}  "
              f"{events[i].elapsed_time(events[i + 1]):.2f} ms")
    if moe.moe_device_errors():
        raise RuntimeError("a kernel reported an error")


if __name__ == "__main__":
    main()
