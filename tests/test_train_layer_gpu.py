"""The operators together, as examples/train_layer.py runs them: the whole
layer's gradients against torch's derivative of the same layer in 64 bits.

The layer's bf16 tensors (up, act, y, out and their gradients) are each rounded
once, a relative 2^-8 at most; five such roundings lie between a gradient and
its inputs, and sums of products keep the relative 2-norm error of their terms
to first order (independent roundings, so no worse than their number times
2^-8 in the 2-norm): 5 * 2^-8 = 2 %.
"""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

F64 = torch.float64
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    spec = importlib.util.spec_from_file_location(
        "train_layer", os.path.join(ROOT, "examples", "train_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def inputs(S, D, F, E, K, lost, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    idx = rand(S, E).topk(K).indices.to(torch.int32)
    idx[rand(S, K) < -2.0] = -1 if lost else 0
    return (rand(S, D).to(torch.bfloat16), idx, rand(S, K).softmax(-1),
            (rand(E, F, D) * D ** -0.5).to(torch.bfloat16),
            (rand(E, D, F) * F ** -0.5).to(torch.bfloat16), rand(S, D))


def plain(x, idx, w, w_up, w_down, keep):
    """The layer in 64 bits over every (token, k) entry."""
    out = torch.zeros(x.shape, dtype=F64, device="cuda")
    for e in range(w_up.shape[0]):
        s, k = ((idx == e) & keep).nonzero(as_tuple=True)
        y = torch.nn.functional.silu(x[s] @ w_up[e].T) @ w_down[e].T
        out = out.index_add(0, s, w[s, k, None] * y)
    return out


@pytest.mark.parametrize("capacity", [0, 24])
def test_layer_gradients(layer, capacity):
    import combine_moe_plan_02_gb300 as moe
    S, D, F, E, K = 90, 256, 136, 12, 3
    x, idx, w, w_up, w_down, dout = inputs(S, D, F, E, K, lost=True)
    out, saved = layer.forward(x, idx, w, w_up, w_down, capacity)
    got = layer.backward(dout, w, w_up, w_down, saved)
    torch.cuda.synchronize()
    assert moe.moe_device_errors() == 0
    leaves = [t.to(F64).requires_grad_() for t in (x, w, w_up, w_down)]
    want_out = plain(leaves[0], idx, leaves[1], leaves[2], leaves[3], saved[0].tok_map >= 0)
    want = torch.autograd.grad((want_out * dout.to(F64)).sum(), leaves)
    assert (out.to(F64) - want_out).norm() <= 3 * 2.0 ** -8 * want_out.norm()
    for a, b in zip(got, want):
        assert (a.to(F64) - b).norm() <= 5 * 2.0 ** -8 * b.norm()


def test_training_lowers_the_loss(layer):
    S, D, F, E, K = 256, 128, 64, 8, 2
    x, idx, w, w_up, w_down, target = inputs(S, D, F, E, K, lost=False, seed=1)
    weights = [w_up.float(), w_down.float()]
    losses = [float(layer.train_step(x, target, idx, w, weights, 20.0, 1.0)[0])
              for _ in range(8)]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_a_batch_without_tokens(layer):
    x, idx, w, w_up, w_down, dout = inputs(4, 64, 72, 8, 2, lost=False)
    out, saved = layer.forward(x[:0], idx[:0].contiguous(), w[:0].contiguous(), w_up, w_down)
    dx, dw, dup, ddown = layer.backward(dout[:0], w[:0].contiguous(), w_up, w_down, saved)
    assert out.shape == (0, 64) and dx.shape == (0, 64) and dw.shape == (0, 2)
    assert not dup.any() and not ddown.any()


def test_a_batch_without_tokens_call_by_call():
    """moe_plan and moe_dispatch make no row at all for no tokens."""
    import combine_moe_plan_02_gb300 as moe
    x, idx, w, w_up, _, _ = inputs(4, 64, 72, 8, 2, lost=False)
    plan = moe.moe_plan(idx[:0].contiguous(), 8)
    packed, _ = moe.moe_dispatch(x[:0], plan.tok_map)
    y = moe.moe_expert_gemm(packed, w_up, plan)
    out = moe.moe_combine(y, w[:0].contiguous(), plan.tok_map)
    dy, dw = moe.moe_combine_backward(out, y, w[:0].contiguous(), plan)
    dwe = moe.moe_expert_gemm_wgrad(dy, packed, plan)
    dx = moe.moe_dispatch_backward(moe.moe_expert_gemm_dgrad(dy, w_up, plan), plan)
    assert out.shape == (0, 72) and dy.shape == (0, 72) and dw.shape == (0, 2)
    assert dx.shape == (0, 64) and not dwe.any()
    assert moe.moe_device_errors() == 0
