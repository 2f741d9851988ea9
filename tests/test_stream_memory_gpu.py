"""Calls on another stream than the current one, while the current stream is
behind and goes on using the memory of tensors that are already freed: no
output, workspace or temporary of a call may lie there.

Blocks of every size that the calls ask for are freed while fills of them with
NaN bytes are pending on the current stream; the calls then run on a stream of
their own.  Their inputs are ready, so their results have to be those of the
same calls on the current stream alone.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16 = torch.bfloat16


def busy():
    a = torch.ones(8192, 8192, dtype=BF16, device="cuda")
    b = torch.empty_like(a)
    for _ in range(40):
        torch.mm(a, a, out=b)
    return a, b


def flat(result):
    if torch.is_tensor(result):
        return [result]
    return [t for r in result if torch.is_tensor(r) or isinstance(r, tuple) for t in flat(r)]


def compare(f):
    """f(stream) on the current stream, then on another beside pending fills."""
    torch.cuda.synchronize()
    want = [t.clone() for t in flat(f(None))]
    sizes = [t.numel() * t.element_size() for t in want] + [512, 4096, 65536, 1 << 20]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        torch.cuda.synchronize()
        keep = busy()
        trash = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
                 for n in sizes for _ in range(3)]
        for t in trash:
            t.fill_(255)
        del trash, t
        got = flat(f(stream))
        side.synchronize()
        torch.cuda.synchronize()
        assert len(got) == len(want)
        for a, b in zip(got, want):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        del keep


@pytest.fixture(scope="module")
def data():
    g = torch.Generator(device="cuda").manual_seed(0)
    S, H, E, K = 20000, 64, 64, 8
    idx = torch.rand(S, E, generator=g, device="cuda").topk(K).indices.to(torch.int32).contiguous()
    return dict(S=S, H=H, E=E, K=K, idx=idx,
                x=torch.randn(S, H, generator=g, device="cuda").to(BF16),
                w=torch.rand(S, K, generator=g, device="cuda"),
                y=torch.randn(S * K, H, generator=g, device="cuda").to(BF16),
                we=torch.randn(E, 128, H, generator=g, device="cuda").to(BF16))


def test_plan_dispatch_and_combine(data):
    import combine_moe_plan_02_gb300 as moe
    d = data

    def f(stream):
        plan, px, _ = moe.moe_plan_dispatch(d["idx"], d["x"], d["E"], stream=stream)
        out = moe.moe_combine(px, d["w"], plan.tok_map, stream=stream)
        return plan, px, out
    compare(f)
    compare(lambda s: moe.moe_plan(d["idx"], d["E"], stream=s))

    def g(stream):                               # entries of packed_src without a row are not written
        plan = moe.moe_plan_capacity(d["idx"], d["E"], 2600, stream=stream)
        return plan.cnt, plan.off, plan.tok_map, plan.n_invalid, plan.n_dropped
    compare(g)


def test_products_and_gradients(data):
    import combine_moe_plan_02_gb300 as moe
    d = data
    plan = moe.moe_plan(d["idx"], d["E"])
    y = moe.moe_expert_gemm(d["y"], d["we"], plan)

    def f(stream):
        return (moe.moe_expert_gemm(d["y"], d["we"], plan, stream=stream),
                moe.moe_expert_gemm_dgrad(y, d["we"], plan, stream=stream),
                moe.moe_expert_gemm_wgrad(y, d["y"], plan, stream=stream),
                moe.moe_combine_backward(d["x"], d["y"], d["w"], plan, stream=stream),
                moe.moe_dispatch_backward(d["y"], plan, stream=stream))
    compare(f)


@pytest.mark.parametrize("kw", [dict(), dict(capacity=2600), dict(quant_block=64)])
def test_op(data, kw):
    import combine_moe_plan_02_gb300 as moe
    d = data
    op = moe.MoeOp(d["E"], **kw)
    rows = d["E"] * 2600 if "capacity" in kw else d["S"] * d["K"]
    y = torch.randn(rows, d["H"], device="cuda").to(BF16)

    def f(stream):
        _, total, routing = op.dispatch(d["x"], d["w"], d["idx"], stream=stream)
        return (total, routing.plan.tok_map, op.combine(y, routing, stream=stream),
                op.combine_backward(d["x"], y, routing, stream=stream),
                op.dispatch_backward(y, routing, stream=stream))
    compare(f)


@pytest.mark.parametrize("kw", [dict(), dict(group_size=8), dict(capacity=2600)])
def test_op_with_64_bit_ids(data, kw):
    import combine_moe_plan_02_gb300 as moe
    d = data
    op = moe.MoeOp(d["E"], **kw)
    idx = d["idx"].long()

    def f(stream):
        _, total, routing = op.dispatch(d["x"], d["w"], idx, stream=stream)
        return total, routing.plan.cnt, routing.plan.tok_map
    compare(f)
