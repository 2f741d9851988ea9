"""The combine's and the dispatch's gradients against plain sums in 64 bits.

dy is one product in f32 and one rounding: it has to be equal.  dw is a sum of
H products in f32, each addition off by at most 2^-24 of the magnitudes
summed: H * 2^-24 * sum |dout * y|.  Rows of y that no entry fills, and every
output before the call, hold NaN.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def route(S, E, K, seed, lost=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.rand(S, E, generator=g, device="cuda").topk(K).indices.to(torch.int32)
    idx[torch.rand(S, K, generator=g, device="cuda") < lost] = -1
    return idx.contiguous()


def case(S, H, E, K, ytype, dtype, cap=0, lost=0.0, seed=0):
    import combine_moe_plan_02_gb300 as moe
    idx = route(S, E, K, seed, lost)
    plan = moe.moe_plan_capacity(idx, E, cap) if cap else moe.moe_plan(idx, E)
    rows = E * cap if cap else S * K + 2
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    y = torch.full((rows, H), float("nan"), dtype=ytype, device="cuda")
    used = plan.tok_map[plan.tok_map >= 0]
    y[used] = torch.randn(used.numel(), H, generator=g, device="cuda").to(ytype)
    w = torch.randn(S, K, generator=g, device="cuda").softmax(-1)
    dout = torch.randn(S, H, generator=g, device="cuda").to(dtype)
    return plan, y, w, dout


def check(plan, y, w, dout):
    import combine_moe_plan_02_gb300 as moe
    S, K = w.shape
    dy = torch.full_like(y, float("nan"))
    dw = torch.full_like(w, float("nan"))
    got = moe.moe_combine_backward(dout, y, w, plan, dy=dy, dw=dw)
    assert got[0] is dy and got[1] is dw
    torch.cuda.synchronize()
    assert moe.moe_device_errors() == 0
    want = torch.zeros_like(y)
    ok = plan.tok_map >= 0
    at = plan.tok_map[ok]
    token = torch.arange(S, device="cuda")[:, None].expand(S, K)[ok]
    want[at] = (w[ok][:, None] * dout[token].float()).to(y.dtype)
    assert torch.equal(dy, want)
    product = dout[token].to(F64) * y[at].to(F64)
    ref = torch.zeros(S, K, dtype=F64, device="cuda")
    bound = ref.clone()
    ref[ok] = product.sum(-1)
    bound[ok] = product.abs().sum(-1) * y.shape[1] * 2.0 ** -24
    assert ((dw.to(F64) - ref).abs() <= bound).all()


@pytest.mark.parametrize("ytype,dtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("S,H,E,K,cap,lost", [
    (1, 8, 1, 1, 0, 0.0),
    (1, 7168, 8, 8, 0, 0.0),
    (3, 264, 16, 5, 0, 0.5),
    (40, 1032, 12, 9, 0, 0.1),          # more entries than are held at once
    (17, 640, 40, 32, 0, 0.2),
    (300, 512, 24, 3, 31, 0.05),        # padded, some dropped
    (700, 2056, 64, 8, 0, 0.0),
    (9, 4104, 8, 2, 0, 1.0),            # no entry has a row
])
def test_shapes(S, H, E, K, cap, lost, ytype, dtype):
    check(*case(S, H, E, K, ytype, dtype, cap, lost, seed=S + K))


def test_no_tokens_clears_the_rows():
    import combine_moe_plan_02_gb300 as moe
    idx = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    plan = moe.moe_plan_capacity(idx, 4, 3)
    y = torch.ones(12, 64, dtype=BF16, device="cuda")
    dy, dw = moe.moe_combine_backward(torch.empty(0, 64, dtype=BF16, device="cuda"), y,
                                      torch.empty(0, 2, device="cuda"), plan,
                                      dy=torch.full_like(y, float("nan")))
    torch.cuda.synchronize()
    assert not dy.any() and dw.shape == (0, 2)


def test_an_entry_outside_the_rows_is_dropped():
    import combine_moe_plan_02_gb300 as moe
    plan, y, w, dout = case(6, 64, 4, 2, F32, F32)
    plan.tok_map[2, 1] = 1 << 40
    dy, dw = moe.moe_combine_backward(dout, y, w, plan)
    torch.cuda.synchronize()
    assert moe.moe_device_errors() == 4
    assert dw[2, 1] == 0 and moe.moe_device_errors() == 0


def test_repeated_calls_agree():
    import combine_moe_plan_02_gb300 as moe
    plan, y, w, dout = case(500, 3080, 32, 6, BF16, BF16)
    dy, dw = moe.moe_combine_backward(dout, y, w, plan)
    for _ in range(3):
        dy2, dw2 = moe.moe_combine_backward(dout, y, w, plan)
        assert torch.equal(dw, dw2)


def test_against_differences():
    """The combine is linear in w: with whole numbers and f32 outputs,
    <dout, C(w + e) - C(w)> equals the gradient for that weight exactly."""
    import combine_moe_plan_02_gb300 as moe
    S, H, E, K = 5, 64, 6, 3
    plan = moe.moe_plan(route(S, E, K, 4, 0.2), E)
    g = torch.Generator(device="cuda").manual_seed(9)
    y = torch.randint(-3, 4, (S * K, H), generator=g, device="cuda").float()
    w = torch.randint(-2, 3, (S, K), generator=g, device="cuda").float()
    dout = torch.randint(-3, 4, (S, H), generator=g, device="cuda").float()
    dy, dw = moe.moe_combine_backward(dout, y, w, plan)
    base = moe.moe_combine(y, w, plan.tok_map, out_dtype=F32)
    for k in range(K):
        step = w.clone()
        step[:, k] += 1
        diff = moe.moe_combine(y, step, plan.tok_map, out_dtype=F32) - base
        assert torch.equal((diff * dout).sum(-1), dw[:, k])
    step = torch.randint(-1, 2, y.shape, generator=g, device="cuda").float()
    diff = moe.moe_combine(y + step, w, plan.tok_map, out_dtype=F32) - base
    live = torch.zeros(S * K, dtype=torch.bool, device="cuda")
    live[plan.tok_map[plan.tok_map >= 0]] = True
    assert (diff * dout).sum() == (step * dy)[live].sum()


@pytest.mark.parametrize("kw", [dict(), dict(capacity=20), dict(group_size=4),
                                dict(weighted=False, fold=False), dict(quant_block=64)])
def test_op_round_trip(kw):
    """MoeOp's gradients from the handle: sums in 64 bits over the map."""
    import combine_moe_plan_02_gb300 as moe
    S, H, E, K = 33, 128, 8, 3
    op = moe.MoeOp(E, **kw)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(S, H, generator=g, device="cuda").to(BF16)
    w = torch.randn(S, K, generator=g, device="cuda").softmax(-1)
    out, total, routing = op.dispatch(x, w, route(S, E, K, 3, 0.1))
    y = torch.randn(routing.rows, H, generator=g, device="cuda").to(BF16)
    dout = torch.randn(S, H, generator=g, device="cuda").to(BF16)
    dy, dw = op.combine_backward(dout, y, routing)
    dx = op.dispatch_backward(y, routing, out_dtype=F32)
    m = routing.plan.tok_map
    ok = m >= 0
    rows = y[m.clamp(min=0)].to(F64) * ok[..., None]
    assert ((dx.to(F64) - rows.sum(1)).abs() <= K * 2.0 ** -23 * rows.abs().sum(1)).all()
    token = torch.arange(S, device="cuda")[:, None].expand(S, K)[ok]
    c = w[ok] if kw.get("weighted", True) else torch.ones_like(w[ok])
    assert torch.equal(dy[m[ok]], (c[:, None] * dout[token].float()).to(BF16))
    if not kw.get("weighted", True):
        assert dw is None
    else:
        ref = (rows * dout.to(F64)[:, None]).sum(-1)
        mass = (rows * dout.to(F64)[:, None]).abs().sum(-1)
        assert ((dw.to(F64) - ref).abs() <= H * 2.0 ** -24 * mass).all()


def busy():
    """Work that keeps the current stream at it for some tens of ms."""
    a = torch.ones(8192, 8192, dtype=BF16, device="cuda")
    for _ in range(40):
        a = (a @ a).clamp_(max=1)


@pytest.mark.parametrize("raw", [False, True])
def test_unweighted_op_beside_a_busy_stream(raw):
    """The gradient of an unweighted op on a stream of its own, while the
    current stream is behind and reuses the memory of what was freed: before
    the call with NaN in it, after the call filled at once."""
    import combine_moe_plan_02_gb300 as moe
    S, H, E, K = 3000, 512, 8, 3
    op = moe.MoeOp(E, weighted=False, fold=False)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(S, H, generator=g, device="cuda").to(BF16)
    w = torch.full((S, K), 0.25, device="cuda")
    _, _, routing = op.dispatch(x, w, route(S, E, K, 3))
    dout = torch.randn(S, H, generator=g, device="cuda").to(BF16)
    y = torch.randn(routing.rows, H, generator=g, device="cuda").to(BF16)
    m = routing.plan.tok_map
    side = torch.cuda.Stream()
    for _ in range(5):
        trash = [torch.full((S, K), float("nan"), device="cuda") for _ in range(8)]
        busy()
        torch.cuda.synchronize()
        del trash
        busy()                                   # the current stream is behind from here on
        dy, dw = op.combine_backward(dout, y, routing,
                                     stream=side.cuda_stream if raw else side)
        mine = [torch.full((S, K), 7.0, device="cuda") for _ in range(8)]
        side.synchronize()
        torch.cuda.synchronize()
        assert dw is None and torch.equal(dy[m], dout[:, None].expand(S, K, H))
        assert all((t == 7).all() for t in mine)
    assert moe.moe_device_errors() == 0
