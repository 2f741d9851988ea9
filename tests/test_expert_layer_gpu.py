"""The few-token layer against plain sums in 64 bits.

Bounds, all relative to the sums of the magnitudes that a value is made of:
products are exact, sums f32 with the tensor core's truncation (2^-23 a step of 16
products, at most K / 16 + 16 steps), so (K / 16 + 16) 2^-23 of each projection;
silu adds 2^-20 relative and at most 1.1 of its input's error.  With bf16 weights h
is cut to 16 bits, of which half a step is lost (24 for f32 outputs); with MXFP4 weights x and
h lose at most 2^-23 of the largest of 32 neighbours.  The output's rounding is 2^-8
(bf16) or 2^-24 of the value."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

from tests import mxfp4  # noqa: E402

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def make(S, E, K, H, F, mx, seed, low=-1, scale=1.0):
    """x, ids from low to E - 1 (repeats among them), weights of the entries and of the layer."""
    import combine_moe_plan_02_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(S, H, generator=g, device="cuda") * scale).to(BF16)
    idx = torch.randint(low, E, (S, K), generator=g, device="cuda").to(torch.int32)
    w = torch.randn(S, K, generator=g, device="cuda")
    up = torch.randn(E, 2 * F, H, generator=g, device="cuda") * H ** -0.5
    down = torch.randn(E, H, F, generator=g, device="cuda") * F ** -0.5
    weights = (moe.moe_quant_mxfp4(up), moe.moe_quant_mxfp4(down)) if mx else (up.to(BF16), down.to(BF16))
    return x, idx, w, *weights


def plain(x, idx, w, up, down):
    """(out, bound on its error before the last rounding, for bf16 and f32 outputs)."""
    mx = not isinstance(up, torch.Tensor)
    f = (lambda q, e: mxfp4.values(q.codes[e], q.scales[e])) if mx else (lambda q, e: q[e].to(F64))
    E, F2, H = up.shape
    F = F2 // 2
    step = lambda n: (n / 16 + 16) * 2.0 ** -23  # noqa: E731
    top = lambda v: v.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)  # noqa: E731
    out = torch.zeros(x.shape, dtype=F64, device="cuda")
    wide, fine = torch.zeros_like(out), torch.zeros_like(out)
    for e in idx.unique().tolist():
        if not 0 <= e < E:
            continue
        s, k = (idx == e).nonzero(as_tuple=True)
        v, wu, wd = x[s].to(F64), f(up, e), f(down, e)
        p, off = v @ wu.T, step(H) * (v.abs() @ wu.abs().T)
        if mx:
            off = off + 2.0 ** -23 * (top(v) @ wu.abs().T)
        gate, lift = p[:, :F], p[:, F:]
        act = gate / (1 + torch.exp(-gate))
        h = act * lift
        off = (1.1 * off[:, :F] + 2.0 ** -20 * act.abs()) * (lift.abs() + off[:, F:]) + act.abs() * off[:, F:]
        c = w[s, k].to(F64)[:, None]
        out.index_add_(0, s, c * (h @ wd.T))
        for total, bits in ((wide, 17), (fine, 24)):
            part = off + step(F) * h.abs() + (2.0 ** -23 * top(h.abs() + off) if mx else 2.0 ** -bits * h.abs())
            total.index_add_(0, s, c.abs() * (part @ wd.abs().T) + 2.0 ** -22 * (c * (h @ wd.T)).abs())
    return out, wide, fine


def check(args, **more):
    import combine_moe_plan_02_gb300 as moe
    want, wide, fine = plain(*args)
    for dtype, bound, eps in ((BF16, wide, 2.0 ** -8), (F32, fine, 2.0 ** -24)):
        out = torch.full(args[0].shape, float("nan"), dtype=dtype, device="cuda")
        assert moe.moe_expert_layer(*args, out=out, **more) is out
        off = (out.to(F64) - want).abs()
        bad = (~(off <= bound + eps * want.abs())).nonzero()
        assert not len(bad), (dtype, len(bad), bad[:4].tolist(), float(off.max()), float(want.abs().max()))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("S,E,K,H,F", [
    (1, 1, 1, 32, 32), (1, 8, 2, 64, 32), (2, 4, 3, 96, 160), (3, 16, 8, 224, 96), (5, 24, 3, 1440, 544),
    (7, 3, 2, 512, 256), (8, 2, 1, 256, 64), (16, 256, 8, 2048, 512), (33, 8, 2, 320, 288),
    (64, 8, 8, 544, 128), (128, 1024, 8, 128, 64), (32, 5, 32, 128, 96), (1024, 4, 1, 64, 32)])
def test_sizes(S, E, K, H, F, mx):
    check(make(S, E, K, H, F, mx, S + H))


@pytest.mark.parametrize("S,E,K,H,F", [(1, 3, 2, 8, 8), (4, 5, 2, 40, 24), (5, 24, 3, 1416, 520), (9, 6, 2, 72, 1000)])
def test_odd_widths(S, E, K, H, F):
    check(make(S, E, K, H, F, False, S + H))


@pytest.mark.parametrize("mx", [False, True])
def test_large(mx):
    check(make(1, 16, 8, 6144, 2048, mx, 1, low=0))
    check(make(24, 16, 8, 7168, 2048, mx, 2, low=0))
    check(make(3, 4, 2, 16384, 256, mx, 3))
    check(make(3, 4, 2, 256, 16384, mx, 4))


@pytest.mark.parametrize("mx", [False, True])
def test_all_on_one_expert(mx):
    """Many tokens of one expert, and the same expert several times in a token."""
    args = list(make(48, 6, 4, 512, 160, mx, 5))
    args[1] = torch.full_like(args[1], 3)
    check(args)
    args[1][:, 2:] = -1
    check(args)


@pytest.mark.parametrize("mx", [False, True])
def test_no_expert(mx):
    """Tokens, and whole batches, without a valid id; their weights are not read."""
    import combine_moe_plan_02_gb300 as moe
    args = list(make(6, 4, 2, 256, 96, mx, 6, low=0))
    args[1][2] = torch.tensor([-1, 4], device="cuda")
    args[1][4, 0] = 1 << 30
    args[2][2], args[2][4, 0] = float("nan"), float("inf")
    clean = [t.clone() if isinstance(t, torch.Tensor) else t for t in args]
    clean[2][2], clean[2][4, 0] = 0, 0
    want = plain(*clean)[0]
    got = moe.moe_expert_layer(*args, out_dtype=F32)
    assert (got[2] == 0).all() and torch.isfinite(got).all()
    assert (got.to(F64) - want).abs().max() < 1e-3 * want.abs().max()
    args[1].fill_(-1)
    for dtype in (BF16, F32):
        out = torch.full((6, 256), float("nan"), dtype=dtype, device="cuda")
        assert (moe.moe_expert_layer(*args, out=out) == 0).all()
    assert moe.moe_expert_layer(args[0][:0], args[1][:0], args[2][:0], *args[3:]).shape == (0, 256)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("scale", [1e-15, 1e-4, 3e4])
def test_sizes_of_values(mx, scale):
    """Rows of very small and large values, and a row whose values span 2^60."""
    args = list(make(6, 4, 2, 512, 96, mx, 7, scale=scale))
    x = args[0].float()
    x[1] *= torch.pow(2.0, torch.linspace(-50, 10, 512, device="cuda")) * 1e-3
    args[0] = x.to(BF16)
    check(args)


@pytest.mark.parametrize("mx", [False, True])
def test_nan_and_infinity_stay_in_their_token(mx):
    import combine_moe_plan_02_gb300 as moe
    args = list(make(9, 3, 2, 256, 96, mx, 8, low=0))
    clean = moe.moe_expert_layer(*args)
    args[0] = args[0].clone()
    args[0][2, 5], args[0][7, 250] = float("nan"), float("inf")
    got = moe.moe_expert_layer(*args)
    other = [0, 1, 3, 4, 5, 6, 8]
    assert torch.equal(got[other], clean[other])
    assert got[2].isnan().all() and not torch.isfinite(got[7]).any()
    # an expert that no token has is never read
    idx = args[1].clone()
    idx[idx == 1] = 2
    bad = [q._replace(scales=q.scales.clone()) if mx else q.clone() for q in args[3:]]
    for q in bad:
        (q.scales if mx else q)[1] = 255 if mx else float("nan")
    x = torch.randn_like(args[0])
    assert torch.equal(moe.moe_expert_layer(x, idx, args[2], *bad), moe.moe_expert_layer(x, idx, args[2], *args[3:]))


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_largest_h(sign):
    """h = 2^128 - 2^118 is an f32, but above the largest bf16: every step is exact."""
    import combine_moe_plan_02_gb300 as moe
    up = torch.zeros(1, 16, 8, device="cuda")
    up[0, 0, 0], up[0, 0, 1], up[0, 8, 0] = 2.0 ** 101, -2.0 ** 91, sign * 2.0 ** 27
    down = torch.zeros(1, 8, 8, device="cuda")
    down[0, 3, 0] = 2.0 ** -100
    idx = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    out = moe.moe_expert_layer(torch.ones(1, 8, dtype=BF16, device="cuda"), idx, torch.ones(1, 1, device="cuda"),
                               up.to(BF16), down.to(BF16), out_dtype=F32)
    want = torch.zeros(1, 8, device="cuda")
    want[0, 3] = sign * (2.0 ** 28 - 2.0 ** 18)
    assert torch.equal(out, want)


def test_scales_of_every_size():
    """Weights' scales from the smallest to 2^100, among them rows of zeros."""
    import combine_moe_plan_02_gb300 as moe
    x, idx, w, up, down = make(3, 2, 2, 512, 128, True, 9, low=0, scale=1e-3)
    g = torch.Generator(device="cuda").manual_seed(1)
    up = moe.MxFp4(up.codes, torch.randint(60, 126, up.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    down = moe.MxFp4(down.codes, torch.randint(0, 227, down.scales.shape, generator=g, device="cuda", dtype=torch.uint8))
    up.codes[1, 7] = 0
    check((x, idx, w, up, down))


@pytest.mark.parametrize("mx", [False, True])
def test_reproducible_graph_and_streams(mx):
    import combine_moe_plan_02_gb300 as moe
    sets = [make(16, 8, 4, 1024, 256, mx, 20 + i) for i in range(3)]
    weights = sets[0][3:]
    x, idx, w = (t.clone() for t in sets[0][:3])
    first = [moe.moe_expert_layer(*s[:3], *weights) for s in sets]
    for _ in range(5):
        for s, f in zip(sets, first):
            assert torch.equal(moe.moe_expert_layer(*s[:3], *weights), f)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):   # calls that follow each other on one workspace
            moe.moe_expert_layer(x, idx, w, *weights, out=out)
    for s, f in zip(sets, first):
        for to, t in zip((x, idx, w), s):
            to.copy_(t)
        graph.replay()
        assert torch.equal(out, f)
    ws = torch.empty(moe.moe_expert_layer_workspace_size(16, 1024, 4, 8, 256, mx), dtype=torch.uint8, device="cuda")
    ws.fill_(0xff)   # needs no initialisation
    assert torch.equal(moe.moe_expert_layer(*sets[1][:3], *weights, workspace=ws), first[1])
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(12):
        streams[i % 3].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[i % 3]):
            outs.append(moe.moe_expert_layer(*sets[i % 3][:3], *weights))
    for i in range(3):
        outs.append(moe.moe_expert_layer(*sets[i][:3], *weights, stream=streams[i]))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, first[i % 3])


def test_offsets_past_32_bits():
    """Weights past 2^32 bytes: the last of 180 experts of 2 x 2048 x 4096."""
    import combine_moe_plan_02_gb300 as moe
    E, H, F = 180, 4096, 2048
    up = torch.zeros(E, 2 * F, H, dtype=BF16, device="cuda")
    down = torch.zeros(E, H, F, dtype=BF16, device="cuda")
    x, idx, w, a, b = make(2, 2, 2, H, F, False, 11, low=0)
    up[-2:], down[-2:] = a, b
    got = moe.moe_expert_layer(x, idx + E - 2, w, up, down)
    assert torch.equal(got, moe.moe_expert_layer(x, idx, w, a, b))


def test_against_the_calls_for_batches():
    """The same layer by dispatch, two products and combine, in bf16."""
    import combine_moe_plan_02_gb300 as moe
    x, idx, w, up, down = make(12, 8, 3, 512, 128, False, 12)
    plan, rows, _ = moe.moe_plan_dispatch(idx, x, 8)
    u = moe.moe_expert_gemm(rows, up, plan, out_dtype=F32)
    h = (torch.nn.functional.silu(u[:, :128]) * u[:, 128:]).to(BF16)
    want = moe.moe_combine(moe.moe_expert_gemm(h, down, plan, out_dtype=F32), w, plan.tok_map, out_dtype=F32)
    got = moe.moe_expert_layer(x, idx, w, up, down, out_dtype=F32)
    assert (got - want).norm() < 4e-3 * want.norm()   # h in bf16 there


def test_at_once_with_the_products():
    """Layers of both kinds and products of both kinds on four streams at once: they
    share tensor memory and SMs and must neither wait for one another nor mix."""
    import combine_moe_plan_02_gb300 as moe
    E, H, F = 8, 1024, 256
    layers = [make(12, E, 4, H, F, mx, 30 + mx) for mx in (False, True)]
    x, idx, _, up, _ = layers[0]
    plan, rows, _ = moe.moe_plan_dispatch(idx, x, E)
    qplan = moe.moe_plan(layers[1][1], E)
    q, qup = moe.moe_dispatch_quant_mxfp4(layers[1][0], qplan.tok_map), layers[1][3]
    jobs = [lambda: moe.moe_expert_layer(*layers[0]), lambda: moe.moe_expert_layer(*layers[1]),
            lambda: moe.moe_expert_gemm(rows, up, plan), lambda: moe.moe_expert_gemm_mxfp4(q, qup, qplan)]
    want = [job() for job in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        for job, stream in zip(jobs, streams):
            with torch.cuda.stream(stream):
                got.append(job())
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 4]), i
    assert moe.moe_device_errors() == 0


@pytest.mark.parametrize("mx", [False, True])
def test_two_graphs_share_a_workspace(mx):
    import combine_moe_plan_02_gb300 as moe
    a, b = (make(S, 6, 2, 512, 96, mx, 40 + S) for S in (3, 40))
    ws = torch.empty(max(moe.moe_expert_layer_workspace_size(S, 512, 2, 6, 96, mx) for S in (3, 40)),
                     dtype=torch.uint8, device="cuda")
    want = [moe.moe_expert_layer(*t) for t in (a, b)]
    graphs, outs = [], []
    for t in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(moe.moe_expert_layer(*t, workspace=ws))
    for i in (0, 1, 1, 0, 1, 0, 0):
        outs[i].zero_()
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])


def test_views_and_alignment():
    """Weights and rows inside larger tensors; rows that do not begin on 16 bytes are refused."""
    import combine_moe_plan_02_gb300 as moe
    x, idx, w, up, down = make(5, 4, 2, 256, 96, False, 50)
    more = [torch.cat([t[:1], t, t[:1]]) for t in (up, down)]
    long = torch.cat([x, x])
    want = moe.moe_expert_layer(x, idx, w, up, down)
    assert torch.equal(moe.moe_expert_layer(long[5:], idx, w, more[0][1:5], more[1][1:5]), want)
    flat = torch.zeros(x.numel() + 8, dtype=BF16, device="cuda")
    flat[4:4 + x.numel()] = x.flatten()
    with pytest.raises(moe.MoeError):
        moe.moe_expert_layer(flat[4:4 + x.numel()].view_as(x), idx, w, up, down)
    with pytest.raises(ValueError):
        moe.moe_expert_layer(x, idx.t().contiguous().t(), w, up, down)
    with pytest.raises(ValueError):
        moe.moe_expert_layer(x, idx.cpu(), w, up, down)
    with pytest.raises(moe.MoeError):   # more entries than the call takes
        moe.moe_expert_layer(x.repeat(110, 1), idx.repeat(110, 1), w.repeat(110, 1), up, down)
