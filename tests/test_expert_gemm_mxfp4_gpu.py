"""The experts' product in MXFP4 against plain sums in 64 bits.

Codes are random and scales of two neighbouring sizes: products are multiples of
a quarter, below 36 * 4 a pair, so every sum of up to 2^16 of them is exact in f32 whatever
the order (2^16 * 144 * 4 < 2^26, and random signs keep the partial sums of the lengths
used here below 2^22): f32 outputs equal the 64-bit sums, bf16 outputs their one rounding.  With scales
of many sizes the bound is derived: 64 products enter the accumulator at a time,
each addition off by at most 2^-23 of what has been summed, so (len / 64 + 64) *
2^-23 times the sum of the products' magnitudes.

Rows in no bucket hold codes and scales of anything (255, NaN, among them), and
outputs before the call NaN."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

from tests import mxfp4  # noqa: E402
from tests.test_expert_gemm_gpu import filled, make_plan  # noqa: E402

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def operand(shape, seed, low=126, high=127):
    import combine_moe_plan_02_gb300 as moe
    return moe.MxFp4(*mxfp4.random(shape, seed, low=low, high=high))


def poison(x, plan):
    """Rows in no bucket: NaN scales over codes that are not zero."""
    dead = ~filled(plan, x.shape[0])
    x.codes[dead] = 0x7e
    x.scales[:, dead] = 255
    return x


def reference(x, w, plan, absolute=False):
    """Sums in 64 bits, bucket by bucket."""
    f = (lambda t: t.abs()) if absolute else (lambda t: t)
    out = torch.zeros(x.shape[0], w.shape[1], dtype=F64, device="cuda")
    cnt, off = plan.cnt.tolist(), plan.off.tolist()
    for e, c in enumerate(cnt):
        if c:
            s = slice(off[e], off[e] + c)
            rows = mxfp4.values(x.codes[s].contiguous(), x.scales[:, s].contiguous())
            out[s] = f(rows) @ f(mxfp4.values(w.codes[e], w.scales[e])).T
    return out


def check(counts, N, D, capacity=0, tail=0, seed=0):
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan(counts, capacity, tail)
    rows += -rows % 4
    x = poison(operand((rows, D), seed), plan)
    w = operand((len(counts), N, D), seed + 1)
    want = reference(x, w, plan)
    for dtype in (F32, BF16):
        y = torch.full((rows, N), float("nan"), dtype=dtype, device="cuda")
        got = moe.moe_expert_gemm_mxfp4(x, w, plan, out=y)
        assert got is y
        bad = (y != want.to(F32).to(dtype)).nonzero()
        assert not len(bad), (dtype, len(bad), bad[:8].tolist())
    assert moe.moe_device_errors() == 0


@pytest.mark.parametrize("counts,N,D", [
    ([4], 8, 32), ([1], 8, 64), ([128], 256, 256), ([128], 256, 128), ([256], 256, 512),
    ([3, 1, 2], 24, 96), ([5, 0, 7, 1], 264, 160), ([129], 136, 224), ([130, 127, 1], 512, 288),
    ([600, 0, 33, 257], 320, 1440), ([31, 32, 33, 34, 35, 36], 520, 2048)])
def test_small(counts, N, D):
    check(counts, N, D)


@pytest.mark.parametrize("seed", range(3))
def test_ragged(seed):
    g = torch.Generator().manual_seed(seed)
    counts = torch.randint(0, 300, (24,), generator=g).tolist()
    check(counts, 8 * (40 + seed), 32 * (30 + 7 * seed), seed=seed)


@pytest.mark.parametrize("capacity", [4, 13, 172])
def test_padded(capacity):
    g = torch.Generator().manual_seed(capacity)
    counts = torch.randint(0, capacity + 1, (24,), generator=g).tolist()
    check(counts, 1048, 1440, capacity=capacity, tail=5)


def test_many_experts():
    check([1] * 1024, 72, 96)
    check([0] * 1000 + [7] * 24, 264, 64)
    check([0, 0, 0], 64, 64, tail=9)


def test_every_start_and_length():
    """Buckets of every length to 70 behind every place in a group of four rows."""
    for lead in range(4):
        check([lead] + list(range(1, 71)), 64, 96, seed=lead)
    check([1, 253, 2, 254, 3, 255, 0, 256, 1, 257, 383, 384, 385, 509, 513], 40, 288)


def test_large():
    check([512 + 7 * (i % 5) - 14 for i in range(64)], 2048, 7168)
    check([i % 9 for i in range(256)], 4096, 2048)


def test_scales_of_many_sizes():
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([100, 31, 300, 1])
    D, N = 7168, 264
    x, w = operand((rows, D), 1, 90, 150), operand((4, N, D), 2, 100, 140)
    want, most = reference(x, w, plan), reference(x, w, plan, True)
    y = moe.moe_expert_gemm_mxfp4(x, w, plan, out_dtype=F32)
    bound = (D / 64 + 64) * 2.0 ** -23 * most
    assert ((y.to(F64) - want).abs() <= bound).all()
    y = moe.moe_expert_gemm_mxfp4(x, w, plan)
    assert ((y.to(F64) - want).abs() <= bound + 2.0 ** -8 * want.abs()).all()


def test_long_positive_sums():
    """The sum's low bits: 32768 positive products."""
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([8])
    D, N = 32768, 64
    x, w = operand((rows, D), 3, 120, 130), operand((1, N, D), 4, 127, 127)
    x, w = (moe.MxFp4(t.codes & 0x77, t.scales) for t in (x, w))
    want = reference(x, w, plan)
    for dtype, off in ((F32, 2e-5), (BF16, 2.0 ** -8 + 1e-4)):
        y = moe.moe_expert_gemm_mxfp4(x, w, plan, out_dtype=dtype)
        assert ((y.to(F64) - want).abs() <= off * want).all(), float(((y.to(F64) - want) / want).abs().max())


def test_nan_stays_in_its_row():
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([40, 8])
    x, w = operand((rows, 256), 5), operand((2, 64, 256), 6)
    x.scales[1, 7, 2] = 255
    w.scales[0, 0, 3, 1] = 255
    y = moe.moe_expert_gemm_mxfp4(x, w, plan, out_dtype=F32)
    want = torch.zeros(rows, 64, dtype=torch.bool, device="cuda")
    want[7] = True
    want[:40, 3] = True
    assert torch.equal(y.isnan(), want)


def test_bad_bucket():
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([8, 8, 8])
    plan.cnt[1] = 30
    x, w = operand((rows, 64), 7), operand((3, 64, 64), 8)
    y = torch.full((rows, 64), 7.0, device="cuda")
    moe.moe_expert_gemm_mxfp4(x, w, plan, out=y)
    assert moe.moe_device_errors() == 32
    plan.cnt[1] = 0
    want = reference(x, w, plan).to(F32)
    assert torch.equal(y[:8], want[:8]) and torch.equal(y[16:], want[16:])


def test_offsets_past_32_bits():
    """Rows and outputs whose bytes and elements pass 2^32."""
    import combine_moe_plan_02_gb300 as moe
    rows, D, N = 1 << 20, 32, 2304
    plan, _ = make_plan([3, 5, 2])
    plan.off[1:] = torch.tensor([3, rows // 2 + 1, rows], device="cuda")
    plan.off[0], plan.off[1], plan.off[2] = 0, rows // 2 - 4, rows - 2
    x, w = operand((rows, D), 9), operand((3, N, D), 10)
    y = torch.empty(rows, N, device="cuda")
    moe.moe_expert_gemm_mxfp4(x, w, plan, out=y)
    at = torch.cat([torch.arange(o, o + c) for o, c in zip(plan.off.tolist(), plan.cnt.tolist())])
    rows_of = torch.repeat_interleave(torch.arange(3), plan.cnt.cpu().long())
    for r, e in zip(at.tolist(), rows_of.tolist()):
        v = mxfp4.values(x.codes[r:r + 1], x.scales[:, r:r + 1].contiguous())
        assert torch.equal(y[r].to(F64), (v @ mxfp4.values(w.codes[e], w.scales[e]).T)[0])
    y[at.cuda()] = 0
    assert int(torch.count_nonzero(y)) == 0


def test_whole_layer_graph_and_streams():
    """Dispatch, both products with the activation between, combine: in a graph,
    replayed on new rows, and on two streams at once."""
    import combine_moe_plan_02_gb300 as moe
    S, E, K, H, F = 96, 8, 3, 256, 160
    g = torch.Generator(device="cuda").manual_seed(0)
    w_up = moe.moe_quant_mxfp4(torch.randn(E, 2 * F, H, generator=g, device="cuda") * H ** -0.5)
    w_down = moe.moe_quant_mxfp4(torch.randn(E, H, F, generator=g, device="cuda") * F ** -0.5)
    idx = torch.rand(S, E, generator=g, device="cuda").topk(K).indices.to(torch.int32)
    topk_w = torch.rand(S, K, generator=g, device="cuda")
    xs = [torch.randn(S, H, generator=g, device="cuda").to(BF16) for _ in range(3)]

    def layer(x):
        plan = moe.moe_plan(idx, E)
        u = moe.moe_expert_gemm_mxfp4(moe.moe_dispatch_quant_mxfp4(x, plan.tok_map), w_up, plan)
        y = moe.moe_expert_gemm_mxfp4(moe.moe_swiglu_quant_mxfp4(u), w_down, plan)
        return moe.moe_combine(y, topk_w, plan.tok_map, out_dtype=F32)

    def plain(x):
        """The same roundings, in 64 bits."""
        out = torch.zeros(S, H, dtype=F64)
        up, down = (mxfp4.values(w.codes, w.scales).cpu() for w in (w_up, w_down))
        v = mxfp4.values(*mxfp4.quant(x))
        for s in range(S):
            for k, e in enumerate(idx[s].tolist()):
                u = (up[e] @ v[s]).to(BF16).to(F64)
                h = u[:F] / (1 + torch.exp(-u[:F])) * u[F:]
                h = mxfp4.values(*mxfp4.quant(h[None]))[0]
                out[s] += float(topk_w[s, k]) * (down[e] @ h).to(BF16).to(F64)
        return out

    x = xs[0].clone()
    layer(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x)
    for v in xs:
        x.copy_(v)
        graph.replay()
        want = plain(v)
        # a value next to a border may take the other code: a step of a third of one of
        # 160 products at most, in few of them
        off = (out.cpu().to(F64) - want).norm() / want.norm()
        assert off < 2e-3, float(off)
        assert torch.equal(out, layer(v))
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for i in range(6):
        streams[i % 2].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(streams[i % 2]):
            outs.append(layer(xs[i % 3]))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, layer(xs[i % 3]))
    assert moe.moe_device_errors() == 0


def test_rows_of_a_buffer():
    """A buffer's rows are a multiple of four; one that is not is refused."""
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([3, 2])
    x, w = operand((6, 64), 1), operand((2, 64, 64), 2)
    with pytest.raises(moe.MoeError):
        moe.moe_expert_gemm_mxfp4(x, w, plan)
    x = operand((8, 64), 1)
    want = reference(x, w, plan).to(F32)
    assert torch.equal(moe.moe_expert_gemm_mxfp4(x, w, plan, out_dtype=F32), want)
    assert (want[5:] == 0).all()
