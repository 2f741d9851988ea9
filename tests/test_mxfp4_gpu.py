"""MXFP4 quantisation and its inverse: bit for bit the definition in 64 bits.

Scaling by a power of two is exact, so codes and scales have one right value,
whatever the order of the work.  The gated activation rounds in f32 first: its
scale and code may be those of any value within 2^-16 of the 64-bit one (the
fast exponential and division for gates above -60)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

from tests import mxfp4  # noqa: E402

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def same(q, want):
    codes, scales = want
    assert torch.equal(q.scales.cpu(), scales)
    assert torch.equal(q.codes.cpu(), codes)


def spread(shape, seed, dtype, low=-20, high=20):
    """Normal values, each block of 32 of another size."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    e = torch.randint(low, high + 1, (*shape[:-1], shape[-1] // 32), generator=g, device="cuda")
    return (x * torch.pow(2.0, e.float()).repeat_interleave(32, -1)).to(dtype)


def poisoned(rows, D, device="cuda"):
    import combine_moe_plan_02_gb300 as moe
    return moe.MxFp4(torch.full((rows, D // 2), 0x5a, dtype=torch.uint8, device=device),
                     torch.full((-(-D // 128), rows, 4), 0x5a, dtype=torch.uint8, device=device))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (5, 96), (7, 160), (2, 512), (3, 544),
                                   (33, 1440), (4, 7168), (3, 5, 224), (2, 8, 4096), (1, 1, 32)])
def test_quant(shape, dtype):
    import combine_moe_plan_02_gb300 as moe
    x = spread(shape, len(shape) + shape[-1], dtype)
    q = moe.moe_quant_mxfp4(x)
    assert q.shape == x.shape
    same(q, mxfp4.quant(x))
    back = mxfp4.values(q.codes, q.scales)
    for out in (F32, BF16):
        assert torch.equal(moe.moe_dequant_mxfp4(q, out_dtype=out).to(F64), back)
    # half a step of the scale: at most 2 of 8 by rounding, or 2 by saturation
    top = x.to(F64).abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
    assert ((back - x.to(F64)).abs() <= top / 4).all()


def test_every_bf16_value_and_every_border():
    """All finite bf16 values under block maxima of every size, and in f32 every
    border between two codes with its neighbours."""
    import combine_moe_plan_02_gb300 as moe
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16).view(BF16)
    x = bits[torch.isfinite(bits.float())]
    x = torch.cat([x, x.flip(0)])
    n = x.numel() // 31 * 31
    x = x[:n].view(-1, 31)
    for shift in (1, 8, 200):   # each value beside a maximum of its own size and far larger ones
        lead = torch.roll(x[:, :1], shift, 0)
        y = torch.cat([lead, x], 1).contiguous().cuda()
        same(moe.moe_quant_mxfp4(y), mxfp4.quant(y))
    borders = torch.tensor([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, 7.9])
    ends = torch.nextafter(borders, torch.zeros(())), borders, torch.nextafter(borders, torch.full((), 9.0))
    v = torch.cat(ends)
    rows = []
    for e in (-149, -140, -130, -126, -125, -60, 0, 1, 60, 120, 124):
        for sign in (1.0, -1.0):
            row = torch.zeros(64, dtype=F64)
            row[0], row[32] = 4.0, 7.75
            row[1:32] = v[:31] * sign
            row[33:33 + v.numel() - 31] = v[31:] * sign
            rows.append((row * 2.0 ** e).float())
    y = torch.stack(rows).cuda()
    same(moe.moe_quant_mxfp4(y), mxfp4.quant(y))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_zeros_infinities_and_nan(dtype):
    import combine_moe_plan_02_gb300 as moe
    x = spread((6, 256), 3, dtype)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 70] = float("nan")
    x[3, 128:160] = -0.0
    x[4, 200] = -float("inf")
    x[5, 0], x[5, 1] = float("nan"), float("inf")
    q = moe.moe_quant_mxfp4(x)
    same(q, mxfp4.quant(x))
    back = moe.moe_dequant_mxfp4(q)
    bad = (~torch.isfinite(x)).unflatten(-1, (-1, 32)).any(-1).repeat_interleave(32, -1)
    assert torch.equal(back.isnan(), bad)
    # every scale byte, against the definition
    codes = torch.arange(256, dtype=torch.uint8).repeat(16, 1).repeat(1, 2).view(16, 512).cuda()
    scales = torch.arange(256, dtype=torch.uint8).view(16, 16)
    scales = scales.repeat(1, 2).view(16, 8, 4).transpose(0, 1).contiguous().cuda()
    q = moe.MxFp4(codes, scales)
    want = mxfp4.values(codes, scales).to(F32)
    got = moe.moe_dequant_mxfp4(q, out_dtype=F32)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))


@pytest.mark.parametrize("S,D,E,K", [(1, 32, 4, 1), (3, 96, 5, 3), (17, 544, 8, 8), (130, 1440, 16, 2),
                                     (5, 7168, 40, 32), (300, 256, 64, 8)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_dispatch(S, D, E, K, dtype):
    import combine_moe_plan_02_gb300 as moe
    g = torch.Generator().manual_seed(S)
    idx = torch.randint(-1, E, (S, K), generator=g).to(torch.int32).cuda()   # repeats and none
    x = spread((S, D), S + D, dtype)
    codes, scales = mxfp4.quant(x)
    for plan, rows in ((moe.moe_plan(idx, E), -(-S * K // 4) * 4), (moe.moe_plan_capacity(idx, E, 3), E * 3)):
        out = poisoned(rows, D)
        assert moe.moe_dispatch_quant_mxfp4(x, plan.tok_map, out=out) is out
        want = poisoned(rows, D, "cpu")
        for s, row in enumerate(plan.tok_map.tolist()):
            for r in row:
                if r >= 0:
                    want.codes[r] = codes[s]
                    want.scales[:, r] = scales[:, s]
        same(out, want)
    plan = moe.moe_plan(idx, E)
    assert moe.moe_dispatch_quant_mxfp4(x, plan.tok_map).shape == (max(-(-S * K // 4) * 4, 4), D)
    assert moe.moe_device_errors() == 0


def test_dispatch_bad_rows():
    """Entries outside the packed rows are skipped and reported, the others stored."""
    import combine_moe_plan_02_gb300 as moe
    x = spread((3, 64), 1, BF16)
    tok_map = torch.tensor([[0, 4], [-1, 2], [3, -7]], device="cuda")
    out = poisoned(4, 64)
    moe.moe_dispatch_quant_mxfp4(x, tok_map, out=out)
    assert moe.moe_device_errors() == 2
    codes, _ = mxfp4.quant(x)
    assert torch.equal(out.codes[[0, 2, 3]].cpu(), codes)
    assert (out.codes[1] == 0x5a).all()


def swiglu_64(u):
    gate, up = u.to(F64).chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,F", [(1, 32), (3, 96), (9, 544), (40, 2048), (130, 1440)])
def test_swiglu(rows, F, dtype):
    import combine_moe_plan_02_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(F)
    u = (torch.randn(rows, 2 * F, generator=g, device="cuda") * 3).to(dtype)
    u[0, ::3] = -40.0
    q = moe.moe_swiglu_quant_mxfp4(u)
    h = swiglu_64(u)
    got = mxfp4.values(q.codes, q.scales)
    # monotone in the value for a given scale: between the codes of the two ends
    near = 2.0 ** -16
    top = h.abs().unflatten(-1, (-1, 32)).amax(-1)
    scale = mxfp4.power(q.scales.transpose(0, 1).flatten(1)[:, :F // 32].to(torch.int64) - 127)
    assert (top * (1 - near) < scale * 8).all() and (top * (1 + near) >= scale * 4).all()
    unit = scale.repeat_interleave(32, -1)
    magnitudes = mxfp4.MAGNITUDES.cuda()
    middle = (magnitudes[1:] + magnitudes[:-1]) / 2
    low = magnitudes[torch.searchsorted(middle, (h.abs() * (1 - near) / unit).contiguous())]
    high = magnitudes[torch.searchsorted(middle, (h.abs() * (1 + near) / unit).contiguous(), right=True)]
    assert (got.abs() >= low * unit).all() and (got.abs() <= high * unit).all()
    assert (torch.sign(got) * torch.sign(h) >= 0).all()


def test_swiglu_extremes():
    import combine_moe_plan_02_gb300 as moe
    u = torch.zeros(4, 128, device="cuda")
    u[0, :32], u[0, 64:96] = 100.0, 1.0            # gate as it is
    u[1, :32], u[1, 64:96] = -200.0, 1.0           # nothing is left
    u[2, 3], u[2, 67] = float("nan"), 1.0
    u[3, 40], u[3, 104] = float("inf"), 2.0
    q = moe.moe_swiglu_quant_mxfp4(u)
    v = moe.moe_dequant_mxfp4(q, out_dtype=F32)
    assert (v[0, :32] == 96.0).all() and (v[0, 32:] == 0).all()   # 100 = 6.25 * 16
    assert (v[1] == 0).all()
    assert v[2, :32].isnan().all() and (v[2, 32:] == 0).all()
    assert v[3, 32:].isnan().all() and (v[3, :32] == 0).all()


def test_strided_offset_and_large():
    """Rows that begin inside a larger tensor, and tensors past 2^31 bytes and elements."""
    import combine_moe_plan_02_gb300 as moe
    base = spread((9, 256), 2, BF16)
    same(moe.moe_quant_mxfp4(base[2:7]), mxfp4.quant(base[2:7]))
    with pytest.raises(ValueError):
        moe.moe_quant_mxfp4(base[:, :128])
    with pytest.raises(moe.MoeError):   # rows that do not begin on 16 bytes
        moe.moe_quant_mxfp4(base.flatten()[4:4 + 512].view(2, 256))
    rows, D = 70001, 32768
    x = torch.zeros(rows, D, dtype=BF16, device="cuda")
    x[-1] = spread((1, D), 5, BF16)
    x[rows // 2] = x[-1]
    q = moe.moe_quant_mxfp4(x)
    want = mxfp4.quant(x[-1:])
    for r in (rows - 1, rows // 2):
        assert torch.equal(q.codes[r].cpu(), want[0][0])
        assert torch.equal(q.scales[:, r].cpu(), want[1][:, 0])
    assert int(torch.count_nonzero(q.codes[:rows // 2]) + torch.count_nonzero(q.codes[rows // 2 + 1:-1])) == 0
    x.fill_(1.0)
    back = moe.moe_dequant_mxfp4(q, out=x)
    assert torch.equal(back[-1].to(F64).cpu(), mxfp4.values(*want)[0])
    assert int(torch.count_nonzero(back[:rows // 2])) == 0


def test_empty():
    import combine_moe_plan_02_gb300 as moe
    q = moe.moe_quant_mxfp4(torch.empty(0, 64, dtype=BF16, device="cuda"))
    assert q.shape == (0, 64) and moe.moe_dequant_mxfp4(q).shape == (0, 64)
    assert moe.moe_swiglu_quant_mxfp4(torch.empty(0, 128, dtype=BF16, device="cuda")).shape == (0, 64)
    out = poisoned(4, 64)
    moe.moe_dispatch_quant_mxfp4(torch.empty(0, 64, dtype=BF16, device="cuda"),
                                 torch.empty(0, 2, dtype=torch.int64, device="cuda"), out=out)
    assert (out.codes == 0x5a).all()


def test_graph_and_streams():
    import combine_moe_plan_02_gb300 as moe
    xs = [spread((64, 512), i, BF16) for i in range(3)]
    x, u = xs[0].clone(), torch.cat([xs[1], xs[2]], 1)
    tok_map = torch.arange(128, device="cuda").view(64, 2)
    out = poisoned(128, 512)
    act = poisoned(64, 512)
    back = torch.empty(128, 512, dtype=BF16, device="cuda")

    def step():
        moe.moe_dispatch_quant_mxfp4(x, tok_map, out=out)
        moe.moe_dequant_mxfp4(out, out=back)
        moe.moe_swiglu_quant_mxfp4(u, out=act)
    step()
    torch.cuda.synchronize()
    first = act.codes.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for v in xs:
        x.copy_(v)
        graph.replay()
        q = moe.moe_quant_mxfp4(v)
        assert torch.equal(out.codes[::2], q.codes) and torch.equal(out.codes[1::2], q.codes)
        assert torch.equal(back[::2].to(F64), mxfp4.values(q.codes, q.scales))
        assert torch.equal(act.codes, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = [moe.moe_quant_mxfp4(v) for v in xs]
    b = [moe.moe_quant_mxfp4(v, stream=side) for v in xs]
    torch.cuda.synchronize()
    for p, q, v in zip(a, b, xs):
        same(p, mxfp4.quant(v))
        same(q, mxfp4.quant(v))
