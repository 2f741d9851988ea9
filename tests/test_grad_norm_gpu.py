"""The global gradient norm and clipping against sums in 64 bits.

A value passes through at most 64 f32 additions at these sizes (a thread's sum,
then lanes, warps and CTAs), each off by 2^-24 of the sum, all terms positive,
so the norm is off by at most 64 * 2^-24 of itself; a clipped value
by that, four f32 roundings, and 2^-8 of it for bf16.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
NORM = 64 * 2.0 ** -24


def grads(sizes, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(t) for n, t in sizes]


def norm64(gs):
    return math.sqrt(sum(float(g.to(F64).square().sum()) for g in gs))


def check_out(gs, out, max_norm):
    norm = norm64(gs)
    c = min(1.0, max_norm / (norm + 1e-6))
    for g, o in zip(gs, out):
        assert o.dtype == g.dtype and o.shape == g.shape
        want = g.to(F64) * c
        off = (NORM + 2.0 ** -22 + (2.0 ** -8 if g.dtype == BF16 else 0.0)) * want.abs()
        assert ((o.to(F64) - want).abs() <= off + (1e-40 if g.dtype == BF16 else 0)).all()


SIZES = [
    [(1, F32)],
    [(1, BF16)],
    [(0, F32), (7, BF16), (0, BF16), (9, F32)],
    [(8192, F32), (8193, F32), (16384, BF16), (16385, BF16), (8191, F32)],
    [(1000003, F32), (1, BF16), (77777, BF16), (3, F32)],
    [(i * 37 + 1, F32 if i % 3 else BF16) for i in range(64)],
    [(i * 5, F32 if i % 2 else BF16) for i in range(700)],     # more than one table
]


@pytest.mark.parametrize("sizes", range(len(SIZES)))
@pytest.mark.parametrize("part", [0.25, 4.0])
def test_norm_and_clip(sizes, part):
    import combine_moe_plan_02_gb300 as moe
    gs = grads(SIZES[sizes], seed=sizes)
    norm = norm64(gs)
    got = moe.moe_grad_norm(gs)
    assert abs(float(got) - norm) <= NORM * norm
    out = [torch.full_like(g, float("nan")) for g in gs]
    kept = [g.clone() for g in gs]
    got = moe.moe_clip_grad_norm(gs, part * norm, out=out)
    assert abs(float(got) - norm) <= NORM * norm
    check_out(gs, out, part * norm)
    assert all(torch.equal(a, b) for a, b in zip(gs, kept))
    got2 = moe.moe_clip_grad_norm(gs, part * norm)       # in place
    assert torch.equal(got, got2)
    assert all(torch.equal(a, b) for a, b in zip(gs, out))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("a,b", [(0, 0), (1, 1), (3, 1), (0, 5), (7, 7)])
def test_any_alignment(dtype, a, b):
    import combine_moe_plan_02_gb300 as moe
    n = 50021
    base = grads([(n + 8, dtype)])[0]
    gs = [base[a:a + n], base[:5]]
    room = torch.full((n + 8,), 3.0, dtype=dtype, device="cuda")
    out = [room[b:b + n], torch.empty(5, dtype=dtype, device="cuda")]
    moe.moe_clip_grad_norm(gs, 1.0, out=out)
    check_out(gs, out, 1.0)
    assert (room[:b] == 3).all() and (room[b + n:] == 3).all()


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinities_and_nan(value, dtype):
    import combine_moe_plan_02_gb300 as moe
    gs = grads([(1000, dtype), (30, F32)])
    gs[0][999] = value
    norm = moe.moe_clip_grad_norm(gs, 1.0)
    if math.isnan(value):
        assert torch.isnan(norm).all() and all(torch.isnan(g).all() for g in gs)
    else:
        assert torch.isinf(norm).all() and torch.isnan(gs[0][999])
        assert not gs[0][:999].any() and not gs[1].any()


def test_limits():
    import combine_moe_plan_02_gb300 as moe
    gs = grads([(100, F32), (100, BF16)])
    kept = [g.clone() for g in gs]
    moe.moe_clip_grad_norm(gs, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(gs, kept))
    moe.moe_clip_grad_norm(gs, 0.0)
    assert not any(g.any() for g in gs)
    assert float(moe.moe_clip_grad_norm(gs, 1.0)) == 0.0      # the norm of zeros
    assert not any(g.any() for g in gs)
    assert float(moe.moe_grad_norm([torch.empty(0, device="cuda")])) == 0.0


def test_more_than_32_bit_offsets():
    import combine_moe_plan_02_gb300 as moe
    n = (1 << 31) + 12345                                     # bf16: 4 GiB
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-1], g[7], g[1 << 30] = 3.0, 4.0, 12.0
    norm = moe.moe_clip_grad_norm([g], 6.5)
    assert abs(float(norm) - 13.0) <= NORM * 13
    got = g[torch.tensor([7, 1 << 30, n - 1], device="cuda")].tolist()
    assert got == [2.0, 6.0, 1.5] and int((g != 0).sum()) == 3


def test_side_stream_and_graph():
    import combine_moe_plan_02_gb300 as moe
    gs = grads([(200001, F32), (333, BF16)])
    out = [torch.empty_like(g) for g in gs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    moe.moe_clip_grad_norm(gs, 1.0, out=out, stream=side)
    side.synchronize()
    check_out(gs, out, 1.0)
    norm = torch.empty(1, device="cuda")
    ws = torch.empty(65536, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_clip_grad_norm(gs, 1.0, out=out, norm=norm, workspace=ws)
    for s in (5, 6):
        for g, new in zip(gs, grads([(200001, F32), (333, BF16)], seed=s)):
            g.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        check_out(gs, out, 1.0)


@pytest.mark.parametrize("raw", [False, True])
def test_calls_that_overlap_on_two_streams(raw):
    """A call on the current stream and one on another, with no wait between:
    neither may use the other's partial sums, and neither norm's memory may be
    one that earlier work of the current stream still writes."""
    import combine_moe_plan_02_gb300 as moe
    big, small = grads([(60_000_000, F32)], seed=1), grads([(300_001, F32), (7, BF16)], seed=2)
    out = [[torch.empty_like(g) for g in gs] for gs in (big, small)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        for n in (1, 16384):                       # freed while the fills below are pending
            for t in [torch.empty(n, device="cuda") for _ in range(4)]:
                moe.moe_clip_grad_norm(big, 1.0, out=out[0])
                t.fill_(float("nan"))
        del t
        a = moe.moe_clip_grad_norm(big, 1.0, out=out[0])
        b = moe.moe_clip_grad_norm(small, 1.0, out=out[1],
                                   stream=side.cuda_stream if raw else side)
        c = moe.moe_grad_norm(small, stream=side)
        torch.cuda.synchronize()
        assert abs(float(a) - norm64(big)) <= 2 * NORM * norm64(big)  # at most 128 additions
        for t in (b, c):
            assert abs(float(t) - norm64(small)) <= NORM * norm64(small)
        check_out(small, out[1], 1.0)


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_an_infinite_limit_scales_nothing(value, dtype):
    import combine_moe_plan_02_gb300 as moe
    gs = grads([(1000, dtype), (30, F32)])
    gs[0][7] = value
    out = [torch.full_like(g, 3.0) for g in gs]
    norm = moe.moe_clip_grad_norm(gs, float("inf"), out=out)
    assert not torch.isfinite(norm).any()
    assert all(torch.equal(torch.nan_to_num(g, nan=9.0), torch.nan_to_num(o, nan=9.0))
               for g, o in zip(gs, out))
    kept = [g.clone() for g in gs]
    moe.moe_clip_grad_norm(gs, float("inf"))
    assert all(torch.equal(torch.nan_to_num(g, nan=9.0), torch.nan_to_num(o, nan=9.0))
               for g, o in zip(gs, kept))
