"""f32 outputs of the MXFP4 product over long reductions whose terms are of different sizes.

An accumulator takes 64 elements a step and cuts off what lies below its last place; f32
outputs have one for 4096 elements, 64 steps, and the parts are added in f32.  So off by at most
64 last places of an accumulator and half a one for each part."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

from tests import mxfp4  # noqa: E402
from tests.test_expert_gemm_gpu import make_plan  # noqa: E402

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def reference(x, w, plan, absolute=False):
    f = torch.abs if absolute else (lambda t: t)
    out = torch.zeros(x.shape[0], w.shape[1], dtype=F64, device="cuda")
    for e, (o, c) in enumerate(zip(plan.off.tolist(), plan.cnt.tolist())):
        rows = mxfp4.values(x.codes[o:o + c], x.scales[:, o:o + c].contiguous())
        out[o:o + c] = f(rows) @ f(mxfp4.values(w.codes[e], w.scales[e])).T
    return out


def lost_at_most(D):
    return (64 + D / 4096 / 2 + 1) * 2.0 ** -23


@pytest.mark.parametrize("counts", [[4], [100, 28], [256, 0, 300]])
@pytest.mark.parametrize("D", [4096, 4128, 6144, 20512, 32768])
def test_small_terms(D, counts):
    """1, then 0.75 of f32's last place at 1 in every step of 64 elements: cut off at each
    step the sum would stay 1."""
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan(counts)
    E, N = len(counts), 264
    w = torch.zeros(E, N, D, device="cuda")
    w[..., 0], w[..., 64::64] = 1.0, 0.75 * 2.0 ** -23
    want = 1 + len(range(64, D, 64)) * 0.75 * 2.0 ** -23
    y = moe.moe_expert_gemm_mxfp4(moe.moe_quant_mxfp4(torch.ones(rows, D, device="cuda")),
                                  moe.moe_quant_mxfp4(w), plan, out_dtype=F32)
    off = float((y.to(F64) - want).abs().max())
    assert off <= lost_at_most(D), (off * 2 ** 23, (want - 1) * 2 ** 23)


@pytest.mark.parametrize("D", [4096, 4352, 7168, 32768])
@pytest.mark.parametrize("spread", [0, 8, 20])
def test_scales_apart(spread, D):
    """Random codes under scales 2^0 .. 2^-spread on either side, wide and narrow tiles, all
    starts in a group of four rows; relative to the sum of the magnitudes."""
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([3, 130, 1, 70, 0, 259], 0, 1)
    x = moe.MxFp4(*mxfp4.random((rows, D), D + spread, low=127 - spread, high=127))
    w = moe.MxFp4(*mxfp4.random((6, 136, D), D + 1, low=127 - spread, high=127))
    want, most = reference(x, w, plan), reference(x, w, plan, True)
    for dtype, eps in ((F32, 2.0 ** -24), (BF16, 2.0 ** -8)):
        y = torch.full((rows, 136), float("nan"), dtype=dtype, device="cuda")
        moe.moe_expert_gemm_mxfp4(x, w, plan, out=y)
        steps = lost_at_most(D) if dtype is F32 else (D / 64 + 1) * 2.0 ** -23
        assert ((y.to(F64) - want).abs() <= steps * most + eps * want.abs()).all()
        assert (y[-1] == 0).all()
    assert moe.moe_device_errors() == 0


def test_reproducible_in_a_graph_and_on_streams():
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([40, 300, 7, 129, 4])
    D, N = 6176, 520
    x = moe.MxFp4(*mxfp4.random((rows, D), 1, low=110))
    w = moe.MxFp4(*mxfp4.random((5, N, D), 2, low=110))
    first = moe.moe_expert_gemm_mxfp4(x, w, plan, out_dtype=F32)
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            moe.moe_expert_gemm_mxfp4(x, w, plan, out=out)
    for _ in range(5):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            outs.append(moe.moe_expert_gemm_mxfp4(x, w, plan, out_dtype=F32))
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)
    assert moe.moe_device_errors() == 0
