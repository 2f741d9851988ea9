"""The gated activation for gates far below zero, where exp(-gate) nears f32's end and
large ups bring the product back into range.

h = gate / (1 + exp(-gate)) * up in 64 bits.  The kernel's h is off by at most 2^-16 of it
(its fast exponential at -80, and below -174 the halves of the exponential as subnormals of
17 bits and more, wherever h is above half of the smallest code), and by half of f32's
smallest step, 2^-150.  So each code lies between those of the two ends, under the scale that the block's largest
magnitude sets."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

from tests import mxfp4  # noqa: E402

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
NEAR, STEP = 2.0 ** -16, 2.0 ** -150


def check(u):
    import combine_moe_plan_02_gb300 as moe
    q = moe.moe_swiglu_quant_mxfp4(u)
    rows, F = q.shape
    gate, up = u.to(F64).chunk(2, -1)
    h = gate / (1 + torch.exp(-gate)) * up
    ends = [(h.abs() * (1 - NEAR) - STEP).clamp(min=0), h.abs() * (1 + NEAR) + STEP]
    byte = q.scales.transpose(0, 1).flatten(1)[:, :F // 32].to(torch.int64)
    scale = mxfp4.power(byte - 127)
    low, high = (v.unflatten(-1, (-1, 32)).amax(-1) for v in ends)
    assert (low < scale * 8).all() and ((high >= scale * 4) | (byte == 0)).all()
    unit = scale.repeat_interleave(32, -1)
    magnitudes = mxfp4.MAGNITUDES.cuda()
    middle = (magnitudes[1:] + magnitudes[:-1]) / 2
    code = [magnitudes[torch.searchsorted(middle, (v / unit).contiguous(), right=bool(i))] * unit
            for i, v in enumerate(ends)]
    got = mxfp4.values(q.codes, q.scales)
    assert (got.abs() >= code[0]).all() and (got.abs() <= code[1]).all()
    assert (torch.sign(got) * torch.sign(h) >= 0).all()
    return got, h


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("low,high", [(-88.72, -87.34), (-89.5, -79.5), (-104.0, -80.0), (-184.0, -100.0)])
@pytest.mark.parametrize("size", [(0, 10), (60, 126)])
def test_far_gates(low, high, size, dtype):
    """Every gate of a block there, ups of one block from 2^size."""
    g = torch.Generator(device="cuda").manual_seed(int(-10 * low) + size[0])
    rows, F = 33, 544
    u = torch.randn(rows, 2 * F, generator=g, device="cuda")
    u[:, :F] = low + (high - low) * torch.rand(rows, F, generator=g, device="cuda")
    e = size[0] + (size[1] - size[0]) * torch.rand(rows, F // 32, generator=g, device="cuda")
    u[:, F:] = u[:, F:].clamp(-2, 2) * torch.exp2(e).repeat_interleave(32, -1)
    got, h = check(u.to(dtype))
    if size[1] > 100 and low > -110:
        assert (got.unflatten(-1, (-1, 32)).abs().amax(-1) > 0).all()   # no block is lost


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_among_ordinary_gates(dtype):
    """A few far gates, whose ups make them their block's largest, beside ordinary ones."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, F = 64, 2048
    u = torch.randn(rows, 2 * F, generator=g, device="cuda") * 3
    at = torch.rand(rows, F, generator=g, device="cuda") < 0.01
    u[:, :F][at] = -80 - 8.7 * torch.rand(int(at.sum()), generator=g, device="cuda")
    u[:, F:][at] *= 2.0 ** 116
    check(u.to(dtype))


def test_one_value():
    """gate -88 and up 1e37: -88 exp(-88) 1e37 = -5.33, held as -6 (4, 6 are the codes around it)."""
    import combine_moe_plan_02_gb300 as moe
    u = torch.full((1, 64), -88.0, device="cuda")
    u[:, 32:] = 1e37
    v = moe.moe_dequant_mxfp4(moe.moe_swiglu_quant_mxfp4(u), out_dtype=F32)
    assert (v == -6).all()
