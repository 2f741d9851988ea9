"""The few-token layer where exp(-gate) is beyond f32 and the lift brings h back.

Gates and lifts are exact here (one element each), h = silu(gate) * lift is off by 2^-20 and
enters the second product with 2^-23 of itself, the output is h: 2^-19 in all."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("low,high", [(-88.5, -60.0), (-104.0, -88.5), (-160.0, -80.0)])
def test_far_gates(low, high, mx):
    import combine_moe_plan_02_gb300 as moe
    S, H, F = 96, 64, 32
    gate = torch.linspace(low, high, S, device="cuda").to(BF16)
    x = torch.zeros(S, H, dtype=BF16, device="cuda")
    x[:, 0], x[:, 32] = gate, 1.0
    up, down = torch.zeros(1, 2 * F, H, device="cuda"), torch.zeros(1, H, F, device="cuda")
    lift = torch.exp2(126.0 - torch.arange(F, device="cuda") % 8)
    up[0, :F, 0], up[0, F:, 32] = 1.0, lift
    down[0, torch.arange(F), torch.arange(F)] = 1.0
    weights = (moe.moe_quant_mxfp4(up), moe.moe_quant_mxfp4(down)) if mx else (up.to(BF16), down.to(BF16))
    idx, w = torch.zeros(S, 1, dtype=torch.int32, device="cuda"), torch.ones(S, 1, device="cuda")
    out = moe.moe_expert_layer(x, idx, w, *weights, out_dtype=F32)[:, :F].to(F64)
    g = gate.to(F64)[:, None]
    want = g / (1 + torch.exp(-g)) * lift.to(F64)
    # of the largest of 32 neighbours, 2^7 of the smallest here
    off = 2.0 ** -19 * want.abs() + 2.0 ** -23 * want.abs().amax(1, keepdim=True)
    assert ((out - want).abs() <= off).all(), float(((out - want) / want).abs().max())


@pytest.mark.parametrize("mx", [False, True])
def test_infinite_and_nan_gates(mx):
    """An infinite gate gives what the formula gives: the lift times it, or NaN below zero (0 times
    infinity in the product), and a NaN stays one."""
    import combine_moe_plan_02_gb300 as moe
    x = torch.zeros(4, 32, dtype=BF16, device="cuda")
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = float("inf"), -float("inf"), float("nan"), -1000.0
    x[:, 1] = 1.0
    up, down = torch.zeros(1, 64, 32, device="cuda"), torch.ones(1, 32, 32, device="cuda")
    up[0, :32, 0], up[0, 32:, 1] = 1.0, 1.0
    weights = (moe.moe_quant_mxfp4(up), moe.moe_quant_mxfp4(down)) if mx else (up.to(BF16), down.to(BF16))
    idx, w = torch.zeros(4, 1, dtype=torch.int32, device="cuda"), torch.ones(4, 1, device="cuda")
    out = moe.moe_expert_layer(x, idx, w, *weights, out_dtype=F32)
    assert not torch.isfinite(out[:3]).any() and out[2].isnan().all()
    assert (out[3] == 0).all()
