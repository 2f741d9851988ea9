"""The few-token layer against the bounds that its header states, in 64 bits.

Of each projection: sums in f32 with the tensor core's truncation, (n / 16 + 16) 2^-23 of
the sum of the magnitudes of its n products; with MXFP4 weights x and h are off by 2^-23 of
the largest of 32 neighbours or by 2^-129, whichever is more; with bf16 weights x is exact and h
keeps 24 bits, for outputs of either type.  silu adds 2^-20 of itself and 1.1 of its input's
error, the sum over k and the experts' weights 2^-22 of each term, the output its rounding."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

from tests import mxfp4  # noqa: E402
from tests.test_expert_layer_gpu import make  # noqa: E402

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def held(v, mx):
    """The error of rows v as they enter a product."""
    if not mx:
        return 2.0 ** -24 * v.abs()
    top = v.abs().unflatten(-1, (-1, 32)).amax(-1).repeat_interleave(32, -1)
    return (2.0 ** -23 * top).clamp(min=2.0 ** -129)


def reference(x, idx, w, up, down):
    """(out, bound before the last rounding)"""
    mx = not isinstance(up, torch.Tensor)
    f = (lambda q, e: mxfp4.values(q.codes[e], q.scales[e])) if mx else (lambda q, e: q[e].to(F64))
    E, F = up.shape[0], up.shape[1] // 2
    step = lambda n: (n / 16 + 16) * 2.0 ** -23  # noqa: E731
    out = torch.zeros(x.shape, dtype=F64, device="cuda")
    bound = torch.zeros_like(out)
    for e in idx.unique().tolist():
        if not 0 <= e < E:
            continue
        s, k = (idx == e).nonzero(as_tuple=True)
        v, wu, wd = x[s].to(F64), f(up, e), f(down, e)
        p = v @ wu.T
        off = step(v.shape[1]) * (v.abs() @ wu.abs().T) + (held(v, True) @ wu.abs().T if mx else 0)
        gate, lift = p[:, :F], p[:, F:]
        act = gate / (1 + torch.exp(-gate))
        h = act * lift
        d = (1.1 * off[:, :F] + 2.0 ** -20 * act.abs()) * (lift.abs() + off[:, F:]) + act.abs() * off[:, F:]
        d = d + step(F) * h.abs() + held(h.abs() + d, mx)
        c = w[s, k].to(F64)[:, None]
        out.index_add_(0, s, c * (h @ wd.T))
        bound.index_add_(0, s, c.abs() * (d @ wd.abs().T) + 2.0 ** -22 * (c * (h @ wd.T)).abs())
    return out, bound


def check(args):
    import combine_moe_plan_02_gb300 as moe
    want, bound = reference(*args)
    assert torch.isfinite(bound).all() and float(want.abs().max()) > 1e-30
    for dtype, eps in ((BF16, 2.0 ** -8), (F32, 2.0 ** -24)):
        out = moe.moe_expert_layer(*args, out_dtype=dtype)
        off = (out.to(F64) - want).abs()
        worst = float((off / (bound + eps * want.abs() + 1e-300)).max())
        assert worst <= 1, (dtype, worst)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("S,E,K,H,F", [(1, 8, 2, 64, 32), (5, 24, 3, 1440, 544), (16, 256, 8, 2048, 512),
                                       (64, 8, 8, 544, 128), (3, 4, 2, 256, 4096)])
def test_sizes(S, E, K, H, F, mx):
    check(make(S, E, K, H, F, mx, S + H))


def scaled(q, power):
    """MXFP4 weights times 2^power."""
    import combine_moe_plan_02_gb300 as moe
    scales = torch.where(q.scales > 0, q.scales.int() + power, 0)
    assert int(scales.max()) < 255
    return moe.MxFp4(q.codes, scales.to(torch.uint8))


@pytest.mark.parametrize("H", [64, 512])
def test_rows_near_the_last_scale(H):
    """x of 2^-100 .. 2^-126, a size a token, on weights that bring its sums back."""
    x, idx, w, up, down = make(14, 4, 2, H, 96, True, 7, low=0)
    x = (x.float() * torch.exp2(-100 - 2.0 * torch.arange(14, device="cuda"))[:, None]).to(BF16)
    check((x, idx, w, scaled(up, 100), down))


def test_hidden_rows_near_the_last_scale():
    """h of 2^-100 .. 2^-126: projections of 2^-50 .. 2^-63."""
    x, idx, w, up, down = make(14, 4, 2, 256, 160, True, 8, low=0)
    x = (x.float() * torch.exp2(-50.0 - torch.arange(14, device="cuda"))[:, None]).to(BF16)
    check((x, idx, w, up, scaled(down, 100)))


def one_hot(rows, columns, value):
    """[1, len(columns), rows] weights: row f takes element columns[f] times value."""
    import combine_moe_plan_02_gb300 as moe
    w = torch.zeros(1, len(columns), rows, device="cuda")
    w[0, torch.arange(len(columns)), torch.tensor(columns)] = value
    return moe.moe_quant_mxfp4(w)


@pytest.mark.parametrize("hidden", [False, True])
def test_each_value_near_the_last_scale(hidden):
    """Each element by itself, so that no sum hides its error: gate f is x[f], the lifts are the
    first and largest one, and the outputs are h."""
    g = torch.Generator(device="cuda").manual_seed(9)
    S, n = 28, 32
    x = torch.rand(S, n, generator=g, device="cuda") + 0.01
    x[:, 0] = 1.0
    low, step = (-50.0, 0.5) if hidden else (-100.0, 1.0)
    x = (x * torch.exp2(low - step * torch.arange(S, device="cuda"))[:, None]).to(BF16)
    up = one_hot(n, list(range(n)) + [0] * n, 1.0 if hidden else 2.0 ** 100)
    down = one_hot(n, list(range(n)), 2.0 ** 100 if hidden else 1.0)
    idx, w = torch.zeros(S, 1, dtype=torch.int32, device="cuda"), torch.ones(S, 1, device="cuda")
    check((x, idx, w, up, down))


def small_steps(n):
    """[n / 64 terms of a row]: 1, then 0.75 of f32's last place at 1 in each step of 64
    elements, and their sum.  Cut off at each step, the sum stays 1."""
    row = torch.zeros(n)
    row[0], row[64::64] = 1.0, 0.75 * 2.0 ** -23
    return row, 1 + (n // 64 - 1) * 0.75 * 2.0 ** -23


# An accumulator of at most 16 steps is cut off by a last place in each; the parts are added
# in f32, half a place each.
def lost_at_most(n):
    return (16 + n / 1024 / 2 + 1) * 2.0 ** -23


@pytest.mark.parametrize("n", [1024, 6144, 16384])
@pytest.mark.parametrize("first", [True, False])
def test_small_terms_of_long_sums(first, n):
    """f32 outputs on MXFP4 weights: gates of 64, which silu leaves as they are, lifts of 1 / 64 of
    the sum in the first product, or of 1 / 64 and the sum in the second."""
    import combine_moe_plan_02_gb300 as moe
    row, want = small_steps(n)
    H, F = (n, 32) if first else (32, n)
    up, down = torch.zeros(1, 2 * F, H, device="cuda"), torch.zeros(1, H, F, device="cuda")
    up[0, :F, 0] = 64.0
    if first:
        up[0, F:] = row.cuda() / 64
        down[0, torch.arange(F), torch.arange(F)] = 1.0
    else:
        up[0, F:, 0] = 1 / 64
        down[0] = row.cuda()
    x = torch.ones(2, H, dtype=BF16, device="cuda")
    idx, w = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), torch.ones(2, 1, device="cuda")
    out = moe.moe_expert_layer(x, idx, w, moe.moe_quant_mxfp4(up), moe.moe_quant_mxfp4(down), out_dtype=F32)
    off = (out[:, :32].to(F64) - want).abs().max()
    assert float(off) <= lost_at_most(n), (float(off) * 2 ** 23, (want - 1) * 2 ** 23)
