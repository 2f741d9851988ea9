"""A bucket that begins outside the rows is left out and reported, and costs no other bucket
its output: starts below zero, past the rows, and so far out that start + count does not fit 64 bits.

The right outputs are those of the same plan with that bucket empty, bit for bit."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

from tests import mxfp4  # noqa: E402
from tests.test_expert_gemm_gpu import make_plan  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
LAST = (1 << 63) - 1
COUNTS, N, D = [8, 12, 5, 16, 3, 8], 72, 96
STARTS = [LAST, LAST - 2, LAST - (1 << 31), 1 << 40, 57, -1, -8, -LAST - 1]


def calls(rows, E):
    import combine_moe_plan_02_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(0)
    x, dy = (torch.randn(rows, n, generator=g, device="cuda").to(BF16) for n in (D, N))
    w = torch.randn(E, N, D, generator=g, device="cuda").to(BF16)
    q = moe.MxFp4(*mxfp4.random((rows, D), 1))
    qw = moe.MxFp4(*mxfp4.random((E, N, D), 2))

    def out(n, dtype):
        return torch.full((rows, n), float("nan"), dtype=dtype, device="cuda")
    return [lambda p: moe.moe_expert_gemm(x, w, p, out=out(N, BF16)),
            lambda p: moe.moe_expert_gemm(x, w, p, out=out(N, F32)),
            lambda p: moe.moe_expert_gemm_dgrad(dy, w, p, out=out(D, BF16)),
            lambda p: moe.moe_expert_gemm_wgrad(dy, x, p),
            lambda p: moe.moe_expert_gemm_mxfp4(q, qw, p, out=out(N, BF16)),
            lambda p: moe.moe_expert_gemm_mxfp4(q, qw, p, out=out(N, F32))]


@pytest.mark.parametrize("start", STARTS)
@pytest.mark.parametrize("bad", [1, 3, 5])
def test_other_buckets_keep_their_output(bad, start):
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan(COUNTS, 0, 4)
    assert rows == 56
    for i, call in enumerate(calls(rows, len(COUNTS))):
        empty = plan._replace(cnt=plan.cnt.clone())
        empty.cnt[bad] = 0
        want = call(empty)
        assert moe.moe_device_errors() == 0
        broken = plan._replace(off=plan.off.clone())
        broken.off[bad] = start
        for _ in range(3):
            got = call(broken)
            assert moe.moe_device_errors() == 32
            assert torch.equal(got, want), i


def test_several_and_the_first():
    """Buckets 0, 2 and 3; the rows before the first one that begins inside are in nobody's gap."""
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan(COUNTS, 0, 4)
    for i, call in enumerate(calls(rows, len(COUNTS))):
        empty = plan._replace(cnt=plan.cnt.clone())
        empty.cnt[[0, 2, 3]] = 0
        want = call(empty)
        broken = plan._replace(off=plan.off.clone())
        broken.off[0], broken.off[2], broken.off[3] = -3, LAST, 1 << 33
        got = call(broken)
        assert moe.moe_device_errors() == 32
        from_row = 8 if i != 3 else 0
        assert torch.equal(got[from_row:], want[from_row:]), i


def test_many_buckets():
    """300 buckets, every seventh of them outside."""
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([1 + i % 5 for i in range(300)], 0, 0)
    rows += -rows % 4
    bad = torch.arange(3, 300, 7, device="cuda")
    for i, call in enumerate(calls(rows, 300)):
        empty = plan._replace(cnt=plan.cnt.clone())
        empty.cnt[bad] = 0
        broken = plan._replace(off=plan.off.clone())
        broken.off[bad] = torch.tensor([LAST, -1, rows + 1], device="cuda").repeat(50)[:len(bad)]
        assert torch.equal(call(broken), call(empty)), i
        assert moe.moe_device_errors() == 32
