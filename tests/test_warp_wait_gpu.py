"""A bounded wait by a whole warp: its lanes never part, whenever each began to wait and
whether the phase completes, completes in time for some of them only, or never does."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

MS = 1_000_000


# limit, completion (-1: never) and the second half's delay in ms; the warp's answer
@pytest.mark.parametrize("limit,complete,late,answer", [
    (5, 0, 0, 1), (20, 1, 0, 1), (20, 1, 10, 1),
    (1, -1, 0, 0), (1, -1, 3, 0),
    (1, 4, 8, 0)])   # over for the first half, complete before the second one looks
def test_lanes_agree(limit, complete, late, answer):
    import combine_moe_plan_02_gb300 as moe
    out = torch.full((32,), -1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    status = moe.lib().moe_selftest_warp_wait(limit * MS, -1 if complete < 0 else complete * MS, late * MS,
                                              out.data_ptr(), stream)
    assert status == 0
    assert out.tolist() == [answer] * 32
    assert moe.moe_device_errors() == 0
