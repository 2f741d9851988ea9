"""What the warp wait's self-test refuses (no GPU)."""
import pytest

from combine_moe_plan_02_gb300 import _abi, build


def test_ranges():
    pytest.importorskip("torch")
    build.build()
    f, fake = _abi.load().moe_selftest_warp_wait, 0x10000
    for bad in ((999, 0, 0, fake), (100_000_001, 0, 0, fake), (1000, -2, 0, fake), (1000, 200_000_001, 0, fake),
                (1000, 0, -1, fake), (1000, 0, 200_000_001, fake), (1000, 0, 0, None)):
        assert f(*bad, None) == _abi.MOE_EINVAL, bad
