"""The few-token layer's grids: where one counts on two CTAs of an SM, the SM holds two."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("mx", [0, 3])
@pytest.mark.parametrize("E", [1, 8, 24, 64, 128, 256, 1000, 1024])
def test_ctas_fit(E, mx):
    import combine_moe_plan_02_gb300 as moe
    f, counts, seen = moe.lib().moe_selftest_layer_ctas, (ctypes.c_int32 * 4)(), set()
    for K in (1, 2, 3, 8, 32):
        for S in range(1, 1024 // K + 1):
            assert f(S, 7168, K, E, 2048, mx, counts) == 0
            for asked, held in (counts[:2], counts[2:]):
                assert 1 <= asked <= held, (S, K, asked, held)
                seen.add(asked)
    assert 2 in seen


def test_the_widest_lists_have_a_form():
    """Sizes at which two CTAs of four (five) stages just do and just do not fit."""
    import combine_moe_plan_02_gb300 as moe
    f, counts = moe.lib().moe_selftest_layer_ctas, (ctypes.c_int32 * 4)()
    # lists of 8 tokens' 64 entries and of 1024 entries of 1024 experts
    for S, E, ctas in ((8, 64, 2), (128, 1024, 1)):
        assert f(S, 7168, 8, E, 2048, 3, counts) == 0
        assert counts[0] == counts[2] == ctas
    for bad in ((0, 64, 1, 8, 32, 0), (1, 0, 1, 8, 32, 0), (1, 64, 33, 8, 32, 0), (1, 64, 1, 8, 32, 1)):
        assert f(*bad, counts) == 1
    assert f(1, 64, 1, 8, 32, 0, None) == 1
