"""What the MXFP4 and few-token calls refuse, on the host (no GPU), and the
tests' own definition of the format against its published table."""
import pytest

from combine_moe_plan_02_gb300 import _abi, build

torch = pytest.importorskip("torch")
EINVAL, EALIGN, OK = _abi.MOE_EINVAL, _abi.MOE_EALIGN, _abi.MOE_OK
FAKE, MIS8, MIS4 = 0x10000, 0x10008, 0x10002     # aligned, not to 16 bytes, not to 4; never read


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.load()


def test_definition():
    """Block maxima 4 .. 8 times the scale; ties to even; saturation at 6."""
    from tests import mxfp4
    x = torch.zeros(1, 64)
    x[0, :12] = torch.tensor([4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 0.26, -0.74, 7.9, -0.1])
    codes, scales = mxfp4.quant(x)
    assert scales.shape == (1, 1, 4) and scales.flatten().tolist() == [127, 0, 0, 0]
    v = mxfp4.values(codes, scales)[0, :12].tolist()
    assert v == [4, 0, 1, 1, 2, 2, 4, 4, 0.5, -0.5, 6, 0]
    assert codes[0, 0] == 6 and codes[0, 1] == 0x22 and codes[0, 5] == 0x87
    assert mxfp4.quant(x * 2.0 ** -140)[1][0, 0, 0] == 0
    assert mxfp4.quant(x.double() * 2.0 ** 125)[1][0, 0, 0] == 252
    x[0, 40] = float("nan")
    assert mxfp4.quant(x)[1].flatten().tolist() == [127, 255, 0, 0]


def test_quant_validation(L):
    f = lambda **k: L.moe_quant_mxfp4(
        k.get("x", FAKE), k.get("dt", 0), k.get("groups", 1), k.get("rows", 8), k.get("D", 64),
        k.get("codes", FAKE), k.get("scales", FAKE), None)
    for bad in (dict(dt=2), dict(dt=-1), dict(groups=-1), dict(rows=-1), dict(D=0), dict(D=1 << 24),
                dict(groups=1 << 16, rows=1 << 15), dict(x=None), dict(codes=None), dict(scales=None)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(D=16), dict(D=48), dict(x=MIS8), dict(codes=MIS8), dict(scales=MIS4)):
        assert f(**bad) == EALIGN, bad
    assert f(rows=0) == OK and f(groups=0) == OK


def test_dispatch_validation(L):
    f = lambda **k: L.moe_dispatch_quant_mxfp4(
        k.get("x", FAKE), k.get("dt", 0), k.get("S", 4), k.get("D", 64), k.get("K", 2),
        k.get("map", FAKE), k.get("codes", FAKE), k.get("scales", FAKE), k.get("rows", 8), None)
    for bad in (dict(dt=2), dict(S=-1), dict(K=0), dict(K=33), dict(S=1 << 30), dict(D=0), dict(rows=0),
                dict(rows=-1), dict(rows=1 << 31), dict(x=None), dict(map=None), dict(codes=None),
                dict(scales=None)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(D=40), dict(x=MIS8), dict(codes=MIS8), dict(scales=MIS4)):
        assert f(**bad) == EALIGN, bad
    assert f(S=0) == OK


def test_swiglu_and_dequant_validation(L):
    f = lambda **k: L.moe_swiglu_quant_mxfp4(
        k.get("u", FAKE), k.get("dt", 0), k.get("rows", 8), k.get("F", 64), k.get("codes", FAKE),
        k.get("scales", FAKE), None)
    g = lambda **k: L.moe_dequant_mxfp4(
        k.get("codes", FAKE), k.get("scales", FAKE), k.get("groups", 1), k.get("rows", 8),
        k.get("F", 64), k.get("u", FAKE), k.get("dt", 0), None)
    for h in (f, g):
        for bad in (dict(dt=2), dict(rows=-1), dict(rows=1 << 31), dict(F=0), dict(F=1 << 24), dict(u=None),
                    dict(codes=None), dict(scales=None)):
            assert h(**bad) == EINVAL, bad
        for bad in (dict(F=33), dict(u=MIS8), dict(codes=MIS8), dict(scales=MIS4)):
            assert h(**bad) == EALIGN, bad
        assert h(rows=0) == OK


def test_binding_refuses():
    import combine_moe_plan_02_gb300 as moe
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = moe.MxFp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8))
    assert q.shape == (4, 64)
    for bad, error in ((x.half(), TypeError), (x[0], ValueError), (x[:, :40], ValueError),
                       (x[:, :0], ValueError)):
        with pytest.raises(error):
            moe.moe_quant_mxfp4(bad)
    for bad in (q._replace(codes=q.codes.int()), q._replace(scales=q.scales.float())):
        with pytest.raises(TypeError):
            moe.moe_dequant_mxfp4(bad)
    for bad in (q._replace(scales=q.scales[:, :2]), q._replace(scales=q.scales[0]),
                q._replace(codes=q.codes[:, :12])):
        with pytest.raises(ValueError):
            moe.moe_dequant_mxfp4(bad)
    with pytest.raises(ValueError):
        moe.moe_dequant_mxfp4(q, out=torch.zeros(4, 32))
    with pytest.raises(TypeError):
        moe.moe_dequant_mxfp4(q, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.moe_quant_mxfp4(torch.zeros(3, 64), out=q)
    tok_map = torch.zeros(4, 2, dtype=torch.int64)
    for args, error in (((x, tok_map.int()), TypeError), ((x, tok_map[:3]), ValueError),
                        ((x[None], tok_map), ValueError), ((x.half(), tok_map), TypeError)):
        with pytest.raises(error):
            moe.moe_dispatch_quant_mxfp4(*args)
    with pytest.raises(ValueError):
        moe.moe_swiglu_quant_mxfp4(torch.zeros(4, 33))
    with pytest.raises(ValueError):   # tensors of the host are refused before the call
        moe.moe_quant_mxfp4(x)
