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
    with pytest.raises(ValueError):   # three dimensions
        moe.moe_dispatch_quant_mxfp4(x, tok_map, out=moe.MxFp4(q.codes[None], q.scales[None]))
    with pytest.raises(ValueError):
        moe.moe_swiglu_quant_mxfp4(torch.zeros(4, 33))
    with pytest.raises(ValueError):   # tensors of the host are refused before the call
        moe.moe_quant_mxfp4(x)


def test_product_validation(L):
    f = lambda **k: L.moe_expert_gemm_mxfp4(
        k.get("x", FAKE), k.get("xs", FAKE), k.get("rows", 8), k.get("w", FAKE), k.get("ws", FAKE),
        k.get("N", 64), k.get("D", 64), k.get("E", 4), k.get("cnt", FAKE), k.get("off", FAKE), k.get("y", FAKE),
        k.get("dt", 0), None)
    for bad in (dict(dt=2), dict(dt=3), dict(rows=-1), dict(rows=1 << 31), dict(E=0), dict(E=1025), dict(N=0),
                dict(N=1 << 24), dict(D=0), dict(D=32800), dict(x=None), dict(xs=None), dict(w=None), dict(ws=None),
                dict(cnt=None), dict(off=None), dict(y=None), dict(rows=1 << 28, E=1024, N=4096)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(rows=6), dict(N=12), dict(D=48), dict(x=MIS8), dict(xs=MIS8), dict(w=MIS8), dict(ws=MIS8),
                dict(y=MIS8)):
        assert f(**bad) == EALIGN, bad
    assert f(rows=0) == OK


def test_layer_validation(L):
    def f(**k):
        a = dict(x=FAKE, S=2, H=64, idx=FAKE, w=FAKE, K=2, E=8, F=32, dt=0, up=FAKE, us=FAKE, down=FAKE, ds=FAKE,
                 out=FAKE, odt=0, ws=FAKE, bytes=1 << 30)
        a.update(k)
        return L.moe_expert_layer(a["x"], a["S"], a["H"], a["idx"], a["w"], a["K"], a["E"], a["F"], a["dt"], a["up"],
                                  a["us"], a["down"], a["ds"], a["out"], a["odt"], a["ws"], a["bytes"], None)
    for bad in (dict(dt=1), dict(dt=2), dict(dt=4), dict(odt=2), dict(odt=3), dict(S=-1), dict(S=513), dict(H=0),
                dict(H=16392), dict(K=0), dict(K=33), dict(E=0), dict(E=1025), dict(F=0), dict(F=16392), dict(x=None),
                dict(idx=None), dict(w=None), dict(up=None), dict(down=None), dict(out=None), dict(ws=None),
                dict(bytes=64), dict(dt=3, us=None), dict(dt=3, ds=None)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(H=60), dict(F=28), dict(dt=3, H=48), dict(dt=3, F=40), dict(x=MIS8), dict(up=MIS8),
                dict(down=MIS8), dict(out=MIS8), dict(ws=MIS8), dict(dt=3, us=MIS8), dict(dt=3, ds=MIS8)):
        assert f(**bad) == EALIGN, bad
    assert f(S=0) == OK
    need = L.moe_expert_layer_workspace_size(2, 64, 2, 8, 32, 0)
    assert need == 4 * 32 * 64 + 1024 + 256   # four parts of 32 rows
    assert f(bytes=need - 1) == EINVAL
    need = L.moe_expert_layer_workspace_size(2, 64, 2, 8, 32, 3)
    assert need == 4 * 64 * 32 + 4 * 512 + 4 * 64 * 16 + 4 * 512 + 1024 + 256   # four parts of 64 rows
    assert f(dt=3, bytes=need - 1) == EINVAL
    for out_of_range in ((-1, 64, 2, 8, 32, 0), (2, 0, 2, 8, 32, 0), (1024, 64, 2, 8, 32, 3), (2, 64, 2, 0, 32, 0),
                         (2, 64, 2, 8, 32, 1)):
        assert L.moe_expert_layer_workspace_size(*out_of_range) == 0


def test_layer_binding_refuses():
    import combine_moe_plan_02_gb300 as moe
    bf = torch.bfloat16
    x, idx, w = torch.zeros(2, 64, dtype=bf), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    up, down = torch.zeros(4, 64, 64, dtype=bf), torch.zeros(4, 64, 32, dtype=bf)
    q = moe.MxFp4(torch.zeros(4, 64, 32, dtype=torch.uint8), torch.zeros(4, 1, 64, 4, dtype=torch.uint8))
    for args, error in (((x.float(), idx, w, up, down), TypeError), ((x, idx.long(), w, up, down), TypeError),
                        ((x, idx, w.double(), up, down), TypeError), ((x, idx, w[:, :1], up, down), TypeError),
                        ((x, idx[:1], w[:1], up, down), TypeError), ((x, idx, w, up.float(), down), TypeError),
                        ((x, idx, w, q, down), TypeError), ((x, idx, w, up, q), TypeError),
                        ((x, idx, w, up[:, :63], down), ValueError), ((x, idx, w, up, down[:3]), ValueError),
                        ((x, idx, w, up[0], down), ValueError), ((x[:, :32], idx, w, up, down), ValueError)):
        with pytest.raises(error):
            moe.moe_expert_layer(*args)
    with pytest.raises(ValueError):
        moe.moe_expert_layer(x, idx, w, up, down, out=torch.zeros(2, 32, dtype=bf))


def test_product_binding_refuses():
    import combine_moe_plan_02_gb300 as moe
    rows = moe.MxFp4(torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(1, 8, 4, dtype=torch.uint8))
    w = moe.MxFp4(torch.zeros(4, 64, 32, dtype=torch.uint8), torch.zeros(4, 1, 64, 4, dtype=torch.uint8))
    none = torch.zeros(0)
    plan = moe.Plan(torch.zeros(4, dtype=torch.int32), torch.zeros(5, dtype=torch.int64), none, none, none)
    for args, error in (((w, w, plan), ValueError), ((rows, rows, plan), ValueError),
                        ((rows, w, plan._replace(cnt=plan.cnt.long())), TypeError),
                        ((rows, w, plan._replace(cnt=plan.cnt[:3])), ValueError),
                        ((rows, w._replace(codes=w.codes[:, :, :16].contiguous()), plan), ValueError)):
        with pytest.raises(error):
            moe.moe_expert_gemm_mxfp4(*args)
    with pytest.raises(TypeError):
        moe.moe_expert_gemm_mxfp4(rows, w, plan, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.moe_expert_gemm_mxfp4(rows, w, plan, out=torch.zeros(8, 32))


def test_calls_run_on_their_tensors_device(monkeypatch):
    """A call whose tensors are on another device than the current one switches to it."""
    import contextlib

    import combine_moe_plan_02_gb300 as moe
    seen, entered = [], []

    class Fake:
        def moe_fake(self, *args):
            seen.append((args, bool(entered)))
            return 0

    class Tensor:
        def get_device(self):
            return 2

    @contextlib.contextmanager
    def device(index):
        entered.append(index)
        yield
        entered.clear()

    monkeypatch.setattr(moe, "lib", Fake)
    monkeypatch.setattr(torch.cuda, "device", device)
    for current, switched in ((2, False), (0, True)):
        monkeypatch.setattr(moe, "_current_device", lambda: current)
        moe._run("moe_fake", Tensor(), 1, 2)
        assert seen.pop() == ((1, 2), switched) and not entered
