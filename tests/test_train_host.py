"""What the gradient and product calls refuse, on the host (no GPU): nothing
is enqueued before the arguments are checked."""
import ctypes

import pytest

from combine_moe_plan_02_gb300 import _abi, build

torch = pytest.importorskip("torch")
EINVAL, EALIGN, OK = _abi.MOE_EINVAL, _abi.MOE_EALIGN, _abi.MOE_OK
FAKE, MIS = 0x10000, 0x10008     # 16-byte aligned and not; never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.load()


def test_combine_backward_validation(L):
    f = lambda **k: L.moe_combine_backward(
        k.get("dout", FAKE), k.get("ddt", 0), k.get("y", FAKE), k.get("rows", 8),
        k.get("ydt", 0), k.get("w", FAKE), k.get("tm", FAKE), k.get("cnt", FAKE),
        k.get("off", FAKE), k.get("S", 4), k.get("H", 64), k.get("K", 2), k.get("E", 8),
        k.get("dy", FAKE), k.get("dw", FAKE), None)
    for bad in (dict(ddt=2), dict(ydt=2), dict(S=-1), dict(H=0), dict(K=0), dict(K=33),
                dict(E=0), dict(E=1025), dict(rows=0), dict(rows=1 << 31), dict(dout=None),
                dict(y=None), dict(w=None), dict(tm=None), dict(cnt=None), dict(off=None),
                dict(dy=None), dict(dw=None), dict(S=1 << 30, K=2)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(H=12), dict(dout=MIS), dict(y=MIS), dict(dy=MIS)):
        assert f(**bad) == EALIGN, bad


def test_expert_gemm_validation(L):
    def f(fn, **k):
        a = dict(rows_a=FAKE, rows=8, other=FAKE, N=64, D=64, E=4, cnt=FAKE, off=FAKE, out=FAKE,
                 dt=0)
        a.update(k)
        if fn == "moe_expert_gemm_wgrad":
            return L.moe_expert_gemm_wgrad(a["rows_a"], a["other"], a["rows"], a["N"], a["D"],
                                           a["E"], a["cnt"], a["off"], a["out"], a["dt"], None)
        return getattr(L, fn)(a["rows_a"], a["rows"], a["other"], a["N"], a["D"], a["E"],
                              a["cnt"], a["off"], a["out"], a["dt"], None)
    for fn in ("moe_expert_gemm", "moe_expert_gemm_dgrad", "moe_expert_gemm_wgrad"):
        for bad in (dict(dt=2), dict(rows=-1), dict(rows=1 << 31), dict(E=0), dict(E=1025),
                    dict(N=0), dict(D=0), dict(N=1 << 24), dict(D=1 << 24), dict(rows_a=None),
                    dict(other=None), dict(cnt=None), dict(off=None), dict(out=None)):
            assert f(fn, **bad) == EINVAL, (fn, bad)
        for bad in (dict(N=12), dict(D=60), dict(rows_a=MIS), dict(other=MIS), dict(out=MIS)):
            assert f(fn, **bad) == EALIGN, (fn, bad)
    assert f("moe_expert_gemm", rows=0) == OK          # no rows: nothing is enqueued
    assert f("moe_expert_gemm_dgrad", rows=0) == OK


def test_grad_norm_validation(L):
    def f(**k):
        n = k.get("n", 1)
        ptr = (ctypes.c_void_p * 1)(k.get("ptr", FAKE))
        out = (ctypes.c_void_p * 1)(k.get("out", FAKE))
        numel = (ctypes.c_int64 * 1)(k.get("numel", 5))
        dt = (ctypes.c_int * 1)(k.get("dt", 1))
        return L.moe_clip_grad_norm(k.get("ptrs", ptr), k.get("outs", out), numel, dt, n,
                                    k.get("most", 1.0), k.get("norm", FAKE), k.get("ws", FAKE),
                                    k.get("ws_bytes", 1 << 20), None)
    size = L.moe_grad_norm_workspace_size()
    assert size > 0 and size % 256 == 0
    for bad in (dict(n=-1), dict(n=65537), dict(dt=2), dict(numel=-1), dict(ptr=None),
                dict(out=None), dict(ptrs=None), dict(outs=None), dict(most=-1.0),
                dict(most=float("nan")), dict(norm=None), dict(ws=None),
                dict(ws_bytes=size - 1)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(ptr=FAKE + 2), dict(out=FAKE + 1), dict(dt=0, ptr=FAKE + 1),
                dict(norm=FAKE + 2), dict(ws=FAKE + 128)):
        assert f(**bad) == EALIGN, bad


def test_binding_checks():
    import combine_moe_plan_02_gb300 as moe
    bf = torch.bfloat16
    plan = moe.Plan(torch.zeros(4, dtype=torch.int32), torch.zeros(5, dtype=torch.int64),
                    torch.zeros(6, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int64),
                    torch.zeros(1, dtype=torch.int32))
    x, w = torch.zeros(6, 16, dtype=bf), torch.zeros(4, 8, 16, dtype=bf)
    dy = torch.zeros(6, 8, dtype=bf)
    with pytest.raises(TypeError, match="bfloat16"):
        moe.moe_expert_gemm(x.float(), w, plan)
    with pytest.raises(TypeError, match="bfloat16"):
        moe.moe_expert_gemm_wgrad(dy, x.half(), plan)
    with pytest.raises(ValueError, match="rows, D"):
        moe.moe_expert_gemm(dy, w, plan)
    with pytest.raises(ValueError, match="rows, N"):
        moe.moe_expert_gemm_dgrad(x, w, plan)
    with pytest.raises(ValueError, match="experts"):
        moe.moe_expert_gemm(x, w[:3], plan)
    with pytest.raises(ValueError, match="rows"):
        moe.moe_expert_gemm_wgrad(dy[:4], x, plan)
    with pytest.raises(ValueError, match="out must"):
        moe.moe_expert_gemm(x, w, plan, out=torch.zeros(6, 16, dtype=bf))
    with pytest.raises(TypeError, match="unsupported"):
        moe.moe_expert_gemm(x, w, plan, out=torch.zeros(6, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_expert_gemm(x, w, plan)
    y, tw = torch.zeros(6, 16), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="dout"):
        moe.moe_combine_backward(torch.zeros(2, 16), y, tw, plan)
    with pytest.raises(TypeError, match="topk_w"):
        moe.moe_combine_backward(torch.zeros(3, 16), y, tw.double(), plan)
    with pytest.raises(ValueError, match="dy"):
        moe.moe_combine_backward(torch.zeros(3, 16), y, tw, plan, dy=y.to(bf))
    with pytest.raises(ValueError, match="dw"):
        moe.moe_combine_backward(torch.zeros(3, 16), y, tw, plan, dw=torch.zeros(3, 3))
    with pytest.raises(ValueError, match="no gradients"):
        moe.moe_grad_norm([])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        moe.moe_grad_norm([torch.zeros(4, dtype=torch.float16)],
                          workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="types and sizes"):
        moe.moe_clip_grad_norm([torch.zeros(4)], 1.0, out=[torch.zeros(5)],
                               workspace=torch.zeros(1 << 20, dtype=torch.uint8))


def test_plans_of_other_types_or_lengths():
    """The kernels read cnt as int32 [E] and off as int64 [E + 1]: anything
    else would be read as other numbers or past its end."""
    import combine_moe_plan_02_gb300 as moe
    bf = torch.bfloat16
    good = moe.Plan(torch.zeros(4, dtype=torch.int32), torch.zeros(5, dtype=torch.int64),
                    torch.zeros(6, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int64),
                    torch.zeros(1, dtype=torch.int32))
    x, w, dy = torch.zeros(6, 16, dtype=bf), torch.zeros(4, 8, 16, dtype=bf), torch.zeros(6, 8, dtype=bf)
    dout, y, tw = torch.zeros(3, 16), torch.zeros(6, 16), torch.zeros(3, 2)
    calls = [lambda p: moe.moe_expert_gemm(x, w, p), lambda p: moe.moe_expert_gemm_dgrad(dy, w, p),
             lambda p: moe.moe_expert_gemm_wgrad(dy, x, p),
             lambda p: moe.moe_combine_backward(dout, y, tw, p),
             lambda p: moe.moe_dispatch_backward(y, p)]
    for call in calls:
        with pytest.raises(TypeError, match="cnt must be int32"):
            call(good._replace(cnt=good.cnt.long()))
        with pytest.raises(TypeError, match="off int64"):
            call(good._replace(off=good.off.int()))
        with pytest.raises(ValueError, match="experts"):
            call(good._replace(off=good.off[:4]))
        with pytest.raises(ValueError, match="CUDA"):
            call(good)
    for call in calls[3:]:
        with pytest.raises(TypeError, match="tok_map"):
            call(good._replace(tok_map=good.tok_map.int()))
    with pytest.raises(ValueError, match="out must"):
        moe.moe_dispatch_backward(y, good, out=torch.zeros(3, 8, dtype=bf))


def test_combine_backward_of_nothing(L):
    """No tokens and no rows: nothing to do, as in the calls before it."""
    f = lambda **k: L.moe_combine_backward(
        None, 0, None, k.get("rows", 0), k.get("ydt", 0), None, None, FAKE, FAKE, 0, k.get("H", 64),
        2, 8, None, None, None)
    assert f() == OK
    assert f(rows=1) == EINVAL and f(H=0) == EINVAL and f(ydt=2) == EINVAL


def test_combine_backward_of_more_tokens_than_a_grid_has(L):
    """One CTA a token beside those that clear rows: refused, not left to the
    launch."""
    f = lambda S: L.moe_combine_backward(FAKE, 0, FAKE, 8, 0, FAKE, FAKE, FAKE, FAKE, S, 64, 1, 8,
                                         FAKE, FAKE, None)
    assert f((1 << 31) - 1) == EINVAL and f((1 << 31) - 152) == EINVAL
