"""The experts' products and their gradients against plain sums in 64 bits.

Most inputs are small whole numbers, so that every product and every partial
sum is exact in f32 whatever the order: the f32 output then has to equal the
64-bit one, and the bf16 output its one rounding.  Normal inputs have the
derived bound: 16 products enter the accumulator at a time, each addition off
by at most 2^-23 of what has been summed, so (len / 16 + 16) * 2^-23 times the
sum of the products' magnitudes, and 2^-8 of the value for a bf16 output.

Rows in no bucket and outputs before the call hold NaN.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def make_plan(counts, capacity=0, tail=0, dev="cuda"):
    """A plan over buckets of the given sizes (the products read cnt and off
    only) and its number of rows."""
    import combine_moe_plan_02_gb300 as moe
    cnt = torch.tensor(counts, dtype=torch.int32, device=dev)
    off = torch.zeros(len(counts) + 1, dtype=torch.int64, device=dev)
    if capacity:
        off[:] = torch.arange(len(counts) + 1, device=dev) * capacity
    else:
        off[1:] = cnt.cumsum(0)
    none = torch.empty(0, 1, dtype=torch.int64, device=dev)
    rows = int(off[-1]) + tail
    return moe.Plan(cnt, off, none, none, none), rows


def filled(plan, rows):
    live = torch.zeros(rows, dtype=torch.bool)
    cnt, off = plan.cnt.tolist(), plan.off.tolist()
    for e, c in enumerate(cnt):
        live[off[e]:off[e] + c] = True
    return live.cuda()


def ints(shape, seed, most=4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device="cuda").to(BF16)


def packed(plan, rows, width, seed, maker=ints):
    x = maker((rows, width), seed)
    x[~filled(plan, rows)] = float("nan")
    return x


def normal(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=BF16)


def reference(op, plan, a, b, absolute=False):
    """Sums in 64 bits, bucket by bucket."""
    f = (lambda t: t.to(F64).abs()) if absolute else (lambda t: t.to(F64))
    cnt, off = plan.cnt.tolist(), plan.off.tolist()
    E = len(cnt)
    if op == "dw":
        out = torch.zeros(E, a.shape[1], b.shape[1], dtype=F64, device="cuda")
    else:
        out = torch.zeros(a.shape[0], b.shape[1] if op == "y" else b.shape[2], dtype=F64,
                          device="cuda")
    for e in range(E):
        s = slice(off[e], off[e] + cnt[e])
        if not cnt[e]:
            continue
        if op == "y":
            out[s] = f(a[s]) @ f(b[e]).T
        elif op == "dx":
            out[s] = f(a[s]) @ f(b[e])
        else:
            out[e] = f(a[s]).T @ f(b[s])
    return out


def call(op, plan, a, b, dtype):
    import combine_moe_plan_02_gb300 as moe
    E = plan.cnt.numel()
    fn = {"y": moe.moe_expert_gemm, "dx": moe.moe_expert_gemm_dgrad,
          "dw": moe.moe_expert_gemm_wgrad}[op]
    shape = {"y": lambda: (a.shape[0], b.shape[1]), "dx": lambda: (a.shape[0], b.shape[2]),
             "dw": lambda: (E, a.shape[1], b.shape[1])}[op]()
    out = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    assert fn(*((a, b, plan)), out=out) is out
    torch.cuda.synchronize()
    assert moe.moe_device_errors() == 0
    return out


def operands(op, plan, rows, N, D, seed, maker=ints):
    E = plan.cnt.numel()
    if op == "y":
        return packed(plan, rows, D, seed, maker), maker((E, N, D), seed + 1)
    if op == "dx":
        return packed(plan, rows, N, seed, maker), maker((E, N, D), seed + 1)
    return packed(plan, rows, N, seed, maker), packed(plan, rows, D, seed + 1, maker)


SHAPES = [
    # counts, N, D, capacity, rows after the last bucket
    ([1], 8, 8, 0, 0),                                  # one token, the smallest sizes
    ([1, 0, 2, 0], 136, 72, 0, 3),                      # empty experts, a tail
    ([0, 0, 0], 64, 64, 0, 5),                          # nothing at all
    ([17, 255, 256, 257, 1, 15, 16], 128, 64, 0, 0),    # around the cuts of a bucket
    ([513, 31, 600], 392, 200, 0, 0),
    ([5, 9, 0, 12], 264, 520, 12, 4),                   # padded buckets
    ([63, 64, 65, 127, 128, 129], 256, 256, 130, 0),
    ([33] * 40, 48, 1032, 0, 0),                        # many experts
    ([1] * 300, 24, 136, 0, 1),
    ([700, 3], 2056, 1544, 0, 0),                       # several tiles each way
]


@pytest.mark.parametrize("op", ["y", "dx", "dw"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_whole_numbers_are_exact(op, dtype, shape):
    counts, N, D, cap, tail = SHAPES[shape]
    plan, rows = make_plan(counts, cap, tail)
    a, b = operands(op, plan, rows, N, D, 10 * shape)
    got = call(op, plan, a, b, dtype)
    want = reference(op, plan, a, b)
    assert want.abs().max() < 2 ** 24
    assert torch.equal(got, want.to(F32).to(dtype))


@pytest.mark.parametrize("op", ["y", "dx", "dw"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_normal_inputs(op, dtype):
    plan, rows = make_plan([300, 0, 77, 512, 1], 0, 0)
    N, D = 640, 2048
    a, b = operands(op, plan, rows, N, D, 5, normal)
    got = call(op, plan, a, b, dtype).to(F64)
    want, mass = reference(op, plan, a, b), reference(op, plan, a, b, absolute=True)
    length = {"y": D, "dx": N, "dw": 512}[op]
    bound = (length / 16 + 16) * 2.0 ** -23 * mass
    if dtype == BF16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    assert ((got - want).abs() <= bound).all()


def test_infinities_stay_in_their_rows():
    """An infinite or NaN row spoils its own outputs and no others."""
    plan, rows = make_plan([40, 24, 70])
    x, w = ints((rows, 64), 1), ints((3, 128, 64), 2)
    x[39, 3], x[40, 5] = float("inf"), float("nan")
    y = call("y", plan, x, w, F32)
    want = reference("y", plan, x, w).to(F32)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[39] = keep[40] = False
    assert torch.equal(y[keep], want[keep])
    assert torch.isnan(y[40]).all() and not torch.isfinite(y[39][w[0, :, 3] != 0]).any()
    dw = call("dw", plan, ints((rows, 128), 3), x, F32)
    assert torch.isfinite(dw[2]).all()                   # the third expert's rows are finite
    cols = [d for d in range(64) if d not in (3, 5)]
    assert torch.isfinite(dw[:, :, cols]).all()


def test_gradients_against_differences():
    """The products are linear in each operand: for whole numbers the
    difference <dy, F(x + v) - F(x)> equals <dx, v> exactly, and likewise for
    the weights."""
    plan, rows = make_plan([19, 0, 130, 64], 0, 2)
    N, D = 72, 96
    live = filled(plan, rows)
    x, v = ints((rows, D), 1, 2), ints((rows, D), 2, 1)
    w, u = ints((4, N, D), 3, 2), ints((4, N, D), 4, 1)
    dy = ints((rows, N), 5, 2)
    x[~live], v[~live], dy[~live] = 0, 0, 0
    y = call("y", plan, x, w, F32).to(F64)
    dx = call("dx", plan, dy, w, F32).to(F64)
    dw = call("dw", plan, dy, x, F32).to(F64)
    along_x = (call("y", plan, x + v, w, F32).to(F64) - y) * dy.to(F64)
    along_w = (call("y", plan, x, w + u, F32).to(F64) - y) * dy.to(F64)
    assert along_x.sum() == (dx * v.to(F64)).sum()
    assert along_w.sum() == (dw * u.to(F64)).sum()


def test_matches_a_real_plan_on_another_stream_and_in_a_graph():
    import combine_moe_plan_02_gb300 as moe
    g = torch.Generator(device="cuda").manual_seed(3)
    S, E, K, N, D = 77, 16, 4, 144, 256
    idx = torch.rand(S, E, generator=g, device="cuda").topk(K).indices.to(torch.int32)
    idx[5] = -1
    x, w = ints((S, D), 1), ints((E, N, D), 2)
    plan, px, _ = moe.moe_plan_dispatch(idx, x, E)
    torch.cuda.synchronize()
    live = filled(plan, px.shape[0])
    px[~live] = float("nan")
    want = reference("y", plan, px, w).to(BF16)
    out = torch.full((S * K, N), float("nan"), dtype=BF16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    moe.moe_expert_gemm(px, w, plan, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_expert_gemm(px, w, plan, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert moe.moe_device_errors() == 0


def test_long_offsets():
    """Rows and weights whose byte offsets pass 32 bits."""
    N, D = 8, 7168
    rows = 340000                                        # x: 4.9 GB
    plan, _ = make_plan([7, rows - 7 - 20, 20])
    x = torch.zeros(rows, D, dtype=BF16, device="cuda")
    w = ints((3, N, D), 2)
    x[-20:] = ints((20, D), 1)
    y = call("y", plan, x, w, F32)
    want = x[-20:].to(F64) @ w[2].to(F64).T
    assert torch.equal(y[-20:], want.to(F32)) and not y[:-20].any()
    dx = call("dx", plan, y.to(BF16), w, BF16)           # dx: 4.9 GB
    assert torch.equal(dx[-20:], (y[-20:].to(BF16).to(F64) @ w[2].to(F64)).to(F32).to(BF16))
    assert not dx[:-20].any()


def test_a_bucket_outside_the_rows_is_left_out():
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([4, 4, 4])
    x, w = ints((rows, 64), 1), ints((3, 64, 64), 2)
    want = reference("y", plan, x, w).to(F32)
    plan.cnt[2] = 100
    out = torch.full((rows, 64), 5.0, dtype=F32, device="cuda")
    moe.moe_expert_gemm(x, w, plan, out=out)
    torch.cuda.synchronize()
    assert moe.moe_device_errors() == 32
    assert torch.equal(out[:8], want[:8])
    assert moe.moe_device_errors() == 0


def test_the_most_experts_and_no_rows():
    import combine_moe_plan_02_gb300 as moe
    plan, rows = make_plan([e % 3 for e in range(1024)], 0, 0)
    for op in ("y", "dx", "dw"):
        a, b = operands(op, plan, rows, 40, 72, 3)
        assert torch.equal(call(op, plan, a, b, F32), reference(op, plan, a, b).to(F32))
    none, _ = make_plan([0] * 4)
    x, dy, w = (torch.empty(0, 64, dtype=BF16, device="cuda"),
                torch.empty(0, 32, dtype=BF16, device="cuda"), ints((4, 32, 64), 1))
    assert moe.moe_expert_gemm(x, w, none).shape == (0, 32)
    assert moe.moe_expert_gemm_dgrad(dy, w, none).shape == (0, 64)
    dw = call("dw", none, dy, x, F32)
    assert dw.shape == (4, 32, 64) and not dw.any()


def test_large_weights_with_rows_of_odd_sixteenths():
    """A bf16 weights' gradient of 390 MB whose rows are not whole 32-byte
    sectors (stored in wider boxes), with ragged and empty buckets and sizes
    that end inside a box."""
    plan, rows = make_plan([(7 * e) % 75 for e in range(96)], 0, 3)
    a, b = operands("dw", plan, rows, 712, 2856, 4)
    got = call("dw", plan, a, b, BF16)
    assert torch.equal(got, reference("dw", plan, a, b).to(F32).to(BF16))


@pytest.mark.parametrize("op", ["y", "dx"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("counts,out,length,cap,tail", [
    ([1], 8, 1024, 0, 0),                       # the fewest rows, the shortest reduction
    ([1, 0, 2], 600, 1032, 0, 0),               # nine tiles, four pairs each
    ([64], 256, 4104, 0, 0),                    # the most rows
    ([33, 31], 1280, 2048, 0, 0),               # ten tiles, blocks of 33 and 31 rows
    ([3, 0, 1, 4], 1000, 520, 0, 0),            # 32 tiles, two pairs each
    ([2, 5], 264, 3000, 6, 3),                  # padded, rows after the last bucket
    ([0, 0, 0], 64, 1024, 0, 7),                # no tile at all
])
def test_few_rows_share_a_reduction(op, dtype, counts, out, length, cap, tail):
    plan, rows = make_plan(counts, cap, tail)
    N, D = (out, length) if op == "y" else (length, out)
    a, b = operands(op, plan, rows, N, D, 7)
    got = call(op, plan, a, b, dtype)
    want = reference(op, plan, a, b)
    assert want.abs().max() < 2 ** 24
    assert torch.equal(got, want.to(F32).to(dtype))
    assert torch.equal(got, call(op, plan, a, b, dtype))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,D", [(264, 392), (8, 8), (40, 264)])
def test_the_weights_gradient_ends_where_a_bucket_ends(dtype, N, D):
    """Buckets of 1 to 130 rows, so every length of a last block, the next one
    all NaN: a row read past an end, by either CTA of a pair, would show."""
    counts = [c for n in range(1, 131) for c in (n, 1 + n % 3)]
    plan, rows = make_plan(counts, 0, 5)
    a, b = operands("dw", plan, rows, N, D, 11)
    off = plan.off.tolist()
    for e in range(1, len(counts), 2):
        a[off[e]:off[e + 1]], b[off[e]:off[e + 1]] = float("nan"), float("nan")
    want = reference("dw", plan, a, b)[::2].to(F32).to(dtype)
    for _ in range(5):
        got = call("dw", plan, a, b, dtype)
        assert torch.equal(got[::2], want) and torch.isnan(got[1::2]).all()


def test_overlapping_buckets_of_a_few_rows():
    """Buckets that share rows may have more tiles than a call of few rows
    launches; those past it are left out and reported."""
    import combine_moe_plan_02_gb300 as moe
    plan, _ = make_plan([1] * 8)
    plan.off.zero_()
    x, w = ints((2, 1024), 1), ints((8, 64, 1024), 2)
    out = torch.full((2, 64), 5.0, dtype=F32, device="cuda")
    moe.moe_expert_gemm(x, w, plan, out=out)
    torch.cuda.synchronize()
    assert moe.moe_device_errors() == 32
    assert moe.moe_device_errors() == 0


# Long reductions.  At every step of 16 products the accumulator loses at most
# 2^-23 of what it holds; 8192 products (bf16 outputs) or 768 (f32) are summed
# there, and the parts of a sum are added in f32, each off by at most 2^-24.  For
# sums of positive terms that is relative to the sum, and a rounded output lies
# between the rounded ends of that interval.

def positive(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(shape, generator=g, device="cuda") + 0.5).to(BF16)


def check_long(got, want, length, dtype):
    per = 768 if dtype == F32 else 8192
    bound = per / 16 * 2.0 ** -23 + (length / per + 1) * 2.0 ** -24
    low, high = ((want * f).to(F32).to(dtype) for f in (1 - bound, 1 + bound))
    assert ((low <= got) & (got <= high)).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("op,counts,out", [("y", [2], 8), ("y", [70, 3], 40), ("dx", [1], 16),
                                           ("dx", [80], 8)])
def test_long_products(op, counts, out, dtype):
    """2^23 products for each output: more than one accumulator may sum, with
    the pairs of a cluster sharing the reduction and without."""
    length = 1 << 23
    plan, rows = make_plan(counts)
    N, D = (out, length) if op == "y" else (length, out)
    a, b = operands(op, plan, rows, N, D, 3, positive)
    got = call(op, plan, a, b, dtype)
    check_long(got, reference(op, plan, a, b), length, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("N,D", [(8, 8), (136, 264)])
def test_long_buckets(dtype, N, D):
    """The weights' gradient over millions of rows, beside short buckets."""
    length = (1 << 24) + 5 if N == 8 else (1 << 22) + 5
    plan, rows = make_plan([3, length, 0, 9000])
    a, b = operands("dw", plan, rows, N, D, 3, positive)
    got = call("dw", plan, a, b, dtype)
    check_long(got, reference("dw", plan, a, b), length, dtype)


def test_large_weights_with_long_buckets():
    """As test_large_weights_with_rows_of_odd_sixteenths, with reductions of more
    than one accumulator in some buckets."""
    plan, rows = make_plan([(7 * e) % 75 for e in range(94)] + [45000, 9001], 0, 3)
    a, b = operands("dw", plan, rows, 712, 2856, 4)
    got = call("dw", plan, a, b, BF16)
    want = reference("dw", plan, a, b)
    assert want.abs().max() < 2 ** 24
    assert torch.equal(got, want.to(F32).to(BF16))


@pytest.mark.parametrize("op", ["y", "dx", "dw"])
def test_f32_sums_of_thousands_of_products(op):
    """The 2-norm of an f32 output's error.  A step loses half of 2^-23 of the
    running sum on average at most, which in a part of 48 steps is a walk to
    the part's sum: 48 * 2^-24 * sqrt(1/4 + 1/12) of it (the mean and the
    spread of the walk), and the parts' additions 2^-25 each.  8192 products in
    one accumulator lose ten times as much."""
    length = 8192
    plan, rows = make_plan([length, length] if op == "dw" else [90, 300])
    N, D = {"y": (256, length), "dx": (length, 256), "dw": (256, 320)}[op]
    a, b = operands(op, plan, rows, N, D, 3, normal)
    got, want = call(op, plan, a, b, F32).to(F64), reference(op, plan, a, b)
    bound = 48 * 2.0 ** -24 * 3 ** -0.5 + (length / 768 + 1) * 2.0 ** -25
    assert (got - want).norm() <= bound * want.norm()


def test_a_bucket_that_takes_seconds():
    """The weights' gradient of 1.1 billion rows: its waits are for parts of
    the sum, each of which is done in time, not for the whole of it."""
    import combine_moe_plan_02_gb300 as moe
    rows = 1_100_000_003                                  # dy and x: 17.6 GB each
    plan, _ = make_plan([rows])
    a = torch.zeros(rows, 8, dtype=BF16, device="cuda")
    b = torch.zeros(rows, 8, dtype=BF16, device="cuda")
    at = torch.tensor([0, 1, 12345, rows // 2, rows - 70, rows - 1], device="cuda")
    a[at], b[at] = ints((6, 8), 1), ints((6, 8), 2)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    events[0].record()
    dw = moe.moe_expert_gemm_wgrad(a, b, plan, out_dtype=BF16)
    events[1].record()
    torch.cuda.synchronize()
    print(f"{events[0].elapsed_time(events[1]):.0f} ms")
    assert moe.moe_device_errors() == 0
    assert torch.equal(dw[0], (a[at].to(F64).T @ b[at].to(F64)).to(F32).to(BF16))


def test_random_shapes():
    """Shapes and buckets of no pattern, each over memory that is mapped anew, so
    that operands begin and end where mapped memory may."""
    import random
    r = random.Random(41)
    for n in range(60):
        counts = [0 if r.random() < 0.2 else r.randint(0, r.choice([3, 20, 80, 300]))
                  for _ in range(r.choice([1, 2, 5, 16, 64]))]
        N, D = 8 * r.randint(1, 80), 8 * r.randint(1, 120)
        plan, rows = make_plan(counts, max(counts) + 1 if n % 4 == 0 else 0, r.choice([0, 0, 5]))
        if rows == 0:
            continue
        for op in ("y", "dx", "dw"):
            torch.cuda.empty_cache()
            dtype = r.choice([F32, BF16])
            a, b = operands(op, plan, rows, N, D, n)
            want = reference(op, plan, a, b).to(F32).to(dtype)
            assert torch.equal(call(op, plan, a, b, dtype), want), (op, counts, N, D)
