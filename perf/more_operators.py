"""Operators of an expert layer that is served with 4-bit weights, or to a few tokens, and the cases that measure them.

  quant   rows on their way into the experts' buckets, or weights, to MXFP4 and the values that they then stand for
  expert  the experts' product over packed rows, both operands in MXFP4
  act     the gated activation between the two products, in MXFP4, and the product that takes it
  layer   a whole layer (up, gate, down, combine) for a few tokens, weights in bf16 or MXFP4

MXFP4 is the OCP Microscaling format v1.0: E2M1 elements (two a byte, the first in the low half) and one E8M0 scale for
32 elements of a row.  The scales of a [rows, D] tensor are laid out as [D / 128 rounded up, rows, 4].

`run` computes them with elementary torch operations in 32 bits, or with the package's own calls where `own` is set.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # prefill of the benchmark's batch: every token's row, quantised, in the buckets of its 8 experts
        {"name": "quant_dispatch_4096x7168", "op": "quant", "S": 4096, "D": 7168, "E": 64, "K": 8},
        # decoding 16 tokens: the call's latency
        {"name": "quant_dispatch_16x6144", "op": "quant", "S": 16, "D": 6144, "E": 256, "K": 8},
        # a checkpoint's weights, once as they are loaded: f32 masters of odd sizes
        {"name": "quant_weights_24x1048x7136", "op": "quant", "S": 0, "D": 7136, "E": 24, "N": 1048, "type": "f32"},
        # prefill: the up and gate product of the benchmark's batch, 512 rows an expert on average
        {"name": "expert_32768x7168x4096", "op": "expert", "S": 4096, "E": 64, "K": 8, "N": 4096, "D": 7168, "type": "bf16",
         "cap": 0},
        # serving, a batch of 128 decoded tokens: nearly all experts with a few rows each
        {"name": "expert_128_tokens", "op": "expert", "S": 128, "E": 256, "K": 8, "N": 4096, "D": 6144, "type": "bf16",
         "cap": 0},
        # a small odd-sized layer with padded buckets and f32 output
        {"name": "expert_odd_padded", "op": "expert", "S": 1001, "E": 24, "K": 3, "N": 1048, "D": 1440, "type": "f32",
         "cap": 172},
        # prefill: the activation of the same batch and its down product
        {"name": "act_32768x2048x7168", "op": "act", "S": 4096, "E": 64, "K": 8, "N": 7168, "D": 2048, "type": "bf16",
         "cap": 0},
        # 8 decoded tokens: 64 rows
        {"name": "act_8_tokens", "op": "act", "S": 8, "E": 256, "K": 8, "N": 6144, "D": 2048, "type": "bf16", "cap": 0},
        # serving one token with bf16 weights: eight experts, bound by their weights
        {"name": "layer_1_token", "op": "layer", "S": 1, "E": 256, "K": 8, "H": 6144, "F": 2048, "weights": "bf16",
         "type": "bf16"},
        # the same with 4-bit weights
        {"name": "layer_1_token_mxfp4", "op": "layer", "S": 1, "E": 256, "K": 8, "H": 6144, "F": 2048, "weights": "mxfp4",
         "type": "bf16"},
        # 32 decoded tokens: nearly all of 64 experts with a few rows each
        {"name": "layer_32_tokens_mxfp4", "op": "layer", "S": 32, "E": 64, "K": 8, "H": 7168, "F": 2048, "weights": "mxfp4",
         "type": "bf16"},
        # a small odd-sized layer with f32 output
        {"name": "layer_5_tokens_odd", "op": "layer", "S": 5, "E": 24, "K": 3, "H": 1416, "F": 520, "weights": "bf16",
         "type": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


MOST_BYTES, MOST_FLOPS, MOST_WEIGHTS = 3.2e9, 1.9e12, 3.4e9


def draw(rng):
    while True:
        op = rng.choice(["quant", "expert", "act", "layer"])
        E, K = rng.choice([8, 24, 64, 128, 256]), rng.randint(1, 8)
        if op == "quant":
            if rng.random() < 0.3:
                case = {"op": op, "S": 0, "D": 32 * _log(rng, 4, 224), "E": rng.randint(1, 32), "N": 8 * _log(rng, 8, 256),
                        "type": rng.choice(["bf16", "f32"])}
            else:
                case = {"op": op, "S": _log(rng, 1, 4096), "D": 32 * _log(rng, 4, 224), "E": E, "K": K}
        elif op == "layer":
            weights = rng.choice(["bf16", "mxfp4"])
            step = 8 if weights == "bf16" else 32
            case = {"op": op, "S": _log(rng, 1, 64), "E": E, "K": K, "H": step * _log(rng, 512 // step, 7168 // step),
                    "F": step * _log(rng, 256 // step, 2048 // step), "weights": weights, "type": rng.choice(["bf16", "f32"])}
        else:
            S = _log(rng, 1, 4096)
            case = {"op": op, "S": S, "E": E, "K": K, "N": 8 * _log(rng, 32, 512), "D": 32 * _log(rng, 8, 224),
                    "type": rng.choice(["bf16", "bf16", "f32"]),
                    "cap": 0 if rng.random() < 0.7 else 4 * max(1, int(S * K / E * rng.uniform(0.9, 1.5) / 4))}
        w = work(case)
        weights = E * 3 * case["F"] * case["H"] if op == "layer" else E * case.get("N", 0) * case["D"]
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS and weights <= MOST_WEIGHTS:
            return case


# ---------------------------------------------------------------------------
# MXFP4 with elementary operations
# ---------------------------------------------------------------------------

# the value of each code, and of both codes of each byte
_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
_PAIRS = [[_VALUES[i & 15], _VALUES[i >> 4]] for i in range(256)]


def _power(exponent):
    """2 ** exponent for whole exponents in -126 .. 127, from their bits."""
    return ((exponent.to(torch.int32) + 127) << 23).view(F32)


def _scaled(v, exponent):
    """v * 2 ** exponent, rounded once: in two factors, so that neither leaves 32 bits."""
    half = torch.div(exponent, 2, rounding_mode="floor")
    return (v * _power(half)[..., None]) * _power(exponent - half)[..., None]


def _blocks(x):
    """(codes, scale bytes) of x [..., D], D a multiple of 32; the scales as [..., D / 32]."""
    v = x.unflatten(-1, (-1, 32))
    a = v.abs().amax(-1)
    bad = ~torch.isfinite(a)
    e = (torch.frexp(torch.where(bad, 1.0, a))[1] - 3).clamp(-127, 127)
    e = torch.where(a == 0, -127, e)
    m = _scaled(v.abs(), -e)
    c = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0))
    c = c + 8 * torch.signbit(v).to(torch.uint8)
    s = torch.where(bad, 255, e + 127).to(torch.uint8)
    return c.flatten(-2), s


def _pack(x):
    """(codes [..., rows, D / 2], scales [..., D / 128, rows, 4]) of x [..., rows, D]."""
    c, s = _blocks(x)
    s = torch.nn.functional.pad(s, (0, -s.shape[-1] % 4)).unflatten(-1, (-1, 4)).transpose(-2, -3)
    return c[..., ::2] | (c[..., 1::2] << 4), s.contiguous()


def _unpack(codes, scales):
    """The values of [..., rows, D]."""
    table = torch.tensor(_PAIRS, device=codes.device)
    v = table[codes.int()].flatten(-2).unflatten(-1, (-1, 32))
    s = scales.transpose(-2, -3).flatten(-2)[..., :v.shape[-2]]
    v = _scaled(v, s.clamp(max=254).to(torch.int32) - 127)
    return v.masked_fill_((s == 255)[..., None], float("nan")).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _route(case, g):
    """Distinct experts for each token."""
    u = torch.rand(case["S"], case["E"], generator=g, device="cuda")
    return u.topk(case["K"], dim=1).indices.to(torch.int32)


def _plan(case, idx):
    """Counts, first rows, and the row of each (token, k) entry in stable order; -1 for one past its bucket's room."""
    S, E, K, cap = case["S"], case["E"], case["K"], case.get("cap", 0)
    key = idx.flatten().long()
    order = key.argsort(stable=True)
    full = torch.bincount(key, minlength=E)
    first = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    first[1:] = full.cumsum(0)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(S * K, device="cuda")
    slot = rank - first[key]
    if cap:
        cnt, off = full.clamp(max=cap), torch.arange(E + 1, device="cuda") * cap
        row = torch.where(slot < cap, key * cap + slot, -1)
        rows = E * cap
    else:
        cnt, off, row, rows = full, first, rank, S * K + -S * K % 4
    src = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")
    src[torch.where(row >= 0, row, rows)] = torch.arange(S * K, dtype=torch.int32, device="cuda")
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    return {"cnt": cnt.to(torch.int32), "off": off.contiguous(), "tok_map": row.view(S, K).contiguous(),
            "packed_src": src[:rows].contiguous(), "none": none, "dropped": (row < 0).sum().to(torch.int32).view(1),
            "rows": rows, "cap": cap}


def _live(plan):
    """True for the rows that hold a token."""
    r = torch.arange(plan["rows"], device="cuda")
    e = (torch.searchsorted(plan["off"], r, right=True) - 1).clamp(max=plan["cnt"].numel() - 1)
    return r < plan["off"][e] + plan["cnt"][e]


def _weights(E, N, D, g, mx):
    """A layer's weights, of both kinds an expert at a time: no copy in 32 bits of all of them is ever held."""
    if not mx:
        return torch.randn(E, N, D, generator=g, device="cuda", dtype=BF16).mul_(D ** -0.5)
    codes = torch.empty(E, N, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, -(-D // 128), N, 4, dtype=torch.uint8, device="cuda")
    for e in range(E):
        codes[e], scales[e] = _pack(torch.randn(N, D, generator=g, device="cuda").mul_(D ** -0.5))
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "quant":
        D = case["D"]
        if not case["S"]:
            x = torch.randn(case["E"], case["N"], D, generator=g, device="cuda").mul_(D ** -0.5)
            return {"op": "quant", "x": x.to(TYPES[case["type"]]), "plan": None}
        plan = _plan(case, _route(case, g))
        rows = plan["rows"]
        return {"op": op, "x": torch.randn(case["S"], D, generator=g, device="cuda").to(BF16), "plan": plan,
                "codes": torch.zeros(rows, D // 2, dtype=torch.uint8, device="cuda"),
                "scales": torch.zeros(-(-D // 128), rows, 4, dtype=torch.uint8, device="cuda")}
    idx = _route(case, g)
    s = {"op": op, "type": TYPES[case["type"]], "E": case["E"]}
    if op == "layer":
        S, H, F = case["S"], case["H"], case["F"]
        s.update(x=torch.randn(S, H, generator=g, device="cuda").to(BF16), idx=idx,
                 w=torch.randn(S, case["K"], generator=g, device="cuda").softmax(-1))
        s["up"] = _weights(case["E"], 2 * F, H, g, case["weights"] == "mxfp4")
        s["down"] = _weights(case["E"], H, F, g, case["weights"] == "mxfp4")
        return s
    plan = _plan(case, idx)
    rows, D = plan["rows"], case["D"]
    live = _live(plan)
    # rows that no token fills hold what was in memory before
    if op == "act":
        s["x"] = torch.randn(rows, 2 * D, generator=g, device="cuda", dtype=BF16).masked_fill_(~live[:, None], float("nan"))
    else:
        codes, scales = _pack(torch.randn(rows, D, generator=g, device="cuda", dtype=BF16).float())
        codes[~live], scales[:, ~live] = 0x7e, 255
        s["x"] = codes, scales
    s["w"], s["plan"] = _weights(case["E"], case["N"], D, g, True), plan
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(s):
    import combine_moe_plan_02_gb300 as moe
    op = s["op"]
    if op == "quant":
        if s["plan"] is None:
            q = moe.moe_quant_mxfp4(s["x"])
        else:
            q = moe.moe_dispatch_quant_mxfp4(s["x"], s["plan"]["tok_map"], out=moe.MxFp4(s["codes"], s["scales"]))
        return moe.moe_dequant_mxfp4(q)
    if op == "layer":
        up, down = (w if isinstance(w, torch.Tensor) else moe.MxFp4(*w) for w in (s["up"], s["down"]))
        return moe.moe_expert_layer(s["x"], s["idx"], s["w"], up, down, out_dtype=s["type"])
    p = s["plan"]
    if p["cap"]:
        plan = moe.CapacityPlan(p["cnt"], p["off"], p["packed_src"], p["tok_map"], p["none"], p["dropped"], p["cap"])
    else:
        plan = moe.Plan(p["cnt"], p["off"], p["packed_src"], p["tok_map"], p["none"])
    x = moe.moe_swiglu_quant_mxfp4(s["x"]) if op == "act" else moe.MxFp4(*s["x"])
    return moe.moe_expert_gemm_mxfp4(x, moe.MxFp4(*s["w"]), plan, out_dtype=s["type"])


def _quant(s):
    x, p = s["x"].float(), s["plan"]
    v = _unpack(*_pack(x)).to(BF16)
    if p is None:
        return v
    out = torch.zeros(p["rows"], v.shape[1], dtype=BF16, device=v.device)
    out[p["tok_map"].flatten()] = v.repeat_interleave(p["tok_map"].shape[1], 0)
    return out


def _buckets(p):
    """The experts that have rows, their rows in a rectangle, and which places of it hold one."""
    live = p["cnt"].nonzero().flatten()
    cnt = p["cnt"][live]
    places = torch.arange(int(cnt.max()) if live.numel() else 0, device=cnt.device)
    ok = places < cnt[:, None]
    return live, torch.where(ok, p["off"][live][:, None] + places, p["rows"]), ok


def _product(s, x):
    live, at, ok = _buckets(s["plan"])
    w = _unpack(s["w"][0][live], s["w"][1][live])
    y = torch.bmm(torch.where(ok[..., None], x[at.clamp(max=x.shape[0] - 1)], 0.0), w.transpose(1, 2))
    out = y.new_zeros(s["plan"]["rows"] + 1, y.shape[-1])
    out[at.flatten()] = y.flatten(0, 1)
    return out[:-1].to(s["type"])


def _expert(s):
    return _product(s, _unpack(*s["x"]))


def _act(s):
    gate, up = s["x"].float().chunk(2, -1)
    return _product(s, _unpack(*_pack(gate / (1 + torch.exp(-gate)) * up)))


def _layer(s):
    S, K = s["idx"].shape
    key = s["idx"].flatten().long()
    live, at = key.unique(return_inverse=True)  # one expert of `live` for each entry
    slot = (at[:, None] == at).tril(-1).sum(1)  # entries of the same expert before this one
    up, down = (w[live].float() if isinstance(w, torch.Tensor) else _unpack(w[0][live], w[1][live]) for w in (s["up"], s["down"]))
    x = up.new_zeros(live.numel(), int(slot.max()) + 1, up.shape[2])
    x[at, slot] = s["x"].float().repeat_interleave(K, 0)
    gate, lift = torch.bmm(x, up.transpose(1, 2)).chunk(2, -1)
    y = torch.bmm(gate / (1 + torch.exp(-gate)) * lift, down.transpose(1, 2))
    return (y[at, slot].view(S, K, -1) * s["w"][..., None]).sum(1).to(s["type"])


_PLAIN = {"quant": _quant, "expert": _expert, "act": _act, "layer": _layer}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

MX = 17 / 32  # bytes of an element and its share of a scale


def work(case):
    op, E = case["op"], case["E"]
    if op == "quant" and not case["S"]:
        n = float(E * case["N"] * case["D"])
        return {"bytes": n * ((4 if case["type"] == "f32" else 2) + 2), "flops": n}
    S, K = case["S"], case["K"]
    if op == "quant":
        return {"bytes": float(S * case["D"] * 2 + S * K * (8 + case["D"] * 2)), "flops": float(S * case["D"])}
    touched = min(E * (1 - (1 - K / E) ** S), S * K)
    b = 4 if case["type"] == "f32" else 2
    if op == "layer":
        H, F = case["H"], case["F"]
        return {"bytes": touched * 3 * F * H * (2 if case["weights"] == "bf16" else MX) + S * H * (2 + b), "flops": 6.0 * S * K * F * H}
    N, D, rows = case["N"], case["D"], E * case["cap"] if case["cap"] else S * K
    V = min(S * K, rows)
    return {"bytes": V * D * (MX if op == "expert" else 4) + touched * N * D * MX + rows * N * b, "flops": 2.0 * V * N * D}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _nearest(x):
    """x [..., D] as MXFP4 holds it: each value the nearest multiple of a step that its own size and its block's largest set."""
    v = x.double().unflatten(-1, (-1, 32))
    top = v.abs().amax(-1, keepdim=True)
    unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 2).clamp(min=-127))
    r = v / unit
    step = torch.exp2(torch.floor(torch.log2(r.abs().clamp(min=1.0))) - 1)
    return ((r / step).round() * step).clamp(-6, 6).mul(unit).flatten(-2)


def _read(codes, scales, rows=None):
    """The values of a [rows, D] tensor, or of some of its rows."""
    if rows is not None:
        codes, scales = codes[rows], scales[:, rows]
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    e, m = (c >> 1) & 3, c & 1
    v = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * torch.exp2(e.double() - 1)) * (1 - 2 * (c >> 3))
    s = torch.exp2(scales.double() - 127).permute(1, 0, 2).flatten(1).repeat_interleave(32, 1)
    return v * s[:, :v.shape[1]]


def _swish(u):
    gate, up = u.double().chunk(2, -1)
    return gate * torch.sigmoid(gate) * up


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if s["op"] == "quant":
        if s["plan"] is None:
            return torch.stack([_nearest(x) for x in s["x"]])
        out = torch.zeros(s["plan"]["rows"], case["D"], dtype=f64, device="cuda")
        v = _nearest(s["x"])
        for k in range(case["K"]):
            out[s["plan"]["tok_map"][:, k]] = v
        return out
    if s["op"] == "layer":
        out = torch.zeros(case["S"], case["H"], dtype=f64, device="cuda")
        for e in s["idx"].unique().tolist():
            t, k = (s["idx"] == e).nonzero(as_tuple=True)
            up, down = (w[e].double() if isinstance(w, torch.Tensor) else _read(w[0][e], w[1][e]) for w in (s["up"], s["down"]))
            y = _swish(s["x"][t].double() @ up.T) @ down.T
            out.index_add_(0, t, y * s["w"][t, k].double()[:, None])
        return out
    p = s["plan"]
    cnt, off = p["cnt"].tolist(), p["off"].tolist()
    out = torch.zeros(p["rows"], case["N"], dtype=f64, device="cuda")
    for e in range(case["E"]):
        a, z = off[e], off[e] + cnt[e]
        if a < z:
            at = torch.arange(a, z, device="cuda")
            x = _nearest(_swish(s["x"][at])) if s["op"] == "act" else _read(*s["x"], at)
            out[a:z] = x @ _read(s["w"][0][e], s["w"][1][e]).T
    return out
