"""Operators of a trained or served expert layer, and the cases that measure them.

  combine_grad  the gradient of the weighted combine: of the expert rows and of the routing weights
  expert        the experts' product over packed rows, y = x w[e]^T
  expert_dx     its gradient for the rows, dx = dy w[e]
  expert_dw     its gradient for the weights, dw[e] = dy^T x over the rows of e
  clip          the global norm over many gradients, and the gradients scaled to a limit

`run` computes them with elementary torch operations in 32 bits, or with the package's own calls where `own` is set.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # training, the benchmark's batch: the backward pass of the combine behind 64 experts
        {"name": "combine_grad_4096x7168", "op": "combine_grad", "S": 4096, "H": 7168, "E": 64, "K": 8, "type": "bf16",
         "dtype": "bf16", "cap": 0, "route": "uniform", "lost": 0.0},
        # training with f32 rows, padded buckets and entries that the router left out
        {"name": "combine_grad_f32_padded", "op": "combine_grad", "S": 4096, "H": 4096, "E": 64, "K": 8, "type": "f32",
         "dtype": "f32", "cap": 576, "route": "uniform", "lost": 0.02},
        # a few tokens (adapting on single requests): the call's latency
        {"name": "combine_grad_16x6144", "op": "combine_grad", "S": 16, "H": 6144, "E": 256, "K": 8, "type": "bf16",
         "dtype": "f32", "cap": 0, "route": "uniform", "lost": 0.0},
        # training and prefill: the up product of the benchmark's batch, 512 rows an expert on average
        {"name": "expert_32768x7168x2048", "op": "expert", "S": 4096, "E": 64, "K": 8, "N": 2048, "D": 7168, "type": "bf16",
         "cap": 0, "route": "uniform", "lost": 0.0},
        # serving, one token: eight experts with one row each, bound by their weights
        {"name": "expert_1_token", "op": "expert", "S": 1, "E": 256, "K": 8, "N": 2048, "D": 6144, "type": "bf16",
         "cap": 0, "route": "uniform", "lost": 0.0},
        # serving, a batch of 128 decoded tokens: nearly all experts with a few rows each
        {"name": "expert_128_tokens", "op": "expert", "S": 128, "E": 256, "K": 8, "N": 2048, "D": 6144, "type": "bf16",
         "cap": 0, "route": "uniform", "lost": 0.0},
        # training, the same batch: the gradient for the rows
        {"name": "expert_dx_32768x2048x7168", "op": "expert_dx", "S": 4096, "E": 64, "K": 8, "N": 2048, "D": 7168, "type": "bf16",
         "cap": 0, "route": "uniform", "lost": 0.0},
        # a small odd-sized layer with padded buckets and f32 output
        {"name": "expert_dx_odd_padded", "op": "expert_dx", "S": 1001, "E": 24, "K": 3, "N": 1048, "D": 1416, "type": "f32",
         "cap": 173, "route": "uniform", "lost": 0.05},
        # training, the same batch: the gradient for the weights, in 32 bits
        {"name": "expert_dw_64x2048x7168", "op": "expert_dw", "S": 4096, "E": 64, "K": 8, "N": 2048, "D": 7168, "type": "f32",
         "cap": 0, "route": "uniform", "lost": 0.0},
        # skewed routing: some experts with many rows, some with none
        {"name": "expert_dw_skewed", "op": "expert_dw", "S": 1024, "E": 256, "K": 8, "N": 1024, "D": 2048, "type": "bf16",
         "cap": 0, "route": "zipf", "lost": 0.0},
        # an optimiser step over an expert layer's gradients in 32 bits: two large tensors and the small ones
        {"name": "clip_f32_layer", "op": "clip", "count": 12, "largest": 469762048, "type": "f32", "limit": 0.5},
        # a small model's gradients: many odd-sized tensors of both types, bound by latency
        {"name": "clip_small_mixed", "op": "clip", "count": 40, "largest": 50001, "type": "mixed", "limit": 0.5},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


MOST_BYTES, MOST_FLOPS = 4.5e9, 9.0e11


def draw(rng):
    while True:
        op = rng.choice(["combine_grad", "expert", "expert_dx", "expert_dw", "clip"])
        if op == "clip":
            case = {"op": op, "count": rng.randint(1, 48), "largest": _log(rng, 1000, 400000000),
                    "type": rng.choice(["f32", "bf16", "mixed"]), "limit": rng.choice([0.1, 0.5, 2.0])}
        else:
            S, E = _log(rng, 1, 4096), rng.choice([8, 24, 64, 128, 256])
            K = rng.randint(1, 8)
            case = {"op": op, "S": S, "E": E, "K": K, "type": rng.choice(["bf16", "f32"]),
                    "cap": 0 if rng.random() < 0.7 else max(1, int(S * K / E * rng.uniform(0.9, 1.5))),
                    "route": "zipf" if rng.random() < 0.2 and S * K <= 8192 else "uniform",
                    "lost": rng.choice([0.0, 0.0, 0.03])}
            if op == "combine_grad":
                case.update(H=8 * _log(rng, 32, 896), dtype=rng.choice(["bf16", "f32"]))
            else:
                case.update(N=8 * _log(rng, 32, 320), D=8 * _log(rng, 32, 896))
                if case["type"] == "f32" and op == "expert" and rng.random() < 0.5:
                    case["type"] = "bf16"
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS:
            return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _route(case, g):
    """Distinct experts for each token, and some entries that go nowhere (-1)."""
    S, E, K = case["S"], case["E"], case["K"]
    u = torch.rand(S, E, generator=g, device="cuda").clamp_(min=1e-9).log_().neg_()
    if case["route"] == "zipf":
        p = torch.arange(1, E + 1, device="cuda", dtype=F32).pow(-1.2)
        u = u / p[torch.randperm(E, generator=g, device="cuda")]
    idx = u.topk(K, dim=1, largest=False).indices.to(torch.int32)
    if case["lost"] > 0:
        idx[torch.rand(S, K, generator=g, device="cuda") < case["lost"]] = -1
    return idx


def _plan(case, idx):
    """Counts, first rows, and the row of each (token, k) entry in stable order; -1 for one that has none."""
    S, E, K, cap = case["S"], case["E"], case["K"], case["cap"]
    flat = idx.flatten().long()
    key = torch.where(flat < 0, E, flat)
    order = key.argsort(stable=True)
    full = torch.bincount(key, minlength=E + 1)[:E]
    first = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    first[1:] = full.cumsum(0)
    rank = torch.empty_like(order)
    rank[order] = torch.arange(S * K, device="cuda")
    slot = rank - first[key]
    if cap:
        cnt, off = full.clamp(max=cap), torch.arange(E + 1, device="cuda") * cap
        row = torch.where((flat >= 0) & (slot < cap), key * cap + slot, -1)
        rows = E * cap
    else:
        cnt, off = full, first
        row = torch.where(flat >= 0, rank, -1)
        rows = S * K
    src = torch.zeros(rows + 1, dtype=torch.int32, device="cuda")
    src[torch.where(row >= 0, row, rows)] = torch.arange(S * K, dtype=torch.int32, device="cuda")
    return {"cnt": cnt.to(torch.int32), "off": off.contiguous(), "tok_map": row.view(S, K).contiguous(),
            "packed_src": src[:rows].contiguous(), "invalid": (flat < 0).sum().to(torch.int32).view(1),
            "dropped": ((flat >= 0) & (row < 0)).sum().to(torch.int32).view(1), "rows": rows, "cap": cap}


def _live(plan):
    """True for the rows that hold a token."""
    r = torch.arange(plan["rows"], device="cuda")
    e = (torch.searchsorted(plan["off"], r, right=True) - 1).clamp(max=plan["cnt"].numel() - 1)
    return r < plan["off"][e] + plan["cnt"][e]


def _rows(plan, width, dtype, g, scale=1.0):
    """Packed rows; those that no token fills hold what was in memory before, here NaN."""
    x = torch.randn(plan["rows"], width, generator=g, device="cuda", dtype=dtype).mul_(scale)
    return x.masked_fill_(~_live(plan)[:, None], float("nan"))


def _sizes(case):
    rng = np.random.RandomState(case["count"] * 7919 + case["largest"] % 65521)
    n, big = case["count"], case["largest"]
    sizes = [big] + [max(1, int(big * rng.rand() ** 6)) for _ in range(n - 1)]
    if n > 2:
        sizes[1] = max(1, big // 2 - 1)
    types = [F32 if case["type"] == "f32" or (case["type"] == "mixed" and i % 2) else BF16 for i in range(n)]
    return list(zip(sizes, types))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op = case["op"]
    if op == "clip":
        grads = [torch.randn(n, generator=g, device="cuda", dtype=t).mul_(0.01) for n, t in _sizes(case)]
        total = sum(x.numel() for x in grads)
        return {"op": op, "grads": grads, "out": [torch.empty_like(x) for x in grads], "limit": case["limit"] * 0.01 * math.sqrt(total)}
    idx = _route(case, g)
    plan = _plan(case, idx)
    s = {"op": op, "plan": plan, "type": TYPES[case["type"]]}
    if op == "combine_grad":
        S, H, K = case["S"], case["H"], case["K"]
        s["w"] = torch.randn(S, K, generator=g, device="cuda").softmax(-1)
        s["y"] = _rows(plan, H, s["type"], g)
        s["dout"] = torch.randn(S, H, generator=g, device="cuda", dtype=TYPES[case["dtype"]]).mul_(0.01)
        return s
    E, N, D = case["E"], case["N"], case["D"]
    if op != "expert_dw":
        s["w"] = torch.randn(E, N, D, generator=g, device="cuda", dtype=BF16).mul_(D ** -0.5)
    if op != "expert_dx":
        s["x"] = _rows(plan, D, BF16, g)
    if op != "expert":
        s["dy"] = _rows(plan, N, BF16, g, 0.01)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _PLAIN[state["op"]](state)


def _run_own(s):
    import combine_moe_plan_02_gb300 as moe
    op = s["op"]
    if op == "clip":
        return [moe.moe_clip_grad_norm(s["grads"], s["limit"], out=s["out"]), s["out"]]
    p = s["plan"]
    if p["cap"]:
        plan = moe.CapacityPlan(p["cnt"], p["off"], p["packed_src"], p["tok_map"], p["invalid"], p["dropped"], p["cap"])
    else:
        plan = moe.Plan(p["cnt"], p["off"], p["packed_src"], p["tok_map"], p["invalid"])
    if op == "combine_grad":
        return list(moe.moe_combine_backward(s["dout"], s["y"], s["w"], plan))
    if op == "expert":
        return moe.moe_expert_gemm(s["x"], s["w"], plan, out_dtype=s["type"])
    if op == "expert_dx":
        return moe.moe_expert_gemm_dgrad(s["dy"], s["w"], plan, out_dtype=s["type"])
    return moe.moe_expert_gemm_wgrad(s["dy"], s["x"], plan, out_dtype=s["type"])


def _combine_grad(s):
    p, w, y, dout = s["plan"], s["w"], s["y"], s["dout"].float()
    S, K = w.shape
    ok = p["tok_map"] >= 0
    at = torch.where(ok, p["tok_map"], p["rows"])
    got = y[at.clamp(max=p["rows"] - 1)].float()
    dw = torch.where(ok, (got * dout[:, None]).sum(-1), 0.0)
    src = torch.full((p["rows"] + 1,), -1, dtype=torch.int64, device=y.device)
    src[at.flatten()] = torch.arange(S * K, device=y.device)
    src = src[:-1]
    e = src.clamp(min=0)
    dy = torch.where((src >= 0)[:, None], w.flatten()[e][:, None] * dout[e // K], 0.0)
    return [dy.to(y.dtype), dw]


def _buckets(p):
    """The experts that have rows, their rows in a rectangle, and which places of it hold one."""
    live = p["cnt"].nonzero().flatten()
    cnt = p["cnt"][live]
    places = torch.arange(int(cnt.max()) if live.numel() else 0, device=cnt.device)
    ok = places < cnt[:, None]
    return live, torch.where(ok, p["off"][live][:, None] + places, p["rows"]), ok


def _take(x, at, ok):
    return torch.where(ok[..., None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)


def _put(p, at, values, dtype):
    out = values.new_zeros(p["rows"] + 1, values.shape[-1])
    out[at.flatten()] = values.flatten(0, 1)
    return out[:-1].to(dtype)


def _expert(s):
    live, at, ok = _buckets(s["plan"])
    y = torch.bmm(_take(s["x"], at, ok), s["w"][live].float().transpose(1, 2))
    return _put(s["plan"], at, y, s["type"])


def _expert_dx(s):
    live, at, ok = _buckets(s["plan"])
    return _put(s["plan"], at, torch.bmm(_take(s["dy"], at, ok), s["w"][live].float()), s["type"])


def _expert_dw(s):
    live, at, ok = _buckets(s["plan"])
    dy, x = _take(s["dy"], at, ok), _take(s["x"], at, ok)
    dw = torch.zeros(s["plan"]["cnt"].numel(), dy.shape[-1], x.shape[-1], dtype=s["type"], device=x.device)
    dw[live] = torch.bmm(dy.transpose(1, 2), x).to(s["type"])
    return dw


def _clip(s):
    norm = torch.stack([g.float().square().sum() for g in s["grads"]]).sum().sqrt().view(1)
    c = (s["limit"] / (norm + 1e-6)).clamp(max=1.0)
    return [norm, [(g.float() * c).to(g.dtype) for g in s["grads"]]]


_PLAIN = {"combine_grad": _combine_grad, "expert": _expert, "expert_dx": _expert_dx, "expert_dw": _expert_dw, "clip": _clip}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _reach(case):
    """Entries with a row, and experts with one, as expected over the draws of a case."""
    S, E, K = case["S"], case["E"], case["K"]
    n = S * K * (1.0 - case["lost"])
    if case["cap"]:
        n = min(n, float(E * case["cap"]))
    if case["route"] == "zipf":
        p = np.arange(1, E + 1) ** -1.2
        touched = float(np.sum(1 - (1 - p / p.sum()) ** (S * K)))
    else:
        touched = E * (1 - (1 - K / E) ** S)
    return n, max(1.0, min(touched, n))


def work(case):
    op = case["op"]
    if op == "clip":
        n = [(k, 4 if t is F32 else 2) for k, t in _sizes(case)]
        return {"bytes": float(sum(2 * k * b for k, b in n)), "flops": float(sum(3 * k for k, _ in n))}
    V, touched = _reach(case)
    S, E, K = case["S"], case["E"], case["K"]
    R = E * case["cap"] if case["cap"] else S * K
    b = 4 if case["type"] == "f32" else 2
    if op == "combine_grad":
        H, d = case["H"], 4 if case["dtype"] == "f32" else 2
        return {"bytes": float(S * H * d + V * H * b + R * H * b + S * K * 16), "flops": 3.0 * V * H}
    N, D = case["N"], case["D"]
    flops = 2.0 * V * N * D
    if op == "expert":
        moved = V * D * 2 + touched * N * D * 2 + R * N * b
    elif op == "expert_dx":
        moved = V * N * 2 + touched * N * D * 2 + R * D * b
    else:
        moved = V * (N + D) * 2 + E * N * D * b
    return {"bytes": float(moved), "flops": flops}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "clip":
        squares = 0.0
        for g in s["grads"]:
            for part in g.split(1 << 26):
                squares += float(part.to(f64).pow(2).sum())
        norm = math.sqrt(squares)
        c = min(1.0, s["limit"] / (norm + 1e-6))
        if sum(g.numel() for g in s["grads"]) > 1 << 31:
            return [torch.tensor([norm], dtype=f64), [None] * len(s["grads"])]
        return [torch.tensor([norm], dtype=f64, device="cuda"), [g.to(f64) * c for g in s["grads"]]]
    p = s["plan"]
    if case["op"] == "combine_grad":
        S, K = s["w"].shape
        dy = torch.zeros(p["rows"], case["H"], dtype=f64, device="cuda")
        dw = torch.zeros(S, K, dtype=f64, device="cuda")
        for k in range(K):
            t = (p["tok_map"][:, k] >= 0).nonzero().flatten()
            r = p["tok_map"][t, k]
            d = s["dout"][t].to(f64)
            dy[r] = d * s["w"][t, k, None].to(f64)
            dw[t, k] = torch.einsum("th,th->t", d, s["y"][r].to(f64))
        return [dy, dw]
    cnt, off = p["cnt"].tolist(), p["off"].tolist()
    if case["op"] == "expert_dw":
        out = torch.zeros(case["E"], case["N"], case["D"], dtype=f64, device="cuda")
    else:
        out = torch.zeros(p["rows"], case["N"] if case["op"] == "expert" else case["D"], dtype=f64, device="cuda")
    for e in range(case["E"]):
        a, z = off[e], off[e] + cnt[e]
        if a == z:
            continue
        if case["op"] == "expert":
            out[a:z] = s["x"][a:z].to(f64) @ s["w"][e].to(f64).T
        elif case["op"] == "expert_dx":
            out[a:z] = s["dy"][a:z].to(f64) @ s["w"][e].to(f64)
        else:
            out[e] = s["dy"][a:z].to(f64).T @ s["x"][a:z].to(f64)
    return out
