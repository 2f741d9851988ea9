"""Single-GPU MoE token dispatch and combine for GB300 (sm_103a).

Python binding of the C ABI in include/moe_plan.h: each function checks and
marshals torch tensors (device pointers, sizes, the current stream) into one
C call; all work runs in the library's CUDA kernels.  Output tensors are
allocated with torch when not passed in, as memory of the stream that the call
runs on.

    plan  = moe_plan(topk_idx, E)                  # counts, offsets, maps
    px, _ = moe_dispatch(x, plan.tok_map)          # packed_x[off[e] + slot]
    y     = experts(px, plan)                      # caller's expert stage
    out   = moe_combine(y, topk_w, plan.tok_map)   # sum_k w * y[tok_map]

The experts' products and the way back:

    y      = moe_expert_gemm(px, w, plan)              # y[r] = w[e] px[r]
    dy, dw = moe_combine_backward(dout, y, topk_w, plan)
    dpx    = moe_expert_gemm_dgrad(dy, w, plan)
    dwe    = moe_expert_gemm_wgrad(dy, px, plan)
    dx     = moe_dispatch_backward(dpx, plan)          # sum_k dpx[tok_map]
    norm   = moe_clip_grad_norm([dwe, ...], 1.0)       # in place
"""
from __future__ import annotations

import ctypes
from array import array
from contextlib import nullcontext
from operator import attrgetter
from typing import NamedTuple, Optional, Sequence, Union

import torch

from . import _abi
from ._abi import MoeError, MOE_BF16, MOE_F32, MOE_FP8_E4M3  # noqa: F401

__all__ = [
    "moe_plan", "moe_group_plan", "moe_dispatch", "moe_plan_dispatch", "moe_dispatch_dedup", "moe_dispatch_quant_fp8",
    "moe_combine", "moe_combine_fold",
    "moe_combine_dedup", "moe_plan_workspace_size", "moe_group_plan_workspace_size",
    "moe_combine_backward", "moe_dispatch_backward", "moe_expert_gemm", "moe_expert_gemm_dgrad",
    "moe_expert_gemm_wgrad", "moe_grad_norm", "moe_clip_grad_norm",
    "moe_device_errors", "moe_plan_capacity", "Plan", "GroupPlan", "CapacityPlan", "MoeError",
    "MoeOp", "Routing", "lib",
]


def lib():
    return _abi.load()


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype in (torch.float8_e4m3fn, torch.uint8):
        return MOE_FP8_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


_TORCH_DT = {MOE_BF16: torch.bfloat16, MOE_F32: torch.float32}


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


# the raw handle of a device's current stream without building a Stream
# object (about 0.2 against 2.9 us per call on a Grace host)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, like: Optional[torch.Tensor]) -> int:
    """The stream to enqueue on: the given one, else the current stream of
    the device that holds `like`."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(like.get_device())
        return torch.cuda.current_stream(like.device).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream, device: torch.device):
    """The context in which what a call allocates or fills for itself belongs
    to the stream that the call runs on.  torch hands a freed block on in the
    order of the stream it was allocated on, so a temporary of another stream
    may still be in use when it is handed out, or be handed on while the call
    uses it."""
    if stream is None:
        return _AS_IT_IS
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream, None), device=device)
    return torch.cuda.stream(stream)


_AS_IT_IS = nullcontext()


def _empty(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """A new output or workspace of a call on `stream`: the stream's own memory,
    which is not handed on before what the current stream does with it until
    then is done."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    if here.cuda_stream == _stream(stream, None):
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream, device):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(here)
    return t


class Plan(NamedTuple):
    cnt: torch.Tensor          # int32 [E]
    off: torch.Tensor          # int64 [E+1]
    packed_src: torch.Tensor   # int32 [S*K] (first off[E] valid)
    tok_map: torch.Tensor      # int64 [S, K]
    n_invalid: torch.Tensor    # int32 [1]


class GroupPlan(NamedTuple):
    gcnt: torch.Tensor         # int32 [G]
    goff: torch.Tensor         # int64 [G+1]
    gtok_map: torch.Tensor     # int64 [S, K]
    grp_src: torch.Tensor      # int32 [max_rows]
    grp_tok_map: torch.Tensor  # int64 [max_rows, K]
    group_size: int

    @property
    def G(self) -> int:
        return self.gcnt.numel()

    @property
    def max_rows(self) -> int:
        return self.grp_src.numel()


def moe_plan_workspace_size(S: int, K: int, E: int) -> int:
    return int(lib().moe_plan_workspace_size(S, K, E))


def moe_group_plan_workspace_size(S: int, K: int, E: int, group_size: int) -> int:
    return int(lib().moe_group_plan_workspace_size(S, K, E, group_size))


def _workspace(nbytes: int, device, ws: Optional[torch.Tensor], stream):
    if nbytes == 0:
        return ws
    if ws is None or ws.numel() * ws.element_size() < nbytes:
        ws = _empty(nbytes, torch.uint8, device, stream)
    return ws


def moe_plan(topk_idx: torch.Tensor, E: int, *, out: Optional[Plan] = None,
             workspace: Optional[torch.Tensor] = None, stream=None) -> Plan:
    """Histogram, exclusive scan and stable (token, k)-order slot map."""
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise TypeError("topk_idx must be int32 [S, K]")
    S, K = topk_idx.shape
    dev = topk_idx.device
    if out is None:
        out = Plan(_empty(E, torch.int32, dev, stream),
                   _empty(E + 1, torch.int64, dev, stream),
                   _empty(max(S * K, 1), torch.int32, dev, stream),
                   _empty((S, K), torch.int64, dev, stream),
                   _empty(1, torch.int32, dev, stream))
    L = lib()
    nws = int(L.moe_plan_workspace_size(S, K, E))
    ws = _workspace(nws, dev, workspace, stream)
    _abi.check("moe_plan", L.moe_plan(
        _ptr(topk_idx), S, K, E, _ptr(out.cnt), _ptr(out.off), _ptr(out.packed_src),
        _ptr(out.tok_map), _ptr(out.n_invalid), _ptr(ws), nws, _stream(stream, topk_idx)))
    return out


class CapacityPlan(NamedTuple):
    cnt: torch.Tensor          # int32 [E] rows filled per bucket
    off: torch.Tensor          # int64 [E+1] = e * capacity
    packed_src: torch.Tensor   # int32 [E*capacity]
    tok_map: torch.Tensor      # int64 [S, K], -1 for dropped entries
    n_invalid: torch.Tensor    # int32 [1]
    n_dropped: torch.Tensor    # int32 [1]
    capacity: int


def moe_plan_capacity(topk_idx: torch.Tensor, E: int, capacity: int, *,
                      out: Optional[CapacityPlan] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> CapacityPlan:
    """Plan into padded buckets of `capacity` rows; entries past a bucket's
    capacity (later tokens first to go) are dropped to -1."""
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise TypeError("topk_idx must be int32 [S, K]")
    S, K = topk_idx.shape
    dev = topk_idx.device
    if out is None:
        out = CapacityPlan(_empty(E, torch.int32, dev, stream),
                           _empty(E + 1, torch.int64, dev, stream),
                           _empty(E * capacity, torch.int32, dev, stream),
                           _empty((S, K), torch.int64, dev, stream),
                           _empty(1, torch.int32, dev, stream),
                           _empty(1, torch.int32, dev, stream), capacity)
    L = lib()
    nws = int(L.moe_plan_workspace_size(S, K, E))
    ws = _workspace(nws, dev, workspace, stream)
    _abi.check("moe_plan_capacity", L.moe_plan_capacity(
        _ptr(topk_idx), S, K, E, capacity, _ptr(out.cnt), _ptr(out.off), _ptr(out.packed_src),
        _ptr(out.tok_map), _ptr(out.n_invalid), _ptr(out.n_dropped), _ptr(ws), nws,
        _stream(stream, topk_idx)))
    return out


def moe_group_plan(topk_idx: torch.Tensor, tok_map: torch.Tensor, E: int, group_size: int, *,
                   out: Optional[GroupPlan] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> GroupPlan:
    """Dedup plan: one group row per (token, virtual group) it reaches."""
    S, K = topk_idx.shape
    G = E // group_size
    dev = topk_idx.device
    if out is None:
        rmax = max(S * min(K, G), 1)
        out = GroupPlan(_empty(G, torch.int32, dev, stream),
                        _empty(G + 1, torch.int64, dev, stream),
                        _empty((S, K), torch.int64, dev, stream),
                        _empty(rmax, torch.int32, dev, stream),
                        _empty((rmax, K), torch.int64, dev, stream),
                        group_size)
    L = lib()
    nws = int(L.moe_group_plan_workspace_size(S, K, E, group_size))
    ws = _workspace(nws, dev, workspace, stream)
    _abi.check("moe_group_plan", L.moe_group_plan(
        _ptr(topk_idx), _ptr(tok_map), S, K, E, group_size, _ptr(out.gcnt), _ptr(out.goff),
        _ptr(out.gtok_map), _ptr(out.grp_src), _ptr(out.grp_tok_map), _ptr(ws), nws,
        _stream(stream, topk_idx)))
    return out


def moe_dispatch(x: torch.Tensor, tok_map: torch.Tensor, *, packed_x: Optional[torch.Tensor] = None,
                 x_scales: Optional[torch.Tensor] = None,
                 packed_scales: Optional[torch.Tensor] = None, stream=None):
    """packed_x[tok_map[s,k]] = x[s] (and the scale rows with them).
    Returns (packed_x, packed_scales)."""
    S, H = x.shape
    K = tok_map.shape[1]
    if packed_x is None:
        packed_x = _empty((S * K, H), x.dtype, x.device, stream)
    n_scales = 0
    if x_scales is not None:
        n_scales = x_scales.shape[1]
        if packed_scales is None:
            packed_scales = _empty((S * K, n_scales), torch.float32, x.device, stream)
    if packed_scales is not None and packed_scales.shape[0] < packed_x.shape[0]:
        raise ValueError("packed_scales needs as many rows as packed_x")
    _abi.check("moe_dispatch", lib().moe_dispatch(
        _ptr(x), S, H, _dt(x), K, _ptr(tok_map), _ptr(packed_x), packed_x.shape[0],
        _ptr(x_scales), n_scales, _ptr(packed_scales), _stream(stream, x)))
    return packed_x, packed_scales


_fused_max_cache: list = []


def _fused_max(L) -> int:
    """Entries up to which moe_plan_dispatch runs as one launch (a constant
    of the loaded library)."""
    if not _fused_max_cache:
        _fused_max_cache.append(int(L.moe_plan_dispatch_fused_max()))
    return _fused_max_cache[0]


def moe_plan_dispatch(topk_idx: torch.Tensor, x: torch.Tensor, E: int, *,
                      x_scales: Optional[torch.Tensor] = None, out: Optional[Plan] = None,
                      packed_x: Optional[torch.Tensor] = None,
                      packed_scales: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """moe_plan followed by moe_dispatch, in one launch for small batches.
    Returns (plan, packed_x, packed_scales)."""
    if topk_idx.dtype != torch.int32 or topk_idx.dim() != 2:
        raise TypeError("topk_idx must be int32 [S, K]")
    S, K = topk_idx.shape
    H = x.shape[1]
    dev = topk_idx.device
    if out is None:
        out = Plan(_empty(E, torch.int32, dev, stream),
                   _empty(E + 1, torch.int64, dev, stream),
                   _empty(max(S * K, 1), torch.int32, dev, stream),
                   _empty((S, K), torch.int64, dev, stream),
                   _empty(1, torch.int32, dev, stream))
    if packed_x is None:
        packed_x = _empty((max(S * K, 1), H), x.dtype, dev, stream)
    n_scales = 0
    if x_scales is not None:
        n_scales = x_scales.shape[1]
        if packed_scales is None:
            packed_scales = _empty((packed_x.shape[0], n_scales), torch.float32, dev, stream)
    if packed_scales is not None and packed_scales.shape[0] < packed_x.shape[0]:
        raise ValueError("packed_scales needs as many rows as packed_x")
    L = lib()
    nws = 0
    if S * K > _fused_max(L):
        nws = int(L.moe_plan_workspace_size(S, K, E))
    ws = _workspace(nws, dev, workspace, stream)
    _abi.check("moe_plan_dispatch", L.moe_plan_dispatch(
        _ptr(topk_idx), _ptr(x), S, H, _dt(x), K, E, _ptr(x_scales), n_scales, _ptr(out.cnt),
        _ptr(out.off), _ptr(out.packed_src), _ptr(out.tok_map), _ptr(out.n_invalid),
        _ptr(packed_x), packed_x.shape[0], _ptr(packed_scales), _ptr(ws), nws,
        _stream(stream, topk_idx)))
    return out, packed_x, packed_scales


def moe_dispatch_quant_fp8(x: torch.Tensor, tok_map: torch.Tensor, *, block: int = 128,
                           packed_q: Optional[torch.Tensor] = None,
                           packed_scales: Optional[torch.Tensor] = None, stream=None):
    """bf16 rows -> blockwise E4M3 codes + f32 scales in the K packed rows of
    each token.  Returns (packed_q as float8_e4m3fn, packed_scales)."""
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    S, H = x.shape
    K = tok_map.shape[1]
    if packed_q is None:
        packed_q = _empty((S * K, H), torch.float8_e4m3fn, x.device, stream)
    if packed_scales is None:
        packed_scales = _empty((S * K, H // block), torch.float32, x.device, stream)
    rows = min(packed_q.shape[0], packed_scales.shape[0])
    _abi.check("moe_dispatch_quant_fp8", lib().moe_dispatch_quant_fp8(
        _ptr(x), S, H, K, _ptr(tok_map), block, _ptr(packed_q), _ptr(packed_scales), rows,
        _stream(stream, x)))
    return packed_q, packed_scales


def moe_dispatch_dedup(x: torch.Tensor, gp: GroupPlan, *, packed_x: Optional[torch.Tensor] = None,
                       grp_x: Optional[torch.Tensor] = None, stream=None):
    """Copy each token once per group row, then expand per expert.
    Returns (grp_x, packed_x)."""
    S, H = x.shape
    K = gp.gtok_map.shape[1]
    if grp_x is None:
        grp_x = _empty((gp.max_rows, H), x.dtype, x.device, stream)
    if packed_x is None:
        packed_x = _empty((S * K, H), x.dtype, x.device, stream)
    _abi.check("moe_dispatch_dedup", lib().moe_dispatch_dedup(
        _ptr(x), S, H, _dt(x), K, gp.G, _ptr(gp.goff), _ptr(gp.grp_src), _ptr(gp.grp_tok_map),
        _ptr(gp.gtok_map), gp.max_rows, _ptr(grp_x), _ptr(packed_x), packed_x.shape[0],
        _stream(stream, x)))
    return grp_x, packed_x


def moe_combine(y: torch.Tensor, topk_w: torch.Tensor, tok_map: torch.Tensor, *,
                out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """out[s] = sum_k topk_w[s,k] * y[tok_map[s,k]] in f32, increasing k."""
    S, K = tok_map.shape
    H = y.shape[1]
    if out is None:
        out = _empty((S, H), out_dtype, y.device, stream)
    _abi.check("moe_combine", lib().moe_combine(
        _ptr(y), y.shape[0], _dt(y), _ptr(topk_w), _ptr(tok_map), S, H, K, _ptr(out), _dt(out),
        _stream(stream, y)))
    return out


def moe_combine_dedup(y: torch.Tensor, topk_w: torch.Tensor, gp: GroupPlan, *,
                      out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                      gtok: Optional[torch.Tensor] = None, stream=None):
    """Per group row weighted sum, then per token unweighted sum of its group
    rows.  Returns (gtok, out)."""
    S, K = gp.gtok_map.shape
    H = y.shape[1]
    if gtok is None:
        gtok = _empty((gp.max_rows, H), torch.float32, y.device, stream)
    if out is None:
        out = _empty((S, H), out_dtype, y.device, stream)
    _abi.check("moe_combine_dedup", lib().moe_combine_dedup(
        _ptr(y), y.shape[0], _dt(y), _ptr(topk_w), _ptr(gp.goff), gp.G, _ptr(gp.grp_src),
        _ptr(gp.grp_tok_map), _ptr(gp.gtok_map), S, H, K, gp.max_rows, _ptr(gtok), _ptr(out),
        _dt(out), _stream(stream, y)))
    return gtok, out


def moe_combine_fold(y: torch.Tensor, topk_w: Optional[torch.Tensor], token_map: torch.Tensor,
                     *, weighted: bool = False, fold: bool = True,
                     out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                     out_weights: Optional[torch.Tensor] = None, stream=None):
    """out[s] = sum over valid k of (topk_w[s,k] if weighted else 1) *
    y[token_map[s,k]]; out_weights[s,i] = sum over valid k of topk_w[s,i].
    token_map is tok_map (packed rows) or gtok_map (group rows).
    Returns (out, out_weights or None)."""
    S, K = token_map.shape
    H = y.shape[1]
    if out is None:
        out = _empty((S, H), out_dtype, y.device, stream)
    if fold and out_weights is None:
        out_weights = _empty((S, K), torch.float32, y.device, stream)
    if not fold:
        out_weights = None
    _abi.check("moe_combine_fold", lib().moe_combine_fold(
        _ptr(y), y.shape[0], _dt(y), _ptr(topk_w), int(weighted), _ptr(token_map), S, H, K,
        _ptr(out), _dt(out), _ptr(out_weights), _stream(stream, y)))
    return out, out_weights


def _check_plan(plan, E: int, tok_map: bool = False):
    """The kernels read cnt, off and tok_map as these types, and so many of
    them."""
    cnt, off = plan.cnt, plan.off
    if cnt.dtype != torch.int32 or off.dtype != torch.int64:
        raise TypeError("the plan's cnt must be int32 and its off int64")
    if cnt.numel() != E or off.numel() != E + 1:
        raise ValueError("the plan must have cnt [E] and off [E + 1] of as many experts")
    if tok_map and (plan.tok_map.dtype != torch.int64 or plan.tok_map.dim() != 2):
        raise TypeError("the plan's tok_map must be int64 [S, K]")


def moe_dispatch_backward(dpacked: torch.Tensor, plan: Union[Plan, CapacityPlan], *,
                          out_dtype: torch.dtype = torch.bfloat16,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of moe_dispatch: dx[s] = sum over valid k of
    dpacked[tok_map[s,k]], in f32, increasing k."""
    _check_plan(plan, plan.cnt.numel(), True)
    if dpacked.dim() != 2:
        raise ValueError("dpacked must be [rows, H]")
    if out is not None and out.shape != (plan.tok_map.shape[0], dpacked.shape[1]):
        raise ValueError("out must be [S, H]")
    return moe_combine_fold(dpacked, None, plan.tok_map, weighted=False, fold=False,
                            out_dtype=out_dtype, out=out, stream=stream)[0]


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, topk_w: torch.Tensor,
                         plan: Union[Plan, CapacityPlan], *, dy: Optional[torch.Tensor] = None,
                         dw: Optional[torch.Tensor] = None, stream=None):
    """Gradient of moe_combine: dy[tok_map[s,k]] = topk_w[s,k] * dout[s], zero
    on rows that no entry fills, and dw[s,k] = <dout[s], y[tok_map[s,k]]>,
    zero without a row.  Returns (dy in y's type, dw f32 [S, K])."""
    _check_plan(plan, plan.cnt.numel(), True)
    S, K = shape = plan.tok_map.shape
    if y.dim() != 2 or dout.shape != (S, y.shape[1]):
        raise ValueError("dout must be [S, H] and y [rows, H]")
    rows, H = y.shape
    if topk_w.dtype != torch.float32 or topk_w.shape != shape:
        raise TypeError("topk_w must be float32 with the shape of tok_map")
    if dy is None:
        dy = _empty(y.shape, y.dtype, y.device, stream)
    elif dy.dtype != y.dtype or dy.shape != y.shape:
        raise ValueError("dy must have y's type and shape")
    if dw is None:
        dw = _empty(shape, torch.float32, y.device, stream)
    elif dw.dtype != torch.float32 or dw.shape != shape:
        raise ValueError("dw must be float32 [S, K]")
    _abi.check("moe_combine_backward", lib().moe_combine_backward(
        _ptr(dout), _dt(dout), _ptr(y), rows, _dt(y), _ptr(topk_w), _ptr(plan.tok_map),
        _ptr(plan.cnt), _ptr(plan.off), S, H, K, plan.cnt.numel(), _ptr(dy), _ptr(dw),
        _stream(stream, y)))
    return dy, dw


def _expert_args(rows: torch.Tensor, name: str, w: torch.Tensor, width: int, plan):
    if rows.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError(f"{name} and w must be bfloat16")
    if w.dim() != 3 or rows.dim() != 2 or rows.shape[1] != w.shape[width]:
        raise ValueError(f"w must be [E, N, D] and {name} [rows, {'N' if width == 1 else 'D'}]")
    _check_plan(plan, w.shape[0])


def _expert_out(out, shape, dtype, device, stream):
    if out is None:
        if dtype not in _TORCH_DT.values():
            raise TypeError(f"unsupported output dtype {dtype}")
        return _empty(shape, dtype, device, stream)
    if tuple(out.shape) != tuple(shape):
        raise ValueError(f"out must be {list(shape)}")
    if out.dtype not in _TORCH_DT.values():
        raise TypeError(f"unsupported output dtype {out.dtype}")
    return out


def moe_expert_gemm(x: torch.Tensor, w: torch.Tensor, plan: Union[Plan, CapacityPlan], *,
                    out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """y[r] = w[e] x[r] for the rows of each bucket e of the plan, zero on rows
    in no bucket.  x bf16 [rows, D], w bf16 [E, N, D]; y [rows, N]."""
    _expert_args(x, "x", w, 2, plan)
    E, N, D = w.shape
    out = _expert_out(out, (x.shape[0], N), out_dtype, x.device, stream)
    _abi.check("moe_expert_gemm", lib().moe_expert_gemm(
        _ptr(x), x.shape[0], _ptr(w), N, D, E, _ptr(plan.cnt), _ptr(plan.off), _ptr(out),
        _dt(out), _stream(stream, x)))
    return out


def moe_expert_gemm_dgrad(dy: torch.Tensor, w: torch.Tensor, plan: Union[Plan, CapacityPlan], *,
                          out_dtype: torch.dtype = torch.bfloat16,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of moe_expert_gemm for its rows: dx[r] = w[e]^T dy[r], zero on
    rows in no bucket.  dy bf16 [rows, N]; dx [rows, D]."""
    _expert_args(dy, "dy", w, 1, plan)
    E, N, D = w.shape
    out = _expert_out(out, (dy.shape[0], D), out_dtype, dy.device, stream)
    _abi.check("moe_expert_gemm_dgrad", lib().moe_expert_gemm_dgrad(
        _ptr(dy), dy.shape[0], _ptr(w), N, D, E, _ptr(plan.cnt), _ptr(plan.off), _ptr(out),
        _dt(out), _stream(stream, dy)))
    return out


def moe_expert_gemm_wgrad(dy: torch.Tensor, x: torch.Tensor, plan: Union[Plan, CapacityPlan], *,
                          out_dtype: torch.dtype = torch.float32,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of moe_expert_gemm for its weights: dw[e] = sum over the rows
    of bucket e of dy[r] x[r]^T, zero for an empty bucket.  Returns
    [E, N, D]."""
    if dy.dtype != torch.bfloat16 or x.dtype != torch.bfloat16:
        raise TypeError("dy and x must be bfloat16")
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0]:
        raise ValueError("dy must be [rows, N] and x [rows, D]")
    E, N, D = plan.cnt.numel(), dy.shape[1], x.shape[1]
    _check_plan(plan, E)
    out = _expert_out(out, (E, N, D), out_dtype, x.device, stream)
    _abi.check("moe_expert_gemm_wgrad", lib().moe_expert_gemm_wgrad(
        _ptr(dy), _ptr(x), x.shape[0], N, D, E, _ptr(plan.cnt), _ptr(plan.off), _ptr(out),
        _dt(out), _stream(stream, x)))
    return out


_dtype_of = attrgetter("dtype")


def _addresses(name: str, tensors: Sequence[torch.Tensor], device: int):
    if device < 0 or set(map(torch.Tensor.get_device, tensors)) != {device}:
        raise ValueError(f"{name} must live on one CUDA device")
    if not all(map(torch.Tensor.is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    return array("Q", list(map(torch.Tensor.data_ptr, tensors)))


def _grad_call(fn: str, grads: Sequence[torch.Tensor], max_norm, out, norm, workspace, stream):
    # one attribute of all tensors at a time: a call over 40 tensors costs the
    # host a third of what one tensor at a time does
    if not grads:
        raise ValueError("no gradients")
    dtypes = list(map(_dtype_of, grads))
    n, n32 = len(dtypes), dtypes.count(torch.float32)
    if n32 + dtypes.count(torch.bfloat16) != n:
        raise TypeError("grads must be float32 or bfloat16")
    sizes = list(map(torch.Tensor.numel, grads))
    if out is grads:
        out = None
    if out is not None and (list(map(_dtype_of, out)) != dtypes or
                            list(map(torch.Tensor.numel, out)) != sizes):
        raise ValueError("out must have the types and sizes of grads")
    like = grads[0]
    device = like.get_device()
    ptrs = _addresses("grads", grads, device)
    outs = ptrs if out is None else _addresses("out", out, device)
    if norm is None:
        norm = _empty(1, torch.float32, like.device, stream)
    elif norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be float32 [1]")
    L = lib()
    ws = _workspace(int(L.moe_grad_norm_workspace_size()), like.device, workspace, stream)
    numel = array("q", sizes)
    codes = array("i", [MOE_F32 if n32 == n else MOE_BF16]) * n if n32 in (0, n) else \
        array("i", [MOE_F32 if d is torch.float32 else MOE_BF16 for d in dtypes])
    args = (ptrs.buffer_info()[0],)
    if max_norm is not None:
        args += (outs.buffer_info()[0],)
    args += (numel.buffer_info()[0], codes.buffer_info()[0], n)
    if max_norm is not None:
        args += (float(max_norm),)
    _abi.check(fn, getattr(L, fn)(*args, _ptr(norm), _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream, like)))
    return norm


def moe_grad_norm(grads: Sequence[torch.Tensor], *, norm: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The L2 norm over all gradients (float32 or bfloat16, any mix), as a
    float32 [1] device tensor."""
    return _grad_call("moe_grad_norm", grads, None, None, norm, workspace, stream)


def moe_clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, *,
                       out: Optional[Sequence[torch.Tensor]] = None,
                       norm: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or
    into `out` (tensors of the same types and sizes).  Returns the norm before
    it, float32 [1] on the device."""
    return _grad_call("moe_clip_grad_norm", grads, max_norm, out, norm, workspace, stream)


def moe_device_errors() -> int:
    """Reads and clears the kernels' device error bits (synchronous): bit 0
    dispatch wait timeout, bit 1 dispatch row index out of range, bit 2
    combine row index out of range, bit 4 expert product wait timeout, bit 5
    expert product bucket out of range."""
    v = ctypes.c_uint32(0)
    _abi.check("moe_device_errors", lib().moe_device_errors(ctypes.byref(v)))
    return int(v.value)


from .op import MoeOp, Routing  # noqa: E402  (the op interface over the calls above)
