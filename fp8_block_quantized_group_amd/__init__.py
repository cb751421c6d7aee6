"""Python binding of the gfx950 fp8 block-quantized MoE expert layer.

Argument marshalling only: every step runs in ``libmoe_fp8.so`` (HIP,
gfx950), declared in ``include/moe_fp8.h``.  PyTorch supplies device memory
and the current HIP stream.  Importing this package does not load the
library; the first call does, and raises if it is missing (build it with
``python -m fp8_block_quantized_group_amd.build``).  There is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, fields, replace
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_fp8.so")

Q_FP8_UE8M0, Q_FP8_F32, Q_BF16, Q_MXFP8 = 0, 1, 2, 3
W_FP8_BLOCK128, W_MXFP8, W_MXFP4 = 0, 1, 2
_ACT_QUANT = {"ue8m0": Q_FP8_UE8M0, "fp32": Q_FP8_F32, "bf16": Q_BF16, "mxfp8": Q_MXFP8}
_WEIGHT_QUANT = {"fp8_block128": W_FP8_BLOCK128, "mxfp8": W_MXFP8, "mxfp4": W_MXFP4}
ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "silu_no_mul", "gelu_no_mul", "gelu_tanh_no_mul",
               "relu2_no_mul", "swigluoai", "swiglustep")   # moe_act_t order
LAYOUT_CONTIGUOUS, LAYOUT_BATCHED, LAYOUT_INDEXED = 0, 1, 2
_LAYOUT = {"contiguous": LAYOUT_CONTIGUOUS, "batched": LAYOUT_BATCHED, "indexed": LAYOUT_INDEXED}
_STATUS = {0: "MOE_OK", -1: "MOE_ERR_INVALID_ARG", -2: "MOE_ERR_UNSUPPORTED",
           -3: "MOE_ERR_WORKSPACE", -4: "MOE_ERR_LAUNCH"}


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_STATUS.get(status, status)}: {msg}")
        self.status = status


class _Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_tokens", "hidden", "intermediate", "num_experts", "top_k", "layout",
        "max_tokens_per_expert", "act_quant", "weight_quant", "activation")] + [
        ("act_limit", ctypes.c_float)]


class _Router(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_tokens", "num_experts", "top_k", "dtype", "score", "num_groups", "topk_groups",
        "group_top", "renormalize")] + [("scale", ctypes.c_float)]


class _Rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_tokens", "hidden", "num_experts", "top_k", "dtype")]


class _BlockNorm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_tokens", "hidden", "dtype", "weight_dtype", "post_norm", "gate",
        "gate_sigmoid")] + [(n, ctypes.c_float) for n in (
            "eps", "residual_scale", "weight_offset")]


class _ExpertLinear(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_rows", "in_features", "out_features", "num_experts", "dtype", "activation")] + [
        ("act_limit", ctypes.c_float)]


class _ExpertLinearW4(ctypes.Structure):
    _fields_ = _ExpertLinear._fields_ + [(n, ctypes.c_int32) for n in (
        "format", "group_size", "scale_dtype")]


class _Eplb(ctypes.Structure):
    _fields_ = [("logical_to_physical", ctypes.c_void_p), ("map_stride", ctypes.c_int32),
                ("replica_count", ctypes.c_void_p), ("num_logical", ctypes.c_int32),
                ("expert_load", ctypes.c_void_p), ("record_flag", ctypes.c_void_p),
                ("num_unpadded_tokens", ctypes.c_void_p)]


class _Routing(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "expert_num_tokens", "expert_offsets", "row_src", "slot_row", "tile_list")]


class _Sizes(ctypes.Structure):
    _fields_ = [("slots", ctypes.c_int64), ("tile_list", ctypes.c_int64),
                ("stage_rows", ctypes.c_int64), ("expert_rows", ctypes.c_int64),
                ("x_sf_row", ctypes.c_int64), ("a2_sf_row", ctypes.c_int64),
                ("padded_rows", ctypes.c_int64), ("blocks", ctypes.c_int64),
                ("tile_m", ctypes.c_int32), ("tall_tile_m", ctypes.c_int32),
                ("max_tiles", ctypes.c_int64), ("tall_list_offset", ctypes.c_int64),
                ("max_tiles_tall", ctypes.c_int64)]


EXPORTS = ("moe_routing_sizes", "moe_stage_workspace_size", "moe_workspace_size",
           "moe_w2_workspace_size", "moe_stage",
           "moe_grouped_gemm_w13", "moe_grouped_gemm_w13_act", "moe_act_requant",
           "moe_grouped_gemm_w2", "moe_topk_reduce", "moe_align_capacity",
           "moe_align_block_size", "moe_grouped_gemm_w13_act_indexed",
           "moe_grouped_gemm_w2_indexed", "moe_fused_mul_sum", "moe_forward",
           "moe_forward_static", "moe_last_error",
           "moe_router_topk", "moe_router_topk_backward", "moe_permute_workspace_size",
           "moe_permute", "moe_permute_backward", "moe_unpermute", "moe_unpermute_backward",
           "moe_block_norm", "moe_block_norm_workspace_size", "moe_block_norm_backward",
           "moe_expert_linear", "moe_expert_linear_workspace_size",
           "moe_expert_linear_backward", "moe_expert_linear_w4",
           "moe_block_norm_quant", "moe_stage_routing", "moe_forward_quantized")

_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m fp8_block_quantized_group_amd.build`")
    lib = ctypes.CDLL(path)
    P, V, S = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t
    lib.moe_last_error.restype = ctypes.c_char_p
    lib.moe_routing_sizes.argtypes = [P(_Problem), P(_Sizes)]
    lib.moe_stage_workspace_size.argtypes = [P(_Problem), P(S)]
    lib.moe_workspace_size.argtypes = [P(_Problem), P(S)]
    lib.moe_w2_workspace_size.argtypes = [P(_Problem), P(S)]
    lib.moe_stage.argtypes = [P(_Problem), V, V, V, V, V, P(_Eplb), V, V, V, V, P(_Routing),
                              V, S, V]
    lib.moe_grouped_gemm_w13.argtypes = [P(_Problem), V, V, P(_Routing), V, V, V, V]
    lib.moe_grouped_gemm_w13_act.argtypes = [P(_Problem), V, V, P(_Routing), V, V, V, V, V]
    lib.moe_act_requant.argtypes = [P(_Problem), V, P(_Routing), V, V, V]
    lib.moe_grouped_gemm_w2.argtypes = [P(_Problem), V, V, P(_Routing), V, V, V, V, S, V]
    lib.moe_topk_reduce.argtypes = [P(_Problem), V, V, V, V, V]
    I32, I64 = ctypes.c_int32, ctypes.c_int64
    lib.moe_align_capacity.argtypes = [P(_Problem), I32, P(I64), P(I64)]
    lib.moe_align_block_size.argtypes = [P(_Problem), V, P(_Routing), I32, V, V, V, V]
    lib.moe_grouped_gemm_w13_act_indexed.argtypes = [P(_Problem), V, V, V, V, V, I32, V, V, V,
                                                     V, V]
    lib.moe_grouped_gemm_w2_indexed.argtypes = [P(_Problem), V, V, V, V, V, I32, V, V, V, V,
                                                S, V]
    lib.moe_fused_mul_sum.argtypes = [P(_Problem), V, V, V, V, V]
    lib.moe_forward.argtypes = [P(_Problem), V, V, V, V, V, P(_Eplb), V, V, V, V, V, V, S, V]
    lib.moe_forward_static.argtypes = [P(_Problem), V, V, V, V, V, P(_Eplb), V, V, V, V, V, V]
    lib.moe_router_topk.argtypes = [P(_Router)] + [V] * 6
    lib.moe_router_topk_backward.argtypes = [P(_Router)] + [V] * 5
    lib.moe_permute_workspace_size.argtypes = [P(_Rows), P(S)]
    lib.moe_permute.argtypes = [P(_Rows)] + [V] * 8 + [S, V]
    lib.moe_permute_backward.argtypes = [P(_Rows)] + [V] * 4
    lib.moe_unpermute.argtypes = [P(_Rows)] + [V] * 5
    lib.moe_unpermute_backward.argtypes = [P(_Rows)] + [V] * 7
    lib.moe_block_norm.argtypes = [P(_BlockNorm)] + [V] * 8
    lib.moe_block_norm_workspace_size.argtypes = [P(_BlockNorm), P(S)]
    lib.moe_block_norm_backward.argtypes = [P(_BlockNorm)] + [V] * 13 + [S, V]
    lib.moe_expert_linear.argtypes = [P(_ExpertLinear)] + [V] * 6
    lib.moe_expert_linear_workspace_size.argtypes = [P(_ExpertLinear), P(S)]
    lib.moe_expert_linear_backward.argtypes = [P(_ExpertLinear)] + [V] * 8 + [S, V]
    lib.moe_expert_linear_w4.argtypes = [P(_ExpertLinearW4)] + [V] * 7
    lib.moe_block_norm_quant.argtypes = [P(_BlockNorm), I32] + [V] * 10
    lib.moe_stage_routing.argtypes = [P(_Problem)] + [V] * 4 + [P(_Eplb), V, V, P(_Routing), V, S,
                                                               V]
    lib.moe_forward_quantized.argtypes = [P(_Problem)] + [V] * 6 + [P(_Eplb)] + [V] * 6 + [S, V]
    lib.moe_last_error.argtypes = []
    for name in EXPORTS:
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int if name != "moe_last_error" else ctypes.c_char_p
        # without argtypes ctypes passes Python ints as 32-bit C ints, which
        # would truncate every device pointer
        if fn.argtypes is None:
            raise RuntimeError(f"{name}: no ctypes signature declared")
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise MoeError(status, load_library().moe_last_error().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    return t.data_ptr()


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@dataclass(frozen=True)
class Problem:
    num_tokens: int
    hidden: int
    intermediate: int
    num_experts: int
    top_k: int
    layout: int = LAYOUT_CONTIGUOUS
    max_tokens_per_expert: int = 0
    act_quant: int = Q_FP8_UE8M0
    weight_quant: int = W_FP8_BLOCK128
    activation: int = 0                             # index into ACTIVATIONS
    act_limit: float = 0.0                          # clamp limit (moe_problem_t)

    def c(self) -> _Problem:
        return _Problem(self.num_tokens, self.hidden, self.intermediate, self.num_experts,
                        self.top_k, self.layout, self.max_tokens_per_expert, self.act_quant,
                        self.weight_quant, self.activation, self.act_limit)

    @staticmethod
    def from_config(cfg, act_quant: Optional[int] = None) -> "Problem":
        """From a ``moe_synth.MoeConfig``."""
        q = act_quant if act_quant is not None else _ACT_QUANT[cfg.act_quant]
        return Problem(cfg.T, cfg.K, cfg.N, cfg.E, cfg.top_k, _LAYOUT[cfg.layout],
                       cfg.max_tokens, q, _WEIGHT_QUANT[cfg.weight_quant],
                       ACTIVATIONS.index(cfg.activation), float(cfg.act_limit))


def sizes(p: Problem) -> dict:
    s = _Sizes()
    _check(load_library().moe_routing_sizes(ctypes.byref(p.c()), ctypes.byref(s)))
    return {f: getattr(s, f) for f, _ in _Sizes._fields_}


def stage_workspace_size(p: Problem) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_stage_workspace_size(ctypes.byref(p.c()), ctypes.byref(n)))
    return n.value


def workspace_size(p: Problem) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_workspace_size(ctypes.byref(p.c()), ctypes.byref(n)))
    return n.value


def w2_workspace_size(p: Problem) -> int:
    """Bytes of the w2 call's split-K workspace (0: w2 does not split)."""
    n = ctypes.c_size_t()
    _check(load_library().moe_w2_workspace_size(ctypes.byref(p.c()), ctypes.byref(n)))
    return n.value


def alloc_w2_workspace(p: Problem, device="cuda") -> Optional[torch.Tensor]:
    n = w2_workspace_size(p)
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def _ws(ws: Optional[torch.Tensor]):
    return (_ptr(ws), ws.numel()) if ws is not None else (None, 0)


def _eplb(eplb: Optional[dict]):
    if eplb is None:
        return None
    l2p = eplb["l2p"]
    e = _Eplb(_ptr(l2p), l2p.shape[1], _ptr(eplb["replica_count"]), l2p.shape[0],
              _ptr(eplb.get("expert_load")), _ptr(eplb.get("record")),
              _ptr(eplb.get("num_unpadded")))
    return ctypes.byref(e), e


def _routing(r: dict) -> _Routing:
    return _Routing(*[_ptr(r[n]) for n in ("expert_num_tokens", "expert_offsets", "row_src",
                                          "slot_row", "tile_list")])


def scale_dtype(p: Problem):
    """torch dtype of the activation scales (E8M0 bytes or fp32)."""
    return torch.float32 if p.act_quant == Q_FP8_F32 else torch.uint8


def alloc_act_outputs(p: Problem, device="cuda", rows: Optional[int] = None):
    """(a2_q, a2_sf) for the w2 input: fp8 codes and scales, or bf16 values
    and None for unquantized activations; ``rows`` defaults to the layout's
    expert rows."""
    s = sizes(p)
    rows = s["expert_rows"] if rows is None else rows
    if p.act_quant == Q_BF16:
        return torch.empty((rows, p.intermediate), dtype=torch.bfloat16, device=device), None
    return (torch.empty((rows, p.intermediate), dtype=torch.uint8, device=device),
            torch.empty((rows, s["a2_sf_row"]), dtype=scale_dtype(p), device=device))


def alloc_stage_outputs(p: Problem, device="cuda") -> dict:
    """Caller-side buffers for moe_stage (allocated by torch)."""
    s = sizes(p)
    dev = torch.device(device)
    out = {
        "x_q": torch.empty((s["stage_rows"], p.hidden),
                           dtype=torch.bfloat16 if p.act_quant == Q_BF16 else torch.uint8,
                           device=dev),
        "x_sf": None if p.act_quant == Q_BF16 else torch.empty(
            (s["stage_rows"], s["x_sf_row"]), dtype=scale_dtype(p), device=dev),
        "topk_idx": torch.empty((p.num_tokens, p.top_k), dtype=torch.int64, device=dev),
        "topk_w": torch.empty((p.num_tokens, p.top_k), dtype=torch.float32, device=dev),
        "expert_num_tokens": torch.empty(p.num_experts, dtype=torch.int32, device=dev),
        "expert_offsets": torch.empty(p.num_experts + 1, dtype=torch.int32, device=dev),
        "row_src": torch.empty(max(s["slots"], 1), dtype=torch.int32, device=dev),
        "slot_row": torch.empty(max(s["slots"], 1), dtype=torch.int32, device=dev),
        "tile_list": torch.empty(s["tile_list"], dtype=torch.int32, device=dev),
        "ws": torch.empty(stage_workspace_size(p), dtype=torch.uint8, device=dev),
    }
    return out


def stage(p: Problem, hidden, topk_ids, topk_weights, bufs: dict, is_padding=None,
          expert_num_tokens=None, eplb=None):
    """moe_stage: fills bufs' x_q, x_sf, topk_idx, topk_w and the routing layout."""
    lib = load_library()
    e = _eplb(eplb)
    r = _routing(bufs)
    _check(lib.moe_stage(ctypes.byref(p.c()), _ptr(hidden), _ptr(expert_num_tokens),
                         _ptr(topk_ids), _ptr(topk_weights), _ptr(is_padding),
                         e[0] if e else None, _ptr(bufs["x_q"]), _ptr(bufs["x_sf"]),
                         _ptr(bufs["topk_idx"]), _ptr(bufs["topk_w"]), ctypes.byref(r),
                         _ptr(bufs["ws"]), bufs["ws"].numel(), _stream()))


def stage_routing(p: Problem, topk_ids, topk_weights, bufs: dict, is_padding=None,
                  expert_num_tokens=None, eplb=None):
    """moe_stage_routing: stage without its rows, for x_q and x_sf made elsewhere."""
    e = _eplb(eplb)
    r = _routing(bufs)
    _check(load_library().moe_stage_routing(
        ctypes.byref(p.c()), _ptr(expert_num_tokens), _ptr(topk_ids), _ptr(topk_weights),
        _ptr(is_padding), e[0] if e else None, _ptr(bufs["topk_idx"]), _ptr(bufs["topk_w"]),
        ctypes.byref(r), _ptr(bufs["ws"]), bufs["ws"].numel(), _stream()))


def grouped_gemm_w13(p: Problem, a_q, a_sf, routing: dict, w13, w13_sf, gate_up):
    r = _routing(routing)
    _check(load_library().moe_grouped_gemm_w13(ctypes.byref(p.c()), _ptr(a_q), _ptr(a_sf),
                                                ctypes.byref(r), _ptr(w13), _ptr(w13_sf),
                                                _ptr(gate_up), _stream()))


def grouped_gemm_w13_act(p: Problem, a_q, a_sf, routing: dict, w13, w13_sf, a2_q, a2_sf):
    """w13 GEMM with SiLU(gate)*up and the fp8 re-quantization in its epilogue;
    a2_q / a2_sf equal grouped_gemm_w13 followed by act_requant bit for bit."""
    r = _routing(routing)
    _check(load_library().moe_grouped_gemm_w13_act(ctypes.byref(p.c()), _ptr(a_q), _ptr(a_sf),
                                                    ctypes.byref(r), _ptr(w13), _ptr(w13_sf),
                                                    _ptr(a2_q), _ptr(a2_sf), _stream()))


def act_requant(p: Problem, gate_up, routing: dict, a2_q, a2_sf):
    r = _routing(routing)
    _check(load_library().moe_act_requant(ctypes.byref(p.c()), _ptr(gate_up), ctypes.byref(r),
                                           _ptr(a2_q), _ptr(a2_sf), _stream()))


def grouped_gemm_w2(p: Problem, a2_q, a2_sf, routing: dict, w2, w2_sf, down, ws="auto"):
    """ws: the split-K workspace (alloc_w2_workspace); "auto" allocates it."""
    r = _routing(routing)
    if isinstance(ws, str):
        ws = alloc_w2_workspace(p, down.device)
    wp, wn = _ws(ws)
    _check(load_library().moe_grouped_gemm_w2(ctypes.byref(p.c()), _ptr(a2_q), _ptr(a2_sf),
                                               ctypes.byref(r), _ptr(w2), _ptr(w2_sf),
                                               _ptr(down), wp, wn, _stream()))


def topk_reduce(p: Problem, down, slot_row, topk_w, out):
    _check(load_library().moe_topk_reduce(ctypes.byref(p.c()), _ptr(down), _ptr(slot_row),
                                           _ptr(topk_w), _ptr(out), _stream()))


def align_capacity(p: Problem, block_size: int):
    """(sorted_ids length, expert_ids length) for ``block_size``."""
    n, b = ctypes.c_int64(), ctypes.c_int64()
    _check(load_library().moe_align_capacity(ctypes.byref(p.c()), block_size, ctypes.byref(n),
                                             ctypes.byref(b)))
    return n.value, b.value


def alloc_indexed(p: Problem, block_size: int, device="cuda") -> dict:
    """sorted_ids / expert_ids / num_tokens_padded buffers of the block map."""
    n, b = align_capacity(p, block_size)
    return {"sorted_ids": torch.empty(max(n, 1), dtype=torch.int32, device=device),
            "expert_ids": torch.empty(max(b, 1), dtype=torch.int32, device=device),
            "num_tokens_padded": torch.empty(1, dtype=torch.int32, device=device),
            "block_size": block_size}


def align_block_size(p: Problem, topk_idx, routing: dict, ix: dict):
    """moe_align_block_size: fills ix (from alloc_indexed) from moe_stage's
    topk_idx and routing."""
    r = _routing(routing)
    _check(load_library().moe_align_block_size(
        ctypes.byref(p.c()), _ptr(topk_idx), ctypes.byref(r), ix["block_size"],
        _ptr(ix["sorted_ids"]), _ptr(ix["expert_ids"]), _ptr(ix["num_tokens_padded"]),
        _stream()))


def grouped_gemm_w13_act_indexed(p: Problem, a_q, a_sf, ix: dict, w13, w13_sf, a2_q, a2_sf):
    _check(load_library().moe_grouped_gemm_w13_act_indexed(
        ctypes.byref(p.c()), _ptr(a_q), _ptr(a_sf), _ptr(ix["sorted_ids"]),
        _ptr(ix["expert_ids"]), _ptr(ix["num_tokens_padded"]), ix["block_size"], _ptr(w13),
        _ptr(w13_sf), _ptr(a2_q), _ptr(a2_sf), _stream()))


def grouped_gemm_w2_indexed(p: Problem, a2_q, a2_sf, ix: dict, w2, w2_sf, down, ws="auto"):
    if isinstance(ws, str):
        ws = alloc_w2_workspace(p, down.device)
    wp, wn = _ws(ws)
    _check(load_library().moe_grouped_gemm_w2_indexed(
        ctypes.byref(p.c()), _ptr(a2_q), _ptr(a2_sf), _ptr(ix["sorted_ids"]),
        _ptr(ix["expert_ids"]), _ptr(ix["num_tokens_padded"]), ix["block_size"], _ptr(w2),
        _ptr(w2_sf), _ptr(down), wp, wn, _stream()))


def fused_mul_sum(p: Problem, down, topk_idx, topk_w, out):
    _check(load_library().moe_fused_mul_sum(ctypes.byref(p.c()), _ptr(down), _ptr(topk_idx),
                                             _ptr(topk_w), _ptr(out), _stream()))


def forward(p: Problem, hidden, topk_ids, topk_weights, w13, w13_sf, w2, w2_sf, out, ws,
            is_padding=None, expert_num_tokens=None, eplb=None):
    """moe_forward: the whole layer; ``ws`` is a uint8 device tensor of at
    least workspace_size(p) bytes."""
    e = _eplb(eplb)
    _check(load_library().moe_forward(
        ctypes.byref(p.c()), _ptr(hidden), _ptr(expert_num_tokens), _ptr(topk_ids),
        _ptr(topk_weights), _ptr(is_padding), e[0] if e else None, _ptr(w13), _ptr(w13_sf),
        _ptr(w2), _ptr(w2_sf), _ptr(out), _ptr(ws), ws.numel(), _stream()))


def forward_quantized(p: Problem, x_q, x_sf, topk_ids, topk_weights, w13, w13_sf, w2, w2_sf, out,
                      ws, is_padding=None, expert_num_tokens=None, eplb=None):
    """moe_forward_quantized: the layer on staged rows (block_norm_quant, stage)."""
    e = _eplb(eplb)
    _check(load_library().moe_forward_quantized(
        ctypes.byref(p.c()), _ptr(x_q), _ptr(x_sf), _ptr(expert_num_tokens), _ptr(topk_ids),
        _ptr(topk_weights), _ptr(is_padding), e[0] if e else None, _ptr(w13), _ptr(w13_sf),
        _ptr(w2), _ptr(w2_sf), _ptr(out), _ptr(ws), ws.numel(), _stream()))


STATIC_SCRATCH_BYTES = 64 << 20      # MOE_STATIC_SCRATCH_BYTES


def forward_static(p: Problem, hidden, topk_ids, topk_weights, w13, w13_sf, w2, w2_sf, out,
                   is_padding=None, expert_num_tokens=None, eplb=None):
    """moe_forward_static: the whole layer with the library's static
    per-GPU workspace (no allocation; calls on one GPU must not overlap)."""
    e = _eplb(eplb)
    _check(load_library().moe_forward_static(
        ctypes.byref(p.c()), _ptr(hidden), _ptr(expert_num_tokens), _ptr(topk_ids),
        _ptr(topk_weights), _ptr(is_padding), e[0] if e else None, _ptr(w13), _ptr(w13_sf),
        _ptr(w2), _ptr(w2_sf), _ptr(out), _stream()))


class MoeLayer:
    """The expert layer with its weights and a preallocated workspace."""

    def __init__(self, p: Problem, w13, w13_sf, w2, w2_sf):
        self.p = p
        self.w13, self.w13_sf, self.w2, self.w2_sf = w13, w13_sf, w2, w2_sf
        self.ws = torch.empty(workspace_size(p), dtype=torch.uint8, device=w13.device)

    def __call__(self, hidden, topk_ids, topk_weights, out=None, is_padding=None,
                 expert_num_tokens=None, eplb=None):
        if out is None:
            out = torch.empty((self.p.num_tokens, self.p.hidden), dtype=torch.bfloat16,
                              device=hidden.device)
        forward(self.p, hidden, topk_ids, topk_weights, self.w13, self.w13_sf, self.w2,
                self.w2_sf, out, self.ws, is_padding, expert_num_tokens, eplb)
        return out


    def quantized(self, x_q, x_sf, topk_ids, topk_weights, out=None, is_padding=None,
                  expert_num_tokens=None, eplb=None):
        """The layer on rows that are staged already."""
        if out is None:
            out = torch.empty((self.p.num_tokens, self.p.hidden), dtype=torch.bfloat16,
                              device=x_q.device)
        forward_quantized(self.p, x_q, x_sf, topk_ids, topk_weights, self.w13, self.w13_sf,
                          self.w2, self.w2_sf, out, self.ws, is_padding, expert_num_tokens, eplb)
        return out


# ---- around the layer: router, sorted rows, block norms ----------------------
# Unlike the layer's calls these check shapes, types and devices here, and run
# on the tensors' device, on its current stream, whatever device is current.

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}     # moe_dtype_t
SCORES = ("softmax", "sigmoid")                                        # moe_score_t
_EIGHT_BITS = {k: v for k, v in _ACT_QUANT.items() if v != Q_BF16}
GATES = ("none", "token", "channel", "full")                           # moe_gate_t


def _choice(value, names, what: str) -> int:
    if value not in names:
        raise ValueError(f"{what} must be one of {tuple(names)}, got {value!r}")
    return names[value] if isinstance(names, dict) else names.index(value)


class _Descriptor:
    """A frozen dataclass whose C struct is made once."""

    def __post_init__(self):
        c = self._struct()
        for name, kind in c._fields_:
            value = getattr(self, name)
            whole = kind is ctypes.c_int32 and hasattr(value, "__index__")
            if whole and getattr(c, name) != value:
                raise ValueError(f"{name} = {value} does not fit 32 bits")
        object.__setattr__(self, "_c", c)
        object.__setattr__(self, "_ref", ctypes.byref(c))

    def __reduce__(self):                   # a reference to a C struct has no copy
        return type(self), tuple(getattr(self, f.name) for f in fields(self))


@dataclass(frozen=True)
class Router(_Descriptor):
    """moe_router_t: how a token's experts are chosen from its logits."""
    num_tokens: int
    num_experts: int
    top_k: int
    score: str = "softmax"                  # "softmax" | "sigmoid"
    num_groups: int = 1
    topk_groups: int = 1
    group_top: int = 1
    renormalize: bool = True
    scale: float = 1.0
    dtype: torch.dtype = torch.float32      # of the logits

    def _struct(self):
        return _Router(self.num_tokens, self.num_experts, self.top_k,
                       _choice(self.dtype, _DTYPES, "dtype"),
                       _choice(self.score, SCORES, "score"), self.num_groups,
                       self.topk_groups, self.group_top, int(self.renormalize), self.scale)


@dataclass(frozen=True)
class ExpertRows(_Descriptor):
    """moe_rows_t: token rows sorted by expert."""
    num_tokens: int
    hidden: int
    num_experts: int
    top_k: int
    dtype: torch.dtype = torch.bfloat16

    def _struct(self):
        return _Rows(self.num_tokens, self.hidden, self.num_experts, self.top_k,
                     _choice(self.dtype, _DTYPES, "dtype"))


@dataclass(frozen=True)
class BlockNorm(_Descriptor):
    """moe_block_norm_t: the norms before and after a block with its gate and
    residual scale."""
    num_tokens: int
    hidden: int
    dtype: torch.dtype = torch.bfloat16
    weight_dtype: Optional[torch.dtype] = None      # None: dtype
    post_norm: bool = False
    gate: str = "none"                              # "none" | "token" | "channel" | "full"
    gate_sigmoid: bool = False
    eps: float = 1e-6
    residual_scale: float = 1.0
    weight_offset: float = 0.0

    def _struct(self):
        return _BlockNorm(self.num_tokens, self.hidden, _choice(self.dtype, _DTYPES, "dtype"),
                          _choice(self.weight_dtype or self.dtype, _DTYPES, "weight_dtype"),
                          int(self.post_norm), _choice(self.gate, GATES, "gate"),
                          int(self.gate_sigmoid), self.eps, self.residual_scale,
                          self.weight_offset)

    def __post_init__(self):
        super().__post_init__()
        T, H = self.num_tokens, self.hidden
        shape = {"none": (), "token": (T,), "channel": (H,), "full": (T, H)}[self.gate]
        object.__setattr__(self, "gate_shape", shape)


def _arg(t, name: str, dtype, shape, device):
    """The address of an argument, checked; None for one that is not given."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _device(t: torch.Tensor, name: str) -> torch.device:
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return t.device


def _scratch(ws: Optional[torch.Tensor], device):
    if ws is None:
        return None, 0
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


# The current stream's address; the raw form costs a tenth of a microsecond,
# building a torch.cuda.Stream most of two, as much as a kernel of these takes.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(fn, device: torch.device, *args):
    """fn(*args, stream) on the device and its current stream."""
    index = device.index
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status)


def router_topk(r: Router, logits, topk_ids, topk_weights, bias=None, is_padding=None):
    """moe_router_topk: fills topk_ids int32 and topk_weights fp32 [T, top_k]
    from logits [T, E]."""
    d = _device(logits, "logits")
    T, E, k = r.num_tokens, r.num_experts, r.top_k
    _run(load_library().moe_router_topk, d, r._ref,
         _arg(logits, "logits", r.dtype, (T, E), d),
         _arg(bias, "bias", torch.float32, (E,), d),
         _arg(is_padding, "is_padding", torch.uint8, (T,), d),
         _arg(topk_ids, "topk_ids", torch.int32, (T, k), d),
         _arg(topk_weights, "topk_weights", torch.float32, (T, k), d))


def router_topk_backward(r: Router, logits, topk_ids, grad_topk_weights, grad_logits):
    """moe_router_topk_backward: fills grad_logits [T, E]."""
    d = _device(logits, "logits")
    T, E, k = r.num_tokens, r.num_experts, r.top_k
    _run(load_library().moe_router_topk_backward, d, r._ref,
         _arg(logits, "logits", r.dtype, (T, E), d),
         _arg(topk_ids, "topk_ids", torch.int32, (T, k), d),
         _arg(grad_topk_weights, "grad_topk_weights", torch.float32, (T, k), d),
         _arg(grad_logits, "grad_logits", r.dtype, (T, E), d))


def permute_workspace_size(p: ExpertRows) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_permute_workspace_size(p._ref, ctypes.byref(n)))
    return n.value


def alloc_permute_workspace(p: ExpertRows, device="cuda") -> torch.Tensor:
    return torch.empty(permute_workspace_size(p), dtype=torch.uint8, device=device)


def alloc_permute_outputs(p: ExpertRows, device="cuda") -> dict:
    """The outputs and the workspace of permute, by its parameters' names."""
    n = p.num_tokens * p.top_k
    i32 = dict(dtype=torch.int32, device=device)
    return {"rows": torch.empty((n, p.hidden), dtype=p.dtype, device=device),
            "expert_offsets": torch.empty(p.num_experts + 1, **i32),
            "slot_row": torch.empty((p.num_tokens, p.top_k), **i32),
            "row_slot": torch.empty(n, **i32), "ws": alloc_permute_workspace(p, device)}


def permute(p: ExpertRows, x, topk_ids, rows, expert_offsets, slot_row, row_slot, ws,
            is_padding=None):
    """moe_permute: the tokens' rows sorted by expert."""
    d = _device(x, "x")
    T, k = p.num_tokens, p.top_k
    wp, wn = _scratch(ws, d)
    _run(load_library().moe_permute, d, p._ref, _arg(x, "x", p.dtype, (T, p.hidden), d),
         _arg(topk_ids, "topk_ids", torch.int32, (T, k), d),
         _arg(is_padding, "is_padding", torch.uint8, (T,), d),
         _arg(rows, "rows", p.dtype, (T * k, p.hidden), d),
         _arg(expert_offsets, "expert_offsets", torch.int32, (p.num_experts + 1,), d),
         _arg(slot_row, "slot_row", torch.int32, (T, k), d),
         _arg(row_slot, "row_slot", torch.int32, (T * k,), d), wp, wn)


def permute_backward(p: ExpertRows, grad_rows, slot_row, grad_x):
    """moe_permute_backward: the sum of every token's rows."""
    d = _device(grad_rows, "grad_rows")
    T, k = p.num_tokens, p.top_k
    _run(load_library().moe_permute_backward, d, p._ref,
         _arg(grad_rows, "grad_rows", p.dtype, (T * k, p.hidden), d),
         _arg(slot_row, "slot_row", torch.int32, (T, k), d),
         _arg(grad_x, "grad_x", p.dtype, (T, p.hidden), d))


def unpermute(p: ExpertRows, rows, slot_row, topk_weights, out):
    """moe_unpermute: the weighted sum of every token's rows (weights None: 1)."""
    d = _device(rows, "rows")
    T, k = p.num_tokens, p.top_k
    _run(load_library().moe_unpermute, d, p._ref,
         _arg(rows, "rows", p.dtype, (T * k, p.hidden), d),
         _arg(slot_row, "slot_row", torch.int32, (T, k), d),
         _arg(topk_weights, "topk_weights", torch.float32, (T, k), d),
         _arg(out, "out", p.dtype, (T, p.hidden), d))


def unpermute_backward(p: ExpertRows, grad_out, rows, slot_row, topk_weights, grad_rows,
                       grad_topk_weights):
    """moe_unpermute_backward: the gradients of the rows and of the weights."""
    d = _device(grad_out, "grad_out")
    T, k = p.num_tokens, p.top_k
    _run(load_library().moe_unpermute_backward, d, p._ref,
         _arg(grad_out, "grad_out", p.dtype, (T, p.hidden), d),
         _arg(rows, "rows", p.dtype, (T * k, p.hidden), d),
         _arg(slot_row, "slot_row", torch.int32, (T, k), d),
         _arg(topk_weights, "topk_weights", torch.float32, (T, k), d),
         _arg(grad_rows, "grad_rows", p.dtype, (T * k, p.hidden), d),
         _arg(grad_topk_weights, "grad_topk_weights", torch.float32, (T, k), d))


def block_norm_workspace_size(p: BlockNorm) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_block_norm_workspace_size(p._ref, ctypes.byref(n)))
    return n.value


def alloc_block_norm_workspace(p: BlockNorm, device="cuda") -> torch.Tensor:
    """Scratch of block_norm_backward when it returns a weight's or a
    per-channel gate's gradient."""
    return torch.empty(block_norm_workspace_size(p), dtype=torch.uint8, device=device)


def _block_args(p: BlockNorm, y, post_weight, gate, pre_weight, d):
    wt = p.weight_dtype or p.dtype
    H = p.hidden
    return (_arg(y, "y", p.dtype, (p.num_tokens, H), d),
            _arg(post_weight, "post_weight", wt, (H,), d),
            _arg(gate, "gate", p.dtype, p.gate_shape, d),
            _arg(pre_weight, "pre_weight", wt, (H,), d))


def block_norm(p: BlockNorm, residual, normed=None, y=None, residual_out=None,
               pre_weight=None, post_weight=None, gate=None):
    """moe_block_norm: fills residual_out = residual + scale * gate * n(y) and
    normed, its norm; y None: normed is the norm of residual."""
    d = _device(residual, "residual")
    shape = (p.num_tokens, p.hidden)
    _run(load_library().moe_block_norm, d, p._ref,
         _arg(residual, "residual", p.dtype, shape, d),
         *_block_args(p, y, post_weight, gate, pre_weight, d),
         _arg(residual_out, "residual_out", p.dtype, shape, d),
         _arg(normed, "normed", p.dtype, shape, d))


def quant_shape(rows: int, hidden: int, quant: str):
    """(dtype, shape) of the scales of ``rows`` staged rows."""
    if quant == "fp32":
        return torch.float32, (rows, hidden // 128)
    return torch.uint8, (rows, hidden // 32 if quant == "mxfp8" else
                         (hidden // 128 + 3) // 4 * 4)


def alloc_quant_outputs(p: BlockNorm, quant: str = "ue8m0", device="cuda") -> dict:
    """The 8-bit outputs of block_norm_quant, by its parameters' names."""
    dtype, shape = quant_shape(p.num_tokens, p.hidden, quant)
    return {"x_q": torch.empty((p.num_tokens, p.hidden), dtype=torch.uint8, device=device),
            "x_sf": torch.empty(shape, dtype=dtype, device=device)}


def block_norm_quant(p: BlockNorm, residual, x_q, x_sf, quant: str = "ue8m0", normed=None, y=None,
                     residual_out=None, pre_weight=None, post_weight=None, gate=None):
    """moe_block_norm_quant: block_norm whose normed rows leave as the layer's
    staged input, x_q and x_sf (quant: "ue8m0" | "fp32" | "mxfp8"), and as they
    are too where normed is given."""
    d = _device(residual, "residual")
    shape = (p.num_tokens, p.hidden)
    kind = _choice(quant, _EIGHT_BITS, "quant")
    _run(load_library().moe_block_norm_quant, d, p._ref, kind,
         _arg(residual, "residual", p.dtype, shape, d),
         *_block_args(p, y, post_weight, gate, pre_weight, d),
         _arg(residual_out, "residual_out", p.dtype, shape, d),
         _arg(normed, "normed", p.dtype, shape, d), _arg(x_q, "x_q", torch.uint8, shape, d),
         _arg(x_sf, "x_sf", *quant_shape(*shape, quant), d))


def block_norm_backward(p: BlockNorm, residual_out, grad_normed, grad_residual, y=None,
                        grad_residual_out=None, pre_weight=None, post_weight=None, gate=None,
                        grad_y=None, grad_pre_weight=None, grad_post_weight=None,
                        grad_gate=None, ws="auto"):
    """moe_block_norm_backward at the stored stream residual_out (y None: the
    forward call's residual); ws: "auto" allocates it where it is needed."""
    d = _device(residual_out, "residual_out")
    shape, H = (p.num_tokens, p.hidden), p.hidden
    if isinstance(ws, str):
        sums = (grad_pre_weight is not None or grad_post_weight is not None
                or (grad_gate is not None and p.gate == "channel"))
        ws = alloc_block_norm_workspace(p, d) if sums else None
    wp, wn = _scratch(ws, d)
    _run(load_library().moe_block_norm_backward, d, p._ref,
         _arg(residual_out, "residual_out", p.dtype, shape, d),
         *_block_args(p, y, post_weight, gate, pre_weight, d),
         _arg(grad_normed, "grad_normed", p.dtype, shape, d),
         _arg(grad_residual_out, "grad_residual_out", p.dtype, shape, d),
         _arg(grad_residual, "grad_residual", p.dtype, shape, d),
         _arg(grad_y, "grad_y", p.dtype, shape, d),
         _arg(grad_pre_weight, "grad_pre_weight", torch.float32, (H,), d),
         _arg(grad_post_weight, "grad_post_weight", torch.float32, (H,), d),
         _arg(grad_gate, "grad_gate", p.dtype if p.gate == "full" else torch.float32,
              p.gate_shape, d), wp, wn)


# ---- the experts' own products --------------------------------------------------

_LINEAR_ACTS = {"none": -1, **{name: i for i, name in enumerate(ACTIVATIONS)}}
_SINGLE_ACTS = ("none", "silu_no_mul", "gelu_no_mul", "gelu_tanh_no_mul", "relu2_no_mul")


@dataclass(frozen=True)
class ExpertLinear(_Descriptor):
    """moe_expert_linear_t: a linear layer of rows sorted by expert, with the
    activation that follows it."""
    num_rows: int
    in_features: int
    out_features: int
    num_experts: int = 1
    dtype: torch.dtype = torch.bfloat16
    activation: str = "none"                # "none" or one of ACTIVATIONS
    act_limit: float = 0.0

    def _struct(self):
        return _ExpertLinear(self.num_rows, self.in_features, self.out_features,
                             self.num_experts, _choice(self.dtype, _DTYPES, "dtype"),
                             _choice(self.activation, _LINEAR_ACTS, "activation"),
                             self.act_limit)

    def __post_init__(self):
        super().__post_init__()
        wide = self.out_features * (1 if self.activation in _SINGLE_ACTS else 2)
        object.__setattr__(self, "wide", wide)      # weight rows of an expert


def _offsets(p, expert_offsets, d):
    return _arg(expert_offsets, "expert_offsets", torch.int32, (p.num_experts + 1,), d)


def expert_linear(p: ExpertLinear, x, weight, out, expert_offsets=None, pre_act=None):
    """moe_expert_linear: out = F(x W_e^T) for every expert's rows (expert_offsets
    None: the one expert has all); pre_act: the product before F, for the gradient."""
    d = _device(x, "x")
    R, K, N, dt = p.num_rows, p.in_features, p.out_features, p.dtype
    _run(load_library().moe_expert_linear, d, p._ref, _arg(x, "x", dt, (R, K), d),
         _offsets(p, expert_offsets, d),
         _arg(weight, "weight", dt, (p.num_experts, p.wide, K), d),
         _arg(out, "out", dt, (R, N), d), _arg(pre_act, "pre_act", dt, (R, p.wide), d))


def expert_linear_workspace_size(p: ExpertLinear) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_expert_linear_workspace_size(p._ref, ctypes.byref(n)))
    return n.value


def alloc_expert_linear_workspace(p: ExpertLinear, device="cuda") -> Optional[torch.Tensor]:
    """Scratch of expert_linear_backward; None where it needs none."""
    n = expert_linear_workspace_size(p)
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def expert_linear_backward(p: ExpertLinear, x, weight, grad_out, grad_x=None, grad_weight=None,
                           expert_offsets=None, pre_act=None, ws="auto"):
    """moe_expert_linear_backward: grad_x and grad_weight (either may be None;
    x is needed for grad_weight, weight for grad_x); ws: "auto" allocates it
    where it is needed."""
    d = _device(grad_out, "grad_out")
    R, K, N, dt = p.num_rows, p.in_features, p.out_features, p.dtype
    shape = (p.num_experts, p.wide, K)
    if isinstance(ws, str):
        ws = alloc_expert_linear_workspace(p, d)
    wp, wn = _scratch(ws, d)
    _run(load_library().moe_expert_linear_backward, d, p._ref, _arg(x, "x", dt, (R, K), d),
         _offsets(p, expert_offsets, d), _arg(weight, "weight", dt, shape, d),
         _arg(pre_act, "pre_act", dt, (R, p.wide), d),
         _arg(grad_out, "grad_out", dt, (R, N), d), _arg(grad_x, "grad_x", dt, (R, K), d),
         _arg(grad_weight, "grad_weight", dt, shape, d), wp, wn)


W4_FORMATS = ("int4", "int4_zero", "mxfp4")                            # moe_w4_t


@dataclass(frozen=True)
class ExpertLinearW4(_Descriptor):
    """moe_expert_linear_w4_t: the same with 4-bit weights and group scales."""
    num_rows: int
    in_features: int
    out_features: int
    num_experts: int = 1
    dtype: torch.dtype = torch.bfloat16
    activation: str = "none"
    act_limit: float = 0.0
    format: str = "int4"                            # "int4" | "int4_zero" | "mxfp4"
    group_size: int = 128
    scale_dtype: Optional[torch.dtype] = None       # None: dtype; mxfp4: uint8

    def _struct(self):
        mx = self.format == "mxfp4"
        if mx and self.scale_dtype not in (None, torch.uint8):
            raise ValueError(f"mxfp4 scales are torch.uint8, got {self.scale_dtype}")
        scale = self.dtype if mx or self.scale_dtype is None else self.scale_dtype
        return _ExpertLinearW4(self.num_rows, self.in_features, self.out_features,
                               self.num_experts, _choice(self.dtype, _DTYPES, "dtype"),
                               _choice(self.activation, _LINEAR_ACTS, "activation"),
                               self.act_limit, _choice(self.format, W4_FORMATS, "format"),
                               self.group_size, _choice(scale, _DTYPES, "scale_dtype"))

    def __post_init__(self):
        super().__post_init__()
        wide = self.out_features * (1 if self.activation in _SINGLE_ACTS else 2)
        scales = torch.uint8 if self.format == "mxfp4" else self.scale_dtype or self.dtype
        object.__setattr__(self, "wide", wide)
        object.__setattr__(self, "scales", scales)  # the scales' type


def expert_linear_w4(p: ExpertLinearW4, x, codes, scales, out, expert_offsets=None, zeros=None):
    """moe_expert_linear_w4: out = F(x W_e^T) with W_e from 4-bit codes uint8
    [E, wide, in / 2] and scales (and zeros uint8) [E, wide, in / group_size]."""
    d = _device(x, "x")
    R, K, E, dt = p.num_rows, p.in_features, p.num_experts, p.dtype
    groups = (E, p.wide, K // p.group_size if p.group_size > 0 else 0)
    _run(load_library().moe_expert_linear_w4, d, p._ref, _arg(x, "x", dt, (R, K), d),
         _offsets(p, expert_offsets, d),
         _arg(codes, "codes", torch.uint8, (E, p.wide, K // 2), d),
         _arg(scales, "scales", p.scales, groups, d),
         _arg(zeros, "zeros", torch.uint8, groups, d),
         _arg(out, "out", dt, (R, p.out_features), d))


class MoeBlock:
    """One block of a model around its expert layer: pre norm, router, MoeLayer,
    then post norm, gate, residual scale and add, and the next block's pre norm
    in the same pass.  Buffers between the steps are kept with the block, as the
    layer keeps its workspace: calls of one block must not overlap.

    ``norm`` describes both norms (dtype bfloat16, the layer's); ``router_weight``
    is [num_experts, hidden] and makes the logits, router.dtype, by a product of
    torch's: a float32 router copies the normed rows to float32 for it on every
    call (16384 x 7168 by 256 experts: 550 us, 71 with a bfloat16 one).  The batched layout has no place here: its slabs come from a
    dispatch that already routed.

    ``staged``: the pre norm's rows leave it in the layer's 8 bits too, beside the 16
    that the router reads, and the layer does not stage them again.  The codes then come
    from the norm before its rounding: the block's bits are not those without it.
    """

    def __init__(self, layer: MoeLayer, router: Router, router_weight, norm: BlockNorm,
                 pre_weight=None, post_weight=None, bias=None, staged: bool = False):
        p = layer.p
        if staged and p.act_quant == Q_BF16:
            raise ValueError("bf16 activations are not quantized: staged has no place")
        if p.layout == LAYOUT_BATCHED:
            raise ValueError("MoeBlock needs the contiguous or the indexed layout")
        if norm.dtype != torch.bfloat16:
            raise ValueError(f"the layer's streams are bfloat16, got {norm.dtype}")
        sizes_ = (p.num_tokens, p.hidden, p.top_k)
        for what, have in (("router", (router.num_tokens, p.hidden, router.top_k)),
                           ("norm", (norm.num_tokens, norm.hidden, p.top_k))):
            if have != sizes_:
                raise ValueError(f"{what} and layer differ in (tokens, hidden, top_k): "
                                 f"{have}, {sizes_}")
        if tuple(router_weight.shape) != (router.num_experts, p.hidden) \
                or router_weight.dtype != router.dtype:
            raise ValueError(f"router_weight must be {router.dtype} "
                             f"{(router.num_experts, p.hidden)}, got {router_weight.dtype} "
                             f"{tuple(router_weight.shape)}")
        self.layer, self.router, self.norm = layer, router, norm
        self.pre = replace(norm, post_norm=False, gate="none")
        self.router_weight, self.bias = router_weight, bias
        self.pre_weight, self.post_weight = pre_weight, post_weight
        dev, shape = router_weight.device, (p.num_tokens, p.hidden)
        self.hidden = torch.empty(shape, dtype=norm.dtype, device=dev)
        self.y = torch.empty(shape, dtype=norm.dtype, device=dev)
        k = (p.num_tokens, p.top_k)
        self.topk_ids = torch.empty(k, dtype=torch.int32, device=dev)
        self.topk_weights = torch.empty(k, dtype=torch.float32, device=dev)
        self.quant = {v: n for n, v in _ACT_QUANT.items()}[p.act_quant]
        self.staged = alloc_quant_outputs(norm, self.quant, dev) if staged else None

    def __call__(self, residual, normed=None, gate=None, is_padding=None, eplb=None,
                 residual_out=None, next_normed=None, next_weight=None, staged=None,
                 next_staged=None):
        """residual_out (new unless given; may be residual).  ``normed``: the
        residual's pre norm where the block before this one left it, and
        ``staged``, a dict of x_q and x_sf, the same in the layer's 8 bits where
        it left that too; with ``next_normed`` (and ``next_staged``) the next
        block's are written there, by next_weight.  With ``eplb`` the router's
        experts are its logical ones."""
        p, r = self.layer.p, self.router
        experts = p.num_experts if eplb is None else eplb["l2p"].shape[0]
        if r.num_experts != experts:
            raise ValueError(f"the router chooses from {r.num_experts} experts, the layer has "
                             f"{experts}{'' if eplb is None else ' logical ones'}")
        _arg(normed, "normed", self.norm.dtype, (p.num_tokens, p.hidden), residual.device)
        if staged is not None:
            if normed is None:
                raise ValueError("staged rows come with the normed ones the router reads")
            if p.act_quant == Q_BF16:
                raise ValueError("bf16 activations are not quantized: staged has no place")
            _arg(staged["x_q"], "x_q", torch.uint8, (p.num_tokens, p.hidden), residual.device)
            _arg(staged["x_sf"], "x_sf", *quant_shape(p.num_tokens, p.hidden, self.quant),
                 residual.device)
        with torch.cuda.device(_device(residual, "residual")):
            if normed is None:
                normed, staged = self.hidden, self.staged
                if staged is None:
                    block_norm(self.pre, residual, normed, pre_weight=self.pre_weight)
                else:
                    block_norm_quant(self.pre, residual, **staged, quant=self.quant,
                                     normed=normed, pre_weight=self.pre_weight)
            logits = torch.matmul(normed.to(self.router.dtype), self.router_weight.t())
            router_topk(self.router, logits, self.topk_ids, self.topk_weights, bias=self.bias,
                        is_padding=is_padding)
            run = self.layer if staged is None else self.layer.quantized
            rows = (normed,) if staged is None else (staged["x_q"], staged["x_sf"])
            run(*rows, self.topk_ids, self.topk_weights, out=self.y, is_padding=is_padding,
                eplb=eplb)
            if residual_out is None:
                residual_out = torch.empty_like(residual)
            after = dict(y=self.y, residual_out=residual_out, pre_weight=next_weight,
                         post_weight=self.post_weight, gate=gate)
            if next_staged is None:
                block_norm(self.norm, residual, next_normed, **after)
            else:
                block_norm_quant(self.norm, residual, **next_staged, quant=self.quant,
                                 normed=next_normed, **after)
        return residual_out
