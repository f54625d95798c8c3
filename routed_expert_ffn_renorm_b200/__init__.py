"""B200 (sm_100a) routed Mixture-of-Experts FFN forward.

Thin Python binding over the C ABI of ``libmoe.so`` (declared in
``include/moe.h``): the functions below have the C entry points' names and
only marshal arguments -- torch tensors in, device pointers and the current
CUDA stream out.  Every step of the layer runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback, and a missing or unbuildable
library raises.

    cfg = MoEConfig(hidden=5120, n_routed_experts=16, moe_intermediate_size=1024,
                    num_experts_per_tok=2, shared_intermediate_size=2048)
    ws = torch.empty(workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    status_clear(ws)
    moe_forward(cfg, x, logits, weights, out, ws)
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from functools import lru_cache
from math import prod
from typing import Optional

__all__ = [
    "MoEConfig", "MoEWeights", "MoEError", "load_library", "workspace_bytes", "moe_router_logits", "moe_route",
    "moe_budget",
    "moe_dispatch", "moe_expert_ffn", "moe_expert_gate_up", "moe_expert_down", "moe_expert_ffn_noalloc",
    "moe_combine", "moe_forward", "moe_quantize_mxfp8", "moe_quantize_nvfp4",
    "MoEWeightsMXFP8", "moe_mxfp8_pack_scales", "moe_expert_ffn_mxfp8", "moe_forward_mxfp8", "pack_mxfp8",
    "MoEWeightsNVFP4", "moe_nvfp4_pack_scales", "moe_expert_ffn_nvfp4", "moe_forward_nvfp4", "pack_nvfp4",
    "moe_ep_rank_ids", "moe_ep_pack", "moe_ep_unpack",
    "moe_forward_few", "moe_forward_few_mxfp8", "moe_forward_few_nvfp4", "FEW_MAX_TOKENS",
    "moe_linear", "linear_workspace_bytes", "moe_verify",
    "status_read", "status_clear",
    "EXPORTED_SYMBOLS", "MOE_STATUS_TIMEOUT",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")
CHECKED_LIB_PATH = os.path.join(_HERE, "libmoe_checked.so")  # built with MOE_DEBUG_BOUNDS

EXPORTED_SYMBOLS = (
    "moe_workspace_bytes", "moe_route", "moe_budget", "moe_dispatch", "moe_expert_ffn", "moe_combine",
    "moe_forward", "moe_status_read", "moe_status_clear", "moe_error_string", "moe_expert_gate_up",
    "moe_expert_down", "moe_expert_ffn_noalloc", "moe_router_logits", "moe_quantize_mxfp8", "moe_quantize_nvfp4",
    "moe_mxfp8_pack_scales", "moe_expert_ffn_mxfp8", "moe_forward_mxfp8",
    "moe_nvfp4_pack_scales", "moe_expert_ffn_nvfp4", "moe_forward_nvfp4",
    "moe_ep_rank_ids", "moe_ep_pack", "moe_ep_unpack",
    "moe_forward_few", "moe_forward_few_mxfp8", "moe_forward_few_nvfp4",
    "moe_linear_workspace_bytes", "moe_linear", "moe_verify",
)
NOALLOC_SCRATCH_BYTES = 8 << 20  # MOE_NOALLOC_SCRATCH_BYTES
FEW_MAX_TOKENS = 16  # MOE_FEW_MAX_TOKENS
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}  # MOE_ACT_*
MOE_STATUS_TIMEOUT = 1
MOE_STATUS_BOUNDS = 2
MOE_STATUS_NONFINITE = 4


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed: {msg} (code {code})")
        self.code = code


class _Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "hidden", "n_routed_experts", "moe_intermediate_size", "num_experts_per_tok",
        "shared_intermediate_size", "norm_topk", "budget")] + [("topp", ctypes.c_float)]


class _Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down", "ws_gate_vec", "w_router")]


class _WeightsMXFP8(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_gate", "w_up", "w_down", "w_gate_scale", "w_up_scale", "w_down_scale", "ws_gate", "ws_up", "ws_down",
        "ws_gate_scale", "ws_up_scale", "ws_down_scale", "ws_gate_vec", "w_router")]


class _WeightsNVFP4(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "w_gate", "w_up", "w_down", "w_gate_scale", "w_up_scale", "w_down_scale", "w_gate_tscale", "w_up_tscale",
        "w_down_tscale", "ws_gate", "ws_up", "ws_down", "ws_gate_scale", "ws_up_scale", "ws_down_scale",
        "ws_tscale", "ws_gate_vec", "w_router")]


class _Aux(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_idx", "topk_w", "sgate", "keff", "expert_kept", "n_dropped", "counts", "offsets", "perm",
        "slot_pos", "logits")]


@dataclass(frozen=True)
class MoEConfig:
    """The layer's configuration keys (names as in the drafter config files)."""
    hidden: int
    n_routed_experts: int
    moe_intermediate_size: int
    num_experts_per_tok: int
    shared_intermediate_size: int = 0
    norm_topk: bool = True
    budget: int = 0
    topp: float = 0.0  # per-token top-p trim; 0 (or >= 1) = off

    def _c(self) -> _Config:
        return _Config(self.hidden, self.n_routed_experts, self.moe_intermediate_size, self.num_experts_per_tok,
                       self.shared_intermediate_size, int(bool(self.norm_topk)), self.budget, float(self.topp))


@dataclass
class MoEWeights:
    """Device bf16 weights: w_gate, w_up [E, I, H]; w_down [E, H, I];
    optional shared expert ws_gate, ws_up [Is, H], ws_down [H, Is], ws_gate_vec [H];
    optional router projection w_router [E, H] (used when moe_forward gets no logits)."""
    w_gate: "torch.Tensor"
    w_up: "torch.Tensor"
    w_down: "torch.Tensor"
    ws_gate: Optional["torch.Tensor"] = None
    ws_up: Optional["torch.Tensor"] = None
    ws_down: Optional["torch.Tensor"] = None
    ws_gate_vec: Optional["torch.Tensor"] = None
    w_router: Optional["torch.Tensor"] = None

    def _c(self) -> _Weights:
        return _Weights(*(_ptr(getattr(self, n), allow_none=True) for n in (
            "w_gate", "w_up", "w_down", "ws_gate", "ws_up", "ws_down", "ws_gate_vec", "w_router")))


@dataclass
class MoEWeightsMXFP8:
    """Device MXFP8 expert weights: E4M3 codes (uint8) in the bf16 weights'
    shapes -- w_gate, w_up [E, I, H], w_down [E, H, I], optional shared
    ws_gate, ws_up [Is, H], ws_down [H, Is] -- and each matrix's UE8M0 scales
    in the FFN's packed layout (moe_mxfp8_pack_scales); ws_gate_vec [H] and
    w_router [E, H] stay bf16.  pack_mxfp8() builds one from MoEWeights."""
    w_gate: "torch.Tensor"
    w_up: "torch.Tensor"
    w_down: "torch.Tensor"
    w_gate_scale: "torch.Tensor"
    w_up_scale: "torch.Tensor"
    w_down_scale: "torch.Tensor"
    ws_gate: Optional["torch.Tensor"] = None
    ws_up: Optional["torch.Tensor"] = None
    ws_down: Optional["torch.Tensor"] = None
    ws_gate_scale: Optional["torch.Tensor"] = None
    ws_up_scale: Optional["torch.Tensor"] = None
    ws_down_scale: Optional["torch.Tensor"] = None
    ws_gate_vec: Optional["torch.Tensor"] = None
    w_router: Optional["torch.Tensor"] = None

    def _c(self) -> _WeightsMXFP8:
        return _WeightsMXFP8(*(_ptr(getattr(self, n), allow_none=True) for n, _ in _WeightsMXFP8._fields_))


@dataclass
class MoEWeightsNVFP4:
    """Device NVFP4 expert weights: E2M1 codes (uint8, two per byte, the
    lower K in the low nibble) -- w_gate, w_up [E, I, H // 2], w_down
    [E, H, I // 2], optional shared ws_gate, ws_up [Is, H // 2], ws_down
    [H, Is // 2] -- each matrix's E4M3 block scales in the FFN's packed
    layout (moe_nvfp4_pack_scales), and the fp32 matrix scales: w_*_tscale
    [E] and ws_tscale [3] (shared gate, up, down).  ws_gate_vec [H] and
    w_router [E, H] stay bf16.  pack_nvfp4() builds one from MoEWeights."""
    w_gate: "torch.Tensor"
    w_up: "torch.Tensor"
    w_down: "torch.Tensor"
    w_gate_scale: "torch.Tensor"
    w_up_scale: "torch.Tensor"
    w_down_scale: "torch.Tensor"
    w_gate_tscale: "torch.Tensor"
    w_up_tscale: "torch.Tensor"
    w_down_tscale: "torch.Tensor"
    ws_gate: Optional["torch.Tensor"] = None
    ws_up: Optional["torch.Tensor"] = None
    ws_down: Optional["torch.Tensor"] = None
    ws_gate_scale: Optional["torch.Tensor"] = None
    ws_up_scale: Optional["torch.Tensor"] = None
    ws_down_scale: Optional["torch.Tensor"] = None
    ws_tscale: Optional["torch.Tensor"] = None
    ws_gate_vec: Optional["torch.Tensor"] = None
    w_router: Optional["torch.Tensor"] = None

    def _c(self) -> _WeightsNVFP4:
        return _WeightsNVFP4(*(_ptr(getattr(self, n), allow_none=True) for n, _ in _WeightsNVFP4._fields_))


_torch_module = None  # imported by the first call that takes a tensor
_lib = None
_checked = None
_lock = threading.Lock()


def load_library(build_if_stale: bool = True, variant: str = "release"):
    """Load libmoe.so (building it first when missing or older than its
    sources).  variant="checked" loads libmoe_checked.so instead, the same
    library built with MOE_DEBUG_BOUNDS (range checks on the caller's index
    inputs, reported as MOE_STATUS_BOUNDS); the functions below always call
    the release library unless a test swaps it in."""
    global _lib, _checked
    if variant == "release" and _lib is not None:
        return _lib
    with _lock:
        if variant == "release" and _lib is not None:
            return _lib
        if variant == "checked" and _checked is not None:
            return _checked
        path = LIB_PATH if variant == "release" else CHECKED_LIB_PATH
        if build_if_stale:
            from . import _build
            if _build.stale(variant):
                _build.build(variant=variant)
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m routed_expert_ffn_renorm_b200._build`")
        lib = ctypes.CDLL(path)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        cfg = ctypes.POINTER(_Config)
        lib.moe_workspace_bytes.restype = sz
        lib.moe_workspace_bytes.argtypes = [cfg, i32]
        lib.moe_route.argtypes = [cfg, i32, P, P, P, P, P, P, P, P]
        lib.moe_router_logits.argtypes = [cfg, i32, P, P, P, P, sz, P]
        lib.moe_budget.argtypes = [cfg, i32, P, P, P, P, P, P, sz, P]
        lib.moe_dispatch.argtypes = [cfg, i32, P, P, P, P, P, P, P, P, P, sz, P]
        lib.moe_expert_ffn.argtypes = [cfg, i32, P, P, P, P, P, P, ctypes.POINTER(_Weights), P, P, sz, P]
        lib.moe_combine.argtypes = [cfg, i32, P, P, P, P]
        lib.moe_expert_gate_up.argtypes = [cfg, i32, P, P, P, ctypes.POINTER(_Weights), P, sz, P]
        lib.moe_expert_down.argtypes = [cfg, i32, P, P, P, P, ctypes.POINTER(_Weights), P, P, sz, P]
        lib.moe_expert_ffn_noalloc.argtypes = [cfg, i32, P, P, P, P, P, P, ctypes.POINTER(_Weights), P, P, P]
        lib.moe_forward.argtypes = [cfg, i32, P, P, ctypes.POINTER(_Weights), P, ctypes.POINTER(_Aux), P, sz, P]
        lib.moe_status_read.argtypes = [P, ctypes.POINTER(i32), P]
        lib.moe_status_clear.argtypes = [P, P]
        i64 = ctypes.c_int64
        lib.moe_quantize_mxfp8.argtypes = [i64, i32, P, P, P, P]
        lib.moe_quantize_nvfp4.argtypes = [i32, i64, i32, P, P, P, P, P]
        lib.moe_mxfp8_pack_scales.argtypes = [i64, i32, P, P, P]
        lib.moe_ep_rank_ids.argtypes = [i32, i32, i32, P, P, P]
        lib.moe_ep_pack.argtypes = [i32, P, i32, P, P, P, P, P, P]
        lib.moe_ep_unpack.argtypes = [cfg, i32, i32, P, P, P, P, P]
        lib.moe_expert_ffn_mxfp8.argtypes = [cfg, i32, P, P, P, P, P, P, ctypes.POINTER(_WeightsMXFP8), P, P, sz, P]
        lib.moe_forward_mxfp8.argtypes = [cfg, i32, P, P, ctypes.POINTER(_WeightsMXFP8), P, ctypes.POINTER(_Aux), P,
                                          sz, P]
        lib.moe_nvfp4_pack_scales.argtypes = [i64, i32, P, P, P]
        lib.moe_expert_ffn_nvfp4.argtypes = [cfg, i32, P, P, P, P, P, P, ctypes.POINTER(_WeightsNVFP4), P, P, sz, P]
        lib.moe_forward_nvfp4.argtypes = [cfg, i32, P, P, ctypes.POINTER(_WeightsNVFP4), P, ctypes.POINTER(_Aux), P,
                                          sz, P]
        for name, wt in (("moe_forward_few", _Weights), ("moe_forward_few_mxfp8", _WeightsMXFP8),
                         ("moe_forward_few_nvfp4", _WeightsNVFP4)):
            getattr(lib, name).argtypes = [cfg, i32, P, P, ctypes.POINTER(wt), P, ctypes.POINTER(_Aux), P, sz, P]
        lib.moe_linear_workspace_bytes.restype = sz
        lib.moe_linear_workspace_bytes.argtypes = [i32, i32, i32]
        lib.moe_linear.argtypes = [i32, i32, i32, P, P, P, i32, P, P, i32, P, sz, P]
        lib.moe_verify.argtypes = [i32, i32, i32, P, P, P, P, P, P, P, P, P]
        lib.moe_error_string.restype = ctypes.c_char_p
        lib.moe_error_string.argtypes = [ctypes.c_int]
        for name in EXPORTED_SYMBOLS:
            if name not in ("moe_workspace_bytes", "moe_linear_workspace_bytes", "moe_error_string"):
                getattr(lib, name).restype = ctypes.c_int
        if variant == "release":
            _lib = lib
        else:
            _checked = lib
        return lib


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t, allow_none: bool = False):
    if t is None:
        if allow_none:
            return None
        raise ValueError("tensor argument is None")
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _expect(t, dtype, numel: int, name: str):
    """Host-side size check of a tensor the library writes or reads in full:
    a wrong dtype or a short buffer would otherwise become an out-of-bounds
    device access."""
    if t.dtype != dtype or t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements of {dtype}, got {t.numel()} of {t.dtype}")


def _stream(stream):
    if stream is None:  # torch.cuda.current_stream() without building the Stream object: 4 us of a 15 us call
        c = _torch()._C
        return c._cuda_getCurrentRawStream(c._cuda_getDevice())
    return stream.cuda_stream


def _check(fn: str, rc: int):
    if rc != 0:
        msg = load_library().moe_error_string(rc).decode()
        raise MoEError(fn, rc, msg)


def workspace_bytes(cfg: MoEConfig, T: int) -> int:
    n = load_library().moe_workspace_bytes(ctypes.byref(cfg._c()), T)
    if n == 0:
        raise MoEError("moe_workspace_bytes", -1, "invalid configuration")
    return int(n)


def moe_router_logits(cfg: MoEConfig, x, w_router, logits, ws, stream=None):
    """logits [T, E] f32 = x [T, H] . w_router [E, H]^T on the tensor cores."""
    T = x.shape[0]
    _check("moe_router_logits", load_library().moe_router_logits(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(w_router), _ptr(logits), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_quantize_mxfp8(w, codes, scales, stream=None):
    """MXFP8 weights: w [..., K] bf16 -> codes [..., K] uint8 (E4M3) and
    scales [..., K // 32] uint8 (UE8M0), blocks along the last axis."""
    import torch
    K = w.shape[-1]
    _expect(w, torch.bfloat16, w.numel(), "w")
    _expect(codes, torch.uint8, w.numel(), "codes")
    _expect(scales, torch.uint8, w.numel() // 32, "scales")
    _check("moe_quantize_mxfp8", load_library().moe_quantize_mxfp8(
        w.numel() // K, K, _ptr(w), _ptr(codes), _ptr(scales), _stream(stream)))


def moe_quantize_nvfp4(w, codes, scales, tensor_scale, stream=None):
    """NVFP4 weights: w [nmat, rows, K] bf16 -> codes [nmat, rows, K // 2]
    uint8 (two E2M1 per byte, element 2i low), scales [nmat, rows, K // 16]
    uint8 (E4M3), tensor_scale [nmat] fp32 (one per matrix)."""
    import torch
    nmat, rows, K = w.shape
    _expect(w, torch.bfloat16, w.numel(), "w")
    _expect(codes, torch.uint8, w.numel() // 2, "codes")
    _expect(scales, torch.uint8, w.numel() // 16, "scales")
    _expect(tensor_scale, torch.float32, nmat, "tensor_scale")
    _check("moe_quantize_nvfp4", load_library().moe_quantize_nvfp4(
        nmat, rows, K, _ptr(w), _ptr(codes), _ptr(scales), _ptr(tensor_scale), _stream(stream)))


def moe_mxfp8_pack_scales(scales, packed, stream=None):
    """MXFP8 scales [rows, K // 32] uint8 -> the FFN's layout
    [rows / 64][K / 128][64][4] (rows % 64 == 0, K % 128 == 0)."""
    import torch
    kb = scales.shape[-1]
    _expect(scales, torch.uint8, scales.numel(), "scales")
    _expect(packed, torch.uint8, scales.numel(), "packed")
    _check("moe_mxfp8_pack_scales", load_library().moe_mxfp8_pack_scales(
        scales.numel() // kb, kb * 32, _ptr(scales), _ptr(packed), _stream(stream)))


def pack_mxfp8(weights: MoEWeights, stream=None) -> MoEWeightsMXFP8:
    """Quantise every expert matrix of `weights` to MXFP8 on the GPU
    (moe_quantize_mxfp8, then moe_mxfp8_pack_scales); the gate vector and
    the router projection are passed through.  Allocates the outputs."""
    import torch

    def one(w):
        codes = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
        scales = torch.empty(w.shape[:-1] + (w.shape[-1] // 32,), dtype=torch.uint8, device=w.device)
        moe_quantize_mxfp8(w, codes, scales, stream=stream)
        packed = torch.empty_like(scales)
        moe_mxfp8_pack_scales(scales, packed, stream=stream)
        return codes, packed

    (g, gs), (u, us), (d, ds) = one(weights.w_gate), one(weights.w_up), one(weights.w_down)
    out = MoEWeightsMXFP8(g, u, d, gs, us, ds, ws_gate_vec=weights.ws_gate_vec, w_router=weights.w_router)
    if weights.ws_gate is not None:
        (out.ws_gate, out.ws_gate_scale), (out.ws_up, out.ws_up_scale), (out.ws_down, out.ws_down_scale) = (
            one(weights.ws_gate), one(weights.ws_up), one(weights.ws_down))
    return out


def moe_expert_ffn_mxfp8(cfg: MoEConfig, x, x_perm, offsets, perm, topk_w, weights: MoEWeightsMXFP8, ybuf, ws, *,
                         sgate=None, stream=None):
    """moe_expert_ffn with MXFP8 expert weights."""
    T = x.shape[0]
    w = weights._c()
    _check("moe_expert_ffn_mxfp8", load_library().moe_expert_ffn_mxfp8(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(x_perm), _ptr(offsets), _ptr(perm), _ptr(topk_w),
        _ptr(sgate, True), ctypes.byref(w), _ptr(ybuf), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_forward_mxfp8(cfg: MoEConfig, x, logits, weights: MoEWeightsMXFP8, out, ws, *, aux: Optional[dict] = None,
                      stream=None):
    """moe_forward with MXFP8 expert weights (arguments as moe_forward)."""
    T = x.shape[0]
    w = weights._c()
    a = _Aux()
    if aux:
        for name, t in aux.items():
            setattr(a, name, _ptr(t))
    _check("moe_forward_mxfp8", load_library().moe_forward_mxfp8(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(logits, True), ctypes.byref(w), _ptr(out), ctypes.byref(a),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_nvfp4_pack_scales(scales, packed, stream=None):
    """NVFP4 block scales [rows, K // 16] uint8 -> the FFN's layout
    [rows / 64][K / 128][64][8] (rows % 64 == 0, K % 128 == 0)."""
    import torch
    kb = scales.shape[-1]
    _expect(scales, torch.uint8, scales.numel(), "scales")
    _expect(packed, torch.uint8, scales.numel(), "packed")
    _check("moe_nvfp4_pack_scales", load_library().moe_nvfp4_pack_scales(
        scales.numel() // kb, kb * 16, _ptr(scales), _ptr(packed), _stream(stream)))


def pack_nvfp4(weights: MoEWeights, stream=None) -> MoEWeightsNVFP4:
    """Quantise every expert matrix of `weights` to NVFP4 on the GPU
    (moe_quantize_nvfp4 with one matrix scale per expert matrix, then
    moe_nvfp4_pack_scales); the gate vector and the router projection are
    passed through.  Allocates the outputs."""
    import torch

    def one(w, tscale):
        w3 = w.reshape((-1,) + tuple(w.shape[-2:]))
        codes = torch.empty(w.shape[:-1] + (w.shape[-1] // 2,), dtype=torch.uint8, device=w.device)
        scales = torch.empty(w.shape[:-1] + (w.shape[-1] // 16,), dtype=torch.uint8, device=w.device)
        moe_quantize_nvfp4(w3, codes, scales, tscale, stream=stream)
        packed = torch.empty_like(scales)
        moe_nvfp4_pack_scales(scales, packed, stream=stream)
        return codes, packed

    E = weights.w_gate.shape[0]
    ts = torch.empty(3, E, dtype=torch.float32, device=weights.w_gate.device)
    (g, gs), (u, us), (d, ds) = (one(weights.w_gate, ts[0]), one(weights.w_up, ts[1]), one(weights.w_down, ts[2]))
    out = MoEWeightsNVFP4(g, u, d, gs, us, ds, ts[0], ts[1], ts[2], ws_gate_vec=weights.ws_gate_vec,
                          w_router=weights.w_router)
    if weights.ws_gate is not None:
        out.ws_tscale = torch.empty(3, dtype=torch.float32, device=weights.ws_gate.device)
        (out.ws_gate, out.ws_gate_scale), (out.ws_up, out.ws_up_scale), (out.ws_down, out.ws_down_scale) = (
            one(weights.ws_gate, out.ws_tscale[0:1]), one(weights.ws_up, out.ws_tscale[1:2]),
            one(weights.ws_down, out.ws_tscale[2:3]))
    return out


def moe_expert_ffn_nvfp4(cfg: MoEConfig, x, x_perm, offsets, perm, topk_w, weights: MoEWeightsNVFP4, ybuf, ws, *,
                         sgate=None, stream=None):
    """moe_expert_ffn with NVFP4 expert weights."""
    T = x.shape[0]
    w = weights._c()
    _check("moe_expert_ffn_nvfp4", load_library().moe_expert_ffn_nvfp4(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(x_perm), _ptr(offsets), _ptr(perm), _ptr(topk_w),
        _ptr(sgate, True), ctypes.byref(w), _ptr(ybuf), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_forward_nvfp4(cfg: MoEConfig, x, logits, weights: MoEWeightsNVFP4, out, ws, *, aux: Optional[dict] = None,
                      stream=None):
    """moe_forward with NVFP4 expert weights (arguments as moe_forward)."""
    T = x.shape[0]
    w = weights._c()
    a = _Aux()
    if aux:
        for name, t in aux.items():
            setattr(a, name, _ptr(t))
    _check("moe_forward_nvfp4", load_library().moe_forward_nvfp4(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(logits, True), ctypes.byref(w), _ptr(out), ctypes.byref(a),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_ep_rank_ids(topk_idx, rank_idx, experts_per_rank: int, stream=None):
    """rank_idx = topk_idx // experts_per_rank (-1 stays -1): the rank holding each slot's expert."""
    T, k = topk_idx.shape
    _check("moe_ep_rank_ids", load_library().moe_ep_rank_ids(T, k, experts_per_rank, _ptr(topk_idx), _ptr(rank_idx),
                                                             _stream(stream)))


def moe_ep_pack(n_sent, perm, topk_idx, topk_w, local_idx, local_w, experts_per_rank: int, stream=None):
    """For the first n_sent[0] (device) entries p of perm: local_idx[p] =
    topk_idx[perm[p]] % experts_per_rank, local_w[p] = topk_w[perm[p]]."""
    _check("moe_ep_pack", load_library().moe_ep_pack(
        local_idx.numel(), _ptr(n_sent), experts_per_rank, _ptr(perm), _ptr(topk_idx), _ptr(topk_w), _ptr(local_idx),
        _ptr(local_w), _stream(stream)))


def moe_ep_unpack(cfg: MoEConfig, T: int, n_returned, perm, rows, ybuf, stream=None):
    """ybuf[s + s // k] = rows[p] for p < n_returned[0] (device), s = perm[p]."""
    _check("moe_ep_unpack", load_library().moe_ep_unpack(
        ctypes.byref(cfg._c()), T, rows.shape[0], _ptr(n_returned), _ptr(perm), _ptr(rows), _ptr(ybuf),
        _stream(stream)))


def moe_route(cfg: MoEConfig, logits, topk_idx, topk_w, *, x=None, ws_gate_vec=None, sgate=None, keff=None,
              stream=None):
    T = logits.shape[0]
    _check("moe_route", load_library().moe_route(
        ctypes.byref(cfg._c()), T, _ptr(logits), _ptr(x, True), _ptr(ws_gate_vec, True), _ptr(topk_idx),
        _ptr(topk_w), _ptr(sgate, True), _ptr(keff, True), _stream(stream)))


def moe_budget(cfg: MoEConfig, topk_idx, topk_w, keff, expert_kept, n_dropped, ws, stream=None):
    T = topk_idx.shape[0]
    _check("moe_budget", load_library().moe_budget(
        ctypes.byref(cfg._c()), T, _ptr(topk_idx), _ptr(topk_w), _ptr(keff), _ptr(expert_kept), _ptr(n_dropped),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_dispatch(cfg: MoEConfig, topk_idx, counts, offsets, perm, slot_pos, ws, *, keff=None, x=None, x_perm=None,
                 stream=None):
    T = topk_idx.shape[0]
    _check("moe_dispatch", load_library().moe_dispatch(
        ctypes.byref(cfg._c()), T, _ptr(topk_idx), _ptr(keff, True), _ptr(x, True), _ptr(counts), _ptr(offsets),
        _ptr(perm), _ptr(slot_pos), _ptr(x_perm, True), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_expert_ffn(cfg: MoEConfig, x, x_perm, offsets, perm, topk_w, weights: MoEWeights, ybuf, ws, *, sgate=None,
                   stream=None):
    T = x.shape[0]
    w = weights._c()
    _check("moe_expert_ffn", load_library().moe_expert_ffn(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(x_perm), _ptr(offsets), _ptr(perm), _ptr(topk_w),
        _ptr(sgate, True), ctypes.byref(w), _ptr(ybuf), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def moe_expert_gate_up(cfg: MoEConfig, x, x_perm, offsets, weights: MoEWeights, ws, stream=None):
    T = x.shape[0]
    w = weights._c()
    _check("moe_expert_gate_up", load_library().moe_expert_gate_up(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(x_perm), _ptr(offsets), ctypes.byref(w), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def moe_expert_down(cfg: MoEConfig, T: int, offsets, perm, topk_w, weights: MoEWeights, ybuf, ws, *, sgate=None,
                    stream=None):
    w = weights._c()
    _check("moe_expert_down", load_library().moe_expert_down(
        ctypes.byref(cfg._c()), T, _ptr(offsets), _ptr(perm), _ptr(topk_w), _ptr(sgate, True), ctypes.byref(w),
        _ptr(ybuf), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_expert_ffn_noalloc(cfg: MoEConfig, x, x_perm, offsets, perm, topk_w, weights: MoEWeights, ybuf, *,
                           sgate=None, device_status=None, stream=None):
    """moe_expert_ffn without a workspace, for callers that cannot allocate
    device memory: the scratch lives in a fixed 8 MiB device array inside the
    library (batches needing more raise MoEError with code -3).  Calls whose
    work overlaps on the GPU share that array and must not run concurrently."""
    T = x.shape[0]
    w = weights._c()
    _check("moe_expert_ffn_noalloc", load_library().moe_expert_ffn_noalloc(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(x_perm), _ptr(offsets), _ptr(perm), _ptr(topk_w), _ptr(sgate, True),
        ctypes.byref(w), _ptr(ybuf), _ptr(device_status, True), _stream(stream)))


def moe_combine(cfg: MoEConfig, ybuf, out, *, keff=None, stream=None):
    T = out.shape[0]
    _check("moe_combine", load_library().moe_combine(
        ctypes.byref(cfg._c()), T, _ptr(ybuf), _ptr(keff, True), _ptr(out), _stream(stream)))


def moe_forward(cfg: MoEConfig, x, logits, weights: MoEWeights, out, ws, *, aux: Optional[dict] = None,
                stream=None):
    """The whole layer on the current stream.  ``logits`` may be None when
    ``weights.w_router`` is set: the router projection computes them.
    ``aux`` may map moe_aux_t member names (topk_idx, topk_w, sgate, keff,
    expert_kept, n_dropped, counts, offsets, perm, slot_pos, logits) to
    device tensors to receive them."""
    T = x.shape[0]
    w = weights._c()
    a = _Aux()
    if aux:
        for name, t in aux.items():
            setattr(a, name, _ptr(t))
    _check("moe_forward", load_library().moe_forward(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(logits, True), ctypes.byref(w), _ptr(out), ctypes.byref(a),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def _expect_like(t, dtype, shape, device, name: str):
    """Host-side check of one tensor of a call: type, shape (a tuple) and device index."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)} on cuda:{device}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")


def _expect_device(t, device: int, name: str):
    if t.get_device() != device:
        raise ValueError(f"{name}: expected on cuda:{device}, got {t.device}")


def _current_device(t, name: str):
    """The launch goes to the current device (its index is returned): its tensors have to live there."""
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}: tensors must live on a CUDA device")
    if t.get_device() != _torch()._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_torch().cuda.current_device()}")
    return t.get_device()


@lru_cache(maxsize=64)
def _few_weight_spec(fn: str, H: int, E: int, I: int, Is: int, router: bool):
    """(field, type, shape, or element count where the layout is packed) of the weights the call reads."""
    torch = _torch()
    bits = {"moe_forward_few": 16, "moe_forward_few_mxfp8": 8, "moe_forward_few_nvfp4": 4}[fn]
    per = 2 if bits == 4 else 1  # weights per element
    mats = [("w_gate", (E, I, H)), ("w_up", (E, I, H)), ("w_down", (E, H, I))]
    if Is:
        mats += [("ws_gate", (Is, H)), ("ws_up", (Is, H)), ("ws_down", (H, Is))]
    spec = []
    for name, shape in mats:
        spec.append((name, torch.bfloat16 if bits == 16 else torch.uint8, shape[:-1] + (shape[-1] // per,)))
        if bits < 16:
            spec.append((name + "_scale", torch.uint8, prod(shape) // (4 * bits)))  # 32 or 16 weights a scale
        if bits == 4 and len(shape) == 3:
            spec.append((name + "_tscale", torch.float32, E))
    if Is:
        spec.append(("ws_gate_vec", torch.bfloat16, (H,)))
        if bits == 4:
            spec.append(("ws_tscale", torch.float32, 3))
    if router:
        spec.append(("w_router", torch.bfloat16, (E, H)))
    return tuple(spec)


def _check_few_weights(fn: str, cfg: MoEConfig, weights, device: int, router: bool):
    """The call's weight pointers.  The kernel reads every weight in full: a tensor of another type, size or
    device would become an out-of-bounds access."""
    ptrs = {}
    for name, dtype, shape in _few_weight_spec(fn, cfg.hidden, cfg.n_routed_experts, cfg.moe_intermediate_size,
                                               cfg.shared_intermediate_size, router):
        t = getattr(weights, name, None)
        if t is None:
            raise ValueError(f"{name} is missing from the weights")
        if t.dtype is not dtype or t.get_device() != device or (
                t.numel() if type(shape) is int else t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} {shape} on cuda:{device}, got {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
        ptrs[name] = t.data_ptr()
    return _FEW_STRUCTS[fn](**ptrs)


_FEW_STRUCTS = {"moe_forward_few": _Weights, "moe_forward_few_mxfp8": _WeightsMXFP8,
                "moe_forward_few_nvfp4": _WeightsNVFP4}


def _few_aux(cfg: MoEConfig, T: int, aux: dict, device: int) -> _Aux:
    torch = _torch()
    E, Tk = cfg.n_routed_experts, T * cfg.num_experts_per_tok
    least = {"topk_idx": (torch.int32, Tk), "topk_w": (torch.float32, Tk), "sgate": (torch.float32, T),
             "keff": (torch.int32, T), "expert_kept": (torch.uint8, E), "n_dropped": (torch.int32, 1),
             "logits": (torch.float32, T * E)}
    a = _Aux()
    for name, t in aux.items():
        if not hasattr(a, name):
            raise ValueError(f"aux: no output {name!r}")
        if name in least and t is not None:  # (the others the call refuses)
            dtype, n = least[name]
            if t.dtype is not dtype or t.numel() < n or t.get_device() != device:
                raise ValueError(f"aux {name}: expected {n} elements of {dtype} on cuda:{device}, got {t.numel()} of "
                                 f"{t.dtype} on {t.device}")
        setattr(a, name, _ptr(t))
    return a


def _forward_few(fn: str, cfg: MoEConfig, x, logits, weights, out, ws, aux, stream):
    torch = _torch()
    dev = _current_device(x, "x")
    T, H, E = x.shape[0], cfg.hidden, cfg.n_routed_experts
    _expect_like(x, torch.bfloat16, (T, H), dev, "x")
    _expect_like(out, torch.bfloat16, (T, H), dev, "out")
    if logits is not None:
        _expect_like(logits, torch.float32, (T, E), dev, "logits")
    elif weights.w_router is None:
        raise ValueError("logits is None and the weights have no w_router")
    w = _check_few_weights(fn, cfg, weights, dev, logits is None)
    _expect_device(ws, dev, "ws")
    a = _few_aux(cfg, T, aux, dev) if aux else _Aux()
    _check(fn, getattr(load_library(), fn)(
        ctypes.byref(cfg._c()), T, _ptr(x), _ptr(logits, True), ctypes.byref(w), _ptr(out), ctypes.byref(a),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_forward_few(cfg: MoEConfig, x, logits, weights: MoEWeights, out, ws, *, aux: Optional[dict] = None,
                    stream=None):
    """The whole layer for at most FEW_MAX_TOKENS tokens in one kernel
    (arguments as moe_forward; aux without counts, offsets, perm, slot_pos)."""
    _forward_few("moe_forward_few", cfg, x, logits, weights, out, ws, aux, stream)


def moe_forward_few_mxfp8(cfg: MoEConfig, x, logits, weights: MoEWeightsMXFP8, out, ws, *,
                          aux: Optional[dict] = None, stream=None):
    """moe_forward_few with MXFP8 expert weights."""
    _forward_few("moe_forward_few_mxfp8", cfg, x, logits, weights, out, ws, aux, stream)


def moe_forward_few_nvfp4(cfg: MoEConfig, x, logits, weights: MoEWeightsNVFP4, out, ws, *,
                          aux: Optional[dict] = None, stream=None):
    """moe_forward_few with NVFP4 expert weights."""
    _forward_few("moe_forward_few_nvfp4", cfg, x, logits, weights, out, ws, aux, stream)


def linear_workspace_bytes(T: int, N: int, K: int) -> int:
    """Workspace of moe_linear for x [T, K] and w [N, K] (status_clear it once)."""
    n = load_library().moe_linear_workspace_bytes(T, N, K)
    if n == 0:
        raise MoEError("moe_linear_workspace_bytes", -1, "invalid sizes")
    return int(n)


def moe_linear(x, w, out, ws, *, bias=None, activation: str = "none", residual=None, stream=None):
    """out [T, N] = residual + act(x [T, K] . w [N, K]^T + bias): bf16 in, out
    bf16 or fp32 by its type; activation "none", "relu", "gelu" (erf) or
    "silu"; out may be `residual` itself."""
    torch = _torch()
    dev = _current_device(x, "x")
    (T, K), N = x.shape, w.shape[0]
    _expect_like(x, torch.bfloat16, (T, K), dev, "x")
    _expect_like(w, torch.bfloat16, (N, K), dev, "w")
    if out.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"out: expected bfloat16 or float32, got {out.dtype}")
    _expect_like(out, out.dtype, (T, N), dev, "out")
    if bias is not None:
        _expect_like(bias, torch.bfloat16, (N,), dev, "bias")
    if residual is not None:
        _expect_like(residual, torch.bfloat16, (T, N), dev, "residual")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation: one of {sorted(ACTIVATIONS)}, got {activation!r}")
    _expect_device(ws, dev, "ws")
    _check("moe_linear", load_library().moe_linear(
        T, N, K, _ptr(x), _ptr(w), _ptr(bias, True), ACTIVATIONS[activation], _ptr(residual, True), _ptr(out),
        int(out.dtype == torch.float32), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def moe_verify(target_probs, draft_tokens, accept_u, sample_u, tokens, n_accepted, *, draft_probs=None,
               draft_len=None, stream=None):
    """Drafted tokens [B, L] against the target's probabilities [B, L + 1, V]
    with given random numbers accept_u [B, L] and sample_u [B]: tokens
    [B, L + 1] receives the kept tokens, the drawn one and -1 behind it,
    n_accepted [B] how many stayed.  draft_probs [B, L, V], or None for a
    drafter that puts all its mass on its token; draft_len [B] for blocks
    shorter than L."""
    torch = _torch()
    dev = _current_device(target_probs, "target_probs")
    B, L1, V = target_probs.shape
    L = L1 - 1
    f32, i32 = torch.float32, torch.int32
    _expect_like(target_probs, f32, (B, L1, V), dev, "target_probs")
    _expect_like(draft_tokens, i32, (B, L), dev, "draft_tokens")
    _expect_like(accept_u, f32, (B, L), dev, "accept_u")
    _expect_like(sample_u, f32, (B,), dev, "sample_u")
    _expect_like(tokens, i32, (B, L1), dev, "tokens")
    _expect_like(n_accepted, i32, (B,), dev, "n_accepted")
    if draft_probs is not None:
        _expect_like(draft_probs, f32, (B, L, V), dev, "draft_probs")
    if draft_len is not None:
        _expect_like(draft_len, i32, (B,), dev, "draft_len")
    _check("moe_verify", load_library().moe_verify(
        B, L, V, _ptr(target_probs), _ptr(draft_probs, True), _ptr(draft_tokens), _ptr(draft_len, True),
        _ptr(accept_u), _ptr(sample_u), _ptr(tokens), _ptr(n_accepted), _stream(stream)))


def status_read(ws, stream=None) -> int:
    v = ctypes.c_int32(0)
    _check("moe_status_read", load_library().moe_status_read(_ptr(ws), ctypes.byref(v), _stream(stream)))
    return int(v.value)


def status_clear(ws, stream=None):
    _check("moe_status_clear", load_library().moe_status_clear(_ptr(ws), _stream(stream)))
