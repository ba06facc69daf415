"""Python binding of libmoelora (ctypes).  Argument marshalling only: every
step of the layer runs in the HIP library; PyTorch provides device memory and
streams.  The functions carry the C ABI's names (``build_pool``,
``moe_lora_forward``, ``moe_lora_backward``, ...); see include/moelora.h for
the contract of each call.

If the shared library is missing or fails to load, every call raises: there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional, Sequence, Tuple

import torch

from . import build as _build

LIB_PATH = _build.OUT

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_ACT_SWIGLU = 0
MOE_ACT_GEGLU = 1
MOE_BASE_BF16, MOE_BASE_MXFP4 = 0, 1
# the saved workspace's device status word (include/moelora.h)
MOE_SAVED_STATUS_OFFSET = 0
MOE_SAVED_FP16_RANGE = 1
MOE_MAX_ADAPTERS = 64
MOE_TYPE_F32, MOE_TYPE_BF16 = 0, 1
MOE_FP8_PLAIN = -1

EXPORTS = (
    "moe_lora_status_string", "moe_lora_version", "moe_lora_block_m", "moe_lora_pool_capacity",
    "moe_lora_workspace_size", "build_pool", "moe_lora_forward", "moe_lora_forward_noalloc", "moe_lora_backward",
    "moe_lora_transform_base", "moe_lora_split_e2m3x2", "moe_lora_trace_enable", "moe_lora_trace_collect", "moe_lora_trace_count",
    "moe_lora_trace_entry", "moe_lora_trace_reset", "moe_lora_multi_pool_capacity",
    "moe_lora_multi_workspace_size", "build_pool_multi", "moe_lora_forward_multi", "moe_lora_backward_multi",
    "moe_router_workspace_size", "moe_router_forward", "moe_router_backward", "moe_adamw_step",
    "moe_fp8_quantize_rows", "moe_fp8_quantize_weight", "moe_fp8_product",
)


class MoeLoraError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {_status_string(status)} ({status})")


class MoeLoraDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("E", ctypes.c_int32), ("topk", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("block_m", ctypes.c_int32), ("scale", ctypes.c_float),
                ("activation", ctypes.c_int32), ("clamp", ctypes.c_float),
                ("base_format", ctypes.c_int32)]


class MoePool(ctypes.Structure):
    _fields_ = [("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("route_to_row", ctypes.c_void_p), ("row_to_route", ctypes.c_void_p),
                ("capacity", ctypes.c_int64), ("block_m", ctypes.c_int32)]


class MoeLoraParams(ctypes.Structure):
    _fields_ = [("W13", ctypes.c_void_p), ("W2", ctypes.c_void_p),
                ("W13_scale", ctypes.c_void_p), ("W2_scale", ctypes.c_void_p),
                ("A1", ctypes.c_void_p), ("A3", ctypes.c_void_p), ("B1", ctypes.c_void_p),
                ("B3", ctypes.c_void_p), ("A2", ctypes.c_void_p), ("B2", ctypes.c_void_p),
                ("W13T", ctypes.c_void_p), ("W2T", ctypes.c_void_p),
                ("W13P", ctypes.c_void_p), ("W2P", ctypes.c_void_p)]


class MoeLoraGrads(ctypes.Structure):
    _fields_ = [("dA1", ctypes.c_void_p), ("dA3", ctypes.c_void_p), ("dB1", ctypes.c_void_p),
                ("dB3", ctypes.c_void_p), ("dA2", ctypes.c_void_p), ("dB2", ctypes.c_void_p),
                ("dW13", ctypes.c_void_p), ("dW2", ctypes.c_void_p)]


class MoeAdapters(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int32), ("offsets", ctypes.POINTER(ctypes.c_int32))]


class MoeRouterDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("logits_type", ctypes.c_int32), ("renorm", ctypes.c_int32)]


class MoeAdamwTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "master", "grad", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64)]


class MoeAdamwDesc(ctypes.Structure):
    _fields_ = [("param_type", ctypes.c_int32), ("grad_type", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("seed", ctypes.c_uint32)] + [
        (n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay", "grad_scale")] + [
        ("step", ctypes.c_int64), ("control", ctypes.c_void_p)]


class MoeFp8Desc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("topk", ctypes.c_int32),
                ("a_rows", ctypes.c_int64)]


def _adapters(roots: Optional[Sequence[int]]):
    """The C struct for the roots 0 = r0 <= ... <= rNA = T (None: single adapter)."""
    if roots is None:
        return None
    arr = (ctypes.c_int32 * len(roots))(*[int(v) for v in roots])
    ad = MoeAdapters(len(roots) - 1, arr)
    ad._keep = arr  # the offsets live as long as the struct
    return ad


_lib: Optional[ctypes.CDLL] = None


def library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libmoelora (once).  Raises if it is not built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libmoelora is not built ({p} missing): run "
                           "python -m mixture_experts_grouped_amd.build")
    lib = ctypes.CDLL(p)
    P = ctypes.POINTER
    vp = ctypes.c_void_p
    lib.moe_lora_status_string.argtypes = [ctypes.c_int32]
    lib.moe_lora_status_string.restype = ctypes.c_char_p
    lib.moe_lora_version.argtypes = []
    lib.moe_lora_version.restype = ctypes.c_int32
    lib.moe_lora_block_m.argtypes = [P(MoeLoraDesc), P(ctypes.c_int32)]
    lib.moe_lora_pool_capacity.argtypes = [P(MoeLoraDesc), P(ctypes.c_int64)]
    lib.moe_lora_workspace_size.argtypes = [P(MoeLoraDesc), P(ctypes.c_size_t), P(ctypes.c_size_t)]
    lib.build_pool.argtypes = [P(MoeLoraDesc), vp, vp, vp, vp, vp, ctypes.c_int64, vp, vp]
    lib.moe_lora_forward.argtypes = [P(MoeLoraDesc), P(MoePool), vp, vp, P(MoeLoraParams), vp,
                                     vp, ctypes.c_size_t, vp, ctypes.c_size_t, vp]
    lib.moe_lora_forward_noalloc.argtypes = [P(MoeLoraDesc), P(MoePool), vp, vp, P(MoeLoraParams), vp,
                                             vp, ctypes.c_size_t, vp]
    lib.moe_lora_backward.argtypes = [P(MoeLoraDesc), P(MoePool), vp, vp, P(MoeLoraParams), vp,
                                      ctypes.c_size_t, vp, vp, P(MoeLoraGrads), vp,
                                      ctypes.c_size_t, vp]
    lib.moe_lora_transform_base.argtypes = [P(MoeLoraDesc), P(MoeLoraParams), vp, vp, vp, vp, vp]
    lib.moe_lora_split_e2m3x2.argtypes = [vp, ctypes.c_int64, ctypes.c_int32, vp, vp, vp]
    lib.moe_lora_trace_enable.argtypes = [ctypes.c_int32]
    lib.moe_lora_trace_enable.restype = None
    lib.moe_lora_trace_collect.argtypes = []
    lib.moe_lora_trace_count.argtypes = []
    lib.moe_lora_trace_count.restype = ctypes.c_int32
    lib.moe_lora_trace_entry.argtypes = [ctypes.c_int32, P(ctypes.c_char_p), P(ctypes.c_int64),
                                         P(ctypes.c_double)]
    lib.moe_lora_trace_reset.argtypes = []
    lib.moe_lora_trace_reset.restype = None
    A = P(MoeAdapters)
    lib.moe_lora_multi_pool_capacity.argtypes = [P(MoeLoraDesc), A, P(ctypes.c_int64)]
    lib.moe_lora_multi_workspace_size.argtypes = [P(MoeLoraDesc), A, P(ctypes.c_size_t), P(ctypes.c_size_t)]
    lib.build_pool_multi.argtypes = [P(MoeLoraDesc), A, vp, vp, vp, vp, vp, ctypes.c_int64, vp, vp]
    lib.moe_lora_forward_multi.argtypes = [P(MoeLoraDesc), A, P(MoePool), vp, vp, P(MoeLoraParams), vp,
                                           vp, ctypes.c_size_t, vp, ctypes.c_size_t, vp]
    lib.moe_lora_backward_multi.argtypes = [P(MoeLoraDesc), A, P(MoePool), vp, vp, P(MoeLoraParams), vp,
                                            ctypes.c_size_t, vp, vp, P(MoeLoraGrads), vp, ctypes.c_size_t, vp]
    i32, i64, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    RD = P(MoeRouterDesc)
    lib.moe_router_workspace_size.argtypes = [RD, A, P(sz)]
    lib.moe_router_forward.argtypes = [RD, A, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_router_backward.argtypes = [RD, A, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.moe_adamw_step.argtypes = [P(MoeAdamwDesc), P(MoeAdamwTensor), i32, vp]
    lib.moe_fp8_quantize_rows.argtypes = [vp, i64, i32, i32, vp, vp, vp]
    lib.moe_fp8_quantize_weight.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp]
    lib.moe_fp8_product.argtypes = [P(MoeFp8Desc), P(MoePool), vp, vp, vp, vp, vp, vp]
    for fn in ("moe_router_workspace_size", "moe_router_forward", "moe_router_backward", "moe_adamw_step",
               "moe_fp8_quantize_rows", "moe_fp8_quantize_weight", "moe_fp8_product",
               "moe_lora_trace_collect", "moe_lora_trace_entry", "moe_lora_block_m", "moe_lora_pool_capacity", "moe_lora_workspace_size",
               "build_pool", "moe_lora_forward", "moe_lora_forward_noalloc", "moe_lora_backward",
               "moe_lora_transform_base", "moe_lora_split_e2m3x2", "moe_lora_multi_pool_capacity",
               "moe_lora_multi_workspace_size", "build_pool_multi", "moe_lora_forward_multi",
               "moe_lora_backward_multi"):
        getattr(lib, fn).restype = ctypes.c_int32
    if path is None:
        _lib = lib
    return lib


def _status_string(status: int) -> str:
    try:
        return library().moe_lora_status_string(status).decode()
    except Exception:  # pragma: no cover - only while reporting another error
        return "status"


def _check(status: int, what: str) -> None:
    if status != MOE_OK:
        raise MoeLoraError(status, what)


def make_desc(T: int, H: int, I: int, E: int, topk: int, rank: int, scale: float = 1.0,
              block_m: int = 0, activation: int = MOE_ACT_SWIGLU, clamp: float = 0.0,
              base_format: int = MOE_BASE_BF16) -> MoeLoraDesc:
    return MoeLoraDesc(T, H, I, E, topk, rank, block_m, scale, activation, clamp, base_format)


def moe_lora_block_m(desc: MoeLoraDesc) -> int:
    v = ctypes.c_int32()
    _check(library().moe_lora_block_m(ctypes.byref(desc), ctypes.byref(v)), "moe_lora_block_m")
    return v.value


def moe_lora_pool_capacity(desc: MoeLoraDesc) -> int:
    v = ctypes.c_int64()
    _check(library().moe_lora_pool_capacity(ctypes.byref(desc), ctypes.byref(v)),
           "moe_lora_pool_capacity")
    return v.value


def moe_lora_workspace_size(desc: MoeLoraDesc) -> Tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(library().moe_lora_workspace_size(ctypes.byref(desc), ctypes.byref(a), ctypes.byref(b)),
           "moe_lora_workspace_size")
    return a.value, b.value


def moe_lora_multi_pool_capacity(desc: MoeLoraDesc, roots: Sequence[int]) -> int:
    v = ctypes.c_int64()
    _check(library().moe_lora_multi_pool_capacity(ctypes.byref(desc), ctypes.byref(_adapters(roots)),
                                                  ctypes.byref(v)), "moe_lora_multi_pool_capacity")
    return v.value


def moe_lora_multi_workspace_size(desc: MoeLoraDesc, roots: Sequence[int]) -> Tuple[int, int]:
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(library().moe_lora_multi_workspace_size(ctypes.byref(desc), ctypes.byref(_adapters(roots)),
                                                   ctypes.byref(a), ctypes.byref(b)),
           "moe_lora_multi_workspace_size")
    return a.value, b.value


def _ptr(t: Optional[torch.Tensor], dtype=None, shape=None, name="tensor") -> Optional[int]:
    if t is None:
        return None
    if t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype is dtype) and (shape is None or t.shape == shape):
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def build_pool(desc: MoeLoraDesc, topk_idx: torch.Tensor, counts: torch.Tensor,
               offsets: torch.Tensor, route_to_row: torch.Tensor, row_to_route: torch.Tensor,
               device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    T, k, E = desc.T, desc.topk, desc.E
    cap = row_to_route.numel()
    i32 = torch.int32
    st = library().build_pool(
        ctypes.byref(desc), _ptr(topk_idx, i32, (T, k), "topk_idx"), _ptr(counts, i32, (E,), "counts"),
        _ptr(offsets, i32, (E + 1,), "offsets"), _ptr(route_to_row, i32, (T * k,), "route_to_row"),
        _ptr(row_to_route, i32, (cap,), "row_to_route"), cap,
        _ptr(device_error, i32, (1,), "device_error"), _stream(stream))
    _check(st, "build_pool")


def build_pool_multi(desc: MoeLoraDesc, roots: Sequence[int], topk_idx: torch.Tensor, counts: torch.Tensor,
                     offsets: torch.Tensor, route_to_row: torch.Tensor, row_to_route: torch.Tensor,
                     device_error: Optional[torch.Tensor] = None, stream=None) -> None:
    """build_pool with (expert, adapter) groups: counts [E * NA], offsets [E * NA + 1]."""
    T, k, G = desc.T, desc.topk, desc.E * (len(roots) - 1)
    cap = row_to_route.numel()
    i32 = torch.int32
    st = library().build_pool_multi(
        ctypes.byref(desc), ctypes.byref(_adapters(roots)), _ptr(topk_idx, i32, (T, k), "topk_idx"),
        _ptr(counts, i32, (G,), "counts"), _ptr(offsets, i32, (G + 1,), "offsets"),
        _ptr(route_to_row, i32, (T * k,), "route_to_row"), _ptr(row_to_route, i32, (cap,), "row_to_route"), cap,
        _ptr(device_error, i32, (1,), "device_error"), _stream(stream))
    _check(st, "build_pool_multi")


def _pool_struct(pool: Dict[str, torch.Tensor], bm: int) -> MoePool:
    return MoePool(pool["counts"].data_ptr(), pool["offsets"].data_ptr(),
                   pool["route_to_row"].data_ptr(), pool["row_to_route"].data_ptr(),
                   pool["row_to_route"].numel(), bm)


def _factor_shapes(desc: MoeLoraDesc, na: Optional[int] = None) -> Dict[str, Tuple[int, ...]]:
    """Adapter factor shapes; with na adapters stacked over a leading axis."""
    E, H, I, r = desc.E, desc.H, desc.I, desc.rank
    shapes = {"A1": (r, H), "A3": (r, H), "B1": (E, I, r), "B3": (E, I, r), "A2": (E, r, I), "B2": (H, r)}
    return shapes if na is None else {n: (na,) + s for n, s in shapes.items()}


def _params_struct(p: Dict[str, torch.Tensor], desc: MoeLoraDesc, na: Optional[int] = None) -> MoeLoraParams:
    """bf16 base: W13, W2 bf16.  MXFP4 base (desc.base_format == MOE_BASE_MXFP4):
    W13 uint8 [E, 2I, H/2] and W2 uint8 [E, H, I/2] packed e2m1 (element 2i in
    the low nibble of byte i), W13_scale uint8 [E, 2I, H/32], W2_scale uint8
    [E, H, I/32] e8m0.  Optional "W13T" [E, H, 2I] and "W2T" [E, I, H] bf16: the
    transformed base (transform_base), read by the backward; optional "W13P",
    "W2P": the forward's packed copies (bf16 [E, 2I, H] and [E, H, I], or for an
    MXFP4 base uint8 of 9/16 byte per weight, see mx_packed_shapes).  With na
    adapters the six factors are stacked [na, ...]."""
    E, H, I, r = desc.E, desc.H, desc.I, desc.rank
    bf = torch.bfloat16
    shapes = _factor_shapes(desc, na)
    ptrs = {n: _ptr(p[n], bf, s, n) for n, s in shapes.items()}
    if desc.base_format == MOE_BASE_MXFP4:
        u8 = torch.uint8
        w13 = _ptr(p["W13"], u8, (E, 2 * I, H // 2), "W13")
        w2 = _ptr(p["W2"], u8, (E, H, I // 2), "W2")
        s13 = _ptr(p["W13_scale"], u8, (E, 2 * I, H // 32), "W13_scale")
        s2 = _ptr(p["W2_scale"], u8, (E, H, I // 32), "W2_scale")
    else:
        w13 = _ptr(p["W13"], bf, (E, 2 * I, H), "W13")
        w2 = _ptr(p["W2"], bf, (E, H, I), "W2")
        s13 = s2 = None
    w13t = _ptr(p.get("W13T"), bf, (E, H, 2 * I), "W13T")
    w2t = _ptr(p.get("W2T"), bf, (E, I, H), "W2T")
    w13p, w2p = _packed_ptrs(desc, p.get("W13P"), p.get("W2P"))
    return MoeLoraParams(w13, w2, s13, s2, ptrs["A1"], ptrs["A3"], ptrs["B1"], ptrs["B3"],
                         ptrs["A2"], ptrs["B2"], w13t, w2t, w13p, w2p)


def mx_packed_shapes(desc: MoeLoraDesc):
    """Storage shapes of the forward's packed copies of an MXFP4 base: per
    expert, N tiles x K stages of 9216-byte stage tiles (256 rows of 32 code
    bytes, then 256 scale words) -- W13P [E, 2I/256, H/64, 9216] and W2P
    [E, H/256, I/64, 9216] uint8."""
    E, H, I = desc.E, desc.H, desc.I
    return (E, 2 * I // 256, H // 64, 9216), (E, H // 256, I // 64, 9216)


def _packed_ptrs(desc: MoeLoraDesc, W13P, W2P):
    E, H, I = desc.E, desc.H, desc.I
    if desc.base_format == MOE_BASE_MXFP4:
        s13, s2 = mx_packed_shapes(desc)
        return _ptr(W13P, torch.uint8, s13, "W13P"), _ptr(W2P, torch.uint8, s2, "W2P")
    bf = torch.bfloat16
    return _ptr(W13P, bf, (E, 2 * I, H), "W13P"), _ptr(W2P, bf, (E, H, I), "W2P")


def moe_lora_transform_base(desc: MoeLoraDesc, params: Dict[str, torch.Tensor],
                            W13T: Optional[torch.Tensor], W2T: Optional[torch.Tensor],
                            W13P: Optional[torch.Tensor] = None, W2P: Optional[torch.Tensor] = None,
                            stream=None) -> None:
    """The transformed base copies (any may be None): W13T, W2T for the
    backward (for an MXFP4 base of the dequantised weights) and W13P, W2P for
    the forward.  Library-private layouts of E x 2I x H and E x H x I bf16
    values, or for the forward copies of an MXFP4 base the byte tiles of
    mx_packed_shapes (shapes are storage only)."""
    E, H, I = desc.E, desc.H, desc.I
    bf = torch.bfloat16
    if desc.base_format == MOE_BASE_MXFP4:
        u8 = torch.uint8
        pp = MoeLoraParams(_ptr(params["W13"], u8, (E, 2 * I, H // 2), "W13"),
                           _ptr(params["W2"], u8, (E, H, I // 2), "W2"),
                           _ptr(params["W13_scale"], u8, (E, 2 * I, H // 32), "W13_scale"),
                           _ptr(params["W2_scale"], u8, (E, H, I // 32), "W2_scale"))
    else:  # the base alone: the adapter factors are not read
        pp = MoeLoraParams(_ptr(params["W13"], bf, (E, 2 * I, H), "W13"), _ptr(params["W2"], bf, (E, H, I), "W2"))
    st = library().moe_lora_transform_base(
        ctypes.byref(desc), ctypes.byref(pp), _ptr(W13T, bf, (E, H, 2 * I), "W13T"),
        _ptr(W2T, bf, (E, I, H), "W2T"), *_packed_ptrs(desc, W13P, W2P), _stream(stream))
    _check(st, "moe_lora_transform_base")


def transform_base(desc: MoeLoraDesc, params: Dict[str, torch.Tensor], stream=None,
                   forward: bool = True) -> Dict[str, torch.Tensor]:
    """Allocate and fill the transformed base copies -- W13T, W2T for the
    backward, and (forward=True) W13P, W2P for the forward -- and return
    them to merge into the params dict.  Redo it whenever W13 / W2 change
    (they are frozen in the side-LoRA setting)."""
    E, H, I = desc.E, desc.H, desc.I
    dev = params["W13"].device
    bf = torch.bfloat16
    out = {"W13T": torch.empty(E, H, 2 * I, dtype=bf, device=dev),
           "W2T": torch.empty(E, I, H, dtype=bf, device=dev)}
    if forward and desc.base_format == MOE_BASE_MXFP4:
        s13, s2 = mx_packed_shapes(desc)
        out["W13P"] = torch.empty(s13, dtype=torch.uint8, device=dev)
        out["W2P"] = torch.empty(s2, dtype=torch.uint8, device=dev)
    elif forward:
        out["W13P"] = torch.empty(E, 2 * I, H, dtype=bf, device=dev)
        out["W2P"] = torch.empty(E, H, I, dtype=bf, device=dev)
    moe_lora_transform_base(desc, params, out["W13T"], out["W2T"], out.get("W13P"), out.get("W2P"), stream)
    return out


def moe_lora_forward(desc: MoeLoraDesc, pool: Dict[str, torch.Tensor], x: torch.Tensor,
                     topk_w: torch.Tensor, params: Dict[str, torch.Tensor], out: torch.Tensor,
                     saved: torch.Tensor, scratch: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    T, H, k = desc.T, desc.H, desc.topk
    bm = moe_lora_block_m(desc)
    ps = _pool_struct(pool, bm)
    pp = _params_struct(params, desc)
    st = library().moe_lora_forward(
        ctypes.byref(desc), ctypes.byref(ps), _ptr(x, torch.bfloat16, (T, H), "x"),
        _ptr(topk_w, torch.float32, (T, k), "topk_w"), ctypes.byref(pp),
        _ptr(out, torch.bfloat16, (T, H), "out"), _ptr(saved, torch.uint8, None, "saved"),
        saved.numel(), _ptr(scratch, torch.uint8, None, "scratch"),
        0 if scratch is None else scratch.numel(), _stream(stream))
    _check(st, "moe_lora_forward")


def moe_lora_forward_noalloc(desc: MoeLoraDesc, pool: Dict[str, torch.Tensor], x: torch.Tensor,
                             topk_w: torch.Tensor, params: Dict[str, torch.Tensor], out: torch.Tensor,
                             saved: torch.Tensor, stream=None) -> None:
    """moe_lora_forward with the library's own static scratch (no scratch
    argument; the library allocates nothing).  Raises MoeLoraError
    (MOE_ERR_WORKSPACE) when the layer needs more than the static array."""
    T, H, k = desc.T, desc.H, desc.topk
    bm = moe_lora_block_m(desc)
    ps = _pool_struct(pool, bm)
    pp = _params_struct(params, desc)
    st = library().moe_lora_forward_noalloc(
        ctypes.byref(desc), ctypes.byref(ps), _ptr(x, torch.bfloat16, (T, H), "x"),
        _ptr(topk_w, torch.float32, (T, k), "topk_w"), ctypes.byref(pp),
        _ptr(out, torch.bfloat16, (T, H), "out"), _ptr(saved, torch.uint8, None, "saved"),
        saved.numel(), _stream(stream))
    _check(st, "moe_lora_forward_noalloc")


def moe_lora_backward(desc: MoeLoraDesc, pool: Dict[str, torch.Tensor], grad_out: torch.Tensor,
                      topk_w: torch.Tensor, params: Dict[str, torch.Tensor], saved: torch.Tensor,
                      grad_x: torch.Tensor, grad_topk_w: torch.Tensor,
                      grads: Dict[str, torch.Tensor], scratch: torch.Tensor, stream=None) -> None:
    T, H, I, E, k, r = desc.T, desc.H, desc.I, desc.E, desc.topk, desc.rank
    bm = moe_lora_block_m(desc)
    ps = _pool_struct(pool, bm)
    pp = _params_struct(params, desc)
    bf = torch.bfloat16
    gshape = {"dA1": (r, H), "dA3": (r, H), "dB1": (E, I, r), "dB3": (E, I, r),
              "dA2": (E, r, I), "dB2": (H, r), "dW13": (E, 2 * I, H), "dW2": (E, H, I)}
    gp = {n: _ptr(grads.get(n), bf, s, n) for n, s in gshape.items()}
    gs = MoeLoraGrads(gp["dA1"], gp["dA3"], gp["dB1"], gp["dB3"], gp["dA2"], gp["dB2"],
                      gp["dW13"], gp["dW2"])
    st = library().moe_lora_backward(
        ctypes.byref(desc), ctypes.byref(ps), _ptr(grad_out, bf, (T, H), "grad_out"),
        _ptr(topk_w, torch.float32, (T, k), "topk_w"), ctypes.byref(pp),
        _ptr(saved, torch.uint8, None, "saved"), saved.numel(),
        _ptr(grad_x, bf, (T, H), "grad_x"), _ptr(grad_topk_w, torch.float32, (T, k), "grad_topk_w"),
        ctypes.byref(gs), _ptr(scratch, torch.uint8, None, "scratch"), scratch.numel(),
        _stream(stream))
    _check(st, "moe_lora_backward")


def moe_lora_forward_multi(desc: MoeLoraDesc, roots: Sequence[int], pool: Dict[str, torch.Tensor],
                           x: torch.Tensor, topk_w: torch.Tensor, params: Dict[str, torch.Tensor],
                           out: torch.Tensor, saved: torch.Tensor, scratch: torch.Tensor, stream=None) -> None:
    """moe_lora_forward over the roots (adapter a: tokens roots[a] .. roots[a+1]-1), factors stacked."""
    T, H, k = desc.T, desc.H, desc.topk
    ps = _pool_struct(pool, moe_lora_block_m(desc))
    pp = _params_struct(params, desc, len(roots) - 1)
    st = library().moe_lora_forward_multi(
        ctypes.byref(desc), ctypes.byref(_adapters(roots)), ctypes.byref(ps), _ptr(x, torch.bfloat16, (T, H), "x"),
        _ptr(topk_w, torch.float32, (T, k), "topk_w"), ctypes.byref(pp),
        _ptr(out, torch.bfloat16, (T, H), "out"), _ptr(saved, torch.uint8, None, "saved"), saved.numel(),
        _ptr(scratch, torch.uint8, None, "scratch"), scratch.numel(), _stream(stream))
    _check(st, "moe_lora_forward_multi")


def moe_lora_backward_multi(desc: MoeLoraDesc, roots: Sequence[int], pool: Dict[str, torch.Tensor],
                            grad_out: torch.Tensor, topk_w: torch.Tensor, params: Dict[str, torch.Tensor],
                            saved: torch.Tensor, grad_x: torch.Tensor, grad_topk_w: torch.Tensor,
                            grads: Dict[str, torch.Tensor], scratch: torch.Tensor, stream=None) -> None:
    """moe_lora_backward over the roots; the six factor gradients stacked per adapter."""
    T, H, k = desc.T, desc.H, desc.topk
    na = len(roots) - 1
    ps = _pool_struct(pool, moe_lora_block_m(desc))
    pp = _params_struct(params, desc, na)
    bf = torch.bfloat16
    gp = {n: _ptr(grads.get("d" + n), bf, s, "d" + n) for n, s in _factor_shapes(desc, na).items()}
    gs = MoeLoraGrads(gp["A1"], gp["A3"], gp["B1"], gp["B3"], gp["A2"], gp["B2"], None, None)
    st = library().moe_lora_backward_multi(
        ctypes.byref(desc), ctypes.byref(_adapters(roots)), ctypes.byref(ps),
        _ptr(grad_out, bf, (T, H), "grad_out"), _ptr(topk_w, torch.float32, (T, k), "topk_w"), ctypes.byref(pp),
        _ptr(saved, torch.uint8, None, "saved"), saved.numel(), _ptr(grad_x, bf, (T, H), "grad_x"),
        _ptr(grad_topk_w, torch.float32, (T, k), "grad_topk_w"), ctypes.byref(gs),
        _ptr(scratch, torch.uint8, None, "scratch"), scratch.numel(), _stream(stream))
    _check(st, "moe_lora_backward_multi")


def _sync(stream, dev: Optional[int] = None) -> None:
    if hasattr(stream, "synchronize"):
        stream.synchronize()
    else:
        torch.cuda.synchronize(dev)


def moe_lora_split_e2m3x2(src: torch.Tensor, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Two-term E2M3 split of bf16 rows src [rows, K] (see include/moelora.h):
    returns (codes uint8 [rows, 2K], scale words int32 [K/64, rows], stage-major)."""
    if src.dim() != 2:
        raise ValueError("src must be [rows, K]")
    rows, K = src.shape
    codes = torch.empty(rows, 2 * K, dtype=torch.uint8, device=src.device)
    scales = torch.empty(K // 64, rows, dtype=torch.int32, device=src.device)
    st = library().moe_lora_split_e2m3x2(_ptr(src, torch.bfloat16, None, "src"), rows, K,
                                         _ptr(codes, torch.uint8, None, "codes"),
                                         _ptr(scales, torch.int32, None, "scale_words"), _stream(stream))
    _check(st, "moe_lora_split_e2m3x2")
    return codes, scales


# the current stream's handle by device index (a Stream object costs 2 us to make)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


def _on(dev: int, t: Optional[torch.Tensor], dtype, shape, name: str) -> Optional[int]:
    """_ptr for a call that runs on device dev: t is there too."""
    if t is None:
        return None
    if t.get_device() == dev and t.is_contiguous() and t.dtype is dtype and (shape is None or t.shape == shape):
        return t.data_ptr()
    p = _ptr(t, dtype, shape, name)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call on cuda:{dev}: one call runs on one device")
    return p


def _device_of(t: torch.Tensor, name: str) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a device tensor")
    return dev


def _launch(what: str, fn, dev: int, stream, *args) -> None:
    """fn(*args, stream) on device dev (made the current one for the call if it
    is not); stream None: that device's current one."""
    if dev < 0:
        raise ValueError(f"{what}: tensors must be device tensors")
    handle = _raw_stream(dev) if stream is None else _stream(stream)
    if torch.cuda.current_device() == dev:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != MOE_OK:
        raise MoeLoraError(st, what)


def _made(stream, make, *shape, **kw) -> torch.Tensor:
    """An output allocated for a call on `stream` (None: the current one): made
    there, so that a fill is ordered before the call and the memory is not
    handed out again too early, and used on the current stream afterwards."""
    if stream is None:
        return make(*shape, **kw)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream, kw["device"])
    with torch.cuda.stream(s):
        t = make(*shape, **kw)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


_FLOAT_TYPES = {torch.float32: MOE_TYPE_F32, torch.bfloat16: MOE_TYPE_BF16}


def _float_type(dtype, name: str) -> int:
    if dtype not in _FLOAT_TYPES:
        raise ValueError(f"{name} must be float32 or bfloat16, got {dtype}")
    return _FLOAT_TYPES[dtype]


# --------------------------------------------------------------------------
# router
# --------------------------------------------------------------------------
def make_router_desc(T: int, E: int, topk: int, dtype=torch.float32, renorm: bool = True) -> MoeRouterDesc:
    return MoeRouterDesc(T, E, topk, _float_type(dtype, "logits"), int(renorm))


def moe_router_workspace_size(desc: MoeRouterDesc, roots: Optional[Sequence[int]] = None) -> int:
    v = ctypes.c_size_t()
    ad = _adapters(roots)
    _check(library().moe_router_workspace_size(ctypes.byref(desc), None if ad is None else ctypes.byref(ad),
                                               ctypes.byref(v)), "moe_router_workspace_size")
    return v.value


class MoeRouter:
    """Top-k routing of one shape: T tokens' logits [T, E] to expert ids and
    weights, expert loads and the balance loss, and the gradient to the
    logits.  Keeps the output buffers and the workspace; every call
    overwrites them, so calls that run at the same time (on two streams, in
    two captured graphs) need a router each.

    roots: several adapters in one pass, as in MoeLoraLayer; loads and loss
    are per root.  renorm: a token's weights divided by their sum.  checked:
    read the count of dropped tokens after the forward (a device-to-host
    sync) and raise if a valid token had a NaN or +inf logit."""

    def __init__(self, T: int, E: int, topk: int, dtype=torch.float32, renorm: bool = True,
                 roots: Optional[Sequence[int]] = None, device="cuda", checked: bool = False):
        self.desc = make_router_desc(T, E, topk, dtype, renorm)
        self.dtype = dtype
        self.checked = checked
        self.roots = None if roots is None else [int(v) for v in roots]
        na = 1 if roots is None else len(roots) - 1
        nbytes = moe_router_workspace_size(self.desc, self.roots)
        self._ad = _adapters(self.roots)
        self._adp = None if self._ad is None else ctypes.byref(self._ad)
        i32, f32 = torch.int32, torch.float32
        self.topk_idx = torch.empty(T, topk, dtype=i32, device=device)
        self.topk_w = torch.empty(T, topk, dtype=f32, device=device)
        self.counts = torch.empty(na, E, dtype=i32, device=device)
        self.active = torch.empty(na, dtype=i32, device=device)
        self.loss = torch.empty(na, dtype=f32, device=device)
        self.device_error = torch.empty(1, dtype=i32, device=device)
        self.grad_logits = torch.empty(T, E, dtype=dtype, device=device)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self._dp = ctypes.byref(self.desc)
        self._dev = self.topk_idx.get_device()
        self._lshape, self._kshape, self._tshape, self._cshape, self._rshape = (T, E), (T, topk), (T,), (na, E), (na,)
        # aliases: the addresses that forward writes stay this router's, whatever the attributes are given
        self._held = [t.detach() for t in (self.topk_idx, self.topk_w, self.counts, self.active, self.loss,
                                           self.device_error, self.workspace)]
        self._results, self._grad = tuple(self._held[:5]), self.grad_logits
        self._outs = tuple(t.data_ptr() for t in self._held) + (nbytes,)

    def forward(self, logits: torch.Tensor, valid: Optional[torch.Tensor] = None, stream=None):
        """logits [T, E]; valid [T] uint8 (0: a padding token) or None.
        Returns (topk_idx, topk_w, counts, active, loss)."""
        dev = self._dev
        _launch("moe_router_forward", library().moe_router_forward, dev, stream, self._dp, self._adp,
                _on(dev, logits, self.dtype, self._lshape, "logits"),
                _on(dev, valid, torch.uint8, self._tshape, "valid"), *self._outs)
        if self.checked:
            bad = self.dropped_tokens(stream)
            if bad:
                raise FloatingPointError(f"moe_router_forward: {bad} valid token(s) with a NaN or +inf logit were dropped")
        return self._results

    def dropped_tokens(self, stream=None) -> int:
        """Valid tokens the last forward dropped for a NaN or +inf logit (syncs)."""
        _sync(stream, self._dev)
        return int(self._held[5].item())

    def backward(self, logits: torch.Tensor, topk_idx: torch.Tensor, counts: torch.Tensor, active: torch.Tensor,
                 grad_topk_w: Optional[torch.Tensor] = None, grad_loss: Optional[torch.Tensor] = None,
                 valid: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The gradient to the logits, [T, E] of their type, from the
        forward's topk_idx, counts and active (the router's own buffers after
        forward, or copies) and the gradients of topk_w [T, k] and of the
        loss [roots] (None: zero).  It is written to self.grad_logits, which
        may be given another tensor of that shape and type, logits itself too."""
        f32, i32, dev = torch.float32, torch.int32, self._dev
        if self.grad_logits is not self._grad:  # another buffer, the logits' own, say
            _on(dev, self.grad_logits, self.dtype, self._lshape, "grad_logits")
            self._grad = self.grad_logits
        _launch("moe_router_backward", library().moe_router_backward, dev, stream, self._dp, self._adp,
                _on(dev, logits, self.dtype, self._lshape, "logits"), _on(dev, valid, torch.uint8, self._tshape, "valid"),
                _on(dev, topk_idx, i32, self._kshape, "topk_idx"), _on(dev, counts, i32, self._cshape, "counts"),
                _on(dev, active, i32, self._rshape, "active"), _on(dev, grad_topk_w, f32, self._kshape, "grad_topk_w"),
                _on(dev, grad_loss, f32, self._rshape, "grad_loss"), self._grad.data_ptr())
        return self._grad


# --------------------------------------------------------------------------
# optimiser
# --------------------------------------------------------------------------
class MoeAdamW:
    """AdamW over a list of tensors (the factors of one or more layers) in one
    call per step.  params: bf16 or fp32, all of one type, updated in place;
    grads: bf16 or fp32 buffers of the same sizes that are read at each step
    (MoeLoraLayer.grads, say; all these tensors stay where they are: the
    optimiser keeps their memory, and goes on with it if a tensor is given
    other memory, by `p.data = ...`, say); masters: fp32 copies of bf16 params that are
    updated instead, the params getting their rounding.  state_bits 32 or 8
    (see include/moelora.h); states: {"m": [...], "v": [...], "m_scale":
    [...], "v_scale": [...]} to go on from, else zeros."""

    def __init__(self, params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                 masters: Optional[Sequence[torch.Tensor]] = None, state_bits: int = 32, lr: float = 1e-3,
                 betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.0,
                 states: Optional[Dict[str, Sequence[torch.Tensor]]] = None):
        if not params or len(grads) != len(params) or (masters is not None and len(masters) != len(params)):
            raise ValueError("params, grads and masters are lists of one length, not empty")
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        self.params, self.grads = list(params), list(grads)
        self.masters = None if masters is None else list(masters)
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits = state_bits
        self.steps = 0  # steps taken
        self._dev = _device_of(params[0], "params")
        self._same = None  # what the descriptor holds of betas, eps and weight_decay
        eight = state_bits == 8
        kinds = {"m": torch.float8_e4m3fn, "v": torch.float8_e5m2} if eight else dict.fromkeys("mv", torch.float32)
        runs = [-(-p.numel() // 128) for p in self.params]
        if states is None:
            states = {n: [torch.zeros(p.shape, dtype=torch.uint8 if eight else t, device=p.device).view(t)
                          for p in self.params] for n, t in kinds.items()}
            if eight:
                states.update({n: [torch.zeros(r, device=p.device) for p, r in zip(self.params, runs)]
                               for n in ("m_scale", "v_scale")})
        names = ("m", "v", "m_scale", "v_scale") if eight else ("m", "v")
        if set(states) != set(names) or any(len(states[n]) != len(params) for n in names):
            raise ValueError(f"states must hold {names}, one tensor each per param")
        self.states = {n: list(states[n]) for n in names}
        self._desc = MoeAdamwDesc(_float_type(params[0].dtype, "params"), _float_type(grads[0].dtype, "grads"), state_bits)
        self._dp = ctypes.byref(self._desc)
        self._table = (MoeAdamwTensor * len(params))()
        ptype, gtype, f32 = params[0].dtype, grads[0].dtype, torch.float32
        if masters is not None and ptype != torch.bfloat16:
            raise ValueError("masters stand beside bf16 params")
        for i, p in enumerate(self.params):
            n = p.numel()
            every = [self.grads[i], *([] if masters is None else [masters[i]]), *(self.states[k][i] for k in names)]
            if any(t.device != params[0].device for t in (p, *every)):
                raise ValueError("one optimiser's tensors are on one device")
            for t, k in [(self.grads[i], "grads")] + ([] if masters is None else [(masters[i], "masters")]) + [
                    (self.states[k][i], k) for k in ("m", "v")]:
                if t.numel() != n:
                    raise ValueError(f"{k}[{i}] has {t.numel()} elements, params[{i}] {n}")
            sc = [_ptr(self.states[k][i], f32, (runs[i],), k) for k in ("m_scale", "v_scale")] if eight else [None, None]
            self._table[i] = MoeAdamwTensor(
                _ptr(p, ptype, None, "params"), None if masters is None else _ptr(masters[i], f32, None, "masters"),
                _ptr(self.grads[i], gtype, None, "grads"), _ptr(self.states["m"][i], kinds["m"], None, "m"),
                _ptr(self.states["v"][i], kinds["v"], None, "v"), *sc, n)
        # the memory outlives a replacement of a tensor's own
        self._held = [t.untyped_storage() for ts in (self.params, self.grads, self.masters or [], *self.states.values()) for t in ts]
        # memory that a step writes belongs to one tensor alone
        spans = [(t.data_ptr(), t.numel() * t.element_size(), k) for k, ts in
                 (("params", self.params), ("grads", self.grads), ("masters", self.masters or []), *self.states.items())
                 for t in ts if t.numel()]
        end, end_written = 0, 0
        for at, size, k in sorted(spans):
            if at < (end_written if k == "grads" else end):
                raise ValueError(f"{k} overlap another tensor of the optimiser")
            end, end_written = max(end, at + size), end_written if k == "grads" else max(end_written, at + size)

    def step(self, lr: Optional[float] = None, step: Optional[int] = None, grad_scale: float = 1.0,
             seed: Optional[int] = None, control: Optional[torch.Tensor] = None, stream=None) -> None:
        """One step.  lr: this step's rate (default: the optimiser's); step:
        its number (default: one more than the last); grad_scale multiplies
        the gradients (a clip coefficient, an accumulation's share); seed of
        the 8-bit states' rounding (default: the step's number).  control:
        those values in device memory (adamw_control), for a captured step."""
        number = self.steps + 1 if step is None else int(step)
        d = self._desc
        same = (*self.betas, self.eps, self.weight_decay)
        if same != self._same:  # fields that seldom change (setting one costs 60 ns)
            d.beta1, d.beta2, d.eps, d.weight_decay = self._same = same
        d.lr = self.lr if lr is None else lr
        d.grad_scale = grad_scale
        d.step = number
        if self.state_bits == 8:
            d.seed = (number if seed is None else seed) & 0xFFFFFFFF
        d.control = _on(self._dev, control, torch.int32, (5,), "control")
        _launch("moe_adamw_step", library().moe_adamw_step, self._dev, stream, self._dp, self._table, len(self._table))
        self.steps = number  # only a step that was taken

    def write_control(self, control: torch.Tensor, lr: float, step: int, grad_scale: float = 1.0,
                      seed: Optional[int] = None) -> None:
        """Fill a control buffer (int32 [5] on the device) with one step's
        values: before each replay of a graph that captured a step with it."""
        _on(self._dev, control, torch.int32, (5,), "control")
        if step < 1:
            raise ValueError("write_control: step >= 1")
        f = torch.tensor([lr, 1.0 - self.betas[0] ** step, 1.0 - self.betas[1] ** step, grad_scale],
                         dtype=torch.float64).to(torch.float32)
        if not (lr >= 0 and bool(torch.isfinite(f).all())):
            raise ValueError("write_control: lr >= 0 and grad_scale, finite in fp32")
        f = f.view(torch.int32)
        s = (step if seed is None else seed) & 0xFFFFFFFF
        control.copy_(torch.cat([f, torch.tensor([s - (1 << 32) if s >> 31 else s], dtype=torch.int32)]))


# --------------------------------------------------------------------------
# 8-bit expert products
# --------------------------------------------------------------------------
_ACTS = {None: MOE_FP8_PLAIN, "swiglu": MOE_ACT_SWIGLU, "geglu": MOE_ACT_GEGLU}
_E4M3 = torch.float8_e4m3fn


def fp8_quantize_rows(src: torch.Tensor, act: Optional[str] = None, codes: Optional[torch.Tensor] = None,
                      scales: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """src bf16 [rows, K] (act None) or [rows, 2K] = gate | up (act "swiglu",
    "geglu") to e4m3 codes [rows, K] and fp32 scales [rows, K/128]."""
    if src.dim() != 2 or act not in _ACTS or (act is not None and src.shape[1] % 2):
        raise ValueError("src must be [rows, K], or [rows, 2K] with act 'swiglu' or 'geglu'")
    rows, K = src.shape
    if act is not None:
        K //= 2
    dev = _device_of(src, "src")
    if codes is None:
        codes = _made(stream, torch.empty, rows, K, dtype=_E4M3, device=src.device)
        to = codes.data_ptr()
    else:
        to = _on(dev, codes, _E4M3, (rows, K), "codes")
    if scales is None:
        scales = _made(stream, torch.empty, rows, K // 128, dtype=torch.float32, device=src.device)
        sto = scales.data_ptr()
    else:
        sto = _on(dev, scales, torch.float32, (rows, K // 128), "scales")
    _launch("moe_fp8_quantize_rows", library().moe_fp8_quantize_rows, dev, stream,
            _on(dev, src, torch.bfloat16, None, "src"), rows, K, _ACTS[act], to, sto)
    return codes, scales


def fp8_quantize_weight(W: torch.Tensor, transposed: bool = False, stream=None) -> Tuple[torch.Tensor, ...]:
    """W bf16 [E, N, K] to (codes [E, N, K], scales [E, N/128, K/128]) by
    128 x 128 blocks; with transposed also the same codes as (codes_t
    [E, K, N], scales_t [E, K/128, N/128]), the data gradient's operand."""
    if W.dim() != 3:
        raise ValueError("W must be [E, N, K]")
    E, N, K = W.shape
    dev = _device_of(W, "W")

    def pair(n, k):
        return [_made(stream, torch.empty, E, n, k, dtype=_E4M3, device=W.device),
                _made(stream, torch.empty, E, n // 128, k // 128, dtype=torch.float32, device=W.device)]
    out = pair(N, K) + (pair(K, N) if transposed else [])
    _launch("moe_fp8_quantize_weight", library().moe_fp8_quantize_weight, dev, stream,
            _on(dev, W, torch.bfloat16, None, "W"), E, N, K, *[t.data_ptr() for t in out], *([] if transposed else [None, None]))
    return tuple(out)


def fp8_product(pool: Dict[str, torch.Tensor], a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor,
                w_scales: torch.Tensor, topk: int = 0, out: Optional[torch.Tensor] = None, block_m: int = 16,
                stream=None) -> torch.Tensor:
    """Every pool row times its expert's weight: out bf16 [capacity, N].
    pool as in MoeLoraLayer.pool; a e4m3 [rows, K] with a_scales [rows,
    K/128]: the tokens (topk > 0: pool row r reads token row_to_route[r] /
    topk), or the pool rows themselves (topk = 0); w e4m3 [E, N, K] with
    w_scales [E, N/128, K/128].  Rows of no route are left as they are (an
    `out` made here holds zeros there).  block_m: the pool's (the library's
    own choice is 16)."""
    if a.dim() != 2 or w.dim() != 3:
        raise ValueError("a must be [rows, K] and w [E, N, K]")
    rows, K = a.shape
    E, N = w.shape[:2]
    cap = pool["row_to_route"].numel()
    dev = _device_of(a, "a")
    if out is None:
        out = _made(stream, torch.zeros, cap, N, dtype=torch.bfloat16, device=a.device)
    i32, f32 = torch.int32, torch.float32
    ps = MoePool(_on(dev, pool["counts"], i32, (E,), "counts"), _on(dev, pool["offsets"], i32, (E + 1,), "offsets"), None,
                 _on(dev, pool["row_to_route"], i32, None, "row_to_route"), cap, block_m)
    d = MoeFp8Desc(E, N, K, topk, rows)
    _launch("moe_fp8_product", library().moe_fp8_product, dev, stream, ctypes.byref(d), ctypes.byref(ps),
            _on(dev, a, _E4M3, None, "a"), _on(dev, a_scales, f32, (rows, K // 128), "a_scales"),
            _on(dev, w, _E4M3, (E, N, K), "w"), _on(dev, w_scales, f32, (E, N // 128, K // 128), "w_scales"),
            _on(dev, out, torch.bfloat16, (cap, N), "out"))
    return out


def moe_lora_trace_enable(on: bool) -> None:
    library().moe_lora_trace_enable(1 if on else 0)


def moe_lora_trace_reset() -> None:
    library().moe_lora_trace_reset()


def moe_lora_trace_collect() -> Dict[str, Tuple[int, float]]:
    """Wait for recorded events; return {kernel: (launches, total_ms)}."""
    lib = library()
    _check(lib.moe_lora_trace_collect(), "moe_lora_trace_collect")
    out = {}
    for i in range(lib.moe_lora_trace_count()):
        name, n, ms = ctypes.c_char_p(), ctypes.c_int64(), ctypes.c_double()
        _check(lib.moe_lora_trace_entry(i, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms)),
               "moe_lora_trace_entry")
        out[name.value.decode()] = (n.value, ms.value)
    return out


class MoeLoraLayer:
    """Device buffers for one layer shape (pool arrays, workspaces, outputs)
    and the three calls in order.  Convenience for tests and the benchmark."""

    def __init__(self, desc: MoeLoraDesc, device="cuda", base_grads: bool = False,
                 checked: bool = False, roots: Optional[Sequence[int]] = None):
        """base_grads: also compute the frozen-weight gradients dW13, dW2.
        checked: after build_pool read the device error count and after the
        forward the saved status word (each a device-to-host sync), and raise
        if either reports a problem (route ids outside [-1, E), or a gate/up
        pre-activation beyond the fp16 range the backward needs).
        roots: several adapters in one pass (the *_multi calls): adapter a
        serves tokens roots[a] .. roots[a+1]-1; factors and their gradients
        are stacked over the adapters."""
        self.desc = desc
        self.device = device
        self.checked = checked
        self.roots = None if roots is None else [int(v) for v in roots]
        na = None if roots is None else len(roots) - 1
        self.block_m = moe_lora_block_m(desc)
        if roots is None:
            self.capacity = moe_lora_pool_capacity(desc)
            self.saved_bytes, self.scratch_bytes = moe_lora_workspace_size(desc)
        else:
            self.capacity = moe_lora_multi_pool_capacity(desc, self.roots)
            self.saved_bytes, self.scratch_bytes = moe_lora_multi_workspace_size(desc, self.roots)
        T, H, I, E, k, r = desc.T, desc.H, desc.I, desc.E, desc.topk, desc.rank
        G = E * (1 if na is None else na)
        i32 = torch.int32
        self.pool = {
            "counts": torch.empty(G, dtype=i32, device=device),
            "offsets": torch.empty(G + 1, dtype=i32, device=device),
            "route_to_row": torch.empty(T * k, dtype=i32, device=device),
            "row_to_route": torch.empty(self.capacity, dtype=i32, device=device),
        }
        self.device_error = torch.empty(1, dtype=i32, device=device)
        self.saved = torch.empty(self.saved_bytes, dtype=torch.uint8, device=device)
        self.scratch = torch.empty(self.scratch_bytes, dtype=torch.uint8, device=device)
        bf = torch.bfloat16
        self.out = torch.empty(T, H, dtype=bf, device=device)
        self.grad_x = torch.empty(T, H, dtype=bf, device=device)
        self.grad_topk_w = torch.empty(T, k, dtype=torch.float32, device=device)
        self.grads = {"d" + n: torch.empty(sh, dtype=bf, device=device)
                      for n, sh in _factor_shapes(desc, na).items()}
        if base_grads:
            self.grads["dW13"] = torch.empty(E, 2 * I, H, dtype=bf, device=device)
            self.grads["dW2"] = torch.empty(E, H, I, dtype=bf, device=device)

    def build_pool(self, topk_idx: torch.Tensor, stream=None) -> None:
        if self.roots is None:
            build_pool(self.desc, topk_idx, self.pool["counts"], self.pool["offsets"],
                       self.pool["route_to_row"], self.pool["row_to_route"], self.device_error, stream)
        else:
            build_pool_multi(self.desc, self.roots, topk_idx, self.pool["counts"], self.pool["offsets"],
                             self.pool["route_to_row"], self.pool["row_to_route"], self.device_error, stream)
        if self.checked:
            bad = self.invalid_routes(stream)
            if bad:
                raise ValueError(f"build_pool: {bad} route id(s) outside [-1, {self.desc.E}) were dropped")

    def invalid_routes(self, stream=None) -> int:
        """Route ids outside [-1, E) dropped by the last build_pool (syncs)."""
        _sync(stream)
        return int(self.device_error.item())

    def saved_status(self, stream=None) -> int:
        """The saved workspace's status word after the last forward (syncs):
        0, or MOE_SAVED_* bits."""
        _sync(stream)
        off = MOE_SAVED_STATUS_OFFSET
        return int(self.saved[off:off + 4].view(torch.int32).item())

    def forward(self, x, topk_w, params, stream=None) -> torch.Tensor:
        if self.roots is None:
            moe_lora_forward(self.desc, self.pool, x, topk_w, params, self.out, self.saved, self.scratch, stream)
        else:
            moe_lora_forward_multi(self.desc, self.roots, self.pool, x, topk_w, params, self.out, self.saved,
                                   self.scratch, stream)
        if self.checked and self.saved_status(stream) & MOE_SAVED_FP16_RANGE:
            raise FloatingPointError("moe_lora_forward: a gate/up pre-activation is beyond the fp16 range "
                                     "(|g| or |v| >= 65520) without a clamp; the backward would not be finite")
        return self.out

    def backward(self, grad_out, topk_w, params, stream=None):
        if self.roots is None:
            moe_lora_backward(self.desc, self.pool, grad_out, topk_w, params, self.saved,
                              self.grad_x, self.grad_topk_w, self.grads, self.scratch, stream)
        else:
            moe_lora_backward_multi(self.desc, self.roots, self.pool, grad_out, topk_w, params, self.saved,
                                    self.grad_x, self.grad_topk_w, self.grads, self.scratch, stream)
        return self.grad_x, self.grad_topk_w, self.grads

    def step(self, topk_idx, x, topk_w, params, grad_out, stream=None):
        """One pass of the whole path: pool, forward, backward."""
        self.build_pool(topk_idx, stream)
        self.forward(x, topk_w, params, stream)
        return self.backward(grad_out, topk_w, params, stream)
