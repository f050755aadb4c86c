"""Python binding of libedge_moe.so (the shared-matrix sparse-MoE expert layer).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  Functions carry the C names and take torch tensors that live on the
GPU (PyTorch provides device memory and streams here, nothing else); the
library is required - calls raise if it is not built.

    import shared_matrix_expert_amd as em
    ws = torch.empty(em.edge_moe_workspace_bytes(dims), dtype=torch.uint8, device="cuda")
    em.edge_moe_route(dims, x, w_router, bias, idx, w, None, ws)
    em.edge_moe_forward(dims, x, idx, w, weights, y, ws)
"""
from __future__ import annotations

import contextlib
import ctypes
import operator
import os
import struct
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libedge_moe.so")

EDGE_MOE_OK = 0
EDGE_MOE_EINVAL = -1
EDGE_MOE_EUNSUPPORTED = -2
EDGE_MOE_EWORKSPACE = -3
EDGE_MOE_EHIP = -4

EXPORTED = ("edge_moe_workspace_bytes", "edge_moe_route", "edge_moe_forward",
            "edge_moe_forward_traced", "edge_moe_residual", "edge_moe_status_string",
            "edge_moe_abi_version", "edge_moe_copy", "edge_moe_tile_shared",
            "edge_moe_prof_enable", "edge_moe_prof_read", "edge_moe_prof_reset",
            "edge_moe_forward_noalloc", "edge_moe_forward_persistent", "edge_moe_mfma_peak",
            "edge_moe_workspace_bytes_mx", "edge_moe_forward_mx", "edge_moe_prefetch_ws_bytes",
            "edge_moe_prefetch", "edge_moe_cache_create", "edge_moe_cache_destroy", "edge_moe_cache_map",
            "edge_moe_cache_prefetch", "edge_moe_cache_totals", "edge_moe_cache_slot_of",
            "edge_moe_mx_quantize", "edge_moe_mx_dequantize", "edge_moe_mx_product_ws_bytes", "edge_moe_mx_product",
            "edge_moe_mx_product_coded",
            "edge_moe_balance_ws_bytes", "edge_moe_balance", "edge_moe_route_backward_ws_bytes",
            "edge_moe_route_backward", "edge_moe_norm", "edge_moe_norm_backward_ws_bytes", "edge_moe_norm_backward",
            "edge_moe_dense_product_ws_bytes", "edge_moe_dense_product", "edge_moe_dense_product_backward_ws_bytes",
            "edge_moe_dense_product_backward", "edge_moe_packed_product_ws_bytes", "edge_moe_packed_product")

# element formats and dense types of the MX matrix operators
MX_FP4, MX_FP8 = 0, 1
_BF16, _FLOAT = 0, 1


class _cuda:                   # torch's current device, and a device's stream handle (filled by load())
    getDevice = getRawStream = None


_dtypes: dict = {}             # torch's types by name, and those of dense matrices (filled by load())
_dense_types: dict = {}
_half_types: set = set()


class CDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "d", "h", "n_experts", "experts_per_group", "top_k",
                 "delta_rank", "lora_rank", "quant_group")]


_WEIGHT_FIELDS = ("s_up_q", "s_up_scale", "s_dn_q", "s_dn_scale", "a_up_q", "a_up_scale",
                  "b_up_q", "b_up_scale", "a_dn_q", "a_dn_scale", "b_dn_q", "b_dn_scale",
                  "lora_up_u", "lora_up_v", "lora_dn_u", "lora_dn_v",
                  "s_up_t", "s_dn_t", "a_up_t", "a_dn_t")
# keys of the weight dicts made by the input generator -> struct fields (the
# last four, the decode-tiled and column-blocked codes, are optional)
_WEIGHT_KEYS = ("s_up", "s_up_scale", "s_dn", "s_dn_scale", "a_up", "a_up_scale",
                "b_up", "b_up_scale", "a_dn", "a_dn_scale", "b_dn", "b_dn_scale",
                "lora_up_u", "lora_up_v", "lora_dn_u", "lora_dn_v",
                "s_up_t", "s_dn_t", "a_up_t", "a_dn_t")
_OPTIONAL_KEYS = ("s_up_t", "s_dn_t", "a_up_t", "a_dn_t")


class CWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _WEIGHT_FIELDS]


# the MX variant: E8M0 scale bytes in place of the fp16 scales, no tiled copies
_WEIGHT_FIELDS_MX = ("s_up_q", "s_up_e", "s_dn_q", "s_dn_e", "a_up_q", "a_up_e",
                     "b_up_q", "b_up_e", "a_dn_q", "a_dn_e", "b_dn_q", "b_dn_e",
                     "lora_up_u", "lora_up_v", "lora_dn_u", "lora_dn_v")


class CWeightsMX(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _WEIGHT_FIELDS_MX]


# per-expert tensors that an expert cache streams (weight-dict keys, struct order)
EXPERT_TENSOR_KEYS = ("a_up", "a_up_scale", "b_up", "b_up_scale", "a_dn", "a_dn_scale",
                      "b_dn", "b_dn_scale", "a_up_t", "a_dn_t")


class CExpertTensors(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("a_up_q", "a_up_scale", "b_up_q", "b_up_scale", "a_dn_q", "a_dn_scale",
                 "b_dn_q", "b_dn_scale", "a_up_t", "a_dn_t")]


class CCacheStats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("hits", "misses", "evictions", "bytes_copied")]


class CTrace(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("expert_offsets", "row_token", "row_slot", "act", "expert_out")]


class CMxDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "R", "M", "N", "K", "x_format")]


class CRouteGrad(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("logits", "topk_idx", "topk_w", "d_topk_w", "d_loss", "counts",
                                                "seq_offsets")]
                + [("n_seq", ctypes.c_int32)]
                + [(n, ctypes.c_void_p) for n in ("x", "w_router", "dlogits", "dx", "dw_router", "dbias")])


def _fields(spec: str) -> list:
    """ctypes fields of a struct: names by kind (i int32, f float, p pointer, s int64 stride)."""
    kinds = {"i": ctypes.c_int32, "f": ctypes.c_float, "p": ctypes.c_void_p, "s": ctypes.c_int64}
    return [(n, kinds[k]) for k, n in (w.split(":") for w in spec.split())]


class CNormArgs(ctypes.Structure):
    _fields_ = _fields("i:T i:d f:eps i:add_type i:gain_type p:x s:x_stride p:add s:add_stride p:gain p:x_out s:x_out_stride "
                       "p:y s:y_stride p:codes p:scales p:rstd")


class CNormGrad(ctypes.Structure):
    _fields_ = _fields("i:T i:d i:gain_type i:grad_type p:x s:x_stride p:gain p:rstd p:dy s:dy_stride p:dres s:dres_stride "
                       "p:dx s:dx_stride p:dgain")


class CDenseDims(ctypes.Structure):
    _fields_ = _fields("i:T i:R i:M i:N i:K")


class CPackedDims(ctypes.Structure):
    _fields_ = _fields("i:T i:R i:M i:N i:K i:quant_group")


class CDenseGrad(ctypes.Structure):
    _fields_ = _fields("p:dy s:dy_stride p:x s:x_stride p:row_src p:offsets p:token_rows i:per_token p:w p:dx s:dx_stride "
                       "i:dx_type i:dw_type p:dw")


class EdgeMoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m shared_matrix_expert_amd.build`")
    # PyTorch-ROCm ships its own HIP runtime; load it first so that the library
    # binds to the same runtime instance as the streams and memory it is given.
    import torch
    # Where this torch has them, the calls that build no device or stream object
    # (0.1 us against 1); host-only calls need neither.
    _cuda.getDevice = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _cuda.getRawStream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)
    _dtypes.update({n: getattr(torch, n) for n in ("uint8", "int32", "float32")})
    _dense_types.update({getattr(torch, n): kind for n, kind in
                         (("bfloat16", _BF16), ("int16", _BF16), ("uint16", _BF16), ("float32", _FLOAT)) if hasattr(torch, n)})
    _half_types.update(getattr(torch, n) for n in ("float16", "int16", "uint16") if hasattr(torch, n))
    lib = ctypes.CDLL(path)
    missing = [n for n in EXPORTED if not hasattr(lib, n)]
    if missing:
        raise RuntimeError(f"{path} was built from other sources, it lacks {', '.join(missing)}: run "
                           "`python -m shared_matrix_expert_amd.build`")
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    lib.edge_moe_workspace_bytes.argtypes = [ctypes.POINTER(CDims)]
    lib.edge_moe_workspace_bytes.restype = sz
    lib.edge_moe_route.argtypes = [ctypes.POINTER(CDims), vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.edge_moe_route.restype = i32
    lib.edge_moe_forward.argtypes = [ctypes.POINTER(CDims), vp, vp, vp, ctypes.POINTER(CWeights),
                                     vp, vp, sz, vp]
    lib.edge_moe_forward.restype = i32
    lib.edge_moe_forward_traced.argtypes = [ctypes.POINTER(CDims), vp, vp, vp,
                                            ctypes.POINTER(CWeights), vp, vp, sz, vp,
                                            ctypes.POINTER(CTrace)]
    lib.edge_moe_forward_traced.restype = i32
    lib.edge_moe_forward_persistent.argtypes = [ctypes.POINTER(CDims), vp, vp, vp, ctypes.POINTER(CWeights),
                                                vp, vp, sz, vp, ctypes.POINTER(CTrace)]
    lib.edge_moe_forward_persistent.restype = i32
    lib.edge_moe_prefetch_ws_bytes.argtypes = []
    lib.edge_moe_prefetch_ws_bytes.restype = sz
    lib.edge_moe_prefetch.argtypes = [ctypes.POINTER(CDims), ctypes.POINTER(CWeights), vp, i32, i32, vp, sz, vp]
    lib.edge_moe_prefetch.restype = i32
    lib.edge_moe_workspace_bytes_mx.argtypes = [ctypes.POINTER(CDims)]
    lib.edge_moe_workspace_bytes_mx.restype = sz
    lib.edge_moe_forward_mx.argtypes = [ctypes.POINTER(CDims), vp, vp, vp, ctypes.POINTER(CWeightsMX),
                                        vp, vp, sz, vp, ctypes.POINTER(CTrace)]
    lib.edge_moe_forward_mx.restype = i32
    lib.edge_moe_mfma_peak.argtypes = [vp, ctypes.c_int32, ctypes.c_int32, vp]
    lib.edge_moe_mfma_peak.restype = i32
    lib.edge_moe_forward_noalloc.argtypes = [ctypes.POINTER(CDims), vp, vp, vp, ctypes.POINTER(CWeights), vp, vp]
    lib.edge_moe_forward_noalloc.restype = i32
    lib.edge_moe_cache_create.argtypes = [ctypes.POINTER(CDims), i32, ctypes.POINTER(CExpertTensors),
                                          ctypes.POINTER(CExpertTensors)]
    lib.edge_moe_cache_create.restype = vp
    lib.edge_moe_cache_destroy.argtypes = [vp]
    lib.edge_moe_cache_destroy.restype = None
    lib.edge_moe_cache_map.argtypes = [vp, i32, vp, vp, vp, ctypes.POINTER(CCacheStats)]
    lib.edge_moe_cache_map.restype = i32
    lib.edge_moe_cache_prefetch.argtypes = [vp, i32, vp, vp, ctypes.POINTER(CCacheStats)]
    lib.edge_moe_cache_prefetch.restype = i32
    lib.edge_moe_cache_totals.argtypes = [vp, ctypes.POINTER(CCacheStats)]
    lib.edge_moe_cache_totals.restype = i32
    lib.edge_moe_cache_slot_of.argtypes = [vp, i32]
    lib.edge_moe_cache_slot_of.restype = i32
    i64 = ctypes.c_int64
    lib.edge_moe_mx_quantize.argtypes = [i32, i32, i32, i32, i32, vp, i64, vp, vp, vp]
    lib.edge_moe_mx_quantize.restype = i32
    lib.edge_moe_mx_dequantize.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, i64, vp]
    lib.edge_moe_mx_dequantize.restype = i32
    lib.edge_moe_mx_product_ws_bytes.argtypes = [ctypes.POINTER(CMxDims)]
    lib.edge_moe_mx_product_ws_bytes.restype = sz
    lib.edge_moe_mx_product.argtypes = [ctypes.POINTER(CMxDims), vp, i64, vp, vp, vp, vp, vp, i64, vp, sz, vp]
    lib.edge_moe_mx_product.restype = i32
    lib.edge_moe_mx_product_coded.argtypes = [ctypes.POINTER(CMxDims), vp, vp, vp, vp, vp, vp, vp, i64, vp]
    lib.edge_moe_mx_product_coded.restype = i32
    lib.edge_moe_balance_ws_bytes.argtypes = [ctypes.POINTER(CDims), i32]
    lib.edge_moe_balance_ws_bytes.restype = sz
    lib.edge_moe_balance.argtypes = [ctypes.POINTER(CDims), vp, vp, vp, i32, vp, vp, vp, vp, sz, vp]
    lib.edge_moe_balance.restype = i32
    lib.edge_moe_route_backward_ws_bytes.argtypes = [ctypes.POINTER(CDims)]
    lib.edge_moe_route_backward_ws_bytes.restype = sz
    lib.edge_moe_route_backward.argtypes = [ctypes.POINTER(CDims), ctypes.POINTER(CRouteGrad), vp, sz, vp]
    lib.edge_moe_route_backward.restype = i32
    lib.edge_moe_norm.argtypes = [ctypes.POINTER(CNormArgs), vp]
    lib.edge_moe_norm.restype = i32
    lib.edge_moe_norm_backward_ws_bytes.argtypes = [i32, i32]
    lib.edge_moe_norm_backward_ws_bytes.restype = sz
    lib.edge_moe_norm_backward.argtypes = [ctypes.POINTER(CNormGrad), vp, sz, vp]
    lib.edge_moe_norm_backward.restype = i32
    lib.edge_moe_dense_product_ws_bytes.argtypes = [ctypes.POINTER(CDenseDims)]
    lib.edge_moe_dense_product_ws_bytes.restype = sz
    lib.edge_moe_dense_product.argtypes = [ctypes.POINTER(CDenseDims), vp, i64, vp, vp, vp, i32, vp, i64, vp, sz, vp]
    lib.edge_moe_dense_product.restype = i32
    lib.edge_moe_dense_product_backward_ws_bytes.argtypes = [ctypes.POINTER(CDenseDims)]
    lib.edge_moe_dense_product_backward_ws_bytes.restype = sz
    lib.edge_moe_dense_product_backward.argtypes = [ctypes.POINTER(CDenseDims), ctypes.POINTER(CDenseGrad), vp, sz, vp]
    lib.edge_moe_dense_product_backward.restype = i32
    lib.edge_moe_packed_product_ws_bytes.argtypes = [ctypes.POINTER(CPackedDims)]
    lib.edge_moe_packed_product_ws_bytes.restype = sz
    lib.edge_moe_packed_product.argtypes = [ctypes.POINTER(CPackedDims), vp, i64, vp, vp, vp, vp, i32, vp, i64, vp, sz, vp]
    lib.edge_moe_packed_product.restype = i32
    lib.edge_moe_residual.argtypes = [ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp]
    lib.edge_moe_residual.restype = i32
    lib.edge_moe_copy.argtypes = [vp, vp, sz, vp]
    lib.edge_moe_copy.restype = i32
    lib.edge_moe_tile_shared.argtypes = [ctypes.POINTER(CDims), ctypes.c_int32, vp, vp, vp]
    lib.edge_moe_tile_shared.restype = i32
    lib.edge_moe_status_string.argtypes = [i32]
    lib.edge_moe_status_string.restype = ctypes.c_char_p
    lib.edge_moe_abi_version.argtypes = []
    lib.edge_moe_abi_version.restype = i32
    lib.edge_moe_prof_enable.argtypes = [i32]
    lib.edge_moe_prof_enable.restype = i32
    lib.edge_moe_prof_read.argtypes = [vp, vp, vp, i32]
    lib.edge_moe_prof_read.restype = i32
    lib.edge_moe_prof_reset.argtypes = []
    lib.edge_moe_prof_reset.restype = None
    _lib = lib
    return lib


_dim_values = operator.attrgetter(*(n for n, _ in CDims._fields_))


def _i32(v: int) -> int:
    """A size as the library's int32: one past it becomes the largest, which no
    limit of the library allows (ctypes would cut the upper bits off)."""
    if -0x80000000 <= v <= 0x7FFFFFFF:
        return int(v)
    return 0x7FFFFFFF if v > 0 else -0x80000000


def _int32s(kind, pack, *values):
    """Struct of int32 sizes; `pack` refuses what does not fit (or is no int)."""
    try:
        return kind.from_buffer_copy(pack(*values))
    except struct.error:
        return kind(*map(_i32, values))


_pack_dims, _pack_mx_dims, _pack_dense_dims = struct.Struct("9i").pack, struct.Struct("6i").pack, struct.Struct("5i").pack


def cdims(dims) -> CDims:
    return _int32s(CDims, _pack_dims, *_dim_values(dims))


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the library must be on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _stream_handle(device: int) -> int:
    import torch
    return torch.cuda.current_stream(device).cuda_stream


def _stream(stream) -> Optional[int]:
    import torch
    if stream is None:
        return _cuda.getRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _made_on(stream):
    """Context in which new tensors belong to the stream that fills them: torch
    hands out memory in the order of the stream it was asked on, so a block of
    the current stream's may still be read or written there when a kernel on
    another stream fills it."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def cweights(weights: dict) -> CWeights:
    return CWeights(*(_ptr(weights.get(k) if k in _OPTIONAL_KEYS else weights[k]) for k in _WEIGHT_KEYS))


def cweights_mx(weights: dict) -> CWeightsMX:
    """Struct of an MX weight dict (keys as the int4 ones: codes under the
    matrix name, E8M0 bytes under "<name>_scale")."""
    return CWeightsMX(*(_ptr(weights[k]) for k in _WEIGHT_KEYS[:16]))


def edge_moe_prefetch_ws_bytes() -> int:
    return int(load().edge_moe_prefetch_ws_bytes())


def edge_moe_prefetch(dims, weights, groups, parts, ws, stream=None) -> None:
    """Read the listed groups' shared matrices (parts: 1 S_up, 2 S_dn, 3 both)
    so that a later layer call finds them in the memory-side cache."""
    n = 0 if groups is None else int(groups.numel())
    st = load().edge_moe_prefetch(ctypes.byref(cdims(dims)), ctypes.byref(cweights(weights)),
                                  _ptr(groups) if n else None, n, int(parts), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_prefetch", st)


def edge_moe_workspace_bytes_mx(dims) -> int:
    return int(load().edge_moe_workspace_bytes_mx(ctypes.byref(cdims(dims))))


def edge_moe_forward_mx(dims, x, topk_idx, topk_w, weights, y, ws, stream=None, trace=None) -> None:
    """The expert layer with MXFP4 shared and delta matrices."""
    tr = None if trace is None else ctypes.byref(CTrace(*(_ptr(trace.get(n)) for n, _ in CTrace._fields_)))
    st = load().edge_moe_forward_mx(ctypes.byref(cdims(dims)), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                                    ctypes.byref(cweights_mx(weights)), _ptr(y), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream), tr)
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_forward_mx", st)


def edge_moe_tile_shared(dims, which, src_q, dst_q, stream=None) -> None:
    """Decode-tiled copy of the codes of s_up (which=0), s_dn (1) or a_up (2),
    or the column-blocked copy of a_dn (3)."""
    st = load().edge_moe_tile_shared(ctypes.byref(cdims(dims)), int(which), _ptr(src_q), _ptr(dst_q),
                                     _stream(stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_tile_shared", st)


def tile_weights(dims, weights: dict, stream=None) -> dict:
    """A copy of the weight dict with the decode-tiled codes added (new device
    tensors of the sizes of s_up / s_dn / a_up / a_dn; a_up only when its rank
    is a multiple of 128, a_dn only when its rank is 128).  The new tensors
    belong to `stream`; what uses them on another one waits for it."""
    import torch
    out = dict(weights)
    for which, key in ((0, "s_up"), (1, "s_dn"), (2, "a_up"), (3, "a_dn")):
        if which == 2 and dims.delta_rank % 128:
            continue
        if which == 3 and dims.delta_rank != 128:
            continue
        with _made_on(stream):
            q = torch.empty_like(weights[key])
        edge_moe_tile_shared(dims, which, weights[key], q, stream)
        out[key + "_t"] = q
    return out


def status_string(status: int) -> str:
    return load().edge_moe_status_string(int(status)).decode()


def edge_moe_copy(dst, src, stream=None) -> None:
    """Plain device copy of src into dst (same byte size), one library kernel."""
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n:
        raise ValueError("edge_moe_copy: dst and src differ in size")
    st = load().edge_moe_copy(_ptr(dst), _ptr(src), n, _stream(stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_copy", st)


def edge_moe_abi_version() -> int:
    return int(load().edge_moe_abi_version())


def edge_moe_workspace_bytes(dims) -> int:
    return int(load().edge_moe_workspace_bytes(ctypes.byref(cdims(dims))))


def edge_moe_route(dims, x, w_router, bias, topk_idx, topk_w, logits_out, ws, stream=None) -> None:
    lib = load()
    st = lib.edge_moe_route(ctypes.byref(cdims(dims)), _ptr(x), _ptr(w_router), _ptr(bias),
                            _ptr(topk_idx), _ptr(topk_w), _ptr(logits_out), _ptr(ws),
                            ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_route", st)


def edge_moe_forward(dims, x, topk_idx, topk_w, weights, y, ws, stream=None, trace=None) -> None:
    lib = load()
    cw = cweights(weights) if isinstance(weights, dict) else weights
    args = (ctypes.byref(cdims(dims)), _ptr(x), _ptr(topk_idx), _ptr(topk_w), ctypes.byref(cw),
            _ptr(y), _ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0,
            _stream(stream))
    if trace is None:
        st = lib.edge_moe_forward(*args)
    else:
        tr = CTrace(*(_ptr(trace.get(n)) for n, _ in CTrace._fields_))
        st = lib.edge_moe_forward_traced(*args, ctypes.byref(tr))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_forward", st)


def edge_moe_forward_persistent(dims, x, topk_idx, topk_w, weights, y, ws, stream=None, trace=None) -> None:
    """The decode / verify layer as one persistent launch (T <= 8, stored copies
    of kinds 0-3 in `weights`); trace as edge_moe_forward's."""
    tr = None if trace is None else CTrace(*(_ptr(trace.get(n)) for n, _ in CTrace._fields_))
    st = load().edge_moe_forward_persistent(ctypes.byref(cdims(dims)), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                                            ctypes.byref(cweights(weights)), _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                                            _stream(stream), None if tr is None else ctypes.byref(tr))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_forward_persistent", st)


def edge_moe_mfma_peak(out, blocks, iters, stream=None) -> None:
    """Matrix-core calibration launch (blocks * 4 * iters * 8 * 16384 flops)."""
    st = load().edge_moe_mfma_peak(_ptr(out), int(blocks), int(iters), _stream(stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_mfma_peak", st)


def edge_moe_forward_noalloc(dims, x, topk_idx, topk_w, weights, y, stream=None) -> None:
    """edge_moe_forward with the library's own per-device scratch as workspace
    (no allocation; calls that overlap on one GPU race)."""
    st = load().edge_moe_forward_noalloc(ctypes.byref(cdims(dims)), _ptr(x), _ptr(topk_idx), _ptr(topk_w),
                                         ctypes.byref(cweights(weights)), _ptr(y), _stream(stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_forward_noalloc", st)


# ---------------------------------------------- MX matrices, router training ----
# The calls below check types, shapes and devices of what they are given (their
# kernels trust the sizes in the arguments), beyond what the library checks.

def _sized(t, dtype: str, count: int, what: str) -> Optional[int]:
    """Address of a contiguous tensor of `count` values of dtype (None passes)."""
    if t is None:
        return None
    if t.dtype is not _dtypes[dtype] or t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{what}: expected {count} contiguous {dtype} values, got {t.numel()} of {t.dtype}")
    return t.data_ptr()


def _bf16_sized(t, count: int, what: str) -> Optional[int]:
    if t is None:
        return None
    if _dense_type(t) != _BF16 or t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{what}: expected {count} contiguous bfloat16 values (or int16 bits), got {t.numel()} of {t.dtype}")
    return t.data_ptr()


def edge_moe_balance_ws_bytes(dims, n_seq=1) -> int:
    return int(load().edge_moe_balance_ws_bytes(ctypes.byref(cdims(dims)), _i32(n_seq)))


def edge_moe_balance(dims, logits, topk_idx, counts, probs, loss, ws, seq_offsets=None, stream=None) -> None:
    """The router's load: counts [S][E] int32, mean probabilities probs [S][E]
    and loss [2] (balance, z), float32, from logits [T][E] and topk_idx [T][k].
    seq_offsets int32 [S + 1]: the sequences' tokens (None: one sequence)."""
    T, E, k = dims.T, dims.n_experts, dims.top_k
    S = 1 if seq_offsets is None else seq_offsets.numel() - 1
    f, i = "float32", "int32"
    lib = load()
    dev = _same_device(logits, topk_idx, counts, probs, loss, ws, seq_offsets)
    st = lib.edge_moe_balance(cdims(dims), _sized(logits, f, T * E, "logits"),
                                 _sized(topk_idx, i, T * k, "topk_idx"), _sized(seq_offsets, i, S + 1, "seq_offsets"),
                                 _i32(S), _sized(counts, i, S * E, "counts"), _sized(probs, f, S * E, "probs"),
                                 _sized(loss, f, 2, "loss"), _ptr(ws), ws.numel() * ws.element_size(), _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_balance", st)


def edge_moe_route_backward_ws_bytes(dims) -> int:
    return int(load().edge_moe_route_backward_ws_bytes(ctypes.byref(cdims(dims))))


def edge_moe_route_backward(dims, logits, topk_idx, ws, topk_w=None, d_topk_w=None, d_loss=None, counts=None,
                            seq_offsets=None, x=None, w_router=None, dlogits=None, dx=None, dw_router=None, dbias=None,
                            stream=None) -> None:
    """The router's backward pass: from d_topk_w [T][k] and / or d_loss [2] (with
    edge_moe_balance's counts and seq_offsets) to those of dlogits [T][E], dx
    [T][d], dw_router [E][d], dbias [E] (float32) that are given.  dx needs
    w_router, dw_router needs x (bf16)."""
    T, E, k, d = dims.T, dims.n_experts, dims.top_k, dims.d
    S = 1 if seq_offsets is None else seq_offsets.numel() - 1
    f, i = "float32", "int32"
    lib = load()
    dev = _same_device(logits, topk_idx, ws, topk_w, d_topk_w, d_loss, counts, seq_offsets, x, w_router, dlogits, dx,
                       dw_router, dbias)
    g = CRouteGrad(_sized(logits, f, T * E, "logits"), _sized(topk_idx, i, T * k, "topk_idx"),
                   _sized(topk_w, f, T * k, "topk_w"), _sized(d_topk_w, f, T * k, "d_topk_w"),
                   _sized(d_loss, f, 2, "d_loss"), _sized(counts, i, S * E, "counts"),
                   _sized(seq_offsets, i, S + 1, "seq_offsets"), _i32(S), _bf16_sized(x, T * d, "x"),
                   _bf16_sized(w_router, E * d, "w_router"), _sized(dlogits, f, T * E, "dlogits"),
                   _sized(dx, f, T * d, "dx"), _sized(dw_router, f, E * d, "dw_router"), _sized(dbias, f, E, "dbias"))
    st = lib.edge_moe_route_backward(cdims(dims), g, _ptr(ws), ws.numel() * ws.element_size(), _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_route_backward", st)


def _same_device(first, *rest) -> int:
    """Every tensor on the current GPU, where the library launches; its index."""
    dev = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors must be on one GPU, got {first.device} and {t.device}")
    if dev < 0 or dev != _cuda.getDevice():
        raise ValueError(f"tensors must be on the current GPU, got {first.device}")
    return dev


def _stream_on(device: int, stream) -> int:
    """The stream's handle; None: the device's current stream.  A stream of
    another GPU would run the kernels there, on memory of this one."""
    if stream is None:
        return _cuda.getRawStream(device)
    if getattr(stream, "device_index", device) != device:
        raise ValueError(f"the stream must be of the tensors' GPU {device}, got one of GPU {stream.device_index}")
    return _stream(stream)


def _dense_type(t) -> int:
    """bf16 (bfloat16, or int16 / uint16 bit patterns) or float32."""
    kind = _dense_types.get(t.dtype)
    if kind is None:
        raise ValueError(f"expected bfloat16 (or its int16 bits) or float32, got {t.dtype}")
    return kind


def _row_stride(t) -> int:
    """Elements between the rows of t [..., N, K]: one stride for all rows."""
    if t.dim() < 2:
        raise ValueError("expected rows: a tensor of at least two dimensions")
    K = t.shape[-1]
    if t.is_contiguous():
        return K
    if K != 1 and t.stride(-1) != 1:
        raise ValueError("the elements of a row must be contiguous")
    stride, span = None, 1
    for n, s in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n != 1:
            if stride is None:
                stride = s
                if span != 1:
                    raise ValueError("the rows must lie at one stride")
            elif s != stride * span:
                raise ValueError("the rows must lie at one stride")
        span *= n
    return K if stride is None else stride


def _mx_shape(fmt, dense, codes, scales):
    """(M, N, K) of a dense tensor and the addresses of its MX codes and scales,
    checked against each other."""
    if fmt not in (MX_FP4, MX_FP8):
        raise ValueError("format must be MX_FP4 or MX_FP8")
    if dense.dim() < 2:
        raise ValueError("expected rows: a tensor of at least two dimensions")
    N, K = dense.shape[-2:]
    M = dense.numel() // (N * K or 1)
    q = _sized(codes, "uint8", M * N * (K // 2 if fmt == MX_FP4 else K), "codes")
    e = _sized(scales, "uint8", M * N * (K // 32), "scales")
    if max(M, N, K) > 0x7FFFFFFF:
        M, N, K = _i32(M), _i32(N), _i32(K)
    return M, N, K, q, e


def edge_moe_mx_quantize(fmt, src, codes, scales, stream=None) -> None:
    """Dense matrices src [..., N, K] (bf16 or float32, rows at one stride) to
    MX codes [..., N, K/2] (MX_FP4) or [..., N, K] (MX_FP8) and E8M0 scales
    [..., K/128, N, 4], both uint8."""
    lib = load()
    M, N, K, q, e = _mx_shape(fmt, src, codes, scales)
    dev = _same_device(src, codes, scales)
    st = lib.edge_moe_mx_quantize(M, N, K, fmt, _dense_type(src), src.data_ptr(), _row_stride(src), q, e,
                                     _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_mx_quantize", st)


def edge_moe_mx_dequantize(fmt, codes, scales, dst, stream=None) -> None:
    """MX codes and scales back to dense dst [..., N, K] (bf16 or float32)."""
    lib = load()
    M, N, K, q, e = _mx_shape(fmt, dst, codes, scales)
    dev = _same_device(dst, codes, scales)
    st = lib.edge_moe_mx_dequantize(M, N, K, fmt, _dense_type(dst), q, e, dst.data_ptr(), _row_stride(dst),
                                       _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_mx_dequantize", st)


def edge_moe_mx_product_ws_bytes(T, R, M, N, K, x_format) -> int:
    return int(load().edge_moe_mx_product_ws_bytes(ctypes.byref(_int32s(CMxDims, _pack_mx_dims, T, R, M, N, K, x_format))))


def edge_moe_mx_product(x_format, x, codes, scales, y, ws, offsets=None, row_src=None, stream=None) -> None:
    """y [R][N] (bf16) = the rows of x [T][K] (bf16), rounded to x_format, times
    MXFP4 matrices codes [M][N][K/2], scales [M][K/128][N][4] (or one matrix
    without the leading dimension).  offsets int32 [M + 1]: the y rows of each
    matrix; row_src int32 [R]: the x row of each y row."""
    lib = load()
    if x.dim() != 2 or y.dim() != 2 or _dense_type(x) != _BF16 or _dense_type(y) != _BF16:
        raise ValueError("x and y must be bfloat16 (or int16 bits) [rows][columns]")
    (T, K), (R, N) = x.shape, y.shape
    if max(T, R) >= 1 << 31:            # the library's sizes are 32 bits
        raise ValueError(f"x and y have too many rows: {T}, {R}")
    M = 1 if codes.dim() == 2 else codes.shape[0]
    q = _sized(codes, "uint8", M * N * (K // 2), "codes")
    e = _sized(scales, "uint8", M * N * (K // 32), "scales")
    off, src = _sized(offsets, "int32", M + 1, "offsets"), _sized(row_src, "int32", R, "row_src")
    dev = _same_device(x, codes, scales, y, ws, offsets, row_src)
    st = lib.edge_moe_mx_product(_int32s(CMxDims, _pack_mx_dims, T, R, M, N, K, x_format), x.data_ptr(), _row_stride(x), src, off, q, e,
                                    y.data_ptr(), _row_stride(y), _ptr(ws), ws.numel() * ws.element_size(),
                                    _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_mx_product", st)


def edge_moe_mx_product_coded(x_format, x_codes, x_scales, codes, scales, y, offsets=None, row_src=None, stream=None) -> None:
    """edge_moe_mx_product from x in MX codes: x_codes uint8 [T][K] (MX_FP8) or
    [T][K/2] (MX_FP4), x_scales uint8 [K/128][T][4], as edge_moe_norm and
    edge_moe_mx_quantize write them."""
    lib = load()
    if x_format not in (MX_FP4, MX_FP8):
        raise ValueError("x_format must be MX_FP4 or MX_FP8")
    if x_codes.dim() != 2 or y.dim() != 2 or _dense_type(y) != _BF16:
        raise ValueError("x_codes must be [T][K] bytes, y bfloat16 (or int16 bits) [R][N]")
    (T, K), (R, N) = x_codes.shape, y.shape
    K *= 2 if x_format == MX_FP4 else 1
    M = 1 if codes.dim() == 2 else codes.shape[0]
    dev = _same_device(x_codes, x_scales, codes, scales, y, offsets, row_src)
    st = lib.edge_moe_mx_product_coded(
        _int32s(CMxDims, _pack_mx_dims, T, R, M, N, K, x_format), _sized(x_codes, "uint8", x_codes.numel(), "x_codes"),
        _sized(x_scales, "uint8", T * (K // 32), "x_scales"), _sized(row_src, "int32", R, "row_src"),
        _sized(offsets, "int32", M + 1, "offsets"), _sized(codes, "uint8", M * N * (K // 2), "codes"),
        _sized(scales, "uint8", M * N * (K // 32), "scales"), *_rows(y, R, N, "y"), _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_mx_product_coded", st)


def mx_weights(dense: dict, stream=None) -> dict:
    """The MX weight dict of edge_moe_forward_mx from dense matrices: "s_up"
    [G][h][d], "s_dn" [G][d][h], "a_up" [E][r][d], "b_up" [E][h][r], "a_dn"
    [E][r][h], "b_dn" [E][d][r] (bf16 or float32) are quantised to MXFP4; the
    LoRA factors, bf16, are taken as they are.  The new tensors belong to
    `stream`; what uses them on another one waits for it."""
    import torch
    out = {}
    for key in _WEIGHT_KEYS[:12:2]:
        src = dense[key]
        M, N, K = src.shape
        with _made_on(stream):
            out[key] = torch.empty(M, N, K // 2, dtype=torch.uint8, device=src.device)
            out[key + "_scale"] = torch.empty(M, K // 128, N, 4, dtype=torch.uint8, device=src.device)
        edge_moe_mx_quantize(MX_FP4, src, out[key], out[key + "_scale"], stream)
    for key in _WEIGHT_KEYS[12:16]:
        out[key] = dense[key]
    return out


# ------------------------------------------------ norm, dense and int4 matrices ----

def _rows(t, count: int, cols: int, what: str):
    """(address, stride) of a tensor of `count` rows of `cols`, at one stride; (0, 0) for None."""
    if t is None:
        return 0, 0
    if t.numel() != count * cols or t.dim() < 2 or t.size(-1) != cols:
        raise ValueError(f"{what}: expected {count} rows of {cols}, got {tuple(t.shape)}")
    return t.data_ptr(), cols if t.is_contiguous() else _row_stride(t)


def _bf16_rows(t, count: int, cols: int, what: str):
    if t is None:
        return 0, 0
    if _dense_types.get(t.dtype) != _BF16:
        raise ValueError(f"{what}: expected bfloat16 (or int16 bits), got {t.dtype}")
    return _rows(t, count, cols, what)


def _vector(t, count: int, what: str) -> int:
    """Address of a contiguous bf16 or float32 vector."""
    if t.numel() != count or not t.is_contiguous():
        raise ValueError(f"{what}: expected {count} contiguous values, got {t.numel()}")
    return t.data_ptr()


def _rows_of(x):
    """(T, d) of a tensor of T rows of d values."""
    if x.dim() < 2:
        raise ValueError("x must be rows: a tensor of at least two dimensions")
    d = x.size(-1)
    T = x.numel() // (d or 1)
    return (T, d) if T <= 0x7FFFFFFF >= d else (_i32(T), _i32(d))


def edge_moe_norm(x, gain, eps, add=None, x_out=None, y=None, codes=None, scales=None, rstd=None, stream=None) -> None:
    """r = bf16(x + add) to x_out, y = bf16(r rstd gain) with rstd = 1 / sqrt(mean r^2
    + eps), and y's MXFP8 codes [..., T, d] and scales [..., d/128, T, 4]: those of
    the outputs that are given.  x, x_out, y bf16 rows [T][d] at one stride, add bf16
    or float32, gain [d] bf16 or float32."""
    lib = load()
    T, d = _rows_of(x)
    dev = _same_device(x, gain, add, x_out, y, codes, scales, rstd)
    a = _pack_norm(T, d, eps, 0 if add is None else _dense_type(add), _dense_type(gain), *_bf16_rows(x, T, d, "x"),
                   *_rows(add, T, d, "add"), _vector(gain, d, "gain"), *_bf16_rows(x_out, T, d, "x_out"),
                   *_bf16_rows(y, T, d, "y"), _sized(codes, "uint8", T * d, "codes") or 0,
                   _sized(scales, "uint8", T * (d // 32), "scales") or 0, _sized(rstd, "float32", T, "rstd") or 0)
    st = lib.edge_moe_norm(CNormArgs.from_buffer_copy(a), _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_norm", st)


def edge_moe_norm_backward_ws_bytes(T, d) -> int:
    return int(load().edge_moe_norm_backward_ws_bytes(_i32(T), _i32(d)))


def edge_moe_norm_backward(x, gain, rstd, dy, ws, dres=None, dx=None, dgain=None, stream=None) -> None:
    """The norm's backward pass at x (the forward pass's x_out, or its x where nothing
    was added): dx = dres + the gradient through y, dgain [d] float32.  dy, dres and
    dx rows of one type, bf16 or float32."""
    lib = load()
    T, d = _rows_of(x)
    kind = _dense_type(dy)
    if (dres is not None and _dense_type(dres) != kind) or (dx is not None and _dense_type(dx) != kind):
        raise ValueError(f"dres and dx must be of dy's type, {dy.dtype}")
    dev = _same_device(x, gain, rstd, dy, ws, dres, dx, dgain)
    g = _pack_norm_grad(T, d, _dense_type(gain), kind, *_bf16_rows(x, T, d, "x"), _vector(gain, d, "gain"),
                        _sized(rstd, "float32", T, "rstd"), *_rows(dy, T, d, "dy"), *_rows(dres, T, d, "dres"),
                        *_rows(dx, T, d, "dx"), _sized(dgain, "float32", d, "dgain") or 0)
    st = lib.edge_moe_norm_backward(CNormGrad.from_buffer_copy(g), _ptr(ws), ws.numel() * ws.element_size(), _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_norm_backward", st)


# the structs' layouts (native alignment), packed without a conversion per field
_pack_norm = struct.Struct("iifii4xPqPqPPqPqPPP").pack
_pack_norm_grad = struct.Struct("iiiiPqPPPqPqPqP").pack
_pack_dense_grad = struct.Struct("PqPqPPPi4xPPqiiP").pack


def _dense_dims(T, R, M, N, K) -> CDenseDims:
    return _int32s(CDenseDims, _pack_dense_dims, T, R, M, N, K)


def _matrices(w, what: str):
    """(M, N, K) and address of contiguous bf16 matrices [M][N][K] or one [N][K]."""
    n = w.dim()
    if n not in (2, 3) or _dense_type(w) != _BF16 or not w.is_contiguous():
        raise ValueError(f"{what}: expected contiguous bfloat16 matrices [M][N][K]")
    return (1 if n == 2 else w.size(0)), w.size(-2), w.size(-1), w.data_ptr()


def edge_moe_dense_product_ws_bytes(T, R, M, N, K) -> int:
    return int(load().edge_moe_dense_product_ws_bytes(_dense_dims(T, R, M, N, K)))


def edge_moe_dense_product(x, w, y, ws, offsets=None, row_src=None, stream=None) -> None:
    """y [R][N] (bf16 or float32) = the rows of x [T][K] (bf16) times bf16 matrices w
    [M][N][K] (or one matrix [N][K]).  offsets int32 [M + 1]: the y rows of each
    matrix; row_src int32 [R]: the x row of each y row."""
    lib = load()
    M, N, K, wp = _matrices(w, "w")
    if x.dim() != 2 or y.dim() != 2:
        raise ValueError("x and y must be rows: [rows][columns]")
    T, R = x.shape[0], y.shape[0]
    dev = _same_device(x, w, y, ws, offsets, row_src)
    st = lib.edge_moe_dense_product(_dense_dims(T, R, M, N, K), *_bf16_rows(x, T, K, "x"), _sized(row_src, "int32", R, "row_src"),
                                    _sized(offsets, "int32", M + 1, "offsets"), wp, _dense_type(y), *_rows(y, R, N, "y"),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_dense_product", st)


def edge_moe_dense_product_backward_ws_bytes(T, R, M, N, K) -> int:
    return int(load().edge_moe_dense_product_backward_ws_bytes(_dense_dims(T, R, M, N, K)))


def edge_moe_dense_product_backward(dy, ws, x=None, w=None, dx=None, dw=None, offsets=None, row_src=None, token_rows=None,
                                    stream=None) -> None:
    """Gradients of edge_moe_dense_product from dy [R][N] (bf16), bf16 or float32 each:
    dx from w, [R][K] by rows or, with token_rows int32 [T][k] (the rows of each
    token, -1 for none), [T][K] by tokens; dw [M][N][K] from x and row_src."""
    lib = load()
    if dy.dim() != 2 or (dx is None and dw is None):
        raise ValueError("dy must be rows [R][N], and dx or dw given")
    if (dx is not None and w is None) or (dw is not None and x is None):
        raise ValueError("dx needs w, dw needs x")
    R, N = dy.shape
    like = dw if dx is None else w
    M, K = (1 if like.dim() == 2 else like.size(0)), like.size(-1)
    for t in (w if dx is not None else None, dw):
        if t is not None and (t.dim() not in (2, 3) or not t.is_contiguous() or t.size(-2) != N or t.size(-1) != K or t.numel() != M * N * K):
            raise ValueError(f"w and dw: expected contiguous matrices {M} x {N} x {K}, got {tuple(t.shape)}")
    if dx is not None and _dense_type(w) != _BF16:
        raise ValueError(f"w: expected bfloat16 (or int16 bits), got {w.dtype}")
    k = 0
    if token_rows is not None:
        if token_rows.dim() != 2 or token_rows.size(1) < 1:
            raise ValueError("token_rows must be [T][k], k at least 1")
        k = token_rows.size(1)
    if dw is not None and x.dim() != 2:
        raise ValueError("x must be rows [T][K]")
    T = x.size(0) if dw is not None else token_rows.size(0) if token_rows is not None else 1
    dev = _same_device(dy, ws, x, w, dx, dw, offsets, row_src, token_rows)
    g = _pack_dense_grad(*_bf16_rows(dy, R, N, "dy"), *(_bf16_rows(x, T, K, "x") if dw is not None else (0, 0)),
                         _sized(row_src, "int32", R, "row_src") or 0, _sized(offsets, "int32", M + 1, "offsets") or 0,
                         _sized(token_rows, "int32", T * k, "token_rows") or 0, _i32(k), 0 if dx is None else w.data_ptr(),
                         *_rows(dx, T if k else R, K, "dx"), 0 if dx is None else _dense_type(dx),
                         0 if dw is None else _dense_type(dw), 0 if dw is None else dw.data_ptr())
    st = lib.edge_moe_dense_product_backward(_dense_dims(T, R, M, N, K), CDenseGrad.from_buffer_copy(g), _ptr(ws),
                                             ws.numel() * ws.element_size(), _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_dense_product_backward", st)


def _packed_dims(T, R, M, N, K, quant_group) -> CPackedDims:
    return _int32s(CPackedDims, _pack_mx_dims, T, R, M, N, K, quant_group)


def edge_moe_packed_product_ws_bytes(T, R, M, N, K, quant_group) -> int:
    return int(load().edge_moe_packed_product_ws_bytes(_packed_dims(T, R, M, N, K, quant_group)))


def edge_moe_packed_product(quant_group, x, codes, scales, y, ws, offsets=None, row_src=None, stream=None) -> None:
    """y [R][N] (bf16 or float32) = the rows of x [T][K] (bf16) times int4 matrices:
    codes uint8 [M][N][K/2] and fp16 scales [M][N][K/min(quant_group, K)] (or one
    matrix without the leading dimension), as in the layer's weight dicts.  offsets
    int32 [M + 1]: the y rows of each matrix; row_src int32 [R]: the x row of each."""
    lib = load()
    if x.dim() != 2 or y.dim() != 2 or quant_group < 1:
        raise ValueError("x and y must be rows: [rows][columns], quant_group a group's elements")
    (T, K), (R, N) = x.shape, y.shape
    M = 1 if codes.dim() == 2 else codes.shape[0]
    if scales.dtype not in _half_types or not scales.is_contiguous() or scales.numel() != M * N * (K // (min(quant_group, K) or 1)):
        raise ValueError(f"scales: expected {M} x {N} x {K} / {quant_group} contiguous float16 values (or int16 bits)")
    dev = _same_device(x, codes, scales, y, ws, offsets, row_src)
    st = lib.edge_moe_packed_product(_packed_dims(T, R, M, N, K, quant_group), *_bf16_rows(x, T, K, "x"),
                                   _sized(row_src, "int32", R, "row_src"), _sized(offsets, "int32", M + 1, "offsets"),
                                   _sized(codes, "uint8", M * N * (K // 2), "codes"), scales.data_ptr(), _dense_type(y),
                                   *_rows(y, R, N, "y"), _ptr(ws), ws.numel() * ws.element_size(), _stream_on(dev, stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_packed_product", st)


def edge_moe_residual(x, y, x_out, stream=None) -> None:
    T, d = x.shape
    st = load().edge_moe_residual(int(T), int(d), _ptr(x), _ptr(y), _ptr(x_out), _stream(stream))
    if st != EDGE_MOE_OK:
        raise EdgeMoeError("edge_moe_residual", st)


def _host_ptr(t) -> Optional[int]:
    if t is None:
        return None
    if t.is_cuda:
        raise ValueError("this argument must be in host memory")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _stats(c: CCacheStats) -> dict:
    return {n: int(getattr(c, n)) for n, _ in CCacheStats._fields_}


class ExpertCache:
    """edge_moe_cache_*: an LRU of `slots_per_group` HBM slots per group for one
    layer's expert tensors, filled from host memory.

    host:  dict with EXPERT_TENSOR_KEYS (the last two optional) of host tensors
           holding the layer's E experts (pin them for the copies to overlap);
    slots: dict of device tensors with G * S experts each, the same keys set,
           or None for a cache that only plans.
    map() renames a batch's expert ids to slots and issues the copies of the
    misses; the layer then runs on slot_dims() with the slot tensors in place
    of the expert tensors (slot_weights())."""

    def __init__(self, dims, slots_per_group: int, host: dict, slots: Optional[dict] = None):
        self._lib = load()
        self.S = int(slots_per_group)
        self._keep = (host, slots)
        # the library trusts the buffers to hold E experts (host) and G * S
        # slots (device) of the per-expert sizes its dims imply: check them here
        per = expert_tensor_bytes(dims)
        G = dims.n_experts // dims.experts_per_group
        for k in EXPERT_TENSOR_KEYS:
            for side, tensors, count in (("host", host, dims.n_experts), ("slot", slots, G * self.S)):
                t = None if tensors is None else tensors.get(k)
                if t is not None and t.numel() * t.element_size() != count * per[k]:
                    raise ValueError(f"{side} tensor {k}: {t.numel() * t.element_size()} bytes, "
                                     f"expected {count} x {per[k]}")
        ch = CExpertTensors(*(_host_ptr(host.get(k)) for k in EXPERT_TENSOR_KEYS))
        cs = None if slots is None else CExpertTensors(*(_ptr(slots.get(k)) for k in EXPERT_TENSOR_KEYS))
        self._h = self._lib.edge_moe_cache_create(ctypes.byref(cdims(dims)), self.S, ctypes.byref(ch),
                                                  None if cs is None else ctypes.byref(cs))
        if not self._h:
            raise ValueError("edge_moe_cache_create rejected its arguments")

    def map(self, topk_idx, slot_idx, stream=None) -> dict:
        """topk_idx, slot_idx: host int32 [T][k] tensors; returns this call's counts."""
        T = topk_idx.shape[0] if topk_idx.dim() else 0
        st = CCacheStats()
        r = self._lib.edge_moe_cache_map(self._h, int(T), _host_ptr(topk_idx), _host_ptr(slot_idx),
                                         _stream(stream) if self._keep[1] is not None else None, ctypes.byref(st))
        if r != EDGE_MOE_OK:
            raise EdgeMoeError("edge_moe_cache_map", r)
        return _stats(st)

    def prefetch(self, experts, stream=None) -> dict:
        st = CCacheStats()
        r = self._lib.edge_moe_cache_prefetch(self._h, int(experts.numel()), _host_ptr(experts),
                                              _stream(stream) if self._keep[1] is not None else None,
                                              ctypes.byref(st))
        if r != EDGE_MOE_OK:
            raise EdgeMoeError("edge_moe_cache_prefetch", r)
        return _stats(st)

    def totals(self) -> dict:
        st = CCacheStats()
        r = self._lib.edge_moe_cache_totals(self._h, ctypes.byref(st))
        if r != EDGE_MOE_OK:
            raise EdgeMoeError("edge_moe_cache_totals", r)
        return _stats(st)

    def slot_of(self, expert: int) -> int:
        return int(self._lib.edge_moe_cache_slot_of(self._h, int(expert)))

    def close(self) -> None:
        if self._h:
            self._lib.edge_moe_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def expert_tensor_bytes(dims) -> dict:
    """Bytes of one expert's tensor of each EXPERT_TENSOR_KEYS key (packed int4
    codes, fp16 scales per min(quant_group, K) elements; the decode copies are
    the size of the codes they copy)."""
    r, d, h, q = dims.delta_rank, dims.d, dims.h, dims.quant_group
    sc = lambda n, k: n * (k // min(q, k)) * 2  # noqa: E731
    out = {"a_up": r * d // 2, "a_up_scale": sc(r, d), "b_up": h * r // 2, "b_up_scale": sc(h, r),
           "a_dn": r * h // 2, "a_dn_scale": sc(r, h), "b_dn": d * r // 2, "b_dn_scale": sc(d, r)}
    out["a_up_t"], out["a_dn_t"] = out["a_up"], out["a_dn"]
    return out


class _SlotDims:
    def __init__(self, dims, S: int):
        for f, _ in CDims._fields_:
            setattr(self, f, int(getattr(dims, f)))
        self.n_experts = (self.n_experts // self.experts_per_group) * S
        self.experts_per_group = S


def slot_dims(dims, slots_per_group: int):
    """The dims of the slot layer: G groups of S experts."""
    return _SlotDims(dims, slots_per_group)


def slot_weights(weights: dict, slots: dict) -> dict:
    """The resident layer's weights with the slot tensors in place of the
    per-expert tensors (missing optional slot tensors drop the key)."""
    out = {k: v for k, v in weights.items() if k not in EXPERT_TENSOR_KEYS}
    out.update({k: v for k, v in slots.items() if v is not None})
    return out


def edge_moe_prof_enable(on: bool) -> bool:
    return bool(load().edge_moe_prof_enable(1 if on else 0))


def edge_moe_prof_reset() -> None:
    load().edge_moe_prof_reset()


def edge_moe_prof_read() -> dict:
    """{kernel name: (launches, total ms)} accumulated since the last reset."""
    lib = load()
    n = lib.edge_moe_prof_read(None, None, None, 0)
    names = (ctypes.c_char * 64 * max(n, 1))()
    launches = (ctypes.c_int64 * max(n, 1))()
    total = (ctypes.c_double * max(n, 1))()
    n = lib.edge_moe_prof_read(ctypes.cast(names, ctypes.c_void_p), ctypes.cast(launches, ctypes.c_void_p),
                               ctypes.cast(total, ctypes.c_void_p), n)
    return {names[i].value.decode(): (int(launches[i]), float(total[i])) for i in range(n)}
