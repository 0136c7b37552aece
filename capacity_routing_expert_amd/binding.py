"""Thin ctypes binding of libmoe (include/moe.h): argument marshalling only.

Every step of the layer runs in the HIP library; this module only turns torch tensors into
device pointers, picks torch's current stream, checks the dtype, device, contiguity and size
(number of elements against what the shape needs) of every tensor it is handed, and raises on
a non-OK status.  torch is imported before the library is
loaded so that both use torch's HIP runtime (one runtime per process).

The library is loaded on first use; if it has not been built the call raises, there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_F32, MOE_BF16 = 0, 1
MOE_WEIGHTS_ROW_MAJOR, MOE_WEIGHTS_PACKED = 0, 1
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARGUMENT", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_DEVICE"}

EXPORTS = ("moe_capacity", "moe_workspace_bytes", "moe_max_kept_rows", "moe_status_string",
           "moe_last_error", "moe_route", "moe_dispatch", "moe_expert_ffn", "moe_combine",
           "moe_layer_forward", "moe_layer_forward_profiled", "moe_workspace_bytes_padded",
           "moe_layer_forward_padded", "moe_layer_forward_gated", "moe_workspace_bytes_dropless",
           "moe_dispatch_pairs", "moe_expert_ffn_pairs", "moe_sum", "moe_layer_forward_dropless",
           "moe_layer_forward_dropless_gated", "moe_workspace_bytes_batches",
           "moe_schedule_batches", "moe_layer_forward_batches", "moe_packed_weights_bytes",
           "moe_pack_weights", "moe_set_gemm_timing", "moe_set_stage_timing",
           "moe_layer_forward_noalloc", "moe_workspace_bytes_balance", "moe_balance_loss",
           "moe_workspace_bytes_route_backward", "moe_route_backward", "moe_quantized_codes_bytes",
           "moe_quantized_scales_bytes", "moe_quantize_weights", "moe_dequantize_weights",
           "moe_expert_ffn_quantized", "moe_layer_forward_quantized",
           "moe_workspace_bytes_route_scored", "moe_route_scored", "moe_route_scored_backward",
           "moe_combine_backward", "moe_combine_backward_rows", "moe_workspace_bytes_balance_bias", "moe_balance_bias", "moe_adamw_check",
           "moe_adamw_step", "moe_adamw_moments")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("capacity", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("weight_layout", ctypes.c_int32)]


class MoeQuantizedExperts(ctypes.Structure):
    """moe_quantized_experts; QuantizedExperts fills it and keeps the tensors."""
    _fields_ = [("w1_codes", ctypes.c_void_p), ("w1_scales", ctypes.c_void_p),
                ("b1", ctypes.c_void_p), ("w2_codes", ctypes.c_void_p),
                ("w2_scales", ctypes.c_void_p), ("b2", ctypes.c_void_p),
                ("group", ctypes.c_int32), ("gated", ctypes.c_int32)]


class MoeRouting(ctypes.Structure):
    """moe_routing; make_routing fills it."""
    _fields_ = [("score", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


class MoeAdamWTensor(ctypes.Structure):
    """moe_adamw_tensor; AdamWTensors fills an array of them and keeps the tensors."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "m_steps", "v_steps",
                                               "copy")] + [
        ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float)]


class MoeAdamWConfig(ctypes.Structure):
    """moe_adamw_config."""
    _fields_ = [("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("state_bits", ctypes.c_int32), ("lr", ctypes.c_float), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("eps", ctypes.c_float), ("grad_scale", ctypes.c_float),
                ("step", ctypes.c_int64), ("dynamic", ctypes.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m capacity_routing_expert_amd.build` (no fallback exists)")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        SP = ctypes.POINTER(MoeShape)
        L.moe_capacity.argtypes = [I64, I32, I32, ctypes.c_double]
        L.moe_capacity.restype = I32
        L.moe_workspace_bytes.argtypes = [SP]
        L.moe_workspace_bytes.restype = SZ
        L.moe_max_kept_rows.argtypes = [SP]
        L.moe_max_kept_rows.restype = I64
        L.moe_status_string.argtypes = [I32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_route.argtypes = [SP, P, P, P, P, P, P, P, SZ, P]
        L.moe_dispatch.argtypes = [SP, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.moe_expert_ffn.argtypes = [SP, P, P, P, P, P, P, P, P, P, SZ, P]
        L.moe_combine.argtypes = [SP, P, P, P, P, P, P]
        L.moe_layer_forward.argtypes = [SP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.moe_layer_forward_profiled.argtypes = L.moe_layer_forward.argtypes + [P]
        # moe_layer_forward's arguments without ws and ws_bytes
        L.moe_layer_forward_noalloc.argtypes = [SP] + [P] * 13 + [P]
        L.moe_workspace_bytes_padded.argtypes = [SP]
        L.moe_workspace_bytes_padded.restype = SZ
        # shape, x, w_router, b_router, w1, b1, w2, b2, out, ids, gates, slot_of, drop, counts,
        # y_rows, ws, ws_bytes, stream, events
        L.moe_layer_forward_padded.argtypes = [SP] + [P] * 15 + [SZ, P, P]
        # shape, x, w_router, b_router, w13, w2, out, ids, gates, slot_of, drop, counts, ws,
        # ws_bytes, stream, events
        L.moe_layer_forward_gated.argtypes = [SP] + [P] * 12 + [SZ, P, P]
        L.moe_workspace_bytes_dropless.argtypes = [SP]
        L.moe_workspace_bytes_dropless.restype = SZ
        L.moe_dispatch_pairs.argtypes = [SP, P, P, P, P, P, P, SZ, P]
        # shape, x, sorted_pairs, row_token, offsets, w1, b1, w2, b2, weights, gated, pair_rows,
        # ws, ws_bytes, stream
        L.moe_expert_ffn_pairs.argtypes = [SP] + [P] * 9 + [I32, P, P, SZ, P]
        L.moe_sum.argtypes = [SP, P, P, P, P, P]
        # shape, x, w_router, b_router, w1, b1, w2, b2, out, ids, gates, counts, pair_rows, ws,
        # ws_bytes, stream, events
        L.moe_layer_forward_dropless.argtypes = [SP] + [P] * 13 + [SZ, P, P]
        # shape, x, w_router, b_router, w13, w2, out, ids, gates, counts, pair_rows, ws,
        # ws_bytes, stream, events
        L.moe_layer_forward_dropless_gated.argtypes = [SP] + [P] * 11 + [SZ, P, P]
        L.moe_packed_weights_bytes.argtypes = [SP, I32, I32]
        L.moe_packed_weights_bytes.restype = SZ
        L.moe_pack_weights.argtypes = [SP, P, I32, I32, P, P]
        L.moe_pack_weights.restype = I32
        L.moe_workspace_bytes_batches.argtypes = [SP, I32]
        L.moe_workspace_bytes_batches.restype = SZ
        L.moe_schedule_batches.argtypes = [SP, I32, P, P, P, P, P]
        # shape, n_batches, consolidate, x, w_router, b_router, w1, b1, w2, b2, out, ids, gates,
        # order, batch_experts, ws, ws_bytes, stream, events
        L.moe_layer_forward_batches.argtypes = [SP, I32, I32] + [P] * 13 + [SZ, P, P]
        L.moe_set_gemm_timing.argtypes = [P]
        L.moe_set_gemm_timing.restype = I32
        L.moe_set_stage_timing.argtypes = [P]
        L.moe_set_stage_timing.restype = I32
        for name in ("moe_workspace_bytes_balance", "moe_workspace_bytes_route_backward"):
            getattr(L, name).argtypes = [SP]
            getattr(L, name).restype = SZ
        # shape, logits, topk_ids, token_mask, coef, grad_scale, loss, counts, probs, dlogits, ws,
        # ws_bytes, stream
        L.moe_balance_loss.argtypes = ([SP, P, P, P, ctypes.c_float, ctypes.c_float] + [P] * 5 +
                                       [SZ, P])
        # shape, x, w_router, logits, topk_ids, dgates, dlogits, token_mask, dx_add, dx, dw, db,
        # ws, ws_bytes, stream
        L.moe_route_backward.argtypes = [SP] + [P] * 12 + [SZ, P]
        L.moe_quantized_codes_bytes.argtypes = [SP, I32, I32]
        L.moe_quantized_codes_bytes.restype = SZ
        L.moe_quantized_scales_bytes.argtypes = [SP, I32, I32, I32]
        L.moe_quantized_scales_bytes.restype = SZ
        L.moe_quantize_weights.argtypes = [SP, P, I32, I32, I32, P, P, P]
        L.moe_dequantize_weights.argtypes = [SP, P, P, I32, I32, I32, P, P]
        QP = ctypes.POINTER(MoeQuantizedExperts)
        L.moe_expert_ffn_quantized.argtypes = [SP, P, P, P, QP, P, P, SZ, P]
        # shape, x, w_router, b_router, experts, out, ids, gates, slot_of, drop, counts, ws,
        # ws_bytes, stream, events
        L.moe_layer_forward_quantized.argtypes = [SP, P, P, P, QP] + [P] * 7 + [SZ, P, P]
        for name in ("moe_workspace_bytes_route_scored", "moe_workspace_bytes_balance_bias"):
            getattr(L, name).argtypes = [SP]
            getattr(L, name).restype = SZ
        RP = ctypes.POINTER(MoeRouting)
        # shape, routing, x, w_router, b_router, score_bias, token_mask, ids, gates, logits, ws,
        # ws_bytes, stream
        L.moe_route_scored.argtypes = [SP, RP] + [P] * 9 + [SZ, P]
        # shape, routing, logits, ids, dgates, dlogits_add, token_mask, dlogits, stream
        L.moe_route_scored_backward.argtypes = [SP, RP] + [P] * 7
        # shape, dout, gates, slot_of, y_rows, dgates, dy_rows, stream
        L.moe_combine_backward.argtypes = [SP] + [P] * 7
        # shape, dout, gates, slot_of, y_rows, n_rows, dgates, dy_rows, stream
        L.moe_combine_backward_rows.argtypes = [SP] + [P] * 4 + [I64] + [P] * 3
        # shape, topk_ids, token_mask, rate, score_bias, counts, ws, ws_bytes, stream
        L.moe_balance_bias.argtypes = [SP, P, P, ctypes.c_float, P, P, P, SZ, P]
        CP, TP = ctypes.POINTER(MoeAdamWConfig), ctypes.POINTER(MoeAdamWTensor)
        L.moe_adamw_check.argtypes = [CP, TP, I32]
        L.moe_adamw_step.argtypes = [CP, TP, I32, P]
        # config, tensors, n, m_out, v_out, stream
        L.moe_adamw_moments.argtypes = [CP, TP, I32, P, P, P]
        for name in ("moe_route_scored", "moe_route_scored_backward", "moe_combine_backward",
                     "moe_combine_backward_rows", "moe_balance_bias", "moe_adamw_check", "moe_adamw_step", "moe_adamw_moments",
                     "moe_quantize_weights", "moe_dequantize_weights", "moe_expert_ffn_quantized",
                     "moe_layer_forward_quantized", "moe_balance_loss", "moe_route_backward", "moe_route", "moe_dispatch", "moe_expert_ffn", "moe_combine",
                     "moe_layer_forward", "moe_layer_forward_profiled", "moe_layer_forward_padded",
                     "moe_layer_forward_noalloc",
                     "moe_layer_forward_gated", "moe_dispatch_pairs", "moe_expert_ffn_pairs",
                     "moe_sum", "moe_layer_forward_dropless", "moe_layer_forward_dropless_gated",
                     "moe_schedule_batches", "moe_layer_forward_batches"):
            getattr(L, name).restype = I32
        _lib = L
    return _lib


def make_shape(T: int, d_model: int, d_ff: int, n_experts: int, top_k: int, capacity: int,
               dtype: int, weight_layout: int = MOE_WEIGHTS_ROW_MAJOR) -> MoeShape:
    return MoeShape(int(T), int(d_model), int(d_ff), int(n_experts), int(top_k), int(capacity),
                    int(dtype), int(weight_layout))


def capacity(T: int, top_k: int, n_experts: int, capacity_factor: float) -> int:
    return int(lib().moe_capacity(int(T), int(top_k), int(n_experts), float(capacity_factor)))


def workspace_bytes(shape: MoeShape) -> int:
    return int(lib().moe_workspace_bytes(ctypes.byref(shape)))


def workspace_bytes_padded(shape: MoeShape) -> int:
    return int(lib().moe_workspace_bytes_padded(ctypes.byref(shape)))


def workspace_bytes_dropless(shape: MoeShape) -> int:
    return int(lib().moe_workspace_bytes_dropless(ctypes.byref(shape)))


def max_kept_rows(shape: MoeShape) -> int:
    return int(lib().moe_max_kept_rows(ctypes.byref(shape)))


def last_error() -> str:
    return lib().moe_last_error().decode()


def _ptr(t: torch.Tensor | None, name: str, dtype=None, device=None,
         numel: int | None = None) -> ctypes.c_void_p | None:
    """Device pointer of `t` after checking its dtype, device, contiguity and that it holds at
    least `numel` elements (the library writes or reads that many through the raw pointer)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, the shape needs {numel}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _n(shape: MoeShape) -> dict:
    """Element counts the shape needs per argument kind."""
    T, d, f, E, k = int(shape.T), int(shape.d_model), int(shape.d_ff), int(shape.n_experts), int(shape.top_k)
    rows = max(int(max_kept_rows(shape)), 0)
    return {"x": T * d, "wr": E * d, "E": E, "E1": E + 1, "Tk": T * k, "TE": T * E,
            "rows": rows, "yrows": rows * d, "f": f, "d": d, "T": T, "k": k}


def _w(shape: MoeShape, rows: int, cols: int) -> int:
    """Elements of one expert weight array of [E, rows, cols] in the shape's layout."""
    E = int(shape.n_experts)
    if shape.weight_layout == MOE_WEIGHTS_PACKED and shape.dtype == MOE_BF16:
        return E * ((cols + 31) // 32) * rows * 32
    return E * rows * cols  # row-major (other layouts and dtypes are refused by the library)


# the handle alone: torch.cuda.current_stream() makes an object around it, 3 us of the 10 us that a
# small call takes on the host
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev: int | None = None) -> ctypes.c_void_p:
    """The handle of `stream`, or of the current one (of device `dev`, if it has been looked up)."""
    if stream is None and _raw_stream is not None:
        if dev is not None and dev >= 0:
            return _raw_stream(dev)
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise MoeError(status, where, last_error())


def _dtype_of(shape: MoeShape):
    return torch.bfloat16 if shape.dtype == MOE_BF16 else torch.float32


def moe_route(shape, x, w_router, b_router, topk_ids, topk_gates, logits, ws, stream=None):
    dt, n = _dtype_of(shape), _n(shape)
    _check(lib().moe_route(ctypes.byref(shape), _ptr(x, "x", dt, numel=n["x"]),
                           _ptr(w_router, "w_router", dt, numel=n["wr"]),
                           _ptr(b_router, "b_router", torch.float32, numel=n["E"]),
                           _ptr(topk_ids, "topk_ids", torch.int32, numel=n["Tk"]),
                           _ptr(topk_gates, "topk_gates", torch.float32, numel=n["Tk"]),
                           _ptr(logits, "logits", torch.float32, numel=n["TE"]),
                           _ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)), "moe_route")


def moe_dispatch(shape, topk_ids, topk_gates, expert_counts, expert_offsets, slot_of, row_token,
                 drop_mask, ws, x=None, x_routed=None, stream=None):
    """x and x_routed (optional, together): the token rows copied into slot order."""
    dt, n = _dtype_of(shape), _n(shape)
    _check(lib().moe_dispatch(ctypes.byref(shape),
                              _ptr(topk_ids, "topk_ids", torch.int32, numel=n["Tk"]),
                              _ptr(topk_gates, "topk_gates", torch.float32, numel=n["Tk"]),
                              _ptr(expert_counts, "expert_counts", torch.int32, numel=n["E"]),
                              _ptr(expert_offsets, "expert_offsets", torch.int32, numel=n["E1"]),
                              _ptr(slot_of, "slot_of", torch.int32, numel=n["Tk"]),
                              _ptr(row_token, "row_token", torch.int32, numel=n["rows"])
                              if row_token.numel() else None,
                              _ptr(drop_mask, "drop_mask", torch.uint8, numel=n["Tk"]),
                              _ptr(x, "x", dt, numel=n["x"]),
                              _ptr(x_routed, "x_routed", dt, numel=n["yrows"])
                              if x_routed is not None and x_routed.numel() else None,
                              _ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)),
           "moe_dispatch")


def moe_expert_ffn(shape, x, row_token, expert_offsets, w1, b1, w2, b2, y_rows, ws, stream=None):
    dt, n = _dtype_of(shape), _n(shape)
    f, d = n["f"], n["d"]
    _check(lib().moe_expert_ffn(ctypes.byref(shape), _ptr(x, "x", dt, numel=n["x"]),
                                _ptr(row_token, "row_token", torch.int32, numel=n["rows"])
                                if row_token.numel() else None,
                                _ptr(expert_offsets, "expert_offsets", torch.int32, numel=n["E1"]),
                                _ptr(w1, "w1", dt, numel=_w(shape, f, d)),
                                _ptr(b1, "b1", dt, numel=n["E"] * f),
                                _ptr(w2, "w2", dt, numel=_w(shape, d, f)),
                                _ptr(b2, "b2", dt, numel=n["E"] * d),
                                _ptr(y_rows, "y_rows", dt, numel=n["yrows"]) if y_rows.numel() else None,
                                _ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)),
           "moe_expert_ffn")


def moe_combine(shape, x, topk_gates, slot_of, y_rows, out, stream=None):
    dt, n = _dtype_of(shape), _n(shape)
    _check(lib().moe_combine(ctypes.byref(shape), _ptr(x, "x", dt, numel=n["x"]),
                             _ptr(topk_gates, "topk_gates", torch.float32, numel=n["Tk"]),
                             _ptr(slot_of, "slot_of", torch.int32, numel=n["Tk"]),
                             _ptr(y_rows, "y_rows", dt, numel=n["yrows"]) if y_rows.numel() else None,
                             _ptr(out, "out", dt, numel=n["x"]), _stream(stream)), "moe_combine")


def _forward_args(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids, topk_gates,
                  slot_of, drop_mask, expert_counts, ws, gated=False):
    dt, n = _dtype_of(shape), _n(shape)
    f, d, E = n["f"], n["d"], n["E"]
    return [ctypes.byref(shape), _ptr(x, "x", dt, numel=n["x"]),
            _ptr(w_router, "w_router", dt, numel=n["wr"]),
            _ptr(b_router, "b_router", torch.float32, numel=E),
            _ptr(w1, "w1", dt, numel=_w(shape, 2 * f if gated else f, d)),
            _ptr(b1, "b1", dt, numel=E * f), _ptr(w2, "w2", dt, numel=_w(shape, d, f)),
            _ptr(b2, "b2", dt, numel=E * d), _ptr(out, "out", dt, numel=n["x"]),
            _ptr(topk_ids, "topk_ids", torch.int32, numel=n["Tk"]),
            _ptr(topk_gates, "topk_gates", torch.float32, numel=n["Tk"]),
            _ptr(slot_of, "slot_of", torch.int32, numel=n["Tk"]),
            _ptr(drop_mask, "drop_mask", torch.uint8, numel=n["Tk"]),
            _ptr(expert_counts, "expert_counts", torch.int32, numel=E), _ptr(ws, "ws", torch.uint8),
            ws.numel() if ws is not None else 0]


def moe_layer_forward(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids=None,
                      topk_gates=None, slot_of=None, drop_mask=None, expert_counts=None, ws=None,
                      stream=None):
    args = _forward_args(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids, topk_gates,
                         slot_of, drop_mask, expert_counts, ws)
    _check(lib().moe_layer_forward(*args, _stream(stream)), "moe_layer_forward")


NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES


def moe_layer_forward_noalloc(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids=None,
                              topk_gates=None, slot_of=None, drop_mask=None, expert_counts=None,
                              stream=None):
    """moe_layer_forward with the library's fixed device scratch as its workspace (no
    allocation anywhere in the call)."""
    args = _forward_args(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids, topk_gates,
                         slot_of, drop_mask, expert_counts, None)
    _check(lib().moe_layer_forward_noalloc(*args[:-2], _stream(stream)),
           "moe_layer_forward_noalloc")


def moe_layer_forward_profiled(shape, x, w_router, b_router, w1, b1, w2, b2, out, events,
                               topk_ids=None, topk_gates=None, slot_of=None, drop_mask=None,
                               expert_counts=None, ws=None, stream=None):
    """`events`: 6 torch.cuda.Event(enable_timing=True) objects, already recorded once (so the
    underlying hipEvent_t exists)."""
    handles = (ctypes.c_void_p * 6)(*[ctypes.c_void_p(ev.cuda_event) for ev in events])
    args = _forward_args(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids, topk_gates,
                         slot_of, drop_mask, expert_counts, ws)
    _check(lib().moe_layer_forward_profiled(*args, _stream(stream), handles),
           "moe_layer_forward_profiled")


def moe_set_gemm_timing(events):
    """Arms kernel timing of the two expert GEMMs for the next layer or expert-FFN call on this
    thread: `events` are 4 torch.cuda.Event(enable_timing=True) objects (or None in place of
    one GEMM's pair), already recorded once (so the underlying hipEvent_t exists), receiving
    the up-projection's start and end and the down-projection's start and end; None
    disarms."""
    if events is None:
        _check(lib().moe_set_gemm_timing(None), "moe_set_gemm_timing")
        return
    handles = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(ev.cuda_event if ev is not None else None)
                                      for ev in events])
    _check(lib().moe_set_gemm_timing(handles), "moe_set_gemm_timing")


def moe_set_stage_timing(events):
    """Arms kernel timing of the router and the combine for the next layer call on this thread:
    `events` are 4 torch.cuda.Event(enable_timing=True) objects (or None in place of one
    kernel's pair), already recorded once, receiving the router kernel's start and end and the
    combine kernel's start and end; None disarms."""
    if events is None:
        _check(lib().moe_set_stage_timing(None), "moe_set_stage_timing")
        return
    handles = (ctypes.c_void_p * 4)(*[ctypes.c_void_p(ev.cuda_event if ev is not None else None)
                                      for ev in events])
    _check(lib().moe_set_stage_timing(handles), "moe_set_stage_timing")


def moe_layer_forward_padded(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids=None,
                             topk_gates=None, slot_of=None, drop_mask=None, expert_counts=None,
                             y_rows=None, ws=None, events=None, stream=None):
    """The padded fixed-buffer layout; `y_rows` [n_experts * capacity, d_model] optional;
    `events` None or 6 recorded torch.cuda.Event(enable_timing=True)."""
    dt = _dtype_of(shape)
    args = _forward_args(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids, topk_gates,
                         slot_of, drop_mask, expert_counts, ws)
    handles = None
    if events is not None:
        handles = (ctypes.c_void_p * 6)(*[ctypes.c_void_p(ev.cuda_event) for ev in events])
    y = (_ptr(y_rows, "y_rows", dt, numel=int(shape.n_experts) * int(shape.capacity) * int(shape.d_model))
         if y_rows is not None and y_rows.numel() else None)
    # the padded call takes y_rows before the workspace
    _check(lib().moe_layer_forward_padded(*args[:-2], y, args[-2], args[-1], _stream(stream),
                                          handles), "moe_layer_forward_padded")


def moe_layer_forward_gated(shape, x, w_router, b_router, w13, w2, out, topk_ids=None,
                            topk_gates=None, slot_of=None, drop_mask=None, expert_counts=None,
                            ws=None, events=None, stream=None):
    """Gated experts: w13 [E, 2 d_ff, d_model] (gate rows first), w2 [E, d_model, d_ff], no
    biases; bf16 only.  `events` None or 6 recorded torch.cuda.Event(enable_timing=True)."""
    handles = None
    if events is not None:
        handles = (ctypes.c_void_p * 6)(*[ctypes.c_void_p(ev.cuda_event) for ev in events])
    a = _forward_args(shape, x, w_router, b_router, w13, None, w2, None, out, topk_ids,
                      topk_gates, slot_of, drop_mask, expert_counts, ws, gated=True)
    # the gated call has no biases: shape, x, w_router, b_router, w13, w2, out, ...
    _check(lib().moe_layer_forward_gated(*a[:5], a[6], *a[8:], _stream(stream), handles),
           "moe_layer_forward_gated")


def _events(events, n=6):
    if events is None:
        return None
    if len(events) != n:
        raise ValueError(f"expected {n} events, got {len(events)}")
    return (ctypes.c_void_p * n)(*[ctypes.c_void_p(ev.cuda_event) for ev in events])


def moe_dispatch_pairs(shape, topk_ids, expert_counts, expert_offsets, sorted_pairs, row_token,
                       ws, stream=None):
    n = _n(shape)
    _check(lib().moe_dispatch_pairs(ctypes.byref(shape),
                                    _ptr(topk_ids, "topk_ids", torch.int32, numel=n["Tk"]),
                                    _ptr(expert_counts, "expert_counts", torch.int32, numel=n["E"]),
                                    _ptr(expert_offsets, "expert_offsets", torch.int32,
                                         numel=n["E1"]),
                                    _ptr(sorted_pairs, "sorted_pairs", torch.int32, numel=n["Tk"]),
                                    _ptr(row_token, "row_token", torch.int32, numel=n["Tk"]),
                                    _ptr(ws, "ws", torch.uint8), ws.numel(), _stream(stream)),
           "moe_dispatch_pairs")


def moe_expert_ffn_pairs(shape, x, sorted_pairs, row_token, expert_offsets, w1, b1, w2, b2,
                         topk_weights, pair_rows, ws, gated=False, stream=None):
    """gated: w1 is w13 [E, 2 d_ff, d_model] and b1, b2 are ignored (pass None)."""
    dt, n = _dtype_of(shape), _n(shape)
    f, d, E = n["f"], n["d"], n["E"]
    _check(lib().moe_expert_ffn_pairs(
        ctypes.byref(shape), _ptr(x, "x", dt, numel=n["x"]),
        _ptr(sorted_pairs, "sorted_pairs", torch.int32, numel=n["Tk"]),
        _ptr(row_token, "row_token", torch.int32, numel=n["Tk"]),
        _ptr(expert_offsets, "expert_offsets", torch.int32, numel=n["E1"]),
        _ptr(w1, "w1", dt, numel=_w(shape, 2 * f if gated else f, d)),
        _ptr(b1, "b1", dt, numel=E * f), _ptr(w2, "w2", dt, numel=_w(shape, d, f)),
        _ptr(b2, "b2", dt, numel=E * d),
        _ptr(topk_weights, "topk_weights", torch.float32, numel=n["Tk"]), int(bool(gated)),
        _ptr(pair_rows, "pair_rows", dt, numel=n["Tk"] * d), _ptr(ws, "ws", torch.uint8),
        ws.numel(), _stream(stream)), "moe_expert_ffn_pairs")


def moe_sum(shape, x, topk_ids, pair_rows, out, stream=None):
    """out[t] = (x[t] +) the sum of pair rows t*k .. t*k + k - 1; x and topk_ids may be None."""
    dt, n = _dtype_of(shape), _n(shape)
    _check(lib().moe_sum(ctypes.byref(shape), _ptr(x, "x", dt, numel=n["x"]),
                         _ptr(topk_ids, "topk_ids", torch.int32, numel=n["Tk"]),
                         _ptr(pair_rows, "pair_rows", dt, numel=n["Tk"] * n["d"]),
                         _ptr(out, "out", dt, numel=n["x"]), _stream(stream)), "moe_sum")


def _dropless_args(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids, topk_gates,
                   expert_counts, pair_rows, ws, gated):
    dt, n = _dtype_of(shape), _n(shape)
    f, d, E = n["f"], n["d"], n["E"]
    return [_ptr(x, "x", dt, numel=n["x"]), _ptr(w_router, "w_router", dt, numel=n["wr"]),
            _ptr(b_router, "b_router", torch.float32, numel=E),
            _ptr(w1, "w1", dt, numel=_w(shape, 2 * f if gated else f, d)),
            _ptr(b1, "b1", dt, numel=E * f), _ptr(w2, "w2", dt, numel=_w(shape, d, f)),
            _ptr(b2, "b2", dt, numel=E * d), _ptr(out, "out", dt, numel=n["x"]),
            _ptr(topk_ids, "topk_ids", torch.int32, numel=n["Tk"]),
            _ptr(topk_gates, "topk_gates", torch.float32, numel=n["Tk"]),
            _ptr(expert_counts, "expert_counts", torch.int32, numel=E),
            _ptr(pair_rows, "pair_rows", dt, numel=n["Tk"] * d), _ptr(ws, "ws", torch.uint8),
            ws.numel()]


def moe_layer_forward_dropless(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids=None,
                               topk_gates=None, expert_counts=None, pair_rows=None, ws=None,
                               events=None, stream=None):
    """Dropless pair-order layer; `pair_rows` [T * k, d_model] optional; `events` None or 6
    recorded torch.cuda.Event(enable_timing=True)."""
    a = _dropless_args(shape, x, w_router, b_router, w1, b1, w2, b2, out, topk_ids, topk_gates,
                       expert_counts, pair_rows, ws, False)
    _check(lib().moe_layer_forward_dropless(ctypes.byref(shape), *a, _stream(stream),
                                            _events(events)), "moe_layer_forward_dropless")


def moe_layer_forward_dropless_gated(shape, x, w_router, b_router, w13, w2, out, topk_ids=None,
                                     topk_gates=None, expert_counts=None, pair_rows=None,
                                     ws=None, events=None, stream=None):
    a = _dropless_args(shape, x, w_router, b_router, w13, None, w2, None, out, topk_ids,
                       topk_gates, expert_counts, pair_rows, ws, True)
    # no biases: x, w_router, b_router, w13, w2, out, ...
    _check(lib().moe_layer_forward_dropless_gated(ctypes.byref(shape), *a[:4], a[5], *a[7:],
                                                  _stream(stream), _events(events)),
           "moe_layer_forward_dropless_gated")


def workspace_bytes_batches(batch_shape: MoeShape, n_batches: int) -> int:
    return int(lib().moe_workspace_bytes_batches(ctypes.byref(batch_shape), int(n_batches)))


def moe_schedule_batches(batch_shape, n_batches, topk_ids, order, batch_experts=None,
                         orig_batch_experts=None, stream=None):
    Tp = int(batch_shape.T) * int(n_batches)
    _check(lib().moe_schedule_batches(
        ctypes.byref(batch_shape), int(n_batches),
        _ptr(topk_ids, "topk_ids", torch.int32, numel=Tp * int(batch_shape.top_k)),
        _ptr(order, "order", torch.int32, numel=Tp),
        _ptr(batch_experts, "batch_experts", torch.int32, numel=int(n_batches)),
        _ptr(orig_batch_experts, "orig_batch_experts", torch.int32, numel=int(n_batches)),
        _stream(stream)), "moe_schedule_batches")


def moe_layer_forward_batches(batch_shape, n_batches, consolidate, x, w_router, b_router, w1, b1,
                              w2, b2, out, topk_ids=None, topk_gates=None, order=None,
                              batch_experts=None, ws=None, events=None, stream=None):
    """A pool of n_batches batches of batch_shape.T tokens, one batch after another, regrouped
    by the Token Scheduler when `consolidate`; `events` None or 5 recorded
    torch.cuda.Event(enable_timing=True)."""
    dt, n = _dtype_of(batch_shape), _n(batch_shape)
    M = int(n_batches)
    Tp = n["T"] * M
    f, d, E = n["f"], n["d"], n["E"]
    _check(lib().moe_layer_forward_batches(
        ctypes.byref(batch_shape), M, int(bool(consolidate)), _ptr(x, "x", dt, numel=Tp * d),
        _ptr(w_router, "w_router", dt, numel=n["wr"]),
        _ptr(b_router, "b_router", torch.float32, numel=E),
        _ptr(w1, "w1", dt, numel=_w(batch_shape, f, d)), _ptr(b1, "b1", dt, numel=E * f),
        _ptr(w2, "w2", dt, numel=_w(batch_shape, d, f)), _ptr(b2, "b2", dt, numel=E * d),
        _ptr(out, "out", dt, numel=Tp * d),
        _ptr(topk_ids, "topk_ids", torch.int32, numel=Tp * n["k"]),
        _ptr(topk_gates, "topk_gates", torch.float32, numel=Tp * n["k"]),
        _ptr(order, "order", torch.int32, numel=Tp),
        _ptr(batch_experts, "batch_experts", torch.int32, numel=M), _ptr(ws, "ws", torch.uint8),
        ws.numel(), _stream(stream), _events(events, 5)), "moe_layer_forward_batches")


def packed_weights_bytes(shape: MoeShape, rows: int, cols: int) -> int:
    return int(lib().moe_packed_weights_bytes(ctypes.byref(shape), int(rows), int(cols)))


def moe_pack_weights(shape, w, w_packed, stream=None):
    """w [E, rows, cols] bf16 -> w_packed (at least moe_packed_weights_bytes bytes)."""
    E, rows, cols = w.shape
    if w_packed.numel() * w_packed.element_size() < packed_weights_bytes(shape, rows, cols):
        raise ValueError("w_packed is too small")
    _check(lib().moe_pack_weights(ctypes.byref(shape), _ptr(w, "w", torch.bfloat16), int(rows),
                                  int(cols), _ptr(w_packed, "w_packed"), _stream(stream)),
           "moe_pack_weights")


_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device() -> int:
    """The current device (-1 without one): looked up once a call."""
    try:
        return _get_device()
    except (RuntimeError, AssertionError):
        return -1


def _cur(dev: int, t, name: str, dtype=None, numel: int = 0):
    """_ptr, and the tensor has to be on device `dev`, the current one (whose stream the call
    takes).  Everything is looked at once; only a tensor that something is wrong with takes the
    long way."""
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and (dtype is None or t.dtype is dtype) and
            t.get_device() == dev and t.numel() >= numel and t.is_contiguous() and dev >= 0):
        return t.data_ptr()
    _ptr(t, name, dtype, numel=numel)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def workspace_bytes_balance(shape: MoeShape) -> int:
    return int(lib().moe_workspace_bytes_balance(ctypes.byref(shape)))


def workspace_bytes_route_backward(shape: MoeShape) -> int:
    return int(lib().moe_workspace_bytes_route_backward(ctypes.byref(shape)))


def moe_balance_loss(shape, logits, topk_ids, loss, expert_counts=None, expert_probs=None,
                     dlogits=None, token_mask=None, coef=1.0, grad_scale=1.0, ws=None,
                     stream=None):
    """Balance loss [1] and, where given, the counts [E], mean probabilities [E] and gradient on
    the logits [T, E]; token_mask [T] uint8, 0 for padding."""
    T, E, k = shape.T, shape.n_experts, shape.top_k
    dev = _device()
    _check(lib().moe_balance_loss(
        ctypes.byref(shape), _cur(dev, logits, "logits", torch.float32, numel=T * E),
        _cur(dev, topk_ids, "topk_ids", torch.int32, numel=T * k),
        _cur(dev, token_mask, "token_mask", torch.uint8, numel=T), float(coef), float(grad_scale),
        _cur(dev, loss, "loss", torch.float32, numel=1),
        _cur(dev, expert_counts, "expert_counts", torch.int32, numel=E),
        _cur(dev, expert_probs, "expert_probs", torch.float32, numel=E),
        _cur(dev, dlogits, "dlogits", torch.float32, numel=T * E), _cur(dev, ws, "ws", torch.uint8),
        ws.numel() if ws is not None else 0, _stream(stream)), "moe_balance_loss")


def moe_route_backward(shape, x, w_router, logits, topk_ids, dgates, dlogits, dx=None,
                       dw_router=None, db_router=None, dx_add=None, token_mask=None, ws=None,
                       stream=None):
    """Gradients of the router: dx [T, d] in the shape's dtype, dw_router [E, d] and db_router [E]
    in fp32, each optional; dgates [T, k] or dlogits [T, E] (or both) come in."""
    dt, f32 = _dtype_of(shape), torch.float32
    T, d, E, k = shape.T, shape.d_model, shape.n_experts, shape.top_k
    dev = _device()
    _check(lib().moe_route_backward(
        ctypes.byref(shape), _cur(dev, x, "x", dt, numel=T * d),
        _cur(dev, w_router, "w_router", dt, numel=E * d), _cur(dev, logits, "logits", f32, numel=T * E),
        _cur(dev, topk_ids, "topk_ids", torch.int32, numel=T * k),
        _cur(dev, dgates, "dgates", f32, numel=T * k), _cur(dev, dlogits, "dlogits", f32, numel=T * E),
        _cur(dev, token_mask, "token_mask", torch.uint8, numel=T),
        _cur(dev, dx_add, "dx_add", dt, numel=T * d), _cur(dev, dx, "dx", dt, numel=T * d),
        _cur(dev, dw_router, "dw_router", f32, numel=E * d),
        _cur(dev, db_router, "db_router", f32, numel=E), _cur(dev, ws, "ws", torch.uint8),
        ws.numel() if ws is not None else 0, _stream(stream)), "moe_route_backward")


def quantized_codes_bytes(shape: MoeShape, rows: int, cols: int) -> int:
    return int(lib().moe_quantized_codes_bytes(ctypes.byref(shape), int(rows), int(cols)))


def quantized_scales_bytes(shape: MoeShape, rows: int, cols: int, group: int) -> int:
    return int(lib().moe_quantized_scales_bytes(ctypes.byref(shape), int(rows), int(cols),
                                                int(group)))


def moe_quantize_weights(shape, w, group, codes, scales, stream=None):
    """w [E, rows, cols] in the shape's dtype -> codes (uint8) and scales (bf16)."""
    E, rows, cols = w.shape
    if E != shape.n_experts:
        raise ValueError(f"w has {E} experts, the shape {shape.n_experts}")
    dev = _device()
    _check(lib().moe_quantize_weights(
        ctypes.byref(shape), _cur(dev, w, "w", _dtype_of(shape)), int(rows), int(cols), int(group),
        _cur(dev, codes, "codes", torch.uint8, numel=quantized_codes_bytes(shape, rows, cols)),
        _cur(dev, scales, "scales", torch.bfloat16,
             numel=quantized_scales_bytes(shape, rows, cols, group) // 2), _stream(stream)),
        "moe_quantize_weights")


def moe_dequantize_weights(shape, codes, scales, group, w, stream=None):
    """The values of codes and scales -> w [E, rows, cols] fp32."""
    E, rows, cols = w.shape
    if E != shape.n_experts:
        raise ValueError(f"w has {E} experts, the shape {shape.n_experts}")
    dev = _device()
    _check(lib().moe_dequantize_weights(
        ctypes.byref(shape),
        _cur(dev, codes, "codes", torch.uint8, numel=quantized_codes_bytes(shape, rows, cols)),
        _cur(dev, scales, "scales", torch.bfloat16,
             numel=quantized_scales_bytes(shape, rows, cols, group) // 2),
        int(rows), int(cols), int(group), _cur(dev, w, "w", torch.float32), _stream(stream)),
        "moe_dequantize_weights")


class QuantizedExperts:
    """The 4-bit experts of one layer: the tensors of moe_quantized_experts, checked once against
    the layer's E, d_model and d_ff."""

    def __init__(self, E, d_model, d_ff, group, gated, w1_codes, w1_scales, b1, w2_codes,
                 w2_scales, b2):
        self.E, self.d_model, self.d_ff = int(E), int(d_model), int(d_ff)
        self.group, self.gated = int(group), bool(gated)
        shape = make_shape(0, d_model, d_ff, E, 1, 0, MOE_BF16)
        rows1 = (2 if gated else 1) * self.d_ff
        u8, bf = torch.uint8, torch.bfloat16
        sizes = {n: quantized_codes_bytes(shape, r, c)
                 for n, r, c in (("w1", rows1, d_model), ("w2", d_model, d_ff))}
        scales = {n: quantized_scales_bytes(shape, r, c, group) // 2
                  for n, r, c in (("w1", rows1, d_model), ("w2", d_model, d_ff))}
        if not sizes["w1"] or not sizes["w2"] or not scales["w1"]:
            raise MoeError(2, "QuantizedExperts", last_error())
        if gated and (b1 is not None or b2 is not None):
            raise ValueError("gated experts have no biases")
        self.tensors = (w1_codes, w1_scales, b1, w2_codes, w2_scales, b2)
        if len({t.device for t in self.tensors if t is not None}) > 1:
            raise ValueError("the experts' tensors are on different devices")
        self.struct = MoeQuantizedExperts(
            _ptr(w1_codes, "w1_codes", u8, numel=sizes["w1"]),
            _ptr(w1_scales, "w1_scales", bf, numel=scales["w1"]),
            _ptr(b1, "b1", bf, numel=self.E * self.d_ff),
            _ptr(w2_codes, "w2_codes", u8, numel=sizes["w2"]),
            _ptr(w2_scales, "w2_scales", bf, numel=scales["w2"]),
            _ptr(b2, "b2", bf, numel=self.E * self.d_model), self.group, int(self.gated))

    def of(self, shape):
        """The struct, for a call of this shape on the current device."""
        if (shape.n_experts, shape.d_model, shape.d_ff) != (self.E, self.d_model, self.d_ff):
            raise ValueError(f"experts of E {self.E}, d_model {self.d_model}, d_ff {self.d_ff}; the "
                             f"shape has {shape.n_experts}, {shape.d_model}, {shape.d_ff}")
        if self.tensors[0].get_device() != _device():
            raise ValueError(f"experts are on {self.tensors[0].device}, the current device is "
                             f"cuda:{_device()}")
        return ctypes.byref(self.struct)


def moe_expert_ffn_quantized(shape, x, row_token, expert_offsets, experts, y_rows, ws,
                             stream=None):
    """moe_expert_ffn with QuantizedExperts."""
    dt, T, d = _dtype_of(shape), shape.T, shape.d_model
    rows = min(T * shape.top_k, shape.n_experts * shape.capacity)  # moe_max_kept_rows
    dev = _device()
    _check(lib().moe_expert_ffn_quantized(
        ctypes.byref(shape), _cur(dev, x, "x", dt, T * d),
        _cur(dev, row_token, "row_token", torch.int32, rows) if row_token.numel() else None,
        _cur(dev, expert_offsets, "expert_offsets", torch.int32, shape.n_experts + 1),
        experts.of(shape), _cur(dev, y_rows, "y_rows", dt, rows * d) if y_rows.numel() else None,
        _cur(dev, ws, "ws", torch.uint8), ws.numel(), _stream(stream)), "moe_expert_ffn_quantized")


def moe_layer_forward_quantized(shape, x, w_router, b_router, experts, out, topk_ids=None,
                                topk_gates=None, slot_of=None, drop_mask=None,
                                expert_counts=None, ws=None, events=None, stream=None):
    """moe_layer_forward (or _gated) with QuantizedExperts; `events` None or 6 recorded
    torch.cuda.Event(enable_timing=True)."""
    dt, n = _dtype_of(shape), _n(shape)
    i32 = torch.int32
    dev = _device()
    _check(lib().moe_layer_forward_quantized(
        ctypes.byref(shape), _cur(dev, x, "x", dt, numel=n["x"]),
        _cur(dev, w_router, "w_router", dt, numel=n["wr"]),
        _cur(dev, b_router, "b_router", torch.float32, numel=n["E"]), experts.of(shape),
        _cur(dev, out, "out", dt, numel=n["x"]), _cur(dev, topk_ids, "topk_ids", i32, numel=n["Tk"]),
        _cur(dev, topk_gates, "topk_gates", torch.float32, numel=n["Tk"]),
        _cur(dev, slot_of, "slot_of", i32, numel=n["Tk"]),
        _cur(dev, drop_mask, "drop_mask", torch.uint8, numel=n["Tk"]),
        _cur(dev, expert_counts, "expert_counts", i32, numel=n["E"]), _cur(dev, ws, "ws", torch.uint8),
        ws.numel() if ws is not None else 0, _stream(stream), _events(events)),
        "moe_layer_forward_quantized")


# ---------------------------------------------------------------- routing by scores
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP_TWO = 0, 1
_SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
_GROUP_SCORES = {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP_TWO}


def make_routing(score: str = "softmax", n_groups: int = 1, topk_groups: int = 1,
                 group_score: str = "max", renormalize: bool = False,
                 scale: float = 1.0) -> MoeRouting:
    """How experts are chosen and gates formed (moe_routing)."""
    if score not in _SCORES:
        raise ValueError(f"score {score!r} is not one of {sorted(_SCORES)}")
    if group_score not in _GROUP_SCORES:
        raise ValueError(f"group_score {group_score!r} is not one of {sorted(_GROUP_SCORES)}")
    return MoeRouting(_SCORES[score], int(n_groups), int(topk_groups), _GROUP_SCORES[group_score],
                      int(bool(renormalize)), float(scale))


def workspace_bytes_route_scored(shape: MoeShape) -> int:
    return int(lib().moe_workspace_bytes_route_scored(ctypes.byref(shape)))


def moe_route_scored(shape, routing, x, w_router, b_router, score_bias, topk_ids, topk_gates,
                     logits=None, token_mask=None, ws=None, stream=None):
    """moe_route with the scores, bias, groups and gates of `routing`; b_router, score_bias [E] and
    token_mask [T] uint8 may be None."""
    dt, f32 = _dtype_of(shape), torch.float32
    T, d, E, k = shape.T, shape.d_model, shape.n_experts, shape.top_k
    dev = _device()
    _check(lib().moe_route_scored(
        ctypes.byref(shape), ctypes.byref(routing), _cur(dev, x, "x", dt, numel=T * d),
        _cur(dev, w_router, "w_router", dt, numel=E * d),
        _cur(dev, b_router, "b_router", f32, numel=E),
        _cur(dev, score_bias, "score_bias", f32, numel=E),
        _cur(dev, token_mask, "token_mask", torch.uint8, numel=T),
        _cur(dev, topk_ids, "topk_ids", torch.int32, numel=T * k),
        _cur(dev, topk_gates, "topk_gates", f32, numel=T * k),
        _cur(dev, logits, "logits", f32, numel=T * E), _cur(dev, ws, "ws", torch.uint8),
        ws.numel() if ws is not None else 0, _stream(stream, dev)), "moe_route_scored")


def moe_route_scored_backward(shape, routing, logits, topk_ids, dgates, dlogits, dlogits_add=None,
                              token_mask=None, stream=None):
    """dlogits [T, E] (+ dlogits_add, which may be dlogits) from the gradient dgates [T, k]."""
    f32 = torch.float32
    T, E, k = shape.T, shape.n_experts, shape.top_k
    dev = _device()
    _check(lib().moe_route_scored_backward(
        ctypes.byref(shape), ctypes.byref(routing), _cur(dev, logits, "logits", f32, numel=T * E),
        _cur(dev, topk_ids, "topk_ids", torch.int32, numel=T * k),
        _cur(dev, dgates, "dgates", f32, numel=T * k),
        _cur(dev, dlogits_add, "dlogits_add", f32, numel=T * E),
        _cur(dev, token_mask, "token_mask", torch.uint8, numel=T),
        _cur(dev, dlogits, "dlogits", f32, numel=T * E), _stream(stream, dev)),
        "moe_route_scored_backward")


def moe_combine_backward(shape, dout, topk_gates, slot_of, y_rows, dgates=None, dy_rows=None,
                         stream=None):
    """Gradients of moe_combine: dgates [T, k] fp32 (needs y_rows) and dy_rows (needs topk_gates),
    each optional.  slot_of in either layout: y_rows and dy_rows hold moe_max_kept_rows rows, or the
    padded layout's n_experts * capacity; a slot past what they hold counts as dropped."""
    dt, T, d, k = _dtype_of(shape), shape.T, shape.d_model, shape.top_k
    n, padded = T * k, shape.n_experts * shape.capacity
    rows, most = (n, padded) if n < padded else (padded, n)  # moe_max_kept_rows, and of any layout
    dev = _device()
    y, dy = _cur(dev, y_rows, "y_rows", dt, rows * d), _cur(dev, dy_rows, "dy_rows", dt, rows * d)
    if y is not None and dgates is not None:
        rows = min(most, y_rows.numel() // d, 0x7FFFFFFF)
        if dy is not None:
            rows = min(rows, dy_rows.numel() // d)
    elif dy is not None:
        rows = min(most, dy_rows.numel() // d, 0x7FFFFFFF)
    _check(lib().moe_combine_backward_rows(
        ctypes.byref(shape), _cur(dev, dout, "dout", dt, T * d),
        _cur(dev, topk_gates, "topk_gates", torch.float32, n),
        _cur(dev, slot_of, "slot_of", torch.int32, n), y, rows,
        _cur(dev, dgates, "dgates", torch.float32, n), dy, _stream(stream, dev)),
        "moe_combine_backward")


def workspace_bytes_balance_bias(shape: MoeShape) -> int:
    return int(lib().moe_workspace_bytes_balance_bias(ctypes.byref(shape)))


def moe_balance_bias(shape, rate, score_bias, expert_counts=None, topk_ids=None, token_mask=None,
                     ws=None, stream=None):
    """score_bias [E] moved by `rate` towards even counts, in place: the counts of topk_ids (written
    to expert_counts where given), or expert_counts where topk_ids is None."""
    T, E, k = shape.T, shape.n_experts, shape.top_k
    dev = _device()
    bias = _cur(dev, score_bias, "score_bias", torch.float32, numel=E)
    ids = _cur(dev, topk_ids, "topk_ids", torch.int32, numel=T * k)
    if topk_ids is not None and T == 0:
        ids = bias  # an empty tensor has no address, and None would mean given counts; never read
    _check(lib().moe_balance_bias(
        ctypes.byref(shape), ids, _cur(dev, token_mask, "token_mask", torch.uint8, numel=T),
        float(rate), bias, _cur(dev, expert_counts, "expert_counts", torch.int32, numel=E),
        _cur(dev, ws, "ws", torch.uint8), ws.numel() if ws is not None else 0, _stream(stream, dev)),
        "moe_balance_bias")


# ---------------------------------------------------------------- AdamW
class AdamWTensors:
    """The tensors of one optimiser: lists of params, grads and moments (any shapes; entry i of every
    list has the elements of params[i], all contiguous and on one device), checked once.  m and v are
    fp32, or int8 and uint8 with m_steps and v_steps ([ceil(n / 256)] fp32 each); copies, bf16, are
    written after each step; weight_decay is a number or one per tensor.  Their addresses are taken
    here and in set_grads: a tensor whose storage is exchanged afterwards (`t.data = ...`) has to be
    handed over again.  grads may be None until set_grads: moe_adamw_moments needs none."""

    def __init__(self, params, grads, m, v, m_steps=None, v_steps=None, copies=None,
                 weight_decay=0.0):
        n = len(params)
        quantized = m_steps is not None or v_steps is not None
        decay = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        lists = {"params": params, "m": m, "v": v, "weight_decay": decay}
        if grads is not None:
            lists["grads"] = grads
        for name, x in (("m_steps", m_steps), ("v_steps", v_steps)):
            if quantized:
                lists[name] = x
        if copies is not None:
            lists["copies"] = copies
        for name, x in lists.items():
            if x is None or len(x) != n:
                raise ValueError(f"{name} has {0 if x is None else len(x)} entries, params {n}")
        self.device = params[0].device if n else None
        self.bits = 8 if quantized else 32
        self.param_dtype = self._one_dtype(params, "params")
        self.params, self.m, self.v = list(params), list(m), list(v)
        self.others = [list(x) for x in (m_steps, v_steps, copies) if x is not None]  # kept alive
        self.array = (MoeAdamWTensor * max(n, 1))()
        self.n = n
        f32 = torch.float32
        sdt = (torch.int8, torch.uint8) if quantized else (f32, f32)
        for i in range(n):
            a, k = self.array[i], params[i].numel()
            a.param = self._at(params[i], f"params[{i}]", self.param_dtype, k)
            a.m = self._at(m[i], f"m[{i}]", sdt[0], k)
            a.v = self._at(v[i], f"v[{i}]", sdt[1], k)
            if quantized:
                a.m_steps = self._at(m_steps[i], f"m_steps[{i}]", f32, (k + 255) // 256)
                a.v_steps = self._at(v_steps[i], f"v_steps[{i}]", f32, (k + 255) // 256)
            if copies is not None and copies[i] is not None:
                a.copy = self._at(copies[i], f"copies[{i}]", torch.bfloat16, k)
            a.n = k
            a.weight_decay = float(decay[i])
        self.grads, self.grad_dtype = None, f32
        if grads is not None:
            self.set_grads(grads)

    def _one_dtype(self, tensors, name):
        kinds = {t.dtype for t in tensors}
        if len(kinds) > 1 or not kinds <= {torch.float32, torch.bfloat16}:
            raise TypeError(f"{name}: one dtype, float32 or bfloat16, not {sorted(map(str, kinds))}")
        return kinds.pop() if kinds else torch.float32

    def _at(self, t, name, dtype, numel):
        p = _ptr(t, name, dtype, self.device, numel)
        if t.numel() != numel:
            raise ValueError(f"{name} holds {t.numel()} elements, {numel} are expected")
        return p

    def set_grads(self, grads):
        """Other gradients for the steps to come; checks that all tensors are apart.  Those that are
        refused leave the list as it was."""
        if len(grads) != self.n:
            raise ValueError(f"grads has {len(grads)} entries, params {self.n}")
        dtype = self._one_dtype(grads, "grads")
        at = [self._at(g, f"grads[{i}]", dtype, self.params[i].numel()) for i, g in enumerate(grads)]
        old = self.grads, self.grad_dtype, [a.grad for a in self.array]
        self.grads, self.grad_dtype = list(grads), dtype
        for a, p in zip(self.array, at):
            a.grad = p
        c = self.config(0.0, 0.0, 0.0, 1.0, 1, 1.0, None)
        try:
            _check(lib().moe_adamw_check(ctypes.byref(c), self.array, self.n), "moe_adamw_check")
        except MoeError:
            self.grads, self.grad_dtype = old[:2]
            for a, p in zip(self.array, old[2]):
                a.grad = p
            raise

    def config(self, lr, beta1, beta2, eps, step, grad_scale, dynamic):
        code = lambda t: MOE_BF16 if t is torch.bfloat16 else MOE_F32
        return MoeAdamWConfig(code(self.param_dtype), code(self.grad_dtype), self.bits, lr, beta1,
                              beta2, eps, grad_scale, step, dynamic)

    def on(self, dev):
        if self.n and self.device.index != dev:
            raise ValueError(f"the tensors are on {self.device}, the current device is cuda:{dev}")


def moe_adamw_step(tensors: AdamWTensors, lr, beta1, beta2, eps, step, grad_scale=1.0, dynamic=None,
                   stream=None):
    """One AdamW step of all tensors; `step` counts from 1.  dynamic [4] fp32 on the device (lr,
    grad_scale, step, skip) takes the place of lr, grad_scale and step."""
    dev = _device()
    tensors.on(dev)
    c = tensors.config(lr, beta1, beta2, eps, step, grad_scale,
                       _cur(dev, dynamic, "dynamic", torch.float32, numel=4))
    _check(lib().moe_adamw_step(ctypes.byref(c), tensors.array, tensors.n, _stream(stream, dev)),
           "moe_adamw_step")


def moe_adamw_moments(tensors: AdamWTensors, m_out=None, v_out=None, stream=None):
    """The fp32 moments [n] each of all tensors: lists of outputs (or None, or None entries)."""
    dev = _device()
    tensors.on(dev)
    outs = []
    for name, x in (("m_out", m_out), ("v_out", v_out)):
        if x is not None and len(x) != tensors.n:
            raise ValueError(f"{name} has {len(x)} entries, the optimiser {tensors.n}")
        outs.append(x if x is None else (ctypes.c_void_p * max(tensors.n, 1))(*[
            None if t is None else tensors._at(t, f"{name}[{i}]", torch.float32,
                                               tensors.params[i].numel())
            for i, t in enumerate(x)]))
    c = tensors.config(0.0, 0.0, 0.0, 1.0, 1, 1.0, None)
    _check(lib().moe_adamw_moments(ctypes.byref(c), tensors.array, tensors.n, *outs,
                                   _stream(stream, dev)), "moe_adamw_moments")
