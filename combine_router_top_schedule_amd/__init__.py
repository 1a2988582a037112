"""Python binding of libmok, the MI355X (gfx950) deterministic fused MoE layer.

Argument marshalling only: every step of the layer runs in the HIP kernels of libmok.so. The
functions keep the C names (``mok_schedule``, ``mok_dispatch``, ``mok_expert_ffn``,
``mok_combine``, ``mok_layer_fwd``, ``mok_layer_bwd``, ``mok_quantize_mx``) and take torch
tensors for device buffers; torch is used for device memory and the current stream only.

The library is built in place by ``combine_router_top_schedule_amd.build`` (``__graft_entry__``
calls it). Importing this package without the built library raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmok.so")

MOK_BF16, MOK_MXFP8 = 0, 1
MOK_FLAG_SKIP_ONE_SIGNAL = 0x1
MOK_FLAG_TRACE = 0x2
MOK_FLAG_POISON = 0x4
STATUS = {0: "MOK_OK", 1: "MOK_ERR_NULL", 2: "MOK_ERR_SHAPE", 3: "MOK_ERR_DTYPE",
          4: "MOK_ERR_ALIGN", 5: "MOK_ERR_WORKSPACE", 6: "MOK_ERR_RING", 7: "MOK_ERR_HIP",
          8: "MOK_ERR_DEVICE_TIMEOUT", 9: "MOK_ERR_UNSUPPORTED", 10: "MOK_ERR_SCRATCH"}
MOK_SCRATCH_BYTES = 1 << 20


class MokDesc(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("intermediate", ctypes.c_int32),
                ("num_segments", ctypes.c_int32), ("tokens_per_segment", ctypes.c_int32),
                ("expert_begin", ctypes.c_int32), ("num_local_experts", ctypes.c_int32),
                ("minibatch_tokens", ctypes.c_int32), ("comm_cus", ctypes.c_int32),
                ("ring_bytes", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_uint32)]


class MokSizes(ctypes.Structure):
    _fields_ = [("saved_bytes", ctypes.c_size_t), ("ws_bytes", ctypes.c_size_t),
                ("bwd_ws_bytes", ctypes.c_size_t),
                ("slots_bytes", ctypes.c_size_t), ("xd_bytes", ctypes.c_size_t),
                ("act_bytes", ctypes.c_size_t), ("wq_bytes", ctypes.c_size_t),
                ("rows_max", ctypes.c_int64), ("ring_slots", ctypes.c_int32),
                ("minibatch", ctypes.c_int32), ("slot_bytes", ctypes.c_int64),
                ("perm_offset", ctypes.c_int64), ("tokpos_offset", ctypes.c_int64),
                ("touched_offset", ctypes.c_int64), ("x_slot_bytes", ctypes.c_int64),
                ("ring_min_bytes", ctypes.c_int64), ("tiles_offset", ctypes.c_int64),
                ("tiles_max", ctypes.c_int64), ("trace_offset", ctypes.c_int64),
                ("trace_records", ctypes.c_int64), ("h_slot_bytes", ctypes.c_int64),
                ("packed_bytes", ctypes.c_int64)]


_P = ctypes.c_void_p

MOK_ELEM_F32, MOK_ELEM_BF16 = 0, 1
MOK_SCORE_SOFTMAX, MOK_SCORE_SIGMOID = 0, 1
MOK_GROUP_MAX, MOK_GROUP_TOP2 = 0, 1
MOK_STATE_F32, MOK_STATE_MX8 = 0, 1
MOK_ADJUST_RMS, MOK_ADJUST_SPECTRAL, MOK_ADJUST_NONE = 0, 1, 2
MOK_BLOCK_FEW_ROWS, MOK_BLOCK_TILES_128, MOK_BLOCK_TILES_256 = 0, 1, 2


class MokRouteDesc(ctypes.Structure):
    _fields_ = [("num_tokens", ctypes.c_int64), ("logits_stride", ctypes.c_int64),
                ("num_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("score", ctypes.c_int32), ("num_groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_score", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("elem", ctypes.c_int32), ("scale", ctypes.c_float)]


class MokSumsqTensor(ctypes.Structure):
    _fields_ = [("g", _P), ("n", ctypes.c_int64)]


class MokAdamwTensor(ctypes.Structure):
    _fields_ = [("p", _P), ("copy", _P), ("g", _P), ("m", _P), ("v", _P), ("m_scale", _P),
                ("v_scale", _P), ("n", ctypes.c_int64)]


class MokAdamwConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("max_norm", ctypes.c_double), ("step", ctypes.c_int64), ("seed", ctypes.c_uint32),
                ("grad_elem", ctypes.c_int32), ("param_elem", ctypes.c_int32),
                ("state", ctypes.c_int32), ("sumsq_dev", _P), ("lr_dev", _P), ("step_dev", _P)]


class MokNewtonSchulz(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_double), ("steps", ctypes.c_int32), ("coefficients", ctypes.c_float * 48)]


class MokMuonTensor(ctypes.Structure):
    _fields_ = [("p", _P), ("copy", _P), ("g", _P), ("m", _P), ("batch", ctypes.c_int32),
                ("rows", ctypes.c_int32), ("cols", ctypes.c_int32)]


class MokMuonConfig(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("momentum", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("max_norm", ctypes.c_double), ("nesterov", ctypes.c_int32), ("adjust", ctypes.c_int32),
                ("grad_elem", ctypes.c_int32), ("ns", MokNewtonSchulz), ("sumsq_dev", _P), ("lr_dev", _P)]


class MokOrthogonalizeTensor(ctypes.Structure):
    _fields_ = [("src", _P), ("out", _P), ("batch", ctypes.c_int32), ("rows", ctypes.c_int32),
                ("cols", ctypes.c_int32)]


class MokBlockDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("stride", ctypes.c_int64), ("groups", ctypes.c_int32),
                ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("elem", ctypes.c_int32)]


class MokWeights(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("wg", "wu", "wd", "wg_q", "wg_s", "wu_q", "wu_s", "wd_q",
                                  "wd_s", "wgt_q", "wgt_s", "wut_q", "wut_s", "wdt_q", "wdt_s",
                                  "packed")]


class MokTuneResult(ctypes.Structure):
    _fields_ = [("minibatch_tokens", ctypes.c_int32), ("comm_cus", ctypes.c_int32),
                ("ms", ctypes.c_float)]


class MokWeightGrads(ctypes.Structure):
    _fields_ = [("dwg", _P), ("dwu", _P), ("dwd", _P)]


# name -> (restype, argtypes); mirrors include/mok.h
_SIGS = {
    "mok_abi_version": (ctypes.c_int, []),
    "mok_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "mok_query_sizes": (ctypes.c_int, [ctypes.POINTER(MokDesc), ctypes.POINTER(MokSizes)]),
    "mok_workspace_size": (ctypes.c_int, [ctypes.POINTER(MokDesc), ctypes.POINTER(ctypes.c_size_t),
                                          ctypes.POINTER(ctypes.c_size_t),
                                          ctypes.POINTER(ctypes.c_size_t)]),
    "mok_two_wave_floor": (ctypes.c_int64, [ctypes.c_int32] * 4),
    "mok_schedule": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, _P, _P, _P, _P]),
    "mok_schedule_routed": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, _P, _P, _P]),
    "mok_layer_fwd_routed": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, ctypes.POINTER(MokWeights), _P,
                                            _P, _P, _P, _P, _P, _P, _P]),
    "mok_schedule_noalloc": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, _P, _P, _P]),
    "mok_router_fwd": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, _P, _P]),
    "mok_router_ws_size": (ctypes.c_int, [ctypes.POINTER(MokDesc), ctypes.POINTER(ctypes.c_size_t)]),
    "mok_router_bwd": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, _P, _P, _P, _P, _P]),
    "mok_dispatch": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, _P, _P, _P]),
    "mok_expert_ffn": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, ctypes.POINTER(MokWeights),
                                      _P, _P, _P, _P]),
    "mok_combine": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, _P, _P, _P, _P, _P]),
    "mok_layer_fwd": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, ctypes.POINTER(MokWeights),
                                     _P, _P, _P, _P, _P, _P, _P, _P]),
    "mok_macro_ws_size": (ctypes.c_int, [ctypes.POINTER(MokDesc), ctypes.c_int32,
                                         ctypes.POINTER(ctypes.c_size_t)]),
    "mok_layer_fwd_macro": (ctypes.c_int, [ctypes.POINTER(MokDesc), ctypes.c_int32, _P, _P,
                                           ctypes.POINTER(MokWeights), _P, _P, _P, _P, _P, _P,
                                           _P, _P]),
    "mok_layer_bwd": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, ctypes.POINTER(MokWeights),
                                     _P, _P, _P, _P, _P, _P, _P, _P,
                                     ctypes.POINTER(MokWeightGrads), _P, _P]),
    "mok_quantize_mx": (ctypes.c_int, [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P,
                                       ctypes.c_int32, _P, _P, _P]),
    "mok_pack_weights": (ctypes.c_int, [ctypes.POINTER(MokDesc), ctypes.POINTER(MokWeights), _P,
                                        _P]),
    "mok_device_status": (ctypes.c_int, [_P, _P, ctypes.POINTER(ctypes.c_int)]),
    "mok_autotune": (ctypes.c_int, [ctypes.POINTER(MokDesc), _P, _P, ctypes.POINTER(MokWeights),
                                    _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_int32,
                                    ctypes.POINTER(MokDesc), ctypes.POINTER(ctypes.c_float),
                                    ctypes.POINTER(MokTuneResult), ctypes.c_int32,
                                    ctypes.POINTER(ctypes.c_int32)]),
    "mok_route_fwd": (ctypes.c_int, [ctypes.POINTER(MokRouteDesc), _P, _P, _P, _P, _P, _P, _P]),
    "mok_route_bwd": (ctypes.c_int, [ctypes.POINTER(MokRouteDesc), _P, _P, _P, _P, _P]),
    "mok_sumsq_ws_size": (ctypes.c_int, [ctypes.c_int32, ctypes.POINTER(ctypes.c_size_t)]),
    "mok_grad_sumsq": (ctypes.c_int, [ctypes.c_int32, _P, ctypes.c_int32, _P, _P, _P]),
    "mok_adamw": (ctypes.c_int, [ctypes.c_int32, _P, ctypes.POINTER(MokAdamwConfig), _P]),
    "mok_muon_ws_size": (ctypes.c_int, [ctypes.c_int32, _P, ctypes.POINTER(ctypes.c_size_t)]),
    "mok_muon": (ctypes.c_int, [ctypes.c_int32, _P, ctypes.POINTER(MokMuonConfig), _P, _P]),
    "mok_orthogonalize_ws_size": (ctypes.c_int, [ctypes.c_int32, _P, ctypes.POINTER(ctypes.c_size_t)]),
    "mok_orthogonalize": (ctypes.c_int, [ctypes.c_int32, _P, ctypes.c_int32, ctypes.POINTER(MokNewtonSchulz), _P,
                                         _P]),
    "mok_block_padded_rows": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int32]),
    "mok_block_quantize": (ctypes.c_int, [ctypes.POINTER(MokBlockDesc), _P, _P, _P, _P, _P, _P, _P]),
    "mok_block_quantize_weights": (ctypes.c_int, [ctypes.POINTER(MokBlockDesc), _P, _P, _P, _P, _P, _P]),
    "mok_block_gemm": (ctypes.c_int, [ctypes.POINTER(MokBlockDesc), _P, _P, _P, _P, _P, _P, _P]),
    "mok_block_gemm_kernel": (ctypes.c_int32, [ctypes.POINTER(MokBlockDesc)]),
    "mok_block_wgrad": (ctypes.c_int, [ctypes.POINTER(MokBlockDesc), _P, _P, _P, _P, _P, _P, ctypes.c_int32, _P]),
    "mok_device_cus": (ctypes.c_int32, []),
    "mok_trace_kernel": (ctypes.c_int, [ctypes.c_int32, _P, _P]),
}

(MOK_TRACE_NONE, MOK_TRACE_FUSED_FWD, MOK_TRACE_BWD_GEMM1, MOK_TRACE_BWD_GEMM2, MOK_TRACE_DISPATCH,
 MOK_TRACE_COMBINE) = range(6)

_lib = None


def lib():
    """Load libmok.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmok.so not found at {LIB_PATH}; build it first "
                               "(python -m combine_router_top_schedule_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class MokError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} "
                         f"({lib().mok_status_str(code).decode()})")
        self.code = code


def _check(fn: str, code: int):
    if code != 0:
        raise MokError(fn, code)


def desc(H, E, K, I, S, T, e0, E_loc, M=0, ring_bytes=0, dtype="bf16", comm_cus=0, flags=0) -> MokDesc:
    dt = {"bf16": MOK_BF16, "mxfp8": MOK_MXFP8}[dtype] if isinstance(dtype, str) else int(dtype)
    return MokDesc(H, E, K, I, S, T, e0, E_loc, M, comm_cus, ring_bytes, dt, flags)


def desc_from_config(cfg, M: Optional[int] = None, ring_bytes: Optional[int] = None, **kw) -> MokDesc:
    """Descriptor for a ``datagen.Config``-like object (fields S, T, H, E, K, I, e0, E_loc, M,
    ring_bytes, dtype)."""
    return desc(cfg.H, cfg.E, cfg.K, cfg.I, cfg.S, cfg.T, cfg.e0, cfg.E_loc,
                cfg.M if M is None else M, cfg.ring_bytes if ring_bytes is None else ring_bytes,
                cfg.dtype, **kw)


def query_sizes(d: MokDesc) -> MokSizes:
    s = MokSizes()
    _check("mok_query_sizes", lib().mok_query_sizes(ctypes.byref(d), ctypes.byref(s)))
    return s


def workspace_size(d: MokDesc):
    """(ws_bytes, saved_bytes, slot_bytes) of the fused entry points."""
    ws, sv, sl = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check("mok_workspace_size", lib().mok_workspace_size(ctypes.byref(d), ctypes.byref(ws),
                                                          ctypes.byref(sv), ctypes.byref(sl)))
    return int(ws.value), int(sv.value), int(sl.value)


def two_wave_floor(cus: int, tile_m: int, tile_n: int, intermediate: int) -> int:
    return int(lib().mok_two_wave_floor(cus, tile_m, tile_n, intermediate))


def abi_version() -> int:
    return int(lib().mok_abi_version())


def device_cus() -> int:
    return int(lib().mok_device_cus())


# ------------------------------------------------------------------------ tensor marshalling

def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libmok takes device tensors only")


def seg_table(rows, S: int, T: int):
    """Device array of S base pointers into a [S*T][H] tensor (one [T][H] block per segment)."""
    import torch
    base = rows.data_ptr()
    step = T * rows.shape[1] * rows.element_size()
    ptrs = torch.tensor([base + s * step for s in range(S)], dtype=torch.int64)
    return ptrs.to(rows.device)


def weights_struct(wg=None, wu=None, wd=None, **mx) -> MokWeights:
    w = MokWeights()
    w.wg, w.wu, w.wd = _ptr(wg), _ptr(wu), _ptr(wd)
    for k, v in mx.items():
        setattr(w, k, _ptr(v))
    return w


def mok_schedule(d: MokDesc, logits, topk_idx, topk_p, saved, ws, stream=None):
    _need_cuda(logits, topk_idx, topk_p, saved, ws)
    _check("mok_schedule", lib().mok_schedule(ctypes.byref(d), _ptr(logits), _ptr(topk_idx),
                                              _ptr(topk_p), _ptr(saved), _ptr(ws), _stream(stream)))


def mok_schedule_routed(d: MokDesc, topk_idx, topk_p, saved, ws, stream=None):
    """The schedule table of a given choice (topk_idx int32, topk_p float32, both tidied in place)."""
    _need_cuda(topk_idx, topk_p, saved, ws)
    _check("mok_schedule_routed", lib().mok_schedule_routed(ctypes.byref(d), _ptr(topk_idx),
                                                            _ptr(topk_p), _ptr(saved), _ptr(ws),
                                                            _stream(stream)))


def mok_schedule_noalloc(d: MokDesc, logits, topk_idx, topk_p, saved, stream=None):
    _need_cuda(logits, topk_idx, topk_p, saved)
    _check("mok_schedule_noalloc", lib().mok_schedule_noalloc(ctypes.byref(d), _ptr(logits),
                                                              _ptr(topk_idx), _ptr(topk_p),
                                                              _ptr(saved), _stream(stream)))


def mok_router_fwd(d: MokDesc, x_seg, wr, logits, stream=None):
    _need_cuda(x_seg, wr, logits)
    _check("mok_router_fwd", lib().mok_router_fwd(ctypes.byref(d), _ptr(x_seg), _ptr(wr),
                                                  _ptr(logits), _stream(stream)))


def router_ws_size(d: MokDesc) -> int:
    n = ctypes.c_size_t()
    _check("mok_router_ws_size", lib().mok_router_ws_size(ctypes.byref(d), ctypes.byref(n)))
    return int(n.value)


def mok_router_bwd(d: MokDesc, x_seg, wr, dlogits, dwr, dx_seg, ws, stream=None):
    _need_cuda(x_seg, wr, dlogits, dwr, dx_seg, ws)
    _check("mok_router_bwd", lib().mok_router_bwd(ctypes.byref(d), _ptr(x_seg), _ptr(wr),
                                                  _ptr(dlogits), _ptr(dwr), _ptr(dx_seg),
                                                  _ptr(ws), _stream(stream)))


def mok_dispatch(d: MokDesc, saved, x_seg, xd, ws, stream=None):
    _need_cuda(saved, x_seg, xd, ws)
    _check("mok_dispatch", lib().mok_dispatch(ctypes.byref(d), _ptr(saved), _ptr(x_seg), _ptr(xd),
                                              _ptr(ws), _stream(stream)))


def mok_expert_ffn(d: MokDesc, saved, xd, w: MokWeights, act, slots, ws, stream=None):
    _need_cuda(saved, xd, act, slots, ws)
    _check("mok_expert_ffn", lib().mok_expert_ffn(ctypes.byref(d), _ptr(saved), _ptr(xd),
                                                  ctypes.byref(w), _ptr(act), _ptr(slots),
                                                  _ptr(ws), _stream(stream)))


def mok_combine(d: MokDesc, saved, topk_idx, topk_p, slots, out_seg, ws, stream=None):
    _need_cuda(saved, topk_idx, topk_p, slots, out_seg, ws)
    _check("mok_combine", lib().mok_combine(ctypes.byref(d), _ptr(saved), _ptr(topk_idx),
                                            _ptr(topk_p), _ptr(slots), _ptr(out_seg), _ptr(ws),
                                            _stream(stream)))


def mok_layer_fwd(d: MokDesc, x_seg, logits, w: MokWeights, out_seg, topk_idx, topk_p, saved,
                  ring, slots, ws, stream=None):
    _need_cuda(x_seg, logits, out_seg, topk_idx, topk_p, saved, ring, slots, ws)
    _check("mok_layer_fwd", lib().mok_layer_fwd(ctypes.byref(d), _ptr(x_seg), _ptr(logits),
                                                ctypes.byref(w), _ptr(out_seg), _ptr(topk_idx),
                                                _ptr(topk_p), _ptr(saved), _ptr(ring),
                                                _ptr(slots), _ptr(ws), _stream(stream)))


def mok_layer_fwd_routed(d: MokDesc, x_seg, w: MokWeights, out_seg, topk_idx, topk_p, saved, ring,
                         slots, ws, stream=None):
    _need_cuda(x_seg, out_seg, topk_idx, topk_p, saved, ring, slots, ws)
    _check("mok_layer_fwd_routed", lib().mok_layer_fwd_routed(
        ctypes.byref(d), _ptr(x_seg), ctypes.byref(w), _ptr(out_seg), _ptr(topk_idx), _ptr(topk_p),
        _ptr(saved), _ptr(ring), _ptr(slots), _ptr(ws), _stream(stream)))


def macro_ws_size(d: MokDesc, num_macro: int) -> int:
    n = ctypes.c_size_t()
    _check("mok_macro_ws_size", lib().mok_macro_ws_size(ctypes.byref(d), int(num_macro),
                                                        ctypes.byref(n)))
    return int(n.value)


def mok_layer_fwd_macro(d: MokDesc, x_segs, logits, w: MokWeights, out_segs, topk_idx, topk_p,
                        saved, ring, slots, ws, stream=None):
    """Lists (one entry per macrobatch) for every per-call argument."""
    B = len(x_segs)
    for lst in (logits, out_segs, topk_idx, topk_p, saved, slots):
        if len(lst) != B:
            raise ValueError("one entry per macrobatch in every list")
        _need_cuda(*lst)
    _need_cuda(*x_segs, ring, ws)
    arr = lambda ts: (ctypes.c_void_p * B)(*[_ptr(t) for t in ts])
    _check("mok_layer_fwd_macro", lib().mok_layer_fwd_macro(
        ctypes.byref(d), B, arr(x_segs), arr(logits), ctypes.byref(w), arr(out_segs),
        arr(topk_idx), arr(topk_p), arr(saved), _ptr(ring), arr(slots), _ptr(ws),
        _stream(stream)))


def mok_layer_bwd(d: MokDesc, dout_seg, x_seg, w: MokWeights, topk_idx, topk_p, saved, ring,
                  slots, dx_seg, dp, dlogits, dwg, dwu, dwd, ws, stream=None):
    _need_cuda(dout_seg, x_seg, topk_idx, topk_p, saved, ring, slots, dx_seg, dp, dwg, dwu, dwd, ws)
    g = MokWeightGrads(_ptr(dwg), _ptr(dwu), _ptr(dwd))
    _check("mok_layer_bwd", lib().mok_layer_bwd(ctypes.byref(d), _ptr(dout_seg), _ptr(x_seg),
                                                ctypes.byref(w), _ptr(topk_idx), _ptr(topk_p),
                                                _ptr(saved), _ptr(ring), _ptr(slots),
                                                _ptr(dx_seg), _ptr(dp), _ptr(dlogits),
                                                ctypes.byref(g), _ptr(ws), _stream(stream)))


def mok_quantize_mx(src, transpose: bool, codes, scales, stream=None):
    """Quantise a BF16 tensor [batch][rows][cols] (or [rows][cols]) to MXFP8."""
    _need_cuda(src, codes, scales)
    shape = tuple(src.shape)
    batch, rows, cols = (1,) + shape if len(shape) == 2 else shape
    _check("mok_quantize_mx", lib().mok_quantize_mx(batch, rows, cols, _ptr(src), int(transpose),
                                                    _ptr(codes), _ptr(scales), _stream(stream)))


def mok_pack_weights(d: MokDesc, w: MokWeights, packed, stream=None):
    """Pack the weights of `w` (BF16 values or MXFP8 codes and scales) into `packed`
    (sizes.packed_bytes, 256-byte aligned)."""
    _need_cuda(packed)
    _check("mok_pack_weights", lib().mok_pack_weights(ctypes.byref(d), ctypes.byref(w),
                                                      _ptr(packed), _stream(stream)))


def mok_autotune(d: MokDesc, x_seg, logits, w: MokWeights, out_seg, topk_idx, topk_p, saved,
                 ring, slots, ws, reps: int = 3, stream=None):
    """Returns (tuned descriptor, best ms, [(minibatch, comm_cus, ms), ...])."""
    _need_cuda(x_seg, logits, out_seg, topk_idx, topk_p, saved, ring, slots, ws)
    tuned, best = MokDesc(), ctypes.c_float()
    res = (MokTuneResult * 64)()
    n = ctypes.c_int32(0)
    _check("mok_autotune", lib().mok_autotune(ctypes.byref(d), _ptr(x_seg), _ptr(logits),
                                              ctypes.byref(w), _ptr(out_seg), _ptr(topk_idx),
                                              _ptr(topk_p), _ptr(saved), _ptr(ring), _ptr(slots),
                                              _ptr(ws), _stream(stream), int(reps),
                                              ctypes.byref(tuned), ctypes.byref(best), res, 64,
                                              ctypes.byref(n)))
    return tuned, float(best.value), [(r.minibatch_tokens, r.comm_cus, float(r.ms))
                                      for r in res[:n.value]]


def mok_device_status(ws, stream=None) -> int:
    out = ctypes.c_int(0)
    _check("mok_device_status", lib().mok_device_status(_ptr(ws), _stream(stream), ctypes.byref(out)))
    return int(out.value)


def mok_trace_kernel(kernel: int, before=None, after=None):
    """Record torch.cuda.Event `before` / `after` around one kernel group of the next calls
    (benchmark measurement; MOK_TRACE_NONE switches it off)."""
    b = None if before is None else int(before.cuda_event)
    a = None if after is None else int(after.cuda_event)
    _check("mok_trace_kernel", lib().mok_trace_kernel(int(kernel), b, a))


# ------------------------------------------------------------------------ expert routing

def route_desc(E: int, K: int, score: str = "softmax", groups: int = 1, top_groups: int = 1,
               group_score: str = "max", renorm: bool = True, scale: float = 1.0) -> MokRouteDesc:
    """What stays the same from call to call of mok_route_fwd / mok_route_bwd: experts, choices per
    token, score ("softmax" or "sigmoid"), groups of experts ("max" or "top2" scored) and weights.
    The tokens, their row stride and type are taken from the logits of each call."""
    return MokRouteDesc(0, E, E, K, {"softmax": MOK_SCORE_SOFTMAX, "sigmoid": MOK_SCORE_SIGMOID}[score],
                        groups, top_groups, {"max": MOK_GROUP_MAX, "top2": MOK_GROUP_TOP2}[group_score],
                        int(renorm), MOK_ELEM_F32, scale)


_torch = None


def _tch():
    """torch, imported at the first call that needs it."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _elem(t, name: str) -> int:
    torch = _tch()
    if t.dtype is torch.float32:
        return MOK_ELEM_F32
    if t.dtype is torch.bfloat16:
        return MOK_ELEM_BF16
    raise ValueError(f"{name} must be float32 or bfloat16, not {t.dtype}")


def _want(t, name: str, dtype, count: int, dev: int) -> int:
    """Address of a contiguous tensor of `count` elements of `dtype` on device number `dev`."""
    if t.dtype is not dtype or t.numel() != count or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {count} elements on device {dev}, "
                         f"not {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _device_of(t) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("libmok takes device tensors only")
    return dev


def _raw_stream(dev: int) -> int:
    """The current stream of device number `dev` (torch's own short way to its handle where it has one:
    a tenth of a microsecond instead of one)."""
    short = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
    return short(dev) if short is not None else _torch.cuda.current_stream(dev).cuda_stream


class _on_device:
    """Makes device number `dev` current around a call (the library launches on the current device) and
    gives the stream to use: the one asked for, or the device's current one."""

    __slots__ = ("guard", "raw")

    def __init__(self, dev: int, stream):
        torch = _tch()
        if stream is None:
            self.raw = _raw_stream(dev)
        elif stream.device.index != dev:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on device {dev}")
        else:
            self.raw = stream.cuda_stream
        self.guard = None if torch.cuda.current_device() == dev else torch.cuda.device(dev)

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _route_call(d: MokRouteDesc, logits, topk_idx, dev: int):
    """(`d` for these logits [N][E], whose rows may be strided; address of topk_idx)"""
    if logits.dim() != 2 or logits.shape[1] != d.num_experts:
        raise ValueError(f"logits must be [N][{d.num_experts}], not {tuple(logits.shape)}")
    N, E = logits.shape
    ld, step = logits.stride()
    if (E > 1 and step != 1) or (N > 1 and ld < E):
        raise ValueError("logits rows must be contiguous and must not overlap")
    c = MokRouteDesc.from_buffer_copy(d)
    c.num_tokens = N
    c.logits_stride = ld if N > 1 else E
    c.elem = _elem(logits, "logits")
    return c, _want(topk_idx, "topk_idx", _torch.int32, N * d.top_k, dev)


def mok_route_fwd(d: MokRouteDesc, logits, topk_idx, topk_w, bias=None, token_mask=None, load=None,
                  stream=None):
    torch, dev = _tch(), _device_of(logits)
    c, idx = _route_call(d, logits, topk_idx, dev)
    N, E = c.num_tokens, c.num_experts
    w = _want(topk_w, "topk_w", torch.float32, N * c.top_k, dev)
    if bias is not None:
        bias = _want(bias, "bias", torch.float32, E, dev)
    if token_mask is not None:
        token_mask = _want(token_mask.view(torch.uint8) if token_mask.dtype is torch.bool else token_mask,
                           "token_mask", torch.uint8, N, dev)
    if load is not None:
        load = _want(load, "load", torch.int32, E, dev)
    with _on_device(dev, stream) as s:
        _check("mok_route_fwd", lib().mok_route_fwd(ctypes.byref(c), logits.data_ptr(), bias, token_mask,
                                                    idx, w, load, s))


def mok_route_bwd(d: MokRouteDesc, logits, topk_idx, dw, dlogits, stream=None):
    torch, dev = _tch(), _device_of(logits)
    c, idx = _route_call(d, logits, topk_idx, dev)
    w = _want(dw, "dw", torch.float32, c.num_tokens * c.top_k, dev)
    dx = _want(dlogits, "dlogits", logits.dtype, c.num_tokens * c.num_experts, dev)
    with _on_device(dev, stream) as s:
        _check("mok_route_bwd", lib().mok_route_bwd(ctypes.byref(c), logits.data_ptr(), idx, w, dx, s))


# ------------------------------------------------------------------------ the optimizer step

class SumsqPlan:
    """The tensors of a mok_grad_sumsq call, and scratch for it."""

    def __init__(self, grads):
        if not grads:
            raise ValueError("no tensors")
        self.keep, self.dev, self.elem = list(grads), _device_of(grads[0]), _elem(grads[0], "a gradient")
        self.table = (MokSumsqTensor * len(grads))(*[
            (_want(g, "a gradient", grads[0].dtype, g.numel(), self.dev), g.numel()) for g in grads])
        n = ctypes.c_size_t()
        _check("mok_sumsq_ws_size", lib().mok_sumsq_ws_size(len(grads), ctypes.byref(n)))
        self.ws = _tch().zeros(int(n.value), dtype=_torch.uint8, device=grads[0].device)
        self.ws_at = self.ws.data_ptr()


def sumsq_plan(grads) -> SumsqPlan:
    return SumsqPlan(grads)


def mok_grad_sumsq(plan: SumsqPlan, out, ws=None, stream=None):
    """out (float64 [1]) = sum of squares over every tensor of the plan. Calls that may overlap in time
    need scratch `ws` of their own (as large as plan.ws, which is used without it, and zero-filled before its
    first use)."""
    at = _want(out, "out", _tch().float64, 1, plan.dev)
    ws_at = plan.ws_at
    if ws is not None:
        if ws.numel() * ws.element_size() < plan.ws.numel():
            raise ValueError(f"ws must hold {plan.ws.numel()} bytes")
        ws_at = _want(ws, "ws", ws.dtype, ws.numel(), plan.dev)
    with _on_device(plan.dev, stream) as s:
        _check("mok_grad_sumsq", lib().mok_grad_sumsq(len(plan.table), plan.table, plan.elem, at, ws_at, s))


class AdamwPlan:
    """The tensors of a mok_adamw call, checked once: lists of equal length of parameters (float32 or
    bfloat16), gradients (float32 or bfloat16), moments (float32; or uint8 E4M3 codes, with their uint8
    scales of 32 elements in m_scale and v_scale) and, for float32 parameters, bfloat16 copies (None in
    the place of a parameter that has none)."""

    def __init__(self, p, g, m, v, copy=None, m_scale=None, v_scale=None):
        torch = _tch()
        if not p:
            raise ValueError("no tensors")
        if (m_scale is None) != (v_scale is None):
            raise ValueError("m_scale and v_scale go together")
        lists = dict(p=p, g=g, m=m, v=v, copy=copy, m_scale=m_scale, v_scale=v_scale)
        self.keep = {k: list(ts) for k, ts in lists.items() if ts is not None}
        for name, ts in self.keep.items():
            if len(ts) != len(p):
                raise ValueError(f"{name} has {len(ts)} tensors, p {len(p)}")
        mx = m_scale is not None
        self.dev, param, grad = _device_of(p[0]), _elem(p[0], "a parameter"), _elem(g[0], "a gradient")
        if copy is not None and param != MOK_ELEM_F32:
            raise ValueError("only float32 parameters have a bfloat16 copy")
        types = dict(p=p[0].dtype, g=g[0].dtype, copy=torch.bfloat16, m=torch.uint8 if mx else torch.float32,
                     v=torch.uint8 if mx else torch.float32, m_scale=torch.uint8, v_scale=torch.uint8)
        sizes = [t.numel() for t in p]
        runs = [-(-n // 32) for n in sizes]
        columns, spans = {}, []
        for name, ts in self.keep.items():
            counts, dtype, read = runs if name.endswith("_scale") else sizes, types[name], name == "g"
            columns[name] = at = [
                None if t is None and name == "copy" else
                t.data_ptr() if t.dtype is dtype and t.numel() == n and t.get_device() == self.dev
                and t.is_contiguous() else _want(t, name, dtype, n, self.dev) for t, n in zip(ts, counts)]
            spans += [(a, a + n * dtype.itemsize, read, name) for a, n in zip(at, counts) if n and a is not None]
        # what is written overlaps nothing else (gradients may be given twice)
        spans.sort()
        read_end = written_end = 0   # the furthest ends so far
        for a, end, read, name in spans:
            if a < written_end or a < read_end and not read:
                raise ValueError(f"memory of {name} is shared with another tensor")
            if read:
                read_end = max(read_end, end)
            else:
                written_end = max(written_end, end)
        none = [None] * len(p)
        self.table = (MokAdamwTensor * len(p))(*zip(*[
            columns.get(name, none) for name in ("p", "copy", "g", "m", "v", "m_scale", "v_scale")], sizes))
        self.config = MokAdamwConfig(grad_elem=grad, param_elem=param,
                                     state=MOK_STATE_MX8 if mx else MOK_STATE_F32)


def adamw_plan(p, g, m, v, copy=None, m_scale=None, v_scale=None) -> AdamwPlan:
    return AdamwPlan(p, g, m, v, copy, m_scale, v_scale)


def mok_adamw(plan: AdamwPlan, lr, step, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
              weight_decay: float = 0.0, seed: int = 0, sumsq=None, max_norm: Optional[float] = None,
              stream=None):
    """One AdamW step over the plan's tensors, in place. `lr` and `step` may be device tensors (float64
    [1], int64 [1]), read when the step runs (a step's number is then added to `seed`; a number below 1, or a
    rate that is negative or not finite, changes nothing). With `sumsq`
    (float64 [1], the squared norm of all gradients) gradients are clipped to `max_norm` (None: not
    clipped) and a step whose norm is not finite changes nothing."""
    torch = _tch()
    c = MokAdamwConfig.from_buffer_copy(plan.config)
    if isinstance(lr, torch.Tensor):
        c.lr_dev = _want(lr, "lr", torch.float64, 1, plan.dev)
    else:
        c.lr = lr
    if isinstance(step, torch.Tensor):
        c.step_dev, c.step = _want(step, "step", torch.int64, 1, plan.dev), 1
    else:
        c.step = step
    if sumsq is not None:
        if not isinstance(sumsq, torch.Tensor):
            raise ValueError("sumsq is a device tensor")
        c.sumsq_dev = _want(sumsq, "sumsq", torch.float64, 1, plan.dev)
    elif max_norm is not None:
        raise ValueError("max_norm needs sumsq, the squared norm of all gradients")
    c.beta1, c.beta2, c.eps, c.weight_decay = beta1, beta2, eps, weight_decay
    c.max_norm = float("inf") if max_norm is None else max_norm
    c.seed = seed & 0xFFFFFFFF
    with _on_device(plan.dev, stream) as s:
        _check("mok_adamw", lib().mok_adamw(len(plan.table), plan.table, ctypes.byref(c), s))


# ------------------------------------------------------------------------ Muon

NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)
"""Coefficients of a step that takes singular values of 0..1 towards 1, small ones 3.4 times a step."""


def _newton_schulz(eps, steps, coefficients) -> MokNewtonSchulz:
    rows = list(coefficients)
    if rows and not hasattr(rows[0], "__len__"):
        rows = [tuple(rows)] * steps
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise ValueError(f"coefficients are (a, b, c), or {steps} of them")
    if not 1 <= steps <= 16:
        raise ValueError(f"steps are 1..16, not {steps}")
    ns = MokNewtonSchulz(eps, steps)
    ns.coefficients[:3 * steps] = [float(c) for r in rows for c in r]
    return ns


def _matrices(t, name: str):
    """(batch, rows, cols) of a tensor [..][rows][cols]."""
    if t.dim() < 2:
        raise ValueError(f"{name} must be matrices [..][rows][cols], not {tuple(t.shape)}")
    batch = 1
    for n in t.shape[:-2]:
        batch *= n
    return batch, t.shape[-2], t.shape[-1]


def _no_overlap(spans):
    """spans: (address, end, read only, name). What is written overlaps nothing else; what is read may be given twice."""
    spans.sort()
    read_end = written_end = 0   # the furthest ends so far
    for a, end, read, name in spans:
        if a < written_end or a < read_end and not read:
            raise ValueError(f"memory of {name} is shared with another tensor")
        if read:
            read_end = max(read_end, end)
        else:
            written_end = max(written_end, end)


class MuonPlan:
    """The tensors of a mok_muon call, checked once, and scratch for it: lists of equal length of float32 parameters
    [..][rows][cols], gradients (float32 or bfloat16), momenta (float32) and bfloat16 copies (None in the place of a
    parameter that has none). Calls that may overlap in time need plans of their own."""

    def __init__(self, p, g, m, copy=None):
        torch = _tch()
        if not p:
            raise ValueError("no tensors")
        lists = dict(p=p, g=g, m=m, copy=copy)
        self.keep = {k: list(ts) for k, ts in lists.items() if ts is not None}
        for name, ts in self.keep.items():
            if len(ts) != len(p):
                raise ValueError(f"{name} has {len(ts)} tensors, p {len(p)}")
        self.dev, self.grad = _device_of(p[0]), _elem(g[0], "a gradient")
        types = dict(p=torch.float32, g=g[0].dtype, m=torch.float32, copy=torch.bfloat16)
        at, spans = {}, []
        for name, ts in self.keep.items():
            at[name] = []
            for t, like in zip(ts, p):
                if t is None and name == "copy":
                    at[name].append(None)
                    continue
                if t.shape != like.shape:
                    raise ValueError(f"{name} must be {tuple(like.shape)}, not {tuple(t.shape)}")
                a = _want(t, name, types[name], like.numel(), self.dev)
                at[name].append(a)
                if t.numel():
                    spans.append((a, a + t.numel() * t.element_size(), name == "g", name))
        _no_overlap(spans)
        none = [None] * len(p)
        self.table = (MokMuonTensor * len(p))(*[
            (pp, c, gg, mm, *_matrices(t, "p")) for pp, c, gg, mm, t in zip(
                at["p"], at.get("copy", none), at["g"], at["m"], p)])
        n = ctypes.c_size_t()
        _check("mok_muon_ws_size", lib().mok_muon_ws_size(len(p), self.table, ctypes.byref(n)))
        self.ws = torch.empty(int(n.value), dtype=torch.uint8, device=p[0].device)


def muon_plan(p, g, m, copy=None) -> MuonPlan:
    return MuonPlan(p, g, m, copy)


def mok_muon(plan: MuonPlan, lr, momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
             eps: float = 1e-7, adjust: str = "rms", steps: int = 5, coefficients=NEWTON_SCHULZ, sumsq=None,
             max_norm: Optional[float] = None, stream=None):
    """One Muon step over the plan's tensors, in place. adjust: "rms" scales the orthogonalised update by 0.2
    sqrt(max(rows, cols)), "spectral" by sqrt(max(1, rows / cols)), "none" not at all. `lr` may be a device tensor
    (float64 [1], read when the step runs; negative or not finite changes nothing). `sumsq` and `max_norm` as
    in mok_adamw."""
    torch = _tch()
    c = MokMuonConfig(momentum=momentum, weight_decay=weight_decay, nesterov=int(nesterov), grad_elem=plan.grad,
                      adjust={"rms": MOK_ADJUST_RMS, "spectral": MOK_ADJUST_SPECTRAL, "none": MOK_ADJUST_NONE}[adjust],
                      ns=_newton_schulz(eps, steps, coefficients),
                      max_norm=float("inf") if max_norm is None else max_norm)
    if isinstance(lr, torch.Tensor):
        c.lr_dev = _want(lr, "lr", torch.float64, 1, plan.dev)
    else:
        c.lr = lr
    if sumsq is not None:
        if not isinstance(sumsq, torch.Tensor):
            raise ValueError("sumsq is a device tensor")
        c.sumsq_dev = _want(sumsq, "sumsq", torch.float64, 1, plan.dev)
    elif max_norm is not None:
        raise ValueError("max_norm needs sumsq, the squared norm of all gradients")
    with _on_device(plan.dev, stream) as s:
        _check("mok_muon", lib().mok_muon(len(plan.table), plan.table, ctypes.byref(c), plan.ws.data_ptr(), s))


class OrthogonalizePlan:
    """The matrices of a mok_orthogonalize call, checked once, and scratch for it: sources (float32 or bfloat16, of one
    type) [..][rows][cols] and bfloat16 outputs of the same shapes."""

    def __init__(self, src, out):
        torch = _tch()
        if not src:
            raise ValueError("no tensors")
        if len(src) != len(out):
            raise ValueError(f"out has {len(out)} tensors, src {len(src)}")
        self.keep, self.dev, self.elem = (list(src), list(out)), _device_of(src[0]), _elem(src[0], "a source")
        rows, spans = [], []
        for a, b in zip(src, out):
            if a.shape != b.shape:
                raise ValueError(f"out must be {tuple(a.shape)}, not {tuple(b.shape)}")
            at = [_want(t, name, dtype, a.numel(), self.dev)
                  for t, name, dtype in ((a, "src", src[0].dtype), (b, "out", torch.bfloat16))]
            rows.append((*at, *_matrices(a, "src")))
            if a.numel():
                spans += [(at[0], at[0] + a.numel() * a.element_size(), True, "src"),
                          (at[1], at[1] + b.numel() * 2, False, "out")]
        _no_overlap(spans)
        self.table = (MokOrthogonalizeTensor * len(src))(*rows)
        n = ctypes.c_size_t()
        _check("mok_orthogonalize_ws_size", lib().mok_orthogonalize_ws_size(len(src), self.table, ctypes.byref(n)))
        self.ws = torch.empty(int(n.value), dtype=torch.uint8, device=src[0].device)


def orthogonalize_plan(src, out) -> OrthogonalizePlan:
    return OrthogonalizePlan(src, out)


def mok_orthogonalize(plan: OrthogonalizePlan, eps: float = 1e-7, steps: int = 5, coefficients=NEWTON_SCHULZ,
                      stream=None):
    """Every output of the plan = its source, orthogonalised by `steps` Newton-Schulz steps. coefficients: (a, b, c) of
    every step, or one such triple for each."""
    ns = _newton_schulz(eps, steps, coefficients)
    with _on_device(plan.dev, stream) as s:
        _check("mok_orthogonalize", lib().mok_orthogonalize(len(plan.table), plan.table, plan.elem, ctypes.byref(ns),
                                                            plan.ws.data_ptr(), s))


# ------------------------------------------------------------------------ linear maps in block-scaled FP8

def _up128(n: int) -> int:
    return -(-n // 128) * 128


def block_padded_rows(rows: int, groups: int = 1) -> int:
    """Columns of the column codes of `rows` rows in `groups` groups, whatever the groups' sizes."""
    n = int(lib().mok_block_padded_rows(rows, groups))
    if n < 0:
        raise ValueError(f"{rows} rows in {groups} groups are out of range")
    return n


def _rows2d(t, name: str):
    """(rows, columns, elements from row to row) of a 2-d tensor with contiguous rows."""
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, not {tuple(t.shape)}")
    rows, cols = t.shape
    ld, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and ld < cols):
        raise ValueError(f"{name}: rows must be contiguous and must not overlap")
    return rows, cols, ld if rows > 1 else max(cols, 1)


def _offsets(offsets, dev: int):
    """(groups, address) of the groups' offsets (None: one group of all rows)."""
    if offsets is None:
        return 1, None
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError(f"offsets must be [groups + 1], not {tuple(offsets.shape)}")
    n = offsets.shape[0]
    return n - 1, _want(offsets, "offsets", _torch.int32, n, dev)


def _shaped(t, name: str, shape, dev: int, codes: bool):
    """Address of a contiguous tensor of `shape`, of E4M3 codes (uint8 or float8_e4m3fn) or of float32 scales."""
    dt = t.dtype
    if (t.shape != shape or not (dt is _torch.uint8 or dt is _torch.float8_e4m3fn if codes else dt is _torch.float32)
            or t.get_device() != dev or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {'uint8 or float8_e4m3fn' if codes else 'float32'} tensor "
                         f"{tuple(shape)} on device {dev}, not {dt} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    return t.data_ptr()


def _launch(fn: str, dev: int, stream, *args):
    """Calls the library with the stream last, on the tensors' device (the short way where that is the current one)."""
    if stream is None and _torch.cuda.current_device() == dev:
        code = getattr(_lib or lib(), fn)(*args, _raw_stream(dev))
    else:
        with _on_device(dev, stream) as s:
            code = getattr(lib(), fn)(*args, s)
    if code:
        raise MokError(fn, code)


def mok_block_quantize(x, codes=None, scales=None, codes_t=None, scales_t=None, offsets=None, stream=None):
    """E4M3 codes of rows x [R][K] (float32 or bfloat16, rows may be strided) with one scale for 128 values. codes
    [R][up(K)] and scales [up(K) / 128][R] are blocked along the row, for products; codes_t [K][P] and scales_t
    [P / 128][K], P = block_padded_rows(R, groups), along the rows of each group, for the weight gradient.
    offsets: int32 [groups + 1] (None: one group of all rows)."""
    _tch()
    dev = _device_of(x)
    R, K, ld = _rows2d(x, "x")
    G, off = _offsets(offsets, dev)
    if (codes is None) != (scales is None) or (codes_t is None) != (scales_t is None):
        raise ValueError("codes and scales go together")
    kb = -(-K // 128)
    c = s = ct = st = None
    if codes is not None:
        c, s = _shaped(codes, "codes", (R, kb * 128), dev, True), _shaped(scales, "scales", (kb, R), dev, False)
    if codes_t is not None:
        P = block_padded_rows(R, G)
        ct, st = _shaped(codes_t, "codes_t", (K, P), dev, True), _shaped(scales_t, "scales_t", (P // 128, K), dev, False)
    _launch("mok_block_quantize", dev, stream, ctypes.byref(MokBlockDesc(R, ld, G, 1, K, _elem(x, "x"))), x.data_ptr(),
            off, c, s, ct, st)


def mok_block_quantize_weights(w, codes, scales, codes_t=None, scales_t=None, stream=None):
    """E4M3 codes of weights w [G][N][K] (contiguous, float32 or bfloat16), one scale for 128 x 128 values: codes
    [G][N][up(K)], scales [G][up(N) / 128][up(K) / 128]; codes_t and scales_t are those of the transposed weights [G][K][N]."""
    _tch()
    dev = _device_of(w)
    if w.dim() != 3:
        raise ValueError(f"w must be [groups][N][K], not {tuple(w.shape)}")
    G, N, K = w.shape
    src = _want(w, "w", w.dtype, w.numel(), dev)
    if (codes_t is None) != (scales_t is None):
        raise ValueError("codes_t and scales_t go together")
    kb, nb = _up128(K) // 128, _up128(N) // 128
    c, s = _shaped(codes, "codes", (G, N, kb * 128), dev, True), _shaped(scales, "scales", (G, nb, kb), dev, False)
    ct = st = None
    if codes_t is not None:
        ct = _shaped(codes_t, "codes_t", (G, K, nb * 128), dev, True)
        st = _shaped(scales_t, "scales_t", (G, kb, nb), dev, False)
    _launch("mok_block_quantize_weights", dev, stream, ctypes.byref(MokBlockDesc(0, K, G, N, K, _elem(w, "w"))), src, c, s,
            ct, st)


def mok_block_gemm(x, x_scales, w, w_scales, out, offsets=None, stream=None):
    """out [R][N] (float32 or bfloat16, rows may be strided) = x w^T by groups of rows: x, x_scales from
    mok_block_quantize, w, w_scales from mok_block_quantize_weights (their transposed ones give the input gradient). Rows
    in no group are left as they are."""
    _tch()
    dev = _device_of(x)
    R, N, ld = _rows2d(out, "out")
    G, off = _offsets(offsets, dev)
    if x.dim() != 2 or x.shape[1] % 128 or x.shape[1] == 0:
        raise ValueError(f"x must be [rows][a multiple of 128], not {tuple(x.shape)}")
    K = x.shape[1]
    if out.get_device() != dev:
        raise ValueError(f"out is on {out.device}, x on device {dev}")
    _launch("mok_block_gemm", dev, stream, ctypes.byref(MokBlockDesc(R, ld, G, N, K, _elem(out, "out"))),
            _shaped(x, "x", (R, K), dev, True), _shaped(x_scales, "x_scales", (K // 128, R), dev, False),
            _shaped(w, "w", (G, N, K), dev, True), _shaped(w_scales, "w_scales", (G, -(-N // 128), K // 128), dev, False),
            off, out.data_ptr())


def mok_block_wgrad(dy_t, dy_scales, x_t, x_scales, dw, offsets=None, accumulate: bool = False, stream=None,
                    rows: Optional[int] = None):
    """dw [G][N][K] (float32, contiguous) = dy^T x by groups of rows, or added to with `accumulate`, from the column codes
    and scales (mok_block_quantize) of dy [R][N] and x [R][K]. rows: R, to which offsets are clamped as they were in
    mok_block_quantize. Without it they must not go past R: the codes' width tells R only to 127 rows, and a group made
    longer than it was would take columns that were never written."""
    _tch()
    dev = _device_of(dw)
    if dw.dim() != 3:
        raise ValueError(f"dw must be [groups][N][K], not {tuple(dw.shape)}")
    G, N, K = dw.shape
    groups, off = _offsets(offsets, dev)
    if groups != G:
        raise ValueError(f"dw has {G} groups, offsets {groups}")
    P = dy_t.shape[1] if dy_t.dim() == 2 else -1
    # (the most rows that need P columns, of the 2^22 that column codes have at most)
    R = min(P + 127 - 127 * G, 1 << 22) if rows is None else rows
    if P < 0 or P % 128 or R < 0 or (R + 127 * G) // 128 * 128 != P:
        raise ValueError(f"dy_t must be [{N}][block_padded_rows({'rows' if rows is None else rows}, {G})], "
                         f"not {tuple(dy_t.shape)}")
    _launch("mok_block_wgrad", dev, stream, ctypes.byref(MokBlockDesc(R, 0, G, N, K, MOK_ELEM_F32)),
            _shaped(dy_t, "dy_t", (N, P), dev, True), _shaped(dy_scales, "dy_scales", (P // 128, N), dev, False),
            _shaped(x_t, "x_t", (K, P), dev, True), _shaped(x_scales, "x_scales", (P // 128, K), dev, False), off,
            _shaped(dw, "dw", (G, N, K), dev, False), int(accumulate))
