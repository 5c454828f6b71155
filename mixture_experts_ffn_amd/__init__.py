"""MI355X (gfx950) MoE expert-FFN layer: Python binding of ``libmoe_ffn.so``.

The binding only marshals arguments: every step of the layer (routing,
gathered up_proj GEMM with SwiGLU, down_proj GEMM, combine, and the backward)
runs in the HIP kernels of the library.  PyTorch provides device memory and
the current stream.  There is no CPU or eager fallback: if the library is not
built, or the tensors are not on a GPU, the calls raise.

Public API (names follow the C ABI of ``include/moe_ffn.h``):

* ``moe_ffn_fwd(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight,
  save_for_backward=False, check_ids=False)`` -> ``y`` (and the saved context)
* ``moe_ffn_route(topk_ids, E)`` -> counts, offsets, sorted_slot, slot_pos
* ``moe_ffn(...)`` autograd-aware layer (forward + backward through the library)
* ``moe_ffn_router(logits, K, ...)`` autograd-aware router -> topk_weights, topk_ids
  (``moe_ffn_router_fwd`` and ``moe_ffn_router_bwd`` are its two halves)
* ``moe_ffn_mxfp4_quantize(weight, panels)`` -> packed 4-bit expert weights
  (``moe_ffn_mxfp4_dequantize`` gives the values back)
* ``moe_ffn_mxfp4_fwd(x, topk_ids, topk_weights, up, down, act="mxfp4")`` -> ``y``
* ``moe_ffn_grouped_mm(x, weight, offsets)`` autograd-aware product of row groups with their own
  weights (``moe_ffn_grouped_mm_fwd`` and ``moe_ffn_grouped_mm_bwd`` are its two halves)
* ``moe_ffn_int8_quantize(weight, panels)`` -> packed int8 weights with a scale for each column
  (``moe_ffn_int8_pack`` takes codes and scales, ``moe_ffn_int8_dequantize`` gives the values back)
* ``moe_ffn_int8_quantize_rows(x)`` -> int8 token rows with a scale for each
* ``moe_ffn_int8_mm(x, weight, offsets=None)`` -> their product, dense or by groups
* ``moe_ffn_int8_fwd(x, topk_ids, topk_weights, up, down)`` -> ``y`` of the layer on int8 weights
"""

from __future__ import annotations

import ctypes
import os
import re
import threading

import torch
from torch.autograd.function import once_differentiable

__all__ = [
    "MoEFFNError",
    "load_library",
    "library_path",
    "exported_symbols",
    "Problem",
    "StageEvents",
    "fwd_workspace_size",
    "route_workspace_size",
    "moe_ffn_fwd",
    "moe_ffn_fwd_noalloc",
    "NOALLOC_WS_BYTES",
    "fwd_stages",
    "fwd_plan",
    "moe_ffn_route",
    "read_status",
    "STAGES",
    "BWD_STAGES",
    "bwd_workspace_size",
    "moe_ffn_bwd_d",
    "moe_ffn_bwd_w",
    "moe_ffn_bwd",
    "moe_ffn",
    "MoEFFNFunction",
    "Router",
    "moe_ffn_router_fwd",
    "moe_ffn_router_bwd",
    "moe_ffn_router",
    "MoERouterFunction",
    "MXFP4Weight",
    "moe_ffn_mxfp4_quantize",
    "moe_ffn_mxfp4_dequantize",
    "mxfp4_workspace_size",
    "moe_ffn_mxfp4_fwd",
    "Grouped",
    "grouped_workspace_size",
    "moe_ffn_grouped_mm_fwd",
    "moe_ffn_grouped_mm_bwd",
    "moe_ffn_grouped_mm",
    "MoEGroupedMMFunction",
    "Int8Weight",
    "Int8Rows",
    "moe_ffn_int8_quantize",
    "moe_ffn_int8_pack",
    "moe_ffn_int8_dequantize",
    "moe_ffn_int8_quantize_rows",
    "int8_mm_workspace_size",
    "moe_ffn_int8_mm",
    "int8_workspace_size",
    "moe_ffn_int8_fwd",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libmoe_ffn.so")
_HEADER = os.path.join(os.path.dirname(_PKG), "include", "moe_ffn.h")
_lock = threading.Lock()
_lib = None

F32, BF16, I32, I64 = 0, 1, 2, 3
CHECK_IDS = 0x1
PIPELINE = 0x2
BULK = 0x10
CHECK_STATUS = 0x8
TEST_ONE_WORKGROUP = 0x400
TEST_DROP_RELEASE = 0x100
TEST_SMALL_GRID = 0x200
CHECK_SAVED = 0x4
DEV_BAD_ID, DEV_TIMEOUT, DEV_BAD_SAVED, DEV_BAD_WS = 0x1, 0x2, 0x4, 0x8
SCORES = {"softmax": 0, "sigmoid": 1}
ACT_FORMATS = {"mxfp4": 4, "mxfp6": 5}
STAGES = ("route", "gemm1", "gemm2", "combine", "pipeline")
BWD_STAGES = ("act_grad", "input_grad", "dx_combine", "w2_grad", "w1_grad")

ERR_NAMES = {0: "OK", 1: "ERR_NULL", 2: "ERR_SHAPE", 3: "ERR_DTYPE", 4: "ERR_ALIGN",
             5: "ERR_WORKSPACE", 6: "ERR_EXPERT_ID", 7: "ERR_SAVED", 8: "ERR_HIP",
             9: "ERR_DEVICE", 10: "ERR_TIMEOUT"}


class MoEFFNError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{ERR_NAMES.get(status, status)}: {message}")
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("H", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E", ctypes.c_int64), ("K", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("ids_dtype", ctypes.c_int32), ("Is", ctypes.c_int64)]


class SharedWeights(ctypes.Structure):
    _fields_ = [("up_proj_weight", ctypes.c_void_p), ("down_proj_weight", ctypes.c_void_p)]


class SharedGrads(ctypes.Structure):
    _fields_ = [("d_up_proj_weight", ctypes.c_void_p), ("d_down_proj_weight", ctypes.c_void_p)]


class Router(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("E", ctypes.c_int64), ("K", ctypes.c_int64),
                ("logits_stride", ctypes.c_int64), ("logits_dtype", ctypes.c_int32),
                ("ids_dtype", ctypes.c_int32), ("score", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class MXFP4Stack(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int64), ("Kd", ctypes.c_int64), ("N", ctypes.c_int64),
                ("panels", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class Grouped(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("E", ctypes.c_int64), ("Kd", ctypes.c_int64),
                ("N", ctypes.c_int64), ("x_stride", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("offsets_dtype", ctypes.c_int32), ("transposed", ctypes.c_int32)]


class Int8Stack(ctypes.Structure):
    _fields_ = MXFP4Stack._fields_


class Int8RowsShape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("Kd", ctypes.c_int64), ("x_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


class Int8Product(ctypes.Structure):
    _fields_ = [("weight", Int8Stack), ("M", ctypes.c_int64), ("offsets_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32)]


class FwdStageLayout(ctypes.Structure):
    """Byte offsets of the forward's intermediate stages in its workspace."""

    _fields_ = [(n, ctypes.c_size_t) for n in
                ("counts", "offsets", "sorted_slot", "slot_pos", "act", "o")] + \
               [("tile_rows", ctypes.c_int32), ("kernel", ctypes.c_int32)]


KERNELS = {0: "generic", 1: "engine", 2: "tiles", 3: "big_tiles", 4: "pipelined",
           5: "tiles_big_gemm2"}


def fwd_plan(problem: Problem, flags: int = 0):
    """(tile rows, kernel family name) the forward runs for this problem."""
    lay = FwdStageLayout()
    _check(load_library().moe_ffn_fwd_stages(ctypes.byref(problem), flags, ctypes.byref(lay)))
    return lay.tile_rows, KERNELS[lay.kernel]


class StageEvents(ctypes.Structure):
    _fields_ = [("begin", ctypes.c_void_p * 8), ("end", ctypes.c_void_p * 8)]


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libmoe_ffn.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is not built; run `python -m mixture_experts_ffn_amd.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, sz, i32, u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint32
        pp = ctypes.POINTER(Problem)
        psz = ctypes.POINTER(ctypes.c_size_t)
        sigs = {
            "moe_ffn_fwd_workspace_size": [pp, u32, psz, psz],
            "moe_ffn_fwd": [pp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp],
            "moe_ffn_fwd_ex": [pp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp,
                               ctypes.POINTER(StageEvents)],
            "moe_ffn_route_workspace_size": [pp, psz],
            "moe_ffn_bwd_workspace_size": [pp, u32, psz],
            "moe_ffn_bwd": [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp],
            "moe_ffn_bwd_ex": [pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp,
                               ctypes.POINTER(StageEvents)],
            "moe_ffn_bwd_d": [pp, vp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp],
            "moe_ffn_fwd_shared": [pp, vp, vp, vp, vp, vp, ctypes.POINTER(SharedWeights), vp, vp,
                                   vp, sz, u32, vp, ctypes.POINTER(StageEvents)],
            "moe_ffn_bwd_shared": [pp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(SharedWeights), vp,
                                   vp, vp, vp, vp, ctypes.POINTER(SharedGrads), vp, sz, u32, vp,
                                   ctypes.POINTER(StageEvents)],
            "moe_ffn_bwd_w": [pp, vp, vp, vp, vp, vp, vp, sz, u32, vp],
            "moe_ffn_route": [pp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_ffn_fwd_noalloc": [pp, vp, vp, vp, vp, vp, vp, u32, vp],
            "moe_ffn_fwd_stages": [pp, u32, ctypes.POINTER(FwdStageLayout)],
            "moe_ffn_router_fwd": [ctypes.POINTER(Router), vp, vp, vp, vp, vp],
            "moe_ffn_router_bwd": [ctypes.POINTER(Router), vp, vp, vp, vp, vp],
            "moe_ffn_mxfp4_weight_size": [ctypes.POINTER(MXFP4Stack), psz],
            "moe_ffn_mxfp4_quantize": [ctypes.POINTER(MXFP4Stack), vp, vp, sz, vp],
            "moe_ffn_mxfp4_dequantize": [ctypes.POINTER(MXFP4Stack), vp, sz, vp, vp],
            "moe_ffn_mxfp4_workspace_size": [pp, i32, u32, psz],
            "moe_ffn_mxfp4_fwd": [pp, i32, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp],
            "moe_ffn_grouped_workspace_size": [ctypes.POINTER(Grouped), psz],
            "moe_ffn_grouped_mm": [ctypes.POINTER(Grouped), vp, vp, vp, vp, vp, sz, vp],
            "moe_ffn_grouped_mm_bwd": [ctypes.POINTER(Grouped), vp, vp, vp, vp, vp, vp, vp, sz, vp],
            "moe_ffn_int8_weight_size": [ctypes.POINTER(Int8Stack), psz],
            "moe_ffn_int8_quantize": [ctypes.POINTER(Int8Stack), vp, vp, sz, vp],
            "moe_ffn_int8_pack": [ctypes.POINTER(Int8Stack), vp, vp, vp, sz, vp],
            "moe_ffn_int8_dequantize": [ctypes.POINTER(Int8Stack), vp, sz, vp, vp],
            "moe_ffn_int8_row_bytes": [ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)],
            "moe_ffn_int8_quantize_rows": [ctypes.POINTER(Int8RowsShape), vp, vp, vp, vp],
            "moe_ffn_int8_mm_workspace_size": [ctypes.POINTER(Int8Product), psz],
            "moe_ffn_int8_mm": [ctypes.POINTER(Int8Product), vp, vp, vp, sz, vp, vp, vp, sz, vp],
            "moe_ffn_int8_workspace_size": [pp, u32, psz],
            "moe_ffn_int8_fwd": [pp, vp, vp, vp, vp, vp, vp, vp, sz, u32, vp],
            "moe_ffn_read_status": [vp, vp, ctypes.POINTER(ctypes.c_int32)],
            "moe_ffn_event_create": [ctypes.POINTER(ctypes.c_void_p)],
            "moe_ffn_event_destroy": [vp],
            "moe_ffn_event_elapsed_ms": [vp, vp, ctypes.POINTER(ctypes.c_float)],
        }
        for name, args in sigs.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = i32
        for name in ("moe_ffn_status_string",):
            getattr(lib, name).argtypes = [i32]
            getattr(lib, name).restype = ctypes.c_char_p
        lib.moe_ffn_last_error.argtypes = []
        lib.moe_ffn_last_error.restype = ctypes.c_char_p
        lib.moe_ffn_version.argtypes = []
        lib.moe_ffn_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def exported_symbols() -> list[str]:
    """Function names declared in include/moe_ffn.h."""
    text = open(_HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(moe_ffn_\w+)\s*\(", text)))


def _check(rc: int):
    if rc != 0:
        lib = load_library()
        detail = lib.moe_ffn_last_error().decode() or lib.moe_ffn_status_string(rc).decode()
        raise MoEFFNError(rc, detail)


def _dtype_code_of(dtype) -> int:
    if dtype == torch.float32:
        return F32
    if dtype == torch.bfloat16:
        return BF16
    raise MoEFFNError(3, f"unsupported dtype {dtype}; use float32 or bfloat16")


def _dtype_code(t: torch.Tensor) -> int:
    return _dtype_code_of(t.dtype)


def _ids_code_of(dtype) -> int:
    if dtype == torch.int32:
        return I32
    if dtype == torch.int64:
        return I64
    raise MoEFFNError(3, f"topk_ids must be int32 or int64, got {dtype}")


def _ids_code(t: torch.Tensor) -> int:
    return _ids_code_of(t.dtype)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _launch(entry, dev, *args):
    """Call a C entry whose last argument is the stream, on ``dev``'s current stream with ``dev``
    current.  A small call is bound by its host time, of which a device guard and a Stream object
    take 3 us: the guard is only for another device, and the stream handle is asked for by itself
    (0.3 us)."""
    if dev.index == torch.cuda.current_device():
        rc = entry(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            rc = entry(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    _check(rc)


def _require_gpu(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise MoEFFNError(1, "all tensors must be on the GPU (no CPU fallback exists)")
        if t is not None and not t.is_contiguous():
            raise MoEFFNError(4, "all tensors must be contiguous")


def _own_gradient(dy):
    """``dy`` as the library takes it.  Autograd hands out views into larger buffers (the gradient
    of a concatenation's part), which may be contiguous and yet start anywhere; those are copied."""
    dy = dy.contiguous()
    return dy if dy.data_ptr() % 16 == 0 else dy.clone()


def make_problem(x, topk_ids, up_proj_weight, down_proj_weight) -> Problem:
    if x.dim() != 2 or topk_ids.dim() != 2 or up_proj_weight.dim() != 3 or down_proj_weight.dim() != 3:
        raise MoEFFNError(2, "expected x [T,H], topk_ids [T,K], up [E,H,2I], down [E,I,H]")
    T, H = x.shape
    E, H2, I2 = up_proj_weight.shape
    E2, I, H3 = down_proj_weight.shape
    if topk_ids.shape[0] != T or H2 != H or H3 != H or E2 != E or I2 != 2 * I:
        raise MoEFFNError(2, f"inconsistent shapes x{tuple(x.shape)} ids{tuple(topk_ids.shape)} "
                             f"up{tuple(up_proj_weight.shape)} down{tuple(down_proj_weight.shape)}")
    if up_proj_weight.dtype != x.dtype or down_proj_weight.dtype != x.dtype:
        raise MoEFFNError(3, "x, up_proj_weight and down_proj_weight must share one dtype")
    return Problem(T, H, I, E, topk_ids.shape[1], _dtype_code(x), _ids_code(topk_ids))


def fwd_workspace_size(problem: Problem, flags: int = 0):
    ws, saved = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().moe_ffn_fwd_workspace_size(ctypes.byref(problem), flags,
                                                     ctypes.byref(ws), ctypes.byref(saved)))
    return ws.value, saved.value


def route_workspace_size(problem: Problem) -> int:
    ws = ctypes.c_size_t()
    _check(load_library().moe_ffn_route_workspace_size(ctypes.byref(problem), ctypes.byref(ws)))
    return ws.value


def _shared_problem(prob, x, shared_up_proj_weight, shared_down_proj_weight):
    """Set prob.Is from the shared-expert weights (both or neither)."""
    if shared_up_proj_weight is None and shared_down_proj_weight is None:
        return None
    if shared_up_proj_weight is None or shared_down_proj_weight is None:
        raise MoEFFNError(2, "pass both shared_up_proj_weight and shared_down_proj_weight")
    _require_gpu(shared_up_proj_weight, shared_down_proj_weight)
    Is, H = shared_down_proj_weight.shape
    if shared_up_proj_weight.shape != (H, 2 * Is) or H != x.shape[1]:
        raise MoEFFNError(2, "expected shared_up [H, 2Is] and shared_down [Is, H]")
    if shared_up_proj_weight.dtype != x.dtype or shared_down_proj_weight.dtype != x.dtype:
        raise MoEFFNError(3, "the shared weights must have the dtype of x")
    prob.Is = Is
    return SharedWeights(shared_up_proj_weight.data_ptr(), shared_down_proj_weight.data_ptr())


def _mode_flag(pipelined):
    """MOE_FFN_PIPELINE for True, MOE_FFN_BULK for False, nothing for None."""
    if pipelined is None:
        return 0
    return PIPELINE if pipelined else BULK


def moe_ffn_fwd(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight, *,
                save_for_backward: bool = False, check_ids: bool = False, ws=None,
                stage_events: StageEvents | None = None, return_ws: bool = False,
                pipelined: bool | None = None, flags: int = 0, shared_up_proj_weight=None,
                shared_down_proj_weight=None):
    """y [T, H] of the MoE expert-FFN layer (see include/moe_ffn.h).

    With ``save_for_backward`` also returns the saved context (a uint8 device
    tensor) that the backward consumes.  ``ws`` may pass a preallocated
    workspace (uint8 tensor of at least ``fwd_workspace_size`` bytes).
    ``pipelined`` True asks for the one-launch forward with tile-granular
    release (bf16, H % 256 == 0, I % 128 == 0; other shapes ignore it), False
    for the two separate GEMM launches, None (the default) leaves the choice
    to the library;
    ``flags`` passes further MOE_FFN_* bits through.  ``shared_up_proj_weight``
    [H, 2Is] and ``shared_down_proj_weight`` [Is, H] (Is a multiple of I) add the
    shared expert's SwiGLU FFN to y; the saved context then covers it too.
    """
    lib = load_library()
    _require_gpu(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight)
    if topk_weights.dtype != torch.float32 or topk_weights.shape != topk_ids.shape:
        raise MoEFFNError(3, "topk_weights must be float32 with the shape of topk_ids")
    prob = make_problem(x, topk_ids, up_proj_weight, down_proj_weight)
    sw = _shared_problem(prob, x, shared_up_proj_weight, shared_down_proj_weight)
    ws_bytes, saved_bytes = fwd_workspace_size(prob)
    dev = x.device
    y = torch.empty_like(x)
    if ws is None:
        ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    elif ws.numel() < ws_bytes:
        raise MoEFFNError(5, f"workspace has {ws.numel()} bytes, {ws_bytes} needed")
    saved = torch.empty(saved_bytes, dtype=torch.uint8, device=dev) if save_for_backward else None
    flags |= (CHECK_IDS if check_ids else 0) | _mode_flag(pipelined)
    ev = ctypes.byref(stage_events) if stage_events is not None else None
    with torch.cuda.device(dev):
        if sw is not None:
            rc = lib.moe_ffn_fwd_shared(ctypes.byref(prob), _ptr(x), _ptr(topk_ids),
                                        _ptr(topk_weights), _ptr(up_proj_weight),
                                        _ptr(down_proj_weight), ctypes.byref(sw), _ptr(y),
                                        _ptr(saved), _ptr(ws), ws.numel(), flags, _stream(dev),
                                        ev)
        else:
            rc = lib.moe_ffn_fwd_ex(ctypes.byref(prob), _ptr(x), _ptr(topk_ids),
                                    _ptr(topk_weights), _ptr(up_proj_weight),
                                    _ptr(down_proj_weight), _ptr(y), _ptr(saved), _ptr(ws),
                                    ws.numel(), flags, _stream(dev), ev)
    _check(rc)
    out = (y,)
    if save_for_backward:
        out += (saved,)
    if return_ws:
        out += (ws,)
    return out[0] if len(out) == 1 else out


def fwd_stages(x, topk_ids, up_proj_weight, down_proj_weight, ws, flags: int = 0):
    """Views of the intermediate stages an inference forward left in ``ws``:
    counts, offsets, sorted_slot, slot_pos (int32) and act [TK, I], o [TK, H]
    in the problem dtype, rows in permuted (expert-major) order."""
    prob = make_problem(x, topk_ids, up_proj_weight, down_proj_weight)
    lay = FwdStageLayout()
    _check(load_library().moe_ffn_fwd_stages(ctypes.byref(prob), flags, ctypes.byref(lay)))
    T, K, E = prob.T, prob.K, prob.E
    I, H = prob.I, prob.H

    def view(off, n, dtype, shape):
        nb = n * torch.empty((), dtype=dtype).element_size()
        return ws[off:off + nb].view(dtype).view(shape)

    return dict(counts=view(lay.counts, E, torch.int32, (E,)),
                offsets=view(lay.offsets, E + 1, torch.int32, (E + 1,)),
                sorted_slot=view(lay.sorted_slot, T * K, torch.int32, (T * K,)),
                slot_pos=view(lay.slot_pos, T * K, torch.int32, (T * K,)),
                act=view(lay.act, T * K * I, x.dtype, (T * K, I)),
                o=view(lay.o, T * K * H, x.dtype, (T * K, H)))


def moe_ffn_fwd_noalloc(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight, y, *,
                        pipelined: bool | None = None, flags: int = 0):
    """The inference forward into the caller's ``y`` [T, H] with no workspace:
    the library's own per-GPU scratch (include/moe_ffn.h, moe_ffn_fwd_noalloc)
    serves as the workspace, so nothing is allocated.  Raises MoEFFNError for
    problems whose workspace exceeds NOALLOC_WS_BYTES."""
    lib = load_library()
    _require_gpu(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight, y)
    if topk_weights.dtype != torch.float32 or topk_weights.shape != topk_ids.shape:
        raise MoEFFNError(3, "topk_weights must be float32 with the shape of topk_ids")
    if y.shape != x.shape or y.dtype != x.dtype or not y.is_contiguous():
        raise MoEFFNError(2, "y must be a contiguous tensor with the shape and dtype of x")
    prob = make_problem(x, topk_ids, up_proj_weight, down_proj_weight)
    flags |= _mode_flag(pipelined)
    dev = x.device
    with torch.cuda.device(dev):
        rc = lib.moe_ffn_fwd_noalloc(ctypes.byref(prob), _ptr(x), _ptr(topk_ids),
                                     _ptr(topk_weights), _ptr(up_proj_weight),
                                     _ptr(down_proj_weight), _ptr(y), flags, _stream(dev))
    _check(rc)
    return y


NOALLOC_WS_BYTES = 64 << 20  # MOE_FFN_NOALLOC_WS_BYTES


def bwd_workspace_size(problem: Problem, flags: int = 0) -> int:
    ws = ctypes.c_size_t()
    _check(load_library().moe_ffn_bwd_workspace_size(ctypes.byref(problem), flags,
                                                     ctypes.byref(ws)))
    return ws.value


def moe_ffn_bwd(dy, x, topk_ids, topk_weights, up_proj_weight, down_proj_weight, saved, *,
                ws=None, stage_events: StageEvents | None = None, check_saved: bool = False,
                return_ws: bool = False, shared_up_proj_weight=None,
                shared_down_proj_weight=None):
    """Gradients (dx, d_up_proj_weight, d_down_proj_weight, d_topk_weights) of the layer.

    With the shared expert's weights (as given to the forward) it also returns
    (d_shared_up_proj_weight, d_shared_down_proj_weight).

    `saved` is the context returned by ``moe_ffn_fwd(..., save_for_backward=True)`` for the
    same inputs.  Outputs are freshly allocated and overwritten (never accumulated).
    ``check_saved`` verifies on the host (synchronously) that `saved` belongs to this
    problem; otherwise the check runs on the device and a mismatch yields zeros and the
    DEV_BAD_SAVED status bit (``read_status`` of the workspace, see ``return_ws``).
    """
    lib = load_library()
    _require_gpu(dy, x, topk_ids, topk_weights, up_proj_weight, down_proj_weight, saved)
    prob = make_problem(x, topk_ids, up_proj_weight, down_proj_weight)
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise MoEFFNError(2, "dy must have the shape and dtype of x")
    sw = _shared_problem(prob, x, shared_up_proj_weight, shared_down_proj_weight)
    ws_bytes = bwd_workspace_size(prob)
    dev = x.device
    dx = torch.empty_like(x)
    d_up = torch.empty_like(up_proj_weight)
    d_down = torch.empty_like(down_proj_weight)
    d_topk = torch.empty(topk_ids.shape, dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    ev = ctypes.byref(stage_events) if stage_events is not None else None
    flags = CHECK_SAVED if check_saved else 0
    with torch.cuda.device(dev):
        if sw is not None:
            d_sup = torch.empty_like(shared_up_proj_weight)
            d_sdown = torch.empty_like(shared_down_proj_weight)
            sg = SharedGrads(d_sup.data_ptr(), d_sdown.data_ptr())
            rc = lib.moe_ffn_bwd_shared(ctypes.byref(prob), _ptr(dy), _ptr(x), _ptr(topk_ids),
                                        _ptr(topk_weights), _ptr(up_proj_weight),
                                        _ptr(down_proj_weight), ctypes.byref(sw), _ptr(saved),
                                        _ptr(dx), _ptr(d_up), _ptr(d_down), _ptr(d_topk),
                                        ctypes.byref(sg), _ptr(ws), ws.numel(), flags,
                                        _stream(dev), ev)
        else:
            rc = lib.moe_ffn_bwd_ex(ctypes.byref(prob), _ptr(dy), _ptr(x), _ptr(topk_ids),
                                    _ptr(topk_weights), _ptr(up_proj_weight),
                                    _ptr(down_proj_weight), _ptr(saved), _ptr(dx), _ptr(d_up),
                                    _ptr(d_down), _ptr(d_topk), _ptr(ws), ws.numel(), flags,
                                    _stream(dev), ev)
    _check(rc)
    if sw is not None:
        return (dx, d_up, d_down, d_topk, d_sup, d_sdown) + ((ws,) if return_ws else ())
    if return_ws:
        return dx, d_up, d_down, d_topk, ws
    return dx, d_up, d_down, d_topk


def moe_ffn_bwd_d(dy, topk_ids, topk_weights, up_proj_weight, down_proj_weight, saved, *,
                  ws=None, check_saved: bool = False):
    """Data half of the backward: (dx, d_topk_weights, ws).

    `ws` then holds the intermediate gradients that ``moe_ffn_bwd_w`` reads; keep it
    untouched until that call has been issued on the same stream.
    """
    lib = load_library()
    _require_gpu(dy, topk_ids, topk_weights, up_proj_weight, down_proj_weight, saved)
    prob = make_problem(dy, topk_ids, up_proj_weight, down_proj_weight)
    ws_bytes = bwd_workspace_size(prob)
    dev = dy.device
    dx = torch.empty_like(dy)
    d_topk = torch.empty(topk_ids.shape, dtype=torch.float32, device=dev)
    if ws is None:
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    flags = CHECK_SAVED if check_saved else 0
    with torch.cuda.device(dev):
        rc = lib.moe_ffn_bwd_d(ctypes.byref(prob), _ptr(dy), _ptr(topk_weights),
                               _ptr(up_proj_weight), _ptr(down_proj_weight), _ptr(saved), _ptr(dx),
                               _ptr(d_topk), _ptr(ws), ws.numel(), flags, _stream(dev))
    _check(rc)
    return dx, d_topk, ws


def moe_ffn_bwd_w(dy, x, topk_ids, up_proj_weight, down_proj_weight, saved, ws, *,
                  check_saved: bool = False):
    """Weight half of the backward: (d_up_proj_weight, d_down_proj_weight).

    `ws` must be the workspace of the ``moe_ffn_bwd_d`` call for the same `saved`
    context; otherwise the gradients are zeros and ``read_status(ws)`` has DEV_BAD_WS
    (with ``check_saved`` the call raises instead).  topk_ids and the weights only
    describe the problem's shape here.
    """
    lib = load_library()
    _require_gpu(dy, x, topk_ids, saved, ws)
    prob = make_problem(x, topk_ids, up_proj_weight, down_proj_weight)
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise MoEFFNError(2, "dy must have the shape and dtype of x")
    dev = x.device
    d_up = torch.empty_like(up_proj_weight)
    d_down = torch.empty_like(down_proj_weight)
    flags = CHECK_SAVED if check_saved else 0
    with torch.cuda.device(dev):
        rc = lib.moe_ffn_bwd_w(ctypes.byref(prob), _ptr(dy), _ptr(x), _ptr(saved), _ptr(d_up),
                               _ptr(d_down), _ptr(ws), ws.numel(), flags, _stream(dev))
    _check(rc)
    return d_up, d_down


class MoEFFNFunction(torch.autograd.Function):
    """Autograd wrapper: forward saves the library's context (route arrays and the
    pre-activation), backward returns one gradient per input (None for topk_ids)."""

    @staticmethod
    def forward(ctx, x, topk_ids, topk_weights, up_proj_weight, down_proj_weight):
        y, saved = moe_ffn_fwd(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight,
                               save_for_backward=True)
        ctx.save_for_backward(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight,
                              saved)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, topk_ids, topk_weights, up, down, saved = ctx.saved_tensors
        dx, d_up, d_down, d_topk = moe_ffn_bwd(_own_gradient(dy), x, topk_ids, topk_weights, up,
                                               down, saved)
        return dx, None, d_topk, d_up, d_down


def moe_ffn(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight):
    """y = MoE expert-FFN layer; differentiable in x, topk_weights and both weights."""
    return MoEFFNFunction.apply(x, topk_ids, topk_weights, up_proj_weight, down_proj_weight)


def moe_ffn_route(topk_ids: torch.Tensor, E: int, H: int = 8, I: int = 8):
    """Routing alone: (counts [E], offsets [E+1], sorted_slot [TK], slot_pos [TK], ws)."""
    lib = load_library()
    _require_gpu(topk_ids)
    T, K = topk_ids.shape
    prob = Problem(T, H, I, E, K, BF16, _ids_code(topk_ids))
    ws_bytes = route_workspace_size(prob)
    dev = topk_ids.device
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    sorted_slot = torch.empty(max(T * K, 1), dtype=torch.int32, device=dev)
    slot_pos = torch.empty(max(T * K, 1), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        rc = lib.moe_ffn_route(ctypes.byref(prob), _ptr(topk_ids), _ptr(counts), _ptr(offsets),
                               _ptr(sorted_slot), _ptr(slot_pos), _ptr(ws), ws_bytes,
                               _stream(dev))
    _check(rc)
    return counts, offsets, sorted_slot[:T * K], slot_pos[:T * K], ws


def _router(logits, K, ids_dtype, score, renormalize, groups, topk_groups, group_top, scale):
    if not logits.is_cuda:
        raise MoEFFNError(1, "all tensors must be on the GPU (no CPU fallback exists)")
    if logits.dim() != 2:
        raise MoEFFNError(2, "expected logits [T, E]")
    if logits.stride(1) != 1 and logits.shape[1] > 1:
        raise MoEFFNError(4, "a token's logits must be consecutive")
    if score not in SCORES:
        raise MoEFFNError(2, f"score must be one of {sorted(SCORES)}, got {score!r}")
    T, E = logits.shape
    stride = logits.stride(0) if T > 1 else max(E, 1)
    return Router(T, E, K, stride, _dtype_code(logits), ids_dtype, SCORES[score],
                  1 if renormalize else 0, groups, topk_groups, group_top, scale)


def _same_device(t, *others):
    index = t.get_device()
    for o in others:
        if o is not None and o.get_device() != index:
            raise MoEFFNError(1, f"tensors on {t.device} and {o.device}: one device is needed")


def moe_ffn_router_fwd(logits, K: int, *, bias=None, score: str = "softmax",
                       renormalize: bool = True, groups: int = 1, topk_groups: int = 1,
                       group_top: int = 1, scale: float = 1.0, ids_dtype=torch.int32):
    """(topk_weights [T, K] fp32, topk_ids [T, K]) of router logits [T, E] (see
    include/moe_ffn.h, moe_ffn_router_fwd).

    ``logits`` are float32 or bfloat16; their rows may be strided.  ``bias`` [E]
    float32 shifts the scores for the selection only.  With ``groups`` > 1 the
    experts come from the ``topk_groups`` best groups.  A slot without an open
    expert (every other logit -inf) has id -1 and weight 0.
    """
    lib = load_library()
    ids_code = _ids_code_of(ids_dtype)
    r = _router(logits, K, ids_code, score, renormalize, groups, topk_groups, group_top, scale)
    if bias is not None:
        _require_gpu(bias)
        _same_device(logits, bias)
        if bias.dtype != torch.float32 or bias.shape != (r.E,):
            raise MoEFFNError(3, "bias must be float32 of shape [E]")
    dev = logits.device
    # sizes the library rejects are not allocated
    shape = (r.T, K) if 0 < K <= 32 else (0, 0)
    weights = torch.empty(shape, dtype=torch.float32, device=dev)
    ids = torch.empty(shape, dtype=ids_dtype, device=dev)
    _launch(lib.moe_ffn_router_fwd, dev, r, logits.data_ptr(), _ptr(bias), ids.data_ptr(),
            weights.data_ptr())
    return weights, ids


def moe_ffn_router_bwd(d_topk_weights, logits, topk_ids, *, score: str = "softmax",
                       renormalize: bool = True, scale: float = 1.0):
    """d_logits [T, E] from d_topk_weights [T, K], the forward's logits and its
    topk_ids.  ``score``, ``renormalize`` and ``scale`` are the forward's; bias
    and groups only enter the selection, which has no gradient."""
    lib = load_library()
    _require_gpu(d_topk_weights, topk_ids)
    _same_device(logits, d_topk_weights, topk_ids)
    if topk_ids.dim() != 2 or logits.dim() != 2 or topk_ids.shape[0] != logits.shape[0]:
        raise MoEFFNError(2, "expected logits [T, E] and topk_ids [T, K]")
    if d_topk_weights.dtype != torch.float32 or d_topk_weights.shape != topk_ids.shape:
        raise MoEFFNError(3, "d_topk_weights must be float32 with the shape of topk_ids")
    r = _router(logits, topk_ids.shape[1], _ids_code(topk_ids), score, renormalize, 1, 1, 1, scale)
    dev = logits.device
    d_logits = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    _launch(lib.moe_ffn_router_bwd, dev, r, d_topk_weights.data_ptr(), logits.data_ptr(),
            topk_ids.data_ptr(), d_logits.data_ptr())
    return d_logits


class MoERouterFunction(torch.autograd.Function):
    """Autograd wrapper of the router: topk_weights is differentiable in logits;
    topk_ids and the selection are not."""

    @staticmethod
    def forward(ctx, logits, K, bias, score, renormalize, groups, topk_groups, group_top, scale,
                ids_dtype):
        weights, ids = moe_ffn_router_fwd(logits, K, bias=bias, score=score,
                                          renormalize=renormalize, groups=groups,
                                          topk_groups=topk_groups, group_top=group_top,
                                          scale=scale, ids_dtype=ids_dtype)
        ctx.save_for_backward(logits, ids)
        ctx.form = dict(score=score, renormalize=renormalize, scale=scale)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, d_weights, _):
        logits, ids = ctx.saved_tensors
        d_logits = moe_ffn_router_bwd(d_weights.contiguous(), logits, ids, **ctx.form)
        return (d_logits,) + (None,) * 9


def moe_ffn_router(logits, K: int, *, bias=None, score: str = "softmax", renormalize: bool = True,
                   groups: int = 1, topk_groups: int = 1, group_top: int = 1, scale: float = 1.0,
                   ids_dtype=torch.int32):
    """(topk_weights, topk_ids) for ``moe_ffn``; differentiable in logits."""
    return MoERouterFunction.apply(logits, K, bias, score, renormalize, groups, topk_groups,
                                   group_top, scale, ids_dtype)


class MXFP4Weight:
    """Expert weights [E, Kd, N] packed by ``moe_ffn_mxfp4_quantize``: ``data`` (uint8, the
    library's layout), the sizes, the number of column panels and the dtype they came in."""

    def __init__(self, data, E, Kd, N, panels, dtype):
        self.data, self.E, self.Kd, self.N, self.panels, self.dtype = data, E, Kd, N, panels, dtype
        self._sized = self._nbytes = None

    @property
    def nbytes(self) -> int:
        """Bytes that ``data`` must hold."""
        sizes = (self.E, self.Kd, self.N, self.panels)
        if self._sized != sizes:
            self._nbytes = _mxfp4_weight_size(self._stack())
            self._sized = sizes
        return self._nbytes

    def _stack(self):
        return MXFP4Stack(self.E, self.Kd, self.N, self.panels, _dtype_code_of(self.dtype))


def _mxfp4_weight_size(stack) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_ffn_mxfp4_weight_size(ctypes.byref(stack), ctypes.byref(n)))
    return n.value


def moe_ffn_mxfp4_quantize(weight, panels: int = 1) -> MXFP4Weight:
    """Pack expert weights [E, Kd, N] (float32 or bfloat16) as MXFP4 with blocks of 32 along Kd.

    up_proj_weight [E, H, 2I] takes ``panels`` 2, down_proj_weight [E, I, H] 1."""
    lib = load_library()
    _require_gpu(weight)
    if weight.dim() != 3:
        raise MoEFFNError(2, "expected weight [E, Kd, N]")
    E, Kd, N = weight.shape
    stack = MXFP4Stack(E, Kd, N, panels, _dtype_code(weight))
    dev = weight.device
    data = torch.empty(_mxfp4_weight_size(stack), dtype=torch.uint8, device=dev)
    _launch(lib.moe_ffn_mxfp4_quantize, dev, stack, weight.data_ptr(), data.data_ptr(),
            data.numel())
    return MXFP4Weight(data, E, Kd, N, panels, weight.dtype)


def moe_ffn_mxfp4_dequantize(packed: MXFP4Weight):
    """The values [E, Kd, N] that ``packed`` stands for, in the dtype it was packed from."""
    lib = load_library()
    stack = packed._stack()
    _require_gpu(packed.data)
    dev = packed.data.device
    w = torch.empty((packed.E, packed.Kd, packed.N), dtype=packed.dtype, device=dev)
    _launch(lib.moe_ffn_mxfp4_dequantize, dev, stack, packed.data.data_ptr(),
            packed.data.numel(), w.data_ptr())
    return w


def _act_code(act: str) -> int:
    if act not in ACT_FORMATS:
        raise MoEFFNError(3, f"act must be one of {sorted(ACT_FORMATS)}, got {act!r}")
    return ACT_FORMATS[act]


def mxfp4_workspace_size(problem: Problem, act: str = "mxfp4", flags: int = 0) -> int:
    ws = ctypes.c_size_t()
    _check(load_library().moe_ffn_mxfp4_workspace_size(ctypes.byref(problem), _act_code(act),
                                                       flags, ctypes.byref(ws)))
    return ws.value


def moe_ffn_mxfp4_fwd(x, topk_ids, topk_weights, up: MXFP4Weight, down: MXFP4Weight, *,
                      act: str = "mxfp4", check_ids: bool = False, ws=None,
                      return_ws: bool = False, flags: int = 0):
    """y [T, H] of the layer on packed 4-bit weights (inference; include/moe_ffn.h,
    moe_ffn_mxfp4_fwd).

    ``act`` is the block format ("mxfp4" or "mxfp6") that the token rows and the SwiGLU output
    are quantised to before their product.  ``ws`` may pass a preallocated workspace (uint8, at
    least ``mxfp4_workspace_size`` bytes).

    There is no backward pass: with gradients enabled, ``x`` and ``topk_weights`` that require one
    are refused (call under ``torch.no_grad()``, or with detached tensors)."""
    lib = load_library()
    if torch.is_grad_enabled() and (x.requires_grad or topk_weights.requires_grad):
        raise MoEFFNError(3, "the MXFP4 forward has no gradient: x and topk_weights must not "
                             "require one")
    _require_gpu(x, topk_ids, topk_weights, up.data, down.data, ws)
    _same_device(x, topk_ids, topk_weights, up.data, down.data, ws)
    if x.dim() != 2 or topk_ids.dim() != 2 or topk_ids.shape[0] != x.shape[0]:
        raise MoEFFNError(2, "expected x [T, H] and topk_ids [T, K]")
    if topk_weights.dtype != torch.float32 or topk_weights.shape != topk_ids.shape:
        raise MoEFFNError(3, "topk_weights must be float32 with the shape of topk_ids")
    T, H = x.shape
    E, I = down.E, down.Kd
    if (up.E, up.Kd, up.N, up.panels) != (E, H, 2 * I, 2) or (down.N, down.panels) != (H, 1):
        raise MoEFFNError(2, "expected up packed from [E, H, 2I] with 2 panels and down from "
                             "[E, I, H] with 1")
    if up.data.nbytes < up.nbytes or down.data.nbytes < down.nbytes:
        raise MoEFFNError(5, "packed weights shorter than their sizes need")
    prob = Problem(T, H, I, E, topk_ids.shape[1], _dtype_code(x), _ids_code(topk_ids))
    flags |= CHECK_IDS if check_ids else 0
    dev = x.device
    if ws is None:
        ws = torch.empty(mxfp4_workspace_size(prob, act, flags), dtype=torch.uint8, device=dev)
    y = torch.empty_like(x)
    _launch(lib.moe_ffn_mxfp4_fwd, dev, prob, _act_code(act), x.data_ptr(), topk_ids.data_ptr(),
            topk_weights.data_ptr(), up.data.data_ptr(), down.data.data_ptr(), y.data_ptr(),
            ws.data_ptr(), ws.nbytes, flags)
    return (y, ws) if return_ws else y


def _require_rows(name, t):
    """A matrix on the GPU whose rows may be strided: the elements from one row to the next."""
    if not t.is_cuda:
        raise MoEFFNError(1, "all tensors must be on the GPU (no CPU fallback exists)")
    if t.dim() != 2:
        raise MoEFFNError(2, f"expected {name} with two dimensions")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise MoEFFNError(4, f"a row of {name} must be consecutive")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _require_offsets(offsets, E):
    _require_gpu(offsets)
    code = _ids_code_of(offsets.dtype)
    if offsets.shape != (E + 1,):
        raise MoEFFNError(2, f"expected offsets [E + 1] = [{E + 1}], got {tuple(offsets.shape)}")
    return code


def _workspace(ws, size, device, *args):
    """(tensor, address, bytes) of the caller's workspace, or of one of ``size(*args)`` bytes; the
    tensor must outlive the call."""
    if ws is None:
        n = size(*args)
        if n == 0:
            return None, None, 0
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    else:
        _require_gpu(ws)
        if ws.device != device:
            raise MoEFFNError(1, f"the workspace is on {ws.device}, the call on {device}")
    return ws, ws.data_ptr(), ws.nbytes


def _grouped(x, weight, offsets, transposed) -> Grouped:
    stride = _require_rows("x", x)
    _require_gpu(weight)
    if weight.dim() != 3:
        raise MoEFFNError(2, "expected weight [E, Kd, N], or [E, N, Kd] with transposed")
    E = weight.shape[0]
    code = _require_offsets(offsets, E)
    _same_device(x, weight, offsets)
    Kd, N = (weight.shape[2], weight.shape[1]) if transposed else weight.shape[1:]
    if x.shape[1] != Kd:
        raise MoEFFNError(2, f"x has {x.shape[1]} columns, weight contracts {Kd}")
    if x.dtype != weight.dtype:
        raise MoEFFNError(3, "x and weight must share one dtype")
    return Grouped(x.shape[0], E, Kd, N, stride, _dtype_code(x), code, 1 if transposed else 0)


def grouped_workspace_size(grouped: Grouped) -> int:
    ws = ctypes.c_size_t()
    _check(load_library().moe_ffn_grouped_workspace_size(ctypes.byref(grouped), ctypes.byref(ws)))
    return ws.value


def moe_ffn_grouped_mm_fwd(x, weight, offsets, *, transposed: bool = False, ws=None):
    """y [M, N]: rows offsets[e] <= m < offsets[e + 1] of x [M, Kd] times weight[e] of weight
    [E, Kd, N] (or, with ``transposed``, weight[e] transposed of [E, N, Kd]); rows outside every
    group are zero (include/moe_ffn.h, moe_ffn_grouped_mm).

    float32 or bfloat16; the rows of ``x`` may be strided, by a multiple of 8 elements.
    ``offsets`` [E + 1] are int32 or int64 and stay on the device.  ``ws`` may pass a preallocated
    workspace (uint8, at least ``grouped_workspace_size`` bytes)."""
    lib = load_library()
    g = _grouped(x, weight, offsets, transposed)
    dev = x.device
    ws = _workspace(ws, grouped_workspace_size, dev, g)
    y = torch.empty((g.M, g.N), dtype=x.dtype, device=dev)
    _launch(lib.moe_ffn_grouped_mm, dev, g, x.data_ptr(), weight.data_ptr(), offsets.data_ptr(),
            y.data_ptr(), ws[1], ws[2])
    return y


def moe_ffn_grouped_mm_bwd(dy, x, weight, offsets, *, transposed: bool = False,
                           need_dx: bool = True, need_dw: bool = True, ws=None):
    """(dx [M, Kd], d_weight) of ``moe_ffn_grouped_mm_fwd`` from dy [M, N]; None for what is not
    needed.  A row outside every group has dx zero and no part in d_weight; an empty group's
    d_weight is zero."""
    lib = load_library()
    g = _grouped(x, weight, offsets, transposed)
    _require_gpu(dy)
    _same_device(x, dy)
    if dy.shape != (g.M, g.N) or dy.dtype != x.dtype:
        raise MoEFFNError(2, f"expected dy [{g.M}, {g.N}] in the dtype of x")
    dev = x.device
    ws = _workspace(ws, grouped_workspace_size, dev, g)
    dx = torch.empty((g.M, g.Kd), dtype=x.dtype, device=dev) if need_dx else None
    dw = torch.empty_like(weight) if need_dw else None
    _launch(lib.moe_ffn_grouped_mm_bwd, dev, g, dy.data_ptr(), x.data_ptr(), weight.data_ptr(),
            offsets.data_ptr(), _ptr(dx), _ptr(dw), ws[1], ws[2])
    return dx, dw


class MoEGroupedMMFunction(torch.autograd.Function):
    """Autograd wrapper of the grouped product: differentiable in x and weight."""

    @staticmethod
    def forward(ctx, x, weight, offsets, transposed):
        ctx.save_for_backward(x, weight, offsets)
        ctx.transposed = transposed
        return moe_ffn_grouped_mm_fwd(x, weight, offsets, transposed=transposed)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, offsets = ctx.saved_tensors
        dx, dw = moe_ffn_grouped_mm_bwd(_own_gradient(dy), x, weight, offsets,
                                        transposed=ctx.transposed,
                                        need_dx=ctx.needs_input_grad[0],
                                        need_dw=ctx.needs_input_grad[1])
        return dx, dw, None, None


def moe_ffn_grouped_mm(x, weight, offsets, *, transposed: bool = False):
    """``moe_ffn_grouped_mm_fwd``, differentiable in x and weight."""
    return MoEGroupedMMFunction.apply(x, weight, offsets, transposed)


class Int8Weight:
    """Weights [E, Kd, N] packed by ``moe_ffn_int8_quantize`` or ``moe_ffn_int8_pack``: ``data``
    (uint8, the library's layout), the sizes, the number of column panels and the dtype that
    ``moe_ffn_int8_dequantize`` gives back."""

    def __init__(self, data, E, Kd, N, panels, dtype):
        self.data, self.E, self.Kd, self.N, self.panels, self.dtype = data, E, Kd, N, panels, dtype
        self._sized = self._nbytes = None

    @property
    def nbytes(self) -> int:
        """Bytes that ``data`` must hold."""
        sizes = (self.E, self.Kd, self.N, self.panels)
        if self._sized != sizes:
            self._nbytes = _int8_weight_size(self._stack())
            self._sized = sizes
        return self._nbytes

    def _stack(self):
        return Int8Stack(self.E, self.Kd, self.N, self.panels, _dtype_code_of(self.dtype))


class Int8Rows:
    """Token rows in int8: ``codes`` [M, Kd rounded up to 64] (int8, zeros behind Kd), ``scales``
    [M] (float32), ``Kd`` and the dtype of the rows they came from."""

    def __init__(self, codes, scales, Kd, dtype):
        self.codes, self.scales, self.Kd, self.dtype = codes, scales, Kd, dtype


def _int8_weight_size(stack) -> int:
    n = ctypes.c_size_t()
    _check(load_library().moe_ffn_int8_weight_size(ctypes.byref(stack), ctypes.byref(n)))
    return n.value


def _no_gradient(what, *ts):
    if torch.is_grad_enabled() and any(t.requires_grad for t in ts):
        raise MoEFFNError(3, f"{what} has no gradient: its inputs must not require one")


def moe_ffn_int8_quantize(weight, panels: int = 1) -> Int8Weight:
    """Pack weights [E, Kd, N] (float32 or bfloat16; [Kd, N] is a stack of one) as int8 with a
    scale for each column: max|w| / 127 along Kd, codes rounded to nearest even.

    up_proj_weight [E, H, 2I] of ``moe_ffn_int8_fwd`` takes ``panels`` 2, all else 1."""
    lib = load_library()
    _require_gpu(weight)
    if weight.dim() not in (2, 3):
        raise MoEFFNError(2, "expected weight [E, Kd, N] or [Kd, N]")
    E, Kd, N = weight.shape if weight.dim() == 3 else (1, *weight.shape)
    stack = Int8Stack(E, Kd, N, panels, _dtype_code(weight))
    dev = weight.device
    data = torch.empty(_int8_weight_size(stack), dtype=torch.uint8, device=dev)
    _launch(lib.moe_ffn_int8_quantize, dev, stack, weight.data_ptr(), data.data_ptr(),
            data.numel())
    return Int8Weight(data, E, Kd, N, panels, weight.dtype)


def moe_ffn_int8_pack(codes, scales, panels: int = 1, dtype=torch.bfloat16) -> Int8Weight:
    """Pack weights that are int8 already: ``codes`` [E, Kd, N] (int8) and ``scales`` [E, N]
    (float32), or [Kd, N] and [N].  ``dtype`` is the one that ``moe_ffn_int8_dequantize`` gives
    back."""
    lib = load_library()
    _require_gpu(codes, scales)
    _same_device(codes, scales)
    if codes.dim() not in (2, 3):
        raise MoEFFNError(2, "expected codes [E, Kd, N] or [Kd, N]")
    if codes.dtype != torch.int8 or scales.dtype != torch.float32:
        raise MoEFFNError(3, "codes must be int8 and scales float32")
    if scales.shape != codes.shape[:-2] + codes.shape[-1:]:
        raise MoEFFNError(2, "expected one scale for each column: [E, N], or [N] for [Kd, N]")
    E, Kd, N = codes.shape if codes.dim() == 3 else (1, *codes.shape)
    stack = Int8Stack(E, Kd, N, panels, _dtype_code_of(dtype))
    dev = codes.device
    data = torch.empty(_int8_weight_size(stack), dtype=torch.uint8, device=dev)
    _launch(lib.moe_ffn_int8_pack, dev, stack, codes.data_ptr(), scales.data_ptr(),
            data.data_ptr(), data.numel())
    return Int8Weight(data, E, Kd, N, panels, dtype)


def moe_ffn_int8_dequantize(packed: Int8Weight):
    """The values code * scale [E, Kd, N] that ``packed`` stands for, rounded to its dtype."""
    lib = load_library()
    stack = packed._stack()
    _require_gpu(packed.data)
    dev = packed.data.device
    w = torch.empty((packed.E, packed.Kd, packed.N), dtype=packed.dtype, device=dev)
    _launch(lib.moe_ffn_int8_dequantize, dev, stack, packed.data.data_ptr(), packed.data.nbytes,
            w.data_ptr())
    return w


def _row_bytes(Kd: int) -> int:
    """Bytes of a row's codes (moe_ffn_int8_row_bytes, without a call)."""
    return -(-Kd // 64) * 64


def moe_ffn_int8_quantize_rows(x) -> Int8Rows:
    """Token rows [M, Kd] (float32 or bfloat16; rows may be strided) as int8 with a scale for each
    row: max|x| / 127, codes rounded to nearest even."""
    lib = load_library()
    stride = _require_rows("x", x)
    _no_gradient("the int8 quantisation", x)
    M, Kd = x.shape
    dev = x.device
    codes = torch.empty((M, _row_bytes(Kd)), dtype=torch.int8, device=dev)
    scales = torch.empty(M, dtype=torch.float32, device=dev)
    _launch(lib.moe_ffn_int8_quantize_rows, dev, Int8RowsShape(M, Kd, stride, _dtype_code(x)),
            x.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return Int8Rows(codes, scales, Kd, x.dtype)


def int8_mm_workspace_size(product: Int8Product) -> int:
    ws = ctypes.c_size_t()
    _check(load_library().moe_ffn_int8_mm_workspace_size(ctypes.byref(product), ctypes.byref(ws)))
    return ws.value


def moe_ffn_int8_mm(x, weight: Int8Weight, offsets=None, *, out_dtype=None, ws=None):
    """y [M, N] of int8 token rows and int8 weights: the exact integer sum times the row's and the
    column's scale, in ``out_dtype`` (float32 or bfloat16; by default the dtype of the rows).

    ``x`` is an ``Int8Rows``, or a matrix [M, Kd] that is quantised first.  With ``offsets``
    [E + 1] (int32 or int64, on the device) rows offsets[e] <= m < offsets[e + 1] meet matrix e and
    rows outside every group are zero; without, the one matrix of a stack of one meets all rows.
    ``ws`` may pass a preallocated workspace (uint8, at least ``int8_mm_workspace_size`` bytes).
    There is no backward pass."""
    lib = load_library()
    rows = x if isinstance(x, Int8Rows) else moe_ffn_int8_quantize_rows(x)
    _require_gpu(rows.codes, rows.scales, weight.data)
    _same_device(rows.codes, rows.scales, weight.data, offsets)
    if rows.Kd != weight.Kd:
        raise MoEFFNError(2, f"the rows have {rows.Kd} values, the weight contracts {weight.Kd}")
    M = rows.codes.shape[0]
    if (rows.codes.dtype != torch.int8 or rows.scales.dtype != torch.float32
            or rows.scales.shape != (M,) or rows.codes.shape[1:] != (_row_bytes(rows.Kd),)):
        raise MoEFFNError(2, "the rows do not hold int8 codes [M, Kd rounded up to 64] and float32 "
                             "scales [M]")
    code = I32 if offsets is None else _require_offsets(offsets, weight.E)
    dtype = rows.dtype if out_dtype is None else out_dtype
    p = Int8Product(weight._stack(), M, code, _dtype_code_of(dtype))
    dev = weight.data.device
    ws = _workspace(ws, int8_mm_workspace_size, dev, p)
    y = torch.empty((M, weight.N), dtype=dtype, device=dev)
    _launch(lib.moe_ffn_int8_mm, dev, p, rows.codes.data_ptr(), rows.scales.data_ptr(),
            weight.data.data_ptr(), weight.data.nbytes, _ptr(offsets), y.data_ptr(), ws[1],
            ws[2])
    return y


def int8_workspace_size(problem: Problem, flags: int = 0) -> int:
    ws = ctypes.c_size_t()
    _check(load_library().moe_ffn_int8_workspace_size(ctypes.byref(problem), flags,
                                                      ctypes.byref(ws)))
    return ws.value


def moe_ffn_int8_fwd(x, topk_ids, topk_weights, up: Int8Weight, down: Int8Weight, *,
                     check_ids: bool = False, ws=None, return_ws: bool = False, flags: int = 0):
    """y [T, H] of the layer on packed int8 weights (inference; include/moe_ffn.h,
    moe_ffn_int8_fwd): token rows and the SwiGLU output are quantised row by row.

    ``ws`` may pass a preallocated workspace (uint8, at least ``int8_workspace_size`` bytes).
    There is no backward pass: with gradients enabled, ``x`` and ``topk_weights`` that require one
    are refused."""
    lib = load_library()
    _no_gradient("the int8 forward", x, topk_weights)
    _require_gpu(x, topk_ids, topk_weights, up.data, down.data, ws)
    _same_device(x, topk_ids, topk_weights, up.data, down.data, ws)
    if x.dim() != 2 or topk_ids.dim() != 2 or topk_ids.shape[0] != x.shape[0]:
        raise MoEFFNError(2, "expected x [T, H] and topk_ids [T, K]")
    if topk_weights.dtype != torch.float32 or topk_weights.shape != topk_ids.shape:
        raise MoEFFNError(3, "topk_weights must be float32 with the shape of topk_ids")
    T, H = x.shape
    E, I = down.E, down.Kd
    if (up.E, up.Kd, up.N, up.panels) != (E, H, 2 * I, 2) or (down.N, down.panels) != (H, 1):
        raise MoEFFNError(2, "expected up packed from [E, H, 2I] with 2 panels and down from "
                             "[E, I, H] with 1")
    if up.data.nbytes < up.nbytes or down.data.nbytes < down.nbytes:
        raise MoEFFNError(5, "packed weights shorter than their sizes need")
    prob = Problem(T, H, I, E, topk_ids.shape[1], _dtype_code(x), _ids_code(topk_ids))
    flags |= CHECK_IDS if check_ids else 0
    dev = x.device
    if ws is None:
        ws = torch.empty(int8_workspace_size(prob, flags), dtype=torch.uint8, device=dev)
    y = torch.empty_like(x)
    _launch(lib.moe_ffn_int8_fwd, dev, prob, x.data_ptr(), topk_ids.data_ptr(),
            topk_weights.data_ptr(), up.data.data_ptr(), down.data.data_ptr(), y.data_ptr(),
            ws.data_ptr(), ws.nbytes, flags)
    return (y, ws) if return_ws else y


def read_status(ws: torch.Tensor) -> int:
    """Device status word of the last forward/route on `ws` (DEV_BAD_ID | DEV_TIMEOUT bits)."""
    lib = load_library()
    st = ctypes.c_int32()
    with torch.cuda.device(ws.device):
        _check(lib.moe_ffn_read_status(_ptr(ws), _stream(ws.device), ctypes.byref(st)))
    return st.value


class EventPool:
    """hipEvents (through the library's helpers) for the per-stage timing hook."""

    def __init__(self, n_sets: int, n_stages: int = 5):
        self.lib = load_library()
        self.sets = []
        for _ in range(n_sets):
            ev = StageEvents()
            for s in range(n_stages):
                for arr in (ev.begin, ev.end):
                    h = ctypes.c_void_p()
                    _check(self.lib.moe_ffn_event_create(ctypes.byref(h)))
                    arr[s] = h
            self.sets.append(ev)
        self.n_stages = n_stages

    def elapsed_ms(self, i: int, stage: int) -> float:
        ms = ctypes.c_float()
        ev = self.sets[i]
        _check(self.lib.moe_ffn_event_elapsed_ms(ev.begin[stage], ev.end[stage], ctypes.byref(ms)))
        return ms.value

    def close(self):
        for ev in self.sets:
            for s in range(self.n_stages):
                for arr in (ev.begin, ev.end):
                    if arr[s]:
                        self.lib.moe_ffn_event_destroy(arr[s])
                        arr[s] = None
        self.sets = []
