"""Python binding of libmoe_mi355x.so, the MI355X (gfx950) routed-MoE FFN library.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  torch supplies device memory and the current stream.  The functions
carry the names of the C entry points in include/moe_mi355x.h; importing this
package raises ImportError when the library has not been built (there is no
fallback of any kind).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmoe_mi355x.so")

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_ALIGN = 0, -1, -2, -3
MOE_ERR_WORKSPACE, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP = -4, -5, -6
MOE_BF16, MOE_MXFP8, MOE_INT8, MOE_MXFP4 = 0, 1, 2, 3
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
KERNELS = {"none": 0, "route": 1, "decode_gate_up": 2, "decode_down": 3, "group": 4,
           "quant": 5, "gemm_gate_up": 6, "gemm_down": 7, "combine": 8, "bwd_gate_up": 9,
           "bwd_down": 10, "bwd_input": 11, "bwd_wdown": 12, "bwd_wgate_up": 13,
           "decode_fused": 14, "bwd_requant": 15, "norm": 16, "norm_backward": 17,
           "route_backward": 18, "int8_gate_up": 19, "int8_down": 20,
           "mxfp4_gate_up": 21, "mxfp4_down": 22, "balance": 23, "balance_backward": 24}
MOE_DEBUG_PERMUTE_ORDER, MOE_DEBUG_DECODE_FUSED = 1, 2

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_SIGS = {
    "moe_route_topk": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_decode_forward": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
    "moe_decode_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_decode_forward_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "moe_quantize_mxfp8": (_I, [_P, ctypes.c_int64, _I, _P, _P, _P]),
    "moe_gate_up_3d_batched": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "moe_down_3d_batched": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moe_backward_batched": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                  _P, _P, _SZ, _P]),
    "moe_gate_up_3d_batched_train": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "moe_backward_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_backward_batched_mxfp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P,
                                        _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_backward_mxfp8_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_add_rmsnorm": (_I, [_P, _P, _P, _I, _I, _F, _P, _P, _I, _P, _P, _P]),
    "moe_add_rmsnorm_backward": (_I, [_P, _P, _P, _P, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "moe_add_rmsnorm_backward_workspace_bytes": (_SZ, [_I, _I]),
    "moe_route_scored": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "moe_route_scored_backward": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _P]),
    "moe_quantize_int8": (_I, [_P, ctypes.c_int64, _I, _P, _P, _P]),
    "moe_experts_int8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_experts_int8_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "moe_quantize_mxfp4": (_I, [_P, ctypes.c_int64, _I, _P, _P, _P]),
    "moe_dequantize_mxfp4": (_I, [_P, _P, ctypes.c_int64, _I, _P, _P]),
    "moe_experts_mxfp4": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _SZ, _P]),
    "moe_experts_mxfp4_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "moe_balance_loss": (_I, [_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_balance_loss_workspace_bytes": (_SZ, [_I, _I, _I]),
    "moe_balance_loss_backward": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P]),
    "moe_profile_kernel": (_I, [_I, _P, _P]),
    "moe_set_debug_options": (_I, [ctypes.c_uint, ctypes.c_uint32]),
    "moe_status_string": (ctypes.c_char_p, [_I]),
    "moe_last_error": (ctypes.c_char_p, []),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python mixture_experts_ffn_07_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        detail = lib.moe_last_error().decode()
        super().__init__(f"{fn}: {lib.moe_status_string(status).decode()} ({status}): {detail}")


def _check(fn: str, status: int) -> None:
    if status != MOE_OK:
        raise MoeError(fn, status)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the library must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)   # 16-bit patterns read as BF16
_MASK = (torch.uint8, torch.bool)


def _u16(t: torch.Tensor) -> torch.Tensor:
    if t.dtype not in _BF16:
        raise TypeError(f"expected BF16 bits, got {t.dtype}")
    return t


def _need(t: Optional[torch.Tensor], name: str, shape, dtypes, optional: bool = False) -> None:
    """Check a tensor argument's shape and element type before any pointer is
    handed to the library (a wrong size would become an out-of-bounds device
    access; a wrong dtype, e.g. int64 indices, would be misread)."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(dtypes, tuple):
        dtypes = (dtypes,)
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {dtypes}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def _need_ws(ws: torch.Tensor, nbytes: int) -> None:
    if ws.dtype != torch.uint8 or ws.dim() != 1:
        raise TypeError("workspace must be a 1-D uint8 tensor")
    if ws.numel() < nbytes:
        raise ValueError(f"workspace holds {ws.numel()} bytes, {nbytes} required")


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A device buffer for the workspace argument (256-byte aligned by torch)."""
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


# Streams: a call runs on `stream`, a torch stream or a raw hipStream_t (None: the current
# one).  What it allocates itself, outputs and workspace, belongs to that stream.  Tensors
# that it is given stay the caller's matter: they have to be ready on that stream, and to
# live, or to be recorded on it, until its work has ended.
def _home(stream, dev):
    """The stream that owns what a call allocates: None for the current one, else the given
    one.  (Memory of the current stream could hold a tensor that its pending work still uses
    when the call's kernels start, and a workspace, once dropped, would go to the current
    stream's next tensor while they still run.)"""
    if stream is None or dev.type != "cuda":
        return None
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
    if handle == torch._C._cuda_getCurrentRawStream(dev.index):
        return None
    if isinstance(stream, torch.cuda.Stream):
        return stream
    return torch.cuda.ExternalStream(handle, device=dev) if handle else torch.cuda.default_stream(dev)


def _make(make, dev, stream) -> torch.Tensor:
    """make() as memory of a call on `stream`.  A tensor that belongs to another stream than
    the current one is known to the allocator as used on both: the caller may read it here,
    after the wait that this takes, and drop it."""
    home = _home(stream, dev)
    if home is None:
        return make()
    with torch.cuda.stream(home):
        t = make()
    t.record_stream(torch.cuda.current_stream(dev))
    return t


def _new(shape, dtype, dev, stream) -> torch.Tensor:
    """Memory for an output of a call on `stream`."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return _make(lambda: torch.empty(shape, dtype=dtype, device=dev), dev, stream)


def _new_ws(nbytes: int, dev, stream) -> torch.Tensor:
    """A workspace for a call on `stream` (the gate/up calls return theirs)."""
    return _make(lambda: workspace(nbytes, dev), dev, stream)


def moe_route_topk(logits: torch.Tensor, k: int, topk_idx: torch.Tensor = None,
                   topk_w: torch.Tensor = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """logits [T, E] float32 -> (topk_idx [T, k] int32, topk_w [T, k] float32)."""
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    T, E = logits.shape
    if logits.dtype != torch.float32:
        raise TypeError("logits must be float32")
    if topk_idx is None:
        topk_idx = _new((T, k), torch.int32, logits.device, stream)
    if topk_w is None:
        topk_w = _new((T, k), torch.float32, logits.device, stream)
    _need(topk_idx, "topk_idx", (T, k), torch.int32)
    _need(topk_w, "topk_w", (T, k), torch.float32)
    _check("moe_route_topk", lib.moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_idx),
                                                _ptr(topk_w), _stream(stream)))
    return topk_idx, topk_w


def moe_decode_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib.moe_decode_workspace_bytes(T, H, I, E, k))


def moe_workspace_bytes(T: int, H: int, I: int, E: int, k: int, dtype: int) -> int:
    return int(lib.moe_workspace_bytes(T, H, I, E, k, dtype))


def moe_decode_forward(x: torch.Tensor, logits: torch.Tensor, w_gate_up: torch.Tensor,
                       w_down: torch.Tensor, k: int, out: torch.Tensor = None,
                       topk_idx: torch.Tensor = None, topk_w: torch.Tensor = None,
                       ws: torch.Tensor = None, stream=None) -> torch.Tensor:
    """Whole layer for a decode batch (T <= 64); BF16 in and out."""
    T, H = x.shape
    E, I2, H2 = w_gate_up.shape
    I = I2 // 2
    if logits.shape != (T, E) or H2 != H or tuple(w_down.shape) != (E, H, I):
        raise ValueError("inconsistent shapes")
    _u16(x), _u16(w_gate_up), _u16(w_down)
    _need(logits, "logits", (T, E), torch.float32)
    if out is None:
        out = _new((T, H), torch.bfloat16, x.device, stream)
    _need(out, "out", (T, H), _BF16)
    _need(topk_idx, "topk_idx", (T, k), torch.int32, optional=True)
    _need(topk_w, "topk_w", (T, k), torch.float32, optional=True)
    need = moe_decode_workspace_bytes(T, H, I, E, k)
    if ws is None:
        ws = _new_ws(need, x.device, stream)
    _need_ws(ws, need)
    _check("moe_decode_forward", lib.moe_decode_forward(
        _ptr(x), _ptr(logits), _ptr(w_gate_up), _ptr(w_down), T, H, I, E, k, _ptr(out),
        _ptr(topk_idx), _ptr(topk_w), _ptr(ws), ws.numel(), _stream(stream)))
    return out


STATIC_SCRATCH_BYTES = 4 << 20      # MOE_STATIC_SCRATCH_BYTES


def moe_decode_forward_noalloc(x: torch.Tensor, logits: torch.Tensor, w_gate_up: torch.Tensor,
                               w_down: torch.Tensor, k: int, out: torch.Tensor,
                               topk_idx: torch.Tensor = None, topk_w: torch.Tensor = None,
                               stream=None) -> torch.Tensor:
    """moe_decode_forward without a workspace (the library's own scratch); the
    caller passes every output, so this call allocates nothing."""
    T, H = x.shape
    E, I2, H2 = w_gate_up.shape
    I = I2 // 2
    if logits.shape != (T, E) or H2 != H or tuple(w_down.shape) != (E, H, I):
        raise ValueError("inconsistent shapes")
    _u16(x), _u16(w_gate_up), _u16(w_down)
    _need(logits, "logits", (T, E), torch.float32)
    _need(out, "out", (T, H), _BF16)
    _need(topk_idx, "topk_idx", (T, k), torch.int32, optional=True)
    _need(topk_w, "topk_w", (T, k), torch.float32, optional=True)
    _check("moe_decode_forward_noalloc", lib.moe_decode_forward_noalloc(
        _ptr(x), _ptr(logits), _ptr(w_gate_up), _ptr(w_down), T, H, I, E, k, _ptr(out),
        _ptr(topk_idx), _ptr(topk_w), _stream(stream)))
    return out


def moe_quantize_mxfp8(src: torch.Tensor, codes: torch.Tensor = None, scales: torch.Tensor = None,
                       stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """src [rows, K] BF16 -> (E4M3 codes [rows, K] uint8, E8M0 scales [rows, K/32] uint8)."""
    rows, K = src.shape
    _u16(src)
    if codes is None:
        codes = _new((rows, K), torch.uint8, src.device, stream)
    if scales is None:
        scales = _new((rows, K // 32), torch.uint8, src.device, stream)
    _need(codes, "codes", (rows, K), torch.uint8)
    _need(scales, "scales", (rows, K // 32), torch.uint8)
    _check("moe_quantize_mxfp8", lib.moe_quantize_mxfp8(_ptr(src), rows, K, _ptr(codes),
                                                        _ptr(scales), _stream(stream)))
    return codes, scales


def moe_gate_up_3d_batched(x, w_gate_up, topk_idx, k: int, dtype: int = MOE_BF16, x_scales=None,
                           w_gate_up_scales=None, h=None, h_scales=None, ws=None, stream=None):
    """Grouped gate/up projection + SwiGLU; returns (h, h_scales, ws)."""
    T, H = x.shape
    E, I2, H2 = w_gate_up.shape
    I = I2 // 2
    if H2 != H:
        raise ValueError("w_gate_up must be [E, 2I, H] with the H of x")
    mx = dtype == MOE_MXFP8
    edt = torch.uint8 if mx else _BF16
    _need(x, "x", (T, H), edt)
    _need(w_gate_up, "w_gate_up", (E, I2, H), edt)
    _need(topk_idx, "topk_idx", (T, k), torch.int32)
    if mx:
        _need(x_scales, "x_scales", (T, H // 32), torch.uint8)
        _need(w_gate_up_scales, "w_gate_up_scales", (E, I2, H // 32), torch.uint8)
    if h is None:
        h = _new((T * k, I), torch.bfloat16 if dtype == MOE_BF16 else torch.uint8, x.device, stream)
    if mx and h_scales is None:
        h_scales = _new((T * k, I // 32), torch.uint8, x.device, stream)
    _need(h, "h", (T * k, I), edt)
    if mx:
        _need(h_scales, "h_scales", (T * k, I // 32), torch.uint8)
    need = moe_workspace_bytes(T, H, I, E, k, dtype)
    if ws is None:
        ws = _new_ws(need, x.device, stream)
    _need_ws(ws, need)
    _check("moe_gate_up_3d_batched", lib.moe_gate_up_3d_batched(
        _ptr(x), _ptr(x_scales), _ptr(w_gate_up), _ptr(w_gate_up_scales), _ptr(topk_idx),
        T, H, I, E, k, dtype, _ptr(h), _ptr(h_scales), _ptr(ws), ws.numel(), _stream(stream)))
    return h, h_scales, ws


def moe_down_3d_batched(h, w_down, topk_idx, topk_w, ws, k: int, dtype: int = MOE_BF16,
                        h_scales=None, w_down_scales=None, out=None, stream=None):
    """Grouped down projection + fixed-order weighted combine -> out [T, H] BF16."""
    T = topk_idx.shape[0]
    E, H, I = w_down.shape
    mx = dtype == MOE_MXFP8
    edt = torch.uint8 if mx else _BF16
    _need(topk_idx, "topk_idx", (T, k), torch.int32)
    _need(topk_w, "topk_w", (T, k), torch.float32)
    _need(h, "h", (T * k, I), edt)
    _need(w_down, "w_down", (E, H, I), edt)
    if mx:
        _need(h_scales, "h_scales", (T * k, I // 32), torch.uint8)
        _need(w_down_scales, "w_down_scales", (E, H, I // 32), torch.uint8)
    if out is None:
        out = _new((T, H), torch.bfloat16, h.device, stream)
    _need(out, "out", (T, H), _BF16)
    _need_ws(ws, moe_workspace_bytes(T, H, I, E, k, dtype))
    _check("moe_down_3d_batched", lib.moe_down_3d_batched(
        _ptr(h), _ptr(h_scales), _ptr(w_down), _ptr(w_down_scales), _ptr(topk_idx),
        _ptr(topk_w), T, H, I, E, k, dtype, _ptr(out), _ptr(ws), ws.numel(), _stream(stream)))
    return out


def moe_backward_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib.moe_backward_workspace_bytes(T, H, I, E, k))


def moe_gate_up_3d_batched_train(x, w_gate_up, topk_idx, k: int, h=None, gu=None, ws=None,
                                 stream=None):
    """moe_gate_up_3d_batched (BF16) that also returns the FP32 pre-activations;
    returns (h, gu, ws)."""
    T, H = x.shape
    E, I2, _ = w_gate_up.shape
    I = I2 // 2
    _need(x, "x", (T, H), _BF16)
    _need(w_gate_up, "w_gate_up", (E, I2, H), _BF16)
    _need(topk_idx, "topk_idx", (T, k), torch.int32)
    if h is None:
        h = _new((T * k, I), torch.bfloat16, x.device, stream)
    if gu is None:
        gu = _new((T * k, I2), torch.float32, x.device, stream)
    _need(h, "h", (T * k, I), _BF16)
    _need(gu, "gu", (T * k, I2), torch.float32)
    need = moe_workspace_bytes(T, H, I, E, k, MOE_BF16)
    if ws is None:
        ws = _new_ws(need, x.device, stream)
    _need_ws(ws, need)
    _check("moe_gate_up_3d_batched_train", lib.moe_gate_up_3d_batched_train(
        _ptr(x), _ptr(w_gate_up), _ptr(topk_idx), T, H, I, E, k, _ptr(h), _ptr(gu), _ptr(ws),
        ws.numel(), _stream(stream)))
    return h, gu, ws


def moe_backward_batched(x, w_gate_up, w_down, topk_idx, topk_w, dout, k: int, gu_saved=None,
                         dx=None, dw_gate_up=None, dw_down=None, d_topk_w=None, dlogits=None,
                         ws=None, stream=None):
    """Backward pass of the layer (BF16); returns (dx, dw_gate_up, dw_down, d_topk_w, dlogits)."""
    T, H = x.shape
    E, I2, _ = w_gate_up.shape
    I = I2 // 2
    dev = x.device
    _need(x, "x", (T, H), _BF16)
    _need(w_gate_up, "w_gate_up", (E, I2, H), _BF16)
    _need(w_down, "w_down", (E, H, I), _BF16)
    _need(topk_idx, "topk_idx", (T, k), torch.int32)
    _need(topk_w, "topk_w", (T, k), torch.float32)
    _need(dout, "dout", (T, H), _BF16)
    _need(gu_saved, "gu_saved", (T * k, I2), torch.float32, optional=True)
    if dx is None:
        dx = _new((T, H), torch.bfloat16, dev, stream)
    if dw_gate_up is None:
        dw_gate_up = _new((E, I2, H), torch.bfloat16, dev, stream)
    if dw_down is None:
        dw_down = _new((E, H, I), torch.bfloat16, dev, stream)
    if d_topk_w is None:
        d_topk_w = _new((T, k), torch.float32, dev, stream)
    if dlogits is None:
        dlogits = _new((T, E), torch.float32, dev, stream)
    _need(dx, "dx", (T, H), _BF16)
    _need(dw_gate_up, "dw_gate_up", (E, I2, H), _BF16)
    _need(dw_down, "dw_down", (E, H, I), _BF16)
    _need(d_topk_w, "d_topk_w", (T, k), torch.float32)
    _need(dlogits, "dlogits", (T, E), torch.float32)
    need = moe_backward_workspace_bytes(T, H, I, E, k)
    if ws is None:
        ws = _new_ws(need, dev, stream)
    _need_ws(ws, need)
    _check("moe_backward_batched", lib.moe_backward_batched(
        _ptr(x), _ptr(w_gate_up), _ptr(w_down), _ptr(topk_idx), _ptr(topk_w), _ptr(dout),
        _ptr(gu_saved), T, H, I, E, k, _ptr(dx), _ptr(dw_gate_up), _ptr(dw_down), _ptr(d_topk_w), _ptr(dlogits),
        _ptr(ws), ws.numel(), _stream(stream)))
    return dx, dw_gate_up, dw_down, d_topk_w, dlogits


def moe_set_debug_options(flags: int = 0, seed: int = 0) -> None:
    """Test options for this thread's later calls: MOE_DEBUG_PERMUTE_ORDER (permuted
    workgroup -> work-item order, seeded) and MOE_DEBUG_DECODE_FUSED (two-launch decode)."""
    _check("moe_set_debug_options", lib.moe_set_debug_options(int(flags), int(seed) & 0xFFFFFFFF))


def moe_backward_mxfp8_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib.moe_backward_mxfp8_workspace_bytes(T, H, I, E, k))


def moe_backward_batched_mxfp8(x, w_gate_up, w_gate_up_scales, w_down, w_down_scales, topk_idx,
                               topk_w, dout, k: int, dx=None, dw_gate_up=None, dw_down=None,
                               d_topk_w=None, dlogits=None, ws=None, stream=None):
    """Backward pass of the MXFP8 layer; returns (dx, dw_gate_up, dw_down, d_topk_w, dlogits)."""
    T, H = x.shape
    E, I2, _ = w_gate_up.shape
    I = I2 // 2
    dev = x.device
    _need(x, "x", (T, H), _BF16)
    _need(w_gate_up, "w_gate_up", (E, I2, H), torch.uint8)
    _need(w_gate_up_scales, "w_gate_up_scales", (E, I2, H // 32), torch.uint8)
    _need(w_down, "w_down", (E, H, I), torch.uint8)
    _need(w_down_scales, "w_down_scales", (E, H, I // 32), torch.uint8)
    _need(topk_idx, "topk_idx", (T, k), torch.int32)
    _need(topk_w, "topk_w", (T, k), torch.float32)
    _need(dout, "dout", (T, H), _BF16)
    if dx is None:
        dx = _new((T, H), torch.bfloat16, dev, stream)
    if dw_gate_up is None:
        dw_gate_up = _new((E, I2, H), torch.bfloat16, dev, stream)
    if dw_down is None:
        dw_down = _new((E, H, I), torch.bfloat16, dev, stream)
    if d_topk_w is None:
        d_topk_w = _new((T, k), torch.float32, dev, stream)
    if dlogits is None:
        dlogits = _new((T, E), torch.float32, dev, stream)
    _need(dx, "dx", (T, H), _BF16)
    _need(dw_gate_up, "dw_gate_up", (E, I2, H), _BF16)
    _need(dw_down, "dw_down", (E, H, I), _BF16)
    _need(d_topk_w, "d_topk_w", (T, k), torch.float32)
    _need(dlogits, "dlogits", (T, E), torch.float32)
    need = moe_backward_mxfp8_workspace_bytes(T, H, I, E, k)
    if ws is None:
        ws = _new_ws(need, dev, stream)
    _need_ws(ws, need)
    _check("moe_backward_batched_mxfp8", lib.moe_backward_batched_mxfp8(
        _ptr(x), _ptr(w_gate_up), _ptr(w_gate_up_scales), _ptr(w_down), _ptr(w_down_scales),
        _ptr(topk_idx), _ptr(topk_w), _ptr(dout), T, H, I, E, k, _ptr(dx), _ptr(dw_gate_up),
        _ptr(dw_down), _ptr(d_topk_w), _ptr(dlogits), _ptr(ws), ws.numel(), _stream(stream)))
    return dx, dw_gate_up, dw_down, d_topk_w, dlogits


# The calls below check each tensor once (a 20-microsecond step is a handful of them: the
# checks and the stream look-up of the calls above cost about 5 us of host time a call,
# these about 2).

def _arg(t, name: str, shape, dtypes, dev) -> Optional[int]:
    """The device pointer of a tensor argument, after checking its element type, shape,
    device and layout (None stays None: the library names what it requires)."""
    if t is None:
        return None
    if t.dtype is not dtypes and not (isinstance(dtypes, tuple) and t.dtype in dtypes):
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtypes}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the call on {dev}: one call takes one device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _gpu(t: torch.Tensor, dims: int, name: str):
    """The GPU that a call runs on: the one of its first tensor."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {t.dim()}")
    return t.device


def _enqueue(name: str, dev, stream, *args) -> None:
    """Call the entry point on the given stream (None: the device's current one), with the
    tensors' device current: the library launches on the current device."""
    if dev.type != "cuda":
        raise ValueError("tensors passed to the library must live on the GPU")
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev.index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        status = getattr(lib, name)(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = getattr(lib, name)(*args, stream)
    if status != MOE_OK:
        raise MoeError(name, status)


def moe_add_rmsnorm(x, weight, eps: float, residual=None, residual_out=None, y=None,
                    qtype: int = MOE_BF16, codes=None, scales=None, stream=None):
    """Residual sum and RMS norm of [T, H] rows; returns (residual_out, y, codes, scales).

    qtype MOE_BF16: y (BF16) only; MOE_MXFP8 / MOE_INT8: codes and scales, and y where a
    buffer for it is given.  residual_out is allocated when a residual is given without it,
    and None without a residual."""
    dev = _gpu(x, 2, "x")
    shape = T, H = x.shape
    px = _arg(x, "x", shape, _BF16, dev)
    pw = _arg(weight, "weight", (H,), _BF16, dev)
    pr = _arg(residual, "residual", shape, _BF16, dev)
    if residual_out is None and residual is not None:
        residual_out = _new(shape, torch.bfloat16, dev, stream)
    ps = _arg(residual_out, "residual_out", shape, _BF16, dev)
    if y is None and qtype == MOE_BF16:
        y = _new(shape, torch.bfloat16, dev, stream)
    py = _arg(y, "y", shape, _BF16, dev)
    pc = pq = None
    if qtype == MOE_BF16:
        codes = scales = None
    else:
        if qtype == MOE_MXFP8:
            cdt, sdt, sshape = torch.uint8, torch.uint8, (T, H // 32)
        else:
            cdt, sdt, sshape = torch.int8, torch.float32, (T,)
        if codes is None:
            codes = _new(shape, cdt, dev, stream)
        if scales is None:
            scales = _new(sshape, sdt, dev, stream)
        pc = _arg(codes, "codes", shape, cdt, dev)
        pq = _arg(scales, "scales", sshape, sdt, dev)
    _enqueue("moe_add_rmsnorm", dev, stream, px, pr, pw, T, H, eps, ps, py, qtype, pc, pq)
    return residual_out, y, codes, scales


def moe_add_rmsnorm_backward_workspace_bytes(T: int, H: int) -> int:
    return int(lib.moe_add_rmsnorm_backward_workspace_bytes(T, H))


def _ws_arg(ws, nbytes, dev, stream):
    """(workspace, pointer, bytes): the caller's workspace, or a new one of nbytes (nbytes None: a
    workspace is given, and the library checks its size).  Who calls
    holds the tensor until the kernels are enqueued: dropped before, its memory could be given
    to work of another thread that is enqueued ahead of them, or be unmapped."""
    if ws is None:
        ws = _new_ws(nbytes, dev, stream)
    _need_ws(ws, nbytes or 0)
    return ws, _arg(ws, "workspace", ws.shape, torch.uint8, dev), ws.numel()


def moe_add_rmsnorm_backward(s, weight, dy, eps: float, ds=None, dx=None, dweight=None, ws=None,
                             stream=None):
    """Gradients of moe_add_rmsnorm from its residual sum s (x without a residual); ds is the
    gradient that reaches s from elsewhere.  Returns (dx, dweight); dx is the gradient of x
    and of the residual."""
    dev = _gpu(s, 2, "s")
    shape = T, H = s.shape
    if dx is None:
        dx = _new(shape, torch.bfloat16, dev, stream)
    if dweight is None:
        dweight = _new((H,), torch.bfloat16, dev, stream)
    ptrs = (_arg(s, "s", shape, _BF16, dev), _arg(weight, "weight", (H,), _BF16, dev),
            _arg(dy, "dy", shape, _BF16, dev), _arg(ds, "ds", shape, _BF16, dev))
    outs = _arg(dx, "dx", shape, _BF16, dev), _arg(dweight, "dweight", (H,), _BF16, dev)
    ws, pws, n = _ws_arg(ws, moe_add_rmsnorm_backward_workspace_bytes(T, H), dev, stream)
    _enqueue("moe_add_rmsnorm_backward", dev, stream, *ptrs, T, H, eps, *outs, pws, n)
    return dx, dweight


def moe_route_scored(logits, k: int, bias=None, score: int = MOE_SCORE_SOFTMAX, n_groups: int = 1,
                     topk_groups: int = 1, group_top: int = 1, renormalize: bool = True,
                     scale: float = 1.0, topk_idx=None, topk_w=None, stream=None):
    """logits [T, E] float32 (-inf masks an expert), bias [E] float32 or None ->
    (topk_idx [T, k] int32, topk_w [T, k] float32)."""
    dev = _gpu(logits, 2, "logits")
    T, E = logits.shape
    shape = (T, max(k, 0))
    if topk_idx is None:
        topk_idx = _new(shape, torch.int32, dev, stream)
    if topk_w is None:
        topk_w = _new(shape, torch.float32, dev, stream)
    _enqueue("moe_route_scored", dev, stream, _arg(logits, "logits", (T, E), torch.float32, dev),
             _arg(bias, "bias", (E,), torch.float32, dev), T, E, k, n_groups, topk_groups, group_top,
             score, 1 if renormalize else 0, scale,
             _arg(topk_idx, "topk_idx", shape, torch.int32, dev),
             _arg(topk_w, "topk_w", shape, torch.float32, dev))
    return topk_idx, topk_w


def moe_route_scored_backward(logits, topk_idx, d_topk_w, score: int = MOE_SCORE_SOFTMAX,
                              renormalize: bool = True, scale: float = 1.0, dlogits=None,
                              stream=None):
    """Gradient of moe_route_scored's weights (selection held fixed) -> dlogits [T, E] float32."""
    dev = _gpu(logits, 2, "logits")
    _gpu(topk_idx, 2, "topk_idx")
    T, E = logits.shape
    k = topk_idx.shape[1]
    if dlogits is None:
        dlogits = _new((T, E), torch.float32, dev, stream)
    _enqueue("moe_route_scored_backward", dev, stream,
             _arg(logits, "logits", (T, E), torch.float32, dev),
             _arg(topk_idx, "topk_idx", (T, k), torch.int32, dev),
             _arg(d_topk_w, "d_topk_w", (T, k), torch.float32, dev), T, E, k, score,
             1 if renormalize else 0, scale, _arg(dlogits, "dlogits", (T, E), torch.float32, dev))
    return dlogits


def moe_quantize_int8(src, codes=None, scales=None, stream=None):
    """src [rows, K] BF16 -> (codes [rows, K] int8, scales [rows] float32)."""
    dev = _gpu(src, 2, "src")
    rows, K = src.shape
    if codes is None:
        codes = _new((rows, K), torch.int8, dev, stream)
    if scales is None:
        scales = _new((rows,), torch.float32, dev, stream)
    _enqueue("moe_quantize_int8", dev, stream, _arg(src, "src", (rows, K), _BF16, dev), rows, K,
             _arg(codes, "codes", (rows, K), torch.int8, dev),
             _arg(scales, "scales", (rows,), torch.float32, dev))
    return codes, scales


def moe_experts_int8_workspace_bytes(T: int, H: int, I: int, E: int, k: int) -> int:
    return int(lib.moe_experts_int8_workspace_bytes(T, H, I, E, k))


def moe_experts_int8(x, x_scales, w_gate_up, w_gate_up_scales, w_down, w_down_scales, topk_idx,
                     topk_w, out=None, ws=None, stream=None):
    """The routed experts' FFN in INT8 (codes with per-token and per-channel scales) -> out
    [T, H] BF16.  Slots whose expert id lies outside [0, E) add nothing."""
    dev = _gpu(x, 2, "x")
    _gpu(w_gate_up, 3, "w_gate_up")
    _gpu(topk_idx, 2, "topk_idx")
    T, H = x.shape
    E, I2, _ = w_gate_up.shape
    I = I2 // 2
    k = topk_idx.shape[1]
    if out is None:
        out = _new((T, H), torch.bfloat16, dev, stream)
    i8, f32 = torch.int8, torch.float32
    ptrs = (_arg(x, "x", (T, H), i8, dev), _arg(x_scales, "x_scales", (T,), f32, dev),
            _arg(w_gate_up, "w_gate_up", (E, 2 * I, H), i8, dev),
            _arg(w_gate_up_scales, "w_gate_up_scales", (E, 2 * I), f32, dev),
            _arg(w_down, "w_down", (E, H, I), i8, dev),
            _arg(w_down_scales, "w_down_scales", (E, H), f32, dev),
            _arg(topk_idx, "topk_idx", (T, k), torch.int32, dev),
            _arg(topk_w, "topk_w", (T, k), f32, dev))
    pout = _arg(out, "out", (T, H), _BF16, dev)
    ws, pws, n = _ws_arg(ws, moe_experts_int8_workspace_bytes(T, H, I, E, k), dev, stream)
    _enqueue("moe_experts_int8", dev, stream, *ptrs, T, H, I, E, k, pout, pws, n)
    return out


def moe_quantize_mxfp4(src, codes=None, scales=None, stream=None):
    """src [rows, K] BF16 -> (E2M1 codes [rows, K/2] uint8, two to a byte with the even element
    in the low four bits, E8M0 scales [rows, K/32] uint8)."""
    dev = _gpu(src, 2, "src")
    rows, K = src.shape
    if codes is None:
        codes = _new((rows, K // 2), torch.uint8, dev, stream)
    if scales is None:
        scales = _new((rows, K // 32), torch.uint8, dev, stream)
    _enqueue("moe_quantize_mxfp4", dev, stream, _arg(src, "src", (rows, K), _BF16, dev), rows, K,
             _arg(codes, "codes", (rows, K // 2), torch.uint8, dev),
             _arg(scales, "scales", (rows, K // 32), torch.uint8, dev))
    return codes, scales


def moe_dequantize_mxfp4(codes, scales, out=None, stream=None):
    """MXFP4 rows (codes [rows, K/2] and scales [rows, K/32], uint8) -> their values [rows, K] BF16."""
    dev = _gpu(codes, 2, "codes")
    rows, K = codes.shape[0], 2 * codes.shape[1]
    if out is None:
        out = _new((rows, K), torch.bfloat16, dev, stream)
    _enqueue("moe_dequantize_mxfp4", dev, stream, _arg(codes, "codes", (rows, K // 2), torch.uint8, dev),
             _arg(scales, "scales", (rows, K // 32), torch.uint8, dev), rows, K,
             _arg(out, "out", (rows, K), _BF16, dev))
    return out


def moe_experts_mxfp4_workspace_bytes(T: int, H: int, I: int, E: int, k: int, xtype: int = MOE_MXFP8) -> int:
    return int(lib.moe_experts_mxfp4_workspace_bytes(T, H, I, E, k, xtype))


def moe_experts_mxfp4(x, x_scales, w_gate_up, w_gate_up_scales, w_down, w_down_scales, topk_idx,
                      topk_w, xtype: int = MOE_MXFP8, out=None, ws=None, stream=None):
    """The routed experts' FFN with MXFP4 weights ([E, 2I, H/2] and [E, H, I/2] bytes) -> out
    [T, H] BF16.  xtype MOE_MXFP8: x [T, H] E4M3 codes; MOE_MXFP4: x [T, H/2] bytes; scales
    [.., K/32].  Slots whose expert id lies outside [0, E) add nothing."""
    dev = _gpu(x, 2, "x")
    _gpu(w_down, 3, "w_down")
    _gpu(topk_idx, 2, "topk_idx")
    T, k = topk_idx.shape
    E, H, I = w_down.shape[0], w_down.shape[1], 2 * w_down.shape[2]
    if out is None:
        out = _new((T, H), torch.bfloat16, dev, stream)
    u8, f32 = torch.uint8, torch.float32
    ptrs = (_arg(x, "x", (T, H // 2 if xtype == MOE_MXFP4 else H), u8, dev),
            _arg(x_scales, "x_scales", (T, H // 32), u8, dev), xtype,
            _arg(w_gate_up, "w_gate_up", (E, 2 * I, H // 2), u8, dev),
            _arg(w_gate_up_scales, "w_gate_up_scales", (E, 2 * I, H // 32), u8, dev),
            _arg(w_down, "w_down", (E, H, I // 2), u8, dev),
            _arg(w_down_scales, "w_down_scales", (E, H, I // 32), u8, dev),
            _arg(topk_idx, "topk_idx", (T, k), torch.int32, dev),
            _arg(topk_w, "topk_w", (T, k), f32, dev))
    pout = _arg(out, "out", (T, H), _BF16, dev)
    need = moe_experts_mxfp4_workspace_bytes(T, H, I, E, k, xtype) if ws is None else None
    ws, pws, n = _ws_arg(ws, need, dev, stream)
    _enqueue("moe_experts_mxfp4", dev, stream, *ptrs, T, H, I, E, k, pout, pws, n)
    return out


def moe_balance_loss_workspace_bytes(T: int, E: int, n_seqs: int = 1) -> int:
    return int(lib.moe_balance_loss_workspace_bytes(T, E, n_seqs))


def moe_balance_loss(logits, topk_idx, score: int = MOE_SCORE_SOFTMAX, n_seqs: int = 1, token_mask=None,
                     losses=None, counts=None, probs=None, tokens=None, ws=None, stream=None):
    """The router's balance loss and z-loss of logits [T, E] float32 and topk_idx [T, k] int32, over
    n_seqs sequences of T / n_seqs tokens; token_mask [T] uint8 or bool (0: no part) or None.  Returns
    (losses [2] float32, counts [n_seqs, E] int32, mean scores [n_seqs, E] float32, tokens [n_seqs]
    int32)."""
    dev = _gpu(logits, 2, "logits")
    _gpu(topk_idx, 2, "topk_idx")
    T, E = logits.shape
    k, S = topk_idx.shape[1], max(n_seqs, 0)
    f32, i32 = torch.float32, torch.int32
    if losses is None:
        losses = _new((2,), f32, dev, stream)
    if counts is None:
        counts = _new((S, E), i32, dev, stream)
    if probs is None:
        probs = _new((S, E), f32, dev, stream)
    if tokens is None:
        tokens = _new((S,), i32, dev, stream)
    ptrs = (_arg(logits, "logits", (T, E), f32, dev), _arg(topk_idx, "topk_idx", (T, k), i32, dev),
            _arg(token_mask, "token_mask", (T,), _MASK, dev))
    outs = (_arg(losses, "losses", (2,), f32, dev), _arg(counts, "counts", (S, E), i32, dev),
            _arg(probs, "probs", (S, E), f32, dev), _arg(tokens, "tokens", (S,), i32, dev))
    need = moe_balance_loss_workspace_bytes(T, E, n_seqs) if ws is None else None
    ws, pws, n = _ws_arg(ws, need, dev, stream)
    _enqueue("moe_balance_loss", dev, stream, *ptrs, T, E, k, n_seqs, score, *outs, pws, n)
    return losses, counts, probs, tokens


def moe_balance_loss_backward(logits, counts, tokens, d_losses, score: int = MOE_SCORE_SOFTMAX,
                              token_mask=None, d_add=None, dlogits=None, stream=None):
    """Gradient of d_losses . losses of moe_balance_loss (counts [n_seqs, E] and tokens [n_seqs] as it
    returned them; d_losses [2] on the GPU), added to d_add [T, E] if given -> dlogits [T, E] float32
    (which may be d_add)."""
    dev = _gpu(logits, 2, "logits")
    _gpu(counts, 2, "counts")
    T, E = logits.shape
    S = counts.shape[0]
    f32, i32 = torch.float32, torch.int32
    if dlogits is None:
        dlogits = _new((T, E), f32, dev, stream)
    _enqueue("moe_balance_loss_backward", dev, stream, _arg(logits, "logits", (T, E), f32, dev),
             _arg(token_mask, "token_mask", (T,), _MASK, dev), _arg(counts, "counts", (S, E), i32, dev),
             _arg(tokens, "tokens", (S,), i32, dev), _arg(d_losses, "d_losses", (2,), f32, dev),
             _arg(d_add, "d_add", (T, E), f32, dev), T, E, S, score,
             _arg(dlogits, "dlogits", (T, E), f32, dev))
    return dlogits


def moe_profile_kernel(kernel, start_event: Optional[int], stop_event: Optional[int]) -> None:
    """Bracket the named kernel's launches with the given hipEvent_t handles."""
    kid = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    _check("moe_profile_kernel", lib.moe_profile_kernel(kid, start_event, stop_event))


__all__ = ["lib", "LIB_PATH", "MoeError", "moe_route_topk", "moe_decode_forward",
           "moe_decode_forward_noalloc", "STATIC_SCRATCH_BYTES",
           "moe_decode_workspace_bytes", "moe_workspace_bytes", "moe_quantize_mxfp8",
           "moe_gate_up_3d_batched", "moe_down_3d_batched", "moe_gate_up_3d_batched_train",
           "moe_backward_batched",
           "moe_backward_workspace_bytes", "moe_backward_batched_mxfp8",
           "moe_backward_mxfp8_workspace_bytes", "moe_profile_kernel", "workspace",
           "moe_set_debug_options", "MOE_DEBUG_PERMUTE_ORDER", "MOE_DEBUG_DECODE_FUSED",
           "moe_add_rmsnorm", "moe_add_rmsnorm_backward",
           "moe_add_rmsnorm_backward_workspace_bytes", "moe_route_scored",
           "moe_route_scored_backward", "moe_quantize_int8", "moe_experts_int8",
           "moe_experts_int8_workspace_bytes", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID",
           "moe_quantize_mxfp4", "moe_dequantize_mxfp4", "moe_experts_mxfp4",
           "moe_experts_mxfp4_workspace_bytes", "moe_balance_loss",
           "moe_balance_loss_workspace_bytes", "moe_balance_loss_backward",
           "MOE_BF16", "MOE_MXFP8", "MOE_INT8", "MOE_MXFP4", "KERNELS"]
