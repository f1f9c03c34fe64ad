"""Python binding of libmxmoe.so: an MXFP4-weight mixture-of-experts layer for MI355X.

Argument marshalling only: every step runs in the library's HIP kernels.
Tensors are torch tensors on the current HIP device; PyTorch provides device
memory and streams.  The library must be built first
(``python -m mxfp4_weight_mixture_amd.build``); importing this package
without it raises ImportError -- there is no other implementation to fall
back to.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxmoe.so")
ABI_VERSION = 3

# mirrors of include/mxmoe.h; checked against the library at import
STATUS = {"MOE_OK": 0, "MOE_ERR_INVALID_ARG": 1, "MOE_ERR_SHAPE": 2, "MOE_ERR_UNSUPPORTED_DEVICE": 3,
          "MOE_ERR_NOT_PINNED": 4, "MOE_ERR_WORKSPACE": 5, "MOE_ERR_HIP": 6, "MOE_ERR_NOT_IMPLEMENTED": 7}
ACT = {"MOE_ACT_BF16": 0, "MOE_ACT_MXFP8_E4M3": 1}
OUT = {"MOE_OUT_FP32": 0, "MOE_OUT_BF16": 1, "MOE_OUT_MXFP8_E4M3": 2}
EPI = {"MOE_EPI_NONE": 0, "MOE_EPI_SWIGLU_SPLIT": 1, "MOE_EPI_SWIGLU_INTERLEAVED": 2}
CHAIN = {"MOE_CHAIN_RMS": 0, "MOE_CHAIN_INDEPENDENT": 1}
WFORMAT = {"MOE_W_CANONICAL": 0, "MOE_W_TILED": 1}
COPY = {"MOE_COPY_ALL": 0, "MOE_COPY_ROUTED": 1, "MOE_COPY_AUTO": 2}
FLOAT = {"MOE_FLOAT_BF16": 0, "MOE_FLOAT_FP16": 1, "MOE_FLOAT_FP32": 2}
GATE = {"MOE_GATE_SILU": 0, "MOE_GATE_GELU": 1}
ENUM_KINDS = {0: STATUS, 1: ACT, 2: OUT, 3: EPI, 4: CHAIN, 5: WFORMAT, 6: COPY, 7: FLOAT, 8: GATE}
EXPERT_COPY = {"all": COPY["MOE_COPY_ALL"], "routed": COPY["MOE_COPY_ROUTED"], "auto": COPY["MOE_COPY_AUTO"]}
W_FORMAT = {"canonical": WFORMAT["MOE_W_CANONICAL"], "tiled": WFORMAT["MOE_W_TILED"]}

GATE_ACT = {"silu": GATE["MOE_GATE_SILU"], "gelu": GATE["MOE_GATE_GELU"]}
FLOAT_DTYPE = {torch.bfloat16: FLOAT["MOE_FLOAT_BF16"], torch.float16: FLOAT["MOE_FLOAT_FP16"],
               torch.float32: FLOAT["MOE_FLOAT_FP32"]}

LAYOUT = {"split": EPI["MOE_EPI_SWIGLU_SPLIT"], "interleaved": EPI["MOE_EPI_SWIGLU_INTERLEAVED"]}

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        name = {v: k for k, v in STATUS.items()}.get(status, str(status))
        super().__init__(f"{name}: {message}")


class GemmArgs(ctypes.Structure):
    _fields_ = [("a", _vp), ("a_scales", _vp), ("a_gather", _vp), ("w_packed", _vp), ("w_scales", _vp),
                ("expert_offsets", _vp), ("c", _vp), ("c_scales", _vp), ("a_dtype", _i32),
                ("a_gather_div", _i32), ("a_rows", _i32), ("rows", _i32), ("E", _i32), ("N", _i32),
                ("K", _i32), ("epilogue", _i32), ("c_dtype", _i32), ("w_format", _i32)]


class LayerArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("I", _i32), ("E", _i32), ("k", _i32), ("layout", _i32),
                ("act_dtype", _i32), ("inter_dtype", _i32), ("logits", _vp), ("x", _vp), ("x_scales", _vp),
                ("w1_packed", _vp), ("w1_scales", _vp), ("w2_packed", _vp), ("w2_scales", _vp),
                ("out", _vp), ("x_next", _vp), ("workspace", _vp), ("workspace_bytes", _sz), ("w_format", _i32)]


class StreamedArgs(ctypes.Structure):
    _fields_ = [("num_layers", _i32), ("T", _i32), ("H", _i32), ("I", _i32), ("E", _i32), ("k", _i32),
                ("layout", _i32), ("chain", _i32), ("depth", _i32), ("num_blobs", _i32),
                ("host_blobs", ctypes.POINTER(_vp)), ("blob_bytes", _sz), ("device_slot", _vp * 2),
                ("logits", _vp), ("x", _vp), ("out", _vp), ("layer_inputs", _vp), ("events", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz), ("w_format", _i32), ("expert_copy", _i32),
                ("routed_copy_max_tokens", _i32)]


class FfnArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("I", _i32), ("layout", _i32), ("gate_act", _i32), ("dtype", _i32),
                ("out_dtype", _i32), ("save_dtype", _i32), ("x", _vp), ("w1", _vp), ("w2", _vp), ("add", _vp),
                ("out", _vp), ("gate_up", _vp), ("x_stride", _i64), ("add_stride", _i64), ("out_stride", _i64),
                ("workspace", _vp), ("workspace_bytes", _sz)]


class FfnGradArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("H", _i32), ("I", _i32), ("layout", _i32), ("gate_act", _i32), ("dtype", _i32),
                ("save_dtype", _i32), ("dx_dtype", _i32), ("dw_dtype", _i32), ("accumulate", _i32), ("dout", _vp),
                ("x", _vp), ("w1", _vp), ("w2", _vp), ("gate_up", _vp), ("dx", _vp), ("dw1", _vp), ("dw2", _vp),
                ("dout_stride", _i64), ("x_stride", _i64), ("dx_stride", _i64), ("workspace", _vp),
                ("workspace_bytes", _sz)]


class AdapterArgs(ctypes.Structure):
    _fields_ = [("T", _i32), ("K", _i32), ("N", _i32), ("num_adapters", _i32), ("R", _i32), ("epilogue", _i32),
                ("gate_act", _i32), ("dtype", _i32), ("out_dtype", _i32), ("x", _vp), ("w", _vp), ("ids", _vp),
                ("a", _vp), ("b", _vp), ("scales", _vp), ("ranks", _vp), ("add", _vp), ("out", _vp),
                ("x_stride", _i64), ("add_stride", _i64), ("out_stride", _i64), ("workspace", _vp),
                ("workspace_bytes", _sz)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m mxfp4_weight_mixture_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    sigs = {
        "moe_abi_version": (ctypes.c_int, []),
        "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_last_error_message": (ctypes.c_char_p, []),
        "moe_enum_name": (ctypes.c_char_p, [ctypes.c_int, ctypes.c_int]),
        "moe_device_supported": (ctypes.c_int, []),
        "moe_route": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp]),
        "moe_permute_workspace_size": (_sz, [_i32, _i32, _i32]),
        "moe_permute": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
        "moe_grouped_gemm_workspace_size": (_sz, [ctypes.POINTER(GemmArgs)]),
        "moe_mxfp4_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(GemmArgs), _vp, _sz, _vp]),
        "moe_mxfp4_grouped_gemm_static": (ctypes.c_int, [ctypes.POINTER(GemmArgs), _vp]),
        "moe_combine": (ctypes.c_int, [_vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
        "moe_layer_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
        "moe_layer_workspace_offset": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32, _i32]),
        "moe_layer_forward": (ctypes.c_int, [ctypes.POINTER(LayerArgs), _vp]),
        "moe_blob_bytes": (_sz, [_i32, _i32, _i32]),
        "moe_blob_section_offset": (_sz, [_i32, _i32, _i32, _i32]),
        "moe_streamed_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32]),
        "moe_layer_prefill_streamed": (ctypes.c_int, [ctypes.POINTER(StreamedArgs), _vp, _vp]),
        "moe_tiled_weight_bytes": (_sz, [_i32, _i32, _i32, _i32]),
        "moe_mxfp4_tile_weights": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
        "moe_mxfp4_untile_weights": (ctypes.c_int, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
        "moe_layer_graph_create": (ctypes.c_int, [ctypes.POINTER(LayerArgs), _vp, ctypes.POINTER(_vp)]),
        "moe_layer_graph_launch": (ctypes.c_int, [_vp, _vp]),
        "moe_layer_graph_destroy": (ctypes.c_int, [_vp]),
        "moe_gated_ffn_workspace_size": (_sz, [_i32, _i32, _i32]),
        "moe_gated_ffn_forward": (ctypes.c_int, [ctypes.POINTER(FfnArgs), _vp]),
        "moe_gated_ffn_check": (ctypes.c_int, [ctypes.POINTER(FfnArgs)]),
        "moe_gated_ffn_grad_workspace_size": (_sz, [_i32, _i32, _i32]),
        "moe_gated_ffn_backward": (ctypes.c_int, [ctypes.POINTER(FfnGradArgs), _vp]),
        "moe_adapter_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32]),
        "moe_adapter_linear": (ctypes.c_int, [ctypes.POINTER(AdapterArgs), _vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.moe_abi_version() != ABI_VERSION:
        raise ImportError(f"libmxmoe ABI {lib.moe_abi_version()} != binding ABI {ABI_VERSION}")
    for kind, table in ENUM_KINDS.items():
        for name, value in table.items():
            got = lib.moe_enum_name(kind, value)
            if got is None or got.decode() != name:
                raise ImportError(f"enum mismatch: kind {kind} value {value}: library says {got}, binding {name}")
        if lib.moe_enum_name(kind, max(table.values()) + 1) is not None:
            raise ImportError(f"enum kind {kind} has values the binding does not know")
    return lib


lib = _load()


def _check(status: int):
    if status != 0:
        raise MoeError(status, (lib.moe_last_error_message() or b"").decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _u8(n: int, device) -> torch.Tensor:
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device=device)


_CURRENT = contextlib.nullcontext()


def _allocate_on(stream):
    """Context in which a call allocates its buffers: on the stream that uses them.

    The caching allocator gives a freed block out again at once, to allocations of the
    stream that the block belongs to: that stream's order protects what still runs.  A
    block of the current stream would reach `stream`, which does not wait for it, while
    earlier work of the current stream still uses it."""
    return _CURRENT if stream is None else torch.cuda.stream(stream)


def _keep_until_done(stream, *tensors):
    """A call's results, allocated on `stream` or given by the caller, and the inputs given with
    the call: both that stream and the current one, where the caller made them or goes on with
    them, use them.  Tell the caching allocator so, so that it does not hand their memory out
    again before either has finished, however soon the caller drops them."""
    if stream is None:
        return
    current = torch.cuda.current_stream(stream.device)
    if stream == current:
        return
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
            t.record_stream(current)


_COPY_STREAMS = {}


def _copy_stream_for(device) -> "torch.cuda.Stream":
    """One side stream per device for the streamed prefill's copies when the caller gives none."""
    idx = torch.device(device).index
    if idx is None:
        idx = torch.cuda.current_device()
    if idx not in _COPY_STREAMS:
        _COPY_STREAMS[idx] = torch.cuda.Stream(device=idx)
    return _COPY_STREAMS[idx]


def device_supported() -> bool:
    return lib.moe_device_supported() == 1


# ----------------------------------------------------------------- calls

def route(logits: torch.Tensor, k: int, stream=None):
    """moe_route: logits fp32 [T][E] -> (topk_ids int32 [T][k], topk_w fp32 [T][k])."""
    T, E = logits.shape
    with _allocate_on(stream):
        ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
        w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib.moe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _stream(stream)))
    _keep_until_done(stream, ids, w, logits)
    return ids, w


def permute(topk_ids: torch.Tensor, E: int, stream=None):
    """moe_permute: topk_ids [T][k] -> (expert_offsets [E+1], perm_src [T*k], dest_row [T*k])."""
    T, k = topk_ids.shape
    dev = topk_ids.device
    n = lib.moe_permute_workspace_size(T, E, k)
    with _allocate_on(stream):
        off = torch.empty(E + 1, dtype=torch.int32, device=dev)
        ps = torch.empty(T * k, dtype=torch.int32, device=dev)
        dr = torch.empty(T * k, dtype=torch.int32, device=dev)
        ws = _u8(n, dev)
    _check(lib.moe_permute(_ptr(topk_ids), T, E, k, _ptr(off), _ptr(ps), _ptr(dr), _ptr(ws), n,
                           _stream(stream)))
    _keep_until_done(stream, off, ps, dr, topk_ids)
    return off, ps, dr


def grouped_gemm(a: torch.Tensor, w_packed: torch.Tensor, w_scales: torch.Tensor,
                 expert_offsets: torch.Tensor, *, a_scales: Optional[torch.Tensor] = None,
                 a_gather: Optional[torch.Tensor] = None, a_gather_div: int = 1, rows: Optional[int] = None,
                 epilogue: str = "none", out_dtype: str = "bf16", w_format: str = "canonical",
                 stream=None) -> torch.Tensor:
    """moe_mxfp4_grouped_gemm.  a: bf16 [a_rows][K] or uint8 E4M3 codes (with a_scales).

    w_packed [E][N][K/2], w_scales [E][N][K/32].  Returns C [rows][N or N/2]
    (fp32 or bf16), or for out_dtype "mxfp8" the pair (E4M3 codes uint8
    [rows][N/2], E8M0 scales uint8 [rows][N/64]).
    """
    E, N, K2 = w_packed.shape
    K = 2 * K2
    if rows is None:
        rows = a_gather.numel() if a_gather is not None else a.shape[0]
    epi = {"none": 0, "split": 1, "interleaved": 2}[epilogue]
    n_out = N if epi == 0 else N // 2
    c_dt = {"fp32": 0, "bf16": 1, "mxfp8": 2}[out_dtype]
    c_scales = None
    with _allocate_on(stream):
        if c_dt == 2:
            c = torch.empty((rows, n_out), dtype=torch.uint8, device=a.device)
            c_scales = torch.empty((rows, n_out // 32), dtype=torch.uint8, device=a.device)
        else:
            c = torch.empty((rows, n_out), dtype=torch.float32 if c_dt == 0 else torch.bfloat16, device=a.device)
    args = GemmArgs(a=a.data_ptr(), a_scales=a_scales.data_ptr() if a_scales is not None else None,
                    a_gather=a_gather.data_ptr() if a_gather is not None else None,
                    w_packed=w_packed.data_ptr(), w_scales=w_scales.data_ptr(),
                    expert_offsets=expert_offsets.data_ptr(), c=c.data_ptr(),
                    c_scales=c_scales.data_ptr() if c_scales is not None else None,
                    a_dtype=1 if a_scales is not None else 0, a_gather_div=a_gather_div,
                    a_rows=a.shape[0], rows=rows, E=E, N=N, K=K, epilogue=epi, c_dtype=c_dt,
                    w_format=W_FORMAT[w_format])
    n = lib.moe_grouped_gemm_workspace_size(ctypes.byref(args))
    with _allocate_on(stream):
        ws = _u8(n, a.device)
    _check(lib.moe_mxfp4_grouped_gemm(ctypes.byref(args), _ptr(ws), n, _stream(stream)))
    _keep_until_done(stream, c, c_scales, a, w_packed, w_scales, expert_offsets, a_scales, a_gather)
    return (c, c_scales) if c_dt == 2 else c


def tile_weights(w_packed: torch.Tensor, w_scales: torch.Tensor, epilogue: str = "none", stream=None):
    """moe_mxfp4_tile_weights: canonical [E][N][K/2] + [E][N][K/32] -> the tiled order.

    Returns uint8 tensors of the same shapes (the bytes are reordered; the
    shapes only carry E, N, K).  epilogue: the one the matrix is used with."""
    E, N, K2 = w_packed.shape
    with _allocate_on(stream):
        tp, ts = torch.empty_like(w_packed), torch.empty_like(w_scales)
    _check(lib.moe_mxfp4_tile_weights(_ptr(w_packed), _ptr(w_scales), E, N, 2 * K2,
                                      {"none": 0, "split": 1, "interleaved": 2}[epilogue], _ptr(tp), _ptr(ts),
                                      _stream(stream)))
    _keep_until_done(stream, tp, ts, w_packed, w_scales)
    return tp, ts


def untile_weights(t_packed: torch.Tensor, t_scales: torch.Tensor, epilogue: str = "none", stream=None):
    """moe_mxfp4_untile_weights: the inverse of tile_weights."""
    E, N, K2 = t_packed.shape
    with _allocate_on(stream):
        wp, ws = torch.empty_like(t_packed), torch.empty_like(t_scales)
    _check(lib.moe_mxfp4_untile_weights(_ptr(t_packed), _ptr(t_scales), E, N, 2 * K2,
                                        {"none": 0, "split": 1, "interleaved": 2}[epilogue], _ptr(wp), _ptr(ws),
                                        _stream(stream)))
    _keep_until_done(stream, wp, ws, t_packed, t_scales)
    return wp, ws


def combine(y: torch.Tensor, dest_row: torch.Tensor, topk_w: torch.Tensor, *, rms_next: bool = False,
            stream=None):
    """moe_combine: y [T*k][H] (fp32 or bf16) -> out fp32 [T][H] (and bf16 x_next if rms_next)."""
    T, k = topk_w.shape
    H = y.shape[1]
    with _allocate_on(stream):
        out = torch.empty((T, H), dtype=torch.float32, device=y.device)
        xn = torch.empty((T, H), dtype=torch.bfloat16, device=y.device) if rms_next else None
    dt = 1 if y.dtype == torch.bfloat16 else 0
    _check(lib.moe_combine(_ptr(y), dt, _ptr(dest_row), _ptr(topk_w), T, k, H, _ptr(out), _ptr(xn),
                           _stream(stream)))
    _keep_until_done(stream, out, xn, y, dest_row, topk_w)
    return (out, xn) if rms_next else out


# --------------------------------------------- dense 16-bit projections

def _rows(name, t, rows, cols, dtypes, device):
    """Check a [rows][cols] tensor whose rows are contiguous; returns its row stride in elements."""
    if t.dim() != 2 or t.shape[1] != cols or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not ({'T' if rows is None else rows}, {cols})")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} is {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the weights on {device}")
    if t.stride(1) != 1:
        raise ValueError(f"{name}'s rows are not contiguous (strides {t.stride()})")
    return t.stride(0) if t.shape[0] > 1 else cols


def _flat(name, t, shape, dtypes, device):
    """Check a contiguous tensor of a given shape."""
    if tuple(t.shape) != tuple(shape) or t.dtype not in dtypes or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {' or '.join(str(d) for d in dtypes)} tensor of shape "
                         f"{tuple(shape)} on {device}: got {t.dtype} {tuple(t.shape)}, strides {t.stride()}, "
                         f"on {t.device}")
    return t


def _on_current_device(device, stream):
    """The library enqueues on the current device: refuse tensors and streams of another."""
    if torch.cuda.current_device() != device.index:
        raise ValueError(f"the weights are on {device}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the weights on {device}")


def _weight(name, w):
    if w.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"{name} is {w.dtype}, not torch.bfloat16 or torch.float16")
    if not w.is_cuda or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")


class GatedFFN:
    """The gated feed-forward block with 16-bit weights: a shared expert beside the routed ones, or a dense layer.

    out = (add +) (act(x Wg^T) * (x Wu^T)) W2^T with w1 [2I][H] holding Wg and Wu ("split": Wg's rows, then
    Wu's; "interleaved": row 2i of Wg, then of Wu), w2 [H][I]; act "silu" or "gelu" (tanh form).  bf16 or
    fp16; fp32 accumulation; h = act(..) * (..) is rounded once to the weights' type.

    The object holds no buffers of its own: calls from several streams or threads, and calls captured into
    graphs, are independent of each other.  Autograd does not record the calls, results carry no history: a
    training step calls backward() itself.  fp16 gradients have fp16's range on the way, too (what backward
    keeps of the gate's and up's gradients is 0 below 2^-25 and infinite from 65520 on): scale the loss.
    """

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, layout: str = "split", act: str = "silu"):
        _weight("w1", w1)
        _weight("w2", w2)
        if w1.dim() != 2 or w2.dim() != 2 or w1.shape != (2 * w2.shape[1], w2.shape[0]):
            raise ValueError(f"w1 {tuple(w1.shape)} and w2 {tuple(w2.shape)} are not [2I][H] and [H][I]")
        if w1.dtype != w2.dtype or w1.device != w2.device:
            raise ValueError("w1 and w2 differ in type or device")
        if layout not in LAYOUT or act not in GATE_ACT:
            raise ValueError(f"layout {layout!r} / act {act!r}: not {list(LAYOUT)} / {list(GATE_ACT)}")
        self.w1, self.w2, self.layout, self.act = w1, w2, layout, act
        self.H, self.I = w2.shape
        self.dtype, self.device = w1.dtype, w1.device
        self._dtypes = (self.dtype, torch.float32)
        dt = FLOAT_DTYPE[self.dtype]
        self._fwd = FfnArgs(H=self.H, I=self.I, layout=LAYOUT[layout], gate_act=GATE_ACT[act], dtype=dt)
        self._bwd = FfnGradArgs(H=self.H, I=self.I, layout=LAYOUT[layout], gate_act=GATE_ACT[act], dtype=dt)

    def forward(self, x: torch.Tensor, add: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, *,
                out_dtype: Optional[torch.dtype] = None, save=False, stream=None):
        """moe_gated_ffn_forward: x [T][H] -> out [T][H], or (out, gate_up) with save.

        add: [T][H], added to the result; `out` may be `add` itself.  out_dtype: the weights' type (default)
        or torch.float32; `add`'s and `out`'s type if they are given.  save: keep the pre-activations
        gate_up [T][2I] for backward(), True in fp32, "half" in the weights' type (half the memory, one more
        rounding in the gradients).
        """
        a, out, gate_up, ws = self._prepare(x, add, out, out_dtype, save, stream)
        _check(lib.moe_gated_ffn_forward(ctypes.byref(a), _stream(stream)))
        _keep_until_done(stream, out, gate_up, x, add, self.w1, self.w2)
        return (out, gate_up) if save else out

    def _prepare(self, x, add, out, out_dtype=None, save=False, stream=None):
        """forward's arguments, checked by the binding, and the buffers of one call: (arguments, out, gate_up,
        workspace)."""
        _on_current_device(self.device, stream)
        a = FfnArgs.from_buffer_copy(self._fwd)
        a.x_stride = _rows("x", x, None, self.H, (self.dtype,), self.device)
        T = a.T = x.shape[0]
        if out is None:
            with _allocate_on(stream):
                out = torch.empty((T, self.H), device=self.device,
                                  dtype=out_dtype or (add.dtype if add is not None else self.dtype))
        a.out_stride = _rows("out", out, T, self.H, self._dtypes, self.device)
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        a.out_dtype = FLOAT_DTYPE[out.dtype]
        if add is not None:
            a.add_stride = _rows("add", add, T, self.H, (out.dtype,), self.device)
            a.add = add.data_ptr()
        gate_up = None
        if save not in (False, True, "half"):
            raise ValueError(f"save is {save!r}, not False, True or 'half'")
        if save:
            with _allocate_on(stream):
                gate_up = torch.empty((T, 2 * self.I), device=self.device,
                                      dtype=self.dtype if save == "half" else torch.float32)
            a.save_dtype, a.gate_up = FLOAT_DTYPE[gate_up.dtype], gate_up.data_ptr()
        else:
            a.save_dtype = a.dtype
        n = lib.moe_gated_ffn_workspace_size(T, self.H, self.I)
        with _allocate_on(stream):
            ws = _u8(n, self.device)
        a.x, a.w1, a.w2, a.out = x.data_ptr(), self.w1.data_ptr(), self.w2.data_ptr(), out.data_ptr()
        a.workspace, a.workspace_bytes = ws.data_ptr(), n
        return a, out, gate_up, ws

    def backward(self, dout: torch.Tensor, x: torch.Tensor, gate_up: torch.Tensor, *, dx=True, dw1=True, dw2=True,
                 dw_dtype: Optional[torch.dtype] = None, accumulate: bool = False, stream=None):
        """moe_gated_ffn_backward: (dx, dw1, dw2) from dout [T][H], x and forward's gate_up.

        dx, dw1, dw2: True allocates the gradient, a tensor receives it, False or None skips it.  dw_dtype:
        type of the weight gradients made here, the weights' (default) or torch.float32.  accumulate: the
        given dw1 and dw2 are added to.
        """
        _on_current_device(self.device, stream)
        a = FfnGradArgs.from_buffer_copy(self._bwd)
        a.dout_stride = _rows("dout", dout, None, self.H, (self.dtype,), self.device)
        T = a.T = dout.shape[0]
        a.x_stride = _rows("x", x, T, self.H, (self.dtype,), self.device)
        _flat("gate_up", gate_up, (T, 2 * self.I), self._dtypes, self.device)

        def grad(g, shape, dtype):
            if g is True:
                with _allocate_on(stream):
                    return torch.empty(shape, dtype=dtype, device=self.device)
            return None if g is None or g is False else g

        if accumulate and (dw1 is True or dw2 is True):
            raise ValueError("accumulate needs the tensors to add to")
        dw_dtype = dw_dtype or next((g.dtype for g in (dw1, dw2) if isinstance(g, torch.Tensor)), self.dtype)
        dx = grad(dx, (T, self.H), self.dtype)
        dw1 = grad(dw1, (2 * self.I, self.H), dw_dtype)
        dw2 = grad(dw2, (self.H, self.I), dw_dtype)
        a.dx_dtype = a.dtype
        if dx is not None:
            a.dx_stride = _rows("dx", dx, T, self.H, self._dtypes, self.device)
            a.dx_dtype, a.dx = FLOAT_DTYPE[dx.dtype], dx.data_ptr()
        a.dw_dtype = FLOAT_DTYPE.get(dw_dtype, -1)
        if dw1 is not None:
            a.dw1 = _flat("dw1", dw1, (2 * self.I, self.H), (dw_dtype,), self.device).data_ptr()
        if dw2 is not None:
            a.dw2 = _flat("dw2", dw2, (self.H, self.I), (dw_dtype,), self.device).data_ptr()
        a.accumulate = int(accumulate)
        a.save_dtype = FLOAT_DTYPE[gate_up.dtype]
        n = lib.moe_gated_ffn_grad_workspace_size(T, self.H, self.I)
        with _allocate_on(stream):
            ws = _u8(n, self.device)
        a.dout, a.x, a.w1, a.w2 = dout.data_ptr(), x.data_ptr(), self.w1.data_ptr(), self.w2.data_ptr()
        a.gate_up, a.workspace, a.workspace_bytes = gate_up.data_ptr(), ws.data_ptr(), n
        _check(lib.moe_gated_ffn_backward(ctypes.byref(a), _stream(stream)))
        _keep_until_done(stream, dx, dw1, dw2, dout, x, gate_up, self.w1, self.w2)
        return dx, dw1, dw2


class AdapterLinear:
    """One projection shared by all tokens, plus each token's own low-rank adapter (many requests in a batch).

    y[t] = (add[t] +) x[t] w^T + scales[a] (x[t] lora_a[a]^T) lora_b[a]^T with a = ids[t]; an id outside
    [0, num_adapters) means no adapter.  w [N][K] (None: the adapters' part alone, for projections computed
    elsewhere), lora_a [num_adapters][R][K], lora_b [num_adapters][N][R], scales fp32 and ranks int32
    [num_adapters].  epilogue "split" or "interleaved": w's rows are gate and up, out = act(gate) * up.

    Adapters may be replaced in place between calls.  No buffers are held and nothing is recorded by autograd
    (see GatedFFN); there is no backward pass.
    """

    def __init__(self, w: Optional[torch.Tensor], lora_a: torch.Tensor, lora_b: torch.Tensor, *,
                 scales: Optional[torch.Tensor] = None, ranks: Optional[torch.Tensor] = None, epilogue: str = "none",
                 act: str = "silu"):
        _weight("lora_a", lora_a)
        _weight("lora_b", lora_b)
        if lora_a.dim() != 3 or lora_b.dim() != 3 or lora_a.shape[0] != lora_b.shape[0] \
                or lora_a.shape[1] != lora_b.shape[2]:
            raise ValueError(f"lora_a {tuple(lora_a.shape)} and lora_b {tuple(lora_b.shape)} are not [n][R][K] "
                             "and [n][N][R]")
        self.n, self.R, self.K = lora_a.shape
        self.N = lora_b.shape[1]
        self.dtype, self.device = lora_a.dtype, lora_a.device
        if lora_b.dtype != self.dtype or lora_b.device != self.device:
            raise ValueError("lora_a and lora_b differ in type or device")
        if w is not None:
            _flat("w", w, (self.N, self.K), (self.dtype,), self.device)
        if scales is not None:
            _flat("scales", scales, (self.n,), (torch.float32,), self.device)
        if ranks is not None:
            _flat("ranks", ranks, (self.n,), (torch.int32,), self.device)
        epi = {"none": 0, **LAYOUT}
        if epilogue not in epi or act not in GATE_ACT:
            raise ValueError(f"epilogue {epilogue!r} / act {act!r}: not {list(epi)} / {list(GATE_ACT)}")
        if epilogue != "none" and w is None:
            raise ValueError("a gated epilogue needs w")
        self.w, self.lora_a, self.lora_b, self.scales, self.ranks = w, lora_a, lora_b, scales, ranks
        self.n_out = self.N if epilogue == "none" else self.N // 2
        self._dtypes = (self.dtype, torch.float32)
        self._tmpl = AdapterArgs(K=self.K, N=self.N, num_adapters=self.n, R=self.R, epilogue=epi[epilogue],
                                 gate_act=GATE_ACT[act], dtype=FLOAT_DTYPE[self.dtype])

    def forward(self, x: torch.Tensor, ids: torch.Tensor, add: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, *, out_dtype: Optional[torch.dtype] = None, stream=None):
        """moe_adapter_linear: x [T][K], ids int32 [T] -> out [T][N] ([T][N/2] for a gated epilogue).

        add: [T][N], added before the epilogue; without one, `out` may be `add` itself.  out_dtype: the
        weights' type (default) or torch.float32; `add`'s and `out`'s type if they are given.
        """
        _on_current_device(self.device, stream)
        a = AdapterArgs.from_buffer_copy(self._tmpl)
        a.x_stride = _rows("x", x, None, self.K, (self.dtype,), self.device)
        T = a.T = x.shape[0]
        _flat("ids", ids, (T,), (torch.int32,), self.device)
        if out is None:
            with _allocate_on(stream):
                out = torch.empty((T, self.n_out), device=self.device,
                                  dtype=out_dtype or (add.dtype if add is not None else self.dtype))
        a.out_stride = _rows("out", out, T, self.n_out, self._dtypes, self.device)
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        a.out_dtype = FLOAT_DTYPE[out.dtype]
        if add is not None:
            a.add_stride = _rows("add", add, T, self.N, (out.dtype,), self.device)
            a.add = add.data_ptr()
        n = lib.moe_adapter_workspace_size(T, self.K, self.N, self.n, self.R)
        with _allocate_on(stream):
            ws = _u8(n, self.device)
        a.x, a.ids, a.out, a.a, a.b = (x.data_ptr(), ids.data_ptr(), out.data_ptr(), self.lora_a.data_ptr(),
                                       self.lora_b.data_ptr())
        if self.w is not None:
            a.w = self.w.data_ptr()
        if self.scales is not None:
            a.scales = self.scales.data_ptr()
        if self.ranks is not None:
            a.ranks = self.ranks.data_ptr()
        a.workspace, a.workspace_bytes = ws.data_ptr(), n
        _check(lib.moe_adapter_linear(ctypes.byref(a), _stream(stream)))
        _keep_until_done(stream, out, x, ids, add, self.w, self.lora_a, self.lora_b, self.scales, self.ranks)
        return out


class Layer:
    """A resident layer: weights stay on the device; forward() runs the five steps on one stream."""

    def __init__(self, w1_packed, w1_scales, w2_packed, w2_scales, k: int, layout: str = "split",
                 inter: str = "bf16", w_format: str = "canonical", tile: bool = False,
                 shared: Optional["GatedFFN"] = None):
        """inter: precision of the SwiGLU output fed to FC2, "bf16" or "mxfp8".
        w_format: the order of the given weights, "canonical" or "tiled" (W1 tiled
        with `layout`, W2 with "none").  tile=True: canonical weights are tiled
        here once and the layer keeps only the tiled copy.
        shared: a GatedFFN that every token passes beside its routed experts (a
        shared expert); forward() adds its result to theirs."""
        if tile:
            if w_format != "canonical":
                raise ValueError("tile=True takes canonical weights")
            w1_packed, w1_scales = tile_weights(w1_packed, w1_scales, layout)
            w2_packed, w2_scales = tile_weights(w2_packed, w2_scales, "none")
            w_format = "tiled"
        self.w_format = W_FORMAT[w_format]
        self.w1p, self.w1s, self.w2p, self.w2s = w1_packed, w1_scales, w2_packed, w2_scales
        self.E, two_i, h2 = w1_packed.shape
        self.I, self.H = two_i // 2, 2 * h2
        self.k = k
        self.layout = LAYOUT[layout]
        self.inter = OUT[{"bf16": "MOE_OUT_BF16", "mxfp8": "MOE_OUT_MXFP8_E4M3"}[inter]]
        if shared is not None and shared.H != self.H:
            raise ValueError(f"the shared expert's width {shared.H} is not the layer's {self.H}")
        self.shared = shared
        self._ws = self._ws_stream = None

    def workspace_bytes(self, T: int) -> int:
        return lib.moe_layer_workspace_size(T, self.H, self.I, self.E, self.k, self.inter)

    def _args(self, T, logits, x, x_scales, out, x_next, ws):
        return LayerArgs(T=T, H=self.H, I=self.I, E=self.E, k=self.k, layout=self.layout,
                         act_dtype=1 if x_scales is not None else 0, inter_dtype=self.inter,
                         logits=logits.data_ptr(), x=x.data_ptr(),
                         x_scales=x_scales.data_ptr() if x_scales is not None else None,
                         w1_packed=self.w1p.data_ptr(), w1_scales=self.w1s.data_ptr(),
                         w2_packed=self.w2p.data_ptr(), w2_scales=self.w2s.data_ptr(), out=out.data_ptr(),
                         x_next=x_next.data_ptr() if x_next is not None else None,
                         workspace=ws.data_ptr(), workspace_bytes=ws.numel(), w_format=self.w_format)

    def _check_out(self, out, T, device):
        """The routed experts' sum is written as contiguous fp32 [T][H]."""
        if out.dtype != torch.float32 or not out.is_contiguous() or out.numel() < T * self.H or out.device != device:
            raise ValueError(f"out must be a contiguous torch.float32 tensor of {(T, self.H)} on {device}: got "
                             f"{out.dtype} {tuple(out.shape)}, strides {out.stride()}, on {out.device}")

    def _shared_input(self, x, x_scales, x_shared, x_next):
        """The shared expert's activations, [T][H] in its type: x itself where that is what x holds."""
        if self.shared is None:
            if x_shared is not None:
                raise ValueError("x_shared without a shared expert")
            return None
        if x_next is not None:
            raise ValueError("x_next is taken from the routed experts' sum: not with a shared expert")
        xs = x if x_shared is None and x_scales is None else x_shared
        if xs is None:
            raise ValueError("MXFP8 activations: the shared expert needs x_shared, their 16-bit values")
        _rows("the shared expert's input", xs, x.shape[0], self.H, (self.shared.dtype,), self.shared.device)
        return xs

    def forward(self, logits: torch.Tensor, x: torch.Tensor, x_scales: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, x_next: Optional[torch.Tensor] = None, stream=None,
                x_shared: Optional[torch.Tensor] = None):
        """x_shared: the shared expert's activations where x does not hold them (MXFP8 x, or another type)."""
        x_shared = self._shared_input(x, x_scales, x_shared, x_next)
        T = logits.shape[0]
        n = self.workspace_bytes(T)
        ws, on = self._ws, torch.cuda.current_stream(logits.device) if stream is None else stream
        with _allocate_on(stream):
            captured = torch.cuda.is_current_stream_capturing()
        # a call on another stream gets a workspace of its own (the kept one may still be in use), and one that
        # the caller captures does too: its graph goes on using it, and owns its memory
        if ws is None or ws.numel() < n or self._ws_stream != on or captured:
            with _allocate_on(stream):
                ws = _u8(n, logits.device)
            self._ws, self._ws_stream = ws, None if captured else on
        if out is None:
            with _allocate_on(stream):
                out = torch.empty((T, self.H), dtype=torch.float32, device=logits.device)
        self._check_out(out, T, logits.device)
        args = self._args(T, logits, x, x_scales, out, x_next, ws)
        # the shared expert may refuse its tensors: before the routed experts are enqueued
        shared = None if x_shared is None else self._prepare_shared(x_shared, out, stream)
        _check(lib.moe_layer_forward(ctypes.byref(args), _stream(stream)))
        if shared is not None:
            _check(lib.moe_gated_ffn_forward(ctypes.byref(shared[0]), _stream(stream)))
        # (routing() shows the workspace to the caller)
        _keep_until_done(stream, ws, out, logits, x, x_scales, x_next, x_shared, self.w1p, self.w1s, self.w2p, self.w2s)
        if shared is not None:
            _keep_until_done(stream, self.shared.w1, self.shared.w2)
        return out

    def _prepare_shared(self, x_shared, out, stream=None):
        """The shared expert's call that adds to `out`, every check made."""
        call = self.shared._prepare(x_shared, out, out, stream=stream)
        _check(lib.moe_gated_ffn_check(ctypes.byref(call[0])))
        return call

    def capture(self, logits: torch.Tensor, x: torch.Tensor, x_scales: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, x_next: Optional[torch.Tensor] = None,
                x_shared: Optional[torch.Tensor] = None) -> "LayerGraph":
        """moe_layer_graph_create: this layer on these buffers, captured once; see LayerGraph."""
        return LayerGraph(self, logits, x, x_scales, out, x_next, x_shared)

    def routing(self, T: int):
        """Views of the routing arrays the last forward() wrote into its workspace."""
        def view(which, count, dtype):
            off = lib.moe_layer_workspace_offset(T, self.H, self.I, self.E, self.k, self.inter, which)
            return self._ws[off: off + 4 * count].view(dtype)
        Tk = T * self.k
        return dict(ids=view(0, Tk, torch.int32).view(T, self.k), w=view(1, Tk, torch.float32).view(T, self.k),
                    offsets=view(2, self.E + 1, torch.int32), perm_src=view(3, Tk, torch.int32),
                    dest_row=view(4, Tk, torch.int32))


class LayerGraph:
    """A resident layer captured into a HIP graph (moe_layer_graph_*).

    The graph owns its workspace and keeps the tensors it was captured on:
    replay() runs the five steps with one launch, reading the current contents
    of logits / x / x_scales and writing `out` (and x_next); a shared expert
    follows as launches of its own, on a workspace that the graph owns too.
    Replays on one graph must not overlap each other.  Capturing waits for what
    the current stream still has to do.
    """

    def __init__(self, layer: Layer, logits, x, x_scales=None, out=None, x_next=None, x_shared=None):
        x_shared = layer._shared_input(x, x_scales, x_shared, x_next)
        T = logits.shape[0]
        dev = logits.device
        self.layer, self.T = layer, T
        self.logits, self.x, self.x_scales, self.x_next = logits, x, x_scales, x_next
        self.out = out if out is not None else torch.empty((T, layer.H), dtype=torch.float32, device=dev)
        layer._check_out(self.out, T, dev)
        self.ws = _u8(layer.workspace_bytes(T), dev)
        args = layer._args(T, logits, x, x_scales, self.out, x_next, self.ws)
        self.shared, self.x_shared = layer.shared, x_shared
        self._shared_call = None if x_shared is None else layer._prepare_shared(x_shared, self.out)
        # replays may run on any stream: what the current one still does with these buffers' memory ends here
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(dev).synchronize()
        # capture needs a created stream; nothing runs during the capture
        side = torch.cuda.Stream(device=dev)
        self._h = ctypes.c_void_p()
        _check(lib.moe_layer_graph_create(ctypes.byref(args), ctypes.c_void_p(side.cuda_stream),
                                          ctypes.byref(self._h)))

    def replay(self, stream=None) -> torch.Tensor:
        if not self._h:
            raise MoeError(STATUS["MOE_ERR_INVALID_ARG"], "graph already destroyed")
        if self._shared_call is not None:
            _on_current_device(self.shared.device, stream)
        _check(lib.moe_layer_graph_launch(self._h, _stream(stream)))
        if self._shared_call is not None:
            _check(lib.moe_gated_ffn_forward(ctypes.byref(self._shared_call[0]), _stream(stream)))
        return self.out

    def routing(self):
        """Views of the routing arrays the last replay wrote into the graph's workspace."""
        L = self.layer
        def view(which, count, dtype):
            off = lib.moe_layer_workspace_offset(self.T, L.H, L.I, L.E, L.k, L.inter, which)
            return self.ws[off: off + 4 * count].view(dtype)
        Tk = self.T * L.k
        return dict(ids=view(0, Tk, torch.int32).view(self.T, L.k), w=view(1, Tk, torch.float32).view(self.T, L.k),
                    offsets=view(2, L.E + 1, torch.int32), perm_src=view(3, Tk, torch.int32),
                    dest_row=view(4, Tk, torch.int32))

    def close(self):
        """moe_layer_graph_destroy; waits for the device first so that no replay is still running."""
        if self._h:
            torch.cuda.synchronize(self.out.device)
            h, self._h = self._h, ctypes.c_void_p()
            _check(lib.moe_layer_graph_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def blob_bytes(H: int, I: int, E: int) -> int:
    return lib.moe_blob_bytes(H, I, E)


def blob_section_offset(H: int, I: int, E: int, which: int) -> int:
    return lib.moe_blob_section_offset(H, I, E, which)


def prefill_streamed(host_blobs: Sequence[torch.Tensor], slots: Sequence[torch.Tensor], logits: torch.Tensor,
                     x: torch.Tensor, out: torch.Tensor, *, T: int, H: int, I: int, E: int, k: int,
                     num_layers: int, layout: str = "split", chain: str = "rms", depth: int = 2,
                     layer_inputs: Optional[torch.Tensor] = None, events=None, workspace=None,
                     compute_stream=None, copy_stream=None, w_format: str = "canonical",
                     expert_copy: str = "all", routed_copy_max_tokens: int = 0):
    """moe_layer_prefill_streamed.  host_blobs: pinned uint8 CPU tensors (layer L uses blob L % n).

    expert_copy: "all" moves every expert of a layer, "routed" only the experts
    its routing hits, "auto" routed when T <= routed_copy_max_tokens.
    copy_stream: the stream the weight copies run on; None uses one dedicated
    side stream per device (never the compute stream, which would serialise the
    pipeline).
    """
    nb = len(host_blobs)
    arr = (_vp * nb)(*[b.data_ptr() for b in host_blobs])
    need = lib.moe_streamed_workspace_size(T, H, I, E, k)
    if workspace is None or workspace.numel() < need:
        # the copy stream waits for the compute stream's earlier work before it begins
        with _allocate_on(compute_stream):
            workspace = _u8(need, x.device)
    ev_arr = None
    if events is not None:
        ev_arr = (_vp * len(events))(*[e.cuda_event for e in events])
    args = StreamedArgs(num_layers=num_layers, T=T, H=H, I=I, E=E, k=k, layout=LAYOUT[layout],
                        chain=CHAIN["MOE_CHAIN_RMS" if chain == "rms" else "MOE_CHAIN_INDEPENDENT"],
                        depth=depth, num_blobs=nb, host_blobs=arr,
                        blob_bytes=min(b.numel() for b in host_blobs),
                        device_slot=(_vp * 2)(slots[0].data_ptr(), slots[1].data_ptr() if len(slots) > 1 else 0),
                        logits=logits.data_ptr(), x=x.data_ptr(), out=out.data_ptr(),
                        layer_inputs=layer_inputs.data_ptr() if layer_inputs is not None else None,
                        events=ctypes.cast(ev_arr, _vp) if ev_arr is not None else None,
                        workspace=workspace.data_ptr(), workspace_bytes=workspace.numel(),
                        w_format=W_FORMAT[w_format], expert_copy=EXPERT_COPY[expert_copy],
                        routed_copy_max_tokens=routed_copy_max_tokens)
    cs = _stream(compute_stream)
    if copy_stream is None:
        # a copy on the compute stream would serialise the pipeline
        copy_stream = _copy_stream_for(x.device)
    _check(lib.moe_layer_prefill_streamed(ctypes.byref(args), cs, _stream(copy_stream)))
    _keep_until_done(compute_stream, workspace, logits, x, out, layer_inputs, *slots)
    _keep_until_done(copy_stream, workspace, logits, *slots)
    return workspace
