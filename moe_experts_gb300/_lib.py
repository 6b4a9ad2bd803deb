"""ctypes binding of libepq.so (include/epq.h): argument marshalling only.

Every function here forwards to the C ABI of the same name.  Tensors are
torch CUDA tensors; their device pointers and torch's current CUDA stream are
passed through.  Output tensors that the caller does not supply are
allocated with torch (device memory is torch's business; the library itself
never allocates).  There is no fallback: if the shared library is missing or
a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libepq.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "epq.h")

EPQ_Q8_0, EPQ_Q4_0, EPQ_Q4_1, EPQ_Q4_K, EPQ_Q2_K, EPQ_Q6_K = 0, 1, 2, 3, 4, 5
FORMATS = {"Q8_0": EPQ_Q8_0, "Q4_0": EPQ_Q4_0, "Q4_1": EPQ_Q4_1, "Q4_K": EPQ_Q4_K, "Q2_K": EPQ_Q2_K,
           "Q6_K": EPQ_Q6_K}

_lib = None


class EpqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = _lib.epq_status_string(status).decode() if _lib else str(status)
        extra = f" (cudaError {_lib.epq_last_cuda_error()})" if _lib and status == 6 else ""
        super().__init__(f"{fn} failed: {msg}{extra}")
        self.status = status


class GemvOpts(ctypes.Structure):
    _fields_ = [("residual", ctypes.c_void_p), ("rms_prenorm", ctypes.c_int), ("rms_eps", ctypes.c_float),
                ("swiglu", ctypes.c_int), ("x_group", ctypes.c_int), ("x_head_dim", ctypes.c_int),
                ("x_ld", ctypes.c_int64), ("weights_ready", ctypes.c_int)]


class GemvOp(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("swiglu", ctypes.c_int), ("rms_prenorm", ctypes.c_int), ("rms_eps", ctypes.c_float),
                ("x_group", ctypes.c_int), ("x_head_dim", ctypes.c_int), ("x_ld", ctypes.c_int64)]


class Router(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("n_experts", ctypes.c_int),
                ("norm_topk", ctypes.c_int)]


class Experts(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("n_experts", ctypes.c_int), ("hidden", ctypes.c_int),
                ("inter", ctypes.c_int), ("gate_up", ctypes.c_void_p), ("gate_up_stride", ctypes.c_int64),
                ("down", ctypes.c_void_p), ("down_stride", ctypes.c_int64), ("shared_gate_up", ctypes.c_void_p),
                ("shared_down", ctypes.c_void_p), ("shared_gate_vec", ctypes.c_void_p),
                ("down_fmt_set", ctypes.c_int), ("down_fmt", ctypes.c_int)]


class MoeOpts(ctypes.Structure):
    _fields_ = [("rms_prenorm", ctypes.c_int), ("rms_eps", ctypes.c_float), ("logits_out", ctypes.c_void_p),
                ("h_out", ctypes.c_void_p), ("stages", ctypes.c_int)]


class Pages(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("table", ctypes.c_void_p), ("length", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("work", ctypes.c_void_p), ("n_layers", ctypes.c_int),
                ("n_pages", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_size", ctypes.c_int), ("n_seq", ctypes.c_int), ("max_pages", ctypes.c_int)]


class AttentionTreeOpts(ctypes.Structure):
    _fields_ = [("mask", ctypes.c_void_p), ("n_tok", ctypes.c_void_p), ("q_ld", ctypes.c_int64),
                ("q_seq_ld", ctypes.c_int64), ("kv_ld", ctypes.c_int64), ("kv_seq_ld", ctypes.c_int64)]


class VerifyOpts(ctypes.Structure):
    _fields_ = [("draft", ctypes.c_void_p), ("n_tok", ctypes.c_void_p), ("temperature", ctypes.c_float),
                ("ld", ctypes.c_int64), ("draft_ld", ctypes.c_int64)]


class RopeScaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("context", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double)]


class Rotation(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("n_pos", ctypes.c_int64), ("rot_dim", ctypes.c_int),
                ("first", ctypes.c_int), ("interleaved", ctypes.c_int)]


class RopeOpts(ctypes.Structure):
    _fields_ = [("position", ctypes.c_void_p), ("start", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("n_tok", ctypes.c_void_p), ("x_ld", ctypes.c_int64), ("x_seq_ld", ctypes.c_int64),
                ("y_ld", ctypes.c_int64), ("y_seq_ld", ctypes.c_int64)]


class AppendOpts(ctypes.Structure):
    _fields_ = [("rotation", ctypes.c_void_p), ("position", ctypes.c_void_p), ("mask", ctypes.c_void_p),
                ("n_tok", ctypes.c_void_p), ("kv_ld", ctypes.c_int64), ("kv_seq_ld", ctypes.c_int64)]


class PromptOpts(ctypes.Structure):
    _fields_ = [("n_tok", ctypes.c_void_p), ("window", ctypes.c_int), ("q_ld", ctypes.c_int64),
                ("q_seq_ld", ctypes.c_int64)]


class LogitsOpts(ctypes.Structure):
    _fields_ = [("penalties", ctypes.c_void_p), ("history", ctypes.c_void_p), ("history_len", ctypes.c_void_p),
                ("prompt_len", ctypes.c_void_p), ("max_history", ctypes.c_int), ("tokens", ctypes.c_void_p),
                ("mask", ctypes.c_void_p), ("n_tok", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("n_bias", ctypes.c_int), ("allowed", ctypes.c_void_p),
                ("ld", ctypes.c_int64), ("out_ld", ctypes.c_int64)]


EPQ_MOE_ROUTE, EPQ_MOE_GATE_UP, EPQ_MOE_DOWN = 1, 2, 4
EPQ_ROPE_PLAIN, EPQ_ROPE_LINEAR, EPQ_ROPE_PARTS, EPQ_ROPE_BANDS = 0, 1, 2, 3


def declared_symbols() -> list[str]:
    """Every function the public header declares."""
    text = open(HEADER, encoding="utf-8").read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(epq_[a-z0-9_]+)\s*\(", text)))


def load(path: str | None = None):
    """Load libepq.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with moe_experts_gb300.build.build()")
    lib = ctypes.CDLL(path)
    i64, vp, i32, f32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    sig = {
        "epq_status_string": (ctypes.c_char_p, [i32]),
        "epq_last_cuda_error": (i32, []),
        "epq_device_error": (i32, []),
        "epq_device_error_detail": (i32, [ctypes.POINTER(i32), ctypes.POINTER(i32), ctypes.POINTER(i32)]),
        "epq_block_weights": (i64, [i32]),
        "epq_block_bytes": (i64, [i32]),
        "epq_row_bytes": (i64, [i32, i64]),
        "epq_set_tuning": (i32, [i32, i32]),
        "epq_quantize": (i32, [i32, vp, i64, i64, vp, vp]),
        "epq_dequantize": (i32, [i32, vp, i64, i64, vp, vp]),
        "epq_gemv": (i32, [i32, vp, vp, vp, i64, i64, i32, vp]),
        "epq_gemv_ex": (i32, [i32, vp, vp, vp, i64, i64, i32, ctypes.POINTER(GemvOpts), vp]),
        "epq_moe_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Router), ctypes.POINTER(Experts), i32, i32]),
        "epq_moe_forward": (i32, [ctypes.POINTER(Router), ctypes.POINTER(Experts), vp, i32, i32,
                                  ctypes.POINTER(MoeOpts), vp, vp, vp, vp, ctypes.c_size_t, vp]),
        "epq_gemv_chain_workspace_bytes": (ctypes.c_size_t, []),
        "epq_gemv_chain": (i32, [i32, ctypes.POINTER(GemvOp), i32, i32, vp, ctypes.c_size_t, vp]),
        "epq_moe_forward_noalloc": (i32, [ctypes.POINTER(Router), ctypes.POINTER(Experts), vp, i32, i32,
                                          ctypes.POINTER(MoeOpts), vp, vp, vp, vp]),
        "epq_kv_row_bytes": (i64, [i32]),
        "epq_attention_decode": (i32, [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, f32, vp, vp, vp]),
        "epq_pages_work_bytes": (ctypes.c_size_t, [ctypes.POINTER(Pages)]),
        "epq_pages_truncate": (i32, [ctypes.POINTER(Pages), vp, vp]),
        "epq_pages_fork": (i32, [ctypes.POINTER(Pages), vp, vp, i32, vp, vp]),
        "epq_pages_reserve": (i32, [ctypes.POINTER(Pages), vp, vp, vp]),
        "epq_pages_compact": (i32, [ctypes.POINTER(Pages), vp, vp, i32, vp]),
        "epq_tree_mask": (i32, [vp, i32, i32, vp, vp]),
        "epq_attention_tree_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Pages), i32, i32]),
        "epq_attention_tree": (i32, [ctypes.POINTER(Pages), i32, vp, vp, vp, i32, i32, f32,
                                     ctypes.POINTER(AttentionTreeOpts), vp, vp, ctypes.c_size_t, vp]),
        "epq_verify_tree_workspace_bytes": (ctypes.c_size_t, [i32, i32, i64]),
        "epq_verify_tree": (i32, [vp, i64, vp, vp, vp, i32, i32, ctypes.POINTER(VerifyOpts), vp, vp, vp, vp, vp,
                                  ctypes.c_size_t, vp]),
        "epq_rope_frequencies": (i32, [i32, ctypes.c_double, ctypes.POINTER(RopeScaling),
                                       ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]),
        "epq_rope_table": (i32, [vp, i32, ctypes.c_double, i64, vp, vp]),
        "epq_rope": (i32, [ctypes.POINTER(Rotation), vp, vp, i32, i32, i32, i32, ctypes.POINTER(RopeOpts), vp]),
        "epq_pages_append": (i32, [ctypes.POINTER(Pages), i32, vp, vp, i32, ctypes.POINTER(AppendOpts), vp]),
        "epq_attention_prompt_workspace_bytes": (ctypes.c_size_t, [ctypes.POINTER(Pages), i32, i32]),
        "epq_attention_prompt": (i32, [ctypes.POINTER(Pages), i32, vp, i32, i32, f32, ctypes.POINTER(PromptOpts), vp,
                                       vp, ctypes.c_size_t, vp]),
        "epq_logits_adjust": (i32, [vp, i64, i32, i32, ctypes.POINTER(LogitsOpts), vp, vp]),
        "epq_pages_advance": (i32, [ctypes.POINTER(Pages), vp, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


# the current stream's handle without a Stream object, where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_object(stream):
    """The torch stream of a `stream` argument that is not None (a handle of 0 is the default stream, for which
    ExternalStream would make a new one)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream(stream)
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _empty_on(stream, shape, dtype, device) -> torch.Tensor:
    """torch.empty for the results or scratch of a call on `stream`.  It comes from that stream's memory, which nothing
    before the call can still be using, and is not given out again before the current stream is done with it either."""
    if device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _allocator(stream):
    """torch.empty, or its like for a call on a stream that is named."""
    return torch.empty if stream is None else functools.partial(_empty_on, stream)


def _check(fn: str, st: int):
    if st != 0:
        raise EpqError(fn, st)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ------------------------------------------------------------------ host-only queries
def epq_row_bytes(fmt: int, cols: int) -> int:
    return int(load().epq_row_bytes(fmt, cols))


def epq_block_weights(fmt: int) -> int:
    return int(load().epq_block_weights(fmt))


def epq_block_bytes(fmt: int) -> int:
    return int(load().epq_block_bytes(fmt))


EPQ_TUNE_TILE_BYTES, EPQ_TUNE_RING_BYTES, EPQ_TUNE_GEMV_ENGINE, EPQ_TUNE_EARLY_STAGES, EPQ_TUNE_TC_SPLIT = 1, 2, 3, 4, 5
EPQ_TUNE_ATTN_CHUNK, EPQ_TUNE_VN_CHUNK, EPQ_TUNE_VN_CLUSTER = 6, 7, 8


def epq_set_tuning(key: int, value: int) -> int:
    return int(load().epq_set_tuning(key, value))


def epq_status_string(st: int) -> str:
    return load().epq_status_string(st).decode()


def epq_device_error() -> int:
    return int(load().epq_device_error())


def epq_device_error_detail() -> tuple[int, int, int, int]:
    """(code, block, pipeline step, thread) of the first wait timeout; clears it."""
    b, w, t = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    code = load().epq_device_error_detail(ctypes.byref(b), ctypes.byref(w), ctypes.byref(t))
    return int(code), b.value, w.value, t.value


# ------------------------------------------------------------------ packing
def epq_quantize(fmt: int, W: torch.Tensor, blocks: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """W float32 [rows, cols] (CUDA) -> packed uint8 [rows, row_bytes]."""
    lib = load()
    rows, cols = W.shape
    rb = lib.epq_row_bytes(fmt, cols)
    if blocks is None:
        blocks = torch.empty((rows, max(rb, 0)), dtype=torch.uint8, device=W.device)
    _check("epq_quantize", lib.epq_quantize(fmt, _ptr(W), rows, cols, _ptr(blocks), _stream(stream)))
    return blocks


def epq_dequantize(fmt: int, blocks: torch.Tensor, rows: int, cols: int, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    lib = load()
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=blocks.device)
    _check("epq_dequantize", lib.epq_dequantize(fmt, _ptr(blocks), rows, cols, _ptr(out), _stream(stream)))
    return out


# ------------------------------------------------------------------ GEMV
def epq_gemv(fmt: int, blocks: torch.Tensor, x: torch.Tensor, rows: int, cols: int, y: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """x float32 [nvec, cols] (or [cols]) -> y float32 [nvec, rows]."""
    lib = load()
    x2 = x if x.dim() == 2 else x.view(1, -1)
    nvec = x2.shape[0]
    if y is None:
        y = torch.empty((nvec, rows), dtype=torch.float32, device=x.device)
    _check("epq_gemv", lib.epq_gemv(fmt, _ptr(blocks), _ptr(x2), _ptr(y), rows, cols, nvec, _stream(stream)))
    return y


def epq_gemv_ex(fmt: int, blocks: torch.Tensor, x: torch.Tensor, rows: int, cols: int, y: torch.Tensor | None = None,
                residual: torch.Tensor | None = None, rms_prenorm: bool = False, rms_eps: float = 0.0,
                swiglu: bool = False, x_group: int = 0, x_head_dim: int = 0, weights_ready: bool = False,
                stream=None) -> torch.Tensor:
    lib = load()
    x2 = x if x.dim() == 2 else x.view(1, -1)
    nvec = x2.shape[0]
    if x2.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    x_ld = x2.stride(0) if nvec > 1 else 0
    rows_out = rows // 2 if swiglu else rows
    if y is None:
        y = torch.empty((nvec, rows_out), dtype=torch.float32, device=x.device)
    o = GemvOpts(residual.data_ptr() if residual is not None else None, int(rms_prenorm), float(rms_eps),
                 int(swiglu), int(x_group), int(x_head_dim), int(x_ld), int(weights_ready))
    _check("epq_gemv_ex", lib.epq_gemv_ex(fmt, _ptr(blocks), _ptr(x2), _ptr(y), rows, cols, nvec,
                                          ctypes.byref(o), _stream(stream)))
    return y


EPQ_CHAIN_MAX_OPS = 256


def epq_gemv_chain_workspace_bytes() -> int:
    return int(load().epq_gemv_chain_workspace_bytes())


def gemv_op(blocks: torch.Tensor, x: torch.Tensor, y: torch.Tensor, rows: int, cols: int,
            residual: torch.Tensor | None = None, swiglu: bool = False, rms_prenorm: bool = False,
            rms_eps: float = 0.0, x_group: int = 0, x_head_dim: int = 0) -> GemvOp:
    """One op of epq_gemv_chain; x and y are [nvec, n] views (rows contiguous)."""
    x2 = x if x.dim() == 2 else x.view(1, -1)
    if x2.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    x_ld = x2.stride(0) if x2.shape[0] > 1 else 0
    return GemvOp(_ptr(blocks), _ptr(x2), _ptr(y), residual.data_ptr() if residual is not None else None,
                  int(rows), int(cols), int(swiglu), int(rms_prenorm), float(rms_eps), int(x_group),
                  int(x_head_dim), int(x_ld))


def epq_gemv_chain(fmt: int, ops: list, nvec: int, workspace: torch.Tensor, stream=None) -> None:
    """Run the ops (GemvOp list) in order in one persistent launch."""
    lib = load()
    arr = (GemvOp * len(ops))(*ops)
    _check("epq_gemv_chain", lib.epq_gemv_chain(fmt, arr, len(ops), nvec, _ptr(workspace),
                                                workspace.numel() * workspace.element_size(), _stream(stream)))


# ------------------------------------------------------------------ MoE layer
def _addr(t):
    return None if t is None else t.data_ptr()


class MoELayer:
    """Device-resident MoE weights in the layout epq_moe_forward expects.

    router [E, H] float32; gate_up uint8 [E, 2*I, row_bytes(H)] (gate rows
    then up rows); down uint8 [E, H, row_bytes(I)]; optional shared expert
    (same shapes without E) and shared gate vector [H].  down_fmt: the
    format of the down projections when it differs from fmt (a mixed
    per-tensor recipe).
    """

    def __init__(self, fmt, router, gate_up, down, router_bias=None, shared_gate_up=None, shared_down=None,
                 shared_gate_vec=None, norm_topk=True, down_fmt=None):
        self.fmt = int(fmt)
        self.down_fmt = self.fmt if down_fmt is None else int(down_fmt)
        self.router, self.router_bias = router, router_bias
        self.gate_up, self.down = gate_up, down
        self.shared_gate_up, self.shared_down, self.shared_gate_vec = shared_gate_up, shared_down, shared_gate_vec
        self.E, self.H = router.shape
        self.I = down.shape[2] * epq_block_weights(self.down_fmt) // epq_block_bytes(self.down_fmt)
        self.norm_topk = bool(norm_topk)
        self._r = Router(_addr(router), _addr(router_bias), self.E, int(self.norm_topk))
        self._x = Experts(self.fmt, self.E, self.H, self.I, _addr(gate_up), gate_up[0].numel(), _addr(down),
                          down[0].numel(), _addr(shared_gate_up), _addr(shared_down), _addr(shared_gate_vec),
                          int(self.down_fmt != self.fmt), self.down_fmt)

    def workspace_bytes(self, ntok: int, topk: int) -> int:
        return int(load().epq_moe_workspace_bytes(ctypes.byref(self._r), ctypes.byref(self._x), ntok, topk))


def epq_moe_workspace_bytes(layer: MoELayer, ntok: int, topk: int) -> int:
    return layer.workspace_bytes(ntok, topk)


def epq_moe_forward(layer: MoELayer, x: torch.Tensor, topk: int, y: torch.Tensor | None = None,
                    topk_idx: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, rms_prenorm: bool = False, rms_eps: float = 0.0,
                    logits_out: torch.Tensor | None = None, h_out: torch.Tensor | None = None, stages: int = 0,
                    stream=None):
    """x float32 [ntok, H] -> y float32 [ntok, H]; returns (y, topk_idx, topk_w)."""
    lib = load()
    ntok = x.shape[0]
    if y is None:
        y = torch.empty_like(x)
    if workspace is None:
        workspace = torch.empty(layer.workspace_bytes(ntok, topk), dtype=torch.uint8, device=x.device)
    o = MoeOpts(int(rms_prenorm), float(rms_eps), _addr(logits_out), _addr(h_out), int(stages))
    _check("epq_moe_forward", lib.epq_moe_forward(
        ctypes.byref(layer._r), ctypes.byref(layer._x), _ptr(x), ntok, topk, ctypes.byref(o), _ptr(y),
        _ptr(topk_idx), _ptr(topk_w), _ptr(workspace), workspace.numel(), _stream(stream)))
    return y, topk_idx, topk_w


def epq_moe_forward_noalloc(layer: MoELayer, x: torch.Tensor, topk: int, y: torch.Tensor,
                            topk_idx: torch.Tensor | None = None, topk_w: torch.Tensor | None = None,
                            rms_prenorm: bool = False, rms_eps: float = 0.0, stream=None):
    """The MoE layer with the library's fixed scratch instead of a workspace.

    For callers that cannot allocate device memory: nothing is allocated
    here either, so y (and the optional top-K outputs) must be supplied.
    """
    lib = load()
    o = MoeOpts(int(rms_prenorm), float(rms_eps), None, None, 0)
    _check("epq_moe_forward_noalloc", lib.epq_moe_forward_noalloc(
        ctypes.byref(layer._r), ctypes.byref(layer._x), _ptr(x), x.shape[0], topk, ctypes.byref(o), _ptr(y),
        _ptr(topk_idx), _ptr(topk_w), _stream(stream)))
    return y


# ------------------------------------------------------------------ attention
def epq_kv_row_bytes(head_dim: int) -> int:
    return int(load().epq_kv_row_bytes(head_dim))


class KVCache:
    """Device Q8_0 key and value caches of one layer: uint8
    [n_kv_heads, max_pos, epq_kv_row_bytes(head_dim)] each."""

    def __init__(self, n_kv_heads: int, head_dim: int, max_pos: int, device):
        rb = epq_kv_row_bytes(head_dim)
        if rb < 0:
            raise ValueError(f"head_dim {head_dim} not supported")
        self.n_kv_heads, self.head_dim, self.max_pos = n_kv_heads, head_dim, max_pos
        self.k = torch.zeros((n_kv_heads, max_pos, rb), dtype=torch.uint8, device=device)
        self.v = torch.zeros_like(self.k)


def epq_attention_decode(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, cache: KVCache, n_heads: int,
                         pos: int, scale: float, skip_log: float = float("-inf"), out: torch.Tensor | None = None,
                         scores_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [n_heads*D], k_new/v_new [n_kv*D] (float32, device) -> out [n_heads*D]."""
    lib = load()
    if out is None:
        out = torch.empty(n_heads * cache.head_dim, dtype=torch.float32, device=q.device)
    _check("epq_attention_decode", lib.epq_attention_decode(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(cache.k), _ptr(cache.v), n_heads, cache.n_kv_heads, cache.head_dim,
        int(pos), cache.max_pos, float(scale), float(skip_log), _ptr(out), _ptr(scores_out), _stream(stream)))
    return out


# ------------------------------------------------------------------ paged cache
# The calls of a speculative step are short next to what Python costs, so the
# functions below compare shapes as tuples, GPUs by their index, and pass
# addresses as integers.
def _place(t):
    """Where t lies: a GPU's index, or the torch.device that is none (argument checks work without a GPU)."""
    return t.get_device() if t.is_cuda else t.device


def _elsewhere(t, name, at):
    if _place(t) != at:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {f'cuda:{at}' if type(at) is int else at}")


def _refuse(t, name, dtype, shape, at):
    _elsewhere(t, name, at)
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need(t, name, dtype, shape, at):
    """t is a contiguous tensor of this type and shape at this place (_place)."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != at or not t.is_contiguous():
        _refuse(t, name, dtype, shape, at)
    return t.data_ptr()


def _result(t, name, dtype, shape, at, new, dev):
    """A result tensor and its address: the caller's, or one made here (which needs no check)."""
    if t is None:
        t = new(shape, dtype=dtype, device=dev)
        return t, t.data_ptr()
    return t, _need(t, name, dtype, shape, at)


def _queue(stream, at):
    """The handle of the stream to launch on: the one named, or the current one of the GPU that the tensors are on."""
    return _raw_stream(at) if stream is None and type(at) is int and _raw_stream is not None else _stream(stream)


def _launch_on(stream, at):
    """_queue, where host tensors are refused on a machine whose GPU would be given their addresses."""
    if type(at) is not int and torch.cuda.is_available():
        raise ValueError(f"the tensors are on {at}, not on a GPU")
    return _queue(stream, at)


def _scratch(t, at):
    """A workspace: its address and bytes."""
    if t.get_device() != at or not t.is_contiguous():
        _refuse(t, "workspace", t.dtype, t.shape, at)
    return t.data_ptr(), t.numel()


class PagedKVCache:
    """Q8_0 key/value cache in pages shared by sequences (epq_pages): pool
    uint8 [n_layers, n_pages, n_kv_heads, 2, page_size, epq_kv_row_bytes(head_dim)],
    table int32 [n_seq, max_pages], length int32 [n_seq], refs int32 [n_pages],
    all on one device, as are the tensors of every call on the cache.  The
    positions of a sequence are appended by epq_attention_tree and committed
    by epq_pages_compact."""

    def __init__(self, n_layers: int, n_pages: int, n_kv_heads: int, head_dim: int, n_seq: int, max_pages: int,
                 page_size: int = 64, device="cuda"):
        rb = epq_kv_row_bytes(head_dim)
        if rb < 0:
            raise ValueError(f"head_dim {head_dim} not supported")
        i32 = dict(dtype=torch.int32, device=device)
        self._bind(torch.zeros((n_layers, n_pages, n_kv_heads, 2, page_size, rb), dtype=torch.uint8, device=device),
                   torch.full((n_seq, max_pages), -1, **i32), torch.zeros(n_seq, **i32), torch.zeros(n_pages, **i32))

    @classmethod
    def over(cls, pool: torch.Tensor, table: torch.Tensor, length: torch.Tensor, refs: torch.Tensor) -> "PagedKVCache":
        """A cache over tensors that the caller holds (layouts as above)."""
        self = cls.__new__(cls)
        self._bind(pool, table, length, refs)
        return self

    def _bind(self, pool, table, length, refs):
        if pool.dim() != 6 or pool.shape[3] != 2 or table.dim() != 2:
            raise ValueError("pool must be [layers, pages, heads, 2, page_size, row] and table [n_seq, max_pages]")
        self.device, self._at = pool.device, _place(pool)
        _need(pool, "pool", torch.uint8, pool.shape, self._at)
        _need(table, "table", torch.int32, table.shape, self._at)
        _need(length, "length", torch.int32, (table.shape[0],), self._at)
        _need(refs, "refs", torch.int32, (pool.shape[1],), self._at)
        self.n_layers, self.n_pages, self.n_kv_heads, _, self.page_size, rb = pool.shape
        self.head_dim = rb * 16 // 17
        if epq_kv_row_bytes(self.head_dim) != rb:
            raise ValueError(f"rows of {rb} bytes are no cache rows")
        self.n_seq, self.max_pages = table.shape
        self.pool, self.table, self.length, self.refs = pool, table, length, refs
        self._p = Pages(_addr(pool), _addr(table), _addr(length), _addr(refs), None, self.n_layers, self.n_pages,
                        self.n_kv_heads, self.head_dim, self.page_size, self.n_seq, self.max_pages)
        n = int(load().epq_pages_work_bytes(ctypes.byref(self._p)))
        if n == 0:
            raise ValueError("sizes of the paged cache not supported")
        self.work = torch.zeros(n, dtype=torch.uint8, device=self.device)
        self._p.work = self.work.data_ptr()
        self._ref = ctypes.byref(self._p)
        self._per_seq = (self.n_seq,)


def epq_pages_truncate(cache: PagedKVCache, new_length: torch.Tensor, stream=None) -> None:
    """new_length int32 [n_seq] (negative: leave): shorten sequences and give their pages back (0 frees one)."""
    at = cache._at
    n = _need(new_length, "new_length", torch.int32, cache._per_seq, at)
    st = _lib.epq_pages_truncate(cache._ref, n, _queue(stream, at))
    if st:
        raise EpqError("epq_pages_truncate", st)


def epq_pages_fork(cache: PagedKVCache, src: torch.Tensor, dst: torch.Tensor, status: torch.Tensor | None = None,
                   stream=None) -> None:
    """Sequences dst (int32 [n], empty) become copies of src, sharing their pages; no entries: nothing happens."""
    n, at = dst.shape[0], cache._at
    a, b = _need(src, "src", torch.int32, (n,), at), _need(dst, "dst", torch.int32, (n,), at)
    c = None if status is None else _need(status, "status", torch.int32, (n,), at)
    if n:
        st = _lib.epq_pages_fork(cache._ref, a, b, n, c, _queue(stream, at))
        if st:
            raise EpqError("epq_pages_fork", st)


def epq_pages_reserve(cache: PagedKVCache, extra: torch.Tensor, status: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """Make extra (int32 [n_seq]) more positions of every sequence writable -> status int32 [n_seq]."""
    at = cache._at
    e = _need(extra, "extra", torch.int32, cache._per_seq, at)
    status, status_at = _result(status, "status", torch.int32, cache._per_seq, at, _allocator(stream), cache.device)
    st = _lib.epq_pages_reserve(cache._ref, e, status_at, _queue(stream, at))
    if st:
        raise EpqError("epq_pages_reserve", st)
    return status


def epq_pages_compact(cache: PagedKVCache, path: torch.Tensor, n_keep: torch.Tensor, stream=None) -> None:
    """Commit the drafted rows path (int32 [n_seq, ntok], n_keep int32 [n_seq] of them) in every layer."""
    ntok, at = path.shape[-1], cache._at
    a = _need(path, "path", torch.int32, (cache.n_seq, ntok), at)
    st = _lib.epq_pages_compact(cache._ref, a, _need(n_keep, "n_keep", torch.int32, cache._per_seq, at), ntok,
                                _queue(stream, at))
    if st:
        raise EpqError("epq_pages_compact", st)


# ------------------------------------------------------------------ tree step
def epq_tree_mask(parent: torch.Tensor, mask: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """parent int32 [n_seq, ntok] -> mask int64 [n_seq, ntok] (bit j: token j is i or an ancestor of i)."""
    if parent.dim() != 2:
        raise ValueError("parent must be [n_seq, ntok]")
    at = _place(parent)
    a = _need(parent, "parent", torch.int32, parent.shape, at)
    mask, b = _result(mask, "mask", torch.int64, parent.shape, at, _allocator(stream), parent.device)
    _check("epq_tree_mask", load().epq_tree_mask(a, parent.shape[0], parent.shape[1], b, _queue(stream, at)))
    return mask


def epq_attention_tree_workspace(cache: PagedKVCache, n_heads: int, ntok: int, stream=None) -> torch.Tensor:
    """A workspace for epq_attention_tree (on `stream`), to be kept between calls."""
    n = int(load().epq_attention_tree_workspace_bytes(cache._ref, n_heads, ntok))
    if n == 0:
        raise ValueError("sizes of the tree attention not supported")
    return _allocator(stream)(n, dtype=torch.uint8, device=cache.device)


def _token_strides(t, name, shape, at):
    """Floats between sequences and tokens of t [n_seq, ntok, n] (0: a dimension of one entry says nothing)."""
    if t.dtype is not torch.float32 or t.shape != shape or t.get_device() != at:
        _elsewhere(t, name, at)
        if t.dtype is not torch.float32 or t.shape != shape:
            raise ValueError(f"{name}: expected float32 {list(shape)}, got {t.dtype} {list(t.shape)}")
    a, b, c = t.stride()
    if c != 1 or (a == 0 and shape[0] > 1) or (b == 0 and shape[1] > 1):
        raise ValueError(f"{name}: rows must be contiguous and not broadcast")
    return a if shape[0] > 1 else 0, b if shape[1] > 1 else 0


def epq_attention_tree(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, cache: PagedKVCache, layer: int,
                       n_heads: int, scale: float, mask: torch.Tensor | None = None,
                       n_tok: torch.Tensor | None = None, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [n_seq, ntok, n_heads*D], k_new/v_new [n_seq, ntok, n_kv*D] (float32; views of one wider buffer are
    read in place) -> out [n_seq, ntok, n_heads*D]; the new rows are stored behind the committed positions."""
    ntok, nseq, D, at = q.shape[1], cache.n_seq, cache.head_dim, cache._at
    shape = (nseq, ntok, n_heads * D)
    q_seq, q_tok = _token_strides(q, "q", shape, at)
    kv = (nseq, ntok, cache.n_kv_heads * D)
    kv_seq, kv_tok = _token_strides(k_new, "k_new", kv, at)
    if _token_strides(v_new, "v_new", kv, at) != (kv_seq, kv_tok):
        raise ValueError("k_new and v_new must have the same strides")
    out, out_at = _result(out, "out", torch.float32, shape, at, _allocator(stream), cache.device)
    if workspace is None:
        workspace = epq_attention_tree_workspace(cache, n_heads, ntok, stream)
    o = AttentionTreeOpts(None if mask is None else _need(mask, "mask", torch.int64, (nseq, ntok), at),
                          None if n_tok is None else _need(n_tok, "n_tok", torch.int32, cache._per_seq, at),
                          q_tok, q_seq, kv_tok, kv_seq)
    st = _lib.epq_attention_tree(cache._ref, layer, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), n_heads, ntok,
                                 scale, ctypes.byref(o), out_at, *_scratch(workspace, at), _queue(stream, at))
    if st:
        raise EpqError("epq_attention_tree", st)
    return out


def epq_verify_tree_workspace(logits: torch.Tensor, stream=None) -> torch.Tensor:
    """A workspace for epq_verify_tree (on `stream`) on logits of this shape."""
    n = int(load().epq_verify_tree_workspace_bytes(logits.shape[0], logits.shape[1], logits.shape[2]))
    if n == 0:
        raise ValueError("sizes of the verification not supported")
    return _allocator(stream)(n, dtype=torch.uint8, device=logits.device)


def epq_verify_tree(logits: torch.Tensor, tokens: torch.Tensor, parent: torch.Tensor, u: torch.Tensor | None = None,
                    draft: torch.Tensor | None = None, n_tok: torch.Tensor | None = None, temperature: float = 1.0,
                    path: torch.Tensor | None = None, n_accept: torch.Tensor | None = None,
                    next_token: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None):
    """logits float32 [n_seq, ntok, vocab], tokens/parent int32 and u float32 [n_seq, ntok], draft None or float32
    like logits -> (path int32 [n_seq, ntok], n_accept int32 [n_seq], next_token int32 [n_seq], lse float32
    [n_seq, ntok])."""
    lib = load()
    i32, f32, dev = torch.int32, torch.float32, logits.device
    if logits.dim() != 3:
        raise ValueError("logits must be [n_seq, ntok, vocab]")
    full = logits.shape
    nseq, ntok, vocab = full
    tree, each = (nseq, ntok), (nseq,)
    at, new = _place(logits), _allocator(stream)
    path, path_at = _result(path, "path", i32, tree, at, new, dev)
    n_accept, n_at = _result(n_accept, "n_accept", i32, each, at, new, dev)
    next_token, next_at = _result(next_token, "next_token", i32, each, at, new, dev)
    lse, lse_at = _result(lse, "lse", f32, tree, at, new, dev)
    if workspace is None:
        workspace = epq_verify_tree_workspace(logits, stream)
    o = VerifyOpts(None if draft is None else _need(draft, "draft", f32, full, at),
                   None if n_tok is None else _need(n_tok, "n_tok", i32, each, at), temperature, 0, 0)
    st = lib.epq_verify_tree(
        _need(logits, "logits", f32, full, at), vocab, _need(tokens, "tokens", i32, tree, at),
        _need(parent, "parent", i32, tree, at), None if u is None else _need(u, "u", f32, tree, at), nseq, ntok,
        ctypes.byref(o), path_at, n_at, next_at, lse_at, *_scratch(workspace, at), _queue(stream, at))
    if st:
        raise EpqError("epq_verify_tree", st)
    return path, n_accept, next_token, lse


# ------------------------------------------------------------------ rotary positions
def epq_rope_frequencies(rot_dim: int, base: float = 10000.0, kind: int = EPQ_ROPE_PLAIN, factor: float = 1.0,
                         context: float | None = None, low: float | None = None, high: float | None = None):
    """(float64 [rot_dim / 2] on the host, magnitude): the angles per position and what the cosines and sines are
    multiplied by; context: the trained one, which EPQ_ROPE_PARTS and EPQ_ROPE_BANDS ask for; low, high: turns over it
    (None: the kind's usual ones)."""
    if context is None:
        if kind in (EPQ_ROPE_PARTS, EPQ_ROPE_BANDS):
            raise ValueError("this kind of scaling needs the context that the frequencies were trained for")
        context = 1.0
    usual = (1.0, 4.0) if kind == EPQ_ROPE_BANDS else (1.0, 32.0)
    sc = RopeScaling(kind, factor, context, usual[0] if low is None else low, usual[1] if high is None else high)
    freq, mag = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.float64), ctypes.c_double()
    _check("epq_rope_frequencies", load().epq_rope_frequencies(
        rot_dim, base, ctypes.byref(sc), ctypes.cast(freq.data_ptr(), ctypes.POINTER(ctypes.c_double)),
        ctypes.byref(mag)))
    return freq, mag.value


class RopeTable:
    """A rotation (epq_rotation): cosines and sines of positions 0..n_pos-1, float32 [n_pos, rot_dim / 2, 2], for
    the elements first .. first + rot_dim - 1 of a head.  The further arguments are those of epq_rope_frequencies."""

    def __init__(self, rot_dim: int, n_pos: int, base: float = 10000.0, first: int = 0, interleaved: bool = False,
                 device="cuda", **scaling):
        freq, magnitude = epq_rope_frequencies(rot_dim, base, **scaling)
        freq = freq.to(device)
        table = torch.empty((n_pos, rot_dim // 2, 2), dtype=torch.float32, device=device)
        _check("epq_rope_table", load().epq_rope_table(freq.data_ptr(), rot_dim, magnitude, n_pos, table.data_ptr(),
                                                       _launch_on(None, _place(table))))
        self._bind(table, first, interleaved)

    @classmethod
    def over(cls, table: torch.Tensor, first: int = 0, interleaved: bool = False) -> "RopeTable":
        """A rotation by a table that the caller holds."""
        self = cls.__new__(cls)
        self._bind(table, first, interleaved)
        return self

    def _bind(self, table, first, interleaved):
        if table.dim() != 3 or table.shape[2] != 2:
            raise ValueError("table must be [n_pos, rot_dim / 2, 2]")
        self._at = _place(table)
        _need(table, "table", torch.float32, table.shape, self._at)
        load()
        self.table, self.first, self.interleaved = table, first, bool(interleaved)
        self.n_pos, self.rot_dim = table.shape[0], 2 * table.shape[1]
        self._r = Rotation(table.data_ptr(), self.n_pos, self.rot_dim, first, int(self.interleaved))
        self._ref, self._address = ctypes.byref(self._r), ctypes.addressof(self._r)


def epq_rope(x: torch.Tensor, rope: RopeTable, n_heads: int, position: torch.Tensor | None = None,
             start: torch.Tensor | None = None, mask: torch.Tensor | None = None, n_tok: torch.Tensor | None = None,
             out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x float32 [n_seq, ntok, n_heads*D] (a view of a wider buffer is read in place) -> out, the heads turned by
    their tokens' positions; out may be x.  position int32 [n_seq, ntok], or start int32 [n_seq] plus the token's
    index (mask int64 [n_seq, ntok]: plus its ancestors in the tree)."""
    if x.dim() != 3:
        raise ValueError("x must be [n_seq, ntok, n_heads * head_dim]")
    nseq, ntok, width = shape = x.shape
    at = rope._at
    if n_heads < 1 or width % n_heads:
        raise ValueError(f"{width} elements are not {n_heads} heads")
    x_seq, x_tok = _token_strides(x, "x", shape, at)
    if out is None:
        out, y_seq, y_tok = _allocator(stream)(shape, dtype=torch.float32, device=x.device), 0, 0
    else:
        y_seq, y_tok = _token_strides(out, "out", shape, at)
    i32 = torch.int32
    o = RopeOpts(None if position is None else _need(position, "position", i32, (nseq, ntok), at),
                 None if start is None else _need(start, "start", i32, (nseq,), at),
                 None if mask is None else _need(mask, "mask", torch.int64, (nseq, ntok), at),
                 None if n_tok is None else _need(n_tok, "n_tok", i32, (nseq,), at), x_tok, x_seq, y_tok, y_seq)
    st = _lib.epq_rope(rope._ref, x.data_ptr(), out.data_ptr(), nseq, ntok, n_heads, width // n_heads,
                       ctypes.byref(o), _launch_on(stream, at))
    if st:
        raise EpqError("epq_rope", st)
    return out


# ------------------------------------------------------------------ a prompt's rows
def epq_pages_append(k: torch.Tensor, v: torch.Tensor, cache: PagedKVCache, layer: int, rope: RopeTable | None = None,
                     position: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                     n_tok: torch.Tensor | None = None, stream=None) -> None:
    """k, v float32 [n_seq, ntok, n_kv*D] (views of one wider buffer are read in place): the rows are stored behind
    the committed positions of one layer, the keys turned by `rope` (positions as in epq_rope, start = the lengths).
    n_tok is 0 for a sequence whose reservation was refused: its last page may be shared."""
    if k.dim() != 3:
        raise ValueError("k must be [n_seq, ntok, n_kv * head_dim]")
    ntok, nseq, at = k.shape[1], cache.n_seq, cache._at
    kv = (nseq, ntok, cache.n_kv_heads * cache.head_dim)
    kv_seq, kv_tok = _token_strides(k, "k", kv, at)
    if _token_strides(v, "v", kv, at) != (kv_seq, kv_tok):
        raise ValueError("k and v must have the same strides")
    if rope is not None and rope._at != at:
        _elsewhere(rope.table, "rope", at)
    o = AppendOpts(None if rope is None else rope._address,
                   None if position is None else _need(position, "position", torch.int32, (nseq, ntok), at),
                   None if mask is None else _need(mask, "mask", torch.int64, (nseq, ntok), at),
                   None if n_tok is None else _need(n_tok, "n_tok", torch.int32, cache._per_seq, at), kv_tok, kv_seq)
    st = _lib.epq_pages_append(cache._ref, layer, k.data_ptr(), v.data_ptr(), ntok, ctypes.byref(o),
                               _launch_on(stream, at))
    if st:
        raise EpqError("epq_pages_append", st)


def epq_pages_advance(cache: PagedKVCache, n: torch.Tensor, stream=None) -> None:
    """Commit n (int32 [n_seq]; 0 where the reservation was refused) appended positions of every sequence."""
    at = cache._at
    st = _lib.epq_pages_advance(cache._ref, _need(n, "n", torch.int32, cache._per_seq, at), _launch_on(stream, at))
    if st:
        raise EpqError("epq_pages_advance", st)


def epq_attention_prompt_workspace(cache: PagedKVCache, n_heads: int, ntok: int, stream=None) -> torch.Tensor:
    """A workspace for epq_attention_prompt (on `stream`), to be kept between calls."""
    n = int(load().epq_attention_prompt_workspace_bytes(cache._ref, n_heads, ntok))
    if n == 0:
        raise ValueError("sizes of the prompt attention not supported")
    return _allocator(stream)(n, dtype=torch.uint8, device=cache.device)


def epq_attention_prompt(q: torch.Tensor, cache: PagedKVCache, layer: int, n_heads: int, scale: float, window: int = 0,
                         n_tok: torch.Tensor | None = None, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q [n_seq, ntok, n_heads*D] (float32; a view of a wider buffer is read in place) -> out [n_seq, ntok, n_heads*D]:
    token i of a sequence attends to its positions 0..length + i, the last `window` of them if that is not 0; the
    tokens' own rows have been stored by epq_pages_append."""
    if q.dim() != 3:
        raise ValueError("q must be [n_seq, ntok, n_heads * head_dim]")
    if window >> 31 > 0:
        raise ValueError("window must be below 2^31")
    ntok, at = q.shape[1], cache._at
    shape = (cache.n_seq, ntok, n_heads * cache.head_dim)
    q_seq, q_tok = _token_strides(q, "q", shape, at)
    out, out_at = _result(out, "out", torch.float32, shape, at, _allocator(stream), cache.device)
    if workspace is None:
        workspace = epq_attention_prompt_workspace(cache, n_heads, ntok, stream)
    o = PromptOpts(None if n_tok is None else _need(n_tok, "n_tok", torch.int32, cache._per_seq, at), window, q_tok,
                   q_seq)
    st = _lib.epq_attention_prompt(cache._ref, layer, q.data_ptr(), n_heads, ntok, scale, ctypes.byref(o), out_at,
                                   *_scratch(workspace, at), _launch_on(stream, at))
    if st:
        raise EpqError("epq_attention_prompt", st)
    return out


# ------------------------------------------------------------------ logits
def epq_logits_adjust(logits: torch.Tensor, penalties: torch.Tensor | None = None, history: torch.Tensor | None = None,
                      history_len: torch.Tensor | None = None, prompt_len: torch.Tensor | None = None,
                      tokens: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                      n_tok: torch.Tensor | None = None, bias_ids: torch.Tensor | None = None,
                      bias: torch.Tensor | None = None, allowed: torch.Tensor | None = None,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """logits float32 [n_seq, ntok, vocab] -> out (may be logits): biases (bias_ids int32, bias float32 [n_seq,
    n_bias]), penalties (float32 [n_seq, 3]: repetition, frequency, presence) for the tokens of history (int32
    [n_seq, max_history]; history_len, prompt_len int32 [n_seq]) and of tokens (int32 [n_seq, ntok]; mask int64
    [n_seq, ntok]: a row's path in the tree), and -inf for what allowed (int32 [n_seq, ntok, ceil(vocab / 32)], bits)
    leaves out."""
    if logits.dim() != 3:
        raise ValueError("logits must be [n_seq, ntok, vocab]")
    full = logits.shape
    nseq, ntok, vocab = full
    at, i32, f32 = _place(logits), torch.int32, torch.float32
    each, tree = (nseq,), (nseq, ntok)
    if bias_ids is not None and (bias is None or bias_ids.dim() != 2) or bias_ids is None and bias is not None:
        raise ValueError("bias_ids and bias must be [n_seq, n_bias] both")
    if history is not None and history.dim() != 2:
        raise ValueError("history must be [n_seq, max_history]")
    nh, nb = 0 if history is None else history.shape[1], 0 if bias is None else bias_ids.shape[1]
    src = _need(logits, "logits", f32, full, at)
    out, dst = _result(out, "out", f32, full, at, _allocator(stream), logits.device)
    o = LogitsOpts(None if penalties is None else _need(penalties, "penalties", f32, (nseq, 3), at),
                   None if history is None else _need(history, "history", i32, (nseq, nh), at),
                   None if history_len is None else _need(history_len, "history_len", i32, each, at),
                   None if prompt_len is None else _need(prompt_len, "prompt_len", i32, each, at), nh,
                   None if tokens is None else _need(tokens, "tokens", i32, tree, at),
                   None if mask is None else _need(mask, "mask", torch.int64, tree, at),
                   None if n_tok is None else _need(n_tok, "n_tok", i32, each, at),
                   None if bias_ids is None else _need(bias_ids, "bias_ids", i32, (nseq, nb), at),
                   None if bias is None else _need(bias, "bias", f32, (nseq, nb), at), nb,
                   None if allowed is None else _need(allowed, "allowed", i32, (nseq, ntok, (vocab + 31) // 32), at),
                   0, 0)
    st = load().epq_logits_adjust(src, vocab, nseq, ntok, ctypes.byref(o), dst, _launch_on(stream, at))
    if st:
        raise EpqError("epq_logits_adjust", st)
    return out
