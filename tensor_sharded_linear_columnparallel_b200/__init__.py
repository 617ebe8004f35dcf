"""Python binding of libtps.so, the tensor-sharded (column/row-parallel) linear
block for one B200 (sm_100a).

Argument marshalling only: every function below checks tensor dtypes/devices,
allocates outputs with torch when none are given (PyTorch is the device-memory
and stream plumbing), and calls the C entry point of the same name declared in
include/tps.h. Every step of the block's arithmetic runs in the library's CUDA
kernels. There is no fallback: if libtps.so is missing or cannot be loaded,
importing this package raises.

Weights use the math orientation W[k, n] (Y = X W) unless ``transposed=True``.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtps.so")

# ---------------------------------------------------------------- constants (tps.h)
TPS_OK = 0
TPS_ERR_ARG = -1
TPS_ERR_DIVISIBILITY = -2
TPS_ERR_ALIGN = -3
TPS_ERR_DTYPE = -4
TPS_ERR_WORKSPACE = -5
TPS_ERR_CUDA = -6
TPS_ERR_TIMEOUT = -7
TPS_ERR_UNIMPLEMENTED = -8
TPS_ERR_DEVICE = -9

KIND_COLUMN, KIND_ROW, KIND_QKV, KIND_GATE_UP = 0, 1, 2, 3
ACT_NONE, ACT_GELU, ACT_SILU_MUL = 0, 1, 2
DTYPE_BF16, DTYPE_F32 = 0, 1
REDUCE_FUSED, REDUCE_PARTIALS, REDUCE_BF16 = 0, 1, 2
FN_COLUMN, FN_ROW, FN_MLP, FN_ATTN, FN_ARGMAX, FN_SAMPLE = 0, 1, 2, 3, 4, 5

PLAN_AUTO, PLAN_TOKEN_MAJOR, PLAN_WEIGHT_MAJOR = 0, 1, 2
PLAN_FORCE_SPLITK, PLAN_NO_SPLITK = 16, 32


def plan_width(cols: int) -> int:
    """Plan-override bits forcing the tile width (16, 32, 64, 128 or 256 columns)."""
    return {16: 1, 32: 2, 64: 3, 128: 4, 256: 5}[cols] << 8

EXPORTED = (
    "tp_head_map", "tp_packed_bytes", "tp_shard_weights", "column_parallel_forward",
    "row_parallel_forward", "shard_partial_reduce", "sharded_mlp_forward",
    "sharded_attn_proj_forward", "tps_workspace_bytes", "tps_status_string",
    "tps_device_error", "tps_set_plan_override", "tps_debug_wait_timeout",
    "row_parallel_forward_noalloc", "vocab_parallel_argmax", "sharded_gqa_attention", "tps_sync_status",
    "shard_partial_reduce_bf16", "sharded_window_attention", "sharded_kv_append", "sharded_window_decode",
    "sharded_prefix_decode", "tps_decode_workspace_bytes", "logits_sample", "vocab_parallel_sample",
)


class TpsError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


class tps_heads(ctypes.Structure):
    _fields_ = [("hq", ctypes.c_int32), ("hkv", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


@dataclass(frozen=True)
class Heads:
    hq: int
    hkv: int
    head_dim: int

    def c(self) -> tps_heads:
        return tps_heads(self.hq, self.hkv, self.head_dim)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python tensor_sharded_linear_columnparallel_b200/build.py` "
            "(there is no CPU or PyTorch fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    HP = ctypes.POINTER(tps_heads)
    I32P = ctypes.POINTER(ctypes.c_int32)
    sig = {
        "tp_head_map": (I, [I, I, I, I32P, I32P, I32P, I32P]),
        "tp_packed_bytes": (SZ, [I, I64, I64, I, HP]),
        "tp_shard_weights": (I, [I, P, I, I64, I64, I, HP, P, SZ, P]),
        "column_parallel_forward": (I, [P, I64, I64, P, I, I64, I, HP, P, I, P, I, P, SZ, P]),
        "row_parallel_forward": (I, [P, I64, I64, P, I64, I, P, I, P, P, I, P, SZ, P]),
        "shard_partial_reduce": (I, [P, I, I64, I64, P, P, I, P]),
        "shard_partial_reduce_bf16": (I, [P, I, I64, I64, P, P, I, P]),
        "sharded_mlp_forward": (I, [P, I64, I64, I64, I, I, P, P, P, P, I, P, SZ, P]),
        "sharded_attn_proj_forward": (I, [P, P, I64, I64, HP, I, P, P, P, P, I, P, SZ, P]),
        "tps_workspace_bytes": (SZ, [I, I64, I64, I64, I]),
        "tps_status_string": (ctypes.c_char_p, [I]),
        "tps_device_error": (I, [P]),
        "tps_set_plan_override": (I, [I]),
        "tps_debug_wait_timeout": (I, [I, P, SZ, P]),
        "tps_sync_status": (I, [P, P]),
        "row_parallel_forward_noalloc": (I, [P, I64, I64, P, I64, I, P, P, I, P]),
        "vocab_parallel_argmax": (I, [P, I64, I64, P, I64, I, P, P, P, SZ, P]),
        "sharded_gqa_attention": (I, [P, I64, I64, HP, I, I, P, P]),
        "sharded_window_attention": (I, [P, I64, I64, HP, I, I64, I64, P, P]),
        "sharded_kv_append": (I, [P, I64, I64, HP, I, P, P, I64, P, P, I64, P]),
        "sharded_window_decode": (I, [P, I64, HP, I, P, I64, I64, P, P, I64, P, P, SZ, P]),
        "sharded_prefix_decode": (I, [P, I64, HP, I, P, P, I64, P, P, P, I64, P, P, SZ, P]),
        "tps_decode_workspace_bytes": (SZ, [I64, HP, I, I64]),
        "logits_sample": (I, [P, I, I64, I64, P, P, P, P, P, P, P, P]),
        "vocab_parallel_sample": (I, [P, I64, I64, P, I64, I, P, P, P, P, P, P, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


# ---------------------------------------------------------------- helpers
def status_string(status: int) -> str:
    return lib.tps_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != TPS_OK:
        raise TpsError(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev(t: torch.Tensor, what: str, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t


def _ydtype(dt) -> int:
    if dt in (torch.bfloat16, DTYPE_BF16):
        return DTYPE_BF16
    if dt in (torch.float32, DTYPE_F32):
        return DTYPE_F32
    raise ValueError(f"unsupported output dtype {dt}")


def _torch_dtype(code: int):
    return torch.bfloat16 if code == DTYPE_BF16 else torch.float32


def _heads_ref(heads):
    if heads is None:
        return None
    h = heads.c() if isinstance(heads, Heads) else heads
    return ctypes.byref(h)


# ---------------------------------------------------------------- host-only queries
def tp_head_map(hq: int, hkv: int, tp: int):
    """(q_first, q_count, kv_first, kv_count) lists of length tp."""
    arrs = [(ctypes.c_int32 * tp)() for _ in range(4)]
    _check(lib.tp_head_map(hq, hkv, tp, *arrs), "tp_head_map")
    return tuple(list(a) for a in arrs)


def tp_packed_bytes(kind: int, k: int, n: int, tp: int, heads=None) -> int:
    h = heads.c() if isinstance(heads, Heads) else heads
    return lib.tp_packed_bytes(kind, k, n, tp, ctypes.byref(h) if h is not None else None)


def tps_workspace_bytes(fn: int, m: int, n: int, k: int, tp: int) -> int:
    return lib.tps_workspace_bytes(fn, m, n, k, tp)


def tps_set_plan_override(plan: int) -> int:
    return lib.tps_set_plan_override(plan)


def tps_device_error(stream=None) -> int:
    return lib.tps_device_error(_stream(stream))


def tps_sync_status(ws: torch.Tensor, stream=None) -> int:
    """Status of the calls given workspace `ws` (its status word, read and cleared)."""
    _dev(ws, "ws")
    return lib.tps_sync_status(_ptr(ws), _stream(stream))


def tps_debug_wait_timeout(timeout_us: int, ws: torch.Tensor | None = None, stream=None) -> None:
    _check(lib.tps_debug_wait_timeout(timeout_us, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                      _stream(stream)), "tps_debug_wait_timeout")


def workspace(fn: int, m: int, n: int, k: int, tp: int, device=None) -> torch.Tensor:
    """Zero-filled workspace buffer of tps_workspace_bytes(...) bytes."""
    nbytes = tps_workspace_bytes(fn, m, n, k, tp)
    return torch.zeros(max(nbytes, 16), dtype=torch.uint8, device="cuda" if device is None else device)


# ---------------------------------------------------------------- entry points
def tp_shard_weights(kind: int, W: torch.Tensor, tp: int, heads=None, transposed: bool = False,
                     out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Packs W (bf16, [k, n], or [n, k] if transposed) into its tp shards."""
    _dev(W, "W", torch.bfloat16)
    if W.dim() != 2:
        raise ValueError("W must be 2-D")
    k, n = (W.shape[1], W.shape[0]) if transposed else (W.shape[0], W.shape[1])
    nbytes = tp_packed_bytes(kind, k, n, tp, heads)
    if nbytes == 0:
        raise TpsError(TPS_ERR_ARG if kind not in (0, 1, 2, 3) else TPS_ERR_DIVISIBILITY, "tp_packed_bytes")
    if out is None:
        out = torch.empty(nbytes // 2, dtype=torch.bfloat16, device=W.device)
    _dev(out, "out")
    _check(lib.tp_shard_weights(kind, _ptr(W), int(transposed), k, n, tp, _heads_ref(heads), _ptr(out),
                                out.numel() * out.element_size(), _stream(stream)), "tp_shard_weights")
    return out


def column_parallel_forward(X: torch.Tensor, packed_w: torch.Tensor, kind: int, n: int, tp: int,
                            heads=None, bias=None, act: int = ACT_NONE, out=None,
                            y_dtype=torch.bfloat16, ws: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """concat_i act(X W_i + b_i); n is the logical column count of the packed weight."""
    _dev(X, "X", torch.bfloat16)
    _dev(packed_w, "packed_w", torch.bfloat16)
    m, k = X.shape
    yd = _ydtype(y_dtype)
    if out is None:
        if kind == KIND_COLUMN:
            n_out = n
        elif kind == KIND_GATE_UP:
            n_out = n // 2
        else:
            _, qc, _, kc = tp_head_map(heads.hq, heads.hkv, tp)
            n_out = tp * (qc[0] + 2 * kc[0]) * heads.head_dim
        out = torch.empty(m, n_out, dtype=_torch_dtype(yd), device=X.device)
    _dev(out, "out")
    if bias is not None:
        _dev(bias, "bias", torch.bfloat16)
    _check(lib.column_parallel_forward(_ptr(X), m, k, _ptr(packed_w), kind, n, tp, _heads_ref(heads), _ptr(bias),
                                       act, _ptr(out), yd, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                       _stream(stream)), "column_parallel_forward")
    return out


def row_parallel_forward(X: torch.Tensor, packed_v: torch.Tensor, n: int, tp: int, bias=None,
                         reduce_mode: int = REDUCE_FUSED, partials: torch.Tensor | None = None, out=None,
                         y_dtype=torch.bfloat16, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """sum_i X_i V_i (+ bias once)."""
    _dev(X, "X", torch.bfloat16)
    _dev(packed_v, "packed_v", torch.bfloat16)
    m, k = X.shape
    yd = _ydtype(y_dtype)
    if out is None:
        out = torch.empty(m, n, dtype=_torch_dtype(yd), device=X.device)
    _dev(out, "out")
    if bias is not None:
        _dev(bias, "bias", torch.bfloat16)
    if reduce_mode == REDUCE_PARTIALS and partials is None:
        partials = torch.empty(tp, m, n, dtype=torch.float32, device=X.device)
    if partials is not None:
        _dev(partials, "partials", torch.float32)
    _check(lib.row_parallel_forward(_ptr(X), m, k, _ptr(packed_v), n, tp, _ptr(bias), reduce_mode, _ptr(partials),
                                    _ptr(out), yd, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                    _stream(stream)), "row_parallel_forward")
    return out


def shard_partial_reduce(partials: torch.Tensor, bias=None, out=None, y_dtype=torch.bfloat16,
                         stream=None, bf16_exchange: bool = False) -> torch.Tensor:
    """Y = sum over dim 0 of partials [tp, m, n] (fp32, shard order) + bias; with
    bf16_exchange, shard_partial_reduce_bf16 (bf16 partials, rounded after every
    addition)."""
    _dev(partials, "partials", torch.float32)
    tp, m, n = partials.shape
    yd = _ydtype(y_dtype)
    if out is None:
        out = torch.empty(m, n, dtype=_torch_dtype(yd), device=partials.device)
    _dev(out, "out")
    if bias is not None:
        _dev(bias, "bias", torch.bfloat16)
    fn = lib.shard_partial_reduce_bf16 if bf16_exchange else lib.shard_partial_reduce
    _check(fn(_ptr(partials), tp, m, n, _ptr(bias), _ptr(out), yd, _stream(stream)),
           "shard_partial_reduce_bf16" if bf16_exchange else "shard_partial_reduce")
    return out


def sharded_mlp_forward(X: torch.Tensor, H: int, I: int, tp: int, act: int, packed_up: torch.Tensor,
                        packed_down: torch.Tensor, h_ws=None, out=None, y_dtype=torch.bfloat16,
                        ws: torch.Tensor | None = None, stream=None):
    """MLP block: h = act(column(X)), Y = row(h). Returns (Y, h)."""
    _dev(X, "X", torch.bfloat16)
    m = X.shape[0]
    yd = _ydtype(y_dtype)
    if h_ws is None:
        h_ws = torch.empty(m, I, dtype=torch.bfloat16, device=X.device)
    if out is None:
        out = torch.empty(m, H, dtype=_torch_dtype(yd), device=X.device)
    _dev(h_ws, "h_ws", torch.bfloat16)
    _dev(out, "out")
    _check(lib.sharded_mlp_forward(_ptr(X), m, H, I, tp, act, _ptr(packed_up), _ptr(packed_down), _ptr(h_ws),
                                   _ptr(out), yd, _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                   _stream(stream)), "sharded_mlp_forward")
    return out, h_ws


def vocab_parallel_argmax(X: torch.Tensor, H: int, V: int, tp: int, packed_w: torch.Tensor,
                          ws: torch.Tensor | None = None, out_idx=None, out_val=None, stream=None):
    """Greedy token per row of X over a vocab-parallel lm_head (COLUMN pack of
    W[H, V]): each shard's local argmax, then the max over shards. Returns
    (indices int32 [m], max logits fp32 [m])."""
    _dev(X, "X", torch.bfloat16)
    m = X.shape[0]
    if ws is None:
        ws = workspace(FN_ARGMAX, m, V, H, tp, device=X.device)
    if out_idx is None:
        out_idx = torch.empty(m, dtype=torch.int32, device=X.device)
    if out_val is None:
        out_val = torch.empty(m, dtype=torch.float32, device=X.device)
    _check(lib.vocab_parallel_argmax(_ptr(X), m, H, _ptr(packed_w), V, tp, _ptr(out_idx), _ptr(out_val), _ptr(ws),
                                     ws.numel() * ws.element_size(), _stream(stream)), "vocab_parallel_argmax")
    return out_idx, out_val


def sharded_gqa_attention(qkv: torch.Tensor, nseq: int, seqlen: int, heads: Heads, tp: int, causal: bool = True,
                          out=None, stream=None):
    """Attention on local heads over a QKV-kind column output (shard-major
    [q | k | v] blocks). Returns attn_out [nseq*seqlen, hq*d] bf16, query head h
    at columns [h*d, (h+1)*d)."""
    _dev(qkv, "qkv", torch.bfloat16)
    m = nseq * seqlen
    if out is None:
        out = torch.empty(m, heads.hq * heads.head_dim, dtype=torch.bfloat16, device=qkv.device)
    _dev(out, "out", torch.bfloat16)
    _check(lib.sharded_gqa_attention(_ptr(qkv), nseq, seqlen, _heads_ref(heads), tp, 1 if causal else 0, _ptr(out),
                                     _stream(stream)), "sharded_gqa_attention")
    return out


def sharded_attn_proj_forward(X: torch.Tensor, attn_out: torch.Tensor, H: int, heads: Heads, tp: int,
                              packed_qkv: torch.Tensor, packed_o: torch.Tensor, qkv_out=None, out=None,
                              y_dtype=torch.bfloat16, ws: torch.Tensor | None = None, stream=None):
    """QKV (column by head) and o_proj (row by head). Returns (Y, qkv_out)."""
    _dev(X, "X", torch.bfloat16)
    _dev(attn_out, "attn_out", torch.bfloat16)
    m = X.shape[0]
    yd = _ydtype(y_dtype)
    if qkv_out is None:
        _, qc, _, kc = tp_head_map(heads.hq, heads.hkv, tp)
        qkv_out = torch.empty(m, tp * (qc[0] + 2 * kc[0]) * heads.head_dim, dtype=torch.bfloat16, device=X.device)
    if out is None:
        out = torch.empty(m, H, dtype=_torch_dtype(yd), device=X.device)
    _dev(qkv_out, "qkv_out", torch.bfloat16)
    _dev(out, "out")
    _check(lib.sharded_attn_proj_forward(_ptr(X), _ptr(attn_out), m, H, _heads_ref(heads), tp, _ptr(packed_qkv),
                                         _ptr(packed_o), _ptr(qkv_out), _ptr(out), yd, _ptr(ws),
                                         0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)),
           "sharded_attn_proj_forward")
    return out, qkv_out


def row_parallel_forward_noalloc(X: torch.Tensor, packed_v: torch.Tensor, n: int, tp: int, bias=None, out=None,
                                 y_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """row_parallel_forward for callers that cannot provide a workspace: the
    split-K scratch is the library's own static device array (m <= 64 tokens;
    concurrent calls on unordered streams race on it)."""
    _dev(X, "X", torch.bfloat16)
    _dev(packed_v, "packed_v", torch.bfloat16)
    m, k = X.shape
    yd = _ydtype(y_dtype)
    if out is None:
        out = torch.empty(m, n, dtype=_torch_dtype(yd), device=X.device)
    _dev(out, "out")
    if bias is not None:
        _dev(bias, "bias", torch.bfloat16)
    _check(lib.row_parallel_forward_noalloc(_ptr(X), m, k, _ptr(packed_v), n, tp, _ptr(bias), _ptr(out), yd,
                                            _stream(stream)), "row_parallel_forward_noalloc")
    return out


# ---------------------------------------------------------------- serving: windows, caches, sampling
# These calls run many times per second on little work, so their host side costs as little
# as it can: one check per tensor, the raw stream (torch.cuda.current_stream() alone takes
# 3 us), and a device or stream switch only where the call needs one.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _here(dev: int, stream) -> bool:
    """Whether the call can run as it is: no stream given, and the tensors' device current."""
    return stream is None and torch.cuda.current_device() == dev


@contextlib.contextmanager
def _there(dev: int, stream):
    """The tensors' device, and the given stream of it, made current: outputs are then
    allocated on the stream that writes them."""
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream of {stream.device}, tensors on cuda:{dev}")
    with torch.cuda.device(dev):
        with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
            yield


def _arg(t, what: str, dtype, shape, dev: int | None) -> int | None:
    """Address of a dense CUDA tensor of the given type and shape (None: any) on device
    dev (None: any), or None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    on = t.get_device()
    if on < 0 or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dev is not None and on != dev:
        raise ValueError(f"{what} is on cuda:{on}, other arguments on cuda:{dev}")
    return t.data_ptr()


def _need(t, what: str):
    if t is None:
        raise TypeError(f"{what} must be a torch.Tensor")
    return t


@functools.lru_cache(maxsize=256)
def _geometry(heads: Heads, tp: int):
    """(columns of a QKV output row, KV head slots tp*kvs, columns of an attention output
    row, the C struct)."""
    _, qc, _, kc = tp_head_map(heads.hq, heads.hkv, tp)
    return tp * (qc[0] + 2 * kc[0]) * heads.head_dim, tp * kc[0], heads.hq * heads.head_dim, heads.c()


def _cache_args(k_cache, v_cache, nseq: int, nkv: int, d: int, dev: int):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [nseq, tp*kvs, cap, d]")
    cap = k_cache.shape[2]
    shape = (nseq, nkv, cap, d)
    return (_arg(_need(k_cache, "k_cache"), "k_cache", torch.bfloat16, shape, dev),
            _arg(_need(v_cache, "v_cache"), "v_cache", torch.bfloat16, shape, dev), cap)


def sharded_window_attention(qkv: torch.Tensor, nseq: int, seqlen: int, heads: Heads, tp: int, window: int,
                             nsink: int = 0, out=None, stream=None):
    """sharded_gqa_attention (causal) where query t sees the last `window` tokens, itself
    included, and the first `nsink`. Returns attn_out [nseq*seqlen, hq*d] bf16."""
    cols, _, ocols, hd = _geometry(heads, tp)
    m = nseq * seqlen
    pq = _arg(_need(qkv, "qkv"), "qkv", torch.bfloat16, (m, cols), None)
    dev = qkv.get_device()
    po = _arg(out, "out", torch.bfloat16, (m, ocols), dev)
    if not _here(dev, stream):
        with _there(dev, stream):
            return sharded_window_attention(qkv, nseq, seqlen, heads, tp, window, nsink, out)
    if out is None:
        out = torch.empty(m, ocols, dtype=torch.bfloat16, device=qkv.device)
        po = out.data_ptr()
    _check(lib.sharded_window_attention(pq, nseq, seqlen, ctypes.byref(hd), tp, window, nsink, po, _raw_stream(dev)),
           "sharded_window_attention")
    return out


def sharded_kv_append(qkv: torch.Tensor, nseq: int, seqlen: int, heads: Heads, tp: int, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, pos=None, count=None, nsink: int = 0, stream=None) -> None:
    """Writes the K and V of a QKV output to the caches [nseq, tp*kvs, cap, d]: token i of
    sequence b, i < count[b], at position pos[b] + i (int32 [nseq]; None: 0 and seqlen)."""
    cols, nkv, _, hd = _geometry(heads, tp)
    pq = _arg(_need(qkv, "qkv"), "qkv", torch.bfloat16, (nseq * seqlen, cols), None)
    dev = qkv.get_device()
    pk, pv, cap = _cache_args(k_cache, v_cache, nseq, nkv, heads.head_dim, dev)
    pp = _arg(pos, "pos", torch.int32, (nseq,), dev)
    pc = _arg(count, "count", torch.int32, (nseq,), dev)
    if not _here(dev, stream):
        with _there(dev, stream):
            return sharded_kv_append(qkv, nseq, seqlen, heads, tp, k_cache, v_cache, pos, count, nsink)
    _check(lib.sharded_kv_append(pq, nseq, seqlen, ctypes.byref(hd), tp, pp, pc, nsink, pk, pv, cap,
                                 _raw_stream(dev)), "sharded_kv_append")


def tps_decode_workspace_bytes(nseq: int, heads: Heads, tp: int, prefix_len: int = 0) -> int:
    return lib.tps_decode_workspace_bytes(nseq, _heads_ref(heads), tp, prefix_len)


def decode_workspace(nseq: int, heads: Heads, tp: int, prefix_len: int = 0, device=None) -> torch.Tensor:
    """Zero-filled workspace of the decode calls (tps_decode_workspace_bytes bytes)."""
    dev = torch.device("cuda" if device is None else device)
    with torch.cuda.device(dev):
        nbytes = tps_decode_workspace_bytes(nseq, heads, tp, prefix_len)
    if nbytes == 0:
        raise TpsError(TPS_ERR_ARG, "tps_decode_workspace_bytes")
    return torch.zeros(nbytes, dtype=torch.uint8, device=dev)


def sharded_window_decode(qkv: torch.Tensor, heads: Heads, tp: int, pos: torch.Tensor, window: int,
                          k_cache: torch.Tensor, v_cache: torch.Tensor, ws: torch.Tensor, nsink: int = 0, out=None,
                          stream=None):
    """One new token per row of qkv: appends it at position pos[b] (int32 [nseq]; negative:
    an unused row, output zero) and returns its attention [nseq, hq*d] bf16 over the last
    `window` positions and the first `nsink`."""
    cols, nkv, ocols, hd = _geometry(heads, tp)
    nseq = _need(qkv, "qkv").shape[0]
    pq = _arg(qkv, "qkv", torch.bfloat16, (nseq, cols), None)
    dev = qkv.get_device()
    pk, pv, cap = _cache_args(k_cache, v_cache, nseq, nkv, heads.head_dim, dev)
    pp = _arg(_need(pos, "pos"), "pos", torch.int32, (nseq,), dev)
    pw = _arg(_need(ws, "ws"), "ws", None, None, dev)
    po = _arg(out, "out", torch.bfloat16, (nseq, ocols), dev)
    if not _here(dev, stream):
        with _there(dev, stream):
            return sharded_window_decode(qkv, heads, tp, pos, window, k_cache, v_cache, ws, nsink, out)
    if out is None:
        out = torch.empty(nseq, ocols, dtype=torch.bfloat16, device=qkv.device)
        po = out.data_ptr()
    _check(lib.sharded_window_decode(pq, nseq, ctypes.byref(hd), tp, pp, window, nsink, pk, pv, cap, po, pw,
                                     ws.nbytes, _raw_stream(dev)), "sharded_window_decode")
    return out


def sharded_prefix_decode(qkv: torch.Tensor, heads: Heads, tp: int, prefix_k, prefix_v, pos: torch.Tensor,
                          k_cache: torch.Tensor, v_cache: torch.Tensor, ws: torch.Tensor, out=None, stream=None):
    """One new token per row of qkv, behind a prefix [tp*kvs, prefix_len, d] that all rows
    share (None: no prefix): appends it at position pos[b] of its own linear cache (a row
    with pos[b] outside [0, cap) is unused, output zero) and returns its attention
    [nseq, hq*d] bf16 over the prefix and positions 0..pos[b]."""
    cols, nkv, ocols, hd = _geometry(heads, tp)
    nseq = _need(qkv, "qkv").shape[0]
    pq = _arg(qkv, "qkv", torch.bfloat16, (nseq, cols), None)
    dev = qkv.get_device()
    pk, pv, cap = _cache_args(k_cache, v_cache, nseq, nkv, heads.head_dim, dev)
    P, fk, fv = 0, None, None
    if prefix_k is not None or prefix_v is not None:
        fk = _arg(_need(prefix_k, "prefix_k"), "prefix_k", torch.bfloat16, None, dev)
        if prefix_k.dim() != 3 or prefix_k.shape[0] != nkv or prefix_k.shape[2] != heads.head_dim:
            raise ValueError(f"prefix_k must have shape ({nkv}, prefix_len, {heads.head_dim}), got {tuple(prefix_k.shape)}")
        P = prefix_k.shape[1]
        fv = _arg(_need(prefix_v, "prefix_v"), "prefix_v", torch.bfloat16, (nkv, P, heads.head_dim), dev)
    pp = _arg(_need(pos, "pos"), "pos", torch.int32, (nseq,), dev)
    pw = _arg(_need(ws, "ws"), "ws", None, None, dev)
    po = _arg(out, "out", torch.bfloat16, (nseq, ocols), dev)
    if not _here(dev, stream):
        with _there(dev, stream):
            return sharded_prefix_decode(qkv, heads, tp, prefix_k, prefix_v, pos, k_cache, v_cache, ws, out)
    if out is None:
        out = torch.empty(nseq, ocols, dtype=torch.bfloat16, device=qkv.device)
        po = out.data_ptr()
    _check(lib.sharded_prefix_decode(pq, nseq, ctypes.byref(hd), tp, fk, fv, P, pp, pk, pv, cap, po, pw,
                                     ws.nbytes, _raw_stream(dev)), "sharded_prefix_decode")
    return out


def _sample_args(m, dev, u, temperature, top_k, top_p, min_p, out_idx, out_logp):
    f32, i32 = torch.float32, torch.int32
    return [_arg(_need(u, "u"), "u", f32, (m,), dev), _arg(temperature, "temperature", f32, (m,), dev),
            _arg(top_k, "top_k", i32, (m,), dev), _arg(top_p, "top_p", f32, (m,), dev),
            _arg(min_p, "min_p", f32, (m,), dev), _arg(out_idx, "out_idx", i32, (m,), dev),
            _arg(out_logp, "out_logp", f32, (m,), dev)]


def _sample_outputs(m, device, par, out_idx, out_logp):
    if out_idx is None:
        out_idx = torch.empty(m, dtype=torch.int32, device=device)
        par[5] = out_idx.data_ptr()
    if out_logp is None:
        out_logp = torch.empty(m, dtype=torch.float32, device=device)
        par[6] = out_logp.data_ptr()
    return out_idx, out_logp


def logits_sample(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None, min_p=None,
                  out_idx=None, out_logp=None, stream=None):
    """Draws one token per row of logits [m, V] (bf16 or fp32) with the uniform numbers u
    [m]: temperature, top-k, top-p, min-p (per-row tensors or None), then the inverse of
    the kept weights' running sum in vocabulary order. Returns (indices int32 [m], log of
    the drawn tokens' shares fp32 [m])."""
    pl = _arg(_need(logits, "logits"), "logits", None, None, None)
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    m, V = logits.shape
    dev = logits.get_device()
    par = _sample_args(m, dev, u, temperature, top_k, top_p, min_p, out_idx, out_logp)
    if not _here(dev, stream):
        with _there(dev, stream):
            return logits_sample(logits, u, temperature, top_k, top_p, min_p, out_idx, out_logp)
    out_idx, out_logp = _sample_outputs(m, logits.device, par, out_idx, out_logp)
    _check(lib.logits_sample(pl, _ydtype(logits.dtype), m, V, *par, _raw_stream(dev)), "logits_sample")
    return out_idx, out_logp


def vocab_parallel_sample(X: torch.Tensor, H: int, V: int, tp: int, packed_w: torch.Tensor, u: torch.Tensor,
                          ws: torch.Tensor | None = None, temperature=None, top_k=None, top_p=None, min_p=None,
                          out_idx=None, out_logp=None, stream=None):
    """logits_sample over a vocab-parallel lm_head (COLUMN pack of W[H, V]); ws is a
    workspace(FN_SAMPLE, m, V, H, tp), which receives the fp32 logits."""
    m = _need(X, "X").shape[0]
    px = _arg(X, "X", torch.bfloat16, (m, H), None)
    dev = X.get_device()
    pw = _arg(_need(packed_w, "packed_w"), "packed_w", torch.bfloat16, None, dev)
    if packed_w.nbytes < tp_packed_bytes(KIND_COLUMN, H, V, tp):
        raise ValueError("packed_w is smaller than the COLUMN pack of W[H, V]")
    _arg(ws, "ws", None, None, dev)
    par = _sample_args(m, dev, u, temperature, top_k, top_p, min_p, out_idx, out_logp)
    if not _here(dev, stream):
        with _there(dev, stream):
            return vocab_parallel_sample(X, H, V, tp, packed_w, u, ws, temperature, top_k, top_p, min_p, out_idx,
                                         out_logp)
    if ws is None:
        ws = workspace(FN_SAMPLE, m, V, H, tp, device=X.device)
    out_idx, out_logp = _sample_outputs(m, X.device, par, out_idx, out_logp)
    _check(lib.vocab_parallel_sample(px, m, H, pw, V, tp, *par, ws.data_ptr(), ws.nbytes, _raw_stream(dev)),
           "vocab_parallel_sample")
    return out_idx, out_logp
