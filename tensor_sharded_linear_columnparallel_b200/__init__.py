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

import ctypes
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
    return torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=device or "cuda")


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
class _On:
    """The call's device and stream: checks that its tensors share one device, makes that
    device current for the call, and allocates outputs on the stream that writes them."""

    def __init__(self, stream, *tensors):
        self.dev = tensors[0].device
        for t in tensors[1:]:
            if t is not None and t.device != self.dev:
                raise ValueError(f"tensors on {self.dev} and {t.device}")
        self.stream = stream

    def __enter__(self):
        self.guard = torch.cuda.device(self.dev)
        self.guard.__enter__()
        if self.stream is None:
            self.stream = torch.cuda.current_stream()
        elif self.stream.device != self.dev:
            self.guard.__exit__(None, None, None)
            raise ValueError(f"stream of {self.stream.device}, tensors on {self.dev}")
        self.on = torch.cuda.stream(self.stream)
        self.on.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        self.on.__exit__(*exc)
        self.guard.__exit__(*exc)


def _qkv_cols(heads: Heads, tp: int) -> tuple[int, int]:
    """Columns of a QKV output row and KV head slots tp*kvs (every shard's KV heads)."""
    _, qc, _, kc = tp_head_map(heads.hq, heads.hkv, tp)
    return tp * (qc[0] + 2 * kc[0]) * heads.head_dim, tp * kc[0]


def _shape(t: torch.Tensor, shape: tuple, what: str) -> None:
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _caches(k_cache, v_cache, nseq: int, nkv: int, d: int) -> int:
    _dev(k_cache, "k_cache", torch.bfloat16)
    _dev(v_cache, "v_cache", torch.bfloat16)
    if k_cache.dim() != 4:
        raise ValueError("k_cache must be [nseq, tp*kvs, cap, d]")
    cap = k_cache.shape[2]
    _shape(k_cache, (nseq, nkv, cap, d), "k_cache")
    _shape(v_cache, (nseq, nkv, cap, d), "v_cache")
    return cap


def _vec(t, n: int, dtype, what: str):
    if t is not None:
        _dev(t, what, dtype)
        _shape(t, (n,), what)
    return t


def sharded_window_attention(qkv: torch.Tensor, nseq: int, seqlen: int, heads: Heads, tp: int, window: int,
                             nsink: int = 0, out=None, stream=None):
    """sharded_gqa_attention (causal) where query t sees the last `window` tokens, itself
    included, and the first `nsink`. Returns attn_out [nseq*seqlen, hq*d] bf16."""
    _dev(qkv, "qkv", torch.bfloat16)
    m = nseq * seqlen
    _shape(qkv, (m, _qkv_cols(heads, tp)[0]), "qkv")
    if out is not None:
        _dev(out, "out", torch.bfloat16)
        _shape(out, (m, heads.hq * heads.head_dim), "out")
    with _On(stream, qkv, out) as st:
        if out is None:
            out = torch.empty(m, heads.hq * heads.head_dim, dtype=torch.bfloat16, device=qkv.device)
        _check(lib.sharded_window_attention(_ptr(qkv), nseq, seqlen, _heads_ref(heads), tp, window, nsink, _ptr(out),
                                            st), "sharded_window_attention")
    return out


def sharded_kv_append(qkv: torch.Tensor, nseq: int, seqlen: int, heads: Heads, tp: int, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, pos=None, count=None, nsink: int = 0, stream=None) -> None:
    """Writes the K and V of a QKV output to the caches [nseq, tp*kvs, cap, d]: token i of
    sequence b, i < count[b], at position pos[b] + i (int32 [nseq]; None: 0 and seqlen)."""
    _dev(qkv, "qkv", torch.bfloat16)
    cols, nkv = _qkv_cols(heads, tp)
    _shape(qkv, (nseq * seqlen, cols), "qkv")
    cap = _caches(k_cache, v_cache, nseq, nkv, heads.head_dim)
    _vec(pos, nseq, torch.int32, "pos")
    _vec(count, nseq, torch.int32, "count")
    with _On(stream, qkv, k_cache, v_cache, pos, count) as st:
        _check(lib.sharded_kv_append(_ptr(qkv), nseq, seqlen, _heads_ref(heads), tp, _ptr(pos), _ptr(count), nsink,
                                     _ptr(k_cache), _ptr(v_cache), cap, st), "sharded_kv_append")


def tps_decode_workspace_bytes(nseq: int, heads: Heads, tp: int, prefix_len: int = 0) -> int:
    return lib.tps_decode_workspace_bytes(nseq, _heads_ref(heads), tp, prefix_len)


def decode_workspace(nseq: int, heads: Heads, tp: int, prefix_len: int = 0, device=None) -> torch.Tensor:
    """Zero-filled workspace of the decode calls (tps_decode_workspace_bytes bytes)."""
    dev = torch.device(device or "cuda")
    with torch.cuda.device(dev):
        nbytes = tps_decode_workspace_bytes(nseq, heads, tp, prefix_len)
    return torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=dev)


def sharded_window_decode(qkv: torch.Tensor, heads: Heads, tp: int, pos: torch.Tensor, window: int,
                          k_cache: torch.Tensor, v_cache: torch.Tensor, ws: torch.Tensor, nsink: int = 0, out=None,
                          stream=None):
    """One new token per row of qkv: appends it at position pos[b] (int32 [nseq]; negative:
    an unused row, output zero) and returns its attention [nseq, hq*d] bf16 over the last
    `window` positions and the first `nsink`."""
    _dev(qkv, "qkv", torch.bfloat16)
    nseq = qkv.shape[0]
    cols, nkv = _qkv_cols(heads, tp)
    _shape(qkv, (nseq, cols), "qkv")
    cap = _caches(k_cache, v_cache, nseq, nkv, heads.head_dim)
    _vec(_dev(pos, "pos", torch.int32), nseq, torch.int32, "pos")
    _dev(ws, "ws")
    if out is not None:
        _dev(out, "out", torch.bfloat16)
        _shape(out, (nseq, heads.hq * heads.head_dim), "out")
    with _On(stream, qkv, k_cache, v_cache, pos, ws, out) as st:
        if out is None:
            out = torch.empty(nseq, heads.hq * heads.head_dim, dtype=torch.bfloat16, device=qkv.device)
        _check(lib.sharded_window_decode(_ptr(qkv), nseq, _heads_ref(heads), tp, _ptr(pos), window, nsink,
                                         _ptr(k_cache), _ptr(v_cache), cap, _ptr(out), _ptr(ws),
                                         ws.numel() * ws.element_size(), st), "sharded_window_decode")
    return out


def sharded_prefix_decode(qkv: torch.Tensor, heads: Heads, tp: int, prefix_k, prefix_v, pos: torch.Tensor,
                          k_cache: torch.Tensor, v_cache: torch.Tensor, ws: torch.Tensor, out=None, stream=None):
    """One new token per row of qkv, behind a prefix [tp*kvs, prefix_len, d] that all rows
    share (None: no prefix): appends it at position pos[b] of its own linear cache (a row
    with pos[b] outside [0, cap) is unused, output zero) and returns its attention
    [nseq, hq*d] bf16 over the prefix and positions 0..pos[b]."""
    _dev(qkv, "qkv", torch.bfloat16)
    nseq = qkv.shape[0]
    cols, nkv = _qkv_cols(heads, tp)
    _shape(qkv, (nseq, cols), "qkv")
    cap = _caches(k_cache, v_cache, nseq, nkv, heads.head_dim)
    P = 0
    if prefix_k is not None or prefix_v is not None:
        _dev(prefix_k, "prefix_k", torch.bfloat16)
        _dev(prefix_v, "prefix_v", torch.bfloat16)
        P = prefix_k.shape[1] if prefix_k.dim() == 3 else -1
        _shape(prefix_k, (nkv, P, heads.head_dim), "prefix_k")
        _shape(prefix_v, (nkv, P, heads.head_dim), "prefix_v")
    _vec(_dev(pos, "pos", torch.int32), nseq, torch.int32, "pos")
    _dev(ws, "ws")
    if out is not None:
        _dev(out, "out", torch.bfloat16)
        _shape(out, (nseq, heads.hq * heads.head_dim), "out")
    with _On(stream, qkv, k_cache, v_cache, pos, ws, out, prefix_k, prefix_v) as st:
        if out is None:
            out = torch.empty(nseq, heads.hq * heads.head_dim, dtype=torch.bfloat16, device=qkv.device)
        _check(lib.sharded_prefix_decode(_ptr(qkv), nseq, _heads_ref(heads), tp, _ptr(prefix_k), _ptr(prefix_v), P,
                                         _ptr(pos), _ptr(k_cache), _ptr(v_cache), cap, _ptr(out), _ptr(ws),
                                         ws.numel() * ws.element_size(), st), "sharded_prefix_decode")
    return out


def _sample_params(m, u, temperature, top_k, top_p, min_p, out_idx, out_logp):
    _vec(_dev(u, "u", torch.float32), m, torch.float32, "u")
    _vec(temperature, m, torch.float32, "temperature")
    _vec(top_k, m, torch.int32, "top_k")
    _vec(top_p, m, torch.float32, "top_p")
    _vec(min_p, m, torch.float32, "min_p")
    _vec(out_idx, m, torch.int32, "out_idx")
    _vec(out_logp, m, torch.float32, "out_logp")
    return u, temperature, top_k, top_p, min_p, out_idx, out_logp


def logits_sample(logits: torch.Tensor, u: torch.Tensor, temperature=None, top_k=None, top_p=None, min_p=None,
                  out_idx=None, out_logp=None, stream=None):
    """Draws one token per row of logits [m, V] (bf16 or fp32) with the uniform numbers u
    [m]: temperature, top-k, top-p, min-p (per-row tensors or None), then the inverse of
    the kept weights' running sum in vocabulary order. Returns (indices int32 [m], log of
    the drawn tokens' shares fp32 [m])."""
    _dev(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D")
    m, V = logits.shape
    par = _sample_params(m, u, temperature, top_k, top_p, min_p, out_idx, out_logp)
    with _On(stream, logits, *par) as st:
        if out_idx is None:
            out_idx = torch.empty(m, dtype=torch.int32, device=logits.device)
        if out_logp is None:
            out_logp = torch.empty(m, dtype=torch.float32, device=logits.device)
        _check(lib.logits_sample(_ptr(logits), _ydtype(logits.dtype), m, V, _ptr(u), _ptr(temperature), _ptr(top_k),
                                 _ptr(top_p), _ptr(min_p), _ptr(out_idx), _ptr(out_logp), st), "logits_sample")
    return out_idx, out_logp


def vocab_parallel_sample(X: torch.Tensor, H: int, V: int, tp: int, packed_w: torch.Tensor, u: torch.Tensor,
                          ws: torch.Tensor | None = None, temperature=None, top_k=None, top_p=None, min_p=None,
                          out_idx=None, out_logp=None, stream=None):
    """logits_sample over a vocab-parallel lm_head (COLUMN pack of W[H, V]); ws is a
    workspace(FN_SAMPLE, m, V, H, tp), which receives the fp32 logits."""
    _dev(X, "X", torch.bfloat16)
    _dev(packed_w, "packed_w", torch.bfloat16)
    m = X.shape[0]
    _shape(X, (m, H), "X")
    if packed_w.numel() * 2 < tp_packed_bytes(KIND_COLUMN, H, V, tp):
        raise ValueError("packed_w is smaller than the COLUMN pack of W[H, V]")
    if ws is not None:
        _dev(ws, "ws")
    par = _sample_params(m, u, temperature, top_k, top_p, min_p, out_idx, out_logp)
    with _On(stream, X, packed_w, ws, *par) as st:
        if ws is None:
            ws = workspace(FN_SAMPLE, m, V, H, tp, device=X.device)
        if out_idx is None:
            out_idx = torch.empty(m, dtype=torch.int32, device=X.device)
        if out_logp is None:
            out_logp = torch.empty(m, dtype=torch.float32, device=X.device)
        _check(lib.vocab_parallel_sample(_ptr(X), m, H, _ptr(packed_w), V, tp, _ptr(u), _ptr(temperature),
                                         _ptr(top_k), _ptr(top_p), _ptr(min_p), _ptr(out_idx), _ptr(out_logp),
                                         _ptr(ws), ws.numel() * ws.element_size(), st), "vocab_parallel_sample")
    return out_idx, out_logp
