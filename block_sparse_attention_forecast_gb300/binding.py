"""ctypes binding of libsparda (include/sparda.h).

Argument marshalling only: every function below takes torch tensors (or plain integers),
passes their device addresses and the current CUDA stream to the C entry point of the same
name, and raises SpardaError on a non-zero status. Every computation happens in the CUDA
kernels of libsparda. There is no fallback: if the library is missing, importing this module
fails with an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import os
import re
from dataclasses import dataclass

import torch

__all__ = [
    "lib", "LIB_PATH", "HEADER_PATH", "SpardaError", "Shape", "LayerKV", "workspace",
    "hot_slot", "fill_hot_from_host",
    "header_functions", "status_string", "num_windows", "c_shape", "c_layer_kv",
    "sparda_abi_version", "sparda_status_string", "sparda_check_shape", "sparda_workspace_bytes",
    "sparda_block_scores_offset", "sparda_device_error", "sparda_get_device_status",
    "sparda_prefetch_default_ctas", "sparda_append_kv", "sparda_compress_keys",
    "sparda_forecast_project", "sparda_forecast_select", "sparda_sparse_decode_attn",
    "sparda_prefetch_blocks", "sparda_multihead_select", "sparda_forecast_select_static", "sparda_attend_and_select",
    "sparda_attend_and_score", "sparda_decode_prologue", "sparda_forecast_score", "sparda_copy",
    "sparda_prefill_forecast_select", "sparda_prefill_multihead_select", "sparda_prefill_attn",
    "sparda_prefetch_blocks_cached", "sparda_sparse_decode_attn_cached", "BlockCache",
    "sparda_prefetch_blocks_copy_engine",
    "LayerKV4", "sparda_kv4_quantize", "sparda_kv4_dequantize", "sparda_kv4_append", "sparda_kv4_decode_attn",
    "sparda_sparse_decode_attn_mass", "sparda_evict_blocks", "sparda_kv4_evict_blocks", "KV4_BLOCK_BYTES",
    "WS_ATTN_MASS", "WS_KV4_ATTN", "WS_KV4_ATTN_MASS",
    "sparda_prompt_attn", "sparda_prompt_append", "sparda_tree_attn", "sparda_tree_commit", "WS_PROMPT", "WS_TREE",
    "TREE_MAX_NODES",
    "OK", "ERR_INVALID_ARG", "ERR_UNSUPPORTED_SHAPE", "ERR_MISALIGNED", "ERR_NOT_MAPPED_HOST",
    "ERR_WORKSPACE_TOO_SMALL", "ERR_CUDA", "ERR_STATIC_SCRATCH_LIMIT", "DEV_WAIT_TIMEOUT", "DEV_BAD_SEQ_LEN", "DEV_BAD_INDEX",
    "WS_SELECT", "WS_ATTN", "WS_MULTIHEAD", "WS_PREFILL", "BLOCK", "WIN_KERNEL", "WIN_STRIDE",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
# SPARDA_LIB may name another build of the same library (the per-CTA timeline variant)
LIB_PATH = os.environ.get("SPARDA_LIB") or os.path.join(_PKG, "_lib", "libsparda.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "sparda.h")

OK = 0
ERR_INVALID_ARG = -1
ERR_UNSUPPORTED_SHAPE = -2
ERR_MISALIGNED = -3
ERR_NOT_MAPPED_HOST = -4
ERR_WORKSPACE_TOO_SMALL = -5
ERR_CUDA = -6
ERR_STATIC_SCRATCH_LIMIT = -7

DEV_WAIT_TIMEOUT = 1
DEV_BAD_SEQ_LEN = 2
DEV_BAD_INDEX = 4

WS_SELECT = 1
WS_ATTN = 2
WS_MULTIHEAD = 3
WS_PREFILL = 4
WS_ATTN_MASS = 5
WS_KV4_ATTN = 6
WS_KV4_ATTN_MASS = 7
WS_PROMPT = 8
WS_TREE = 9

TREE_MAX_NODES = 128        # nodes of a tree of drafted tokens

KV4_BLOCK_BYTES = 10240     # one 64-token block of the 4-bit cache, keys and values

BLOCK = 64
WIN_KERNEL = 32
WIN_STRIDE = 16


class SpardaError(RuntimeError):
    def __init__(self, name, status):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (name, status_string(status), status))


class c_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "n_groups", "heads_per_group", "head_dim", "block", "win_kernel", "win_stride",
        "topk", "max_ctx", "max_batch")]


class c_layer_kv(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ck", ctypes.c_void_p),
                ("hot_k", ctypes.c_void_p), ("hot_v", ctypes.c_void_p),
                ("on_host", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class c_layer_kv4(ctypes.Structure):
    _fields_ = [("kv", ctypes.c_void_p), ("ck", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libsparda.so is not built (%s). Build it with "
            "`python -m block_sparse_attention_forecast_gb300.build` (nvcc, CUDA 13)." % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int64
    SH, LY = ctypes.POINTER(c_shape), ctypes.POINTER(c_layer_kv)
    L4 = ctypes.POINTER(c_layer_kv4)
    sig = {
        "sparda_abi_version": (I32, []),
        "sparda_status_string": (ctypes.c_char_p, [I32]),
        "sparda_check_shape": (I32, [SH]),
        "sparda_workspace_bytes": (SZ, [SH, I32, I32]),
        "sparda_block_scores_offset": (SZ, [SH]),
        "sparda_device_error": (I32, [ctypes.POINTER(I32), I32]),
        "sparda_get_device_status": (I32, [P, I32, P]),
        "sparda_prefetch_default_ctas": (I32, [I32]),
        "sparda_append_kv": (I32, [SH, LY, P, P, P, I32, P]),
        "sparda_compress_keys": (I32, [SH, LY, P, I32, P]),
        "sparda_forecast_project": (I32, [P, P, I32, I32, I32, P, P]),
        "sparda_forecast_select": (I32, [SH, P, P, P, I32, P, P, P, SZ, P]),
        "sparda_sparse_decode_attn": (I32, [SH, LY, P, P, P, P, P, P, I32, P, P, SZ, P]),
        "sparda_prefetch_blocks": (I32, [SH, LY, P, P, P, I32, P, P, I32, P]),
        "sparda_multihead_select": (I32, [SH, P, P, P, I32, P, P, P, SZ, P]),
        "sparda_forecast_select_static": (I32, [SH, P, P, P, I32, P, P, P]),
        "sparda_attend_and_select": (I32, [SH, LY, P, P, P, P, P, P, P, SZ, P, P, P, P, P, SZ, P, I32, P]),
        "sparda_attend_and_score": (I32, [SH, LY, P, P, P, P, P, P, P, SZ, P, P, P, SZ, P, SZ, P, I32, P]),
        "sparda_decode_prologue": (I32, [SH, LY, P, P, P, SZ, P, P, P, P, I32, P, P, I32, P]),
        "sparda_copy": (I32, [P, P, SZ, P]),
        "sparda_forecast_score": (I32, [SH, P, P, P, I32, P, SZ, P]),
        "sparda_prefill_forecast_select": (I32, [SH, P, P, P, I32, P, P, P, SZ, P]),
        "sparda_prefill_multihead_select": (I32, [SH, P, P, P, I32, P, P, P, SZ, P]),
        "sparda_prefill_attn": (I32, [SH, LY, P, P, P, P, I32, P, P]),
        "sparda_prefetch_blocks_cached": (I32, [SH, LY, P, P, P, I32, P, P, P, I32, P, P, P, I32, P]),
        "sparda_prefetch_blocks_copy_engine": (I32, [SH, LY, P, P, P, I32, P, P, P, P]),
        "sparda_sparse_decode_attn_cached": (I32, [SH, LY, P, P, I32, P, P, P, P, P, I32, P, P, SZ, P]),
        "sparda_kv4_quantize": (I32, [SH, L4, P, P, P, I32, P]),
        "sparda_kv4_dequantize": (I32, [SH, L4, P, P, P, I32, P, P, P]),
        "sparda_kv4_append": (I32, [SH, L4, P, P, P, I32, P]),
        "sparda_kv4_decode_attn": (I32, [SH, L4, P, P, P, P, I32, P, P, P, SZ, P]),
        "sparda_sparse_decode_attn_mass": (I32, [SH, LY, P, P, P, P, I32, P, P, P, SZ, P]),
        "sparda_evict_blocks": (I32, [SH, LY, P, P, SH, LY, P, P, I32, I32, I32, P, P]),
        "sparda_kv4_evict_blocks": (I32, [SH, L4, P, P, SH, L4, P, P, I32, I32, I32, P, P]),
        "sparda_prompt_attn": (I32, [SH, LY, P, P, I64, P, P, I64, P, I32, I32, P, P, SZ, P]),
        "sparda_prompt_append": (I32, [SH, LY, P, P, I64, P, I32, P, I32, P, P]),
        "sparda_tree_attn": (I32, [SH, LY, P, I64, P, P, I64, P, P, I32, P, P, P, I32, P, P, SZ, P]),
        "sparda_tree_commit": (I32, [SH, LY, P, P, I64, I32, P, P, P, I32, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def header_functions():
    """Names of the functions include/sparda.h declares."""
    with open(HEADER_PATH) as fh:
        text = fh.read()
    return sorted(set(re.findall(r"^\s*(?:int32_t|size_t|const char\*)\s+(sparda_\w+)\s*\(", text, re.M)))


def status_string(status):
    return lib.sparda_status_string(int(status)).decode()


sparda_status_string = status_string


def _check(name, status):
    if status != OK:
        raise SpardaError(name, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def num_windows(n_tokens):
    return 0 if n_tokens < WIN_KERNEL else (n_tokens - WIN_KERNEL) // WIN_STRIDE + 1


@dataclass
class Shape:
    """Decode-step geometry (sparda_shape)."""
    __slots__ = ("_kept", "__dict__", "__weakref__")     # [sizes(), ref()], no field: not among vars(shape)
    n_groups: int = 2
    heads_per_group: int = 16
    head_dim: int = 128
    topk: int = 32
    max_ctx: int = 32768
    max_batch: int = 1
    block: int = BLOCK
    win_kernel: int = WIN_KERNEL
    win_stride: int = WIN_STRIDE

    def c(self):
        return c_shape(self.n_groups, self.heads_per_group, self.head_dim, self.block,
                       self.win_kernel, self.win_stride, self.topk, self.max_ctx, self.max_batch)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_kept", [None, None])

    def __getstate__(self):
        return self.__dict__

    def __setstate__(self, state):
        for name, value in state.items():
            setattr(self, name, value)

    def sizes(self):
        """(elements of a resident LayerKV's k or v, bytes of a LayerKV4's kv, elements of their ck), kept until
        a field changes."""
        r = self._kept[0]
        if r is None:
            rows = self.max_batch * self.n_groups
            r = self._kept[0] = (rows * self.max_ctx * self.head_dim, rows * (self.max_ctx // BLOCK) * KV4_BLOCK_BYTES,
                                 rows * num_windows(self.max_ctx) * self.head_dim)
        return r

    def ref(self):
        """A pointer to c(), kept until a field changes."""
        r = self._kept[1]
        if r is None:
            r = self._kept[1] = ctypes.byref(self.c())
        return r

    @property
    def w_cap(self):
        return num_windows(self.max_ctx)

    @property
    def kslots(self):
        return self.topk + 2


@dataclass
class LayerKV:
    """One layer's caches (sparda_layer_kv), as torch tensors.

    k, v: bf16 [max_batch, G, max_ctx, d] on the device, or pinned host tensors (on_host).
    ck: bf16 [max_batch, G, w_cap, d] on the device. hot_k, hot_v: bf16
    [max_batch, G, 3, 64, d] on the device for offloaded layers.
    """
    k: torch.Tensor
    v: torch.Tensor
    ck: torch.Tensor
    hot_k: torch.Tensor = None
    hot_v: torch.Tensor = None
    on_host: bool = False

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__.pop("_args", None)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_args"}

    def c(self):
        return c_layer_kv(self.k.data_ptr(), self.v.data_ptr(), self.ck.data_ptr(),
                          self.hot_k.data_ptr() if self.hot_k is not None else None,
                          self.hot_v.data_ptr() if self.hot_v is not None else None,
                          1 if self.on_host else 0, 0)

    @staticmethod
    def empty(shape, device="cuda", on_host=False):
        G, d = shape.n_groups, shape.head_dim
        kv = (shape.max_batch, G, shape.max_ctx, d)
        if on_host:
            k = torch.empty(kv, dtype=torch.bfloat16, pin_memory=True)
            v = torch.empty(kv, dtype=torch.bfloat16, pin_memory=True)
            hot = (shape.max_batch, G, 3, shape.block, d)
            hk = torch.zeros(hot, dtype=torch.bfloat16, device=device)
            hv = torch.zeros(hot, dtype=torch.bfloat16, device=device)
        else:
            k = torch.empty(kv, dtype=torch.bfloat16, device=device)
            v = torch.empty(kv, dtype=torch.bfloat16, device=device)
            hk = hv = None
        ck = torch.zeros((shape.max_batch, G, shape.w_cap, d), dtype=torch.bfloat16, device=device)
        return LayerKV(k, v, ck, hk, hv, on_host)


@dataclass
class LayerKV4:
    """One layer's cache in 4 bits (sparda_layer_kv4), as torch tensors on the device.

    kv: uint8 [max_batch, G, max_ctx / 64, KV4_BLOCK_BYTES]. ck: bf16 [max_batch, G, w_cap, d].
    """
    kv: torch.Tensor
    ck: torch.Tensor

    on_host = False                # a 4-bit cache is resident

    def c(self):
        return c_layer_kv4(self.kv.data_ptr(), self.ck.data_ptr())

    def __setattr__(self, name, value):
        self.__dict__[name] = value
        self.__dict__.pop("_args", None)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_args"}

    @staticmethod
    def empty(shape, device="cuda"):
        B, G = shape.max_batch, shape.n_groups
        kv = torch.empty((B, G, shape.max_ctx // shape.block, KV4_BLOCK_BYTES), dtype=torch.uint8, device=device)
        ck = torch.zeros((B, G, shape.w_cap, shape.head_dim), dtype=torch.bfloat16, device=device)
        return LayerKV4(kv, ck)


def hot_slot(j):
    """Hot-ring slot of block j of an offloaded layer (include/sparda.h, sparda_layer_kv)."""
    return 0 if j == 0 else 1 + (j & 1)


def fill_hot_from_host(layer, n_cached):
    """Set-up after a prefill of an offloaded layer: copy block 0 and the two newest blocks of
    every sequence from the host cache into the hot ring. n_cached[b] = tokens cached so far.
    Plain device copies; not part of the decode step."""
    for b, n in enumerate(n_cached):
        if n < 1:
            continue
        tb = (n - 1) // BLOCK
        for j in sorted({0, tb, max(tb - 1, 0)}):
            rows = slice(j * BLOCK, (j + 1) * BLOCK)
            layer.hot_k[b, :, hot_slot(j)].copy_(layer.k[b, :, rows], non_blocking=False)
            layer.hot_v[b, :, hot_slot(j)].copy_(layer.v[b, :, rows], non_blocking=False)


def workspace(shape, batch, kind, device="cuda"):
    """A zero-filled workspace of the size sparda_workspace_bytes gives."""
    n = sparda_workspace_bytes(shape, batch, kind)
    if n == 0:
        raise SpardaError("sparda_workspace_bytes", ERR_UNSUPPORTED_SHAPE)
    return torch.zeros(n, dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ entry points
def sparda_abi_version():
    return lib.sparda_abi_version()


def sparda_check_shape(shape):
    return lib.sparda_check_shape(ctypes.byref(shape.c()))


def sparda_workspace_bytes(shape, batch, kind):
    return lib.sparda_workspace_bytes(ctypes.byref(shape.c()), int(batch), int(kind))


def sparda_block_scores_offset(shape):
    return lib.sparda_block_scores_offset(ctypes.byref(shape.c()))


def sparda_device_error(clear=True):
    flags = ctypes.c_int32(0)
    _check("sparda_device_error", lib.sparda_device_error(ctypes.byref(flags), 1 if clear else 0))
    return flags.value


def sparda_get_device_status(dev_flag, clear=True, stream=None):
    """Enqueue a stream-ordered copy of the device error word into dev_flag (an int32 tensor
    of one element on the device, or pinned on the host), resetting the word if clear."""
    _check("sparda_get_device_status", lib.sparda_get_device_status(_ptr(dev_flag), 1 if clear else 0,
                                                                      _stream(stream)))


def sparda_prefetch_default_ctas(batch):
    return lib.sparda_prefetch_default_ctas(int(batch))


def sparda_append_kv(shape, layer, k_new, v_new, seq_len, batch, stream=None):
    _check("sparda_append_kv", lib.sparda_append_kv(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(k_new), _ptr(v_new),
        _ptr(seq_len), int(batch), _stream(stream)))


def sparda_compress_keys(shape, layer, seq_len, batch, stream=None):
    _check("sparda_compress_keys", lib.sparda_compress_keys(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(seq_len), int(batch),
        _stream(stream)))


def sparda_forecast_project(W, h, f, stream=None):
    rows, hidden = W.shape
    _check("sparda_forecast_project", lib.sparda_forecast_project(
        _ptr(W), _ptr(h), int(rows), int(hidden), int(h.shape[0]), _ptr(f), _stream(stream)))


def sparda_forecast_select(shape, ck, forecast, seq_len, batch, idx, cnt, ws, stream=None):
    _check("sparda_forecast_select", lib.sparda_forecast_select(
        ctypes.byref(shape.c()), _ptr(ck), _ptr(forecast), _ptr(seq_len), int(batch), _ptr(idx),
        _ptr(cnt), _ptr(ws), ws.numel(), _stream(stream)))


def sparda_sparse_decode_attn(shape, layer, q, idx, cnt, seq_len, batch, out, ws,
                              staging_k=None, staging_v=None, stream=None):
    _check("sparda_sparse_decode_attn", lib.sparda_sparse_decode_attn(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(staging_k), _ptr(staging_v),
        _ptr(q), _ptr(idx), _ptr(cnt), _ptr(seq_len), int(batch), _ptr(out), _ptr(ws),
        ws.numel(), _stream(stream)))


def sparda_attend_and_select(shape, layer, q, idx, cnt, out, ws_attn, ck_next, forecast_next, idx_next,
                             cnt_next, ws_sel, seq_len, batch, staging_k=None, staging_v=None, stream=None):
    _check("sparda_attend_and_select", lib.sparda_attend_and_select(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(staging_k), _ptr(staging_v), _ptr(q), _ptr(idx),
        _ptr(cnt), _ptr(out), _ptr(ws_attn), ws_attn.numel(), _ptr(ck_next), _ptr(forecast_next), _ptr(idx_next),
        _ptr(cnt_next), _ptr(ws_sel), ws_sel.numel(), _ptr(seq_len), int(batch), _stream(stream)))


def sparda_attend_and_score(shape, layer, q, idx, cnt, out, ws_attn, ck_next, forecast_next, ws_scores,
                            seq_len, batch, staging_k=None, staging_v=None, l2_next=None, stream=None):
    """l2_next: an optional tensor the next launches read (pulled into L2 at the end)."""
    _check("sparda_attend_and_score", lib.sparda_attend_and_score(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(staging_k), _ptr(staging_v), _ptr(q), _ptr(idx),
        _ptr(cnt), _ptr(out), _ptr(ws_attn), ws_attn.numel(), _ptr(ck_next), _ptr(forecast_next), _ptr(ws_scores),
        ws_scores.numel(), _ptr(l2_next), l2_next.numel() * l2_next.element_size() if l2_next is not None else 0,
        _ptr(seq_len), int(batch), _stream(stream)))


def sparda_decode_prologue(shape, layer, k_new, v_new, seq_len, batch, ws_scores=None, idx=None, cnt=None,
                           W_next=None, h=None, forecast_next=None, stream=None):
    """Layer L's top-k (from ws_scores, if given), append, and forecast for layer L+1 (if
    W_next is given) in one launch."""
    hidden = int(W_next.shape[1]) if W_next is not None else 0
    _check("sparda_decode_prologue", lib.sparda_decode_prologue(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(k_new), _ptr(v_new), _ptr(ws_scores),
        ws_scores.numel() if ws_scores is not None else 0, _ptr(idx), _ptr(cnt), _ptr(W_next), _ptr(h), hidden,
        _ptr(forecast_next), _ptr(seq_len), int(batch), _stream(stream)))


def sparda_prefetch_blocks(shape, layer, idx, cnt, seq_len, batch, staging_k, staging_v,
                           n_ctas=0, stream=None):
    _check("sparda_prefetch_blocks", lib.sparda_prefetch_blocks(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(idx), _ptr(cnt), _ptr(seq_len),
        int(batch), _ptr(staging_k), _ptr(staging_v), int(n_ctas), _stream(stream)))


def sparda_forecast_score(shape, ck, forecast, seq_len, batch, ws, stream=None):
    """Block scores of the Forecast selector without the top-k, into the select workspace ws
    (for sparda_decode_prologue's ws_scores)."""
    _check("sparda_forecast_score", lib.sparda_forecast_score(
        ctypes.byref(shape.c()), _ptr(ck), _ptr(forecast), _ptr(seq_len), int(batch), _ptr(ws), ws.numel(),
        _stream(stream)))


def sparda_copy(dst, src, stream=None):
    """Device-side copy of src into dst (same byte size, each contiguous): device tensors or
    pinned host tensors (see include/sparda.h)."""
    nbytes = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != nbytes or not dst.is_contiguous() or not src.is_contiguous():
        raise ValueError("sparda_copy needs two contiguous tensors of the same byte size")
    _check("sparda_copy", lib.sparda_copy(_ptr(dst), _ptr(src), nbytes, _stream(stream)))


def sparda_multihead_select(shape, ck, q, seq_len, batch, idx, cnt, ws, stream=None):
    _check("sparda_multihead_select", lib.sparda_multihead_select(
        ctypes.byref(shape.c()), _ptr(ck), _ptr(q), _ptr(seq_len), int(batch), _ptr(idx),
        _ptr(cnt), _ptr(ws), ws.numel(), _stream(stream)))


def sparda_forecast_select_static(shape, ck, forecast, seq_len, batch, idx, cnt, stream=None):
    """sparda_forecast_select without a workspace: for callers that may not allocate device
    memory. Its scratch is a fixed array inside the library (see include/sparda.h)."""
    _check("sparda_forecast_select_static", lib.sparda_forecast_select_static(
        ctypes.byref(shape.c()), _ptr(ck), _ptr(forecast), _ptr(seq_len), int(batch), _ptr(idx),
        _ptr(cnt), _stream(stream)))


# ------------------------------------------------------------------ chunked prefill
def sparda_prefill_forecast_select(shape, ck, forecast, seq_len, batch, idx, cnt, ws, stream=None):
    """Per-chunk selections of a prompt by the Forecast selector. forecast: bf16
    [max_batch, max_ctx, G, d]; idx: int32 [B, G, max_ctx/64, topk+2]; cnt: int32
    [B, G, max_ctx/64]; ws: a WS_PREFILL workspace."""
    _check("sparda_prefill_forecast_select", lib.sparda_prefill_forecast_select(
        ctypes.byref(shape.c()), _ptr(ck), _ptr(forecast), _ptr(seq_len), int(batch), _ptr(idx), _ptr(cnt),
        _ptr(ws), ws.numel(), _stream(stream)))


def sparda_prefill_multihead_select(shape, ck, q, seq_len, batch, idx, cnt, ws, stream=None):
    """Per-chunk selections of a prompt by the baseline multi-head selector. q: bf16
    [max_batch, max_ctx, G*H, d]; outputs as sparda_prefill_forecast_select."""
    _check("sparda_prefill_multihead_select", lib.sparda_prefill_multihead_select(
        ctypes.byref(shape.c()), _ptr(ck), _ptr(q), _ptr(seq_len), int(batch), _ptr(idx), _ptr(cnt),
        _ptr(ws), ws.numel(), _stream(stream)))


def sparda_prefill_attn(shape, layer, q, idx, cnt, seq_len, batch, out, stream=None):
    """Causal block-sparse prefill attention of a resident layer over the per-chunk
    selections. q, out: bf16 [max_batch, max_ctx, G*H, d]."""
    _check("sparda_prefill_attn", lib.sparda_prefill_attn(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(q), _ptr(idx), _ptr(cnt), _ptr(seq_len),
        int(batch), _ptr(out), _stream(stream)))


# ------------------------------------------------------------------ cross-step block cache
class BlockCache:
    """The block cache of one offloaded layer (include/sparda.h): n_cache HBM slots per
    (sequence, group) holding blocks gathered at earlier steps, the block each slot holds
    (-1: none), the slot of each idx entry, and the gather's scratch."""

    def __init__(self, shape, n_cache=None, device="cuda"):
        n = shape.kslots if n_cache is None else int(n_cache)
        B, G = shape.max_batch, shape.n_groups
        self.n_cache = n
        self.k = torch.zeros((B, G, n, shape.block, shape.head_dim), dtype=torch.bfloat16, device=device)
        self.v = torch.zeros_like(self.k)
        self.blocks = torch.full((B, G, n), -1, dtype=torch.int32, device=device)
        self.slot = torch.full((B, G, shape.kslots), -1, dtype=torch.int32, device=device)
        self.fetch = torch.full((B, G, n), -1, dtype=torch.int32, device=device)

    def reset(self):
        self.blocks.fill_(-1)


def sparda_prefetch_blocks_cached(shape, layer, idx, cnt, seq_len, batch, cache, stats=None, n_ctas=0,
                                  stream=None):
    """Gather of the selected blocks not yet in `cache` (a BlockCache); stats: optional int64
    tensor [2] on the device accumulating hits and misses."""
    _check("sparda_prefetch_blocks_cached", lib.sparda_prefetch_blocks_cached(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(idx), _ptr(cnt), _ptr(seq_len), int(batch),
        _ptr(cache.k), _ptr(cache.v), _ptr(cache.blocks), int(cache.n_cache), _ptr(cache.slot), _ptr(cache.fetch),
        _ptr(stats), int(n_ctas), _stream(stream)))


def sparda_sparse_decode_attn_cached(shape, layer, cache, q, idx, cnt, seq_len, batch, out, ws, stream=None):
    """Attention of an offloaded layer over its selected blocks, read from `cache`."""
    _check("sparda_sparse_decode_attn_cached", lib.sparda_sparse_decode_attn_cached(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), _ptr(cache.k), _ptr(cache.v), int(cache.n_cache),
        _ptr(cache.slot), _ptr(q), _ptr(idx), _ptr(cnt), _ptr(seq_len), int(batch), _ptr(out), _ptr(ws),
        ws.numel(), _stream(stream)))


def sparda_prefetch_blocks_copy_engine(shape, layer, idx_host, cnt_host, seq_len_host, batch, staging_k, staging_v,
                                       stream=None):
    """The gather by one cudaMemcpyAsync per run of consecutive selected blocks; the selection
    (idx_host, cnt_host, seq_len_host) must be int32 CPU tensors. Returns the number of copies
    issued."""
    for t in (idx_host, cnt_host, seq_len_host):
        if t.device.type != "cpu" or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError("the copy-engine gather takes the selection as contiguous int32 CPU tensors")
    n = ctypes.c_int32(0)
    _check("sparda_prefetch_blocks_copy_engine", lib.sparda_prefetch_blocks_copy_engine(
        ctypes.byref(shape.c()), ctypes.byref(layer.c()), ctypes.c_void_p(idx_host.data_ptr()),
        ctypes.c_void_p(cnt_host.data_ptr()), ctypes.c_void_p(seq_len_host.data_ptr()), int(batch),
        _ptr(staging_k), _ptr(staging_v), ctypes.byref(n), _stream(stream)))
    return n.value


# ------------------------------------------------------------------ the 4-bit cache, block mass, eviction
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream_handle(stream, dev):
    """The stream's handle as an integer: `stream`, or the current one of device `dev`."""
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _checked(what, t, dtype, n, dev):
    """t's address, if it is a contiguous tensor of `dtype` on CUDA device `dev` (-1: the CPU) with at
    least n elements."""
    if t.dtype is not dtype or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        raise ValueError("%s: a contiguous %s tensor of at least %d elements on %s is wanted, got %s %s on %s%s" % (
            what, dtype, n, "the CPU" if dev < 0 else "cuda:%d" % dev, t.dtype, tuple(t.shape), t.device,
            "" if t.is_contiguous() else ", strided"))
    return t.data_ptr()


def _cache_device(t):
    """The index of the device that holds a layer's cache, which has to be the current one (the call's
    stream and the library's device state are its)."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError("the layer's cache is on %s; it has to be on the current CUDA device" % t.device)
    return dev


def _kv4_layer(shape, layer):
    """(device, pointer to the C layer) of a LayerKV4, its tensors checked. The C struct is kept with the
    layer until one of its fields is set; the tensors' sizes and addresses are checked in every call."""
    kv, ck = layer.kv, layer.ck
    dev = kv.get_device()
    if dev < 0 or dev != _current_device():
        _cache_device(kv)                            # raises
    _, n_kv, n_ck = shape.sizes()
    args = layer.__dict__.get("_args")
    if (args is not None and args[0] == kv.data_ptr() and args[1] == ck.data_ptr() and kv.numel() >= n_kv and
            ck.numel() >= n_ck):
        return dev, args[2]
    c = c_layer_kv4(_checked("kv", kv, torch.uint8, n_kv, dev), _checked("ck", ck, torch.bfloat16, n_ck, dev))
    ref = ctypes.byref(c)
    layer.__dict__["_args"] = (c.kv, c.ck, ref)
    return dev, ref


def _selection_ptrs(shape, idx, cnt, bg, dev):
    if idx is None and cnt is None:
        return None, None
    if idx is None or cnt is None:
        raise ValueError("idx and cnt come together")
    return _checked("idx", idx, torch.int32, bg * (shape.topk + 2), dev), _checked("cnt", cnt, torch.int32, bg, dev)


def sparda_kv4_quantize(shape, layer, k, v, seq_len, batch, stream=None):
    """Tokens 0 .. seq_len[b]-1 of k and v (bf16 [max_batch, G, max_ctx, d]) into a LayerKV4."""
    dev, lc = _kv4_layer(shape, layer)
    B, G, d, ctx = int(batch), shape.n_groups, shape.head_dim, shape.max_ctx
    n = shape.max_batch * G * ctx * d
    _check("sparda_kv4_quantize", lib.sparda_kv4_quantize(
        shape.ref(), lc, _checked("k", k, torch.bfloat16, n, dev), _checked("v", v, torch.bfloat16, n, dev),
        _checked("seq_len", seq_len, torch.int32, B, dev), B, _stream_handle(stream, dev)))


def sparda_kv4_dequantize(shape, layer, seq_len, batch, k, v, idx=None, cnt=None, stream=None):
    """The values of a LayerKV4 as bf16: every token's rows into k and v [max_batch, G, max_ctx, d], or
    with idx and cnt the selected blocks' into staging buffers [max_batch, G, topk+2, 64, d]."""
    dev, lc = _kv4_layer(shape, layer)
    B, G, d, ctx = int(batch), shape.n_groups, shape.head_dim, shape.max_ctx
    pi, pc = _selection_ptrs(shape, idx, cnt, B * G, dev)
    n = shape.max_batch * G * (ctx if pi is None else (shape.topk + 2) * BLOCK) * d
    _check("sparda_kv4_dequantize", lib.sparda_kv4_dequantize(
        shape.ref(), lc, pi, pc, _checked("seq_len", seq_len, torch.int32, B, dev), B,
        _checked("k", k, torch.bfloat16, n, dev), _checked("v", v, torch.bfloat16, n, dev), _stream_handle(stream, dev)))


def sparda_kv4_append(shape, layer, k_new, v_new, seq_len, batch, stream=None):
    """The current token's key and value (bf16 [B, G, d]) into a LayerKV4, with its compressed key."""
    dev, lc = _kv4_layer(shape, layer)
    B, G, d = int(batch), shape.n_groups, shape.head_dim
    _check("sparda_kv4_append", lib.sparda_kv4_append(
        shape.ref(), lc, _checked("k_new", k_new, torch.bfloat16, B * G * d, dev),
        _checked("v_new", v_new, torch.bfloat16, B * G * d, dev), _checked("seq_len", seq_len, torch.int32, B, dev), B,
        _stream_handle(stream, dev)))


def sparda_kv4_decode_attn(shape, layer, q, idx, cnt, seq_len, batch, out, ws, mass=None, stream=None):
    """Decode attention over a LayerKV4: the selected blocks, or with idx = cnt = None every token.
    mass (float32 [max_batch, G, max_ctx / 64]): the block weights to add to; ws is then a
    WS_KV4_ATTN_MASS workspace, else a WS_KV4_ATTN one."""
    dev, lc = _kv4_layer(shape, layer)
    B, G, d, ctx = int(batch), shape.n_groups, shape.head_dim, shape.max_ctx
    n = B * G * shape.heads_per_group * d
    pi, pc = _selection_ptrs(shape, idx, cnt, B * G, dev)
    pm = None if mass is None else _checked("mass", mass, torch.float32, B * G * (ctx // BLOCK), dev)
    _check("sparda_kv4_decode_attn", lib.sparda_kv4_decode_attn(
        shape.ref(), lc, _checked("q", q, torch.bfloat16, n, dev), pi, pc,
        _checked("seq_len", seq_len, torch.int32, B, dev), B, _checked("out", out, torch.bfloat16, n, dev), pm,
        _checked("ws", ws, torch.uint8, 1, dev), ws.numel(), _stream_handle(stream, dev)))


def _layer_ptrs(shape, layer):
    """(device, pointer to the C layer) of a resident LayerKV, its tensors checked. The C struct is kept with the
    layer until one of its fields is set; the tensors' sizes and addresses are checked in every call."""
    if layer.on_host:
        raise ValueError("a resident layer is wanted")
    k, v, ck = layer.k, layer.v, layer.ck
    dev = k.get_device()
    if dev < 0 or dev != _current_device():
        _cache_device(k)                             # raises
    n, _, n_ck = shape.sizes()
    args = layer.__dict__.get("_args")
    if (args is not None and args[0] == k.data_ptr() and args[1] == v.data_ptr() and args[2] == ck.data_ptr() and
            k.numel() >= n and v.numel() >= n and ck.numel() >= n_ck):
        return dev, args[3]
    c = c_layer_kv(_checked("k", k, torch.bfloat16, n, dev), _checked("v", v, torch.bfloat16, n, dev),
                   _checked("ck", ck, torch.bfloat16, n_ck, dev), None, None, 0, 0)
    ref = ctypes.byref(c)
    layer.__dict__["_args"] = (c.k, c.v, c.ck, ref)
    return dev, ref


def sparda_sparse_decode_attn_mass(shape, layer, q, idx, cnt, seq_len, batch, out, ws, mass, stream=None):
    """sparda_sparse_decode_attn of a resident layer that also adds to mass (float32 [max_batch, G,
    max_ctx / 64]) the attention weight each selected block received. ws: WS_ATTN_MASS."""
    dev, lc = _layer_ptrs(shape, layer)
    B, G = int(batch), shape.n_groups
    n = B * G * shape.heads_per_group * shape.head_dim
    pi, pc = _selection_ptrs(shape, idx, cnt, B * G, dev)
    _check("sparda_sparse_decode_attn_mass", lib.sparda_sparse_decode_attn_mass(
        shape.ref(), lc, _checked("q", q, torch.bfloat16, n, dev), pi, pc,
        _checked("seq_len", seq_len, torch.int32, B, dev), B, _checked("out", out, torch.bfloat16, n, dev),
        _checked("mass", mass, torch.float32, B * G * (shape.max_ctx // BLOCK), dev),
        _checked("ws", ws, torch.uint8, 1, dev), ws.numel(), _stream_handle(stream, dev)))


def _evict(name, fn, ptrs, shape, layer, mass, seq_len, batch, keep, recent, kept, dst_shape, dst, dst_mass, dst_seq_len,
           stream):
    dev, lc = ptrs(shape, layer)
    B, G = int(batch), shape.n_groups
    ds = dc = pm = pl = None
    if dst is not None or dst_shape is not None or dst_mass is not None or dst_seq_len is not None:
        if dst is None or dst_shape is None or dst_mass is None or dst_seq_len is None:
            raise ValueError("dst_shape, dst, dst_mass and dst_seq_len come together")
        ds, dc = dst_shape.ref(), ptrs(dst_shape, dst)[1]
        pm = _checked("dst_mass", dst_mass, torch.float32, B * G * (dst_shape.max_ctx // BLOCK), dev)
        pl = _checked("dst_seq_len", dst_seq_len, torch.int32, B, dev)
    _check(name, fn(
        shape.ref(), lc, _checked("mass", mass, torch.float32, B * G * (shape.max_ctx // BLOCK), dev),
        _checked("seq_len", seq_len, torch.int32, B, dev), ds, dc, pm, pl, B, int(keep), int(recent),
        _checked("kept", kept, torch.int32, B * G * max(0, int(keep)), dev), _stream_handle(stream, dev)))


def sparda_evict_blocks(shape, layer, mass, seq_len, batch, keep, recent, kept, dst_shape=None, dst=None,
                        dst_mass=None, dst_seq_len=None, stream=None):
    """Cut every sequence of a resident LayerKV to `keep` blocks: block 0, the `recent` newest and those
    with the largest mass. In place, or into the cache dst with its dst_mass and dst_seq_len. kept
    (int32 [B, G, keep]) receives the old block numbers."""
    _evict("sparda_evict_blocks", lib.sparda_evict_blocks, _layer_ptrs, shape, layer, mass, seq_len, batch, keep, recent,
           kept, dst_shape, dst, dst_mass, dst_seq_len, stream)


def sparda_kv4_evict_blocks(shape, layer, mass, seq_len, batch, keep, recent, kept, dst_shape=None, dst=None,
                            dst_mass=None, dst_seq_len=None, stream=None):
    """sparda_evict_blocks of a LayerKV4."""
    _evict("sparda_kv4_evict_blocks", lib.sparda_kv4_evict_blocks, _kv4_layer, shape, layer, mass, seq_len, batch, keep,
           recent, kept, dst_shape, dst, dst_mass, dst_seq_len, stream)


# ------------------------------------------------------------------ packed prompts and drafted tokens
def _rows(what, t, dims, heads, d, dev):
    """(address, elements from one row to the next) of new tokens' queries, keys or values: a bf16 tensor of `dims`
    leading dimensions (1: rows, 2: sequences of rows) and [heads, d] on CUDA device `dev`, whose rows hold their
    heads densely and lie evenly spaced."""
    n, st = t.shape, t.stride()
    if (t.dtype is torch.bfloat16 and t.get_device() == dev and len(n) == dims + 2 and n[-1] == d and n[-2] == heads and
            st[-1] == 1 and (st[-2] == d or heads == 1)):
        row = st[dims - 1] if n[dims - 1] > 1 else (st[0] if dims == 2 and n[0] > 1 else heads * d)
        if dims == 1 or n[0] == 1 or st[0] == n[1] * row:
            return t.data_ptr(), row
    raise ValueError("%s: a torch.bfloat16 tensor of %d dimensions ending in [%d, %d] on cuda:%d with dense heads and "
                     "evenly spaced rows is wanted, got %s %s on %s, strides %s" % (
                         what, dims + 2, heads, d, dev, t.dtype, tuple(n), t.device, tuple(st)))


def _kv_rows(k, v, dims, G, d, dev):
    pk, sk = _rows("keys", k, dims, G, d, dev)
    if v.shape != k.shape:
        raise ValueError("keys and values need the same shape, got %s and %s" % (tuple(k.shape), tuple(v.shape)))
    pv, sv = _rows("values", v, dims, G, d, dev)
    if sk != sv:
        raise ValueError("keys and values need the same spacing of rows, got %d and %d elements" % (sk, sv))
    return pk, pv, sk


def _same_rows(q, k, dims):
    if q.shape[:dims] != k.shape[:dims]:
        raise ValueError("queries and keys need the same rows, got %s and %s" % (tuple(q.shape), tuple(k.shape)))


def _int_ptr(what, t, n, dev):
    return None if t is None else _checked(what, t, torch.int32, n, dev)


def sparda_prompt_attn(shape, q, k, v, cu_len, batch, out, ws, past=None, past_len=None, stream=None):
    """Causal attention of packed prompts: sequence b's tokens are rows cu_len[b] .. cu_len[b+1]-1 of q
    [n_tokens, G*H, d] and of k and v [n_tokens, G, d] (slices of one projection are fine). past, past_len: a
    resident LayerKV and how many of its tokens come before each prompt. ws: WS_PROMPT."""
    if past is not None:
        dev, lc = _layer_ptrs(shape, past)
    else:
        dev, lc = _cache_device(q), None
    B, G, H, d = int(batch), shape.n_groups, shape.heads_per_group, shape.head_dim
    n = q.shape[0]
    pq, sq = _rows("q", q, 1, G * H, d, dev)
    pk, pv, skv = _kv_rows(k, v, 1, G, d, dev)
    _same_rows(q, k, 1)
    _check("sparda_prompt_attn", lib.sparda_prompt_attn(
        shape.ref(), lc, _int_ptr("past_len", past_len, B, dev), pq, sq, pk, pv, skv,
        _checked("cu_len", cu_len, torch.int32, B + 1, dev), n, B,
        _checked("out", out, torch.bfloat16, n * G * H * d, dev), _checked("ws", ws, torch.uint8, 1, dev), ws.numel(),
        _stream_handle(stream, dev)))


def sparda_prompt_append(shape, layer, k, v, cu_len, seq_len, batch, new_len=None, stream=None):
    """Packed prompts' keys and values [n_tokens, G, d] into a resident LayerKV behind the seq_len[b] tokens it
    holds (None: behind none), with the compressed keys they complete; new_len (int32 [B]) receives the lengths."""
    dev, lc = _layer_ptrs(shape, layer)
    B = int(batch)
    pk, pv, skv = _kv_rows(k, v, 1, shape.n_groups, shape.head_dim, dev)
    _check("sparda_prompt_append", lib.sparda_prompt_append(
        shape.ref(), lc, pk, pv, skv, _checked("cu_len", cu_len, torch.int32, B + 1, dev), k.shape[0],
        _int_ptr("seq_len", seq_len, B, dev), B, _int_ptr("new_len", new_len, B, dev), _stream_handle(stream, dev)))


def sparda_tree_attn(shape, layer, q, k_new, v_new, parent, seq_len, batch, out, ws, n_nodes=None, idx=None, cnt=None,
                     stream=None):
    """Attention of trees of drafted tokens (q [B, N, G*H, d], k_new and v_new [B, N, G, d], parent int32 [B, N] or
    None for chains; slices of one projection are fine) over the seq_len[b] tokens of a resident LayerKV, all of
    them or those of the blocks idx / cnt. n_nodes: int32 [B], the nodes each sequence uses. ws: WS_TREE."""
    dev, lc = _layer_ptrs(shape, layer)
    B, G, H, d = int(batch), shape.n_groups, shape.heads_per_group, shape.head_dim
    pq, sq = _rows("q", q, 2, G * H, d, dev)
    N = q.shape[1]
    pk, pv, skv = _kv_rows(k_new, v_new, 2, G, d, dev)
    _same_rows(q, k_new, 2)
    if q.shape[0] < B:
        raise ValueError("q holds %d sequences, %d are wanted" % (q.shape[0], B))
    pi, pc = _selection_ptrs(shape, idx, cnt, B * G, dev)
    _check("sparda_tree_attn", lib.sparda_tree_attn(
        shape.ref(), lc, pq, sq, pk, pv, skv, _int_ptr("parent", parent, B * N, dev), _int_ptr("n_nodes", n_nodes, B, dev),
        N, pi, pc, _checked("seq_len", seq_len, torch.int32, B, dev), B,
        _checked("out", out, torch.bfloat16, B * N * G * H * d, dev), _checked("ws", ws, torch.uint8, 1, dev), ws.numel(),
        _stream_handle(stream, dev)))


def sparda_tree_commit(shape, layer, k_new, v_new, path, n_path, seq_len, batch, new_len=None, stream=None):
    """The accepted nodes path[b, :n_path[b]] (int32 [B, N]) of trees of drafted tokens (k_new, v_new [B, N, G, d])
    into a resident LayerKV behind its seq_len[b] tokens, with the compressed keys they complete; new_len (int32
    [B]) receives the lengths."""
    dev, lc = _layer_ptrs(shape, layer)
    B = int(batch)
    pk, pv, skv = _kv_rows(k_new, v_new, 2, shape.n_groups, shape.head_dim, dev)
    N = k_new.shape[1]
    if k_new.shape[0] < B:
        raise ValueError("k_new holds %d sequences, %d are wanted" % (k_new.shape[0], B))
    _check("sparda_tree_commit", lib.sparda_tree_commit(
        shape.ref(), lc, pk, pv, skv, N, _checked("path", path, torch.int32, B * N, dev),
        _checked("n_path", n_path, torch.int32, B, dev), _checked("seq_len", seq_len, torch.int32, B, dev), B,
        _int_ptr("new_len", new_len, B, dev), _stream_handle(stream, dev)))
