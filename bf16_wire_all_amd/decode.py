"""Python binding of the decode-step calls (include/xfer_decode.h): argument
marshalling only, as the package's other calls.

Device buffers are torch CUDA tensors on the current device; heads may be
slices of a fused buffer (the last two dimensions dense, any row stride).
Every call takes the current torch stream unless `stream` is given, and
raises XferError on a non-OK status."""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import OK, OUT_BF16, OUT_F32, Shard, _check, _stream, lib as _base_lib

KV_BF16, KV_E4M3 = 0, 1
ROPE_HALVES, ROPE_PAIRS = 0, 1

EXPORTED = ["xfer_qkv_rope_store", "xfer_attn_workspace_bytes", "xfer_attn_paged", "xfer_sample_workspace_bytes",
            "xfer_sample_merge"]

SAMPLE_PARAMS = np.dtype([("temperature", "<f4"), ("top_k", "<u4"), ("top_p", "<f4"), ("min_p", "<f4")])
SAMPLED = np.dtype([("prob", "<f4"), ("idx", "<i4")])


class KVCacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_uint64), ("token_stride", ctypes.c_uint64),
                ("head_stride", ctypes.c_uint64), ("n_pages", ctypes.c_uint32), ("page_tokens", ctypes.c_uint32),
                ("kv_heads", ctypes.c_uint32), ("head_dim", ctypes.c_uint32), ("kind", ctypes.c_int32),
                ("reserved", ctypes.c_uint32)]


class RopeC(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("max_pos", ctypes.c_uint32),
                ("rot_dim", ctypes.c_uint32), ("style", ctypes.c_int32), ("reserved", ctypes.c_uint32)]


class QKVC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q_ld", ctypes.c_uint64),
                ("k_ld", ctypes.c_uint64), ("v_ld", ctypes.c_uint64), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("tokens", ctypes.c_uint32), ("q_heads", ctypes.c_uint32),
                ("eps", ctypes.c_float), ("reserved", ctypes.c_uint32)]


class PagedBatchC(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("table_ld", ctypes.c_uint64),
                ("rows", ctypes.c_uint32), ("max_len", ctypes.c_uint32), ("window", ctypes.c_uint32),
                ("sinks", ctypes.c_uint32)]


_lib = None


def lib():
    """The loaded libxfer.so with the decode-step signatures."""
    global _lib
    if _lib is None:
        L = _base_lib()
        P, S, U32, U64, I, F = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int,
                                ctypes.c_float)
        L.xfer_qkv_rope_store.argtypes = [ctypes.POINTER(KVCacheC), ctypes.POINTER(QKVC), ctypes.POINTER(RopeC), P, P,
                                          U64, P]
        L.xfer_qkv_rope_store.restype = I
        L.xfer_attn_workspace_bytes.argtypes = [ctypes.POINTER(KVCacheC), ctypes.POINTER(PagedBatchC), U32]
        L.xfer_attn_workspace_bytes.restype = S
        L.xfer_attn_paged.argtypes = [ctypes.POINTER(KVCacheC), ctypes.POINTER(PagedBatchC), P, U64, U32, F, P, U64, I,
                                      P, S, P]
        L.xfer_attn_paged.restype = I
        L.xfer_sample_workspace_bytes.argtypes = [U32, U32, U32]
        L.xfer_sample_workspace_bytes.restype = S
        L.xfer_sample_merge.argtypes = [ctypes.POINTER(Shard), ctypes.POINTER(Shard), P, P, P, P, S, P]
        L.xfer_sample_merge.restype = I
        _lib = L
    return _lib


# What a tensor may be of to stand for each format: the type itself, or whole
# numbers of its size as bit patterns.  Another float type would be read as if
# it were this one.
_BF16 = frozenset((torch.bfloat16, torch.int16, torch.uint16))
_E4M3 = frozenset((torch.float8_e4m3fn, torch.uint8, torch.int8))
_F32 = frozenset((torch.float32,))
_INT32 = frozenset((torch.int32, torch.uint32))
_INT64 = frozenset((torch.int64, torch.uint64))


def _names(types) -> str:
    return " or ".join(sorted(str(t) for t in types))


# The checks below run at every call, in front of kernels of a few
# microseconds: each asks a tensor as few things as it can.

def _flat(t, types, device: int, what: str) -> int:
    """Pointer of a contiguous tensor of the call's device (None: NULL); types None: any."""
    if t is None:
        return 0
    if t.get_device() != device or (types is not None and t.dtype not in types) or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor{' of ' + _names(types) if types else ''} on cuda:{device}")
    return t.data_ptr()


def _rows(t, heads, head_dim: int, types, device: int, what: str):
    """(pointer, rows, heads, ld in elements) of a [rows, heads, head_dim] tensor whose rows are dense."""
    rows, h, d = t.shape
    s0, s1, s2 = t.stride()
    if t.get_device() != device or t.dtype not in types or d != head_dim or (heads is not None and h != heads):
        raise ValueError(f"{what}: expected [rows, {heads or 'heads'}, {head_dim}] of {_names(types)} on cuda:{device}")
    if s2 != 1 or (h > 1 and s1 != d):
        raise ValueError(f"{what}: a row's heads must lie one after the other")
    return t.data_ptr(), rows, h, s0 if rows > 1 else h * d


def _stream_on(device: int, stream) -> int:
    """The stream of a call whose tensors are on `device`, which has to be the
    current one: pointers belong to the device that is current at the call."""
    if device < 0 or device != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on device {device}, which is not the current CUDA device")
    return torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


class KVCache:
    """A paged cache of keys and values; keeps its tensors alive."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or v.shape != k.shape or v.stride() != k.stride():
            raise ValueError("k and v must be alike: [pages, page_tokens, heads, head_dim] with the same strides")
        types = next((t for t in (_BF16, _E4M3) if k.dtype in t and v.dtype in t), None)
        if types is None or v.device != k.device or k.device.type != "cuda":
            raise ValueError("k and v must be BF16 or E4M3 CUDA tensors of one device")
        n, p, h, d = k.shape
        s, e = k.stride(), k.element_size()
        if s[3] != 1:
            raise ValueError("a head's elements must lie one after the other")
        for scale in (k_scale, v_scale):
            if scale is not None and scale.numel() != h:
                raise ValueError("one scale for each head")
        self.device, self.kv_heads, self.head_dim, self.page_tokens, self.n_pages = k.get_device(), h, d, p, n
        self.tensors = (k, v, k_scale, v_scale)
        # the stride of a dimension of one element is never walked: any multiple of 16 will do
        stride = [s[i] * e if k.shape[i] > 1 else 0 for i in range(3)]
        self.c = KVCacheC(k.data_ptr(), v.data_ptr(), _flat(k_scale, _F32, self.device, "k_scale") or None,
                          _flat(v_scale, _F32, self.device, "v_scale") or None, stride[0], stride[1], stride[2], n, p, h,
                          d, KV_BF16 if types is _BF16 else KV_E4M3, 0)


def kv_cache(k, v, k_scale=None, v_scale=None) -> KVCache:
    """k, v: [pages, page_tokens, heads, head_dim] CUDA tensors or views (BF16 or
    float8_e4m3fn, or int16, uint16, int8 or uint8 as their bit patterns), any
    strides but a dense last dimension;
    k_scale, v_scale: F32[heads] of an E4M3 cache."""
    return KVCache(k, v, k_scale, v_scale)


def qkv_rope_store(cache: KVCache, q, k, v, positions, cos_sin, slots, q_out, q_weight=None, k_weight=None,
                   eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """q: [tokens, q_heads, head_dim], k, v: [tokens, kv_heads, head_dim] (BF16 or
    its patterns; slices of a fused projection will do); positions: int32[tokens]
    and cos_sin: F32[max_pos, rot_dim] (both None: no rotation); slots:
    int64[tokens]; q_out like q (q itself is computed in place);
    interleaved: dims 2i and 2i + 1 form a pair, not i and i + rot_dim / 2."""
    dev, d = cache.device, cache.head_dim
    stream = _stream_on(dev, stream)
    kp, tokens, _, k_ld = _rows(k, cache.kv_heads, d, _BF16, dev, "k")
    vp, vt, _, v_ld = _rows(v, cache.kv_heads, d, _BF16, dev, "v")
    qp, qt, q_heads, q_ld = _rows(q, None, d, _BF16, dev, "q")
    op, ot, _, o_ld = _rows(q_out, q_heads, d, _BF16, dev, "q_out")
    if not (vt == qt == ot == tokens == slots.numel()):
        raise ValueError("q, k, v, q_out and slots must have one row for each token")
    for w in (q_weight, k_weight):
        if w is not None and w.numel() != d:
            raise ValueError("one weight for each element of a head")
    rope = RopeC(0, 0, 0, 0, ROPE_PAIRS if interleaved else ROPE_HALVES, 0)
    if cos_sin is not None:
        if positions is None or cos_sin.dim() != 2 or positions.numel() != tokens:
            raise ValueError("cos_sin must be [max_pos, rot_dim], with a position for each token")
        rope.cos_sin = _flat(cos_sin, _F32, dev, "cos_sin")
        rope.positions = _flat(positions, _INT32, dev, "positions")
        rope.max_pos, rope.rot_dim = cos_sin.shape
    qkv = QKVC(qp, kp, vp, q_ld, k_ld, v_ld, _flat(q_weight, _BF16, dev, "q_weight"),
               _flat(k_weight, _BF16, dev, "k_weight"), tokens, q_heads, eps, 0)
    status = lib().xfer_qkv_rope_store(ctypes.byref(cache.c), ctypes.byref(qkv), ctypes.byref(rope),
                                       _flat(slots, _INT64, dev, "slots"), op, o_ld, stream)
    if status != OK:
        _check(status, "xfer_qkv_rope_store")


def qkv_rope_store_raw(cache: KVCacheC, qkv: QKVC, rope: RopeC, slots_ptr: int, q_out_ptr: int, q_out_ld: int,
                       stream=None) -> int:
    """Raw-pointer form; returns the status without raising."""
    return lib().xfer_qkv_rope_store(ctypes.byref(cache), ctypes.byref(qkv), ctypes.byref(rope), slots_ptr, q_out_ptr,
                                     q_out_ld, _stream(stream))


# ------------------------------------------------- attention of one new token

def attn_workspace_bytes(cache: KVCache, rows: int, q_heads: int, max_len: int, window: int = 0, sinks: int = 0) -> int:
    """Bytes of workspace that attn_paged needs for these sizes."""
    batch = PagedBatchC(0, 0, 0, rows, max_len, window, sinks)
    return int(lib().xfer_attn_workspace_bytes(ctypes.byref(cache.c), ctypes.byref(batch), q_heads))


def attn_paged(cache: KVCache, q, page_table, lens, max_len: int, scale: float, out, workspace=None, window: int = 0,
               sinks: int = 0, stream=None) -> None:
    """q: [rows, q_heads, head_dim] (BF16 or its patterns); page_table: int32 or
    uint32 [rows, at least ceil(max_len / page_tokens)], dense within a row;
    lens: int32 or uint32 [rows] (a negative one is a large length, cut to
    max_len); out: like q, BF16 (or its patterns) or F32; workspace: a CUDA
    tensor of at least attn_workspace_bytes() bytes (None if that is 0)."""
    dev, d = cache.device, cache.head_dim
    stream = _stream_on(dev, stream)
    qp, rows, q_heads, q_ld = _rows(q, None, d, _BF16, dev, "q")
    f32 = out.dtype in _F32
    op, o_rows, _, o_ld = _rows(out, q_heads, d, _F32 if f32 else _BF16, dev, "out")
    if o_rows != rows or lens.numel() != rows or page_table.dim() != 2 or page_table.shape[0] != rows:
        raise ValueError("q, page_table, lens and out must have the same rows")
    width, ts = page_table.shape[1], page_table.stride()
    if page_table.get_device() != dev or page_table.dtype not in _INT32 or (width > 1 and ts[1] != 1):
        raise ValueError(f"page_table: expected {_names(_INT32)} on cuda:{dev}, dense within a row")
    if width * cache.page_tokens < max_len:
        raise ValueError("page_table is too narrow for max_len")
    ws, ws_bytes = 0, 0
    if workspace is not None:
        ws_bytes, ws = workspace.numel() * workspace.element_size(), _flat(workspace, None, dev, "workspace")
    batch = PagedBatchC(page_table.data_ptr(), _flat(lens, _INT32, dev, "lens"), ts[0] if rows > 1 else width, rows,
                        max_len, window, sinks)
    status = lib().xfer_attn_paged(ctypes.byref(cache.c), ctypes.byref(batch), qp, q_ld, q_heads, scale, op, o_ld,
                                   OUT_F32 if f32 else OUT_BF16, ws, ws_bytes, stream)
    if status != OK:
        _check(status, "xfer_attn_paged")


def attn_paged_raw(cache: KVCacheC, batch: PagedBatchC, q_ptr: int, q_ld: int, q_heads: int, scale: float,
                   out_ptr: int, out_ld: int, out_mode: int, ws_ptr: int, ws_bytes: int, stream=None) -> int:
    """Raw-pointer form; returns the status without raising."""
    return lib().xfer_attn_paged(ctypes.byref(cache), ctypes.byref(batch), q_ptr, q_ld, q_heads, scale, out_ptr,
                                 out_ld, out_mode, ws_ptr, ws_bytes, _stream(stream))


# ------------------------------------------------------------------ sampling

def shard(logits, ncols: int, col_offset: int) -> Shard:
    """A column shard of BF16 logits (or their patterns): a CUDA tensor [rows, at
    least ncols] whose rows are dense, and a multiple of 8 elements apart; the
    shard keeps it alive."""
    rows, width = logits.shape
    ts = logits.stride()
    if not logits.is_cuda or logits.dtype not in _BF16 or width < ncols or (width > 1 and ts[1] != 1):
        raise ValueError(f"expected a CUDA tensor of {_names(_BF16)}, dense within a row and ncols wide")
    # a single row has no distance to the next: any multiple of 8 that holds it will do
    s = Shard(logits.data_ptr(), ts[0] if rows > 1 else -(-width // 8) * 8, rows, ncols, col_offset)
    s.tensor, s.device = logits, logits.get_device()
    return s


def sample_workspace_bytes(rows: int, ncols0: int, ncols1: int) -> int:
    return int(lib().xfer_sample_workspace_bytes(rows, ncols0, ncols1))


def sample_merge(s0: Shard, s1: Shard, params, u, out, workspace, stream=None) -> None:
    """params: CUDA tensor of rows * 16 bytes (SAMPLE_PARAMS records); u: F32[rows]
    in [0, 1); out: CUDA tensor of rows * 8 bytes (SAMPLED records); workspace:
    at least sample_workspace_bytes() bytes, any contents."""
    dev, rows = u.get_device(), s0.rows
    stream = _stream_on(dev, stream)
    # a shard made from a pointer alone does not say where it lies
    if getattr(s0, "device", dev) != dev or getattr(s1, "device", dev) != dev:
        raise ValueError(f"expected shards on cuda:{dev}, where u is")
    if params.numel() * params.element_size() != rows * 16 or u.numel() != rows:
        raise ValueError("params and u must have one record for each row")
    if out.numel() * out.element_size() != rows * 8:
        raise ValueError("out must have 8 bytes for each row")
    status = lib().xfer_sample_merge(ctypes.byref(s0), ctypes.byref(s1), _flat(params, None, dev, "params"),
                                     _flat(u, _F32, dev, "u"), _flat(out, None, dev, "out"),
                                     _flat(workspace, None, dev, "workspace"),
                                     workspace.numel() * workspace.element_size(), stream)
    if status != OK:
        _check(status, "xfer_sample_merge")


def sample_merge_raw(s0: Shard, s1: Shard, params_ptr: int, u_ptr: int, out_ptr: int, ws_ptr: int, ws_bytes: int,
                     stream=None) -> int:
    """Raw-pointer form; returns the status without raising."""
    return lib().xfer_sample_merge(ctypes.byref(s0), ctypes.byref(s1), params_ptr, u_ptr, out_ptr, ws_ptr, ws_bytes,
                                   _stream(stream))
