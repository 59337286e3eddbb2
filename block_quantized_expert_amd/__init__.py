"""Python binding of librfpx (include/rfpx.h and include/rfpx_attn.h):
argument marshalling only.

Every computation runs in the HIP kernels of librfpx.so; PyTorch supplies
device memory and the current stream.  The functions carry the C names and
raise ``RfpxError`` on any non-zero status.  If the library is not built, or
was linked against a different HIP runtime than the one torch loaded, import
of the library fails loudly -- there is no fallback.

Format and layer definitions are in include/rfpx.h; they follow page
"DeepSeek V4 Flash 在 128GB 锐龙 AI MAX+ 上跑到 32 tok/s" (taozi.news),
section "ROCmFPX：把 284B 权重压进 128 GB", and page "Lucebox专攻DeepSeek V4…"
(m.mzlw.cn), section "MoE 专家并行".
"""
from __future__ import annotations

import ctypes as C
import os
import threading
from typing import Optional, Sequence

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "librfpx.so")

RFPX_FP2, RFPX_FP3, RFPX_FP4 = 2, 3, 4
RFPX_X_F32, RFPX_X_BF16 = 0, 1
Q_MAX, K_MAX, E_MAX = 8, 8, 1024
BLOCK_BYTES = {RFPX_FP2: 10, RFPX_FP3: 14, RFPX_FP4: 17}

# every symbol include/rfpx.h declares
SYMBOLS = (
    "rfpx_block_bytes", "rfpx_matrix_bytes", "rfpx_pack", "rfpx_pack_weighted",
    "rfpx_pack_codes",
    "rfpx_unpack", "moe_image_bytes", "moe_image_build", "moe_image_validate",
    "moe_image_unpack",
    "moe_workspace_bytes", "moe_route_topk", "moe_layer_forward",
    "moe_layer_forward_timed", "moe_layer_forward_noalloc", "moe_noalloc_scratch_bytes",
    "moe_prefill_forward", "moe_prefill_forward_timed",
    "rfpx_dense_image_bytes", "rfpx_dense_image_build", "rfpx_dense_image_unpack",
    "rfpx_dense_workspace_bytes", "rfpx_dense_forward",
    "rfpx_stream_read", "rfpx_stream_read_sink_words",
    "rfpx_status_str", "rfpx_last_error",
)

# ... and include/rfpx_attn.h
ATTN_SYMBOLS = (
    "rfpx_kv_pool_bytes", "rfpx_qk_norm_rope", "rfpx_kv_append", "rfpx_kv_unpack",
    "rfpx_attn_workspace_bytes", "rfpx_attn_forward", "rfpx_attn_weights",
    "rfpx_kv_evict_workspace_bytes", "rfpx_kv_evict",
)
RFPX_ROPE_HALF, RFPX_ROPE_PAIRS = 0, 1


class RfpxError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: status {status}: {msg}")
        self.status = status


class MoeLayerC(C.Structure):
    _fields_ = [("d", C.c_int), ("f", C.c_int), ("n_experts", C.c_int),
                ("top_k", C.c_int), ("routed_scale", C.c_float),
                ("router_w", C.c_void_p), ("image", C.c_void_p),
                ("fmts", C.POINTER(C.c_int)), ("image_bytes", C.c_size_t)]


class KvCacheC(C.Structure):
    _fields_ = [("n_kv_heads", C.c_int), ("head_dim", C.c_int), ("page_tokens", C.c_int),
                ("n_pages", C.c_int), ("pool", C.c_void_p), ("pool_bytes", C.c_size_t)]


class KvBatchC(C.Structure):
    _fields_ = [("n_seqs", C.c_int), ("pages_per_seq", C.c_int), ("max_cols", C.c_int),
                ("max_len", C.c_int), ("page_table", C.c_void_p), ("lens", C.c_void_p),
                ("starts", C.c_void_p)]


class RopeC(C.Structure):
    _fields_ = [("dim", C.c_int), ("style", C.c_int), ("inv_freq_host", C.c_void_p)]


_lock = threading.Lock()
_lib = None


def lib():
    """Load librfpx.so once (after torch, so that both share one HIP
    runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        import torch  # noqa: F401  -- torch's HIP runtime must be loaded first
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run __graft_entry__.build() "
                "(hipcc --offload-arch=gfx950)")
        l = C.CDLL(LIB_PATH)
        hips = set()
        with open("/proc/self/maps") as fh:
            for line in fh:
                if "libamdhip64" in line:
                    hips.add(line.split()[-1])
        if len(hips) > 1:
            raise RuntimeError(f"two HIP runtimes in one process: {sorted(hips)}")
        P, I, S = C.c_void_p, C.c_int, C.c_size_t
        LP = C.POINTER(MoeLayerC)
        sig = {
            "rfpx_block_bytes": (S, [I]),
            "rfpx_matrix_bytes": (S, [I, I, I]),
            "rfpx_pack": (I, [I, P, I, I, P, S, P]),
            "rfpx_pack_weighted": (I, [I, P, P, I, I, P, S, P]),
            "rfpx_pack_codes": (I, [I, P, P, I, I, P, S, P]),
            "rfpx_unpack": (I, [I, P, I, I, P, P]),
            "moe_image_bytes": (S, [I, I, I, P]),
            "moe_image_build": (I, [I, I, I, P, P, P, S, P]),
            "moe_image_validate": (I, [LP, P, P]),
            "moe_image_unpack": (I, [LP, I, I, P, P]),
            "moe_workspace_bytes": (S, [LP, I, I]),
            "moe_route_topk": (I, [LP, P, I, I, P, P, P, S, P]),
            "moe_layer_forward": (I, [LP, P, I, I, P, P, S, P]),
            "moe_layer_forward_timed": (I, [LP, P, I, I, P, P, S, P, P]),
            "moe_layer_forward_noalloc": (I, [LP, P, I, I, P, P]),
            "moe_noalloc_scratch_bytes": (S, []),
            "moe_prefill_forward": (I, [LP, P, I, I, P, P, S, P]),
            "moe_prefill_forward_timed": (I, [LP, P, I, I, P, P, S, P, P]),
            "rfpx_dense_image_bytes": (S, [I, I, I]),
            "rfpx_dense_image_build": (I, [I, P, I, I, P, S, P]),
            "rfpx_dense_image_unpack": (I, [I, P, I, I, P, P]),
            "rfpx_dense_workspace_bytes": (S, [I, I, I, I]),
            "rfpx_dense_forward": (I, [I, P, I, I, P, I, I, P, P, S, P]),
            "rfpx_stream_read": (I, [P, S, P, P]),
            "rfpx_stream_read_sink_words": (S, []),
            "rfpx_status_str": (C.c_char_p, [I]),
            "rfpx_last_error": (C.c_char_p, []),
        }
        L, F = C.c_longlong, C.c_float
        KP, BP = C.POINTER(KvCacheC), C.POINTER(KvBatchC)
        sig.update({
            "rfpx_kv_pool_bytes": (S, [I, I, I, I]),
            "rfpx_qk_norm_rope": (I, [P, L, I, P, L, I, I, I, I, P, P, P, F, C.POINTER(RopeC),
                                      P, L, P, L, I, P]),
            "rfpx_kv_append": (I, [KP, BP, P, L, P, L, I, I, P, P, P, P]),
            "rfpx_kv_unpack": (I, [KP, BP, I, P, P, I, P]),
            "rfpx_attn_workspace_bytes": (S, [KP, BP, I, I]),
            "rfpx_attn_forward": (I, [KP, BP, P, L, I, I, I, F, P, L, P, P, S, P]),
            "rfpx_attn_weights": (I, [KP, BP, P, L, I, I, I, F, P, F, P, P, P]),
            "rfpx_kv_evict_workspace_bytes": (S, [KP, BP, I]),
            "rfpx_kv_evict": (I, [KP, BP, I, I, P, P, P, P, P, P, S, P]),
        })
        for name, (res, args) in sig.items():
            fn = getattr(l, name)
            fn.restype = res
            fn.argtypes = args
        _lib = l
        return l


def _check(fn: str, st: int) -> None:
    if st != 0:
        l = lib()
        raise RfpxError(fn, st, (l.rfpx_last_error() or b"").decode())


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _ptr(t) -> C.c_void_p:
    return C.c_void_p(t.data_ptr())


def _new(like, shape, dtype, stream=None):
    """An uninitialized tensor beside `like` for a call on `stream` (None: the
    current one).  Its memory comes from that stream's pool, where nothing
    queued on another stream can still be using it; the caller may go on with
    it on the current stream."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    import torch
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    if stream != here:
        t.record_stream(here)
    return t


def _need_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("tensor must be on the GPU")
        if not t.is_contiguous():
            raise ValueError("tensor must be contiguous")


# ------------------------------------------------------------------- codec

def rfpx_block_bytes(fmt: int) -> int:
    return lib().rfpx_block_bytes(fmt)


def rfpx_matrix_bytes(fmt: int, rows: int, cols: int) -> int:
    return lib().rfpx_matrix_bytes(fmt, rows, cols)


def rfpx_pack(fmt: int, w, out=None, stream=None):
    """Quantize w (cuda fp32 [rows][cols]) into canonical blocks (uint8)."""
    import torch
    _need_cuda(w)
    rows, cols = w.shape
    n = rfpx_matrix_bytes(fmt, rows, cols)
    if out is None:
        out = _new(w, n, torch.uint8, stream)
    _check("rfpx_pack", lib().rfpx_pack(fmt, _ptr(w), rows, cols, _ptr(out),
                                        out.numel(), _stream(stream)))
    return out


def rfpx_pack_weighted(fmt: int, w, imp, out=None, stream=None):
    """Importance-weighted quantizer: w cuda fp32 [rows][cols], imp cuda
    fp32 [cols] (>= 0)."""
    import torch
    _need_cuda(w, imp)
    rows, cols = w.shape
    if imp.numel() != cols:
        raise ValueError("imp must hold one importance per column")
    n = rfpx_matrix_bytes(fmt, rows, cols)
    if out is None:
        out = _new(w, n, torch.uint8, stream)
    _check("rfpx_pack_weighted", lib().rfpx_pack_weighted(
        fmt, _ptr(w), _ptr(imp), rows, cols, _ptr(out), out.numel(), _stream(stream)))
    return out


def rfpx_pack_codes(fmt: int, codes, scale_bits, out=None, stream=None):
    """codes: cuda uint8 [rows][cols]; scale_bits: cuda int16/uint16 bits
    [rows][cols/32]."""
    import torch
    _need_cuda(codes, scale_bits)
    rows, cols = codes.shape
    n = rfpx_matrix_bytes(fmt, rows, cols)
    if out is None:
        out = _new(codes, n, torch.uint8, stream)
    _check("rfpx_pack_codes", lib().rfpx_pack_codes(
        fmt, _ptr(codes), _ptr(scale_bits), rows, cols, _ptr(out), out.numel(),
        _stream(stream)))
    return out


def rfpx_unpack(fmt: int, data, rows: int, cols: int, out=None, stream=None):
    import torch
    _need_cuda(data)
    if out is None:
        out = _new(data, (rows, cols), torch.float32, stream)
    _check("rfpx_unpack", lib().rfpx_unpack(fmt, _ptr(data), rows, cols, _ptr(out),
                                            _stream(stream)))
    return out


# ------------------------------------------------------------------- image

def _fmts_array(fmts) -> C.Array:
    flat = [int(v) for row in fmts for v in (row if hasattr(row, "__len__") else [row])]
    return (C.c_int * len(flat))(*flat)


def moe_image_bytes(d: int, f: int, n_experts: int, fmts) -> int:
    return lib().moe_image_bytes(d, f, n_experts, C.cast(_fmts_array(fmts), C.c_void_p))


def moe_image_build(d: int, f: int, n_experts: int, fmts,
                    canonical: Sequence, out=None, stream=None):
    """canonical: (E+1)*3 cuda uint8 tensors (gate, up, down per expert, the
    shared expert last).  Returns the image (cuda uint8, 256-B aligned)."""
    import torch
    fa = _fmts_array(fmts)
    n = lib().moe_image_bytes(d, f, n_experts, C.cast(fa, C.c_void_p))
    if n == 0:
        raise RfpxError("moe_image_bytes", -2, "unsupported shape or format table")
    for t in canonical:
        _need_cuda(t)
    ptrs = (C.c_void_p * len(canonical))(*[t.data_ptr() for t in canonical])
    if out is None:
        out = _new(canonical[0], n, torch.uint8, stream)
    _check("moe_image_build", lib().moe_image_build(
        d, f, n_experts, C.cast(fa, C.c_void_p), C.cast(ptrs, C.c_void_p), _ptr(out),
        out.numel(), _stream(stream)))
    return out


class MoeLayer:
    """A layer descriptor (moe_layer) plus references that keep its device
    buffers and format table alive.  image_bytes defaults to the size of
    the image tensor."""

    def __init__(self, d: int, f: int, n_experts: int, top_k: int, router_w,
                 image, fmts, routed_scale: float = 1.0,
                 image_bytes: Optional[int] = None):
        _need_cuda(router_w, image)
        self._fmts = _fmts_array(fmts)
        self._router_w = router_w
        self._image = image
        if image_bytes is None:
            image_bytes = image.numel()
        self.c = MoeLayerC(d, f, n_experts, top_k, routed_scale,
                           router_w.data_ptr(), image.data_ptr(),
                           C.cast(self._fmts, C.POINTER(C.c_int)), image_bytes)
        self.d, self.f, self.n_experts, self.top_k = d, f, n_experts, top_k

    @property
    def ref(self):
        return C.byref(self.c)


def moe_image_validate(layer: MoeLayer, report=None, stream=None):
    """Enqueue the device check of the layer's image; returns the report
    tensor (cuda int32 [4], read as uint32: header faults, mismatching table
    entries, blocks with a non-finite scale, 0), valid once the stream
    passes."""
    import torch
    if report is None:
        report = _new(layer._image, 4, torch.int32, stream)
    _need_cuda(report)
    _check("moe_image_validate", lib().moe_image_validate(layer.ref, _ptr(report),
                                                          _stream(stream)))
    return report


def check_image(layer: MoeLayer, stream=None) -> None:
    """moe_image_validate, waited for: raises RfpxError if the image fails."""
    import torch
    rep = moe_image_validate(layer, stream=stream)
    (stream or torch.cuda.current_stream()).synchronize()
    r = [int(v) & 0xFFFFFFFF for v in rep.cpu().tolist()]
    if any(r):
        raise RfpxError("moe_image_validate", -4,
                        f"header faults 0x{r[0]:x}, {r[1]} table entries differ from the "
                        f"format table, {r[2]} blocks with a non-finite scale")


def moe_image_unpack(layer: MoeLayer, expert: int, matrix: int, out=None,
                     stream=None):
    import torch
    rows, cols = (layer.f, layer.d) if matrix < 2 else (layer.d, layer.f)
    if out is None:
        out = _new(layer._image, (rows, cols), torch.float32, stream)
    _check("moe_image_unpack", lib().moe_image_unpack(layer.ref, expert, matrix,
                                                      _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------- forward

def moe_workspace_bytes(layer: MoeLayer, q_or_T: int, prefill: bool = False) -> int:
    return lib().moe_workspace_bytes(layer.ref, q_or_T, 1 if prefill else 0)


def workspace(layer: MoeLayer, q_or_T: int, prefill: bool = False, stream=None):
    """A workspace of the right size (uninitialized: the library needs no
    particular contents) for calls on `stream` (None: the current one)."""
    import torch
    n = moe_workspace_bytes(layer, q_or_T, prefill)
    if n == 0:
        raise RfpxError("moe_workspace_bytes", -2, "unsupported shape")
    return _new(layer._image, n, torch.uint8, stream)


def _xtype(x) -> int:
    import torch
    if x.dtype == torch.bfloat16:
        return RFPX_X_BF16
    if x.dtype == torch.float32:
        return RFPX_X_F32
    raise ValueError("x must be bfloat16 or float32")


def moe_route_topk(layer: MoeLayer, x, ids=None, w=None, ws=None, stream=None):
    import torch
    _need_cuda(x)
    q = x.shape[0]
    if ids is None:
        ids = _new(x, (q, layer.top_k), torch.int32, stream)
    if w is None:
        w = _new(x, (q, layer.top_k), torch.float32, stream)
    if ws is None:
        ws = workspace(layer, q, stream=stream)
    _check("moe_route_topk", lib().moe_route_topk(
        layer.ref, _ptr(x), _xtype(x), q, _ptr(ids), _ptr(w), _ptr(ws), ws.numel(),
        _stream(stream)))
    return ids, w


def moe_layer_forward(layer: MoeLayer, x, y=None, ws=None, stream=None):
    import torch
    _need_cuda(x)
    q = x.shape[0]
    if y is None:
        y = _new(x, (q, layer.d), torch.float32, stream)
    if ws is None:
        ws = workspace(layer, q, stream=stream)
    _check("moe_layer_forward", lib().moe_layer_forward(
        layer.ref, _ptr(x), _xtype(x), q, _ptr(y), _ptr(ws), ws.numel(),
        _stream(stream)))
    return y


def moe_layer_forward_timed(layer: MoeLayer, x, y, ws, events, stream=None):
    """events: a ctypes array of 6 hipEvent_t handles (created by the
    caller on this device), stamped with the start and end of the routing
    kernels, the gate/up kernel and the down kernel."""
    _need_cuda(x)
    if events is not None and len(events) != 6:
        raise ValueError("moe_layer_forward_timed takes 6 events")
    _check("moe_layer_forward_timed", lib().moe_layer_forward_timed(
        layer.ref, _ptr(x), _xtype(x), x.shape[0], _ptr(y), _ptr(ws), ws.numel(),
        _stream(stream), C.cast(events, C.c_void_p) if events is not None else None))
    return y


def moe_layer_forward_noalloc(layer: MoeLayer, x, y, stream=None):
    """moe_layer_forward on the library's own device scratch: y (cuda fp32
    [q][d]) is given by the caller, nothing is allocated."""
    _need_cuda(x, y)
    _check("moe_layer_forward_noalloc", lib().moe_layer_forward_noalloc(
        layer.ref, _ptr(x), _xtype(x), x.shape[0], _ptr(y), _stream(stream)))
    return y


def moe_prefill_forward(layer: MoeLayer, x, y=None, ws=None, stream=None):
    import torch
    _need_cuda(x)
    T = x.shape[0]
    if y is None:
        y = _new(x, (T, layer.d), torch.float32, stream)
    if ws is None:
        ws = workspace(layer, T, prefill=True, stream=stream)
    _check("moe_prefill_forward", lib().moe_prefill_forward(
        layer.ref, _ptr(x), _xtype(x), T, _ptr(y), _ptr(ws), ws.numel(),
        _stream(stream)))
    return y


def moe_prefill_forward_timed(layer: MoeLayer, x, y, ws, events, stream=None):
    """events: a ctypes array of 6 hipEvent_t handles (created by the
    caller on this device), stamped with the start of the router scores, the
    end of the expert grouping, the start and end of the grouped gate/up
    product, the start of the grouped down product and the end of the
    combine."""
    _need_cuda(x)
    if events is not None and len(events) != 6:
        raise ValueError("moe_prefill_forward_timed takes 6 events")
    _check("moe_prefill_forward_timed", lib().moe_prefill_forward_timed(
        layer.ref, _ptr(x), _xtype(x), x.shape[0], _ptr(y), _ptr(ws), ws.numel(),
        _stream(stream), C.cast(events, C.c_void_p) if events is not None else None))
    return y


# ------------------------------------------------------ dense projections

class DenseMatrix:
    """A dense block-quantized matrix in its device image (rows x cols,
    format fmt), built from canonical blocks by rfpx_dense_image_build."""

    def __init__(self, fmt: int, rows: int, cols: int, canonical, stream=None):
        import torch
        _need_cuda(canonical)
        n = lib().rfpx_dense_image_bytes(fmt, rows, cols)
        if n == 0:
            raise RfpxError("rfpx_dense_image_bytes", -2, f"unsupported {rows} x {cols}")
        self.image = _new(canonical, n, torch.uint8, stream)
        _check("rfpx_dense_image_build", lib().rfpx_dense_image_build(
            fmt, _ptr(canonical), rows, cols, _ptr(self.image), n, _stream(stream)))
        self.fmt, self.rows, self.cols = fmt, rows, cols

    def unpack(self, out=None, stream=None):
        import torch
        if out is None:
            out = _new(self.image, (self.rows, self.cols), torch.float32, stream)
        _check("rfpx_dense_image_unpack", lib().rfpx_dense_image_unpack(
            self.fmt, _ptr(self.image), self.rows, self.cols, _ptr(out), _stream(stream)))
        return out

    def workspace(self, q: int, stream=None):
        import torch
        n = lib().rfpx_dense_workspace_bytes(self.fmt, self.rows, self.cols, q)
        if n == 0:
            raise RfpxError("rfpx_dense_workspace_bytes", -2, "unsupported shape")
        return _new(self.image, n, torch.uint8, stream)


def rfpx_dense_forward(m: DenseMatrix, x, y=None, ws=None, stream=None):
    """y[q][rows] = W x_c for the q columns of x (cuda bf16 or fp32
    [q][cols])."""
    import torch
    _need_cuda(x)
    q = x.shape[0]
    if y is None:
        y = _new(x, (q, m.rows), torch.float32, stream)
    if ws is None:
        ws = m.workspace(q, stream)
    _check("rfpx_dense_forward", lib().rfpx_dense_forward(
        m.fmt, _ptr(m.image), m.rows, m.cols, _ptr(x), _xtype(x), q, _ptr(y), _ptr(ws),
        ws.numel(), _stream(stream)))
    return y


# -------------------------------------------------------------- attention
#
# The step between a layer's qkv projection and its output projection, over a
# paged key/value cache in FP4 blocks (include/rfpx_attn.h).  Tensors of rows
# are [rows][heads][head_dim], heads and values adjacent, rows any multiple of
# 16 bytes apart, so that slices of one projection's output go in as they are.
# All tensors of a call live on the current device.

def _rows(what: str, t):
    """(pointer, row stride) of a tensor of rows."""
    if t.dim() != 3:
        raise ValueError(f"{what} must be [rows][heads][head_dim]")
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and h > 1):
        raise ValueError(f"{what}: heads and values must be adjacent")
    return t.data_ptr(), (s0 if n > 1 else h * d)


def _one_out(what, t, out, dtype, stream):
    """out, or a new tensor of t's shape and that dtype."""
    if out is None:
        out = _new(t, t.shape, dtype, stream)
    elif out.shape != t.shape or out.dtype != dtype:
        raise ValueError(f"{what}_out must be a {dtype} tensor of {what}'s shape")
    return out


def _same_device(torch, *ts):
    dev = torch._C._cuda_getDevice()
    for t in ts:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensor must be on the current device, cuda:{dev}")
    return dev


def _raw_stream(torch, dev, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream must be one of the current device, cuda:{dev}")
    return stream.cuda_stream


def _flat(what: str, t, dtype, shape):
    """Pointer of a contiguous tensor of that dtype and shape (None: null)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


class Rope:
    """The rotation of a head's first `dim` values (rfpx_rope): frequencies
    theta^(-2i/dim), or inv_freq (dim/2 numbers, radians a position)."""

    def __init__(self, dim: int, theta: float = 10000.0, style: int = RFPX_ROPE_HALF,
                 inv_freq: Optional[Sequence[float]] = None):
        half = max(0, dim // 2)
        if inv_freq is None:
            inv_freq = [float(theta) ** (-2.0 * i / dim) for i in range(half)]
        if len(inv_freq) != half:
            raise ValueError(f"inv_freq must hold {half} numbers")
        self._freq = (C.c_double * max(1, half))(*[float(f) for f in inv_freq])
        self.c = RopeC(dim, style, C.cast(self._freq, C.c_void_p))
        self.ref = C.byref(self.c)
        self.dim, self.style = dim, style


def rfpx_kv_pool_bytes(n_kv_heads: int, head_dim: int, page_tokens: int, n_pages: int) -> int:
    return lib().rfpx_kv_pool_bytes(n_kv_heads, head_dim, page_tokens, n_pages)


class KvCache:
    """A paged FP4 key/value cache (rfpx_kv_cache) and its pool, which is
    allocated here unless given.  Pages are numbered 0 .. n_pages-1."""

    def __init__(self, n_kv_heads: int, head_dim: int, page_tokens: int, n_pages: int, pool=None,
                 device="cuda"):
        import torch
        n = rfpx_kv_pool_bytes(n_kv_heads, head_dim, page_tokens, n_pages)
        if n == 0:
            raise RfpxError("rfpx_kv_pool_bytes", -2, "unsupported cache shape")
        if pool is None:
            pool = torch.empty(n, dtype=torch.uint8, device=device)
        _need_cuda(pool)
        self.pool = pool
        self.n_kv_heads, self.head_dim = n_kv_heads, head_dim
        self.page_tokens, self.n_pages = page_tokens, n_pages
        self.c = KvCacheC(n_kv_heads, head_dim, page_tokens, n_pages, pool.data_ptr(),
                          pool.numel() * pool.element_size())
        self.ref = C.byref(self.c)


class KvBatch:
    """A step of a batch (rfpx_kv_batch): page_table int32 [seqs][pages], lens
    int32 [seqs] with the step's columns, starts int32 [seqs + 1]; kept by
    reference, so their contents may change between calls.  max_cols and
    max_len are what launches are planned for."""

    def __init__(self, page_table, lens, starts, max_cols: int, max_len: int):
        import torch
        n, pages = page_table.shape
        _need_cuda(page_table, lens, starts)
        _flat("page_table", page_table, torch.int32, (n, pages))
        _flat("lens", lens, torch.int32, (n,))
        _flat("starts", starts, torch.int32, (n + 1,))
        # (a call looks at lens alone, for all three)
        if page_table.device != lens.device or starts.device != lens.device:
            raise ValueError("page_table, lens and starts must be on one device")
        self.page_table, self.lens, self.starts = page_table, lens, starts
        self.n_seqs, self.pages_per_seq = n, pages
        self.max_cols, self.max_len = max_cols, max_len
        self.c = KvBatchC(n, pages, max_cols, max_len, page_table.data_ptr(), lens.data_ptr(),
                          starts.data_ptr())
        self.ref = C.byref(self.c)


def _slots(cache: KvCache, batch: KvBatch):
    return (batch.n_seqs, cache.n_kv_heads, batch.pages_per_seq * cache.page_tokens)


def rfpx_qk_norm_rope(q, k, positions, q_weight=None, k_weight=None, eps: float = 1e-6,
                      rope: Optional[Rope] = None, q_out=None, k_out=None, out_dtype=None,
                      stream=None):
    """RMS norm (where a weight, fp32 [head_dim], is given) and rotation of
    the heads of q and k (either may be None); positions int32 [rows], negative
    for padding rows, which are left as they were.  Returns (q_out, k_out)."""
    import torch
    x = q if q is not None else k
    if x is None:
        raise ValueError("q or k is needed")
    n, _, d = x.shape
    dtype = out_dtype
    if dtype is None:
        given = q_out if q_out is not None else k_out
        dtype = x.dtype if given is None else given.dtype
    qp = qs = qh = qo = qos = kp = ks = kh = ko = kos = 0
    if q is not None:
        q_out = _one_out("q", q, q_out, dtype, stream)
        (qp, qs), (qo, qos), qh = _rows("q", q), _rows("q_out", q_out), q.shape[1]
    if k is not None:
        if k is not x and (k.shape[0] != n or k.shape[2] != d or k.dtype != x.dtype):
            raise ValueError("q and k must agree in rows, head_dim and dtype")
        k_out = _one_out("k", k, k_out, dtype, stream)
        (kp, ks), (ko, kos), kh = _rows("k", k), _rows("k_out", k_out), k.shape[1]
    dev = _same_device(torch, q, k, positions, q_weight, k_weight, q_out, k_out)
    _check("rfpx_qk_norm_rope", lib().rfpx_qk_norm_rope(
        qp, qs, qh, kp, ks, kh, d, _xtype(x), n, _flat("positions", positions, torch.int32, (n,)),
        _flat("q_weight", q_weight, torch.float32, (d,)),
        _flat("k_weight", k_weight, torch.float32, (d,)), eps,
        None if rope is None else rope.ref, qo, qos, ko, kos,
        _xtype(k_out if q is None else q_out), _raw_stream(torch, dev, stream)))
    return (None if q is None else q_out), (None if k is None else k_out)


def rfpx_kv_append(cache: KvCache, batch: KvBatch, k, v, positions=None, pos=None, acc=None,
                   stream=None) -> None:
    """Quantize the step's k and v into the cache; pos (int32) and acc (fp32),
    [seqs][kv heads][slots], get positions[row] and 0 at the new slots."""
    import torch
    dev = _same_device(torch, cache.pool, batch.lens, k, v, positions, pos, acc)
    shape = (k.shape[0], cache.n_kv_heads, cache.head_dim)
    if tuple(k.shape) != shape or tuple(v.shape) != shape or k.dtype != v.dtype:
        raise ValueError(f"k and v must be {shape} tensors of one dtype")
    kp, ks = _rows("k", k)
    vp, vs = _rows("v", v)
    slots = _slots(cache, batch)
    _check("rfpx_kv_append", lib().rfpx_kv_append(
        cache.ref, batch.ref, kp, ks, vp, vs, _xtype(k), k.shape[0],
        _flat("positions", positions, torch.int32, (k.shape[0],)),
        _flat("pos", pos, torch.int32, slots), _flat("acc", acc, torch.float32, slots),
        _raw_stream(torch, dev, stream)))


def rfpx_kv_unpack(cache: KvCache, batch: KvBatch, rows: int, k=None, v=None, stream=None):
    """What the cache holds for the step's columns: (k, v) [rows][kv heads]
    [head_dim], fp32 unless bf16 tensors are given."""
    import torch
    shape = (rows, cache.n_kv_heads, cache.head_dim)
    if k is None:
        k = _new(cache.pool, shape, torch.float32, stream)
    if v is None:
        v = _new(cache.pool, shape, k.dtype, stream)
    dev = _same_device(torch, cache.pool, batch.lens, k, v)
    _check("rfpx_kv_unpack", lib().rfpx_kv_unpack(
        cache.ref, batch.ref, rows, _flat("k", k, k.dtype, shape), _flat("v", v, k.dtype, shape),
        _xtype(k), _raw_stream(torch, dev, stream)))
    return k, v


def rfpx_attn_workspace_bytes(cache: KvCache, batch: KvBatch, heads: int, rows: int) -> int:
    return lib().rfpx_attn_workspace_bytes(cache.ref, batch.ref, heads, rows)


def rfpx_attn_forward(cache: KvCache, batch: KvBatch, q, scale: Optional[float] = None, out=None,
                      lse=None, ws=None, stream=None):
    """Attention of the step's columns q [rows][heads][head_dim] (fp32 or
    bf16) over the cache; scale defaults to head_dim^-0.5.  lse (fp32 [rows]
    [heads]), if given, gets the log of every row's sum of exponentials."""
    import torch
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError(f"q must be [rows][heads][{cache.head_dim}]")
    rows, heads, d = q.shape
    if out is None:
        out = _new(q, q.shape, q.dtype, stream)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and dtype")
    if ws is None:
        n = rfpx_attn_workspace_bytes(cache, batch, heads, rows)
        if n == 0:
            raise RfpxError("rfpx_attn_workspace_bytes", -2, lib().rfpx_last_error().decode())
        ws = _new(q, n, torch.uint8, stream)
    dev = _same_device(torch, cache.pool, batch.lens, q, out, lse, ws)
    qp, qs = _rows("q", q)
    op, os_ = _rows("out", out)
    _check("rfpx_attn_forward", lib().rfpx_attn_forward(
        cache.ref, batch.ref, qp, qs, _xtype(q), heads, rows,
        d ** -0.5 if scale is None else scale, op, os_,
        _flat("lse", lse, torch.float32, (rows, heads)), ws.data_ptr(),
        ws.numel() * ws.element_size(), _raw_stream(torch, dev, stream)))
    return out


def rfpx_attn_weights(cache: KvCache, batch: KvBatch, q, lse, acc, decay: float = 1.0,
                      scale: Optional[float] = None, acc_out=None, stream=None):
    """acc_out = decay * acc + the attention weight that every slot receives
    from the step's columns (acc fp32 [seqs][kv heads][slots]; in place unless
    acc_out is given); q, scale and lse as in rfpx_attn_forward."""
    import torch
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError(f"q must be [rows][heads][{cache.head_dim}]")
    rows, heads, d = q.shape
    if acc_out is None:
        acc_out = acc
    dev = _same_device(torch, cache.pool, batch.lens, q, lse, acc, acc_out)
    slots = _slots(cache, batch)
    qp, qs = _rows("q", q)
    _check("rfpx_attn_weights", lib().rfpx_attn_weights(
        cache.ref, batch.ref, qp, qs, _xtype(q), heads, rows, d ** -0.5 if scale is None else scale,
        _flat("lse", lse, torch.float32, (rows, heads)), decay,
        _flat("acc", acc, torch.float32, slots), _flat("acc_out", acc_out, torch.float32, slots),
        _raw_stream(torch, dev, stream)))
    return acc_out


def rfpx_kv_evict_workspace_bytes(cache: KvCache, batch: KvBatch, keep: int) -> int:
    return lib().rfpx_kv_evict_workspace_bytes(cache.ref, batch.ref, keep)


def rfpx_kv_evict(cache: KvCache, batch: KvBatch, keep: int, recent: int, acc, pos, acc_out=None,
                  pos_out=None, lens_out=None, ws=None, stream=None):
    """Cut every sequence to its `keep` best slots: the `recent` newest by pos
    first, then those of largest acc.  acc, pos and the batch's lens are
    updated in place unless outputs are given.  Returns (acc, pos, lens)."""
    import torch
    acc_out = acc if acc_out is None else acc_out
    pos_out = pos if pos_out is None else pos_out
    lens_out = batch.lens if lens_out is None else lens_out
    if ws is None:
        n = rfpx_kv_evict_workspace_bytes(cache, batch, keep)
        if n == 0:
            raise RfpxError("rfpx_kv_evict_workspace_bytes", -2, lib().rfpx_last_error().decode())
        ws = _new(cache.pool, n, torch.uint8, stream)
    dev = _same_device(torch, cache.pool, batch.lens, acc, pos, acc_out, pos_out, lens_out, ws)
    slots = _slots(cache, batch)
    _check("rfpx_kv_evict", lib().rfpx_kv_evict(
        cache.ref, batch.ref, keep, recent, _flat("acc", acc, torch.float32, slots),
        _flat("pos", pos, torch.int32, slots), _flat("acc_out", acc_out, torch.float32, slots),
        _flat("pos_out", pos_out, torch.int32, slots),
        _flat("lens_out", lens_out, torch.int32, (batch.n_seqs,)), ws.data_ptr(),
        ws.numel() * ws.element_size(), _raw_stream(torch, dev, stream)))
    return acc_out, pos_out, lens_out


# ------------------------------------------------------------ measurement

def rfpx_stream_read(buf, sink=None, stream=None):
    """A plain streaming read of the cuda tensor buf (its bytes); returns the
    sink tensor (int32 [rfpx_stream_read_sink_words()]), whose words XOR to
    the XOR of buf's 32-bit words (words past the workgroup count are left
    as they were: pass a zeroed sink to check)."""
    import torch
    _need_cuda(buf)
    n = lib().rfpx_stream_read_sink_words()
    if sink is None:
        sink = _new(buf, n, torch.int32, stream)
        with torch.cuda.stream(stream):  # (None: the current one)
            sink.zero_()
    _check("rfpx_stream_read", lib().rfpx_stream_read(
        _ptr(buf), buf.numel() * buf.element_size(), _ptr(sink), _stream(stream)))
    return sink


# ----------------------------------------------------------- convenience

def upload_layer(lay, device="cuda", stream=None, validate: bool = True) -> MoeLayer:
    """Build the device image of a synthetic layer (an object with d, f, E,
    k, wr, fmts, blob, offsets, mat(e, m)): one host-to-device copy of all
    canonical bytes, then moe_image_build on the GPU, then (by default)
    moe_image_validate, raising if the image fails it."""
    import numpy as np
    import torch
    blob = torch.from_numpy(np.ascontiguousarray(lay.blob)).to(device)
    canon = []
    for e in range(lay.E + 1):
        for m in range(3):
            i = 3 * e + m
            n = lay.mat(e, m).size
            canon.append(blob[int(lay.offsets[i]):int(lay.offsets[i]) + n])
    image = moe_image_build(lay.d, lay.f, lay.E, lay.fmts, canon, stream=stream)
    wr = torch.from_numpy(np.ascontiguousarray(lay.wr)).to(device)
    L = MoeLayer(lay.d, lay.f, lay.E, lay.k, wr, image, lay.fmts,
                 getattr(lay, "routed_scale", 1.0))
    if validate:
        check_image(L, stream)  # waits for the stream, so the canonical bytes may go
    else:
        (stream or torch.cuda.current_stream()).synchronize()
    del blob, canon
    return L
