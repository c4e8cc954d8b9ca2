"""Python binding of the microscaling-quantized convolution library (libmq.so, gfx950).

Argument marshalling only: every step of the hot path runs in the library's HIP kernels. torch
supplies device memory and the current stream. The functions keep the C ABI's names
(``include/mq.h``) and raise :class:`MQError` on a non-OK status. If the library is not built
this module raises on import: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence, Tuple, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmq.so")

MQ_OK, MQ_ERR_ARG, MQ_ERR_SHAPE, MQ_ERR_UNSUPPORTED, MQ_ERR_WORKSPACE, MQ_ERR_LAUNCH = range(6)
MQ_NVFP4, MQ_NVFP6 = 4, 6
MQ_ROLE_ACT, MQ_ROLE_WEIGHT, MQ_ROLE_GRAD = 0, 1, 2
MQ_RNE, MQ_SR = 0, 1
MQ_QUANTIZE_WS_BYTES = 8192  # tensor-amax workspace (mq_quantize, relayouts)
MQ_QUANTIZE_AMAX_READY = 1   # mq_quantize flag: the workspace already holds this tensor's amax
MQ_SRC_DENSE, MQ_SRC_NCHW, MQ_SRC_OIHW = 0, 1, 2  # mq_quant_job.layout
MQ_QUANTIZE_BATCH_MAX = 4
MQ_NOALLOC_SCRATCH_BYTES = 32 << 20  # library-owned split-K scratch of mq_conv_backward_noalloc
MQ_F16, MQ_BF16 = 1, 2  # mq_dtype: element type of the attention calls
MQ_KV_BLOCK = 16        # tokens that share one scale of the key/value cache

EXPORTS = (
    "mq_status_str", "mq_codes_bytes", "mq_scales_bytes", "mq_relayout_cbf",
    "mq_relayout_weight", "mq_quantize", "mq_quantize_nchw", "mq_quantize_batch",
    "mq_quantize_weight", "mq_conv_fwd",
    "mq_wgrad_workspace_bytes",
    "mq_conv_wgrad", "mq_conv_dgrad", "mq_conv_backward", "mq_conv_backward_noalloc",
    "mq_conv_fwd_amax", "mq_conv_backward_amax",
    "mq_kv_append", "mq_attn_cached_workspace_bytes", "mq_attn_cached", "mq_attn_prompt",
    "mq_kv_evict",
)


class MQError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_lib.mq_status_str(status).decode()}")
        self.status = status


class mq_qtensor(ctypes.Structure):
    _fields_ = [("o0", ctypes.c_int32), ("o1", ctypes.c_int32), ("r", ctypes.c_int32),
                ("s", ctypes.c_int32), ("fmt", ctypes.c_int32), ("role", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tscale", ctypes.c_void_p)]


class mq_quant_job(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("layout", ctypes.c_int32), ("rnd", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("flags", ctypes.c_uint32), ("dst", mq_qtensor),
                ("amax_ws", ctypes.c_void_p), ("amax_ws_bytes", ctypes.c_size_t)]


class mq_conv(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "Cin", "H", "W", "Cout", "Kh", "Kw",
                                              "stride_h", "stride_w", "pad_h", "pad_w")]


class mq_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("tokens", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class mq_kv_cache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() or "
                          f"python microscaling_quantized_convolution_amd/_build.py")
    L = ctypes.CDLL(LIB_PATH)
    P, i32, u64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint64, ctypes.c_size_t
    L.mq_status_str.restype = ctypes.c_char_p
    L.mq_status_str.argtypes = [ctypes.c_int]
    L.mq_codes_bytes.restype = sz
    L.mq_codes_bytes.argtypes = [i32] * 5
    L.mq_scales_bytes.restype = sz
    L.mq_scales_bytes.argtypes = [i32] * 4
    L.mq_relayout_cbf.argtypes = [P, P, i32, i32, i32, i32, i32, P, sz, P]
    L.mq_relayout_weight.argtypes = [P, P, i32, i32, i32, i32, i32, P, sz, P]
    L.mq_quantize.argtypes = [P, ctypes.POINTER(mq_qtensor), i32, u64, P, sz, ctypes.c_uint32, P]
    L.mq_quantize_nchw.argtypes = [P, ctypes.POINTER(mq_qtensor), i32, u64, P, sz,
                                   ctypes.c_uint32, P]
    L.mq_quantize_weight.argtypes = [P, ctypes.POINTER(mq_qtensor), i32, u64, P, sz, P]
    L.mq_quantize_batch.argtypes = [ctypes.POINTER(mq_quant_job), i32, P]
    L.mq_conv_fwd.argtypes = [ctypes.POINTER(mq_conv), ctypes.POINTER(mq_qtensor),
                              ctypes.POINTER(mq_qtensor), P, P]
    L.mq_wgrad_workspace_bytes.restype = sz
    L.mq_wgrad_workspace_bytes.argtypes = [ctypes.POINTER(mq_conv)]
    L.mq_conv_wgrad.argtypes = [ctypes.POINTER(mq_conv), ctypes.POINTER(mq_qtensor),
                                ctypes.POINTER(mq_qtensor), P, P, sz, P]
    L.mq_conv_dgrad.argtypes = [ctypes.POINTER(mq_conv), ctypes.POINTER(mq_qtensor),
                                ctypes.POINTER(mq_qtensor), P, P]
    L.mq_conv_backward.argtypes = [ctypes.POINTER(mq_conv), ctypes.POINTER(mq_qtensor),
                                   ctypes.POINTER(mq_qtensor), ctypes.POINTER(mq_qtensor), P, P,
                                   P, sz, P]
    L.mq_conv_backward_noalloc.argtypes = [ctypes.POINTER(mq_conv), ctypes.POINTER(mq_qtensor),
                                           ctypes.POINTER(mq_qtensor), ctypes.POINTER(mq_qtensor),
                                           P, P, P]
    L.mq_conv_fwd_amax.argtypes = [ctypes.POINTER(mq_conv), ctypes.POINTER(mq_qtensor),
                                   ctypes.POINTER(mq_qtensor), P, P, sz, P]
    L.mq_conv_backward_amax.argtypes = [ctypes.POINTER(mq_conv), ctypes.POINTER(mq_qtensor),
                                        ctypes.POINTER(mq_qtensor), ctypes.POINTER(mq_qtensor),
                                        P, P, P, sz, P, sz, P]
    R, C, f32 = ctypes.POINTER(mq_rows), ctypes.POINTER(mq_kv_cache), ctypes.c_float
    L.mq_kv_append.argtypes = [C, R, R, P, P, P, i32, i32, P]
    L.mq_attn_cached_workspace_bytes.restype = sz
    L.mq_attn_cached_workspace_bytes.argtypes = [i32] * 7
    L.mq_attn_cached.argtypes = [C, R, R, P, P, i32, i32, i32, i32, f32, P, P, sz, P]
    L.mq_attn_prompt.argtypes = [R, R, R, R, P, i32, i32, f32, P]
    L.mq_kv_evict.argtypes = [C, P, P, P, P, P, P, i32, i32, i32, i32, i32, P]
    for name in EXPORTS:
        getattr(L, name).restype = getattr(L, name).restype or ctypes.c_int
    return L


_lib = _load()


def lib() -> ctypes.CDLL:
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(st: int, where: str):
    if st != MQ_OK:
        raise MQError(st, where)


ConvLike = Union[mq_conv, Sequence[int]]


def conv_struct(p: ConvLike) -> mq_conv:
    """(N, Cin, H, W, Cout, Kh, Kw, stride_h, stride_w, pad_h, pad_w) -> mq_conv."""
    return p if isinstance(p, mq_conv) else mq_conv(*[int(v) for v in p])


class QTensor:
    """Device buffers of one quantized tensor (codes, scales, tensor scale) and its shape."""

    def __init__(self, o0: int, o1: int, r: int, s: int, fmt: int, role: int,
                 device: Union[str, torch.device] = "cuda"):
        self.shape = (int(o0), int(o1), int(r), int(s))
        self.fmt, self.role = int(fmt), int(role)
        nc = _lib.mq_codes_bytes(*self.shape, self.fmt)
        ns = _lib.mq_scales_bytes(*self.shape)
        if nc == 0 or ns == 0:
            raise MQError(MQ_ERR_ARG, "QTensor")
        self.codes = torch.empty(nc, dtype=torch.uint8, device=device)
        self.scales = torch.empty(ns, dtype=torch.uint8, device=device)
        self.tscale = torch.empty(1, dtype=torch.float32, device=device)

    def struct(self) -> mq_qtensor:
        return mq_qtensor(*self.shape, self.fmt, self.role, self.codes.data_ptr(),
                          self.scales.data_ptr(), self.tscale.data_ptr())


def mq_codes_bytes(o0, o1, r, s, fmt) -> int:
    return int(_lib.mq_codes_bytes(o0, o1, r, s, fmt))


def mq_scales_bytes(o0, o1, r, s) -> int:
    return int(_lib.mq_scales_bytes(o0, o1, r, s))


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def mq_relayout_cbf(src: torch.Tensor, dst: torch.Tensor, N: int, C: int, H: int, W: int,
                    inverse: int = 0, amax_ws: Optional[torch.Tensor] = None, stream=None):
    _check(_lib.mq_relayout_cbf(_ptr(src), _ptr(dst), N, C, H, W, inverse, _ptr(amax_ws),
                                _nbytes(amax_ws), _stream(stream)), "mq_relayout_cbf")


def mq_relayout_weight(src: torch.Tensor, dst: torch.Tensor, Cout: int, Cin: int, Kh: int,
                       Kw: int, inverse: int = 0, amax_ws: Optional[torch.Tensor] = None,
                       stream=None):
    _check(_lib.mq_relayout_weight(_ptr(src), _ptr(dst), Cout, Cin, Kh, Kw, inverse,
                                   _ptr(amax_ws), _nbytes(amax_ws), _stream(stream)),
           "mq_relayout_weight")


def quantize_workspace(device: Union[str, torch.device] = "cuda") -> torch.Tensor:
    """Device scratch for mq_quantize's amax pass."""
    return torch.empty(MQ_QUANTIZE_WS_BYTES, dtype=torch.uint8, device=device)


def mq_quantize(src: torch.Tensor, dst: QTensor, rnd: int, seed: int, amax_ws: torch.Tensor,
                flags: int = 0, stream=None):
    q = dst.struct()
    _check(_lib.mq_quantize(_ptr(src), ctypes.byref(q), rnd, seed & (2 ** 64 - 1),
                            _ptr(amax_ws), _nbytes(amax_ws), flags, _stream(stream)),
           "mq_quantize")


def mq_quantize_nchw(src_nchw: torch.Tensor, dst: QTensor, rnd: int, seed: int,
                     amax_ws: torch.Tensor, flags: int = 0, stream=None):
    """NCHW fp32 activation / gradient -> quantized channel-batch-first tensor (same result as
    mq_relayout_cbf then mq_quantize, without the fp32 copy)."""
    q = dst.struct()
    _check(_lib.mq_quantize_nchw(_ptr(src_nchw), ctypes.byref(q), rnd, seed & (2 ** 64 - 1),
                                 _ptr(amax_ws), _nbytes(amax_ws), flags, _stream(stream)),
           "mq_quantize_nchw")


def quant_job(src: torch.Tensor, layout: int, dst: QTensor, rnd: int, seed: int,
              amax_ws: torch.Tensor, flags: int = 0) -> mq_quant_job:
    """One mq_quant_job (the caller keeps src, dst and amax_ws alive until the call is done)."""
    return mq_quant_job(ctypes.c_void_p(src.data_ptr()), layout, rnd, seed & (2 ** 64 - 1), flags,
                        dst.struct(), ctypes.c_void_p(amax_ws.data_ptr()), _nbytes(amax_ws))


def mq_quantize_batch(jobs: Sequence[mq_quant_job], stream=None):
    """Several tensors in one amax launch and one quantizing launch (see quant_job)."""
    arr = (mq_quant_job * len(jobs))(*jobs)
    _check(_lib.mq_quantize_batch(arr, len(jobs), _stream(stream)), "mq_quantize_batch")


def mq_quantize_weight(w_oihw: torch.Tensor, dst: QTensor, rnd: int, seed: int,
                       amax_ws: torch.Tensor, stream=None):
    """OIHW fp32 weight -> quantized tap-major weight (same result as mq_relayout_weight then
    mq_quantize, without the fp32 copy)."""
    q = dst.struct()
    _check(_lib.mq_quantize_weight(_ptr(w_oihw), ctypes.byref(q), rnd, seed & (2 ** 64 - 1),
                                   _ptr(amax_ws), _nbytes(amax_ws), _stream(stream)),
           "mq_quantize_weight")


def mq_conv_fwd(p: ConvLike, x: QTensor, w: QTensor, y: torch.Tensor, stream=None):
    c, qx, qw = conv_struct(p), x.struct(), w.struct()
    _check(_lib.mq_conv_fwd(ctypes.byref(c), ctypes.byref(qx), ctypes.byref(qw), _ptr(y),
                            _stream(stream)), "mq_conv_fwd")


def mq_wgrad_workspace_bytes(p: ConvLike) -> int:
    c = conv_struct(p)
    return int(_lib.mq_wgrad_workspace_bytes(ctypes.byref(c)))


def mq_conv_wgrad(p: ConvLike, gy: QTensor, x: QTensor, gw: torch.Tensor,
                  ws: Optional[torch.Tensor], stream=None):
    c, qg, qx = conv_struct(p), gy.struct(), x.struct()
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(_lib.mq_conv_wgrad(ctypes.byref(c), ctypes.byref(qg), ctypes.byref(qx), _ptr(gw),
                              _ptr(ws), nbytes, _stream(stream)), "mq_conv_wgrad")


def mq_conv_dgrad(p: ConvLike, w: QTensor, gy: QTensor, gx: torch.Tensor, stream=None):
    c, qw, qg = conv_struct(p), w.struct(), gy.struct()
    _check(_lib.mq_conv_dgrad(ctypes.byref(c), ctypes.byref(qw), ctypes.byref(qg), _ptr(gx),
                              _stream(stream)), "mq_conv_dgrad")


def mq_conv_backward(p: ConvLike, w: QTensor, gy: QTensor, x: QTensor, gw: torch.Tensor,
                     gx: torch.Tensor, ws: torch.Tensor, stream=None):
    """Both gradients (G_W as mq_conv_wgrad, G_X as mq_conv_dgrad) in one call."""
    c, qw, qg, qx = conv_struct(p), w.struct(), gy.struct(), x.struct()
    _check(_lib.mq_conv_backward(ctypes.byref(c), ctypes.byref(qw), ctypes.byref(qg),
                                 ctypes.byref(qx), _ptr(gw), _ptr(gx), _ptr(ws), _nbytes(ws),
                                 _stream(stream)), "mq_conv_backward")


def mq_conv_backward_noalloc(p: ConvLike, w: QTensor, gy: QTensor, x: QTensor,
                             gw: torch.Tensor, gx: torch.Tensor, stream=None):
    """mq_conv_backward without a workspace argument: the split-K partials live in the
    library's own device array (for callers that cannot allocate)."""
    c, qw, qg, qx = conv_struct(p), w.struct(), gy.struct(), x.struct()
    _check(_lib.mq_conv_backward_noalloc(ctypes.byref(c), ctypes.byref(qw), ctypes.byref(qg),
                                         ctypes.byref(qx), _ptr(gw), _ptr(gx), _stream(stream)),
           "mq_conv_backward_noalloc")


def mq_conv_fwd_amax(p: ConvLike, x: QTensor, w: QTensor, y: torch.Tensor,
                     amax_ws: torch.Tensor, stream=None):
    """mq_conv_fwd, plus the partial maxima of |Y| in amax_ws (for MQ_QUANTIZE_AMAX_READY)."""
    c, qx, qw = conv_struct(p), x.struct(), w.struct()
    _check(_lib.mq_conv_fwd_amax(ctypes.byref(c), ctypes.byref(qx), ctypes.byref(qw), _ptr(y),
                                 _ptr(amax_ws), _nbytes(amax_ws), _stream(stream)),
           "mq_conv_fwd_amax")


def mq_conv_backward_amax(p: ConvLike, w: QTensor, gy: QTensor, x: QTensor, gw: torch.Tensor,
                          gx: torch.Tensor, ws: torch.Tensor, gx_amax_ws: torch.Tensor,
                          stream=None):
    """mq_conv_backward, plus the partial maxima of |G_X| in gx_amax_ws."""
    c, qw, qg, qx = conv_struct(p), w.struct(), gy.struct(), x.struct()
    _check(_lib.mq_conv_backward_amax(ctypes.byref(c), ctypes.byref(qw), ctypes.byref(qg),
                                      ctypes.byref(qx), _ptr(gw), _ptr(gx), _ptr(ws), _nbytes(ws),
                                      _ptr(gx_amax_ws), _nbytes(gx_amax_ws), _stream(stream)),
           "mq_conv_backward_amax")


def out_hw(p: ConvLike) -> Tuple[int, int]:
    c = conv_struct(p)
    return ((c.H + 2 * c.pad_h - c.Kh) // c.stride_h + 1,
            (c.W + 2 * c.pad_w - c.Kw) // c.stride_w + 1)


# ---- attention over an 8-bit key/value cache ---------------------------------------------------
#
# These calls are made once per layer and token, so their marshalling is kept short (a few
# attribute reads a tensor): checks that the library cannot make itself, types, contiguity and
# device, then one foreign call.

_DTYPES = {torch.float16: MQ_F16, torch.bfloat16: MQ_BF16}
if torch.version.hip:
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _rows(t: torch.Tensor, what: str, device: int) -> mq_rows:
    """[tokens][heads][dim] view with a contiguous last dimension -> mq_rows."""
    dt, strides = _DTYPES.get(t.dtype), t.stride()
    if dt is None or len(strides) != 3 or strides[2] != 1 or t.get_device() != device:
        raise ValueError(f"{what}: expected a float16 or bfloat16 tensor [tokens][heads][dim] with "
                         f"contiguous elements on cuda:{device} (the current device), got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}, strides {strides}")
    n, h, d = t.shape
    return mq_rows(t.data_ptr(), strides[0], strides[1], n, h, d, dt)


def _dense(t: torch.Tensor, dtype: torch.dtype, shape, what: str, device: int) -> int:
    """Address of a contiguous tensor of that type and shape on that device."""
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or
            t.get_device() != device):
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor {tuple(shape)} on "
                         f"cuda:{device} (the current device), got {tuple(t.shape)} {t.dtype} on "
                         f"{t.device}, strides {t.stride()}")
    return t.data_ptr()


def _ints(t: torch.Tensor, what: str, device: int) -> Tuple[int, int]:
    """Address and length of an int32 vector."""
    shape = t.shape
    if len(shape) != 1:
        raise ValueError(f"{what}: expected one dimension, got {tuple(shape)}")
    return _dense(t, torch.int32, shape, what, device), shape[0]


def _table(table: torch.Tensor, n: int, device: int) -> Tuple[int, int]:
    """Address and width of a page table of n rows."""
    shape = table.shape
    if len(shape) != 2 or shape[0] != n:
        raise ValueError(f"table: expected [{n} sequences][pages], got {tuple(shape)}")
    return _dense(table, torch.int32, shape, "table", device), shape[1]


class KVCache:
    """A paged key/value cache in 8 bits (mq_kv_cache; the layouts are in include/mq.h).

    Made from its four uint8 tensors, k_codes [pages][heads][page_size][dim],
    v_codes [pages][heads][page_size / 16][dim][16], k_scales and v_scales
    [pages][heads][page_size / 16], or by :meth:`empty`."""

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor):
        if k_codes.dim() != 4 or k_codes.shape[2] % MQ_KV_BLOCK:
            raise ValueError(f"k_codes: expected [pages][heads][page_size][dim] with page_size a "
                             f"multiple of {MQ_KV_BLOCK}, got {tuple(k_codes.shape)}")
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k_codes.shape
        blocks = (self.num_pages, self.kv_heads, self.page_size // MQ_KV_BLOCK)
        dev = k_codes.get_device()
        self.device = k_codes.device
        self.k_codes, self.v_codes = k_codes, v_codes
        self.k_scales, self.v_scales = k_scales, v_scales
        u8 = torch.uint8
        self.struct = mq_kv_cache(
            self.num_pages, self.page_size, self.kv_heads, self.head_dim,
            _dense(k_codes, u8, k_codes.shape, "k_codes", dev),
            _dense(v_codes, u8, blocks + (self.head_dim, MQ_KV_BLOCK), "v_codes", dev),
            _dense(k_scales, u8, blocks, "k_scales", dev), _dense(v_scales, u8, blocks, "v_scales", dev))
        self._ref, self._dev = ctypes.byref(self.struct), dev
        self.weights_shape = torch.Size((self.num_pages, self.kv_heads, self.page_size))

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
              device: Union[str, torch.device] = "cuda") -> "KVCache":
        """A cache that holds nothing yet (its memory is not cleared: mq_kv_append writes whole
        blocks)."""
        new = lambda *shape: torch.empty(shape, dtype=torch.uint8, device=device)
        blocks = (num_pages, kv_heads, page_size // MQ_KV_BLOCK)
        return cls(new(num_pages, kv_heads, page_size, head_dim),
                   new(*blocks, head_dim, MQ_KV_BLOCK), new(*blocks), new(*blocks))

    def ref(self, device: int):
        """The structure, for a call on that device."""
        if device != self._dev:
            raise ValueError(f"cache on {self.device}, but the current device is cuda:{device}")
        return self._ref

    def values(self) -> Tuple[torch.Tensor, torch.Tensor]:
        """Keys and values as fp32 [pages][heads][page_size][dim] (for inspection: every slot is
        decoded, also those that hold no token)."""
        out = []
        for codes, scales in ((self.k_codes.view(*self.k_scales.shape, MQ_KV_BLOCK, -1),
                               self.k_scales), (self.v_codes.transpose(3, 4), self.v_scales)):
            e = scales.to(torch.int32)
            f = torch.where(e == 255, torch.nan, torch.ldexp(torch.ones_like(e, dtype=torch.float32),
                                                             e - 127))
            out.append((codes.view(torch.float8_e4m3fn).float() * f[..., None, None])
                       .reshape(self.k_codes.shape))
        return out[0], out[1]


def mq_kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, table: torch.Tensor,
                 lens: torch.Tensor, cu: torch.Tensor, stream=None):
    """Quantize the packed keys and values k, v [tokens][kv_heads][dim] into the cache behind each
    sequence's lens[s] tokens: sequence s receives rows cu[s]:cu[s + 1]. lens is not changed."""
    dev = _current_device()
    pl, n = _ints(lens, "lens", dev)
    pt, width = _table(table, n, dev)
    st = _lib.mq_kv_append(cache.ref(dev), _rows(k, "k", dev), _rows(v, "v", dev), pt, pl,
                           _dense(cu, torch.int32, (n + 1,), "cu", dev), n, width,
                           _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise MQError(st, "mq_kv_append")


def mq_attn_cached_workspace_bytes(n_seqs: int, q_heads: int, kv_heads: int, head_dim: int,
                                   q_len: int, max_len: int, weights: bool = False) -> int:
    return int(_lib.mq_attn_cached_workspace_bytes(n_seqs, q_heads, kv_heads, head_dim, q_len,
                                                   max_len, int(weights)))


def attn_cached_workspace(n_seqs: int, q_heads: int, kv_heads: int, head_dim: int, q_len: int,
                          max_len: int, weights: bool = False,
                          device: Union[str, torch.device] = "cuda") -> torch.Tensor:
    """Device scratch for mq_attn_cached calls of these sizes."""
    return torch.empty(mq_attn_cached_workspace_bytes(n_seqs, q_heads, kv_heads, head_dim, q_len,
                                                      max_len, weights),
                       dtype=torch.uint8, device=device)


def mq_attn_cached(q: torch.Tensor, cache: KVCache, table: torch.Tensor, lens: torch.Tensor,
                   out: torch.Tensor, ws: Optional[torch.Tensor], scale: float, q_len: int = 1,
                   max_len: int = 0, weights: Optional[torch.Tensor] = None, stream=None):
    """Attention of each sequence's last q_len tokens, q [sequences * q_len][q_heads][dim], over
    its lens[s] cached tokens (these included), into out. weights (fp32, cache.weights_shape)
    gains the attention each cached token received, from every sequence that reads its page."""
    dev = _current_device()
    pl, n = _ints(lens, "lens", dev)
    pt, width = _table(table, n, dev)
    pw = (None if weights is None
          else _dense(weights, torch.float32, cache.weights_shape, "weights", dev))
    st = _lib.mq_attn_cached(cache.ref(dev), _rows(q, "q", dev), _rows(out, "out", dev), pt,
                             pl, n, width, q_len, max_len, scale, pw,
                             None if ws is None else _dense(ws, torch.uint8, ws.shape, "ws", dev),
                             0 if ws is None else ws.numel(),
                             _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise MQError(st, "mq_attn_cached")


def mq_attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                   cu: torch.Tensor, max_len: int, scale: float, stream=None):
    """Causal attention over packed prompts: rows cu[s]:cu[s + 1] of q, out [tokens][q_heads][dim]
    and k, v [tokens][kv_heads][dim] are sequence s, none longer than max_len."""
    dev = _current_device()
    pc, n = _ints(cu, "cu", dev)
    st = _lib.mq_attn_prompt(_rows(q, "q", dev), _rows(k, "k", dev), _rows(v, "v", dev),
                             _rows(out, "out", dev), pc, n - 1, max_len, scale,
                             _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise MQError(st, "mq_attn_prompt")


def mq_kv_evict(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, weights: torch.Tensor,
                new_table: torch.Tensor, new_lens: torch.Tensor, kept: torch.Tensor, recent: int,
                stream=None):
    """Keep at most kept.shape[2] tokens of each sequence and head, the `recent` last ones and those
    with the largest weights, copied to the pages of new_table; kept [sequences][kv_heads][keep]
    receives their former positions, new_lens the sequences' new lengths."""
    dev = _current_device()
    i32, keep = torch.int32, kept.shape[-1]
    pl, n = _ints(lens, "lens", dev)
    pt, width = _table(table, n, dev)
    pn, new_width = _table(new_table, n, dev)
    st = _lib.mq_kv_evict(cache.ref(dev),
                          _dense(weights, torch.float32, cache.weights_shape, "weights", dev), pt, pl, pn,
                          _dense(new_lens, i32, (n,), "new_lens", dev),
                          _dense(kept, i32, (n, cache.kv_heads, keep), "kept", dev), n, width,
                          new_width, keep, recent,
                          _raw_stream(dev) if stream is None else _stream(stream))
    if st:
        raise MQError(st, "mq_kv_evict")
