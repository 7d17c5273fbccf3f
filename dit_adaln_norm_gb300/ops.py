"""Thin ctypes binding of libdan.so (include/dan.h, include/dan_cache.h and
include/dan_train.h): argument marshalling only.

Every function takes CUDA torch tensors (bf16; the group norm also fp16 and
fp32), checks the layout the C ABI
expects, passes raw pointers, strides and the current CUDA stream, and turns
a non-zero status into an exception.  All arithmetic runs in the CUDA
kernels; there is no CPU or eager fallback.  PyTorch only allocates outputs.

The library is loaded on first use.  If it is missing the call raises
(build it with ``python -c "import __graft_entry__ as g; g.build()"``).
"""
from __future__ import annotations

import ctypes
import functools
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdan.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "dan.h")
CACHE_HEADER = os.path.join(os.path.dirname(HERE), "include", "dan_cache.h")
TRAIN_HEADER = os.path.join(os.path.dirname(HERE), "include", "dan_train.h")

DAN_OK, DAN_EINVAL, DAN_EUNSUPPORTED, DAN_EALIGN, DAN_EALIAS, DAN_ECUDA = range(6)

_P = ctypes.c_void_p
_I = ctypes.c_int64
_F = ctypes.c_float
_N = ctypes.c_int
_SIGS = {
    "dan_rms_modulate": [_P, _P, _P, _P, _I, _P, _I, _I, _I, _F, _P],
    "dan_rms_modulate_noalloc": [_P, _P, _P, _P, _I, _P, _I, _I, _I, _F, _P],
    "dan_can_use_rms_modulate": [_P, _P, _P, _P, _I, _P, _I, _I, _I, _F],
    "dan_gated_rms_modulate": [_P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _F, _P],
    "dan_can_use_gated_rms_modulate": [_P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _F],
    "dan_ln_modulate": [_P, _P, _P, _I, _P, _I, _I, _I, _F, _P],
    "dan_can_use_ln_modulate": [_P, _P, _P, _I, _P, _I, _I, _I, _F],
    "dan_ln_modulate_fp8": [_P, _P, _P, _I, _F, _P, _I, _I, _I, _F, _P],
    "dan_gated_residual_transposed": [_P, _P, _P, _I, _P, _I, _I, _I, _P],
    "dan_can_use_gated_residual_transposed": [_P, _P, _P, _I, _P, _I, _I, _I],
    "dan_gated_ln_modulate": [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _F, _P],
    "dan_can_use_gated_ln_modulate": [_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _F],
    "dan_can_use_ln_modulate_fp8": [_P, _P, _P, _I, _F, _P, _I, _I, _I, _F],
    "dan_qk_norm_rope_epilogue": [_P, _P, _P, _I, _I, _P, _P, _P, _I, _I, _I, _I,
                                  _P, _P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _P],
    "dan_can_use_qk_norm_rope_epilogue": [_P, _P, _P, _I, _I, _P, _P, _P, _I, _I, _I, _I,
                                          _P, _P, _P, _P, _P, _P, _F, _F, _P, _P, _P],
    "dan_qk_norm_rope_neox_epilogue": [_P, _P, _P, _I, _I, _P, _P, _P, _I, _I, _I, _I,
                                       _P, _P, _P, _P, _P, _P, _F, _F, _P, _P, _P, _P],
    "dan_can_use_qk_norm_rope_neox_epilogue": [_P, _P, _P, _I, _I, _P, _P, _P, _I, _I, _I, _I,
                                               _P, _P, _P, _P, _P, _P, _F, _F, _P, _P, _P],
    "dan_qk_norm_rope_cache": [_P, _P, _P] + [_I] * 6 + [_P, _P, _P, _I, _P, _P, _F, ctypes.c_int,
                                                         _P, _I, _P, _P, _I, _I, _P],
    "dan_can_use_qk_norm_rope_cache": [_P, _P, _P] + [_I] * 6 + [_P, _P, _P, _I, _P, _P, _F,
                                                                 ctypes.c_int, _P, _I, _P, _P, _I,
                                                                 _I],
    "dan_window_attention": [_P, _I, _I, _P, _P, _I, _I, _P, _I, _I, _P, _P] + [_I] * 8
                            + [_F, _P, _P, _P, _I, _P],
    "dan_can_use_window_attention": [_P, _I, _I, _P, _P, _I, _I, _P, _I, _I, _P, _P] + [_I] * 8
                                    + [_F, _P, _P, _P, _I],
    "dan_window_attention_workspace": [_I] * 11,
    "dan_ln_modulate_save": [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _F, _P],
    "dan_can_use_ln_modulate_save": [_P, _P, _P, _I, _P, _P, _P, _P, _I, _I, _I, _F],
    "dan_ln_modulate_backward_workspace": [_I, _I, _I],
    "dan_ln_modulate_backward": [_P] * 6 + [_I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I, _P],
    "dan_can_use_ln_modulate_backward": [_P] * 6 + [_I, _P, _P, _P, _P, _I, _I, _I, _I, _P, _I],
    "dan_group_norm_workspace": [_I, _I, _I, _I, _N, _N],
    "dan_group_norm": [_P, _N, _P, _P, _N, _P, _P, _I, _N, _P, _P, _P, _P, _I, _I, _I, _I, _F, _P, _I,
                       _P],
    "dan_can_use_group_norm": [_P, _N, _P, _P, _N, _P, _P, _I, _N, _P, _P, _P, _P, _I, _I, _I, _I, _F,
                               _P, _I],
    "dan_group_norm_backward_workspace": [_I, _I, _I, _I, _N, _N],
    "dan_group_norm_backward": [_P, _P, _N, _P, _P, _P, _P, _P, _N, _P, _P, _I, _N] + [_P] * 5
                               + [_I] * 5 + [_P, _I, _P],
    "dan_can_use_group_norm_backward": [_P, _P, _N, _P, _P, _P, _P, _P, _N, _P, _P, _I, _N] + [_P] * 5
                                       + [_I] * 5 + [_P, _I],
}

_lib = None


class DanError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}")


def load():
    """Load libdan.so (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libdan.so not found at {LIB_PATH}: build the CUDA library first")
        lib = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        for name in _SIGS:
            if name.endswith("_workspace"):
                getattr(lib, name).restype = ctypes.c_int64
        lib.dan_status_string.argtypes = [ctypes.c_int]
        lib.dan_status_string.restype = ctypes.c_char_p
        lib.dan_get_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        lib.dan_get_device_status.restype = ctypes.c_int
        lib.dan_selftest_wait_timeout.argtypes = [ctypes.c_ulonglong, _P]
        lib.dan_selftest_wait_timeout.restype = ctypes.c_int
        _lib = lib
    return _lib


def declared_symbols(header: str = HEADER) -> list[str]:
    """Function names declared in a header (include/dan.h by default)."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S) if header != HEADER else text
    return sorted(set(re.findall(r"\b(dan_\w+)\s*\(", text)))


def status_string(status: int) -> str:
    return load().dan_status_string(int(status)).decode()


def device_status() -> int:
    """Read and clear the current device's status word (bit 1: a warp gave
    up waiting for a row it requested, 4: it then also gave up on its other
    copies in flight, 8: an index array of a cache operation held an entry out
    of its range).  Synchronous; 0 when every wait completed."""
    v = ctypes.c_uint(0)
    _check(load().dan_get_device_status(ctypes.byref(v)), "dan_get_device_status")
    return v.value


def selftest_wait_timeout(limit_ns: int):
    """Launch the bounded-wait self-test on the current stream."""
    _check(load().dan_selftest_wait_timeout(int(limit_ns), _stream()), "dan_selftest_wait_timeout")


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


def _check(status: int, what: str):
    if status != DAN_OK:
        raise DanError(status, what)


def _bf16_cuda(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.bfloat16:
        raise TypeError(f"{name}: expected a CUDA bfloat16 tensor")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(x: torch.Tensor, name: str):
    _bf16_cuda(x, name)
    if x.dim() != 3 or not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous [B, T, D] tensor")
    return x.shape


def _vectors(B: int, D: int, named):
    """Per-batch [B, D] (or [D] when B == 1) views sharing one batch stride."""
    strides = set()
    for name, v in named:
        _bf16_cuda(v, name)
        if v.dim() == 1:
            if B != 1 or v.shape[0] != D or v.stride(0) != 1:
                raise ValueError(f"{name}: a 1-D vector needs B == 1, shape [D], unit stride")
            strides.add(None)
            continue
        if tuple(v.shape) != (B, D) or v.stride(1) != 1:
            raise ValueError(f"{name}: expected a [B={B}, D={D}] view with unit column stride")
        strides.add(v.stride(0) if B > 1 else None)
    strides.discard(None)
    if len(strides) > 1:
        raise ValueError("per-batch vectors must share one batch stride")
    return strides.pop() if strides else D


def _weight(w, D):
    if w is None:
        return None
    _bf16_cuda(w, "weight")
    if w.dim() != 1 or w.shape[0] != D or not w.is_contiguous():
        raise ValueError("weight: expected a contiguous [D] tensor")
    return w


def rms_modulate(x, scale, shift, eps: float, weight=None, out=None):
    """y = bf16(RMSNorm(x) [* weight] * (1 + scale) + shift), x [B, T, D]."""
    B, T, D = _rows(x, "x")
    vs = _vectors(B, D, [("scale", scale), ("shift", shift)])
    weight = _weight(weight, D)
    y = torch.empty_like(x) if out is None else out
    _rows(y, "out")
    _check(load().dan_rms_modulate(_ptr(x), _ptr(weight), _ptr(scale), _ptr(shift), vs, _ptr(y),
                                   B, T, D, float(eps), _stream()), "dan_rms_modulate")
    return y


def gated_rms_modulate(r, h, gate, scale, shift, eps: float, weight=None, r_out=None, out=None):
    """r' = bf16(r + bf16(gate * h)); y = rms_modulate(r').  Returns (r', y)."""
    B, T, D = _rows(r, "r")
    _rows(h, "h")
    vs = _vectors(B, D, [("gate", gate), ("scale", scale), ("shift", shift)])
    weight = _weight(weight, D)
    r_out = torch.empty_like(r) if r_out is None else r_out
    y = torch.empty_like(r) if out is None else out
    _rows(r_out, "r_out")
    _rows(y, "out")
    _check(load().dan_gated_rms_modulate(_ptr(r), _ptr(h), _ptr(gate), _ptr(weight), _ptr(scale),
                                         _ptr(shift), vs, _ptr(r_out), _ptr(y), B, T, D,
                                         float(eps), _stream()), "dan_gated_rms_modulate")
    return r_out, y


def ln_modulate(x, scale, shift, eps: float, out=None):
    """y = bf16(LayerNorm(x) * (1 + scale) + shift), LayerNorm without affine."""
    B, T, D = _rows(x, "x")
    vs = _vectors(B, D, [("scale", scale), ("shift", shift)])
    y = torch.empty_like(x) if out is None else out
    _rows(y, "out")
    _check(load().dan_ln_modulate(_ptr(x), _ptr(scale), _ptr(shift), vs, _ptr(y), B, T, D,
                                  float(eps), _stream()), "dan_ln_modulate")
    return y


def gated_ln_modulate(r, h, gate, scale, shift, eps: float, r_out=None, out=None):
    """r' = bf16(r + bf16(gate * h)); y = ln_modulate(r').  Returns (r', y)."""
    B, T, D = _rows(r, "r")
    _rows(h, "h")
    vs = _vectors(B, D, [("gate", gate), ("scale", scale), ("shift", shift)])
    r_out = torch.empty_like(r) if r_out is None else r_out
    y = torch.empty_like(r) if out is None else out
    _rows(r_out, "r_out")
    _rows(y, "out")
    _check(load().dan_gated_ln_modulate(_ptr(r), _ptr(h), _ptr(gate), _ptr(scale), _ptr(shift),
                                        vs, _ptr(r_out), _ptr(y), B, T, D, float(eps),
                                        _stream()), "dan_gated_ln_modulate")
    return r_out, y


def gated_residual_transposed(r, h, gate, out=None):
    """r: the residual [B, D, T] (the [B, hidden, tokens] layout); h: the
    update [B, T, D]; gate [B, D] (or [D] when B == 1).  Returns
    r' = bf16(r + bf16(gate * h^T)) as [B, D, T]."""
    _bf16_cuda(r, "r")
    _bf16_cuda(h, "h")
    if r.dim() != 3 or not r.is_contiguous():
        raise ValueError("r: expected a contiguous [B, D, T] tensor")
    B, D, T = r.shape
    if tuple(h.shape) != (B, T, D) or not h.is_contiguous():
        raise ValueError("h: expected a contiguous [B, T, D] tensor")
    vs = _vectors(B, D, [("gate", gate)])
    y = torch.empty_like(r) if out is None else out
    _bf16_cuda(y, "out")
    if tuple(y.shape) != (B, D, T) or not y.is_contiguous():
        raise ValueError("out: expected a contiguous [B, D, T] tensor")
    _check(load().dan_gated_residual_transposed(_ptr(r), _ptr(h), _ptr(gate), vs, _ptr(y), B, T,
                                                D, _stream()), "dan_gated_residual_transposed")
    return y


def ln_modulate_fp8(x, scale, shift, qscale: float, eps: float, out=None):
    """q = e4m3(ln_modulate(x, scale, shift, eps) * rn(1/qscale)) as a
    torch.uint8 [B, T, D] tensor of E4M3 codes (view it as
    torch.float8_e4m3fn for an FP8 GEMM)."""
    B, T, D = _rows(x, "x")
    vs = _vectors(B, D, [("scale", scale), ("shift", shift)])
    q = torch.empty((B, T, D), dtype=torch.uint8, device=x.device) if out is None else out
    if q.dtype != torch.uint8 or not q.is_cuda or tuple(q.shape) != (B, T, D) or not q.is_contiguous():
        raise ValueError("out: expected a contiguous CUDA uint8 [B, T, D] tensor")
    _check(load().dan_ln_modulate_fp8(_ptr(x), _ptr(scale), _ptr(shift), vs, float(qscale),
                                      _ptr(q), B, T, D, float(eps), _stream()),
           "dan_ln_modulate_fp8")
    return q


def _qkv(views, name, heads, hd):
    q, k, v = views
    T = q.shape[0]
    for t, n in zip(views, "qkv"):
        _bf16_cuda(t, f"{name}.{n}")
        if t.dim() != 2 or t.shape != (T, heads * hd) or (T > 0 and t.stride(1) != 1):
            raise ValueError(f"{name}.{n}: expected a [T, heads*{hd}] view with unit column stride")
    strides = {t.stride(0) for t in views} if T > 1 else {heads * hd}
    if len(strides) != 1:
        raise ValueError(f"{name}: q, k, v must share one row stride")
    return T, strides.pop()


def qk_norm_rope_epilogue(txt, img, wq_txt, wk_txt, wq_img, wk_img, rope_txt, rope_img,
                          eps_txt: float, eps_img: float, heads: int, out=None,
                          head_dim: int = 128, neox: bool = False):
    """txt, img: (q, k, v) views [T_s, heads*head_dim]; weights [head_dim] bf16;
    rope tables fp32 [T_s, head_dim].  Returns joint (q, k, v), each
    [T_txt+T_img, heads, head_dim].  head_dim 128 or 64; neox=True rotates
    the halves' pairs (dan_qk_norm_rope_neox_epilogue) instead of
    interleaved pairs."""
    hd = int(head_dim)
    Tt, st = _qkv(txt, "txt", heads, hd)
    Ti, si = _qkv(img, "img", heads, hd)
    for w, n in ((wq_txt, "wq_txt"), (wk_txt, "wk_txt"), (wq_img, "wq_img"), (wk_img, "wk_img")):
        _bf16_cuda(w, n)
        if w.shape != (hd,) or not w.is_contiguous():
            raise ValueError(f"{n}: expected a contiguous [{hd}] tensor")
    for r, n, T in ((rope_txt, "rope_txt", Tt), (rope_img, "rope_img", Ti)):
        if not r.is_cuda or r.dtype != torch.float32 or r.shape != (T, hd) or not r.is_contiguous():
            raise ValueError(f"{n}: expected a contiguous CUDA float32 [T, {hd}] tensor")
    if out is None:
        dev = txt[0].device
        out = tuple(torch.empty((Tt + Ti, heads, hd), dtype=torch.bfloat16, device=dev)
                    for _ in range(3))
    qo, ko, vo = out
    name = "dan_qk_norm_rope_neox_epilogue" if neox else "dan_qk_norm_rope_epilogue"
    _check(getattr(load(), name)(
        _ptr(txt[0]), _ptr(txt[1]), _ptr(txt[2]), Tt, st,
        _ptr(img[0]), _ptr(img[1]), _ptr(img[2]), Ti, si, heads, hd,
        _ptr(wq_txt), _ptr(wk_txt), _ptr(wq_img), _ptr(wk_img), _ptr(rope_txt), _ptr(rope_img),
        float(eps_txt), float(eps_img), _ptr(qo), _ptr(ko), _ptr(vo), _stream()), name)
    return qo, ko, vo


# ------------------------------------------------------ paged-cache operators
#
# A decode step calls these for a few microseconds of GPU work, so the checks
# of a good call are kept short (dtype, device index, shape and strides, each
# read once); what is wrong with a bad one is worked out only when it is.

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _is(t, dtype, device: int) -> bool:
    try:
        return t.dtype is dtype and t.get_device() == device
    except AttributeError:  # not a tensor
        return False


def _want(t, name: str, dtype, device: int, first: str = "the caches"):
    """Raise for a tensor that is not of this dtype on this CUDA device (that of `first`)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype is not dtype:
        raise TypeError(f"{name}: expected a CUDA {str(dtype).removeprefix('torch.')} tensor")
    if t.get_device() != device:
        raise ValueError(f"{name}: lies on cuda:{t.get_device()}, {first} on cuda:{device}")


def _caches(k_cache, v_cache):
    """([pages, kv_heads, page_size, head_dim], device index) of the caches."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dtype is not _BF16 or not k_cache.is_cuda:
        raise TypeError("k_cache: expected a CUDA bfloat16 tensor")
    device, shape = k_cache.get_device(), k_cache.shape
    if not _is(v_cache, _BF16, device):
        _want(v_cache, "v_cache", _BF16, device)
    if len(shape) != 4 or shape != v_cache.shape or not k_cache.is_contiguous() or \
            not v_cache.is_contiguous():
        raise ValueError("k_cache, v_cache: expected two contiguous [pages, kv_heads, page_size, "
                         "head_dim] tensors of one shape")
    if not shape[3]:
        raise ValueError("k_cache: head_dim is 0")
    return shape, device


def _ints(t, name: str, shape, device: int):
    if not _is(t, _I32, device):
        _want(t, name, _I32, device)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {list(shape)} tensor")


def _token_rows(t, name: str, N: int, heads: int, hd: int, device: int) -> int:
    """Row stride of a [N, heads, hd] or [N, heads*hd] view whose rows are dense."""
    if not _is(t, _BF16, device):
        _want(t, name, _BF16, device)
    shape, stride = t.shape, t.stride()
    width = heads * hd
    if len(shape) == 2:
        good = shape == (N, width) and (stride[1] == 1 or width == 1)
    else:
        good = shape == (N, heads, hd) and (stride[2] == 1 or hd == 1) and (stride[1] == hd or heads == 1)
    if not good and not (N == 0 and t.numel() == 0 and shape in ((0, width), (0, heads, hd))):
        raise ValueError(f"{name}: expected [{N}, {heads}, {hd}] (or [{N}, {width}]) with dense rows")
    return stride[0] if N > 1 else width


def _limit(value, name: str) -> int:
    value = int(value)
    if not 0 <= value <= 0x7FFFFFFF:
        raise ValueError(f"{name}: expected 0 .. 2**31 - 1, got {value}")
    return value


def _on(device: int, name: str, *args):
    """Call an entry point with the device's current stream, on that device."""
    fn = getattr(_lib or load(), name)
    if torch._C._cuda_getDevice() == device:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if status != DAN_OK:
        raise DanError(status, name)


def qk_norm_rope_cache(q, k, v, wq, wk, rope, positions, slots, k_cache, v_cache, eps: float,
                       neox: bool = False, q_out=None):
    """RMSNorm per head and RoPE of Q and K at given positions; K and V go to
    the paged cache (include/dan_cache.h).

    q [N, heads*hd], k, v [N, kv_heads*hd] (or with the heads as a dimension of
    their own): views with dense rows, k and v with one row stride (e.g. column
    slices of a packed projection); wq, wk [hd]; rope fp32 [rows, hd], row p the
    cosines then sines of position p; positions, slots int32 [N], a negative
    slot storing nothing; k_cache, v_cache [pages, kv_heads, page_size, hd],
    written in place.  Returns the queries [N, heads, hd] (q_out if given;
    q_out may be q itself).  All tensors on one device, whose current stream
    the call runs on."""
    (pages, Hkv, page, hd), device = _caches(k_cache, v_cache)
    if not _is(q, _BF16, device):
        _want(q, "q", _BF16, device)
    shape = q.shape
    if len(shape) not in (2, 3) or (len(shape) == 2 and shape[1] % hd):
        raise ValueError(f"q: expected [N, heads*{hd}] or [N, heads, {hd}]")
    N = shape[0]
    H = shape[1] // hd if len(shape) == 2 else shape[1]
    q_stride = _token_rows(q, "q", N, H, hd, device)
    kv_stride = _token_rows(k, "k", N, Hkv, hd, device)
    if _token_rows(v, "v", N, Hkv, hd, device) != kv_stride:
        raise ValueError("k and v must share one row stride")
    for w, name in ((wq, "wq"), (wk, "wk")):
        if not _is(w, _BF16, device):
            _want(w, name, _BF16, device)
        if w.shape != (hd,) or not w.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous [{hd}] tensor")
    if not _is(rope, _F32, device):
        _want(rope, "rope", _F32, device)
    if rope.dim() != 2 or rope.shape[1] != hd or not rope.is_contiguous():
        raise ValueError(f"rope: expected a contiguous [rows, {hd}] tensor")
    _ints(positions, "positions", (N,), device)
    _ints(slots, "slots", (N,), device)
    if q_out is None:
        q_out = torch.empty((N, H, hd), dtype=_BF16, device=k_cache.device)
        out_stride = H * hd
    else:
        out_stride = _token_rows(q_out, "q_out", N, H, hd, device)
    _on(device, "dan_qk_norm_rope_cache", q.data_ptr(), k.data_ptr(), v.data_ptr(), N, q_stride,
        kv_stride, H, Hkv, hd, wq.data_ptr(), wk.data_ptr(), rope.data_ptr(), rope.shape[0],
        positions.data_ptr(), slots.data_ptr(), float(eps), 1 if neox else 0, q_out.data_ptr(), out_stride,
        k_cache.data_ptr(), v_cache.data_ptr(), pages, page)
    return q_out if q_out.dim() == 3 else q_out.unflatten(1, (H, hd))


@functools.lru_cache(maxsize=1024)
def _attention_workspace(*sizes) -> int:
    return load().dan_window_attention_workspace(*sizes)


def window_attention(q, k_cache, v_cache, page_table, q_start, kv_len, window: int, sinks: int = 0,
                     chunk: int = 1, scale: float | None = None, max_q: int | None = None, out=None,
                     lse=None):
    """Attention of ragged sequences over the paged cache
    (include/dan_cache.h): each query sees the first ``sinks`` tokens, the
    ``window`` tokens up to the first of its chunk, and its chunk of ``chunk``
    tokens (chunk=1: causal).

    q [N, heads, hd] with dense rows; page_table int32 [S, max_pages] (rows may
    be strided); q_start int32 [S+1], kv_len int32 [S]: sequence s has the
    query rows q_start[s]..q_start[s+1]-1, its last tokens, and kv_len[s] keys
    in the cache.  scale defaults to hd**-0.5; max_q is a bound on the rows of
    one sequence.  Returns out [N, heads, hd] (rows outside every sequence are
    not written), or (out, lse) when ``lse`` is a float32 [N, heads] tensor or
    True.  All tensors on one device, whose current stream the call runs on."""
    (pages, Hkv, page, hd), device = _caches(k_cache, v_cache)
    if not _is(q, _BF16, device):
        _want(q, "q", _BF16, device)
    if q.dim() != 3:
        raise ValueError("q: expected a [N, heads, head_dim] tensor")
    N, H, _ = q.shape
    q_stride = _token_rows(q, "q", N, H, hd, device)
    if not _is(page_table, _I32, device):
        _want(page_table, "page_table", _I32, device)
    if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table: expected [S, max_pages] with unit column stride")
    S, M = page_table.shape
    table_stride = page_table.stride(0) if S > 1 else M
    _ints(q_start, "q_start", (S + 1,), device)
    _ints(kv_len, "kv_len", (S,), device)
    window, sinks, chunk = _limit(window, "window"), _limit(sinks, "sinks"), _limit(chunk, "chunk")
    max_q = N if max_q is None else _limit(max_q, "max_q")
    if out is None:
        out = torch.empty((N, H, hd), dtype=_BF16, device=k_cache.device)
    else:
        if not _is(out, _BF16, device):
            _want(out, "out", _BF16, device)
        if out.shape != (N, H, hd) or not out.is_contiguous():
            raise ValueError("out: expected a contiguous [N, heads, head_dim] tensor")
    if lse is None or lse is False:
        lse = None
    elif lse is True:
        lse = torch.empty((N, H), dtype=_F32, device=k_cache.device)
    else:
        if not _is(lse, _F32, device):
            _want(lse, "lse", _F32, device)
        if lse.shape != (N, H) or not lse.is_contiguous():
            raise ValueError("lse: expected a contiguous float32 [N, heads] tensor")
    size = _attention_workspace(N, S, H, Hkv, hd, M, page, window, sinks, chunk, max_q)
    # of this call alone: the allocator hands it on in the stream's order
    work = torch.empty(size, dtype=torch.uint8, device=k_cache.device) if size else None
    _on(device, "dan_window_attention", q.data_ptr(), N, q_stride, k_cache.data_ptr(),
        v_cache.data_ptr(), pages, page, page_table.data_ptr(), table_stride, M, q_start.data_ptr(),
        kv_len.data_ptr(), S, H, Hkv, hd, window, sinks, chunk, max_q,
        hd ** -0.5 if scale is None else float(scale), out.data_ptr(), None if lse is None else lse.data_ptr(),
        None if work is None else work.data_ptr(), size)
    return out if lse is None else (out, lse)


# ---------------------------------------------------------- training operators
#
# What a forward pass keeps is a tuple (stats, codes, scales): the rows' or
# groups' mean and 1/std, and the input's 8-bit checkpoint (or None twice).

_U8 = torch.uint8


@functools.lru_cache(maxsize=1024)
def _bytes(name: str, device: int, *sizes) -> int:
    with torch.cuda.device(device):  # the count may follow from the device's SMs
        return getattr(load(), name)(*sizes)


def _two(shape, dtype, device):
    """Two outputs (one of two rows, unbound, takes twice the host's time)."""
    return torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device)


def _dense(t, name: str, dtype, shape, device: int, first: str):
    """A contiguous tensor of this dtype and shape on the device of `first`."""
    if not _is(t, dtype, device):
        _want(t, name, dtype, device, first)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {list(shape)} tensor")


def _batch_rows(t, name: str, dtype, B: int, D: int, device: int, first: str) -> int:
    """Batch stride of a [B, D] view (or [D] when B == 1) with unit column stride."""
    if not _is(t, dtype, device):
        _want(t, name, dtype, device, first)
    shape = t.shape
    if shape == (B, D):
        if t.stride(1) != 1 and B > 0:
            raise ValueError(f"{name}: expected unit column stride")
        return t.stride(0) if B > 1 else D
    if B != 1 or shape != (D,) or t.stride(0) != 1:
        raise ValueError(f"{name}: expected a [{B}, {D}] view with unit column stride")
    return D


def _pair(a, b, names, dtype, B: int, D: int, device: int, first: str) -> int:
    """The one batch stride of two [B, D] views."""
    stride = _batch_rows(a, names[0], dtype, B, D, device, first)
    if b.__class__ is a.__class__ and b.dtype is dtype and b.shape == a.shape and \
            b.stride() == a.stride() and b.get_device() == device:
        return stride  # (a good pair, checked once)
    if _batch_rows(b, names[1], dtype, B, D, device, first) != stride:
        raise ValueError(f"{names[0]} and {names[1]} must share one batch stride")
    return stride


def _kept(saved):
    try:
        stats, codes, scales = saved
    except (TypeError, ValueError):
        raise TypeError("saved: expected the (stats, codes, scales) of the forward pass") from None
    return stats, codes, scales


def ln_modulate_save(x, scale, shift, eps: float, checkpoint: bool = True, out=None):
    """y = LayerNorm(x) * (1 + scale) + shift for training (include/dan_train.h):
    rounded to bf16 once, and what the gradient needs.

    x [B, T, D] contiguous; scale, shift [B, D] (or [D] when B == 1) views that
    share one batch stride; out may be x itself.  Returns (y, saved) with saved
    = (stats, codes, scales): stats float32 [B, T, 2], the rows' mean and 1/std;
    codes uint8 [B, T, D] and scales uint8 [B, T, ceil(D / 32)], x in 8 bits
    (E4M3 codes, an E8M0 power of two for each 32 columns), or None without
    ``checkpoint``."""
    B, T, D = _rows(x, "x")
    device = x.get_device()
    vs = _pair(scale, shift, ("scale", "shift"), _BF16, B, D, device, "x")
    if out is None:
        out = torch.empty_like(x)
    else:
        _dense(out, "out", _BF16, x.shape, device, "x")
    stats = torch.empty((B, T, 2), dtype=_F32, device=x.device)
    codes = scales = None
    if checkpoint:
        codes = torch.empty((B, T, D), dtype=_U8, device=x.device)
        scales = torch.empty((B, T, (D + 31) // 32), dtype=_U8, device=x.device)
    _on(device, "dan_ln_modulate_save", x.data_ptr(), scale.data_ptr(), shift.data_ptr(), vs, out.data_ptr(),
        stats.data_ptr(), _ptr(codes), _ptr(scales), B, T, D, float(eps))
    return out, (stats, codes, scales)


def ln_modulate_backward(dy, x, scale, saved, dres=None, dx=None, dscale=None, dshift=None):
    """The gradients of ``ln_modulate_save`` (include/dan_train.h).

    dy [B, T, D]; x the forward pass's input, or None to take it from the
    checkpoint in ``saved``; scale as there; dres [B, T, D]: a gradient of x from
    elsewhere, added to dx before its rounding.  dx may be dy or dres itself;
    dscale, dshift [B, D] (or [D] when B == 1): views that share one batch stride,
    e.g. of the embedding's gradient.  Returns (dx, dscale, dshift), bf16."""
    B, T, D = _rows(dy, "dy")
    device, shape = dy.get_device(), dy.shape
    stats, codes, scales = _kept(saved)
    _dense(stats, "stats", _F32, (B, T, 2), device, "dy")
    if x is not None:
        _dense(x, "x", _BF16, shape, device, "dy")
        at = x.data_ptr(), None, None
    elif codes is None or scales is None:
        raise ValueError("x: None, but nothing in saved holds it")
    else:
        _dense(codes, "codes", _U8, shape, device, "dy")
        _dense(scales, "scales", _U8, (B, T, (D + 31) // 32), device, "dy")
        at = None, codes.data_ptr(), scales.data_ptr()
    vs = _batch_rows(scale, "scale", _BF16, B, D, device, "dy")
    if dres is not None:
        _dense(dres, "dres", _BF16, shape, device, "dy")
    if dx is None:
        dx = torch.empty_like(dy)
    else:
        _dense(dx, "dx", _BF16, shape, device, "dy")
    if dscale is None and dshift is None:
        dscale, dshift = _two((B, D), _BF16, dy.device)
        gs = D
    elif dscale is None or dshift is None:
        raise ValueError("dscale and dshift: expected both or neither")
    else:
        gs = _pair(dscale, dshift, ("dscale", "dshift"), _BF16, B, D, device, "dy")
    size = _bytes("dan_ln_modulate_backward_workspace", device, B, T, D)
    # of this call alone: the allocator hands it on in the stream's order
    work = torch.empty(size, dtype=_U8, device=dy.device) if size else None
    _on(device, "dan_ln_modulate_backward", dy.data_ptr(), *at, stats.data_ptr(), scale.data_ptr(), vs,
        _ptr(dres), dx.data_ptr(), dscale.data_ptr(), dshift.data_ptr(), gs, B, T, D, _ptr(work), size)
    return dx, dscale, dshift


_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_ACTS = {None: 0, "silu": 1}


def _last(t) -> bool:
    """Whether a tensor's memory is dense with its channels last."""
    if t.dim() == 3:
        return t.is_contiguous()
    return t.is_contiguous(memory_format=torch.channels_last if t.dim() == 4 else torch.channels_last_3d)


def _images(t, name: str):
    """(N, S, C) of a channels-last image tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _TYPES:
        raise TypeError(f"{name}: expected a CUDA bfloat16, float16 or float32 tensor")
    shape = t.shape
    if len(shape) not in (3, 4, 5) or not _last(t):
        raise ValueError(f"{name}: expected [N, C, H, W] (or [N, C, D, H, W]) in channels_last memory, or "
                         "a contiguous [N, S, C] tensor")
    if len(shape) == 4:
        return shape[0], shape[2] * shape[3], shape[1]
    return tuple(shape) if len(shape) == 3 else (shape[0], shape[2] * shape[3] * shape[4], shape[1])


def _like(t, name: str, dtype, shape, device: int, first: str):
    """A channels-last image tensor of this dtype and shape on the device of `first`."""
    if not _is(t, dtype, device):
        _want(t, name, dtype, device, first)
    if t.shape != shape or not _last(t):
        raise ValueError(f"{name}: expected a {list(shape)} tensor, channels last in memory")


def _scale_shape(shape):
    """The shape of the checkpoint's scales for images of a shape."""
    if len(shape) == 3:
        return shape[0], shape[1], shape[2] // 32
    return shape[0], shape[1] // 32, *shape[2:]


def _gains(weight, bias, scale, shift, dtype, N: int, C: int, device: int, first: str):
    """(type of weight and bias, image stride of scale and shift)."""
    ptype, vs = _TYPES[dtype], C
    if weight is not None or bias is not None:
        if weight is None or bias is None:
            raise ValueError("weight and bias: expected both or neither")
        wtype = weight.dtype if isinstance(weight, torch.Tensor) and weight.dtype is _F32 else dtype
        ptype = _TYPES[wtype]
        for t, name in ((weight, "weight"), (bias, "bias")):
            _dense(t, name, wtype, (C,), device, first)
    if scale is not None or shift is not None:
        if scale is None or shift is None:
            raise ValueError("scale and shift: expected both or neither")
        vs = _pair(scale, shift, ("scale", "shift"), dtype, N, C, device, first)
    return ptype, vs


def _act(act) -> int:
    try:
        return _ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act: expected None or 'silu', got {act!r}") from None


def _group_norm(x, groups, weight, bias, eps, act, scale, shift, out, save: bool, checkpoint: bool):
    N, S, C = _images(x, "x")
    device, dtype, shape = x.get_device(), x.dtype, x.shape
    groups, act = int(groups), _act(act)
    if not 1 <= groups <= C:  # before anything is allocated by their number
        raise DanError(DAN_EINVAL if groups < 1 else DAN_EUNSUPPORTED, "dan_group_norm")
    ptype, vs = _gains(weight, bias, scale, shift, dtype, N, C, device, "x")
    if out is None:
        out = torch.empty_like(x)
    else:
        _like(out, "out", dtype, shape, device, "x")
    stats = codes = scales = None
    if save:
        stats = torch.empty((N, groups, 2), dtype=_F32, device=x.device)
        if checkpoint:
            if C % 32:
                raise ValueError(f"checkpoint: expected channels in blocks of 32, got {C}")
            codes = torch.empty_like(x, dtype=_U8)
            scales = torch.empty_strided(*_scale_layout(shape), dtype=_U8, device=x.device)
    size = _bytes("dan_group_norm_workspace", device, N, S, C, groups, _TYPES[dtype], 1 if codes is not None else 0)
    work = torch.empty(size, dtype=_U8, device=x.device) if size else None
    _on(device, "dan_group_norm", x.data_ptr(), _TYPES[dtype], _ptr(weight), _ptr(bias), ptype, _ptr(scale),
        _ptr(shift), vs, act, out.data_ptr(), _ptr(stats), _ptr(codes), _ptr(scales), N, S, C, groups, float(eps),
        _ptr(work), size)
    return out, (stats, codes, scales)


@functools.lru_cache(maxsize=1024)
def _scale_layout(shape):
    """Shape and (channels-last) strides of the checkpoint's scales."""
    shape = _scale_shape(shape)
    if len(shape) == 3:
        return shape, (shape[1] * shape[2], shape[2], 1)
    strides, step = [1] * len(shape), shape[1]
    for i in range(len(shape) - 1, 1, -1):
        strides[i], step = step, step * shape[i]
    strides[0] = step
    return shape, tuple(strides)


def group_norm(x, groups: int, weight, bias, eps: float, act=None, scale=None, shift=None, out=None):
    """Group norm of channels-last images (include/dan_train.h):
    z = (n * weight + bias) * (1 + scale) + shift, y = z, or silu(z) with
    ``act="silu"``.

    x [N, C, H, W] (or [N, C, D, H, W]) in torch's channels_last memory, or
    [N, S, C] contiguous, in bf16, fp16 or fp32; weight, bias [C] in x's type or
    fp32 (or None); scale, shift [N, C] (or [C] when N == 1) in x's type, views
    that share one image stride (or None).  out may be x itself.  Returns y like
    x."""
    return _group_norm(x, groups, weight, bias, eps, act, scale, shift, out, False, False)[0]


def group_norm_save(x, groups: int, weight, bias, eps: float, act=None, scale=None, shift=None,
                    checkpoint: bool = True, out=None):
    """``group_norm`` for training.  Returns (y, saved) with saved = (stats,
    codes, scales): stats float32 [N, groups, 2], the groups' mean and 1/std;
    codes uint8 like x and scales uint8 like x with C / 32 channels, x in 8 bits
    (for C % 32 == 0), or None without ``checkpoint``."""
    return _group_norm(x, groups, weight, bias, eps, act, scale, shift, out, True, checkpoint)


def group_norm_backward(dy, x, groups: int, weight, bias, saved, act=None, scale=None, shift=None, dx=None,
                        dscale=None, dshift=None):
    """The gradients of ``group_norm_save`` (include/dan_train.h).

    dy like the forward pass's x; x that input, or None to take it from the
    checkpoint in ``saved``; the others as there.  dx may be dy itself; dscale,
    dshift [N, C] (or [C] when N == 1): views that share one image stride, e.g. of
    the embedding's gradient.  Returns (dx, dweight, dbias, dscale, dshift), each in
    the type of what it is the gradient of, None where that is."""
    N, S, C = _images(dy, "dy")
    device, dtype, shape = dy.get_device(), dy.dtype, dy.shape
    groups, act = int(groups), _act(act)
    stats, codes, scales = _kept(saved)
    _dense(stats, "stats", _F32, (N, groups, 2), device, "dy")
    if x is not None:
        _like(x, "x", dtype, shape, device, "dy")
        at = x.data_ptr() or 16, None, None  # (no memory is looked at where there is none)
    elif codes is None or scales is None:
        raise ValueError("x: None, but nothing in saved holds it")
    else:
        if C % 32:
            raise ValueError(f"saved: a checkpoint has channels in blocks of 32, dy has {C}")
        _like(codes, "codes", _U8, shape, device, "dy")
        _like(scales, "scales", _U8, _scale_shape(shape), device, "dy")
        at = None, codes.data_ptr(), scales.data_ptr()
    ptype, vs = _gains(weight, bias, scale, shift, dtype, N, C, device, "dy")
    if dx is None:
        dx = torch.empty_like(dy)
    else:
        _like(dx, "dx", dtype, shape, device, "dy")
    dweight = dbias = None
    if weight is not None:
        dweight, dbias = _two((C,), weight.dtype, dy.device)
    gs = C
    if dscale is not None or dshift is not None:
        if dscale is None or dshift is None:
            raise ValueError("dscale and dshift: expected both or neither")
        if scale is None:
            raise ValueError("dscale and dshift: there is no scale and shift")
        gs = _pair(dscale, dshift, ("dscale", "dshift"), dtype, N, C, device, "dy")
    elif scale is not None:
        dscale, dshift = _two((N, C), dtype, dy.device)
    size = _bytes("dan_group_norm_backward_workspace", device, N, S, C, groups, _TYPES[dtype], 1 if x is None else 0)
    work = torch.empty(size, dtype=_U8, device=dy.device) if size else None
    _on(device, "dan_group_norm_backward", dy.data_ptr(), at[0], _TYPES[dtype], at[1], at[2], stats.data_ptr(),
        _ptr(weight), _ptr(bias), ptype, _ptr(scale), _ptr(shift), vs, act, dx.data_ptr(), _ptr(dweight),
        _ptr(dbias), _ptr(dscale), _ptr(dshift), gs, N, S, C, groups, _ptr(work), size)
    return dx, dweight, dbias, dscale, dshift
