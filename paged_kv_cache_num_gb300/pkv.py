"""Python binding of the C ABI in include/pkv.h (ctypes; argument marshalling
only).  Every operation runs in the CUDA kernels of libpkv.so; there is no
fallback: if the library is not built or a call fails, an exception is
raised.  PyTorch provides the device memory and the current stream.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libpkv.so")

# dtype codes (pkv.h)
F16, BF16, E4M3, U3, U8, I32, I64, F32, E5M2, I8, U4 = 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11
# device error bits
DEVERR_SLOT_RANGE, DEVERR_BLOCK_RANGE, DEVERR_CONTEXT_RANGE, DEVERR_POS_RANGE, DEVERR_TIMEOUT = (
    1, 2, 4, 8, 16)
DEVERR_QSTART_RANGE = 32
DEVERR_POOL_RANGE = 64

_TORCH_CODES = {torch.float16: F16, torch.bfloat16: BF16, torch.float8_e4m3fn: E4M3,
                torch.float8_e5m2: E5M2, torch.int8: I8,
                torch.uint8: U8, torch.int32: I32, torch.int64: I64, torch.float32: F32}


class PkvError(RuntimeError):
    """A non-OK status from the library (message from pkv_last_error)."""

    def __init__(self, code: int, msg: str):
        super().__init__("pkv error %d: %s" % (code, msg))
        self.code = code


class _Tensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class _Cache(ctypes.Structure):
    _fields_ = [("k_cache", _Tensor), ("v_cache", _Tensor), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_qscale", _Tensor), ("k_qzero", _Tensor),
                ("v_qscale", _Tensor), ("v_qzero", _Tensor), ("scale_mode", ctypes.c_int32),
                ("k_scales", _Tensor), ("v_scales", _Tensor), ("chunk_stride", ctypes.c_int64)]


# scale granularity of fp8 / int8 caches (pkv.h PKV_SCALE_*)
SCALE_MODES = {"head": 0, "block": 1, "token": 2}


_lib = None
_lock = threading.Lock()


def lib():
    """The loaded libpkv.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError("libpkv.so is not built (%s); run "
                                  "paged_kv_cache_num_gb300.build.build()" % LIB_PATH)
            L = ctypes.CDLL(LIB_PATH)
            P = ctypes.c_void_p
            TP = ctypes.POINTER(_Tensor)
            CP = ctypes.POINTER(_Cache)
            L.pkv_version.restype = ctypes.c_char_p
            L.pkv_last_error.restype = ctypes.c_char_p
            L.pkv_abi_version.restype = ctypes.c_int
            # descriptors of most calls are packed bytes (_packed)
            L.pkv_slot_mapping.argtypes = [P, P, P, ctypes.c_int, P, P, P]
            L.pkv_kv_append.argtypes = [P, P, P, P, P, P]
            L.pkv_kv_append_scaled.argtypes = [TP, TP, TP, TP, TP, CP, P, P]
            L.pkv_paged_decode_workspace.argtypes = [P, P, P, ctypes.c_int, P]
            L.pkv_paged_decode_launches.argtypes = [TP, CP, TP, ctypes.c_int,
                                                    ctypes.POINTER(ctypes.c_int32)]
            L.pkv_paged_decode.argtypes = [P, P, P, P, ctypes.c_float, P, ctypes.c_int, P, ctypes.c_size_t, P, P]
            L.pkv_paged_decode_noalloc.argtypes = [TP, CP, TP, TP, ctypes.c_float, TP,
                                                   ctypes.c_int, P, P]
            L.pkv_decode_step.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_float, P, ctypes.c_int, P,
                                          ctypes.c_size_t, P, P]
            L.pkv_kv_append_dynamic.argtypes = [P, P, P, P, P, P]
            L.pkv_kv_gather.argtypes = [P, P, P, P, P, P]
            L.pkv_paged_prefill_workspace.argtypes = [P, P, P, P]
            L.pkv_paged_prefill_launches.argtypes = [P, P, P, P]
            L.pkv_paged_prefill.argtypes = [P, P, P, P, P, ctypes.c_float, P, P, ctypes.c_size_t, P, P]
            L.pkv_norm_rope.argtypes = [P, P, P, P, ctypes.c_float, P, P, ctypes.c_int, P, P, P, P]
            L.pkv_norm_rope_append.argtypes = [P, P, P, P, P, ctypes.c_float, P, P, ctypes.c_int, P, P, P, P, P]
            L.pkv_extend_tables.argtypes = [P, P, P, P, P, ctypes.c_int, P, P, P, P, P, P, P, P]
            L.pkv_trim_tables.argtypes = [P, P, P, P, P, ctypes.c_int, P, P, P, P]
            L.pkv_noalloc_scratch_bytes.restype = ctypes.c_size_t
            L.pkv_pack3.argtypes = [P, P, ctypes.c_int64, P]
            L.pkv_unpack3.argtypes = [P, P, ctypes.c_int64, P]
            L.pkv_unpack3_words.argtypes = [P, P, ctypes.c_int64, P]
            L.pkv_copy_peak.argtypes = [P, P, ctypes.c_size_t, P]
            for fn in ("pkv_slot_mapping", "pkv_kv_append", "pkv_kv_append_scaled",
                       "pkv_paged_decode_workspace", "pkv_paged_decode_launches",
                       "pkv_paged_decode", "pkv_paged_decode_noalloc", "pkv_decode_step", "pkv_pack3",
                       "pkv_kv_append_dynamic", "pkv_kv_gather", "pkv_paged_prefill_workspace",
                       "pkv_paged_prefill_launches", "pkv_paged_prefill", "pkv_norm_rope", "pkv_norm_rope_append",
                       "pkv_extend_tables", "pkv_trim_tables", "pkv_unpack3", "pkv_unpack3_words", "pkv_copy_peak"):
                getattr(L, fn).restype = ctypes.c_int
            _lib = L
    return _lib


def _check(rc: int):
    if rc != 0:
        raise PkvError(rc, lib().pkv_last_error().decode())


_PACK = struct.Struct("@Pii8q").pack          # pkv_tensor
_PAD = ((0, 0, 0, 0), (0, 0, 0), (0, 0), (0,), ())


def _packed(t: torch.Tensor, code: Optional[int] = None) -> bytes:
    """A pkv_tensor as bytes."""
    sh, st = t.shape, t.stride()
    n = len(sh)
    if n > 4:
        raise ValueError("at most 4 dims")
    pad = _PAD[n]
    return _PACK(t.data_ptr() if 0 not in sh else 0, _TORCH_CODES[t.dtype] if code is None else code, n,
                 *sh, *pad, *st, *pad)


def _desc(t: Optional[torch.Tensor], code: Optional[int] = None) -> _Tensor:
    return _Tensor() if t is None else _Tensor.from_buffer_copy(_packed(t, code))


def _xvec_desc(t: torch.Tensor, code: int) -> _Tensor:
    if t.dim() != 5 or t.stride(4) != 1:
        raise ValueError("an xvec cache is [num_blocks, Hkv, head_dim // x, block_size, x], x contiguous")
    d = _Tensor()
    d.data = t.data_ptr() if t.numel() > 0 else 0
    d.dtype = code
    d.ndim = 4
    P, H, C, BS, x = t.shape
    for i, (n, st) in enumerate(((P, t.stride(0)), (BS, t.stride(3)), (H, t.stride(1)), (C * x, 1))):
        d.shape[i] = n
        d.stride[i] = st
    return d


def _flag(err_flag):
    if err_flag is None:
        return None
    if err_flag.dtype is not torch.int32 or err_flag.numel() < 1:
        raise ValueError("err_flag must be an int32")
    return err_flag.data_ptr()


def _room(t, name: str, nbytes: int = 0):
    """(address, bytes) of a buffer that is taken as one run of bytes."""
    if t is None:
        return None, 0
    n = t.numel() * t.element_size()
    if not t.is_contiguous() or n < nbytes:
        raise ValueError("%s must be contiguous, of %d bytes or more" % (name, nbytes))
    return t.data_ptr(), n


def _one_device(*ts) -> int:
    """The CUDA device that every tensor is on."""
    dev = None
    for t in ts:
        if t is not None:
            i = t.get_device()
            if i != dev:
                if i < 0:
                    raise ValueError("all tensors must be CUDA tensors")
                if dev is not None:
                    raise ValueError("all tensors must be on one device, got cuda:%d and cuda:%d" % (dev, i))
                dev = i
    return dev


def _elsewhere(dev: int, stream):
    """None when device `dev` is current and no stream is given; else a
    context in which they are, so that what the call allocates belongs to the
    stream that uses it."""
    if stream is None:
        if torch.cuda.current_device() == dev:
            return None
        stream = torch.cuda.current_stream(dev)
    elif stream.device_index != dev:
        raise ValueError("the stream is on cuda:%d, the tensors on cuda:%d" % (stream.device_index, dev))
    return torch.cuda.stream(stream)


@dataclass
class KVCache:
    """A paged KV cache [num_blocks, block_size, num_kv_heads, row] in device
    memory.  kind: "f16", "bf16", "e4m3" / "e5m2" / "i8" (+ per-kv-head fp32 scales), or "u3" /
    "u4" (3- or 4-bit codes, row = 3*head_dim/8 or head_dim/2 bytes, + fp16
    scale / uint8 zero per (slot, head)).  layout "xvec" (16-bit and one-byte kinds): k_cache /
    v_cache are stored [num_blocks, num_kv_heads, head_dim // x, block_size,
    x] with x = 16 bytes / element size."""
    kind: str
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None
    k_qscale: Optional[torch.Tensor] = None
    k_qzero: Optional[torch.Tensor] = None
    v_qscale: Optional[torch.Tensor] = None
    v_qzero: Optional[torch.Tensor] = None
    # fp8 / int8 scale granularity: "head" (k_scale / v_scale [Hkv]), "block"
    # (k_scales / v_scales fp32 [num_blocks, Hkv]) or "token" (fp32
    # [num_blocks, block_size, Hkv], filled by kv_append_scaled)
    scale_mode: str = "head"
    k_scales: Optional[torch.Tensor] = None
    v_scales: Optional[torch.Tensor] = None
    layout: str = "flash"

    @property
    def num_blocks(self):
        return self.k_cache.shape[0]

    @property
    def block_size(self):
        return self.k_cache.shape[3 if self.layout == "xvec" else 1]

    @property
    def num_kv_heads(self):
        return self.k_cache.shape[1 if self.layout == "xvec" else 2]

    @property
    def head_dim(self):
        if self.layout == "xvec":
            return self.k_cache.shape[2] * self.k_cache.shape[4]
        r = self.k_cache.shape[3]
        return r * 8 // 3 if self.kind == "u3" else r * 2 if self.kind == "u4" else r

    @staticmethod
    def allocate(kind: str, num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int,
                 device="cuda", k_scale=None, v_scale=None, fill=None, scale_mode: str = "head",
                 k_scales=None, v_scales=None, layout: str = "flash") -> "KVCache":
        """A cache of `kind`; fp8 / int8 caches take per-head scales (k_scale,
        v_scale), per-block scales (scale_mode "block": k_scales / v_scales
        [num_blocks, Hkv]) or per-token scales (scale_mode "token": arrays
        allocated here, written by kv_append_scaled).  layout "xvec": the
        x-vectorised storage [num_blocks, Hkv, head_dim // x, block_size, x]."""
        shape = (num_blocks, block_size, num_kv_heads)
        if layout == "xvec":
            if kind not in ("f16", "bf16", "e4m3", "e5m2", "i8"):
                raise ValueError("layout xvec applies to 16-bit and one-byte caches")
            dt = {"f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}.get(kind, torch.uint8)
            x = 16 // torch.empty((), dtype=dt).element_size()
            if head_dim % x:
                raise ValueError("head_dim must be a multiple of x = %d" % x)
            k = torch.empty((num_blocks, num_kv_heads, head_dim // x, block_size, x), dtype=dt,
                            device=device)
            v = torch.empty_like(k)
            c = KVCache(kind, k, v, k_scale=k_scale, v_scale=v_scale, scale_mode=scale_mode,
                        layout="xvec")
            if scale_mode == "block":
                c.k_scales, c.v_scales = k_scales, v_scales
            elif scale_mode == "token":
                hm = (num_blocks, num_kv_heads, block_size)
                c.k_scales = torch.ones(hm, dtype=torch.float32, device=device).permute(0, 2, 1)
                c.v_scales = torch.ones(hm, dtype=torch.float32, device=device).permute(0, 2, 1)
            if fill is not None:
                for t in (k, v):
                    t.view(torch.uint8).fill_(fill)
            return c
        elif layout != "flash":
            raise ValueError(layout)
        if kind in ("f16", "bf16"):
            dt = torch.float16 if kind == "f16" else torch.bfloat16
            k = torch.empty(shape + (head_dim,), dtype=dt, device=device)
            v = torch.empty_like(k)
            c = KVCache(kind, k, v)
        elif kind in ("e4m3", "e5m2", "i8"):
            k = torch.empty(shape + (head_dim,), dtype=torch.int8 if kind == "i8" else torch.uint8,
                            device=device)
            v = torch.empty_like(k)
            c = KVCache(kind, k, v, k_scale=k_scale, v_scale=v_scale, scale_mode=scale_mode)
            if scale_mode == "block":
                c.k_scales, c.v_scales = k_scales, v_scales
            elif scale_mode == "token":
                # head-major storage behind a [num_blocks, block_size, Hkv] view,
                # as the 3-bit metadata: a decode CTA stages its heads' runs
                hm = (num_blocks, num_kv_heads, block_size)
                c.k_scales = torch.ones(hm, dtype=torch.float32, device=device).permute(0, 2, 1)
                c.v_scales = torch.ones(hm, dtype=torch.float32, device=device).permute(0, 2, 1)
        elif kind in ("u3", "u4"):
            k = torch.empty(shape + (int(kind[1]) * head_dim // 8,), dtype=torch.uint8, device=device)
            v = torch.empty_like(k)
            # scale / zero stored head-major ([num_blocks, num_kv_heads,
            # block_size]) and seen through a [num_blocks, block_size,
            # num_kv_heads] view: a decode CTA then stages only its own heads'
            # runs of each block
            meta = (num_blocks, num_kv_heads, block_size)
            phys = [torch.empty(meta, dtype=dt, device=device)
                    for dt in (torch.float16, torch.uint8, torch.float16, torch.uint8)]
            ks_, kz_, vs_, vz_ = (t.permute(0, 2, 1) for t in phys)
            c = KVCache(kind, k, v, k_qscale=ks_, k_qzero=kz_, v_qscale=vs_, v_qzero=vz_)
        else:
            raise ValueError(kind)
        if fill is not None:
            for t in [c.k_cache, c.v_cache] + (phys if kind in ("u3", "u4") else []):
                t.view(torch.uint8).fill_(fill)
        return c

    def _struct(self) -> _Cache:
        key = [x for t in (self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.k_qscale, self.k_qzero,
                           self.v_qscale, self.v_qzero, self.k_scales, self.v_scales) if t is not None
               for x in (t.data_ptr(), t.dtype, t.shape, t.stride())]
        cached = self.__dict__.get("_cstruct")
        if cached is not None and cached[0] == key:
            return cached[1]
        s = self._build_struct()
        self.__dict__["_cstruct"] = (key, s)
        return s

    def _check_types(self):
        """The descriptors state the kind's own types: other tensors would be
        read, and written, beyond their ends."""
        width = 2 if self.kind in ("f16", "bf16") else 1
        for name, t, size in (("k_cache", self.k_cache, width), ("v_cache", self.v_cache, width),
                              ("k_qscale", self.k_qscale, 2), ("v_qscale", self.v_qscale, 2),
                              ("k_qzero", self.k_qzero, 1), ("v_qzero", self.v_qzero, 1)):
            if t is not None and t.element_size() != size:
                raise ValueError("%s of a %s cache has elements of %d bytes, got %s" % (name, self.kind, size, t.dtype))
        for name in ("k_scale", "v_scale", "k_scales", "v_scales"):
            t = getattr(self, name)
            if t is not None and t.dtype != torch.float32:
                raise ValueError("%s must be float32, got %s" % (name, t.dtype))
        for name in ("k_scale", "v_scale"):
            t = getattr(self, name)
            if t is not None and (t.numel() != self.num_kv_heads or not t.is_contiguous()):
                raise ValueError("%s must be %d contiguous numbers, one for each kv head" % (name, self.num_kv_heads))

    def _build_struct(self) -> _Cache:
        s = _Cache()
        code = {"f16": F16, "bf16": BF16, "e4m3": E4M3, "e5m2": E5M2, "i8": I8, "u3": U3, "u4": U4}[self.kind]
        self._check_types()
        if self.layout == "xvec":
            # [P, Hkv, D/x, BS, x] described as [P, BS, Hkv, D] + the piece stride
            s.k_cache = _xvec_desc(self.k_cache, code)
            s.v_cache = _xvec_desc(self.v_cache, code)
            s.chunk_stride = self.k_cache.stride(2)
        else:
            s.k_cache = _desc(self.k_cache, code)
            s.v_cache = _desc(self.v_cache, code)
        if self.kind in ("e4m3", "e5m2", "i8") and self.scale_mode == "head":
            if self.k_scale is None or self.v_scale is None:
                raise ValueError("fp8 / int8 cache needs k_scale / v_scale")
            s.k_scale = self.k_scale.data_ptr()
            s.v_scale = self.v_scale.data_ptr()
        if self.kind in ("u3", "u4"):
            s.k_qscale = _desc(self.k_qscale, F16)
            s.k_qzero = _desc(self.k_qzero, U8)
            s.v_qscale = _desc(self.v_qscale, F16)
            s.v_qzero = _desc(self.v_qzero, U8)
        s.scale_mode = SCALE_MODES[self.scale_mode]
        if self.scale_mode != "head":
            s.k_scales = _desc(self.k_scales, F32)
            s.v_scales = _desc(self.v_scales, F32)
        return s

    def tensors(self):
        return [t for t in (self.k_cache, self.v_cache, self.k_scale, self.v_scale, self.k_qscale,
                            self.k_qzero, self.v_qscale, self.v_qzero, self.k_scales,
                            self.v_scales) if t is not None]


def version() -> str:
    return lib().pkv_version().decode()


def slot_mapping(block_tables, req, pos, block_size: int, out=None, err_flag=None, stream=None):
    """slot = block_tables[req][pos // bs] * bs + pos % bs (pos < 0 -> -1), on the GPU."""
    dev = _one_device(block_tables, req, pos, out, err_flag)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return slot_mapping(block_tables, req, pos, block_size, out, err_flag)
    if out is None:
        out = torch.empty(req.shape[0], dtype=torch.int64, device=req.device)
    _check(lib().pkv_slot_mapping(_packed(block_tables), _packed(req), _packed(pos), int(block_size), _packed(out),
                                  _flag(err_flag), _raw_stream(dev)))
    return out


def kv_append(k_new, v_new, slot_mapping, cache: KVCache, err_flag=None, stream=None):
    """Scatter new K/V rows [T, Hkv, D] into the cache through slot_mapping."""
    dev = _one_device(k_new, v_new, slot_mapping, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return kv_append(k_new, v_new, slot_mapping, cache, err_flag)
    cs = cache._struct()
    _check(lib().pkv_kv_append(_packed(k_new), _packed(v_new), _packed(slot_mapping), ctypes.byref(cs),
                               _flag(err_flag), _raw_stream(dev)))


def kv_append_scaled(k_new, v_new, k_new_scale, v_new_scale, slot_mapping, cache: KVCache,
                     err_flag=None, stream=None):
    """kv_append for a cache with per-token scales: k_new_scale / v_new_scale
    fp32 [num_tokens, Hkv] are divided out and stored at the tokens' slots."""
    dev = _one_device(k_new, v_new, k_new_scale, v_new_scale, slot_mapping, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return kv_append_scaled(k_new, v_new, k_new_scale, v_new_scale, slot_mapping, cache, err_flag)
    _check(lib().pkv_kv_append_scaled(ctypes.byref(_desc(k_new)), ctypes.byref(_desc(v_new)),
                                      ctypes.byref(_desc(k_new_scale)), ctypes.byref(_desc(v_new_scale)),
                                      ctypes.byref(_desc(slot_mapping)), ctypes.byref(cache._struct()),
                                      _flag(err_flag), _raw_stream(dev)))


def _raw_stream(dev: int) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


if hasattr(torch._C, "_cuda_getCurrentRawStream"):      # the same handle, without a Stream object
    _raw_stream = torch._C._cuda_getCurrentRawStream    # noqa: F811


def kv_append_dynamic(k_new, v_new, slot_mapping, cache: KVCache, err_flag=None, stream=None):
    """kv_append for a cache with per-token scales that computes each row's
    scales, amax / (the format's largest value), and stores them with it."""
    dev = _one_device(k_new, v_new, slot_mapping, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return kv_append_dynamic(k_new, v_new, slot_mapping, cache, err_flag)
    _check(lib().pkv_kv_append_dynamic(_packed(k_new), _packed(v_new), _packed(slot_mapping),
                                       ctypes.byref(cache._struct()),
                                       _flag(err_flag), _raw_stream(dev)))


def kv_gather(cache: KVCache, slot_mapping, dtype: Optional[torch.dtype] = None, k_out=None, v_out=None,
              err_flag=None, stream=None):
    """The cached rows at slot_mapping, dequantised: (k_out, v_out), each
    [num_tokens, Hkv, D].  Without k_out / v_out they are allocated in `dtype`
    (the cache's own for 16-bit caches, else bfloat16), zero where
    slot_mapping < 0; given buffers keep those rows as they were."""
    dev = _one_device(slot_mapping, k_out, v_out, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return kv_gather(cache, slot_mapping, dtype, k_out, v_out, err_flag)
    if k_out is None or v_out is None:
        if dtype is None:
            given = k_out if k_out is not None else v_out
            dtype = given.dtype if given is not None else \
                cache.k_cache.dtype if cache.kind in ("f16", "bf16") else torch.bfloat16
        shape = (slot_mapping.shape[0], cache.num_kv_heads, cache.head_dim)
        if k_out is None:
            k_out = torch.zeros(shape, dtype=dtype, device=slot_mapping.device)
        if v_out is None:
            v_out = torch.zeros(shape, dtype=dtype, device=slot_mapping.device)
    _check(lib().pkv_kv_gather(ctypes.byref(cache._struct()), _packed(slot_mapping), _packed(k_out), _packed(v_out),
                               _flag(err_flag), _raw_stream(dev)))
    return k_out, v_out


def norm_rope(q, k, cos_sin, pos, q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
              q_out=None, k_out=None, err_flag=None, stream=None):
    """Each head row of q [T, Hq, D] and k [T, Hkv, D] normed by its own mean
    square (where a weight [D] is given) and rotated by its token's position:
    row pos[t] of cos_sin [max_pos, rot] fp32, cosines then sines.  Returns
    (q_out, k_out), allocated, with zeros where pos < 0, unless given; they
    may be q and k themselves."""
    dev = _one_device(q, k, cos_sin, pos, q_weight, k_weight, q_out, k_out, err_flag)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return norm_rope(q, k, cos_sin, pos, q_weight, k_weight, eps, interleaved, q_out, k_out, err_flag)
    if q_out is None:
        q_out = torch.zeros_like(q, memory_format=torch.contiguous_format)
    if k_out is None:
        k_out = torch.zeros_like(k, memory_format=torch.contiguous_format)
    _check(lib().pkv_norm_rope(_packed(q), _packed(k), None if q_weight is None else _packed(q_weight),
                               None if k_weight is None else _packed(k_weight), eps, _packed(cos_sin), _packed(pos),
                               int(interleaved), _packed(q_out), _packed(k_out), _flag(err_flag), _raw_stream(dev)))
    return q_out, k_out


def norm_rope_append(q, k_new, v_new, cos_sin, pos, slot_mapping, cache: KVCache, q_weight=None, k_weight=None,
                     eps: float = 1e-6, interleaved: bool = False, q_out=None, err_flag=None, stream=None):
    """norm_rope whose keys go into the cache at slot_mapping, with the values,
    in the same pass: what norm_rope and then kv_append (kv_append_dynamic for
    per-token scales) store.  Returns q_out, allocated, with zeros where pos <
    0, unless given; it may be q itself."""
    dev = _one_device(q, k_new, v_new, cos_sin, pos, slot_mapping, q_weight, k_weight, q_out, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return norm_rope_append(q, k_new, v_new, cos_sin, pos, slot_mapping, cache, q_weight, k_weight, eps,
                                    interleaved, q_out, err_flag)
    if q_out is None:
        q_out = torch.zeros_like(q, memory_format=torch.contiguous_format)
    _check(lib().pkv_norm_rope_append(_packed(q), _packed(k_new), _packed(v_new),
                                      None if q_weight is None else _packed(q_weight),
                                      None if k_weight is None else _packed(k_weight), eps, _packed(cos_sin),
                                      _packed(pos), int(interleaved), _packed(slot_mapping),
                                      ctypes.byref(cache._struct()), _packed(q_out), _flag(err_flag), _raw_stream(dev)))
    return q_out


def extend_tables(block_tables, cached_lens, new_lens, free_blocks, free_count, block_size: int,
                  num_rows: Optional[int] = None, context_lens=None, q_starts=None, req=None, pos=None,
                  slot_mapping=None, free_left=None, err_flag=None, stream=None):
    """Gives request b new_lens[b] tokens behind its cached_lens[b]: blocks from
    the top of the stack free_blocks[:free_count] into block_tables (in
    place), and the step's rows.  Returns (context_lens, q_starts, req, pos,
    slot_mapping, free_left), allocated unless given; context_lens may be
    cached_lens, free_left free_count.  The rows' outputs have num_rows
    entries, -1 behind the last request's rows."""
    dev = _one_device(block_tables, cached_lens, new_lens, free_blocks, free_count, context_lens, q_starts, req, pos,
                      slot_mapping, free_left, err_flag)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return extend_tables(block_tables, cached_lens, new_lens, free_blocks, free_count, block_size, num_rows,
                                 context_lens, q_starts, req, pos, slot_mapping, free_left, err_flag)
    if num_rows is None:
        given = next((t for t in (req, pos, slot_mapping) if t is not None), None)
        if given is None:
            raise ValueError("num_rows, or one of req, pos and slot_mapping, says how many rows there are")
        num_rows = given.shape[0]

    def out(t, n, dtype=torch.int32):
        return torch.empty(n, dtype=dtype, device=block_tables.device) if t is None else t

    batch = block_tables.shape[0]
    context_lens, q_starts, free_left = out(context_lens, batch), out(q_starts, batch + 1), out(free_left, 1)
    req, pos, slot_mapping = out(req, num_rows), out(pos, num_rows), out(slot_mapping, num_rows, torch.int64)
    _check(lib().pkv_extend_tables(_packed(block_tables), _packed(cached_lens), _packed(new_lens), _packed(free_blocks),
                                   _packed(free_count), int(block_size), _packed(context_lens), _packed(q_starts),
                                   _packed(req), _packed(pos), _packed(slot_mapping), _packed(free_left),
                                   _flag(err_flag), _raw_stream(dev)))
    return context_lens, q_starts, req, pos, slot_mapping, free_left


def trim_tables(block_tables, context_lens, keep_lens, free_blocks, free_count, block_size: int, kept_lens=None,
                free_left=None, err_flag=None, stream=None):
    """Request b keeps the first keep_lens[b] of its context_lens[b] tokens; the
    blocks that hold none of them go back on the stack free_blocks (in
    place).  Returns (kept_lens, free_left), allocated unless given; kept_lens
    may be context_lens or keep_lens, free_left free_count."""
    dev = _one_device(block_tables, context_lens, keep_lens, free_blocks, free_count, kept_lens, free_left, err_flag)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return trim_tables(block_tables, context_lens, keep_lens, free_blocks, free_count, block_size, kept_lens,
                               free_left, err_flag)
    if kept_lens is None:
        kept_lens = torch.empty(block_tables.shape[0], dtype=torch.int32, device=block_tables.device)
    if free_left is None:
        free_left = torch.empty(1, dtype=torch.int32, device=block_tables.device)
    _check(lib().pkv_trim_tables(_packed(block_tables), _packed(context_lens), _packed(keep_lens), _packed(free_blocks),
                                 _packed(free_count), int(block_size), _packed(kept_lens), _packed(free_left),
                                 _flag(err_flag), _raw_stream(dev)))
    return kept_lens, free_left


def prefill_workspace_bytes(q, cache: KVCache, block_tables) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().pkv_paged_prefill_workspace(_packed(q), ctypes.byref(cache._struct()), _packed(block_tables),
                                             ctypes.byref(n)))
    return int(n.value)


def prefill_launches(q, cache: KVCache, block_tables) -> int:
    """Kernel launches one paged_prefill call with these arguments makes."""
    n = ctypes.c_int32(0)
    _check(lib().pkv_paged_prefill_launches(_packed(q), ctypes.byref(cache._struct()), _packed(block_tables),
                                            ctypes.byref(n)))
    return int(n.value)


def paged_prefill(q, cache: KVCache, block_tables, q_starts, context_lens,
                  sm_scale: Optional[float] = None, out=None, workspace=None, err_flag=None, stream=None):
    """Causal attention of packed new tokens q [T, Hq, D] over the cache:
    sequence b owns rows q_starts[b] .. q_starts[b + 1] - 1, the last tokens of
    its context_lens[b] cached ones (their K/V are appended before).  Without
    `out` one is allocated, zero in the rows that no sequence owns."""
    dev = _one_device(q, block_tables, q_starts, context_lens, out, workspace, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return paged_prefill(q, cache, block_tables, q_starts, context_lens, sm_scale, out, workspace, err_flag)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(q.shape[-1])
    if out is None:
        out = torch.zeros_like(q, memory_format=torch.contiguous_format)
    if workspace is None:
        workspace = torch.empty(prefill_workspace_bytes(q, cache, block_tables), dtype=torch.uint8, device=q.device)
    _check(lib().pkv_paged_prefill(_packed(q), ctypes.byref(cache._struct()), _packed(block_tables),
                                   _packed(q_starts), _packed(context_lens), sm_scale, _packed(out),
                                   *_room(workspace, "workspace"),
                                   _flag(err_flag), _raw_stream(dev)))
    return out


def decode_workspace_bytes(q, cache: KVCache, block_tables, num_splits: int = 0) -> int:
    n = ctypes.c_size_t(0)
    cs = cache._struct()
    _check(lib().pkv_paged_decode_workspace(_packed(q), ctypes.byref(cs), _packed(block_tables), int(num_splits),
                                            ctypes.byref(n)))
    return int(n.value)


def decode_launches(q, cache: KVCache, block_tables, num_splits: int = 0) -> int:
    """Kernel launches one paged_decode call with these arguments makes."""
    n = ctypes.c_int32(0)
    _check(lib().pkv_paged_decode_launches(ctypes.byref(_desc(q)), ctypes.byref(cache._struct()),
                                           ctypes.byref(_desc(block_tables)), int(num_splits),
                                           ctypes.byref(n)))
    return int(n.value)


def paged_decode(q, cache: KVCache, block_tables, context_lens, sm_scale: Optional[float] = None,
                 out=None, num_splits: int = 0, workspace=None, err_flag=None, stream=None):
    """softmax(sm_scale * q . K^T) V over each sequence's paged context."""
    dev = _one_device(q, block_tables, context_lens, out, workspace, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return paged_decode(q, cache, block_tables, context_lens, sm_scale, out, num_splits, workspace, err_flag)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(q.shape[-1])
    if out is None:
        out = torch.empty_like(q)
    cs = cache._struct()
    if workspace is None:
        need = decode_workspace_bytes(q, cache, block_tables, num_splits)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr, ws_n = _room(workspace, "workspace")
    _check(lib().pkv_paged_decode(_packed(q), ctypes.byref(cs), _packed(block_tables), _packed(context_lens),
                                  float(sm_scale), _packed(out), int(num_splits), ws_ptr, ws_n, _flag(err_flag),
                                  _raw_stream(dev)))
    return out


def decode_step(k_new, v_new, req, pos, q, cache: KVCache, block_tables, context_lens,
                sm_scale: Optional[float] = None, out=None, slots=None, num_splits: int = 0,
                workspace=None, err_flag=None, stream=None):
    """slot_mapping + kv_append + paged_decode in one library call (see
    pkv_decode_step in pkv.h); returns out.  `slots` (int64 [num_tokens])
    receives the slot mapping."""
    dev = _one_device(k_new, v_new, req, pos, q, block_tables, context_lens, out, slots, workspace, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return decode_step(k_new, v_new, req, pos, q, cache, block_tables, context_lens, sm_scale, out, slots,
                               num_splits, workspace, err_flag)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(q.shape[-1])
    if out is None:
        out = torch.empty_like(q)
    if slots is None:
        slots = torch.empty(req.shape[0], dtype=torch.int64, device=q.device)
    cs = cache._struct()
    if workspace is None:
        need = decode_workspace_bytes(q, cache, block_tables, num_splits)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr, ws_n = _room(workspace, "workspace")
    _check(lib().pkv_decode_step(_packed(k_new), _packed(v_new), _packed(req), _packed(pos), _packed(slots), _packed(q),
                                 ctypes.byref(cs), _packed(block_tables), _packed(context_lens), float(sm_scale),
                                 _packed(out), int(num_splits), ws_ptr, ws_n, _flag(err_flag), _raw_stream(dev)))
    return out


def paged_decode_noalloc(q, cache: KVCache, block_tables, context_lens,
                         sm_scale: Optional[float] = None, out=None, num_splits: int = 0,
                         err_flag=None, stream=None):
    """paged_decode without a caller workspace: the split-K scratch is the
    library's fixed device array (see pkv_paged_decode_noalloc in pkv.h)."""
    dev = _one_device(q, block_tables, context_lens, out, err_flag, *cache.tensors())
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return paged_decode_noalloc(q, cache, block_tables, context_lens, sm_scale, out, num_splits, err_flag)
    if sm_scale is None:
        sm_scale = 1.0 / math.sqrt(q.shape[-1])
    if out is None:
        out = torch.empty_like(q)
    cs = cache._struct()
    _check(lib().pkv_paged_decode_noalloc(ctypes.byref(_desc(q)), ctypes.byref(cs),
                                          ctypes.byref(_desc(block_tables)),
                                          ctypes.byref(_desc(context_lens)), float(sm_scale),
                                          ctypes.byref(_desc(out)), int(num_splits),
                                          _flag(err_flag), _raw_stream(dev)))
    return out


def pack3(values, packed=None, stream=None):
    """uint8 [n*8] codes -> uint8 [n*3] packed bytes."""
    dev = _one_device(values, packed)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return pack3(values, packed)
    n = values.numel() // 8
    if packed is None:
        packed = torch.empty(n * 3, dtype=torch.uint8, device=values.device)
    _check(lib().pkv_pack3(_room(values, "values")[0], _room(packed, "packed", 3 * n)[0], n, _raw_stream(dev)))
    return packed


def unpack3(packed, values=None, stream=None):
    """uint8 [n*3] packed bytes -> uint8 [n*8] codes."""
    dev = _one_device(packed, values)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return unpack3(packed, values)
    n = packed.numel() // 3
    if values is None:
        values = torch.empty(n * 8, dtype=torch.uint8, device=packed.device)
    _check(lib().pkv_unpack3(_room(packed, "packed")[0], _room(values, "values", 8 * n)[0], n, _raw_stream(dev)))
    return values


def unpack3_words(words, values=None, stream=None):
    """int32/uint32 words [m*3] (same bytes as packed octets) -> uint8 [m*32]."""
    dev = _one_device(words, values)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return unpack3_words(words, values)
    m = words.numel() // 3
    if values is None:
        values = torch.empty(m * 32, dtype=torch.uint8, device=words.device)
    _check(lib().pkv_unpack3_words(_room(words, "words", 12 * m)[0], _room(values, "values", 32 * m)[0], m, _raw_stream(dev)))
    return values


def copy_peak(src, dst, stream=None):
    """16-byte vectorised copy of src's bytes into dst (bandwidth yardstick)."""
    dev = _one_device(src, dst)
    there = _elsewhere(dev, stream)
    if there is not None:
        with there:
            return copy_peak(src, dst)
    at, nbytes = _room(src, "src")
    _check(lib().pkv_copy_peak(at, _room(dst, "dst", nbytes)[0], nbytes, _raw_stream(dev)))
