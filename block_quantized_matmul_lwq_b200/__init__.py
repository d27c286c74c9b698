"""Python binding of liblwq.so, the block-quantized matmul for B200 (sm_100a).

Argument marshalling only: every step of y = x . dequant(Wq)^T runs in the
library's CUDA kernels.  The names mirror the C ABI in include/lwq.h.
Pointer arguments accept plain integers or objects with ``data_ptr()`` (torch
tensors); ``stream`` accepts an integer cudaStream_t, an object with a
``cuda_stream`` attribute (torch.cuda.Stream), or None (legacy default stream).
The library is loaded on first use; any call fails loudly (ImportError)
when it has not been built -- there is no fallback of any kind.
"""

from __future__ import annotations

import ctypes
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblwq.so")

# codes (include/lwq.h)
LWQ_Q8_0, LWQ_Q4_0, LWQ_Q4_K, LWQ_Q6_K, LWQ_Q5_K, LWQ_Q2_K = 1, 2, 3, 4, 5, 6
LWQ_ACT_F32, LWQ_ACT_F16, LWQ_ACT_BF16 = 0x000, 0x100, 0x200
LWQ_FLAG_OVERLAP = 0x1000   # weights constant: allow programmatic dependent launch
LWQ_FLAG_ACT_I8 = 0x2000    # int8 activation blocks of 32 (integer block dot products)
LWQ_FLAG_OUT16 = 0x4000     # paged attention: out in the cache's 16-bit type
LWQ_ROPE_HALF, LWQ_ROPE_PAIRS = 0, 1
LWQ_OK = 0
LWQ_ERR_INVALID_ARG = 1
LWQ_ERR_UNSUPPORTED = 2
LWQ_ERR_MISALIGNED = 3
LWQ_ERR_NOT_INITIALIZED = 4
LWQ_ERR_WORKSPACE_TOO_SMALL = 5
LWQ_ERR_CUDA = 6
LWQ_ERR_DEVICE_TIMEOUT = 7
LWQ_ERR_BAD_PAGE = 8
STATUS = {0: "LWQ_OK", 1: "LWQ_ERR_INVALID_ARG", 2: "LWQ_ERR_UNSUPPORTED", 3: "LWQ_ERR_MISALIGNED",
          4: "LWQ_ERR_NOT_INITIALIZED", 5: "LWQ_ERR_WORKSPACE_TOO_SMALL", 6: "LWQ_ERR_CUDA",
          7: "LWQ_ERR_DEVICE_TIMEOUT", 8: "LWQ_ERR_BAD_PAGE"}
WEIGHT_FORMATS = {"q8_0": LWQ_Q8_0, "q4_0": LWQ_Q4_0, "q4_k": LWQ_Q4_K, "q6_k": LWQ_Q6_K, "q5_k": LWQ_Q5_K,
                  "q2_k": LWQ_Q2_K}
ACT_DTYPES = {"f32": LWQ_ACT_F32, "f16": LWQ_ACT_F16, "bf16": LWQ_ACT_BF16}

# every symbol the header declares
EXPORTS = ["lwq_row_bytes", "lwq_workspace_size", "lwq_init", "lwq_shutdown", "lwq_matmul",
           "lwq_select_config", "lwq_matmul_config", "lwq_status_string", "lwq_get_device_error",
           "lwq_selftest_timeout", "lwq_last_launch_count", "lwq_version", "lwq_matmul_noalloc",
           "lwq_attention_workspace_size", "lwq_attention_decode", "lwq_rope_init", "lwq_kv_append",
           "lwq_attention_paged_workspace_size", "lwq_attention_paged",
           "lwq_attention_prefill_workspace_size", "lwq_attention_prefill"]


class LwqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({lwq_status_string(status)})")


class lwq_config(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("warps", ctypes.c_int), ("stages", ctypes.c_int),
                ("splits", ctypes.c_int), ("ctas", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("tile_m", ctypes.c_int), ("reserved", ctypes.c_int * 5)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f, _ in self._fields_ if f != "reserved"}


class lwq_paged(ctypes.Structure):
    """The paged key/value cache and one batch of sequences (include/lwq.h).  Keeps the objects it was given
    alive; the tensors' contents (page tables, lengths) may change between calls."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("tables", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("prefix", ctypes.c_void_p), ("prefix_len", ctypes.c_int),
                ("dtype", ctypes.c_int), ("B", ctypes.c_int), ("Hkv", ctypes.c_int), ("D", ctypes.c_int),
                ("page", ctypes.c_int), ("max_pages", ctypes.c_int), ("num_pages", ctypes.c_int)]

    def __init__(self, act: int, k, v, tables, lens, *, B: int, Hkv: int, D: int, page: int, max_pages: int,
                 num_pages: int, prefix=None, prefix_len: int = 0):
        n = num_pages * Hkv * page * D
        super().__init__(_tensor(k, "k", act, n), _tensor(v, "v", act, n), _tensor(tables, "tables", _INDEX, B * max_pages),
                         _tensor(lens, "lens", _INDEX, B),
                         _tensor(prefix, "prefix", _INDEX, -(-prefix_len // max(page, 1))),
                         prefix_len, act, B, Hkv, D, page, max_pages, num_pages)
        self.owners = (k, v, tables, lens, prefix)
        on = {p.get_device() for p in self.owners if hasattr(p, "get_device")}
        if len(on) > 1:
            raise ValueError(f"the cache's tensors are on several devices: {sorted(on)}")
        self.device = on.pop() if on else None

    at = property(ctypes.addressof)
    owners, device = (), None       # of a copied descriptor: its tensors are not known


class lwq_rope(ctypes.Structure):
    """The rotation of lwq_kv_append (include/lwq.h); filled by lwq_rope_init."""

    _fields_ = [("rot_dim", ctypes.c_int), ("layout", ctypes.c_int), ("axes", ctypes.c_int),
                ("reserved", ctypes.c_int), ("turn", ctypes.c_uint64 * 64), ("axis", ctypes.c_uint8 * 64)]

    at = property(ctypes.addressof)


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m block_quantized_matmul_lwq_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(LIB_PATH)
    c = ctypes
    vp, i = c.c_void_p, c.c_int
    lib.lwq_row_bytes.restype, lib.lwq_row_bytes.argtypes = c.c_size_t, [i, c.c_int64]
    lib.lwq_workspace_size.restype, lib.lwq_workspace_size.argtypes = c.c_size_t, [i, i, i, i]
    lib.lwq_init.restype, lib.lwq_init.argtypes = i, [vp, c.c_size_t]
    lib.lwq_shutdown.restype, lib.lwq_shutdown.argtypes = i, []
    lib.lwq_matmul.restype, lib.lwq_matmul.argtypes = i, [i, vp, vp, vp, i, i, i, vp]
    lib.lwq_select_config.restype = i
    lib.lwq_select_config.argtypes = [i, i, i, i, c.POINTER(lwq_config)]
    lib.lwq_matmul_config.restype = i
    lib.lwq_matmul_config.argtypes = [i, vp, vp, vp, i, i, i, c.POINTER(lwq_config), vp]
    lib.lwq_status_string.restype, lib.lwq_status_string.argtypes = c.c_char_p, [i]
    lib.lwq_get_device_error.restype, lib.lwq_get_device_error.argtypes = i, []
    lib.lwq_selftest_timeout.restype, lib.lwq_selftest_timeout.argtypes = i, [c.c_uint, vp]
    lib.lwq_last_launch_count.restype, lib.lwq_last_launch_count.argtypes = i, []
    lib.lwq_version.restype, lib.lwq_version.argtypes = i, []
    lib.lwq_matmul_noalloc.restype, lib.lwq_matmul_noalloc.argtypes = i, [i, vp, vp, vp, i, i, i, vp]
    lib.lwq_attention_workspace_size.restype = c.c_size_t
    lib.lwq_attention_workspace_size.argtypes = [i, i, i, i, i]
    lib.lwq_attention_decode.restype = i
    lib.lwq_attention_decode.argtypes = [i, vp, vp, vp, vp, vp, i, i, i, i, i, c.c_float, vp]
    pc, pr, i64 = vp, vp, c.c_int64   # structs by address (lwq_paged.at, lwq_rope.at): cheaper per call than byref
    lib.lwq_rope_init.restype = i
    lib.lwq_rope_init.argtypes = [c.POINTER(lwq_rope), i, i, c.c_double, c.POINTER(c.c_double), i, c.POINTER(i)]
    lib.lwq_kv_append.restype = i
    lib.lwq_kv_append.argtypes = [pc, pr, i, vp, i64, vp, i64, vp, i64, vp, vp, vp, i, i, vp]
    lib.lwq_attention_paged_workspace_size.restype = c.c_size_t
    lib.lwq_attention_paged_workspace_size.argtypes = [pc, i]
    lib.lwq_attention_paged.restype = i
    lib.lwq_attention_paged.argtypes = [pc, i, vp, vp, i, c.c_float, vp]
    lib.lwq_attention_prefill_workspace_size.restype = c.c_size_t
    lib.lwq_attention_prefill_workspace_size.argtypes = [pc, i, i]
    lib.lwq_attention_prefill.restype = i
    lib.lwq_attention_prefill.argtypes = [pc, i, vp, vp, vp, i, i, c.c_float, vp]
    return lib


_lib_handle = None


def lib() -> ctypes.CDLL:
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _load()
    return _lib_handle


class _LazyLib:
    def __getattr__(self, name):
        f = getattr(lib(), name)
        setattr(self, name, f)   # later calls find it as a plain attribute
        return f


_lib = _LazyLib()


def _ptr(p) -> int:
    if p is None:
        return 0
    if isinstance(p, int):
        return p
    return int(p.data_ptr())


_INDEX = "index"            # what _element_types has int32 arrays under, beside the activation codes
_element_types = {}


def _types(kind):
    """The element types that a tensor of this kind (an activation code, or _INDEX) may have; None for a code that there is
    not (the call itself refuses it).  Integers of 16 bits pass for 16-bit floats: the bits as they are."""
    if not _element_types:
        t = sys.modules["torch"]
        bits = {getattr(t, n) for n in ("int16", "uint16") if hasattr(t, n)}
        _element_types.update({LWQ_ACT_F32: {t.float32}, LWQ_ACT_F16: bits | {t.float16},
                               LWQ_ACT_BF16: bits | {t.bfloat16},
                               _INDEX: {getattr(t, n) for n in ("int32", "uint32") if hasattr(t, n)}})
    return _element_types.get(kind)


def _tensor(p, name: str, kind, count: int = 0, device=None) -> int:
    """_ptr of a tensor that a kernel will index: refused where it is on the host or on another device than the cache's,
    has another element type than the call's, or, given a count, has fewer elements or is not contiguous."""
    if p is None or p.__class__ is int:
        return p or 0
    try:
        on, types = p.get_device(), _element_types.get(kind) or _types(kind)
        if ((on == device if device is not None else on >= 0) and (types is None or p.dtype in types)
                and (not count or p.numel() >= count and p.is_contiguous())):
            return p.data_ptr()
    except AttributeError:      # a pointer of another kind
        return _ptr(p)
    raise ValueError(f"{name}: {f'{count} elements in one piece' if count else 'elements'} of "
                     f"{' or '.join(sorted(str(t) for t in _types(kind) or ()))} on "
                     f"{'the GPU' if device is None else f'cuda:{device}'} are needed, not {tuple(p.shape)} of {p.dtype} on "
                     f"{p.device} with strides {p.stride()}")


def _reaches(*rows) -> None:
    """Each (tensor, name, pointer, bytes from there) ends within its tensor's memory (mostly one tensor's for all)."""
    base = end = 0
    for p, name, at, nbytes in rows:
        if at and not (base <= at and at + nbytes <= end) and hasattr(p, "untyped_storage"):
            s = p.untyped_storage()
            base = s.data_ptr()
            end = base + s.nbytes()
            if at + nbytes > end:
                raise ValueError(f"{name}: its rows end {at + nbytes - end} bytes behind the tensor's memory")


_current = None                 # torch.cuda.current_device


def _current_device(cache) -> None:
    """The device of the cache's tensors is the current one, on which the call launches."""
    global _current
    if cache.device is not None:
        if _current is None:
            _current = sys.modules["torch"].cuda.current_device
        if _current() != cache.device:
            raise ValueError(f"the cache is on cuda:{cache.device}, the current device is cuda:{_current()}")


def _stream(s) -> int:
    if s is None:
        return 0
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _check(rc: int, where: str) -> int:
    if rc != LWQ_OK:
        raise LwqError(rc, where)
    return rc


def fmt_code(weights: str, act: str) -> int:
    """``fmt`` for the C ABI from names: weights in q8_0/q4_0/q4_k/q6_k/q5_k/q2_k, act in f32/f16/bf16."""
    return WEIGHT_FORMATS[weights] | ACT_DTYPES[act]


def lwq_status_string(status: int) -> str:
    return _lib.lwq_status_string(status).decode()


def lwq_row_bytes(fmt: int, K: int) -> int:
    return _lib.lwq_row_bytes(fmt, K)


def lwq_workspace_size(fmt: int, max_M: int, max_N: int, max_K: int) -> int:
    return _lib.lwq_workspace_size(fmt, max_M, max_N, max_K)


def lwq_init(workspace, nbytes: int) -> None:
    _check(_lib.lwq_init(_ptr(workspace), nbytes), "lwq_init")


def lwq_shutdown() -> None:
    _check(_lib.lwq_shutdown(), "lwq_shutdown")


def lwq_matmul(fmt: int, Wq, x, y, M: int, N: int, K: int, stream=None) -> None:
    _check(_lib.lwq_matmul(fmt, _ptr(Wq), _ptr(x), _ptr(y), M, N, K, _stream(stream)), "lwq_matmul")


def lwq_select_config(fmt: int, M: int, N: int, K: int) -> lwq_config:
    cfg = lwq_config()
    _check(_lib.lwq_select_config(fmt, M, N, K, ctypes.byref(cfg)), "lwq_select_config")
    return cfg


def lwq_matmul_config(fmt: int, Wq, x, y, M: int, N: int, K: int, cfg: lwq_config, stream=None) -> None:
    _check(_lib.lwq_matmul_config(fmt, _ptr(Wq), _ptr(x), _ptr(y), M, N, K, ctypes.byref(cfg), _stream(stream)),
           "lwq_matmul_config")


def lwq_get_device_error() -> int:
    """LWQ_OK, LWQ_ERR_DEVICE_TIMEOUT or LWQ_ERR_BAD_PAGE (and clears it); synchronize first."""
    return _lib.lwq_get_device_error()


def lwq_selftest_timeout(timeout_us: int, stream=None) -> None:
    _check(_lib.lwq_selftest_timeout(timeout_us, _stream(stream)), "lwq_selftest_timeout")


def lwq_last_launch_count() -> int:
    return _lib.lwq_last_launch_count()


def lwq_version() -> int:
    return _lib.lwq_version()


def lwq_matmul_noalloc(fmt: int, Wq, x, y, M: int, N: int, K: int, stream=None) -> None:
    """lwq_matmul for callers that cannot allocate: no workspace, static 4 MiB scratch (see include/lwq.h)."""
    _check(_lib.lwq_matmul_noalloc(fmt, _ptr(Wq), _ptr(x), _ptr(y), M, N, K, _stream(stream)),
           "lwq_matmul_noalloc")


def lwq_attention_workspace_size(B: int, H: int, Hkv: int, Lmax: int, D: int) -> int:
    return _lib.lwq_attention_workspace_size(B, H, Hkv, Lmax, D)


def lwq_attention_decode(act: int, q, k, v, seq_lens, out, B: int, H: int, Hkv: int, Lmax: int, D: int,
                         scale: float, stream=None) -> None:
    """Decode attention through the C ABI (act: LWQ_ACT_F16 or LWQ_ACT_BF16; seq_lens may be None)."""
    _check(_lib.lwq_attention_decode(act, _ptr(q), _ptr(k), _ptr(v), _ptr(seq_lens), _ptr(out), B, H, Hkv, Lmax, D,
                                     float(scale), _stream(stream)), "lwq_attention_decode")


def lwq_rope_init(rot_dim: int, base: float = 10000.0, layout: int = LWQ_ROPE_HALF, inv_freq=None,
                  sections=None) -> lwq_rope:
    """A rotation of the first rot_dim elements of each head; sections: pairs per position axis (None: one axis);
    inv_freq: rot_dim // 2 frequencies in place of base ** (-2 i / rot_dim)."""
    if inv_freq is not None and len(inv_freq) != rot_dim // 2:
        raise ValueError(f"inv_freq needs {rot_dim // 2} frequencies, not {len(inv_freq)}")
    rope = lwq_rope()
    freq = None if inv_freq is None else (ctypes.c_double * len(inv_freq))(*[float(f) for f in inv_freq])
    sec = None if sections is None else (ctypes.c_int * len(sections))(*sections)
    _check(_lib.lwq_rope_init(ctypes.byref(rope), rot_dim, layout, float(base), freq,
                              1 if sections is None else len(sections), sec), "lwq_rope_init")
    return rope


def lwq_kv_append(cache: lwq_paged, rope, src: int, q, ldq: int, k, ldk: int, v, ldv: int, q_out, T: int, H: int,
                  cu_tokens=None, positions=None, stream=None) -> None:
    """Rotate q and k by position (rope None: not) and store k and v in the cache (see include/lwq.h)."""
    on, D, last, es = cache.device, cache.D, T - 1, 4 if src == LWQ_ACT_F32 else 2
    n = cache.Hkv * D
    qp, kp, vp = _tensor(q, "q", src, 0, on), _tensor(k, "k", src, 0, on), _tensor(v, "v", src, 0, on)
    _reaches((v, "v", vp, (last * ldv + n) * es), (k, "k", kp, (last * ldk + n) * es),
             (q, "q", qp, (last * ldq + H * D) * es))
    out = _tensor(q_out, "q_out", cache.dtype, T * H * D, on)
    cu = _tensor(cu_tokens, "cu_tokens", _INDEX, cache.B + 1, on)
    pos = _tensor(positions, "positions", _INDEX, T * (1 if rope is None else rope.axes), on)
    _current_device(cache)
    _check(_lib.lwq_kv_append(cache.at, None if rope is None else rope.at, src, qp, ldq, kp, ldk, vp, ldv, out, cu, pos, T,
                              H, _stream(stream)), "lwq_kv_append")


def lwq_attention_paged_workspace_size(cache: lwq_paged, H: int) -> int:
    return _lib.lwq_attention_paged_workspace_size(cache.at, H)


def lwq_attention_paged(cache: lwq_paged, q, out, H: int, scale: float, flags: int = 0, stream=None) -> None:
    """Decode attention, one query token per sequence, over the paged cache and its shared prefix."""
    n, on = cache.B * H * cache.D, cache.device
    ptrs = (_tensor(q, "q", cache.dtype, n, on),
            _tensor(out, "out", cache.dtype if flags & LWQ_FLAG_OUT16 else LWQ_ACT_F32, n, on))
    _current_device(cache)
    _check(_lib.lwq_attention_paged(cache.at, flags, *ptrs, H, float(scale), _stream(stream)), "lwq_attention_paged")


def lwq_attention_prefill_workspace_size(cache: lwq_paged, T: int, H: int) -> int:
    return _lib.lwq_attention_prefill_workspace_size(cache.at, T, H)


def lwq_attention_prefill(cache: lwq_paged, q, out, cu_tokens, T: int, H: int, scale: float, flags: int = 0,
                          stream=None) -> None:
    """Causal attention of the batch's new tokens over the cache that already holds them."""
    n, on = T * H * cache.D, cache.device
    ptrs = (_tensor(q, "q", cache.dtype, n, on),
            _tensor(out, "out", cache.dtype if flags & LWQ_FLAG_OUT16 else LWQ_ACT_F32, n, on),
            _tensor(cu_tokens, "cu_tokens", _INDEX, cache.B + 1, on))
    _current_device(cache)
    _check(_lib.lwq_attention_prefill(cache.at, flags, *ptrs, T, H, float(scale), _stream(stream)),
           "lwq_attention_prefill")
