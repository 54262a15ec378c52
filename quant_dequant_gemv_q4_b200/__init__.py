"""B200-native block-quantized dequant GEMV: y[N,B] = dequant(W[N,K]) . x[K,B], and the operators between
the GEMVs of a decode step: head norms with the position rotation, a paged 4-bit key/value cache with its
append and its attention, and sampling.

A thin ctypes binding over ``libqg.so`` (built from ``csrc/`` for sm_100a by ``build.py``): every
function here only marshals arguments and calls the C ABI of ``include/qg.h`` under the same name;
all computation runs in the library's CUDA kernels.  There is no CPU fallback: if the library is
missing, every call raises.

Pointers may be given as torch tensors (their ``data_ptr()``) or plain integers; ``stream=None``
means torch's current CUDA stream.  The operators around the GEMVs take torch CUDA tensors and read
sizes and strides from them.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

QG_FMT_Q8_0 = 8
QG_FMT_Q4_K = 12
QG_FMT_Q5_K = 13
QG_FMT_Q6_K = 14
QG_FMT_IQ4_XS = 23

QG_VARIANT_AUTO = 0
QG_VARIANT_DIRECT = 1
QG_VARIANT_FACTORED = 2
QG_VARIANT_GENERIC = 3
QG_VARIANT_TENSOR = 4
QG_VARIANT_TCGEN05 = 5

QG_OK = 0
QG_ERR_NULL = 1
QG_ERR_FMT = 2
QG_ERR_SHAPE = 3
QG_ERR_BATCH = 4
QG_ERR_ALIGN = 5
QG_ERR_CUDA = 6
QG_ERR_NOMEM = 7
QG_ERR_RANGE = 8
QG_ERR_VARIANT = 9
QG_ERR_SCRATCH = 10

QG_TYPE_F32 = 0
QG_TYPE_F16 = 1
QG_ROPE_HALVES = 0
QG_ROPE_ADJACENT = 1

# bytes of the fixed device array qg_gemv_noalloc uses as scratch
QG_NOALLOC_SCRATCH_BYTES = 8 << 20

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqg.so")
_lib = None


class qg_heads(ctypes.Structure):
    """A [tokens][heads][dims] view of device memory, strides in elements."""
    _fields_ = [("ptr", ctypes.c_void_p), ("token", ctypes.c_int64), ("head", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("type", ctypes.c_int32)]


class QgError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


def lib() -> ctypes.CDLL:
    """Load libqg.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libqg.so not found at {LIB_PATH}; build it with "
                "`python -m quant_dequant_gemv_q4_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        L.qg_weight_bytes.argtypes = [I, I64, I64]
        L.qg_weight_bytes.restype = SZ
        L.qg_gemv.argtypes = [P, I, I64, I64, P, I, P, P]
        L.qg_gemv.restype = I
        L.qg_gemv_variant.argtypes = [P, I, I64, I64, P, I, P, P, I]
        L.qg_gemv_variant.restype = I
        L.qg_gemv_noalloc.argtypes = [P, I, I64, I64, P, I, P, P]
        L.qg_gemv_noalloc.restype = I
        L.qg_gemv_host.argtypes = [P, I, I64, I64, P, I, P, P]
        L.qg_gemv_host.restype = I
        L.qg_gemv_gate_up_silu.argtypes = [P, P, I, I64, I64, P, I, P, P]
        L.qg_gemv_gate_up_silu.restype = I
        L.qg_gemv_residual.argtypes = [P, I, I64, I64, P, I, P, P, P]
        L.qg_gemv_residual.restype = I
        L.qg_dequant_f32.argtypes = [P, I, I64, I64, P, P]
        L.qg_dequant_f32.restype = I
        L.qg_pack_reference.argtypes = [I, I64, I64, P, P, P, P, P, P]
        L.qg_pack_reference.restype = I
        L.qg_last_variant.argtypes = []
        L.qg_last_variant.restype = I
        L.qg_last_splits.argtypes = []
        L.qg_last_splits.restype = I
        L.qg_plan.argtypes = [I, I64, I64, I, I, I, I, I, ctypes.POINTER(I64)]
        L.qg_plan.restype = I
        L.qg_device_error.argtypes = [P, ctypes.POINTER(I)]
        L.qg_device_error.restype = I
        L.qg_noalloc_device_error.argtypes = [P, ctypes.POINTER(I)]
        L.qg_noalloc_device_error.restype = I
        L.qg_hbm_copy.argtypes = [P, P, SZ, P]
        L.qg_hbm_copy.restype = I
        L.qg_hbm_read.argtypes = [P, SZ, P, P]
        L.qg_hbm_read.restype = I
        F, DBL, HP = ctypes.c_float, ctypes.c_double, ctypes.c_void_p  # (HP: a qg_heads by reference, or its bytes)
        L.qg_qk_norm_rope.argtypes = [HP, HP, I64, I, I, I, P, P, DBL, P, P, I, I, HP, HP, P]
        L.qg_qk_norm_rope.restype = I
        L.qg_kv4_bytes.argtypes = [I64, I, I, I]
        L.qg_kv4_bytes.restype = SZ
        L.qg_kv4_append.argtypes = [HP, HP, I64, I, I, P, DBL, P, P, I, I, P, P, I64, I, P]
        L.qg_kv4_append.restype = I
        L.qg_kv4_read.argtypes = [P, I64, I, I, I, P, I64, HP, HP, P]
        L.qg_kv4_read.restype = I
        L.qg_attn_kv4_workspace.argtypes = [I, I, I, I]
        L.qg_attn_kv4_workspace.restype = SZ
        L.qg_attn_kv4.argtypes = [HP, I64, I, P, I, I, I, I, P, I64, I, P, I, P, F, HP, P, SZ, P]
        L.qg_attn_kv4.restype = I
        L.qg_sample_workspace.argtypes = [I64, I64, I64]
        L.qg_sample_workspace.restype = SZ
        L.qg_sample.argtypes = [P, I64, I64, I64, I64, P, P, P, P, P, P, P, SZ, P]
        L.qg_sample.restype = I
        L.qg_status_string.argtypes = [I]
        L.qg_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _ptr(a) -> int | None:
    if a is None:
        return None
    if isinstance(a, int):
        return a
    if hasattr(a, "data_ptr"):
        return a.data_ptr()
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    raise TypeError(f"cannot take a pointer of {type(a)}")


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ok(rc: int, what: str) -> None:
    if rc != QG_OK:
        raise QgError(rc, what)


def status_string(status: int) -> str:
    return lib().qg_status_string(int(status)).decode()


def qg_status_string(status: int) -> str:
    return status_string(status)


def qg_weight_bytes(fmt: int, N: int, K: int) -> int:
    return int(lib().qg_weight_bytes(int(fmt), int(N), int(K)))


def qg_gemv(W, fmt: int, N: int, K: int, x, B: int, y, stream=None) -> None:
    """Enqueue y = dequant(W) . x (all device pointers / CUDA tensors)."""
    _ok(lib().qg_gemv(_ptr(W), int(fmt), int(N), int(K), _ptr(x), int(B), _ptr(y),
                      _stream(stream)), "qg_gemv")


def qg_gemv_host(W, fmt: int, N: int, K: int, x_host, B: int, y_host, stream=None) -> None:
    """Enqueue x_host -> device, y = dequant(W) . x, y -> y_host (W on the device; x_host, y_host
    host memory: pinned CPU tensors or numpy arrays).  y_host is valid after the stream syncs."""
    _ok(lib().qg_gemv_host(_ptr(W), int(fmt), int(N), int(K), _ptr(x_host), int(B), _ptr(y_host),
                           _stream(stream)), "qg_gemv_host")


def qg_gemv_variant(W, fmt: int, N: int, K: int, x, B: int, y, stream=None,
                    variant: int = QG_VARIANT_AUTO) -> None:
    _ok(lib().qg_gemv_variant(_ptr(W), int(fmt), int(N), int(K), _ptr(x), int(B), _ptr(y),
                              _stream(stream), int(variant)), "qg_gemv_variant")


def qg_gemv_gate_up_silu(Wg, Wu, fmt: int, N: int, K: int, x, B: int, h, stream=None) -> None:
    """h = silu(dequant(Wg) . x) * (dequant(Wu) . x) in one launch (fp32 h [N][B])."""
    _ok(lib().qg_gemv_gate_up_silu(_ptr(Wg), _ptr(Wu), int(fmt), int(N), int(K), _ptr(x), int(B),
                                   _ptr(h), _stream(stream)), "qg_gemv_gate_up_silu")


def qg_gemv_residual(W, fmt: int, N: int, K: int, x, B: int, r, y, stream=None) -> None:
    """y = dequant(W) . x + r (r may be y itself: in-place residual update)."""
    _ok(lib().qg_gemv_residual(_ptr(W), int(fmt), int(N), int(K), _ptr(x), int(B), _ptr(r), _ptr(y),
                               _stream(stream)), "qg_gemv_residual")


def qg_gemv_noalloc(W, fmt: int, N: int, K: int, x, B: int, y, stream=None) -> None:
    """qg_gemv that allocates nothing: scratch in the library's fixed device array (for callers
    that cannot let the library call cudaMalloc; calls that overlap on the GPU race)."""
    _ok(lib().qg_gemv_noalloc(_ptr(W), int(fmt), int(N), int(K), _ptr(x), int(B), _ptr(y),
                              _stream(stream)), "qg_gemv_noalloc")


def qg_dequant_f32(W, fmt: int, N: int, K: int, out, stream=None) -> None:
    _ok(lib().qg_dequant_f32(_ptr(W), int(fmt), int(N), int(K), _ptr(out), _stream(stream)),
        "qg_dequant_f32")


def qg_pack_reference(fmt: int, N: int, K: int, d, dmin, sc, m, q) -> np.ndarray:
    """Host bit packer: fields (numpy) -> uint8 tensor bytes (Q6_K: sc are the int8 group scales,
    q the stored values 0..63; IQ4_XS: sc are the stored 6-bit sub-block scales, q the codebook
    indices; dmin, m unused for both)."""
    out = np.empty(qg_weight_bytes(fmt, N, K), dtype=np.uint8)
    d = np.ascontiguousarray(d, dtype=np.uint16)
    args = [d]
    if fmt in (QG_FMT_Q4_K, QG_FMT_Q5_K):
        dmin = np.ascontiguousarray(dmin, dtype=np.uint16)
        sc = np.ascontiguousarray(sc, dtype=np.uint8)
        m = np.ascontiguousarray(m, dtype=np.uint8)
        q = np.ascontiguousarray(q, dtype=np.uint8)
    elif fmt == QG_FMT_Q6_K:
        dmin = m = None
        sc = np.ascontiguousarray(np.asarray(sc).astype(np.int8).view(np.uint8))
        q = np.ascontiguousarray(q, dtype=np.uint8)
    elif fmt == QG_FMT_IQ4_XS:
        dmin = m = None
        sc = np.ascontiguousarray(sc, dtype=np.uint8)
        q = np.ascontiguousarray(q, dtype=np.uint8)
    else:
        dmin = sc = m = None
        q = np.ascontiguousarray(q, dtype=np.int8)
    args += [dmin, sc, m, q]
    _ok(lib().qg_pack_reference(int(fmt), int(N), int(K), _ptr(d), _ptr(dmin), _ptr(sc), _ptr(m),
                                _ptr(q), _ptr(out)), "qg_pack_reference")
    return out


def qg_last_variant() -> int:
    return int(lib().qg_last_variant())


def qg_last_splits() -> int:
    return int(lib().qg_last_splits())


def qg_plan(fmt: int, N: int, K: int, B: int, variant: int = 0, mats: int = 1, sms: int = 0,
            smem_optin: int = 0) -> dict:
    """The launch plan of a call (host only): variant, K slices, units per slice, CTAs, warps per
    CTA, dynamic shared memory bytes.  sms / smem_optin <= 0: the current device's."""
    out = (ctypes.c_int64 * 6)()
    _ok(lib().qg_plan(int(fmt), int(N), int(K), int(B), int(variant), int(mats), int(sms),
                      int(smem_optin), out), "qg_plan")
    keys = ("variant", "splits", "units_per_slice", "ctas", "warps", "smem")
    return dict(zip(keys, (int(v) for v in out)))


def qg_device_error(stream=None) -> int:
    flag = ctypes.c_int(0)
    _ok(lib().qg_device_error(_stream(stream), ctypes.byref(flag)), "qg_device_error")
    return flag.value


def qg_noalloc_device_error(stream=None) -> int:
    """Reads and clears the error word of qg_gemv_noalloc's fixed array (0: no timeout)."""
    flag = ctypes.c_int(0)
    _ok(lib().qg_noalloc_device_error(_stream(stream), ctypes.byref(flag)),
        "qg_noalloc_device_error")
    return flag.value


def qg_hbm_copy(src, dst, nbytes: int, stream=None) -> None:
    _ok(lib().qg_hbm_copy(_ptr(src), _ptr(dst), int(nbytes), _stream(stream)), "qg_hbm_copy")


def qg_hbm_read(src, nbytes: int, out, stream=None) -> None:
    _ok(lib().qg_hbm_read(_ptr(src), int(nbytes), _ptr(out), _stream(stream)), "qg_hbm_read")


# The operators around the GEMVs are short (a few microseconds on the GPU), so what their wrappers do on the
# host counts: torch is looked up once, views go to C as packed bytes, and the checks are a few attribute reads.
_tc = None
_pack_heads = struct.Struct("@Pqqqi4x").pack  # qg_heads


class _Torch:
    def __init__(self):
        import torch
        self.f32, self.f16, self.f64 = torch.float32, torch.float16, torch.float64
        self.i32, self.i64, self.u8 = torch.int32, torch.int64, torch.uint8
        self.empty, self.device = torch.empty, torch.cuda.current_device
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self.stream = raw or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _torch() -> _Torch:
    global _tc
    if _tc is None:
        _tc = _Torch()
    return _tc


def _where(tc, what: str, *tensors) -> int:
    """The current device; every tensor (None apart) has to be on it, where the kernels run."""
    dev = tc.device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{what}: every tensor must be on the current CUDA device ({dev}), got {t.device}")
    return dev


def _handle(tc, stream, dev: int) -> int:
    if stream is None:
        return tc.stream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _view(tc, t, what: str, name: str) -> bytes:
    """A [tokens, heads, dims] tensor as a qg_heads."""
    dt, st = t.dtype, t.stride()
    if (dt is not tc.f32 and dt is not tc.f16) or len(st) != 3:
        raise ValueError(f"{what}: {name} is fp32 or fp16 [tokens, heads, dims], got {dt} {tuple(t.shape)}")
    return _pack_heads(t.data_ptr(), st[0], st[1], st[2], QG_TYPE_F32 if dt is tc.f32 else QG_TYPE_F16)


def _vec(t, dtype, n: int, what: str, name: str):
    """The address of a contiguous vector of n elements of a type, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what}: {name} is a contiguous {dtype} [{n}], got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _cache_sizes(tc, cache, page: int, what: str):
    if cache.dtype is tc.u8 and cache.dim() == 4 and cache.is_contiguous():
        pages, H, blocks, width = cache.shape
        if page >= 16 and blocks * 16 == page and width % 18 == 0:
            return pages, H, width // 18
    raise ValueError(f"{what}: the cache is contiguous uint8 [pages, heads, page / 16, 18 D] with pages of {page} "
                     f"tokens, got {cache.dtype} {tuple(cache.shape)}")


def _rope(tc, pos, inv_freq, T: int, what: str):
    if inv_freq is None:
        return None, None, 0
    if pos is None:
        raise ValueError(f"{what}: a rotation needs positions")
    n = inv_freq.numel()
    return _vec(pos, tc.i32, T, what, "pos"), _vec(inv_freq, tc.f64, n, what, "inv_freq"), 2 * n


def qg_kv4_bytes(pages: int, page: int, H: int, D: int) -> int:
    """Bytes of a 4-bit cache; 0 for sizes it does not come in."""
    return int(lib().qg_kv4_bytes(int(pages), int(page), int(H), int(D)))


def kv4_cache(pages: int, page: int, H: int, D: int, device=None):
    """An empty 4-bit cache, uint8 [pages, H, page / 16, 18 D]."""
    import torch
    if pages > 0 and qg_kv4_bytes(pages, page, H, D) == 0:
        raise QgError(QG_ERR_SHAPE, "kv4_cache")
    return torch.zeros((pages, H, page // 16, 18 * D), dtype=torch.uint8, device=device or "cuda")


def qg_qk_norm_rope(q, k, wq, wk, eps: float, pos, inv_freq, pairing: int, q_out, k_out, stream=None) -> None:
    """Head norms (weights wq, wk fp32 [D]; None: no norm) and the rotation by pos * inv_freq (int32 [T],
    float64 [R / 2]; inv_freq None: no rotation) of q [T, Hq, D] and k [T, Hk, D] (either may be None)."""
    what = "qg_qk_norm_rope"
    tc = _tc or _torch()
    some = q if q is not None else k
    if some is None or some.dim() != 3:
        raise ValueError(f"{what}: q or k, [tokens, heads, dims]")
    dev = _where(tc, what, q, k, wq, wk, pos, inv_freq, q_out, k_out)
    T, _, D = some.shape
    vq = vk = oq = ok = None
    Hq = Hk = 0
    if q is not None:
        Hq = q.shape[1]
        if q_out is None or q_out.shape != q.shape:
            raise ValueError(f"{what}: q and q_out are [{T}, heads, {D}]")
        vq, oq = _view(tc, q, what, "q"), _view(tc, q_out, what, "q_out")
    if k is not None:
        Hk = k.shape[1]
        if k_out is None or k_out.shape != k.shape or k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"{what}: k and k_out are [{T}, heads, {D}]")
        vk, ok = _view(tc, k, what, "k"), _view(tc, k_out, what, "k_out")
    pp, pf, R = _rope(tc, pos, inv_freq, T, what)
    rc = (_lib or lib()).qg_qk_norm_rope(vq, vk, T, Hq, Hk, D, _vec(wq, tc.f32, D, what, "wq"),
                                         _vec(wk, tc.f32, D, what, "wk"), eps, pp, pf, R, pairing, oq, ok,
                                         _handle(tc, stream, dev))
    if rc:
        raise QgError(rc, what)


def qg_kv4_append(k, v, wk, eps: float, pos, inv_freq, pairing: int, slot, cache, page: int, stream=None) -> None:
    """Appends k, v [T, H, D] to the 4-bit cache at slot int64 [T] (-1: not written), the key with its head
    norm (wk None: none) and rotation (inv_freq None: none) applied on the way."""
    what = "qg_kv4_append"
    tc = _tc or _torch()
    dev = _where(tc, what, k, v, wk, pos, inv_freq, slot, cache)
    pages, H, D = _cache_sizes(tc, cache, page, what)
    T = k.shape[0]
    if k.shape != v.shape or k.shape[1:] != (H, D):
        raise ValueError(f"{what}: k and v are [tokens, {H}, {D}], got {tuple(k.shape)} and {tuple(v.shape)}")
    pp, pf, R = _rope(tc, pos, inv_freq, T, what)
    rc = (_lib or lib()).qg_kv4_append(_view(tc, k, what, "k"), _view(tc, v, what, "v"), T, H, D,
                                       _vec(wk, tc.f32, D, what, "wk"), eps, pp, pf, R, pairing,
                                       _vec(slot, tc.i64, T, what, "slot"), cache.data_ptr(), pages, page,
                                       _handle(tc, stream, dev))
    if rc:
        raise QgError(rc, what)


def qg_kv4_read(cache, page: int, slot, k_out, v_out, stream=None) -> None:
    """The values that the slots (int64 [T]) of the cache hold, into k_out and v_out [T, H, D]."""
    what = "qg_kv4_read"
    tc = _tc or _torch()
    dev = _where(tc, what, cache, slot, k_out, v_out)
    pages, H, D = _cache_sizes(tc, cache, page, what)
    T = slot.numel()
    if k_out.shape != (T, H, D) or v_out.shape != (T, H, D):
        raise ValueError(f"{what}: k_out and v_out are [{T}, {H}, {D}]")
    rc = (_lib or lib()).qg_kv4_read(cache.data_ptr(), pages, page, H, D, _vec(slot, tc.i64, T, what, "slot"), T,
                                     _view(tc, k_out, what, "k_out"), _view(tc, v_out, what, "v_out"),
                                     _handle(tc, stream, dev))
    if rc:
        raise QgError(rc, what)


_attn_ws: dict = {}


def _workspace_bytes(dev: int, Hq: int, Hk: int, D: int, max_q: int) -> int:
    key = (dev, Hq, Hk, D, max_q)
    n = _attn_ws.get(key)
    if n is None:
        n = int(lib().qg_attn_kv4_workspace(Hq, Hk, D, max_q))
        if n == 0:
            raise QgError(QG_ERR_SHAPE, "qg_attn_kv4_workspace")
        if len(_attn_ws) >= 4096:
            _attn_ws.clear()
        _attn_ws[key] = n
    return n


def qg_attn_kv4_workspace(Hq: int, Hk: int, D: int, max_q: int) -> int:
    """Workspace bytes of qg_attn_kv4 on the current device."""
    return _workspace_bytes(_torch().device(), int(Hq), int(Hk), int(D), int(max_q))


def qg_attn_kv4(q, q_start, max_q: int, cache, page: int, table, kv_len, scale: float, out, workspace=None,
                stream=None) -> None:
    """Causal attention of the new tokens q [T, Hq, D] (fp16; sequence s: rows q_start[s] .. q_start[s + 1] - 1)
    over the 4-bit cache, sequence s having kv_len[s] places in the pages table[s], into out [T, Hq, D] (fp16).
    workspace: uint8, qg_attn_kv4_workspace(Hq, Hk, D, max_q) bytes, not shared with a call that may overlap;
    None takes one from torch's allocator for this call."""
    what = "qg_attn_kv4"
    tc = _tc or _torch()
    dev = _where(tc, what, q, q_start, cache, table, kv_len, out, workspace)
    pages, Hk, D = _cache_sizes(tc, cache, page, what)
    if q.dtype is not tc.f16 or out.dtype is not tc.f16 or q.dim() != 3 or q.shape != out.shape or q.shape[2] != D:
        raise ValueError(f"{what}: q and out are fp16 [tokens, heads, {D}]")
    if table.dtype is not tc.i32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError(f"{what}: table is contiguous int32 [sequences, pages]")
    T, Hq, _ = q.shape
    nseq, width = table.shape
    st = _handle(tc, stream, dev)
    if workspace is None:
        if stream is not None and st != tc.stream(dev):
            raise ValueError(f"{what}: a call on a stream that is not torch's current one needs a workspace")
        n = _workspace_bytes(dev, Hq, Hk, D, max_q)
        workspace = tc.empty(n, dtype=tc.u8, device=q.device)
    else:
        n = workspace.numel() * workspace.element_size()
    rc = (_lib or lib()).qg_attn_kv4(_view(tc, q, what, "q"), T, nseq, _vec(q_start, tc.i32, nseq + 1, what, "q_start"),
                                     max_q, Hq, Hk, D, cache.data_ptr(), pages, page, table.data_ptr(), width,
                                     _vec(kv_len, tc.i32, nseq, what, "kv_len"), scale, _view(tc, out, what, "out"),
                                     workspace.data_ptr(), n, st)
    if rc:
        raise QgError(rc, what)


def qg_sample_workspace(rows: int, V: int, elem_stride: int) -> int:
    """Workspace bytes of qg_sample; 0 for rows that stand one after another."""
    return int(lib().qg_sample_workspace(int(rows), int(V), int(elem_stride)))


def qg_sample(logits, temperature, top_k, top_p, min_p, u, token, workspace=None, stream=None) -> None:
    """One token a row of logits [rows, V] (fp32, any strides: a GEMV's y.view(V, B).t()) with the row's
    temperature, top_k (int32), top_p and min_p (None: no such filter) from the random numbers u, into token
    (int32 [rows]).  workspace: uint8, qg_sample_workspace(rows, V, stride) bytes, not shared with a call that
    may overlap; None takes one from torch's allocator for this call."""
    what = "qg_sample"
    tc = _tc or _torch()
    dev = _where(tc, what, logits, temperature, top_k, top_p, min_p, u, token, workspace)
    if logits.dtype is not tc.f32 or logits.dim() != 2:
        raise ValueError(f"{what}: logits are fp32 [rows, V]")
    R, V = logits.shape
    rs, es = logits.stride()
    f32 = tc.f32
    st = _handle(tc, stream, dev)
    wp, wn = None, 0
    if workspace is not None:
        wp, wn = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif es != 1 and R > 1:
        if stream is not None and st != tc.stream(dev):
            raise ValueError(f"{what}: a call on a stream that is not torch's current one needs a workspace")
        workspace = tc.empty(R * V, dtype=f32, device=logits.device)
        wp, wn = workspace.data_ptr(), R * V * 4
    rc = (_lib or lib()).qg_sample(logits.data_ptr(), R, V, rs, es, _vec(temperature, f32, R, what, "temperature"),
                                   _vec(top_k, tc.i32, R, what, "top_k"), _vec(top_p, f32, R, what, "top_p"),
                                   _vec(min_p, f32, R, what, "min_p"), _vec(u, f32, R, what, "u"),
                                   _vec(token, tc.i32, R, what, "token"), wp, wn, st)
    if rc:
        raise QgError(rc, what)


def gemv(W, fmt: int, N: int, K: int, x, variant: int = QG_VARIANT_AUTO, stream=None):
    """Convenience wrapper on torch CUDA tensors: W uint8 bytes, x fp16 [K, B] -> new y fp32 [N, B]."""
    import torch
    B = 1 if x.dim() == 1 else x.shape[1]
    y = torch.empty((N, B), dtype=torch.float32, device=x.device)
    qg_gemv_variant(W, fmt, N, K, x, B, y, stream, variant)
    return y
