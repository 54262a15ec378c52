"""B200-native block-quantized dequant GEMV: y[N,B] = dequant(W[N,K]) . x[K,B], and the operators between
the GEMVs of a decode step: head norms with the position rotation, a paged 4-bit key/value cache with its
append and its attention, and sampling.

A thin ctypes binding over ``libqg.so`` (built from ``csrc/`` for sm_100a by ``build.py``): every
function here only marshals arguments and calls the C ABI of ``include/qg.h`` under the same name;
all computation runs in the library's CUDA kernels.  There is no CPU fallback: if the library is
missing, every call raises.

Pointers may be given as torch tensors (their ``data_ptr()``) or plain integers; ``stream=None``
means torch's current CUDA stream.  The operators around the GEMVs take torch CUDA tensors, whose sizes
and strides a small C++ module (``qg_binding.so``, of ``csrc/qg_binding.cpp``) hands to the same C ABI.
"""
from __future__ import annotations

import ctypes
import os

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
BINDING_PATH = os.path.join(_HERE, "qg_binding.so")
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
        L.qg_attn_kv4_device_error.argtypes = [P, ctypes.POINTER(I)]
        L.qg_attn_kv4_device_error.restype = I
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


# The operators around the GEMVs are short (a few microseconds on the GPU), so what a call does on the host counts:
# their tensors are read and checked in C++ (csrc/qg_binding.cpp), which calls the library.
_binding = None


def _bound():
    """The module that calls the operators around the GEMVs on torch tensors (raises if it has not been built)."""
    global _binding
    if _binding is None:
        import importlib.util

        import torch  # noqa: F401  (its libraries have to be there first)
        L = lib()
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"qg_binding.so not found at {BINDING_PATH}; build it with "
                               "`python -m quant_dequant_gemv_q4_b200.build`")
        spec = importlib.util.spec_from_file_location("qg_binding", BINDING_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        from . import build
        if m.built_for != build.built_for():
            raise RuntimeError(f"{BINDING_PATH} was built for {m.built_for}, this is {build.built_for()}; build it again with "
                               "`python -m quant_dequant_gemv_q4_b200.build`")
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in
                 (L.qg_qk_norm_rope, L.qg_kv4_append, L.qg_kv4_read, L.qg_attn_kv4_workspace, L.qg_attn_kv4, L.qg_sample_workspace,
                  L.qg_sample)))
        _binding = m
    return _binding


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
    rc = (_binding or _bound()).qk_norm_rope(q, k, wq, wk, eps, pos, inv_freq, pairing, q_out, k_out, stream)
    if rc:
        raise QgError(rc, "qg_qk_norm_rope")


def qg_kv4_append(k, v, wk, eps: float, pos, inv_freq, pairing: int, slot, cache, page: int, stream=None) -> None:
    """Appends k, v [T, H, D] to the 4-bit cache at slot int64 [T] (-1: not written), the key with its head
    norm (wk None: none) and rotation (inv_freq None: none) applied on the way."""
    rc = (_binding or _bound()).kv4_append(k, v, wk, eps, pos, inv_freq, pairing, slot, cache, page, stream)
    if rc:
        raise QgError(rc, "qg_kv4_append")


def qg_kv4_read(cache, page: int, slot, k_out, v_out, stream=None) -> None:
    """The values that the slots (int64 [T]) of the cache hold, into k_out and v_out [T, H, D]."""
    rc = (_binding or _bound()).kv4_read(cache, page, slot, k_out, v_out, stream)
    if rc:
        raise QgError(rc, "qg_kv4_read")


def qg_attn_kv4_workspace(Hq: int, Hk: int, D: int, max_q: int) -> int:
    """Workspace bytes of qg_attn_kv4 on the current device."""
    n = int(lib().qg_attn_kv4_workspace(int(Hq), int(Hk), int(D), int(max_q)))
    if n == 0:
        raise QgError(QG_ERR_SHAPE, "qg_attn_kv4_workspace")
    return n


def qg_attn_kv4(q, q_start, max_q: int, cache, page: int, table, kv_len, scale: float, out, workspace=None,
                stream=None) -> None:
    """Causal attention of the new tokens q [T, Hq, D] (fp16; sequence s: rows q_start[s] .. q_start[s + 1] - 1)
    over the 4-bit cache, sequence s having kv_len[s] places in the pages table[s], into out [T, Hq, D] (fp16).
    workspace: uint8, qg_attn_kv4_workspace(Hq, Hk, D, max_q) bytes, not shared with a call that may overlap;
    None takes one from torch's allocator for this call.  Device-side timeouts: qg_attn_kv4_device_error()."""
    rc = (_binding or _bound()).attn_kv4(q, q_start, max_q, cache, page, table, kv_len, scale, out, workspace, stream)
    if rc:
        raise QgError(rc, "qg_attn_kv4")


def qg_attn_kv4_device_error(stream=None) -> int:
    """Nonzero if a wait inside a qg_attn_kv4 call on the current device ran out (its results are void) since this was
    last asked; synchronizes the stream."""
    flag = ctypes.c_int(0)
    _ok(lib().qg_attn_kv4_device_error(_stream(stream), ctypes.byref(flag)), "qg_attn_kv4_device_error")
    return flag.value


def qg_sample_workspace(rows: int, V: int, elem_stride: int) -> int:
    """Workspace bytes of qg_sample; 0 for rows that stand one after another."""
    return int(lib().qg_sample_workspace(int(rows), int(V), int(elem_stride)))


def qg_sample(logits, temperature, top_k, top_p, min_p, u, token, workspace=None, stream=None) -> None:
    """One token a row of logits [rows, V] (fp32, any strides: a GEMV's y.view(V, B).t()) with the row's
    temperature, top_k (int32), top_p and min_p (None: no such filter) from the random numbers u, into token
    (int32 [rows]).  workspace: uint8, qg_sample_workspace(rows, V, stride) bytes, not shared with a call that
    may overlap; None takes one from torch's allocator for this call."""
    rc = (_binding or _bound()).sample(logits, temperature, top_k, top_p, min_p, u, token, workspace, stream)
    if rc:
        raise QgError(rc, "qg_sample")


def gemv(W, fmt: int, N: int, K: int, x, variant: int = QG_VARIANT_AUTO, stream=None):
    """Convenience wrapper on torch CUDA tensors: W uint8 bytes, x fp16 [K, B] -> new y fp32 [N, B]."""
    import torch
    B = 1 if x.dim() == 1 else x.shape[1]
    y = torch.empty((N, B), dtype=torch.float32, device=x.device)
    qg_gemv_variant(W, fmt, N, K, x, B, y, stream, variant)
    return y
