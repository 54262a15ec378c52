// qg_kv4.cuh -- the 4-bit key/value cache format, and the strided head views and host helpers that the
// operators around it share.
//
// A cache is uint8 [pages][H][page / 16][18 D], D = 64, 128 or 256.  A block holds 16 consecutive
// tokens of one head:
//   [K codes 16 x D/2][K scales 16 x D/64 x (fp16 d, fp16 m)][V codes 16 x D/2][V scales ...]
// A value is d * code + m with the (d, m) of its group of 64 dimensions: 4.5 bits a value.  K and V
// of 16 tokens are one contiguous run (4608 bytes at D = 256), so the attention kernels fetch a tile
// with one bulk copy.
//
// A token's codes are D nibbles, the even dimension in the low one, cut in chunks of 16 bytes (32
// dimensions).  Chunk c of token t stands at place c ^ (s(t) & (D/32 - 1)) with
// s(t) = (t & 2) | ((t ^ (t >> 2)) & 1) << 2: the attention kernel's lanes read one chunk each of
// tokens t, t + 2, t + 4, t + 6 (V) or of tokens t, t + 1 (K) at once, whose rows would all start in
// the same shared-memory bank; the permutation spreads those reads over all banks (D = 256).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/qg.h"

namespace qg {

constexpr int kKvBlock = 16;  // tokens of a block
constexpr int kKvGroup = 64;  // dimensions that share a (d, m) pair

template <int D> struct Kv4 {
    static constexpr int kCodeRow = D / 2;                      // code bytes of a token
    static constexpr int kGroups = D / kKvGroup;                // (d, m) pairs of a token
    static constexpr int kCodes = kKvBlock * kCodeRow;          // code bytes of K (or V) of a block
    static constexpr int kPart = kCodes + kKvBlock * kGroups * 4;  // all bytes of K (or V) of a block
    static constexpr int kBlock = 2 * kPart;                    // 18 D
    static constexpr int kChunkMask = D / 32 - 1;
};

// the permutation of a token's 16-byte chunks
__host__ __device__ __forceinline__ int kv4_swizzle(int t) { return (t & 2) | (((t ^ (t >> 2)) & 1) << 2); }

// byte offset in a part (K or V) of a block where dimension `dim` (even) of token t stands
template <int D> __host__ __device__ __forceinline__ int kv4_code_offset(int t, int dim)
{
    return t * Kv4<D>::kCodeRow + (((dim >> 5) ^ (kv4_swizzle(t) & Kv4<D>::kChunkMask)) << 4) + ((dim & 31) >> 1);
}

// A qg_heads as kernels take it.
struct HeadsView {
    void *p;
    int64_t st, sh, sd;  // strides in elements
    int type;            // QG_TYPE_F32 or QG_TYPE_F16
    int vec;             // elements of the widest aligned load along the dimensions (1: none)
};

inline int elem_bytes(int type) { return type == QG_TYPE_F32 ? 4 : 2; }

// Checks a view and finds how wide its rows may be read: dim stride 1 and every row start aligned to
// `want` elements.  `want` elements are at most 16 bytes a load; wider ones are split by the kernels.
inline int check_view(const qg_heads *h, int64_t T, int H, int want, bool f16_only, HeadsView *out)
{
    if (!h || !h->ptr) return QG_ERR_NULL;
    if (h->type != QG_TYPE_F16 && (f16_only || h->type != QG_TYPE_F32)) return QG_ERR_FMT;
    const int eb = elem_bytes(h->type);
    const uintptr_t a = reinterpret_cast<uintptr_t>(h->ptr);
    if (a % eb) return QG_ERR_ALIGN;
    out->p = h->ptr;
    out->st = h->token;
    out->sh = h->head;
    out->sd = h->dim;
    out->type = h->type;
    const int64_t row = (want * eb > 16 ? 16 : want * eb);
    const bool wide = h->dim == 1 && a % row == 0 && (T <= 1 || (h->token * eb) % row == 0) &&
                      (H <= 1 || (h->head * eb) % row == 0);
    out->vec = wide ? want : 1;
    return QG_OK;
}

// The status of a runtime call.  What a failed one leaves behind is taken back: a later launch that looks at the
// runtime's last error would take it for its own.
inline int cuda_status(cudaError_t e)
{
    if (e == cudaSuccess) return QG_OK;
    (void)cudaGetLastError();
    return QG_ERR_CUDA;
}

// Multiprocessors of the current device (a small table, no allocation).
inline int current_sms(int *sms)
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cuda_status(cudaGetDevice(&dev)) != QG_OK) return QG_ERR_CUDA;
    const bool slot = dev >= 0 && dev < 64;
    int n = slot ? known[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cuda_status(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != QG_OK) return QG_ERR_CUDA;
        if (slot) known[dev].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return QG_OK;
}

// Launch with programmatic stream serialization: the kernel may start while its predecessor drains and
// calls griddepcontrol.wait before it touches memory that the stream's earlier work may write.
template <typename... Args>
inline int launch_pdl(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem, void *stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Eight consecutive dimensions (from a multiple of eight on) of one head of one token.
__device__ __forceinline__ void load_dims(const HeadsView &h, int64_t t, int head, int dim, float (&x)[8])
{
    const int64_t at = t * h.st + head * h.sh + dim * h.sd;
    if (h.type == QG_TYPE_F32) {
        const float *p = static_cast<const float *>(h.p) + at;
        if (h.vec > 1) {
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(p + i);
                x[i] = v.x, x[i + 1] = v.y, x[i + 2] = v.z, x[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = p[i * h.sd];
        }
    } else {
        const __half *p = static_cast<const __half *>(h.p) + at;
        if (h.vec > 1) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __half2float(p[i * h.sd]);
        }
    }
}

// V dimensions (4 or 8, from a multiple of V on) written (fp16: each rounded once).
template <int V> __device__ __forceinline__ void store_dims(const HeadsView &h, int64_t t, int head, int dim, const float (&x)[V])
{
    static_assert(V == 4 || V == 8, "one 8- or 16-byte access of fp16, one or two of fp32");
    const int64_t at = t * h.st + head * h.sh + dim * h.sd;
    if (h.type == QG_TYPE_F32) {
        float *p = static_cast<float *>(h.p) + at;
        if (h.vec > 1) {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i * h.sd] = x[i];
        }
    } else {
        __half *p = static_cast<__half *>(h.p) + at;
        if (h.vec > 1) {
            uint32_t w[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&v);
            }
            if constexpr (V == 4)
                *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) p[i * h.sd] = __float2half_rn(x[i]);
        }
    }
}

}  // namespace qg
