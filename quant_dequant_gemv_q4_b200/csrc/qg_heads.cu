// qg_heads.cu -- the per-head operators between the QKV projection and the attention: the head norms
// with the position rotation (qg_qk_norm_rope), the append to the 4-bit cache (qg_kv4_append) and the
// read-back of cache entries (qg_kv4_read).  Declarations and contracts: include/qg.h.
//
// A row is one head of one token.  A lane holds eight consecutive dimensions of it, so D / 8 lanes take a
// row and a warp 32 * 8 / D rows: fp16 rows move in 16-byte accesses whatever D is, and the sums over a row
// are shuffles among its lanes.  The sines and cosines of a token depend on the token alone: a block takes
// one token, fills a table of them in shared memory once, and its warps take the token's heads, the next
// rows' loads in flight while a row is worked on.  The kernels are bound by memory traffic for long inputs
// and by launch and load latency for a few tokens.
#include <algorithm>

#include "qg_kv4.cuh"

namespace {

using namespace qg;

constexpr int kHeadWarps = 8;

struct RopeArgs {
    const int32_t *pos;
    const double *freq;  // [R / 2]
    int R;               // rotated dimensions (0: none)
    int pairing;         // QG_ROPE_HALVES or QG_ROPE_ADJACENT
};

struct NormRopeArgs {
    HeadsView q, k, qo, ko;
    const float *wq, *wk;
    double eps;
    RopeArgs rope;
    int Hq, Hk;
};

struct AppendArgs {
    HeadsView k, v;
    const float *wk;
    double eps;
    RopeArgs rope;
    const int64_t *slot;
    uint8_t *cache;
    int64_t slots;  // pages * page
    int page, H;
};

struct ReadArgs {
    HeadsView ko, vo;
    const int64_t *slot;
    const uint8_t *cache;
    int64_t slots, rows;
    int page, H;
};

constexpr int kV = 8;  // dimensions of a lane

// The rotation partners of a lane's dimensions dim .. dim + 7 < R.  Dimension i < R is the pair (i, i + R/2)
// (halves) or (2j, 2j + 1) (adjacent) of angle index j.  For halves the partners are another lane's eight
// when R/2 is a multiple of eight (`far`: lanes between), and go through shared memory otherwise.
template <typename T>
__device__ __forceinline__ void rope_partners(const T (&x)[kV], T *row, int dim, int R, int pairing, T (&partner)[kV])
{
    if (pairing == QG_ROPE_ADJACENT) {
#pragma unroll
        for (int i = 0; i < kV; ++i) partner[i] = x[i ^ 1];
    } else if (R % (2 * kV) == 0) {
        const int lane = threadIdx.x & 31, far = R / (2 * kV);
        const int from = dim < R / 2 ? lane + far : dim < R ? lane - far : lane;
#pragma unroll
        for (int i = 0; i < kV; ++i) partner[i] = __shfl_sync(0xffffffffu, x[i], from);
    } else {
        const int half = R >> 1;
        __syncwarp();  // the row's last readers are done
#pragma unroll
        for (int i = 0; i < kV; ++i) row[dim + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int d = dim + i;
            partner[i] = row[d < half ? d + half : (d < R ? d - half : d)];
        }
    }
}

__device__ __forceinline__ int rope_index(int d, int R, int pairing)
{
    return pairing == QG_ROPE_ADJACENT ? d >> 1 : (d < (R >> 1) ? d : d - (R >> 1));
}

__device__ __forceinline__ bool rope_first(int d, int R, int pairing)
{
    return pairing == QG_ROPE_ADJACENT ? (d & 1) == 0 : d < (R >> 1);
}

// x_i cos a - x_j sin a, x_j cos a + x_i sin a of the lane's rotated dimensions; cs: (cos, sin) by angle index.
template <typename T, typename T2>
__device__ __forceinline__ void rotate(T (&x)[kV], T *row, const T2 *cs, int dim, const RopeArgs &r)
{
    T p[kV];
    rope_partners(x, row, dim, r.R, r.pairing, p);
    if (dim >= r.R) return;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
        const int d = dim + i;
        if (d < r.R) {
            const T2 c = cs[rope_index(d, r.R, r.pairing)];
            x[i] = rope_first(d, r.R, r.pairing) ? x[i] * c.x - p[i] * c.y : x[i] * c.x + p[i] * c.y;
        }
    }
}

template <int LR, typename T> __device__ __forceinline__ T row_sum(T v)
{
#pragma unroll
    for (int o = LR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// y = x * rsqrt(mean(x^2) + eps) * w, then the rotation.  The sum of squares and the products are in
// fp32.  The angle is reduced to a fraction of a turn in 64 bits, so far positions keep their sine and
// cosine to fp32 (the reduced fraction is off by at most 2^-25 turns).
template <int D> __global__ void __launch_bounds__(kHeadWarps * 32) norm_rope_kernel(const NormRopeArgs a)
{
    constexpr int LR = D / kV, RW = 32 / LR;  // lanes of a row, rows of a warp
    __shared__ float2 cs[D / 2];
    __shared__ float rows[kHeadWarps][RW][D];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dim = kV * (lane % LR), sub = lane / LR;
    pdl_launch_dependents();
    pdl_wait();
    const int R = a.rope.R;
    const int H = a.Hq + a.Hk;
    const int step = gridDim.y * kHeadWarps * RW;
    int h0 = (blockIdx.y * kHeadWarps + warp) * RW;  // the warp's rows: heads h0 .. h0 + RW - 1
    auto load = [&](int h, float (&v)[kV]) {
        if (h < H) load_dims<kV>(h < a.Hq ? a.q : a.k, t, h < a.Hq ? h : h - a.Hq, dim, v);
    };
    float x[kV] = {};
    load(h0 + sub, x);
    for (int i = threadIdx.x; i < (R >> 1); i += blockDim.x) {
        double turns = (double)a.rope.pos[t] * a.rope.freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= rint(turns);
        float s, c;
        sincospif(2.0f * (float)turns, &s, &c);
        cs[i] = make_float2(c, s);
    }
    __syncthreads();
    while (h0 < H) {
        const int h = h0 + sub, hn = h0 + step;
        const bool isq = h < a.Hq;
        float xn[kV] = {};
        load(hn + sub, xn);
        const float *w = isq ? a.wq : a.wk;
        if (a.wq || a.wk) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < kV; ++i) ss = fmaf(x[i], x[i], ss);
            ss = row_sum<LR>(ss);
            if (w) {
                const float r = 1.0f / sqrtf(ss * (1.0f / D) + (float)a.eps);
#pragma unroll
                for (int i = 0; i < kV; ++i) x[i] = x[i] * r * __ldg(w + dim + i);
            }
        }
        if (R) rotate(x, rows[warp][sub], cs, dim, a.rope);
        if (h < H) store_dims<kV>(isq ? a.qo : a.ko, t, isq ? h : h - a.Hq, dim, x);
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] = xn[i];
        h0 = hn;
    }
}

// Appending: rows 0 .. H-1 of a token are its keys, H .. 2H-1 its values.
//
// A code is the nearest of sixteen levels, and a value next to the border of two would go to one or the
// other by the rounding of the sums before it.  So that the stored bytes are those of the formula, the norm,
// the rotation, the group's range and d are in 64 bits; the quotient is in fp32 but where it comes within its
// own error of a border, where it is formed again in 64 bits (for about one value in ten thousand).  d and m
// are rounded to fp16 first and the codes are found against the rounded pair, which is what a reader
// multiplies by.
template <int D> __global__ void __launch_bounds__(kHeadWarps * 32) kv4_append_kernel(const AppendArgs a)
{
    constexpr int LR = D / kV, RW = 32 / LR;
    constexpr int LG = kKvGroup / kV;  // lanes of a group of 64
    using F = Kv4<D>;
    __shared__ double2 cs[D / 2];
    __shared__ double rows[kHeadWarps][RW][D];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dim = kV * (lane % LR), sub = lane / LR;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t slot = a.slot[t];
    if (slot < 0 || slot >= a.slots) return;  // not to be written
    const int R = a.rope.R;
    const int step = gridDim.y * kHeadWarps * RW;
    int h0 = (blockIdx.y * kHeadWarps + warp) * RW;
    auto load = [&](int h, float (&v)[kV]) {
        if (h < 2 * a.H) load_dims<kV>(h < a.H ? a.k : a.v, t, h < a.H ? h : h - a.H, dim, v);
    };
    float xf[kV] = {};
    load(h0 + sub, xf);
    for (int i = threadIdx.x; i < (R >> 1); i += blockDim.x) {
        double s, c;
        sincos((double)a.rope.pos[t] * a.rope.freq[i], &s, &c);
        cs[i] = make_double2(c, s);
    }
    __syncthreads();
    const int64_t pg = slot / a.page;
    const int in_page = (int)(slot - pg * a.page);
    const int blk = in_page / kKvBlock, tok = in_page % kKvBlock;
    while (h0 < 2 * a.H) {
        const int h = h0 + sub, hn = h0 + step;
        const bool isk = h < a.H;
        float xn[kV] = {};
        load(hn + sub, xn);
        double lo, hi;
        double x[kV];
        const bool exact = (a.wk != nullptr || R) && h0 < a.H;  // some row of the warp is a key that is changed
        if (exact) {
#pragma unroll
            for (int i = 0; i < kV; ++i) x[i] = xf[i];
            if (a.wk) {
                double ss = 0.0;
#pragma unroll
                for (int i = 0; i < kV; ++i) ss = fma(x[i], x[i], ss);
                ss = row_sum<LR>(ss);
                if (isk) {
                    const double r = 1.0 / sqrt(ss * (1.0 / D) + a.eps);
#pragma unroll
                    for (int i = 0; i < kV; ++i) x[i] = x[i] * r * (double)__ldg(a.wk + dim + i);
                }
            }
            if (R) {
                double y[kV];
#pragma unroll
                for (int i = 0; i < kV; ++i) y[i] = x[i];
                rotate(y, rows[warp][sub], cs, dim, a.rope);
#pragma unroll
                for (int i = 0; i < kV; ++i) x[i] = isk ? y[i] : x[i];
            }
            lo = x[0], hi = x[0];
#pragma unroll
            for (int i = 1; i < kV; ++i) {
                lo = x[i] < lo ? x[i] : lo;
                hi = x[i] > hi ? x[i] : hi;
            }
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1) {
                const double l = __shfl_xor_sync(0xffffffffu, lo, o), u = __shfl_xor_sync(0xffffffffu, hi, o);
                lo = l < lo ? l : lo;
                hi = u > hi ? u : hi;
            }
#pragma unroll
            for (int i = 0; i < kV; ++i) xf[i] = (float)x[i];
        } else {
            float l = xf[0], u = xf[0];
#pragma unroll
            for (int i = 1; i < kV; ++i) {
                l = fminf(l, xf[i]);
                u = fmaxf(u, xf[i]);
            }
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1) {
                l = fminf(l, __shfl_xor_sync(0xffffffffu, l, o));
                u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
            }
            lo = l, hi = u;
        }
        // a range past fp16 saturates, so that what is read back stays finite
        const __half dh = __float2half_rn(fminf((float)((hi - lo) / 15.0), 65504.0f));
        const __half mh = __float2half_rn(fminf(fmaxf((float)lo, -65504.0f), 65504.0f));
        const float d = __half2float(dh), m = __half2float(mh);
        const float rd = d > 0.0f ? 1.0f / d : 0.0f;
        uint32_t codes = 0;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            // off by at most 2^-23 of the quotient and 2^-24 (|x| + |m|) / d, twice that with x rounded to fp32
            const float y = (xf[i] - m) * rd;
            const float c = fminf(fmaxf(rintf(y), 0.0f), 15.0f);  // (also takes a NaN to 0)
            uint32_t code = (uint32_t)(int)c;
            const float margin = fmaf(fabsf(xf[i]) + fabsf(m), 3e-7f * rd, 1e-5f);
            if (d > 0.0f && 0.5f - fabsf(y - rintf(y)) < margin) {
                const double z = ((exact ? x[i] : (double)xf[i]) - (double)m) / (double)d;
                code = (uint32_t)__double2int_rn(fmin(fmax(z, 0.0), 15.0));
            }
            codes |= code << (4 * i);
        }
        if (h < 2 * a.H) {
            const int head = isk ? h : h - a.H;
            uint8_t *part = a.cache + ((pg * a.H + head) * (a.page / kKvBlock) + blk) * F::kBlock + (isk ? 0 : F::kPart);
            *reinterpret_cast<uint32_t *>(part + kv4_code_offset<D>(tok, dim)) = codes;
            if (lane % LG == 0)
                *reinterpret_cast<__half2 *>(part + F::kCodes + (tok * F::kGroups + dim / kKvGroup) * 4) = __halves2half2(dh, mh);
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) xf[i] = xn[i];
        h0 = hn;
    }
}

// The values that a slot holds, d * code + m with one fp32 rounding; zeros for a slot out of range.
template <int D> __global__ void __launch_bounds__(kHeadWarps * 32) kv4_read_kernel(const ReadArgs a)
{
    constexpr int LR = D / kV, RW = 32 / LR;
    using F = Kv4<D>;
    const int lane = threadIdx.x & 31;
    const int dim = kV * (lane % LR);
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t r = ((int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5)) * RW + lane / LR; r < a.rows;
         r += (int64_t)gridDim.x * kHeadWarps * RW) {
        const int64_t t = r / (2 * a.H);
        const int h = (int)(r - t * 2 * a.H);
        const bool isk = h < a.H;
        const int head = isk ? h : h - a.H;
        const int64_t slot = a.slot[t];
        float x[kV] = {};
        if (slot >= 0 && slot < a.slots) {
            const int64_t pg = slot / a.page;
            const int in_page = (int)(slot - pg * a.page);
            const int blk = in_page / kKvBlock, tok = in_page % kKvBlock;
            const uint8_t *part = a.cache + ((pg * a.H + head) * (a.page / kKvBlock) + blk) * F::kBlock + (isk ? 0 : F::kPart);
            const uint32_t codes = *reinterpret_cast<const uint32_t *>(part + kv4_code_offset<D>(tok, dim));
            const float2 dm = __half22float2(*reinterpret_cast<const __half2 *>(
                part + F::kCodes + (tok * F::kGroups + dim / kKvGroup) * 4));
#pragma unroll
            for (int i = 0; i < kV; ++i) x[i] = fmaf((float)((codes >> (4 * i)) & 15u), dm.x, dm.y);
        }
        store_dims<kV>(isk ? a.ko : a.vo, t, head, dim, x);
    }
}

bool good_dim(int D) { return D == 64 || D == 128 || D == 256; }

int check_rope(const int32_t *pos, const double *freq, int R, int pairing, int D, RopeArgs *out)
{
    if (R < 0 || R > D || R % 2) return QG_ERR_SHAPE;
    if (pairing != QG_ROPE_HALVES && pairing != QG_ROPE_ADJACENT) return QG_ERR_VARIANT;
    if (R > 0 && (!pos || !freq)) return QG_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(pos) % 4 || reinterpret_cast<uintptr_t>(freq) % 8) return QG_ERR_ALIGN;
    out->pos = pos;
    out->freq = freq;
    out->R = R;
    out->pairing = pairing;
    return QG_OK;
}

// Blocks along a token's heads: a warp's rows once each while that leaves the card room, else the whole token
// in one block, so that its sines and cosines are made once.
int head_blocks(int64_t T, int rows, int D, int sms)
{
    const int each = kHeadWarps * 32 * kV / D;
    const int most = (rows + each - 1) / each;
    const int64_t want = (4 * (int64_t)sms + T - 1) / T;
    return (int)std::min<int64_t>(most, std::max<int64_t>(1, want));
}

constexpr int64_t kMostTokens = 0x7fffffff;  // grid limit

int check_cache(const void *cache, int64_t pages, int page, int H, int D)
{
    if (!good_dim(D) || H < 1 || H > QG_MAX_HEADS || pages < 0 || page < kKvBlock || page % kKvBlock) return QG_ERR_SHAPE;
    if (pages > 0 && qg_kv4_bytes(pages, page, H, D) == 0) return QG_ERR_SHAPE;
    if (pages > 0 && !cache) return QG_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(cache) % 16) return QG_ERR_ALIGN;
    return QG_OK;
}

}  // namespace

extern "C" {

size_t qg_kv4_bytes(int64_t pages, int page, int H, int D)
{
    if (!good_dim(D) || H < 1 || H > QG_MAX_HEADS || pages < 0 || page < kKvBlock || page % kKvBlock) return 0;
    const unsigned __int128 n = (unsigned __int128)pages * (unsigned)page / kKvBlock * (unsigned)H * (18u * (unsigned)D);
    return n > (unsigned __int128)INT64_MAX ? 0 : (size_t)n;
}

int qg_qk_norm_rope(const qg_heads *q, const qg_heads *k, int64_t T, int Hq, int Hk, int D, const float *wq,
                    const float *wk, double eps, const int32_t *pos, const double *inv_freq, int R, int pairing,
                    const qg_heads *q_out, const qg_heads *k_out, void *stream)
{
    if (!good_dim(D) || T < 0 || T > kMostTokens || Hq < 0 || Hk < 0 || Hq > QG_MAX_HEADS || Hk > QG_MAX_HEADS)
        return QG_ERR_SHAPE;
    if (!(eps >= 0.0)) return QG_ERR_RANGE;
    NormRopeArgs a = {};
    int rc = check_rope(pos, inv_freq, R, pairing, D, &a.rope);
    if (rc != QG_OK) return rc;
    if (T == 0 || Hq + Hk == 0) return QG_OK;
    if (Hq > 0) {
        if ((rc = check_view(q, T, Hq, kV, false, &a.q)) != QG_OK) return rc;
        if ((rc = check_view(q_out, T, Hq, kV, false, &a.qo)) != QG_OK) return rc;
    }
    if (Hk > 0) {
        if ((rc = check_view(k, T, Hk, kV, false, &a.k)) != QG_OK) return rc;
        if ((rc = check_view(k_out, T, Hk, kV, false, &a.ko)) != QG_OK) return rc;
    }
    if (reinterpret_cast<uintptr_t>(wq) % 4 || reinterpret_cast<uintptr_t>(wk) % 4) return QG_ERR_ALIGN;
    a.wq = wq;
    a.wk = wk;
    a.eps = eps;
    a.Hq = Hq;
    a.Hk = Hk;
    int sms = 0;
    if ((rc = current_sms(&sms)) != QG_OK) return rc;
    const dim3 grid((unsigned)T, head_blocks(T, Hq + Hk, D, sms)), block(kHeadWarps * 32);
    switch (D) {
    case 64: return launch_pdl(norm_rope_kernel<64>, grid, block, 0, stream, a);
    case 128: return launch_pdl(norm_rope_kernel<128>, grid, block, 0, stream, a);
    default: return launch_pdl(norm_rope_kernel<256>, grid, block, 0, stream, a);
    }
}

int qg_kv4_append(const qg_heads *k, const qg_heads *v, int64_t T, int H, int D, const float *wk, double eps,
                  const int32_t *pos, const double *inv_freq, int R, int pairing, const int64_t *slot, void *cache,
                  int64_t pages, int page, void *stream)
{
    int rc = check_cache(cache, pages, page, H, D);
    if (rc != QG_OK) return rc;
    if (T < 0 || T > kMostTokens) return QG_ERR_SHAPE;
    if (!(eps >= 0.0)) return QG_ERR_RANGE;
    AppendArgs a = {};
    if ((rc = check_rope(pos, inv_freq, R, pairing, D, &a.rope)) != QG_OK) return rc;
    if (T == 0 || pages == 0) return QG_OK;
    if (!slot) return QG_ERR_NULL;
    if ((rc = check_view(k, T, H, kV, false, &a.k)) != QG_OK) return rc;
    if ((rc = check_view(v, T, H, kV, false, &a.v)) != QG_OK) return rc;
    if (reinterpret_cast<uintptr_t>(slot) % 8 || reinterpret_cast<uintptr_t>(wk) % 4) return QG_ERR_ALIGN;
    a.wk = wk;
    a.eps = eps;
    a.slot = slot;
    a.cache = static_cast<uint8_t *>(cache);
    a.slots = pages * page;
    a.page = page;
    a.H = H;
    int sms = 0;
    if ((rc = current_sms(&sms)) != QG_OK) return rc;
    const dim3 grid((unsigned)T, head_blocks(T, 2 * H, D, sms)), block(kHeadWarps * 32);
    switch (D) {
    case 64: return launch_pdl(kv4_append_kernel<64>, grid, block, 0, stream, a);
    case 128: return launch_pdl(kv4_append_kernel<128>, grid, block, 0, stream, a);
    default: return launch_pdl(kv4_append_kernel<256>, grid, block, 0, stream, a);
    }
}

int qg_kv4_read(const void *cache, int64_t pages, int page, int H, int D, const int64_t *slot, int64_t T,
                const qg_heads *k_out, const qg_heads *v_out, void *stream)
{
    int rc = check_cache(cache, pages, page, H, D);
    if (rc != QG_OK) return rc;
    if (T < 0 || T > kMostTokens) return QG_ERR_SHAPE;
    if (T == 0) return QG_OK;
    if (!slot) return QG_ERR_NULL;
    ReadArgs a = {};
    if ((rc = check_view(k_out, T, H, kV, false, &a.ko)) != QG_OK) return rc;
    if ((rc = check_view(v_out, T, H, kV, false, &a.vo)) != QG_OK) return rc;
    if (reinterpret_cast<uintptr_t>(slot) % 8) return QG_ERR_ALIGN;
    a.slot = slot;
    a.cache = static_cast<const uint8_t *>(cache);
    a.slots = pages * page;
    a.rows = T * 2 * H;
    a.page = page;
    a.H = H;
    int sms = 0;
    if ((rc = current_sms(&sms)) != QG_OK) return rc;
    const int each = kHeadWarps * 32 * kV / D;  // rows of a block at a time
    const dim3 grid((unsigned)std::min<int64_t>((a.rows + each - 1) / each, (int64_t)sms * 8));
    const dim3 block(kHeadWarps * 32);
    switch (D) {
    case 64: return launch_pdl(kv4_read_kernel<64>, grid, block, 0, stream, a);
    case 128: return launch_pdl(kv4_read_kernel<128>, grid, block, 0, stream, a);
    default: return launch_pdl(kv4_read_kernel<256>, grid, block, 0, stream, a);
    }
}

}  // extern "C"
