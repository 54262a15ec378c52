// qg_heads.cu -- the per-head operators between the QKV projection and the attention: the head norms
// with the position rotation (qg_qk_norm_rope), the append to the 4-bit cache (qg_kv4_append) and the
// read-back of cache entries (qg_kv4_read).  Declarations and contracts: include/qg.h.
//
// A row is one head of one token.  A lane holds eight consecutive dimensions of it, so D / 8 lanes take a
// row and a warp 32 * 8 / D rows: fp16 rows move in 16-byte accesses whatever D is, and the sums over a row
// are shuffles among its lanes.
//
// Norm weights and rotation together are y_i = r (x_i A_i + x_j B_i) with j the dimension's rotation partner,
// A_i = w_i cos a, B_i = -+ w_j sin a and r the norm's factor.  A and B depend on the token alone: a block
// makes them once in shared memory, and its warps take the token's heads with a lane's eight of each in
// registers, the next rows' loads in flight while a row is worked on.  With many tokens a block takes
// four: their tables are made side by side, and what a block waits for before its first row is shared.  For a few tokens
// the kernels are bound by launch and load latency (one token 2.3 us, 16 tokens appended and read back 6.5), for many by
// issuing instructions: 4099 tokens of 32 + 8 heads of 128, fp16, take 26 us (84 MB, 3.2 TB/s) with 74% of the issue slots of
// the active cycles used, and 1.7 waves of blocks; appending 6001 tokens 32 us (68% of the slots; the fp64 pipe 8%
// busy, the XU pipe, which converts between 64 and 32 bits, 38%), reading them back 17 (65%, and a row in flight a
// lane).  With two blocks a multiprocessor instead of three the append of 6001 tokens took 3 us longer.
#include <algorithm>

#include "qg_kv4.cuh"

namespace {

using namespace qg;

constexpr int kHeadWarps = 8;
constexpr int kMostTogether = 4;  // tokens of a block

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
    int64_t T;
    int Hq, Hk, together;  // together: tokens of a block
};

struct AppendArgs {
    HeadsView k, v;
    const float *wk;
    double eps;
    RopeArgs rope;
    const int64_t *slot;
    uint8_t *cache;
    int64_t slots;  // pages * page
    int64_t T;
    int page, H, together;
};

struct ReadArgs {
    HeadsView ko, vo;
    const int64_t *slot;
    const uint8_t *cache;
    int64_t slots, rows;
    int page, H;
};

constexpr int kV = 8;  // dimensions of a lane

// The rotation partners of a lane's dimensions dim .. dim + 7.  Dimension i < R is the pair (i, i + R/2)
// (halves) or (2j, 2j + 1) (adjacent) of angle index j.  For halves the partners are another lane's eight
// when R/2 is a multiple of eight, and go through shared memory otherwise.
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

// Where dimension d stands in a table: a lane's first dimension next to the neighbouring lane's first, and so
// on.  In their own order the lanes' reads would all start in the same banks of shared memory.
template <int D> __device__ __forceinline__ int place(int d) { return (d % kV) * (D / kV) + d / kV; }

// The tables of a block's tokens t0 .. t0 + n - 1: ab[j][y][place(d)] = (A, B) of dimension d of token t0 + j, one
// for each of W weight vectors (null: ones); cs(angle, &c, &s) gives cosine and sine.
template <int D, int W, typename T2, typename F>
__device__ __forceinline__ void make_tables(T2 (*ab)[W][D], const float *const (&w)[W], const RopeArgs &r, int64_t t0, int n, F cs)
{
    const int half = r.R / 2;
    for (int x = threadIdx.x; x < n * half; x += kHeadWarps * 32) {
        const int tok = x / half, f = x - tok * half;
        const int i = r.pairing == QG_ROPE_ADJACENT ? 2 * f : f, j = r.pairing == QG_ROPE_ADJACENT ? 2 * f + 1 : f + half;
        const double angle = (double)r.pos[t0 + tok] * r.freq[f];
        float wi[W], wj[W];
#pragma unroll
        for (int y = 0; y < W; ++y) {
            wi[y] = w[y] ? w[y][i] : 1.0f;
            wj[y] = w[y] ? w[y][j] : 1.0f;
        }
        decltype(ab[0][0][0].x) c, s;
        cs(angle, &c, &s);
#pragma unroll
        for (int y = 0; y < W; ++y) {
            ab[tok][y][place<D>(i)] = T2{wi[y] * c, -(wj[y] * s)};
            ab[tok][y][place<D>(j)] = T2{wj[y] * c, wi[y] * s};
        }
    }
    const int rest = D - r.R;
    for (int x = threadIdx.x; x < n * rest; x += kHeadWarps * 32) {
        const int tok = x / rest, d = r.R + x - tok * rest;
#pragma unroll
        for (int y = 0; y < W; ++y) ab[tok][y][place<D>(d)] = T2{w[y] ? w[y][d] : 1.0f, 0.0f};
    }
}

// The rows of a token in a view, from a lane's dimensions on.  KIND: 1 fp16 in 16-byte accesses, 2 fp32 so, 0 any.
struct RowsAt {
    const HeadsView &v;
    int64_t base;  // elements to the block's first token, head 0, this lane's dimensions
    __device__ __forceinline__ RowsAt(const HeadsView &view, int64_t t0, int dim) : v(view), base(t0 * view.st + dim * view.sd) {}
    // eight dimensions as they come: what is converted at once is waited for at once
    template <int KIND> __device__ __forceinline__ void load(int tok, int head, uint4 (&raw)[2]) const
    {
        const int64_t at = base + tok * v.st + head * v.sh;
        if constexpr (KIND == 1) {
            raw[0] = *reinterpret_cast<const uint4 *>(static_cast<const __half *>(v.p) + at);
        } else if constexpr (KIND == 2) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(v.p) + at);
            raw[0] = p[0], raw[1] = p[1];
        } else {
            float x[kV];
            HeadsView w = v;
            w.p = v.type == QG_TYPE_F32 ? static_cast<void *>(static_cast<float *>(v.p) + at) : static_cast<void *>(static_cast<__half *>(v.p) + at);
            load_dims(w, 0, 0, 0, x);
            raw[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            raw[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
        }
    }
    template <int KIND> static __device__ __forceinline__ void values(const uint4 (&raw)[2], float (&x)[kV])
    {
        if constexpr (KIND == 1) {
            const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
                x[2 * i] = f.x, x[2 * i + 1] = f.y;
            }
        } else {
            x[0] = __uint_as_float(raw[0].x), x[1] = __uint_as_float(raw[0].y), x[2] = __uint_as_float(raw[0].z), x[3] = __uint_as_float(raw[0].w);
            x[4] = __uint_as_float(raw[1].x), x[5] = __uint_as_float(raw[1].y), x[6] = __uint_as_float(raw[1].z), x[7] = __uint_as_float(raw[1].w);
        }
    }
    __device__ __forceinline__ void store(int tok, int head, const float (&x)[kV]) const
    {
        const int64_t at = base + tok * v.st + head * v.sh;
        HeadsView w = v;
        w.p = v.type == QG_TYPE_F32 ? static_cast<void *>(static_cast<float *>(v.p) + at) : static_cast<void *>(static_cast<__half *>(v.p) + at);
        store_dims<kV>(w, 0, 0, 0, x);
    }
};

inline int view_kind(const HeadsView &v) { return v.vec == 1 ? 0 : v.type == QG_TYPE_F16 ? 1 : 2; }

template <int LR, typename T> __device__ __forceinline__ T row_sum(T v)
{
#pragma unroll
    for (int o = LR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// y = x * rsqrt(mean(x^2) + eps) * w, then the rotation.  The sum of squares and the products are in
// fp32.  The angle is reduced to a fraction of a turn in 64 bits, so far positions keep their sine and
// cosine to fp32 (the reduced fraction is off by at most 2^-25 turns).
template <int D, int KIND> __global__ void __launch_bounds__(kHeadWarps * 32, 4) norm_rope_kernel(const NormRopeArgs a)
{
    constexpr int LR = D / kV, RW = 32 / LR;  // lanes of a row, rows of a warp
    __shared__ __align__(16) float2 ab[kMostTogether][2][D];
    __shared__ float rows[kHeadWarps][RW][D];
    const int64_t t0 = (int64_t)blockIdx.x * a.together;
    const int n = (int)(a.T - t0 < a.together ? a.T - t0 : a.together);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dim = kV * (lane % LR), sub = lane / LR;
    pdl_launch_dependents();
    pdl_wait();
    const int R = a.rope.R;
    const bool norm = a.wq || a.wk;
    // a token's rows in groups of RW heads, those of q first (no group holds heads of both)
    const int gq = (a.Hq + RW - 1) / RW, groups = gq + (a.Hk + RW - 1) / RW;
    const int step = gridDim.y * kHeadWarps;
    const RowsAt q(a.q, t0, dim), k(a.k, t0, dim), qo(a.qo, t0, dim), ko(a.ko, t0, dim);
    int g = blockIdx.y * kHeadWarps + warp, tok = 0;  // the group, and the token it is of
    while (g >= groups) {
        g -= groups;
        ++tok;
    }
    auto load = [&](int tok, int g, uint4 (&v)[2]) {
        const int h = (g < gq ? g : g - gq) * RW + sub;
        if (tok >= n) return;
        if (g < gq) {
            if (h < a.Hq) q.load<KIND>(tok, h, v);
        } else if (h < a.Hk) {
            k.load<KIND>(tok, h, v);
        }
    };
    uint4 raw[2] = {};
    load(tok, g, raw);
    const float *const weights[2] = {a.wq, a.wk};
    make_tables<D, 2>(ab, weights, a.rope, t0, n, [](double angle, float *c, float *s) {
        double turns = angle * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= rint(turns);
        sincospif(2.0f * (float)turns, s, c);
    });
    __syncthreads();
    float A[kV], B[kV];
    int which = -1;
    while (tok < n) {
        float x[kV];
        RowsAt::values<KIND>(raw, x);
        int gn = g + step, tn = tok;
        while (gn >= groups) {
            gn -= groups;
            ++tn;
        }
        load(tn, gn, raw);
        const bool isq = g < gq;
        if (which != 2 * tok + !isq) {
            which = 2 * tok + !isq;
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const float2 v = ab[tok][!isq][place<D>(dim + i)];
                A[i] = v.x, B[i] = v.y;
            }
        }
        float r = 1.0f, p[kV];
        if (R) rope_partners(x, rows[warp][sub], dim, R, a.rope.pairing, p);
        if (norm) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < kV; ++i) ss = fmaf(x[i], x[i], ss);
            ss = row_sum<LR>(ss);
            if (isq ? a.wq != nullptr : a.wk != nullptr) r = rsqrtf(ss * (1.0f / D) + (float)a.eps);  // (2 ulp)
        }
#pragma unroll
        for (int i = 0; i < kV; ++i) x[i] = r * (R ? fmaf(p[i], B[i], x[i] * A[i]) : x[i] * A[i]);
        const int h = (isq ? g : g - gq) * RW + sub;
        if (isq) {
            if (h < a.Hq) qo.store(tok, h, x);
        } else if (h < a.Hk) {
            ko.store(tok, h, x);
        }
        g = gn;
        tok = tn;
    }
}

// Appending.
//
// A code is the nearest of sixteen levels, and a value next to the border of two would go to one or the
// other by the rounding of the sums before it.  So that the stored bytes are those of the formula, the norm,
// the rotation, the group's range and d are in 64 bits; the quotient is in fp32 but where it comes within its
// own error of a border, where it is formed again in 64 bits (for about one value in ten thousand).  d and m
// are rounded to fp32 and then to fp16, two steps of the cache's definition (what conversions from 64 to 16 bits
// commonly do), and the codes are found against the rounded pair, which is what a reader multiplies by.
template <int D, int KIND> __global__ void __launch_bounds__(kHeadWarps * 32, 3) kv4_append_kernel(const AppendArgs a)
{
    constexpr int LR = D / kV, RW = 32 / LR;
    constexpr int LG = kKvGroup / kV;  // lanes of a group of 64
    using F = Kv4<D>;
    __shared__ __align__(16) double2 ab[kMostTogether][1][D];
    __shared__ float rows[kHeadWarps][RW][D];
    const int64_t t0 = (int64_t)blockIdx.x * a.together;
    const int n = (int)(a.T - t0 < a.together ? a.T - t0 : a.together);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dim = kV * (lane % LR), sub = lane / LR;
    pdl_launch_dependents();
    pdl_wait();
    const int R = a.rope.R;
    const bool changed = a.wk || R;  // keys are stored as something other than they come
    // a token's rows in groups of RW heads: those of k first
    const int gk = (a.H + RW - 1) / RW, groups = 2 * gk;
    const int step = gridDim.y * kHeadWarps;
    const RowsAt k(a.k, t0, dim), v(a.v, t0, dim);
    int g = blockIdx.y * kHeadWarps + warp, tok = 0;
    while (g >= groups) {
        g -= groups;
        ++tok;
    }
    auto load = [&](int tok, int g, uint4 (&x)[2], int64_t &slot) {
        const int h = (g < gk ? g : g - gk) * RW + sub;
        if (tok >= n) return;
        slot = a.slot[t0 + tok];
        if (h >= a.H) return;
        if (g < gk)
            k.load<KIND>(tok, h, x);
        else
            v.load<KIND>(tok, h, x);
    };
    uint4 raw[2] = {};
    int64_t next_slot = -1;
    load(tok, g, raw, next_slot);
    if (changed) {
        const float *const weights[1] = {a.wk};
        make_tables<D, 1>(ab, weights, a.rope, t0, n, [](double angle, double *c, double *s) { sincos(angle, s, c); });
        __syncthreads();
    }
    while (tok < n) {
        float xf[kV];
        RowsAt::values<KIND>(raw, xf);
        const int64_t slot = next_slot;
        const int gt = g, tt = tok;
        g += step;
        while (g >= groups) {
            g -= groups;
            ++tok;
        }
        load(tok, g, raw, next_slot);
        if (slot < 0 || slot >= a.slots) continue;  // not to be written
        const bool isk = gt < gk, exact = changed && isk;
        double x[kV], lo, hi;
        if (exact) {
            double r = 1.0, p[kV];
#pragma unroll
            for (int i = 0; i < kV; ++i) x[i] = xf[i];
            if (R) {
                // partners are exchanged as they came, in fp32
                float pf[kV];
                rope_partners(xf, rows[warp][sub], dim, R, a.rope.pairing, pf);
#pragma unroll
                for (int i = 0; i < kV; ++i) p[i] = pf[i];
            }
            if (a.wk) {
                double ss = 0.0;
#pragma unroll
                for (int i = 0; i < kV; ++i) ss = fma(x[i], x[i], ss);
                r = rsqrt(row_sum<LR>(ss) * (1.0 / D) + a.eps);
            }
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                const double2 c = ab[tt][0][place<D>(dim + i)];
                x[i] = r * (R ? fma(p[i], c.y, x[i] * c.x) : x[i] * c.x);
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
        const __half dh = __float2half_rn(fminf((float)((hi - lo) * (1.0 / 15.0)), 65504.0f));
        const __half mh = __float2half_rn(fminf(fmaxf((float)lo, -65504.0f), 65504.0f));
        const float d = __half2float(dh), m = __half2float(mh);
        const float rd = d > 0.0f ? 1.0f / d : 0.0f;
        uint32_t codes = 0, close = 0;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            // off by at most 2^-23 of the quotient and 2^-24 (|x| + |m|) / d, twice that with x rounded to fp32
            const float y = (xf[i] - m) * rd, n = rintf(y);
            codes |= (uint32_t)(int)fminf(fmaxf(n, 0.0f), 15.0f) << (4 * i);  // (also takes a NaN to 0)
            const float margin = fmaf(fabsf(xf[i]) + fabsf(m), 3e-7f * rd, 1e-5f);
            if (0.5f - fabsf(y - n) < margin) close |= 1u << i;
        }
        if (close && d > 0.0f) {
#pragma unroll
            for (int i = 0; i < kV; ++i)
                if (close >> i & 1) {
                    const double z = ((exact ? x[i] : (double)xf[i]) - (double)m) / (double)d;
                    codes = (codes & ~(15u << (4 * i))) | (uint32_t)__double2int_rn(fmin(fmax(z, 0.0), 15.0)) << (4 * i);
                }
        }
        const int head = (isk ? gt : gt - gk) * RW + sub;
        if (head < a.H) {
            const int64_t pg = slot / a.page;
            const int in_page = (int)(slot - pg * a.page);
            const int blk = in_page / kKvBlock, place = in_page % kKvBlock;
            uint8_t *part = a.cache + ((pg * a.H + head) * (a.page / kKvBlock) + blk) * F::kBlock + (isk ? 0 : F::kPart);
            *reinterpret_cast<uint32_t *>(part + kv4_code_offset<D>(place, dim)) = codes;
            if (lane % LG == 0)
                *reinterpret_cast<__half2 *>(part + F::kCodes + (place * F::kGroups + dim / kKvGroup) * 4) = __halves2half2(dh, mh);
        }
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

// (without tokens there are no positions: an empty tensor has no address)
int check_rope(const int32_t *pos, const double *freq, int R, int pairing, int D, int64_t T, RopeArgs *out)
{
    if (R < 0 || R > D || R % 2) return QG_ERR_SHAPE;
    if (pairing != QG_ROPE_HALVES && pairing != QG_ROPE_ADJACENT) return QG_ERR_VARIANT;
    if (R > 0 && T > 0 && (!pos || !freq)) return QG_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(pos) % 4 || reinterpret_cast<uintptr_t>(freq) % 8) return QG_ERR_ALIGN;
    out->pos = pos;
    out->freq = freq;
    out->R = R;
    out->pairing = pairing;
    return QG_OK;
}

// Tokens of a block, and blocks along a token's heads: four tokens where that leaves several blocks for each
// multiprocessor, else one, cut along its heads while the card has room.  With one and with four, 40 heads of 128
// took 11.8 and 12.8 us for 1300 tokens, 15.9 and 16.2 for 2000, 30.5 and 26.3 for 4099; the append of eight
// heads 14.4 and 15.0 us for 2000, 27.4 and 24.8 for 4099.
void head_blocks(int64_t T, int rows, int D, int sms, int *together, dim3 *grid)
{
    *together = T >= (int64_t)16 * sms ? kMostTogether : 1;
    const int each = kHeadWarps * 32 * kV / D;
    const int most = (rows + each - 1) / each;
    const int64_t blocks = (T + *together - 1) / *together;
    const int64_t want = (4 * (int64_t)sms + blocks - 1) / blocks;
    *grid = dim3((unsigned)blocks, (unsigned)std::min<int64_t>(most, std::max<int64_t>(1, want)));
}

template <int D> int launch_norm_rope(int kind, dim3 grid, dim3 block, void *stream, const NormRopeArgs &a)
{
    switch (kind) {
    case 1: return launch_pdl(norm_rope_kernel<D, 1>, grid, block, 0, stream, a);
    case 2: return launch_pdl(norm_rope_kernel<D, 2>, grid, block, 0, stream, a);
    default: return launch_pdl(norm_rope_kernel<D, 0>, grid, block, 0, stream, a);
    }
}
template <int D> int launch_append(int kind, dim3 grid, dim3 block, void *stream, const AppendArgs &a)
{
    switch (kind) {
    case 1: return launch_pdl(kv4_append_kernel<D, 1>, grid, block, 0, stream, a);
    case 2: return launch_pdl(kv4_append_kernel<D, 2>, grid, block, 0, stream, a);
    default: return launch_pdl(kv4_append_kernel<D, 0>, grid, block, 0, stream, a);
    }
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
    int rc = check_rope(pos, inv_freq, R, pairing, D, T, &a.rope);
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
    dim3 grid;
    const dim3 block(kHeadWarps * 32);
    a.T = T;
    head_blocks(T, Hq + Hk + 32 * kV / D - 1, D, sms, &a.together, &grid);
    const int kq = Hq ? view_kind(a.q) : view_kind(a.k), kk = Hk ? view_kind(a.k) : kq;
    switch (D) {
    case 64: return launch_norm_rope<64>(kq == kk ? kq : 0, grid, block, stream, a);
    case 128: return launch_norm_rope<128>(kq == kk ? kq : 0, grid, block, stream, a);
    default: return launch_norm_rope<256>(kq == kk ? kq : 0, grid, block, stream, a);
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
    if ((rc = check_rope(pos, inv_freq, R, pairing, D, T, &a.rope)) != QG_OK) return rc;
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
    dim3 grid;
    const dim3 block(kHeadWarps * 32);
    a.T = T;
    head_blocks(T, 2 * (H + 32 * kV / D - 1), D, sms, &a.together, &grid);
    const int kind = view_kind(a.k) == view_kind(a.v) ? view_kind(a.k) : 0;
    switch (D) {
    case 64: return launch_append<64>(kind, grid, block, stream, a);
    case 128: return launch_append<128>(kind, grid, block, stream, a);
    default: return launch_append<256>(kind, grid, block, stream, a);
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
