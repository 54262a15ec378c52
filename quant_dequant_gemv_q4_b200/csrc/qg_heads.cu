// qg_heads.cu -- the per-head operators between the QKV projection and the attention: the head norms
// with the position rotation (qg_qk_norm_rope), the append to the 4-bit cache (qg_kv4_append) and the
// read-back of cache entries (qg_kv4_read).  Declarations and contracts: include/qg.h.
//
// One warp takes one row (one head of one token): lane l holds dimensions V l .. V l + V - 1, V = D/32,
// so a row is one coalesced access and the sums over a row are warp shuffles.  The sines and cosines of
// a token depend on the token alone: a block takes one token, fills a table of them in shared memory
// once, and its warps take the token's heads.  The kernels are bound by memory traffic for long inputs
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

// The row's rotation partners.  Dimension i < R is the pair (i, i + R/2) (halves) or (2j, 2j + 1)
// (adjacent) of angle index j; `mine` of lane l are dimensions V l ...  For halves the partner may be
// in another lane: the row goes through shared memory.
template <int V, typename T>
__device__ __forceinline__ void rope_partners(const T (&x)[V], T *row, int lane, int R, int pairing, T (&partner)[V])
{
    if (pairing == QG_ROPE_ADJACENT) {
#pragma unroll
        for (int i = 0; i < V; ++i) partner[i] = x[i ^ 1];
        return;
    }
    __syncwarp();  // the row's last readers are done
#pragma unroll
    for (int i = 0; i < V; ++i) row[V * lane + i] = x[i];
    __syncwarp();
    const int half = R >> 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = V * lane + i;
        partner[i] = row[d < half ? d + half : (d < R ? d - half : d)];
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

// y = x * rsqrt(mean(x^2) + eps) * w, then the rotation.  The sum of squares and the products are in
// fp32.  The angle is reduced to a fraction of a turn in 64 bits, so far positions keep their sine and
// cosine to fp32 (the reduced fraction is off by at most 2^-25 turns).
template <int D> __global__ void __launch_bounds__(kHeadWarps * 32) norm_rope_kernel(const NormRopeArgs a)
{
    constexpr int V = D / 32;
    __shared__ float2 cs[D / 2];
    __shared__ float rows[kHeadWarps][D];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int R = a.rope.R;
    const int H = a.Hq + a.Hk;
    const int step = gridDim.y * kHeadWarps;
    int h = blockIdx.y * kHeadWarps + warp;
    float x[V];
    if (h < H) load_dims<V>(h < a.Hq ? a.q : a.k, t, h < a.Hq ? h : h - a.Hq, V * lane, x);
    for (int i = threadIdx.x; i < (R >> 1); i += blockDim.x) {
        double turns = (double)a.rope.pos[t] * a.rope.freq[i] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= rint(turns);
        float s, c;
        sincospif(2.0f * (float)turns, &s, &c);
        cs[i] = make_float2(c, s);
    }
    __syncthreads();
    while (h < H) {
        const bool isq = h < a.Hq;
        const int head = isq ? h : h - a.Hq;
        const float *w = isq ? a.wq : a.wk;
        const int hn = h + step;
        float xn[V];  // the next row's load overlaps this row's arithmetic
        if (hn < H) load_dims<V>(hn < a.Hq ? a.q : a.k, t, hn < a.Hq ? hn : hn - a.Hq, V * lane, xn);
        if (w) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = 1.0f / sqrtf(ss * (1.0f / D) + (float)a.eps);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = x[i] * r * __ldg(w + V * lane + i);
        }
        if (R) {
            float p[V];
            rope_partners<V>(x, rows[warp], lane, R, a.rope.pairing, p);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int d = V * lane + i;
                if (d < R) {
                    const float2 c = cs[rope_index(d, R, a.rope.pairing)];
                    x[i] = rope_first(d, R, a.rope.pairing) ? x[i] * c.x - p[i] * c.y : x[i] * c.x + p[i] * c.y;
                }
            }
        }
        store_dims<V>(isq ? a.qo : a.ko, t, head, V * lane, x);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = xn[i];
        h = hn;
    }
}

// Appending: rows 0 .. H-1 of a token are its keys, H .. 2H-1 its values.
//
// Everything that decides a code is in 64 bits (the norm, the rotation, d, the quotient): a code is the
// nearest of sixteen levels, and a value next to the border of two would otherwise go to one or the
// other by the rounding of the sums before it.  With 64 bits the stored bytes are those of the formula
// but for values closer than about 1e-15 to a border.  d and m are rounded to fp16 first and the codes
// are found against the rounded pair, which is what a reader multiplies by.
template <int D> __global__ void __launch_bounds__(kHeadWarps * 32) kv4_append_kernel(const AppendArgs a)
{
    constexpr int V = D / 32;
    constexpr int LG = kKvGroup / V;  // lanes of a group of 64
    using F = Kv4<D>;
    __shared__ double2 cs[D / 2];
    __shared__ double rows[kHeadWarps][D];
    const int64_t t = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t slot = a.slot[t];
    if (slot < 0 || slot >= a.slots) return;  // not to be written
    const int R = a.rope.R;
    for (int i = threadIdx.x; i < (R >> 1); i += blockDim.x) {
        double s, c;
        sincos((double)a.rope.pos[t] * a.rope.freq[i], &s, &c);
        cs[i] = make_double2(c, s);
    }
    __syncthreads();
    const int64_t pg = slot / a.page;
    const int in_page = (int)(slot - pg * a.page);
    const int blk = in_page / kKvBlock, tok = in_page % kKvBlock;
    const int step = gridDim.y * kHeadWarps;
    for (int h = blockIdx.y * kHeadWarps + warp; h < 2 * a.H; h += step) {
        const bool isk = h < a.H;
        const int head = isk ? h : h - a.H;
        float xf[V];
        load_dims<V>(isk ? a.k : a.v, t, head, V * lane, xf);
        double x[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = xf[i];
        if (isk && a.wk) {
            double ss = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fma(x[i], x[i], ss);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const double r = 1.0 / sqrt(ss * (1.0 / D) + a.eps);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = x[i] * r * (double)__ldg(a.wk + V * lane + i);
        }
        if (isk && R) {
            double p[V];
            rope_partners<V>(x, rows[warp], lane, R, a.rope.pairing, p);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int d = V * lane + i;
                if (d < R) {
                    const double2 c = cs[rope_index(d, R, a.rope.pairing)];
                    x[i] = rope_first(d, R, a.rope.pairing) ? x[i] * c.x - p[i] * c.y : x[i] * c.x + p[i] * c.y;
                }
            }
        }
        double lo = x[0], hi = x[0];
#pragma unroll
        for (int i = 1; i < V; ++i) {
            lo = fmin(lo, x[i]);
            hi = fmax(hi, x[i]);
        }
#pragma unroll
        for (int o = LG / 2; o > 0; o >>= 1) {
            lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        // a range past fp16 saturates, so that what is read back stays finite
        const __half dh = __float2half_rn(fminf((float)((hi - lo) / 15.0), 65504.0f));
        const __half mh = __float2half_rn(fminf(fmaxf((float)lo, -65504.0f), 65504.0f));
        const double d = (double)__half2float(dh), m = (double)__half2float(mh);
        uint32_t codes = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            double y = d > 0.0 ? (x[i] - m) / d : 0.0;
            y = fmin(fmax(y, 0.0), 15.0);  // also takes a NaN to 0
            codes |= (uint32_t)__double2int_rn(y) << (4 * i);
        }
        uint8_t *part = a.cache + ((pg * a.H + head) * (a.page / kKvBlock) + blk) * F::kBlock + (isk ? 0 : F::kPart);
        uint8_t *at = part + kv4_code_offset<D>(tok, V * lane);
        if constexpr (V == 8)
            *reinterpret_cast<uint32_t *>(at) = codes;
        else if constexpr (V == 4)
            *reinterpret_cast<uint16_t *>(at) = (uint16_t)codes;
        else
            *at = (uint8_t)codes;
        if (lane % LG == 0)
            *reinterpret_cast<__half2 *>(part + F::kCodes + (tok * F::kGroups + lane / LG) * 4) = __halves2half2(dh, mh);
    }
}

// The values that a slot holds, d * code + m with one fp32 rounding; zeros for a slot out of range.
template <int D> __global__ void __launch_bounds__(kHeadWarps * 32) kv4_read_kernel(const ReadArgs a)
{
    constexpr int V = D / 32;
    using F = Kv4<D>;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t r = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); r < a.rows; r += (int64_t)gridDim.x * kHeadWarps) {
        const int64_t t = r / (2 * a.H);
        const int h = (int)(r - t * 2 * a.H);
        const bool isk = h < a.H;
        const int head = isk ? h : h - a.H;
        const int64_t slot = a.slot[t];
        float x[V] = {};
        if (slot >= 0 && slot < a.slots) {
            const int64_t pg = slot / a.page;
            const int in_page = (int)(slot - pg * a.page);
            const int blk = in_page / kKvBlock, tok = in_page % kKvBlock;
            const uint8_t *part = a.cache + ((pg * a.H + head) * (a.page / kKvBlock) + blk) * F::kBlock + (isk ? 0 : F::kPart);
            const uint8_t *at = part + kv4_code_offset<D>(tok, V * lane);
            uint32_t codes;
            if constexpr (V == 8)
                codes = *reinterpret_cast<const uint32_t *>(at);
            else if constexpr (V == 4)
                codes = *reinterpret_cast<const uint16_t *>(at);
            else
                codes = *at;
            const float2 dm = __half22float2(*reinterpret_cast<const __half2 *>(
                part + F::kCodes + (tok * F::kGroups + V * lane / kKvGroup) * 4));
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = fmaf((float)((codes >> (4 * i)) & 15u), dm.x, dm.y);
        }
        store_dims<V>(isk ? a.ko : a.vo, t, head, V * lane, x);
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

// Blocks along a token's heads: one row a warp while that leaves the card room, else the whole token in
// one block, so that its sines and cosines are made once (4099 tokens of 40 heads: see the kernel).
int head_blocks(int64_t T, int rows, int sms)
{
    const int most = (rows + kHeadWarps - 1) / kHeadWarps;
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
    const int V = D / 32;
    if (Hq > 0) {
        if ((rc = check_view(q, T, Hq, V, false, &a.q)) != QG_OK) return rc;
        if ((rc = check_view(q_out, T, Hq, V, false, &a.qo)) != QG_OK) return rc;
    }
    if (Hk > 0) {
        if ((rc = check_view(k, T, Hk, V, false, &a.k)) != QG_OK) return rc;
        if ((rc = check_view(k_out, T, Hk, V, false, &a.ko)) != QG_OK) return rc;
    }
    if (reinterpret_cast<uintptr_t>(wq) % 4 || reinterpret_cast<uintptr_t>(wk) % 4) return QG_ERR_ALIGN;
    a.wq = wq;
    a.wk = wk;
    a.eps = eps;
    a.Hq = Hq;
    a.Hk = Hk;
    int sms = 0;
    if ((rc = current_sms(&sms)) != QG_OK) return rc;
    const dim3 grid((unsigned)T, head_blocks(T, Hq + Hk, sms)), block(kHeadWarps * 32);
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
    if ((rc = check_view(k, T, H, D / 32, false, &a.k)) != QG_OK) return rc;
    if ((rc = check_view(v, T, H, D / 32, false, &a.v)) != QG_OK) return rc;
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
    const dim3 grid((unsigned)T, head_blocks(T, 2 * H, sms)), block(kHeadWarps * 32);
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
    if ((rc = check_view(k_out, T, H, D / 32, false, &a.ko)) != QG_OK) return rc;
    if ((rc = check_view(v_out, T, H, D / 32, false, &a.vo)) != QG_OK) return rc;
    if (reinterpret_cast<uintptr_t>(slot) % 8) return QG_ERR_ALIGN;
    a.slot = slot;
    a.cache = static_cast<const uint8_t *>(cache);
    a.slots = pages * page;
    a.rows = T * 2 * H;
    a.page = page;
    a.H = H;
    int sms = 0;
    if ((rc = current_sms(&sms)) != QG_OK) return rc;
    const dim3 grid((unsigned)std::min<int64_t>((a.rows + kHeadWarps - 1) / kHeadWarps, (int64_t)sms * 8));
    const dim3 block(kHeadWarps * 32);
    switch (D) {
    case 64: return launch_pdl(kv4_read_kernel<64>, grid, block, 0, stream, a);
    case 128: return launch_pdl(kv4_read_kernel<128>, grid, block, 0, stream, a);
    default: return launch_pdl(kv4_read_kernel<256>, grid, block, 0, stream, a);
    }
}

}  // extern "C"
