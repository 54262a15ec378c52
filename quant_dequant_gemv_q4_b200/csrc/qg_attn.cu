// qg_attn.cu -- attention over the paged 4-bit cache (qg_attn_kv4).  Declaration and contract:
// include/qg.h; cache format: qg_kv4.cuh.
//
//   out[t,h] = sum_p softmax_p(scale * q[t,h] . k[p, h/G]) v[p, h/G],   p <= len - n + i
//
// for the i-th of the n query tokens of a sequence of len places: k, v = d * code + m.
//
// What bounds it.  Each place of a key head is 2 * 4.5 bits a dimension, read once for up to 16 query
// rows (G heads x n tokens): at 12 rows 9 bytes feed 48 multiply-adds, so a step that decodes few
// tokens is bound by the cache's bytes as long as the unpacking (about 1.7 instructions a value) and
// the matrix instructions keep up.
//
// attn_kv4_kernel.  One warp takes 16 query rows and a tile of 16 places:
//   S[16 x 16] = Q K^T  and  O[16 x D] += P V  by mma.sync m16n8k16 (f16 operands, fp32 sums).
// The codes go from shared memory straight into the B fragments: the assignment of dimensions to the
// k index of the first product, and of dimensions to the n index of the second, is free, and is chosen
// so that a lane's 4-byte words hold only nibbles of its own fragments (kq_dims, v_dims).  Nothing is
// transposed, and the unpacked values are never stored.
// Four warps of a CTA take the four tiles of a 64-place unit; each keeps its own running maximum, sum
// and O, with no synchronization in the loop, and the four are joined in shared memory at the end of a
// row tile.  Each warp's lane 0 keeps a ring of bulk copies in flight, a block (18 D bytes) each.
//
// Splitting.  The units of all (sequence, head, row tile) items are numbered in one line and dealt to
// the CTAs in equal runs, so ragged batches and single long sequences fill the card alike.  An item cut
// between CTAs leaves partial (O, maximum, sum) in the workspace, which attn_kv4_join_kernel adds up in
// CTA order: results do not depend on timing.
//
// Softmax in base 2 on fp32 scores.  The reference maximum of a row moves only when a score exceeds it
// by more than 8 (so rarely after the first tiles), and the weights carry a factor 2^7: at most 2^15,
// and full fp16 precision down to 2^-21 of the reference.
#include <algorithm>

#include "qg_kv4.cuh"
#include "qg_ptx.cuh"

namespace {

using namespace qg;

constexpr int kAttnWarps = 4;
constexpr int kUnit = kAttnWarps * kKvBlock;  // places of a unit
constexpr int kRows = 16;                     // query rows of an item
constexpr float kMoveMax = 8.0f;              // a score this far above the reference moves it
constexpr float kWeightShift = 7.0f;          // weights are 2^(s - reference + 7)

template <int D> struct AttnCfg;
template <> struct AttnCfg<256> { static constexpr int kStages = 5, kCtas = 2; };
template <> struct AttnCfg<128> { static constexpr int kStages = 6, kCtas = 3; };
template <> struct AttnCfg<64> { static constexpr int kStages = 8, kCtas = 4; };

constexpr int kJoinStride = 68;  // floats of a row of the joining buffer (64 and a shift of four banks)

template <int D> struct AttnSmem {
    static constexpr int kRing = kAttnWarps * AttnCfg<D>::kStages * Kv4<D>::kBlock;
    static constexpr int kJoin = kAttnWarps * kRows * kJoinStride * 4;
    static constexpr int kBytes = kRing + kJoin;
};

struct AttnArgs {
    HeadsView q, out;
    const uint8_t *cache;
    const int32_t *table, *start, *len;
    int64_t pages, T;
    float *part;     // [2 grid][kRows][D]
    float2 *stat;    // [2 grid][kRows] (reference, sum)
    int4 *cut;       // items cut between CTAs: {sequence, head, row tile, CTAs}, CTAs = 0 for none
    int *err;
    float scale_log2;
    int nseq, page, width, Hk, G, by_item;
};

// What the schedule needs of a sequence.
struct Seq {
    int first, n, len, tiles, units;  // first query row in T, query tokens, places, row tiles, units of an item
};

__device__ __forceinline__ Seq load_seq(const AttnArgs &a, int s)
{
    Seq q;
    const int64_t lo = a.start[s], hi = a.start[s + 1];
    const bool ok = lo >= 0 && hi > lo && lo < a.T;
    q.first = ok ? (int)lo : 0;
    q.n = ok ? (int)((hi < a.T ? hi : a.T) - lo) : 0;
    const int64_t cap = (int64_t)a.width * a.page;
    const int64_t len = a.len[s];
    q.len = (int)(len < 0 ? 0 : len < cap ? len : cap);
    q.tiles = (int)(((int64_t)q.n * a.G + kRows - 1) / kRows);
    q.units = q.len > 0 ? (q.len + kUnit - 1) / kUnit : 1;  // an empty sequence still writes its zeros
    return q;
}

__device__ __forceinline__ int64_t seq_units(const AttnArgs &a, const Seq &q) { return (int64_t)q.tiles * a.Hk * q.units; }

// A place in the line of units.
struct Cursor {
    Seq q;
    int s, item, unit;  // sequence, item of it (head * tiles + row tile), unit of the item
};

__device__ __forceinline__ void next_item(const AttnArgs &a, Cursor &c)
{
    c.unit = 0;
    if (++c.item < c.q.tiles * a.Hk) return;
    c.item = 0;
    do {
        if (++c.s >= a.nseq) return;
        c.q = load_seq(a, c.s);
    } while (c.q.tiles == 0);
}

__device__ __forceinline__ uint32_t lop_and_or(uint32_t x, uint32_t m, uint32_t o)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(m), "r"(o));  // (x & m) | o
    return r;
}

__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// Two codes at bits 0-3 (LO) or 4-7 of each half of x as d * code + m: the nibble under an exponent is
// 1024 + code (or 1024 + 16 code), made the exact code by one f16x2 instruction; the second rounds the
// value to fp16 once (2^-11 relative, far below the step d).
__device__ __forceinline__ uint32_t dequant_lo(uint32_t x, __half2 d, __half2 m)
{
    const __half2 c = __hsub2(as_h2(lop_and_or(x, 0x000f000fu, 0x64006400u)), as_h2(0x64006400u));
    return as_u32(__hfma2(c, d, m));
}
__device__ __forceinline__ uint32_t dequant_hi(uint32_t x, __half2 d, __half2 m)
{
    // (1024 + 16 code) / 16 - 64
    const __half2 c = __hfma2(as_h2(lop_and_or(x, 0x00f000f0u, 0x64006400u)), as_h2(0x2c002c00u), as_h2(0xd400d400u));
    return as_u32(__hfma2(c, d, m));
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t lds32(const uint8_t *a) { return *reinterpret_cast<const uint32_t *>(a); }
template <int W> __device__ __forceinline__ void lds_words(const uint8_t *a, uint32_t *w)
{
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4 *>(a);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(a);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = lds32(a);
    }
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return as_u32(__floats2half2_rn(lo, hi)); }

// First of the 8 dimensions that word i of lane part t4 (lane % 4) holds of a K row.
template <int D> __device__ __forceinline__ int kq_dims(int t4, int i)
{
    if constexpr (D == 256) return 32 * t4 + 8 * (i & 3) + (i >> 2) * 128;
    return (D / 4) * t4 + 8 * i;
}

template <int D> __global__ void __launch_bounds__(kAttnWarps * 32, AttnCfg<D>::kCtas) attn_kv4_kernel(const AttnArgs a)
{
    using F = Kv4<D>;
    constexpr int kStages = AttnCfg<D>::kStages;
    constexpr int KW = D / 32;  // 4-byte words of a K row a lane holds
    constexpr int NT = D / 8;   // n tiles of O
    constexpr int VW = D / 64;  // 4-byte words of a V row a lane holds
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kAttnWarps * kStages];
    __shared__ int tile_ok[kAttnWarps][kStages];
    __shared__ Cursor ahead[kAttnWarps];  // where lane 0's copies are
    __shared__ float2 wstat[kAttnWarps][kRows];
    __shared__ int64_t scan[kAttnWarps + 1];
    __shared__ Cursor found;
    __shared__ int found_item0;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t4 = lane & 3;
    const int cta = blockIdx.x, grid = gridDim.x;
    uint8_t *ring = smem + warp * kStages * F::kBlock;
    const uint32_t bar0 = smem_u32(bars) + warp * kStages * 8;
    float *join = reinterpret_cast<float *>(smem + AttnSmem<D>::kRing);

    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(bar0 + 8 * i, 1);
        mbar_init_fence();
    }
    pdl_launch_dependents();
    pdl_wait();
    if (cta == 0 && threadIdx.x == 0) *a.err = 0;

    // The run of units of this CTA: the units of all sequences, then the sequence its first one is in.
    int64_t total = 0;
    for (int s0 = 0; s0 < a.nseq; s0 += kAttnWarps * 32) {
        const int s = s0 + threadIdx.x;
        if (s < a.nseq) {
            const Seq q = load_seq(a, s);
            total += seq_units(a, q);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) scan[warp] = total;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) total += scan[w];
    const int64_t per = (total + grid - 1) / grid;
    const int64_t begin = per * cta < total ? per * cta : total;
    const int64_t end = begin + per < total ? begin + per : total;
    if (begin == end) {
        if (threadIdx.x == 0 && !a.by_item) a.cut[cta] = make_int4(0, 0, 0, 0);
        if (cta == 0 && a.by_item)
            for (int i = threadIdx.x; i < grid; i += blockDim.x) a.cut[i] = make_int4(0, 0, 0, 0);
        return;
    }
    {
        int64_t base = 0;
        int items = 0;  // items of the sequences before
        for (int s0 = 0; s0 < a.nseq; s0 += kAttnWarps * 32) {
            const int s = s0 + threadIdx.x;
            Seq q = {};
            if (s < a.nseq) q = load_seq(a, s);
            const int64_t u = s < a.nseq ? seq_units(a, q) : 0;
            int64_t up = u;
            int it = q.tiles * a.Hk, itp = it;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, up, o);
                const int w = __shfl_up_sync(0xffffffffu, itp, o);
                if (lane >= o) {
                    up += v;
                    itp += w;
                }
            }
            __syncthreads();
            __shared__ int iscan[kAttnWarps];
            if (lane == 31) {
                scan[warp] = up;
                iscan[warp] = itp;
            }
            __syncthreads();
            int64_t before = base + up - u;
            int ibefore = items + itp - it;
            for (int w = 0; w < kAttnWarps; ++w) {
                if (w < warp) {
                    before += scan[w];
                    ibefore += iscan[w];
                }
                base += scan[w];
                items += iscan[w];
            }
            if (begin >= before && begin < before + u) {
                Cursor c;
                c.q = q;
                c.s = s;
                c.item = (int)((begin - before) / q.units);
                c.unit = (int)((begin - before) % q.units);
                found = c;
                found_item0 = ibefore;
            }
        }
        __syncthreads();
        // the join looks at every entry that the argument sizes allow for
        if (cta == 0 && a.by_item)
            for (int i = items + (int)threadIdx.x; i < grid; i += blockDim.x) a.cut[i] = make_int4(0, 0, 0, 0);
    }
    Cursor cur = found;
    int item_no = found_item0 + cur.item;  // number of the item among all
    const int count = (int)(end - begin);

    // Copies: lane 0 walks the same run, kStages - 1 units ahead.
    int issued = 0;
    if (lane == 0) ahead[warp] = cur;
    auto issue = [&]() {  // lane 0 only
        if (issued >= count) return;
        Cursor &c = ahead[warp];
        const int stage = issued % kStages;
        const int pos = c.unit * kUnit + warp * kKvBlock;
        const int head = c.item / c.q.tiles;
        int64_t pg = -1;
        const int pi = pos / a.page;
        if (pos < c.q.len) pg = a.table[(int64_t)c.s * a.width + pi];
        const bool ok = pg >= 0 && pg < a.pages;
        tile_ok[warp][stage] = ok;
        const uint32_t bar = bar0 + 8 * stage;
        mbar_arrive_expect_tx(bar, ok ? F::kBlock : 0);
        if (ok) {
            const int64_t blk = (pg * a.Hk + head) * (a.page / kKvBlock) + (pos - pi * a.page) / kKvBlock;
            bulk_g2s_plain(smem_u32(ring + stage * F::kBlock), a.cache + blk * F::kBlock, F::kBlock, bar);
        }
        ++issued;
        if (++c.unit == c.q.units) next_item(a, c);
    };
    __syncwarp();
    if (lane == 0)
        for (int i = 0; i < kStages - 1; ++i) issue();

    uint32_t qf[D / 16][4];
    float o[NT][4];
    float ref[2], sum[2];  // rows g and g + 8
    int lim[2];            // the last place each row sees
    bool dead = false, fresh = true;
    bool any_cut = false;

    for (int i = 0; i < count; ++i) {
        const int head = cur.item / cur.q.tiles;
        const int rt = cur.item - head * cur.q.tiles;
        if (fresh) {  // a new item, or this CTA's part of it
            fresh = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                ref[r] = -INFINITY;
                sum[r] = 0.0f;
                const int row = rt * kRows + g + 8 * r;
                const int tok = row / a.G;
                const bool ok = tok < cur.q.n;
                lim[r] = ok ? cur.q.len - cur.q.n + tok : -1;
                const __half *qp = static_cast<const __half *>(a.q.p) + (int64_t)(cur.q.first + tok) * a.q.st +
                                   (int64_t)(head * a.G + row - tok * a.G) * a.q.sh;
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    const int dim = kq_dims<D>(t4, w);
                    uint32_t v[4] = {0, 0, 0, 0};  // dimension pairs (0,1) (2,3) (4,5) (6,7)
                    if (ok) {
                        if (a.q.vec > 1) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(qp + dim);
                            v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[e] = as_u32(__halves2half2(qp[(dim + 2 * e) * a.q.sd], qp[(dim + 2 * e + 1) * a.q.sd]));
                        }
                    }
                    // the pairs that the nibbles of a word come in: (0,4) (1,5) (2,6) (3,7)
                    qf[2 * w][r] = __byte_perm(v[0], v[2], 0x5410);
                    qf[2 * w][2 + r] = __byte_perm(v[0], v[2], 0x7632);
                    qf[2 * w + 1][r] = __byte_perm(v[1], v[3], 0x5410);
                    qf[2 * w + 1][2 + r] = __byte_perm(v[1], v[3], 0x7632);
                }
            }
        }
        const int stage = i % kStages;
        if (lane == 0) issue();  // into the stage that the previous tile left
        if (!dead && !mbar_wait_bounded(bar0 + 8 * stage, (uint32_t)((i / kStages) & 1))) {
            dead = true;
            if (lane == 0) *a.err = 1;
        }
        const int pos = cur.unit * kUnit + warp * kKvBlock;
        // the last place that any row of the item sees
        const int tmax = min(cur.q.n - 1, (rt * kRows + kRows - 1) / a.G);
        const int seen = cur.q.len - cur.q.n + tmax;
        if (!dead && pos <= seen && tile_ok[warp][stage]) {
            const uint8_t *kb = ring + stage * F::kBlock;
            const uint8_t *vb = kb + F::kPart;
            const bool masked = pos + kKvBlock - 1 > cur.q.len - cur.q.n + (rt * kRows) / a.G;
            // S = Q K^T: n tile j holds places 8 j .. 8 j + 7, two accumulator chains each
            float sc[2][2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[j][0][e] = sc[j][1][e] = 0.0f;
                const int tok = g + 8 * j;
                const int sw = kv4_swizzle(tok) & F::kChunkMask;
                uint32_t w[KW];
                __half2 d[2], m[2];
                if constexpr (D == 256) {
                    lds_words<4>(kb + tok * F::kCodeRow + ((t4 ^ sw) << 4), w);
                    lds_words<4>(kb + tok * F::kCodeRow + (((t4 + 4) ^ sw) << 4), w + 4);
                    const uint32_t s0 = lds32(kb + F::kCodes + (tok * F::kGroups + (t4 >> 1)) * 4);
                    const uint32_t s1 = lds32(kb + F::kCodes + (tok * F::kGroups + 2 + (t4 >> 1)) * 4);
                    d[0] = __low2half2(as_h2(s0)), m[0] = __high2half2(as_h2(s0));
                    d[1] = __low2half2(as_h2(s1)), m[1] = __high2half2(as_h2(s1));
                } else if constexpr (D == 128) {
                    lds_words<4>(kb + tok * F::kCodeRow + ((t4 ^ sw) << 4), w);
                    const uint32_t s0 = lds32(kb + F::kCodes + (tok * F::kGroups + (t4 >> 1)) * 4);
                    d[0] = d[1] = __low2half2(as_h2(s0)), m[0] = m[1] = __high2half2(as_h2(s0));
                } else {
                    lds_words<2>(kb + tok * F::kCodeRow + (((t4 >> 1) ^ sw) << 4) + (t4 & 1) * 8, w);
                    const uint32_t s0 = lds32(kb + F::kCodes + tok * F::kGroups * 4);
                    d[0] = d[1] = __low2half2(as_h2(s0)), m[0] = m[1] = __high2half2(as_h2(s0));
                }
#pragma unroll
                for (int k = 0; k < KW; ++k) {
                    const __half2 dd = d[k >> 2], mm = m[k >> 2];
                    const uint32_t w8 = w[k] >> 8;
                    mma16816(sc[j][0], qf[2 * k][0], qf[2 * k][1], qf[2 * k][2], qf[2 * k][3], dequant_lo(w[k], dd, mm),
                             dequant_hi(w[k], dd, mm));
                    mma16816(sc[j][1], qf[2 * k + 1][0], qf[2 * k + 1][1], qf[2 * k + 1][2], qf[2 * k + 1][3],
                             dequant_lo(w8, dd, mm), dequant_hi(w8, dd, mm));
                }
            }
            float s[2][4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j][e] = (sc[j][0][e] + sc[j][1][e]) * a.scale_log2;
            if (masked) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (pos + 8 * j + 2 * t4 + (e & 1) > lim[e >> 1]) s[j][e] = -INFINITY;
            }
            float top[2];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                top[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
            if (__any_sync(0xffffffffu, top[0] > ref[0] + kMoveMax || top[1] > ref[1] + kMoveMax)) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float t = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    t = fmaxf(t, ref[r]);
                    const float f = t == -INFINITY ? 1.0f : ex2(ref[r] - t);
                    ref[r] = t;
                    sum[r] *= f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[n][2 * r] *= f;
                        o[n][2 * r + 1] *= f;
                    }
                }
            }
            uint32_t p[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float base = (ref[r] == -INFINITY ? 0.0f : ref[r]) - kWeightShift;
                float e[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    e[x] = ex2(s[x >> 1][2 * r + (x & 1)] - base);
                    sum[r] += e[x];
                }
                p[r] = pack_h2(e[0], e[1]);
                p[2 + r] = pack_h2(e[2], e[3]);
            }
            // O += P V: the k index is the place, 2 t4 + {0, 1} and 8 more; word i of a lane's V
            // row holds n tiles 8 i .. 8 i + 7 of column g
            uint32_t w[4][VW];
            uint32_t sv[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int tok = 2 * t4 + (x & 1) + 8 * (x >> 1);
                const int sw = kv4_swizzle(tok) & F::kChunkMask;
                const int dim = (D / 8) * g;
                lds_words<VW>(vb + tok * F::kCodeRow + (((dim >> 5) ^ sw) << 4) + ((dim & 31) >> 1), w[x]);
                sv[x] = lds32(vb + F::kCodes + (tok * F::kGroups + dim / kKvGroup) * 4);
                // places past the sequence hold anything, NaN among it
                if (masked && pos + tok >= cur.q.len) sv[x] = 0;
            }
            const __half2 d0 = as_h2(__byte_perm(sv[0], sv[1], 0x5410)), m0 = as_h2(__byte_perm(sv[0], sv[1], 0x7632));
            const __half2 d1 = as_h2(__byte_perm(sv[2], sv[3], 0x5410)), m1 = as_h2(__byte_perm(sv[2], sv[3], 0x7632));
#pragma unroll
            for (int v = 0; v < VW; ++v) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sel = half ? 0x7632 : 0x5410;
                    const uint32_t x = __byte_perm(w[0][v], w[1][v], sel), y = __byte_perm(w[2][v], w[3][v], sel);
                    const uint32_t x8 = x >> 8, y8 = y >> 8;
                    const int n = 8 * v + 4 * half;
                    mma16816(o[n], p[0], p[1], p[2], p[3], dequant_lo(x, d0, m0), dequant_lo(y, d1, m1));
                    mma16816(o[n + 1], p[0], p[1], p[2], p[3], dequant_hi(x, d0, m0), dequant_hi(y, d1, m1));
                    mma16816(o[n + 2], p[0], p[1], p[2], p[3], dequant_lo(x8, d0, m0), dequant_lo(y8, d1, m1));
                    mma16816(o[n + 3], p[0], p[1], p[2], p[3], dequant_hi(x8, d0, m0), dequant_hi(y8, d1, m1));
                }
            }
        }
        __syncwarp();  // every lane has read the stage before lane 0 fills it again
        const bool whole_end = cur.unit + 1 == cur.q.units;
        if (whole_end || i + 1 == count) {
            // ---- end of this CTA's part of the item: join the warps
            const bool from_start = cur.unit + 1 <= i + 1;  // unit 0 was in this run
            const bool complete = whole_end && from_start;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
                sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
                if (t4 == 0) wstat[warp][g + 8 * r] = make_float2(ref[r], sum[r]);
            }
            __syncthreads();
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float t = -INFINITY;
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) t = fmaxf(t, wstat[w][g + 8 * r].x);
                f[r] = ref[r] == -INFINITY ? 0.0f : ex2(ref[r] - t);
            }
            // the thread's element of the joined tile: a row and D / 8 dimensions of it
            const int jr = threadIdx.x >> 3, jn = threadIdx.x & 7;
            float top = -INFINITY, den = 0.0f;
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, wstat[w][jr].x);
#pragma unroll
            for (int w = 0; w < kAttnWarps; ++w) {
                const float2 st = wstat[w][jr];
                if (st.x != -INFINITY) den += st.y * ex2(st.x - top);
            }
            const float inv = den > 0.0f ? 1.0f / den : 0.0f;
            const int row = rt * kRows + jr;
            const int tok = row / a.G;
            const bool row_ok = tok < cur.q.n;
            const int slot = 2 * cta + (from_start ? 1 : 0);
#pragma unroll
            for (int c = 0; c < NT / 8; ++c) {
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float *dst = join + ((warp * kRows) + g + 8 * r) * kJoinStride + (2 * t4 + e) * 8;
#pragma unroll
                        for (int h = 0; h < 8; h += 4)
                            *reinterpret_cast<float4 *>(dst + h) =
                                make_float4(o[8 * c + h][2 * r + e] * f[r], o[8 * c + h + 1][2 * r + e] * f[r],
                                            o[8 * c + h + 2][2 * r + e] * f[r], o[8 * c + h + 3][2 * r + e] * f[r]);
                    }
                __syncthreads();
                float v[8] = {};
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    const float *src = join + (w * kRows + jr) * kJoinStride + jn * 8;
#pragma unroll
                    for (int h = 0; h < 8; h += 4) {
                        const float4 x = *reinterpret_cast<const float4 *>(src + h);
                        v[h] += x.x, v[h + 1] += x.y, v[h + 2] += x.z, v[h + 3] += x.w;
                    }
                }
                const int dim = (D / 8) * jn + 8 * c;
                if (complete) {
                    if (row_ok) {
#pragma unroll
                        for (int h = 0; h < 8; ++h) v[h] *= inv;
                        store_dims<8>(a.out, cur.q.first + tok, head * a.G + row - tok * a.G, dim, v);
                    }
                } else {
                    float *dst = a.part + ((int64_t)slot * kRows + jr) * D + dim;
#pragma unroll
                    for (int h = 0; h < 8; h += 4) *reinterpret_cast<float4 *>(dst + h) = make_float4(v[h], v[h + 1], v[h + 2], v[h + 3]);
                }
                __syncthreads();
            }
            if (!complete && jn == 0) a.stat[slot * kRows + jr] = make_float2(top, den);
            if (from_start && threadIdx.x == 0) {
                const int left = cur.q.units - cur.unit - 1;  // units of the item in the CTAs after this one
                const int4 c = complete ? make_int4(0, 0, 0, 0)
                                        : make_int4(cur.s, head, rt, (int)(1 + (left + per - 1) / per));
                if (a.by_item) {
                    if (item_no < grid) a.cut[item_no] = make_int4(c.x, c.y | (cta << 16), c.z, c.w);
                } else if (!complete) {
                    a.cut[cta] = make_int4(c.x, c.y | (cta << 16), c.z, c.w);
                    any_cut = true;
                }
            }
            fresh = true;
        }
        if (++cur.unit == cur.q.units) {
            next_item(a, cur);
            ++item_no;
        }
    }
    if (!a.by_item && threadIdx.x == 0 && !any_cut) a.cut[cta] = make_int4(0, 0, 0, 0);
}

// The items that were cut between CTAs: out = sum_i 2^(ref_i - ref) O_i / sum_i 2^(ref_i - ref) sum_i,
// in CTA order.  One block takes RB rows of one item; D / 4 threads share a row's dimensions and the
// rest of its threads the parts.
template <int D, int RB> __global__ void __launch_bounds__(256) attn_kv4_join_kernel(const AttnArgs a)
{
    constexpr int TX = D / 4;              // threads across a row
    constexpr int TY = 256 / (TX * RB);    // threads that share its parts
    static_assert(TY >= 1, "a row's threads fit the block");
    __shared__ float4 acc[RB][TY][TX];
    __shared__ float den[RB][TY];
    pdl_launch_dependents();
    pdl_wait();
    const int4 c = a.cut[blockIdx.x];
    if (c.w == 0) return;
    const int head = c.y & 0xffff, cta = c.y >> 16;
    const int x = threadIdx.x % TX, y = threadIdx.x / TX % TY, rl = threadIdx.x / (TX * TY);
    const int r = blockIdx.y * RB + rl;
    const Seq q = load_seq(a, c.x);
    const int row = c.z * kRows + r;
    const int tok = row / a.G;
    float top = -INFINITY;
    for (int i = 0; i < c.w; ++i) top = fmaxf(top, a.stat[(i ? 2 * (cta + i) : 2 * cta + 1) * kRows + r].x);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
#pragma unroll 4
    for (int i = y; i < c.w; i += TY) {
        const int slot = i ? 2 * (cta + i) : 2 * cta + 1;
        const float2 st = a.stat[slot * kRows + r];
        const float f = st.x == -INFINITY ? 0.0f : ex2(st.x - top);
        const float4 u = *reinterpret_cast<const float4 *>(a.part + ((int64_t)slot * kRows + r) * D + 4 * x);
        l = fmaf(st.y, f, l);
        v.x = fmaf(u.x, f, v.x);
        v.y = fmaf(u.y, f, v.y);
        v.z = fmaf(u.z, f, v.z);
        v.w = fmaf(u.w, f, v.w);
    }
    acc[rl][y][x] = v;
    if (x == 0) den[rl][y] = l;
    __syncthreads();
    if (y != 0 || tok >= q.n) return;
    for (int i = 1; i < TY; ++i) {
        const float4 u = acc[rl][i][x];
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    l = 0.0f;
    for (int i = 0; i < TY; ++i) l += den[rl][i];
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const float w[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
    store_dims<4>(a.out, q.first + tok, head * a.G + row - tok * a.G, 4 * x, w);
}

template <int D> int ctas(int sms) { return sms * AttnCfg<D>::kCtas; }

int attn_grid(int D, int sms) { return D == 256 ? ctas<256>(sms) : D == 128 ? ctas<128>(sms) : ctas<64>(sms); }

struct WsLayout {
    size_t part, stat, cut, bytes;
};

WsLayout ws_layout(int D, int grid)
{
    WsLayout w;
    w.part = 256;  // the error word first
    w.stat = w.part + (size_t)2 * grid * kRows * D * sizeof(float);
    w.cut = w.stat + (size_t)2 * grid * kRows * sizeof(float2);
    w.bytes = w.cut + (size_t)grid * sizeof(int4);
    return w;
}

template <int D> int launch_attn(const AttnArgs &a, int grid, int64_t items, void *stream)
{
    static std::atomic<uint64_t> raised{0};  // devices whose shared-memory limit is raised
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QG_ERR_CUDA;
    if (dev >= 64 || !(raised.load() >> dev & 1)) {
        if (cudaFuncSetAttribute(attn_kv4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, AttnSmem<D>::kBytes) != cudaSuccess)
            return QG_ERR_CUDA;
        if (dev < 64) raised.fetch_or(uint64_t(1) << dev);
    }
    int rc = launch_pdl(attn_kv4_kernel<D>, dim3(grid), dim3(kAttnWarps * 32), AttnSmem<D>::kBytes, stream, a);
    if (rc != QG_OK) return rc;
    // no item is cut when none has more than one unit
    if ((int64_t)a.width * a.page <= kUnit) return QG_OK;
    if (a.by_item)
        return launch_pdl(attn_kv4_join_kernel<D, 1>, dim3((unsigned)items, kRows), dim3(256), 0, stream, a);
    return launch_pdl(attn_kv4_join_kernel<D, 4>, dim3(grid, kRows / 4), dim3(256), 0, stream, a);
}

bool good_dim(int D) { return D == 64 || D == 128 || D == 256; }

}  // namespace

extern "C" {

size_t qg_attn_kv4_workspace(int D)
{
    int sms = 0;
    if (!good_dim(D) || current_sms(&sms) != QG_OK) return 0;
    return ws_layout(D, attn_grid(D, sms)).bytes;
}

int qg_attn_kv4(const qg_heads *q, int64_t T, int nseq, const int32_t *q_start, int max_q, int Hq, int Hk, int D,
                const void *cache, int64_t pages, int page, const int32_t *table, int width, const int32_t *kv_len,
                float scale, const qg_heads *out, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!good_dim(D) || T < 0 || T > 0x7fffffff || nseq < 0 || max_q < 0 || Hk < 1 || Hq < Hk || Hq % Hk || Hq > QG_MAX_HEADS ||
        page < kKvBlock || page % kKvBlock || width < 0 || pages < 0 || (int64_t)width * page > 0x7fffff00)
        return QG_ERR_SHAPE;
    if (pages > 0 && qg_kv4_bytes(pages, page, Hk, D) == 0) return QG_ERR_SHAPE;
    if (T == 0 || nseq == 0) return QG_OK;
    if (!q_start || !kv_len || (width > 0 && !table) || (pages > 0 && !cache) || !workspace) return QG_ERR_NULL;
    AttnArgs a = {};
    int rc = check_view(q, T, Hq, 8, true, &a.q);
    if (rc != QG_OK) return rc;
    if ((rc = check_view(out, T, Hq, 8, true, &a.out)) != QG_OK) return rc;
    if (reinterpret_cast<uintptr_t>(cache) % 16 || reinterpret_cast<uintptr_t>(workspace) % 256 ||
        reinterpret_cast<uintptr_t>(table) % 4 || reinterpret_cast<uintptr_t>(q_start) % 4 || reinterpret_cast<uintptr_t>(kv_len) % 4)
        return QG_ERR_ALIGN;
    int sms = 0;
    if ((rc = current_sms(&sms)) != QG_OK) return rc;
    const int grid = attn_grid(D, sms);
    const WsLayout w = ws_layout(D, grid);
    if (workspace_bytes < w.bytes) return QG_ERR_SCRATCH;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    a.err = reinterpret_cast<int *>(base);
    a.part = reinterpret_cast<float *>(base + w.part);
    a.stat = reinterpret_cast<float2 *>(base + w.stat);
    a.cut = reinterpret_cast<int4 *>(base + w.cut);
    a.cache = static_cast<const uint8_t *>(cache);
    a.table = table;
    a.start = q_start;
    a.len = kv_len;
    a.pages = pages;
    a.T = T;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.nseq = nseq;
    a.page = page;
    a.width = width;
    a.Hk = Hk;
    a.G = Hq / Hk;
    // items at most: a row tile may be short in every sequence
    const int64_t items = (int64_t)Hk * (nseq + T * a.G / kRows);
    a.by_item = items <= grid;
    switch (D) {
    case 64: return launch_attn<64>(a, grid, items, stream);
    case 128: return launch_attn<128>(a, grid, items, stream);
    default: return launch_attn<256>(a, grid, items, stream);
    }
}

}  // extern "C"
