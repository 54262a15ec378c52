// qg_attn.cu -- attention over the paged 4-bit cache (qg_attn_kv4).  Declaration and contract:
// include/qg.h; cache format: qg_kv4.cuh.
//
//   out[t,h] = sum_p softmax_p(scale * q[t,h] . k[p, h/G]) v[p, h/G],   p <= len - n + i
//
// for the i-th of the n query tokens of a sequence of len places: k, v = d * code + m.
//
// An item is a key head of a sequence and up to N of its query rows (G heads x n tokens, N = 16 .. 128); it
// is worked through in tiles of 128 places.  Both products run on the fifth-generation tensor cores with
// the cache as the A operand, M = 128, and the query rows as the N columns:
//   S^T[128 places x N] = K[128 x D] Q^T        A: unpacked keys in tensor memory, lane = place
//   O^T[D x N]         += V^T[D x 128] P^T      A: unpacked values in tensor memory, lane = dimension
// so few query rows cost few tensor cycles (at N = 16 both products of a tile take about a tenth of the
// time its bytes take to arrive), accumulators take no registers, and the unpacked cache never passes
// through shared memory, whose bandwidth would bound the kernel (16 KB of fp16 written and read back for
// each 16 places, against 4.6 KB of codes).
//   Keys: a thread unpacks one place's row and writes it to its tensor-memory lane (tcgen05.st 32x32b).
//   Values: ldmatrix.trans on 16-bit elements (four nibbles: four dimensions of a place) gives a thread two
//   neighbouring places of four dimensions; masking out each of the four nibbles leaves the fp16 pair
//   that one tensor-memory column of that dimension's lane holds, and tcgen05.st 16x128b has just this
//   fragment's shape: the transposition costs nothing.
// Which k index a dimension has in the first product, and which lane in the second, is free: the nibble
// order is left as it falls, q is staged in that order and O is unscrambled when it is written.
//
// Roles of a CTA's warps (one CTA an SM): a producer (a bulk copy of 18 D bytes for each 16 places, several
// tiles ahead), four warps that unpack keys, four for values, four (N = 128: eight) for the softmax, and
// one that issues the matrix instructions.  Key and value operands are double-buffered in parts of a tile
// (kSub), scores and weights in tiles, all handed over by mbarriers.
//
// Softmax in base 2 on fp32 scores.  A thread holds one place's scores; the reference maximum of a row is
// shared by the 128 places and moves only when a score exceeds it by more than 8 (so hardly ever after the
// first tile), so that in the common tile nothing is reduced across threads: weights are
// 2^(s - reference + 7), at most 2^15 and of full fp16 precision down to 2^-21 of the reference, and a
// thread adds up its own places' weights until the item ends.
//
// Splitting.  The tiles of all items are numbered in one line and dealt to the CTAs in equal runs, so ragged
// batches and single long sequences fill the card alike.  An item cut between CTAs leaves partial
// (O, reference, sum) in the workspace, which attn_kv4_join_kernel adds up in CTA order: results do not
// depend on timing.
#include <algorithm>
#include <cstddef>

#include "qg_kv4.cuh"
#include "qg_ptx.cuh"
#include "qg_tcgen05.cuh"

namespace {

using namespace qg;

constexpr int kTile = 128;                      // places of a tile
constexpr int kTileBlocks = kTile / kKvBlock;
constexpr float kMoveMax = 8.0f;                // a score this far above the reference moves it
constexpr float kWeightShift = 7.0f;
constexpr int kMetas = 16;                      // tiles whose description is kept (more than any role lags)

// flags of a tile
constexpr int kFirst = 1;      // first of this CTA's part of its item
constexpr int kLast = 2;       // last of it
constexpr int kFromStart = 4;  // the part holds the item's first tile
constexpr int kComplete = 8;   // the part is the whole item

struct AttnArgs {
    HeadsView q, out;
    const uint8_t *cache;
    const int32_t *table, *start, *len;
    int64_t pages, T;
    float *part;   // [2 grid][N][D]
    float2 *stat;  // [2 grid][N] (reference, sum)
    int4 *cut;     // items cut between CTAs: {sequence, head | first CTA << 16, row tile, CTAs}, CTAs = 0: none
    int *err;
    float scale_log2;
    int nseq, page, width, Hk, G, by_item;
};

struct Seq {
    int first, n, len, tiles;  // first query row in T, query tokens, places, row tiles
};

template <int N> __device__ __forceinline__ Seq load_seq(const AttnArgs &a, int s)
{
    Seq q;
    const int64_t lo = a.start[s], hi = a.start[s + 1];
    const bool ok = lo >= 0 && hi > lo && lo < a.T;
    q.first = ok ? (int)lo : 0;
    q.n = ok ? (int)((hi < a.T ? hi : a.T) - lo) : 0;
    const int64_t cap = (int64_t)a.width * a.page;
    const int64_t len = a.len[s];
    q.len = (int)(len < 0 ? 0 : len < cap ? len : cap);
    q.tiles = (int)(((int64_t)q.n * a.G + N - 1) / N);
    return q;
}

// Tiles of the item of row tile rt: down to the last place that any of its rows sees (one for rows that see
// nothing: their zeros are still written).
template <int N> __device__ __forceinline__ int item_units(const AttnArgs &a, const Seq &q, int rt)
{
    const int64_t last = ((int64_t)rt * N + N - 1) / a.G;
    const int tok = (int)(last < q.n - 1 ? last : q.n - 1);
    const int seen = q.len - q.n + tok + 1;
    return seen > 0 ? (seen + kTile - 1) / kTile : 1;
}

template <int N> __device__ __forceinline__ int64_t head_units(const AttnArgs &a, const Seq &q)
{
    int64_t u = 0;
    for (int rt = 0; rt < q.tiles; ++rt) u += item_units<N>(a, q, rt);
    return u;
}

// A place in the line of tiles.
struct Cursor {
    Seq q;
    int s, head, rt, unit, units;
};

template <int N> __device__ __forceinline__ void next_item(const AttnArgs &a, Cursor &c)
{
    c.unit = 0;
    if (++c.rt == c.q.tiles) {
        c.rt = 0;
        if (++c.head == a.Hk) {
            c.head = 0;
            do {
                if (++c.s >= a.nseq) return;
                c.q = load_seq<N>(a, c.s);
            } while (c.q.tiles == 0);
        }
    }
    c.units = item_units<N>(a, c.q, c.rt);
}

// What the roles need to know of a tile.
struct Meta {
    int flags, valid, pos, first, n, len, s, head, rt, ctas, item, pad;
};

__device__ __forceinline__ uint32_t lop_and_or(uint32_t x, uint32_t m, uint32_t o)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(x), "r"(m), "r"(o));  // (x & m) | o
    return r;
}
__device__ __forceinline__ __half2 as_h2(uint32_t x) { return *reinterpret_cast<const __half2 *>(&x); }
__device__ __forceinline__ uint32_t as_u32(__half2 x) { return *reinterpret_cast<const uint32_t *>(&x); }

// Two codes at bits 0-3 (lo) or 4-7 (hi) of each half of x as d * code + m: the nibble under an exponent is
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

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) { return as_u32(__floats2half2_rn(lo, hi)); }
__device__ __forceinline__ int float_order(float x)
{
    const int b = __float_as_int(x);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float order_float(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7fffffff)); }

template <int D, int N> struct Cfg {
    using F = Kv4<D>;
    static constexpr int kSub = (D == 256 && N == 128) ? 4 : 2;  // operand buffers hold 1 / kSub of a tile
    static constexpr int kMh = D >= 128 ? D / 128 : 1;           // M = 128 halves of O^T
    static constexpr int kKCols = D / 2 / kSub;                  // columns of a key buffer: D / kSub dimensions
    static constexpr int kVTok = kTile / kSub;                   // places of a value buffer
    static constexpr int kVCols = kVTok / 2;                     // columns of it in each half
    static constexpr int kSBufs = (D == 256 && N == 128) ? 1 : 2;
    static constexpr int kPBufs = (D == 256 && N == 128) ? 1 : 2;
    static constexpr int kSoft = N > 64 ? 2 : 1;                 // softmax warpgroups
    static constexpr int kNS = N / kSoft;                        // query rows of each
    static constexpr int kWarps = 8 + 4 * kSoft + 2;
    // tensor memory columns
    static constexpr int kK = 0, kV = kK + 2 * kKCols, kS = kV + 2 * kVCols * kMh, kO = kS + kSBufs * N;
    static constexpr int kCols = kO + kMh * N;
    static_assert(kCols <= 512, "tensor memory");
    // shared memory
    static constexpr int kTileBytes = kTileBlocks * F::kBlock;
    static constexpr int kStages = D == 256 ? (N == 128 ? 3 : 4) : D == 128 ? 6 : 8;
    static constexpr int kQ = kStages * kTileBytes;
    static constexpr int kQBytes = N * D * 2;
    static constexpr int kP = kQ + kQBytes;
    static constexpr int kPBytes = N * kTile * 2;
    static constexpr int kOutStride = D + 4;
    static constexpr int kOutRows = 8;
    static constexpr int kOutBytes = kSoft * kOutRows * kOutStride * 4;
    static constexpr int kPAll = kPBufs * kPBytes > kOutBytes ? kPBufs * kPBytes : kOutBytes;
    static constexpr int kBytes = kP + kPAll;
    static_assert(kBytes <= 224 * 1024, "shared memory");
};

template <int N> struct Small {
    uint64_t ring_full[8], ring_empty[8];
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], s_empty[2], p_full[2], p_empty[2];
    uint64_t q_full, o_full, o_empty;
    Meta meta[kMetas];
    Cursor found;
    int found_item;
    int64_t scan[20];
    int iscan[20];
    uint32_t tmem;
    int dead, produced;    // produced: tiles described so far
    alignas(16) float base[N];  // reference - kWeightShift (0 in place of -inf)
    float ref[N];
    alignas(16) int lim[N];     // last place that a row sees
    float wred[8][N];      // by warp
    float inv[N];
    float factor[N];
};

// Waits for a phase; gives up after kWaitNs of wall time, or at once when another warp has.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, int *dead, int *err)
{
    const uint32_t b = smem_u32(bar);
    if (mbar_try_wait(b, parity)) return;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(b, parity)) {
        if (*(volatile int *)dead) return;
        if (global_timer_ns() - t0 > kWaitNs) {
            *(volatile int *)dead = 1;
            *err = 1;
            return;
        }
    }
}

// Waits until `need` tiles are described.
__device__ __forceinline__ void wait_described(int *produced, int need, int *dead, int *err)
{
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        int v;
        asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(produced)) : "memory");
        if (v >= need || *(volatile int *)dead) return;
        if (global_timer_ns() - t0 > kWaitNs) {
            *(volatile int *)dead = 1;
            *err = 1;
            return;
        }
    }
}

__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ bool bar_or(int id, int threads, bool p)
{
    int r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %3, 0;\n\tbarrier.cta.red.or.pred q, %1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((int)p)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Sums v[i] over the warp's lanes for M values: on return lane l holds the total of value l % M.
template <int M> __device__ __forceinline__ float reduce_scatter(float (&v)[M], int lane)
{
#pragma unroll
    for (int o = M / 2; o > 0; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const float give = up ? v[i] : v[i + o];
            const float keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    float r = v[0];
#pragma unroll
    for (int o = M; o < 32; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    return r;
}

// The dimension that lane `l` (0 .. 127) of half mh of O^T holds.
template <int D> __device__ __forceinline__ int o_dim(int l, int mh)
{
    const int w = l >> 5, r = l & 15, j = (l >> 4) & 1;
    if constexpr (D == 256) return 64 * w + 4 * r + 2 * mh + j;
    return 32 * w + 4 * (r & 7) + 2 * j + (r >> 3);
}

template <int D, int N> __global__ void __launch_bounds__(Cfg<D, N>::kWarps * 32, 1) attn_kv4_kernel(const AttnArgs a)
{
    using F = Kv4<D>;
    using C = Cfg<D, N>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) Small<N> sm;
    static_assert(offsetof(Small<N>, base) % 16 == 0 && offsetof(Small<N>, lim) % 16 == 0, "read four at a time");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x, grid = gridDim.x;
    constexpr int kProducer = C::kWarps - 2, kIssuer = C::kWarps - 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&sm.ring_full[i]), 1);
            mbar_init(smem_u32(&sm.ring_empty[i]), 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.k_full[i]), 4);
            mbar_init(smem_u32(&sm.k_empty[i]), 1);
            mbar_init(smem_u32(&sm.v_full[i]), 4);
            mbar_init(smem_u32(&sm.v_empty[i]), 1);
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.s_empty[i]), 4 * C::kSoft);
            mbar_init(smem_u32(&sm.p_full[i]), 4 * C::kSoft);
            mbar_init(smem_u32(&sm.p_empty[i]), 1);
        }
        mbar_init(smem_u32(&sm.q_full), 4 * C::kSoft);
        mbar_init(smem_u32(&sm.o_full), 1);
        mbar_init(smem_u32(&sm.o_empty), 4 * C::kSoft);
        mbar_init_fence();
        sm.dead = 0;
        sm.produced = 0;
    }
    // Tensor memory is taken only when the kernels before are done, and the kernels after may start only when
    // it is taken: neither then holds it while it waits for the other.
    pdl_wait();
    if (warp == kIssuer) tmem_alloc(smem_u32(&sm.tmem), 512);
    if (cta == 0 && threadIdx.x == 0) *a.err = 0;

    // ---- the run of tiles of this CTA: the tiles of all sequences, then the sequence its first one is in
    const int threads = C::kWarps * 32;
    int64_t total = 0;
    for (int s = threadIdx.x; s < a.nseq; s += threads) {
        const Seq q = load_seq<N>(a, s);
        total += head_units<N>(a, q) * a.Hk;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) sm.scan[warp] = total;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = sm.tmem;
    total = 0;
    for (int w = 0; w < C::kWarps; ++w) total += sm.scan[w];
    const int64_t per = (total + grid - 1) / grid;
    const int64_t begin = per * cta < total ? per * cta : total;
    const int64_t end = begin + per < total ? begin + per : total;
    const int count = (int)(end - begin);
    if (count == 0) {
        if (threadIdx.x == 0 && !a.by_item) a.cut[cta] = make_int4(0, 0, 0, 0);
        if (cta == 0 && a.by_item)
            for (int i = threadIdx.x; i < grid; i += threads) a.cut[i] = make_int4(0, 0, 0, 0);
    } else {
        int64_t base = 0;
        int items = 0;
        for (int s0 = 0; s0 < a.nseq; s0 += threads) {
            const int s = s0 + threadIdx.x;
            Seq q = {};
            int64_t hu = 0;
            if (s < a.nseq) {
                q = load_seq<N>(a, s);
                hu = head_units<N>(a, q);
            }
            const int64_t u = hu * a.Hk;
            const int it = q.tiles * a.Hk;
            int64_t up = u;
            int itp = it;
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
            if (lane == 31) {
                sm.scan[warp] = up;
                sm.iscan[warp] = itp;
            }
            __syncthreads();
            int64_t before = base + up - u;
            int ibefore = items + itp - it;
            for (int w = 0; w < C::kWarps; ++w) {
                if (w < warp) {
                    before += sm.scan[w];
                    ibefore += sm.iscan[w];
                }
                base += sm.scan[w];
                items += sm.iscan[w];
            }
            if (begin >= before && begin < before + u) {
                Cursor c;
                c.q = q;
                c.s = s;
                int64_t rest = begin - before;
                c.head = (int)(rest / hu);
                rest -= c.head * hu;
                c.rt = 0;
                c.units = item_units<N>(a, q, 0);
                while (rest >= c.units) {
                    rest -= c.units;
                    c.units = item_units<N>(a, q, ++c.rt);
                }
                c.unit = (int)rest;
                sm.found = c;
                sm.found_item = ibefore + c.head * q.tiles + c.rt;
            }
        }
        // the join looks at every entry that the argument sizes allow for
        if (cta == 0 && a.by_item)
            for (int i = items + (int)threadIdx.x; i < grid; i += threads) a.cut[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
    }

    int *dead = &sm.dead;
    if (warp == kProducer) {
        // ---- copies and descriptions of the tiles
        Cursor c = sm.found;
        int item = sm.found_item;
        bool any_cut = false, from_start = false;
        for (int i = 0; i < count; ++i) {
            const int st = i % C::kStages;
            if (i >= C::kStages) wait(&sm.ring_empty[st], ((i / C::kStages) & 1) ^ 1, dead, a.err);
            if (*(volatile int *)dead) break;
            const int pos = c.unit * kTile;
            const bool first = i == 0 || c.unit == 0;
            if (first) from_start = c.unit == 0;
            const bool whole_end = c.unit + 1 == c.units;
            const bool last = whole_end || i + 1 == count;
            const bool complete = whole_end && from_start;
            // a lane looks up a block's page
            const int p = pos + lane * kKvBlock;
            int64_t pg = -1;
            int in_page = 0;
            if (lane < kTileBlocks && p < c.q.len) {
                const int pi = p / a.page;
                in_page = p - pi * a.page;
                pg = a.table[(int64_t)c.s * a.width + pi];
            }
            const bool ok = pg >= 0 && pg < a.pages;
            const uint32_t valid = __ballot_sync(0xffffffffu, ok);
            const uint32_t bar = smem_u32(&sm.ring_full[st]);
            if (lane == 0) {
                Meta &m = sm.meta[i % kMetas];
                const int left = c.units - c.unit - 1;
                m.flags = (first ? kFirst : 0) | (last ? kLast : 0) | (from_start ? kFromStart : 0) | (complete ? kComplete : 0);
                m.valid = valid;
                m.pos = pos;
                m.first = c.q.first;
                m.n = c.q.n;
                m.len = c.q.len;
                m.s = c.s;
                m.head = c.head;
                m.rt = c.rt;
                m.item = item;
                asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(smem_u32(&sm.produced)), "r"(i + 1) : "memory");
                mbar_arrive_expect_tx(bar, __popc(valid) * F::kBlock);
                if (last && from_start) {
                    const int4 e = complete ? make_int4(0, 0, 0, 0)
                                            : make_int4(c.s, c.head | (cta << 16), c.rt, (int)(1 + (left + per - 1) / per));
                    if (a.by_item) {
                        if (item < grid) a.cut[item] = e;
                    } else if (!complete) {
                        a.cut[cta] = e;
                        any_cut = true;
                    }
                }
            }
            __syncwarp();
            if (ok) {
                const int64_t blk = (pg * a.Hk + c.head) * (a.page / kKvBlock) + in_page / kKvBlock;
                bulk_g2s_plain(smem_u32(smem + st * C::kTileBytes + lane * F::kBlock), a.cache + blk * F::kBlock, F::kBlock, bar);
            }
            if (++c.unit == c.units) {
                next_item<N>(a, c);
                ++item;
            }
        }
        if (*(volatile int *)dead)  // copies in flight land before the shared memory is given up
            for (int st = 0; st < C::kStages; ++st) {
                (void)mbar_wait_bounded(smem_u32(&sm.ring_full[st]), 0);
                (void)mbar_wait_bounded(smem_u32(&sm.ring_full[st]), 1);
            }
        if (lane == 0 && count > 0 && !a.by_item && !any_cut) a.cut[cta] = make_int4(0, 0, 0, 0);
    } else if (warp == kIssuer) {
        // ---- the matrix instructions, one thread
        if (lane == 0) {
            constexpr uint32_t kIdesc1 = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
            constexpr uint32_t kIdesc2 = kIdesc1 | (1u << 16);  // B (the weights) with the query rows contiguous
            const uint32_t qa = smem_u32(smem + C::kQ), pa = smem_u32(smem + C::kP);
            int seg = 0;  // parts of items begun
            auto scores = [&](int i) {
                const int sb = i % C::kSBufs;
                wait_described(&sm.produced, i + 1, dead, a.err);
                if (sm.meta[i % kMetas].flags & kFirst) {
                    wait(&sm.q_full, seg & 1, dead, a.err);
                    ++seg;
                }
                if (i >= C::kSBufs) wait(&sm.s_empty[sb], ((i / C::kSBufs) & 1) ^ 1, dead, a.err);
                for (int h = 0; h < C::kSub; ++h) {
                    const int u = i * C::kSub + h, b = u & 1;
                    wait(&sm.k_full[b], (u >> 1) & 1, dead, a.err);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / C::kSub / 16; ++k) {
                        const int step = h * (D / C::kSub / 16) + k;
                        umma_f16_ts(tmem + C::kS + sb * N, tmem + C::kK + b * C::kKCols + 8 * k,
                                    umma_desc_none(qa + step * 32 * N, 16 * N, 128), kIdesc1, step > 0);
                    }
                    umma_commit(smem_u32(&sm.k_empty[b]));
                }
                umma_commit(smem_u32(&sm.s_full[sb]));
            };
            if (count > 0) scores(0);
            int done = 0;  // parts of items finished
            for (int i = 0; i < count; ++i) {
                const int flags = sm.meta[i % kMetas].flags;
                if (C::kSBufs > 1 && i + 1 < count) scores(i + 1);
                const int pb = i % C::kPBufs;
                if ((flags & kFirst) && done > 0) wait(&sm.o_empty, (done - 1) & 1, dead, a.err);
                wait(&sm.p_full[pb], (i / C::kPBufs) & 1, dead, a.err);
                for (int h = 0; h < C::kSub; ++h) {
                    const int u = i * C::kSub + h, b = u & 1;
                    wait(&sm.v_full[b], (u >> 1) & 1, dead, a.err);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < C::kVTok / 16; ++k)
#pragma unroll
                        for (int mh = 0; mh < C::kMh; ++mh)
                            umma_f16_ts(tmem + C::kO + mh * N, tmem + C::kV + (b * C::kMh + mh) * C::kVCols + 8 * k,
                                        umma_desc_none(pa + pb * C::kPBytes + (h * (C::kVTok / 16) + k) * 256, 128, 16 * kTile), kIdesc2,
                                        !((flags & kFirst) && h == 0 && k == 0));
                    umma_commit(smem_u32(&sm.v_empty[b]));
                }
                umma_commit(smem_u32(&sm.p_empty[pb]));
                if (flags & kLast) {
                    umma_commit(smem_u32(&sm.o_full));
                    ++done;
                }
                if (C::kSBufs == 1 && i + 1 < count) scores(i + 1);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // ---- keys: one place a thread
        const int t = warp * 32 + lane;
        const int blk = t / kKvBlock, tok = t % kKvBlock;
        const int sw = kv4_swizzle(tok) & F::kChunkMask;
        constexpr int kChunks = D / 32 / C::kSub;  // of a buffer
        for (int i = 0; i < count; ++i) {
            const int st = i % C::kStages;
            wait(&sm.ring_full[st], (i / C::kStages) & 1, dead, a.err);
            const uint8_t *kb = smem + st * C::kTileBytes + blk * F::kBlock;
            for (int h = 0; h < C::kSub; ++h) {
                const int u = i * C::kSub + h, b = u & 1;
                uint4 w[kChunks];
                uint32_t sc[kChunks];
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const int ch = h * kChunks + c;
                    w[c] = *reinterpret_cast<const uint4 *>(kb + tok * F::kCodeRow + ((ch ^ sw) << 4));
                    sc[c] = *reinterpret_cast<const uint32_t *>(kb + F::kCodes + (tok * F::kGroups + (ch >> 1)) * 4);
                }
                if (u >= 2) {
                    wait(&sm.k_empty[b], ((u >> 1) & 1) ^ 1, dead, a.err);
                    tc_fence_after();
                }
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const __half2 d = __low2half2(as_h2(sc[c])), m = __high2half2(as_h2(sc[c]));
                    const uint32_t x[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
                    uint32_t r[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t x8 = x[e] >> 8;
                        r[4 * e] = dequant_lo(x[e], d, m);
                        r[4 * e + 1] = dequant_hi(x[e], d, m);
                        r[4 * e + 2] = dequant_lo(x8, d, m);
                        r[4 * e + 3] = dequant_hi(x8, d, m);
                    }
                    tmem_st_32x32b(tmem + ((uint32_t)(warp * 32) << 16) + C::kK + b * C::kKCols + 16 * c, r);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.k_full[b]));
            }
            if (lane == 0) mbar_arrive(smem_u32(&sm.ring_empty[st]));
        }
    } else if (warp < 8) {
        // ---- values: 64 (D = 256) or 32 dimensions a warp, four nibbles of two places a register
        const int w = warp - 4;
        constexpr int kStep = D == 256 ? 16 : 32;  // places of one ldmatrix
        const bool idle = D == 64 && w >= 2;       // lanes 64 .. 127 of O^T hold nothing
        const int group = D == 256 ? w : D == 128 ? w >> 1 : 0;
        // the row this lane addresses: place and 16-byte chunk
        const int at = D == 256 ? (lane >> 4) * 8 + (lane & 7) : lane;
        const int chunk = D == 256 ? 2 * w + ((lane >> 3) & 1) : w & F::kChunkMask;
        for (int i = 0; i < count; ++i) {
            const int st = i % C::kStages;
            wait(&sm.ring_full[st], (i / C::kStages) & 1, dead, a.err);
            const Meta &m = sm.meta[i % kMetas];
            const int valid = m.valid, room = m.len - m.pos;  // places of the tile that are there
            const bool edge = valid != (1 << kTileBlocks) - 1 || room < kTile;
            const uint8_t *vb = smem + st * C::kTileBytes + F::kPart;
            for (int h = 0; h < C::kSub; ++h) {
                const int u = i * C::kSub + h, b = u & 1;
                if (u >= 2) {
                    wait(&sm.v_empty[b], ((u >> 1) & 1) ^ 1, dead, a.err);
                    tc_fence_after();
                }
                if (!idle) {
#pragma unroll
                    for (int p = 0; p < C::kVTok; p += kStep) {
                        const int p0 = h * C::kVTok + p;
                        uint32_t x[4];
                        {
                            const int pl = p0 + at, tok = pl % kKvBlock;
                            ldmatrix_x4_trans(smem_u32(vb + (pl / kKvBlock) * F::kBlock + tok * F::kCodeRow +
                                                       ((chunk ^ (kv4_swizzle(tok) & F::kChunkMask)) << 4)),
                                              x);
                        }
                        // (d, m) of this thread's two places of each group of eight
                        __half2 dd[kStep / 8], mm[kStep / 8];
#pragma unroll
                        for (int e = 0; e < kStep / 8; ++e) {
                            const int pl = p0 + 8 * e + 2 * (lane & 3), tok = pl % kKvBlock;
                            const uint8_t *sp = vb + (pl / kKvBlock) * F::kBlock + F::kCodes + (tok * F::kGroups + group) * 4;
                            uint32_t s0 = *reinterpret_cast<const uint32_t *>(sp);
                            uint32_t s1 = *reinterpret_cast<const uint32_t *>(sp + F::kGroups * 4);
                            if (edge) {  // places that are not there hold anything, NaN among it
                                const bool there = (valid >> (pl / kKvBlock)) & 1;
                                if (!there || pl >= room) s0 = 0;
                                if (!there || pl + 1 >= room) s1 = 0;
                            }
                            dd[e] = as_h2(__byte_perm(s0, s1, 0x5410));
                            mm[e] = as_h2(__byte_perm(s0, s1, 0x7632));
                        }
                        const uint32_t col = tmem + ((uint32_t)(w * 32) << 16) + C::kV + b * C::kMh * C::kVCols + p / 2;
                        uint32_t r[4][4];  // by nibble
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int g = D == 256 ? e >> 1 : e;
                            const uint32_t x8 = x[e] >> 8;
                            r[0][e] = dequant_lo(x[e], dd[g], mm[g]);
                            r[1][e] = dequant_hi(x[e], dd[g], mm[g]);
                            r[2][e] = dequant_lo(x8, dd[g], mm[g]);
                            r[3][e] = dequant_hi(x8, dd[g], mm[g]);
                        }
                        if constexpr (D == 256) {
                            // registers: (chunk 2w, 2w + 1) of places 0-7, then of places 8-15
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                tmem_st_16x128b_x2(col + ((uint32_t)(16 * (j & 1)) << 16) + (j >> 1) * C::kVCols, r[j]);
                        } else {
                            // nibbles 2q and 2q + 1 in lanes 0-7 and 8-15 of a group of 16
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                const uint32_t y[8] = {r[2 * q][0], r[2 * q + 1][0], r[2 * q][1], r[2 * q + 1][1],
                                                       r[2 * q][2], r[2 * q + 1][2], r[2 * q][3], r[2 * q + 1][3]};
                                tmem_st_16x128b_x4(col + ((uint32_t)(16 * q) << 16), y);
                            }
                        }
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.v_full[b]));
            }
            if (lane == 0) mbar_arrive(smem_u32(&sm.ring_empty[st]));
        }
    } else {
        // ---- softmax: one place a thread, kNS query rows; and q in, O out
        constexpr int NS = C::kNS;
        constexpr int NC = NS < 32 ? NS : 32;    // query rows worked at once
        const int wg = (warp - 8) >> 2;          // softmax warpgroup
        const int n0 = wg * NS;                  // its first query row
        const int w = (warp - 8) & 3;            // tensor-memory quadrant
        const int t = w * 32 + lane;
        const int bar_id = 1 + wg;
        const uint32_t quad = tmem + ((uint32_t)(w * 32) << 16);
        float sum[NS];
        int seg = 0;
        float *stage = reinterpret_cast<float *>(smem + C::kP) + wg * C::kOutRows * C::kOutStride;
        // Stages q of an item, rows of other items at zero; k index in the order that the codes are unpacked in.
        auto stage_q = [&](const Meta &m) {
            const int64_t row0 = (int64_t)m.rt * N;
            for (int x = t; x < NS * (D / 8); x += 128) {
                const int n = n0 + x % NS, g = x / NS;
                const int64_t row = row0 + n;
                const int tok = (int)(row / a.G);
                uint32_t v[4] = {0, 0, 0, 0};
                if (tok < m.n) {
                    const __half *qp = static_cast<const __half *>(a.q.p) + (int64_t)(m.first + tok) * a.q.st +
                                       (int64_t)(m.head * a.G + (int)(row - (int64_t)tok * a.G)) * a.q.sh;
                    if (a.q.vec > 1) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(qp + 8 * g);
                        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = as_u32(__halves2half2(qp[(8 * g + 2 * e) * a.q.sd], qp[(8 * g + 2 * e + 1) * a.q.sd]));
                    }
                }
                *reinterpret_cast<uint4 *>(smem + C::kQ + g * 16 * N + (n >> 3) * 128 + (n & 7) * 16) =
                    make_uint4(__byte_perm(v[0], v[2], 0x5410), __byte_perm(v[0], v[2], 0x7632), __byte_perm(v[1], v[3], 0x5410),
                               __byte_perm(v[1], v[3], 0x7632));
            }
            for (int n = t; n < NS; n += 128) {
                const int tok = (int)((row0 + n0 + n) / a.G);
                sm.lim[n0 + n] = tok < m.n ? m.len - m.n + tok : -1;
            }
            fence_proxy_async_smem();
            bar_sync(bar_id, 128);
            if (lane == 0) mbar_arrive(smem_u32(&sm.q_full));
        };
        if (count > 0) {
            wait_described(&sm.produced, 1, dead, a.err);
            stage_q(sm.meta[0]);
        }
        for (int i = 0; i < count; ++i) {
            const int sb = i % C::kSBufs, pb = i % C::kPBufs;
            wait(&sm.s_full[sb], (i / C::kSBufs) & 1, dead, a.err);
            tc_fence_after();
            const Meta m = sm.meta[i % kMetas];
            const bool first = m.flags & kFirst;
            if (first) {
#pragma unroll
                for (int n = 0; n < NS; ++n) sum[n] = 0.0f;
            }
            const int pos = m.pos + t;
            const bool there = ((m.valid >> (t / kKvBlock)) & 1) && pos < m.len;
            const bool edge = m.valid != (1 << kTileBlocks) - 1 || m.pos + kTile > m.len - m.n + (int)(((int64_t)m.rt * N) / a.G) + 1;
#pragma unroll
            for (int c = 0; c < NS; c += NC) {
                const int nc = n0 + c;
                float s[NC];
                TmemRead<NC>::run(quad + C::kS + sb * N + nc, s);
                if (c + NC == NS) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty[sb]));
                }
                if (edge) {
#pragma unroll
                    for (int n = 0; n < NC; n += 4) {
                        const int4 l = *reinterpret_cast<const int4 *>(&sm.lim[nc + n]);
                        if (!there || pos > l.x) s[n] = -INFINITY;
                        if (!there || pos > l.y) s[n + 1] = -INFINITY;
                        if (!there || pos > l.z) s[n + 2] = -INFINITY;
                        if (!there || pos > l.w) s[n + 3] = -INFINITY;
                    }
                }
                bool move = first;
                if (!first) {
                    float over = -INFINITY;
#pragma unroll
                    for (int n = 0; n < NC; n += 4) {
                        const float4 b = *reinterpret_cast<const float4 *>(&sm.base[nc + n]);
                        over = fmaxf(over, fmaf(s[n], a.scale_log2, -b.x));
                        over = fmaxf(over, fmaf(s[n + 1], a.scale_log2, -b.y));
                        over = fmaxf(over, fmaf(s[n + 2], a.scale_log2, -b.z));
                        over = fmaxf(over, fmaf(s[n + 3], a.scale_log2, -b.w));
                    }
                    move = over > kMoveMax + kWeightShift;
                }
                if (bar_or(bar_id, 128, move)) {
                    // the rows' maxima over the 128 places; O and the sums follow the reference
#pragma unroll
                    for (int n = 0; n < NC; ++n) {
                        const int top = __reduce_max_sync(0xffffffffu, float_order(s[n] * a.scale_log2));
                        if (lane == 0) sm.wred[wg * 4 + w][n] = order_float(top);
                    }
                    bar_sync(bar_id, 128);
                    if (t < NC) {
                        const float old = first ? -INFINITY : sm.ref[nc + t];
                        float top = old;
#pragma unroll
                        for (int x = 0; x < 4; ++x) top = fmaxf(top, sm.wred[wg * 4 + x][t]);
                        if (sm.lim[nc + t] < 0) top = fmaxf(top, 0.0f);  // a row that sees nothing stays out of this
                        sm.ref[nc + t] = top;
                        // a row that has seen nothing yet moves at its first score
                        sm.base[nc + t] = top == -INFINITY ? -1e30f : top - kWeightShift;
                        sm.factor[nc + t] = top == -INFINITY ? 1.0f : ex2(old - top);
                    }
                    bar_sync(bar_id, 128);
                    if (!first) {
#pragma unroll
                        for (int n = 0; n < NC; ++n) sum[c + n] *= sm.factor[nc + n];
                        // every product before this tile is in O
                        wait(&sm.p_empty[(i - 1) % C::kPBufs], ((i - 1) / C::kPBufs) & 1, dead, a.err);
                        tc_fence_after();
#pragma unroll 1
                        for (int x = 0; x < C::kMh * NC; x += 16) {
                            const uint32_t at = quad + C::kO + (x / NC) * N + nc + x % NC;
                            float o[16];
                            uint32_t r[16];
                            TmemRead<16>::run(at, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[e] * sm.factor[nc + x % NC + e]);
                            tmem_st_32x32b(at, r);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                }
                if (c == 0 && i >= C::kPBufs) wait(&sm.p_empty[pb], ((i / C::kPBufs) & 1) ^ 1, dead, a.err);
                uint8_t *pp = smem + C::kP + pb * C::kPBytes + (nc >> 3) * (16 * kTile) + (t >> 3) * 128 + (t & 7) * 16;
#pragma unroll
                for (int n = 0; n < NC; n += 8) {
                    const float4 b0 = *reinterpret_cast<const float4 *>(&sm.base[nc + n]);
                    const float4 b1 = *reinterpret_cast<const float4 *>(&sm.base[nc + n + 4]);
                    const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
                    float e[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        e[x] = ex2(fmaf(s[n + x], a.scale_log2, -b[x]));
                        sum[c + n + x] += e[x];
                    }
                    *reinterpret_cast<uint4 *>(pp + (n >> 3) * (16 * kTile)) =
                        make_uint4(pack_h2(e[0], e[1]), pack_h2(e[2], e[3]), pack_h2(e[4], e[5]), pack_h2(e[6], e[7]));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[pb]));
            if (m.flags & kLast) {
                // q of the next item while the last products run (all first products of this one are done:
                // their scores have been read)
                if (C::kSoft > 1) bar_sync(3, 256);  // both warpgroups have
                if (i + 1 < count) {
                    wait_described(&sm.produced, i + 2, dead, a.err);
                    stage_q(sm.meta[(i + 1) % kMetas]);
                }
                // ---- the sums over the places
#pragma unroll
                for (int c = 0; c < NS; c += 16) {
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = sum[c + e];
                    const float r = reduce_scatter<16>(v, lane);
                    if (lane < 16) sm.wred[wg * 4 + w][c + lane] = r;
                }
                bar_sync(bar_id, 128);
                const int slot = 2 * cta + ((m.flags & kFromStart) ? 1 : 0);
                const bool complete = m.flags & kComplete;
                for (int n = t; n < NS; n += 128) {
                    const float den = (sm.wred[wg * 4][n] + sm.wred[wg * 4 + 1][n]) + (sm.wred[wg * 4 + 2][n] + sm.wred[wg * 4 + 3][n]);
                    sm.inv[n0 + n] = complete ? (den > 0.0f ? 1.0f / den : 0.0f) : 1.0f;
                    if (!complete) a.stat[(int64_t)slot * N + n0 + n] = make_float2(sm.ref[n0 + n], den);
                }
                wait(&sm.o_full, seg & 1, dead, a.err);
                ++seg;
                tc_fence_after();
                bar_sync(bar_id, 128);
                // ---- O, eight rows at a time through shared memory (the weights' buffers are free now)
                const int64_t row0 = (int64_t)m.rt * N + n0;
                for (int c = 0; c < NS; c += 8) {
                    if ((row0 + c) / a.G >= m.n) break;  // no more rows
#pragma unroll
                    for (int mh = 0; mh < C::kMh; ++mh) {
                        float o[8];
                        TmemRead<8>::run(quad + C::kO + mh * N + n0 + c, o);
                        const int dim = o_dim<D>(t, mh);
                        if (D > 64 || t < 64) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) stage[e * C::kOutStride + dim] = o[e] * sm.inv[n0 + c + e];
                        }
                    }
                    bar_sync(bar_id, 128);
                    for (int x = t; x < 8 * (D / 8); x += 128) {
                        const int e = x / (D / 8), g = x % (D / 8);
                        const int64_t row = row0 + c + e;
                        const int tok = (int)(row / a.G);
                        const float4 v0 = *reinterpret_cast<const float4 *>(stage + e * C::kOutStride + 8 * g);
                        const float4 v1 = *reinterpret_cast<const float4 *>(stage + e * C::kOutStride + 8 * g + 4);
                        if (tok < m.n) {
                            if (complete) {
                                const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                                store_dims<8>(a.out, m.first + tok, m.head * a.G + (int)(row - (int64_t)tok * a.G), 8 * g, v);
                            } else {
                                float *dst = a.part + ((int64_t)slot * N + n0 + c + e) * D + 8 * g;
                                *reinterpret_cast<float4 *>(dst) = v0;
                                *reinterpret_cast<float4 *>(dst + 4) = v1;
                            }
                        }
                    }
                    bar_sync(bar_id, 128);
                }
                tc_fence_before();
                if (C::kSoft > 1) bar_sync(3, 256);  // the other warpgroup may still read the staging area
                if (lane == 0) mbar_arrive(smem_u32(&sm.o_empty));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kIssuer) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The items that were cut between CTAs: out = sum_i 2^(ref_i - ref) O_i / sum_i 2^(ref_i - ref) sum_i,
// in CTA order.  One block takes RB rows of one item; D / 4 threads share a row's dimensions and the
// rest of its threads the parts.
template <int D, int N, int RB> __global__ void __launch_bounds__(256) attn_kv4_join_kernel(const AttnArgs a)
{
    constexpr int TX = D / 4;            // threads across a row
    constexpr int TY = 256 / (TX * RB);  // threads that share its parts
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
    const Seq q = load_seq<N>(a, c.x);
    const int64_t row = (int64_t)c.z * N + r;
    const int tok = (int)(row / a.G);
    float top = -INFINITY;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    if (tok < q.n) {
        for (int i = 0; i < c.w; ++i) top = fmaxf(top, a.stat[(int64_t)(i ? 2 * (cta + i) : 2 * cta + 1) * N + r].x);
#pragma unroll 4
        for (int i = y; i < c.w; i += TY) {
            const int64_t slot = i ? 2 * (cta + i) : 2 * cta + 1;
            const float2 st = a.stat[slot * N + r];
            const float f = st.x == -INFINITY ? 0.0f : ex2(st.x - top);
            const float4 u = *reinterpret_cast<const float4 *>(a.part + (slot * N + r) * D + 4 * x);
            l = fmaf(st.y, f, l);
            v.x = fmaf(u.x, f, v.x);
            v.y = fmaf(u.y, f, v.y);
            v.z = fmaf(u.z, f, v.z);
            v.w = fmaf(u.w, f, v.w);
        }
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
    store_dims<4>(a.out, q.first + tok, head * a.G + (int)(row - (int64_t)tok * a.G), 4 * x, w);
}

// Query rows of an item: the fewest columns that hold what a sequence has (by the caller's max_q), so that
// few rows leave tensor time and shared memory to the copies; many rows share each unpacked tile.
int rows_of(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

struct WsLayout {
    size_t part, stat, cut, bytes;
};

WsLayout ws_layout(int D, int N, int grid)
{
    WsLayout w;
    w.part = 256;  // the error word first
    w.stat = w.part + (size_t)2 * grid * N * D * sizeof(float);
    w.cut = w.stat + (size_t)2 * grid * N * sizeof(float2);
    w.bytes = w.cut + (size_t)grid * sizeof(int4);
    return w;
}

template <int D, int N> int launch_attn(AttnArgs &a, int grid, int nseq, void *stream)
{
    static std::atomic<uint64_t> raised{0};  // devices whose shared-memory limit is raised
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return QG_ERR_CUDA;
    if (dev >= 64 || !(raised.load() >> dev & 1)) {
        if (cudaFuncSetAttribute(attn_kv4_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, N>::kBytes) != cudaSuccess)
            return QG_ERR_CUDA;
        if (dev < 64) raised.fetch_or(uint64_t(1) << dev);
    }
    // items at most: a row tile may be short in every sequence
    const int64_t items = (int64_t)a.Hk * (nseq + a.T * a.G / N);
    a.by_item = items <= grid;
    const int rc = launch_pdl(attn_kv4_kernel<D, N>, dim3(grid), dim3(Cfg<D, N>::kWarps * 32), Cfg<D, N>::kBytes, stream, a);
    if (rc != QG_OK) return rc;
    // no item is cut when none has more than one tile
    if ((int64_t)a.width * a.page <= kTile) return QG_OK;
    if (a.by_item)
        return launch_pdl(attn_kv4_join_kernel<D, N, 1>, dim3((unsigned)items, N), dim3(256), 0, stream, a);
    return launch_pdl(attn_kv4_join_kernel<D, N, 4>, dim3(grid, N / 4), dim3(256), 0, stream, a);
}

template <int D> int launch_rows(AttnArgs &a, int N, int grid, int nseq, void *stream)
{
    switch (N) {
    case 16: return launch_attn<D, 16>(a, grid, nseq, stream);
    case 32: return launch_attn<D, 32>(a, grid, nseq, stream);
    case 64: return launch_attn<D, 64>(a, grid, nseq, stream);
    default: return launch_attn<D, 128>(a, grid, nseq, stream);
    }
}

bool good_dim(int D) { return D == 64 || D == 128 || D == 256; }

}  // namespace

extern "C" {

size_t qg_attn_kv4_workspace(int Hq, int Hk, int D, int max_q)
{
    int sms = 0;
    if (!good_dim(D) || Hk < 1 || Hq < Hk || Hq % Hk || Hq > QG_MAX_HEADS || max_q < 0 || current_sms(&sms) != QG_OK) return 0;
    return ws_layout(D, rows_of((int64_t)max_q * (Hq / Hk)), sms).bytes;
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
    a.G = Hq / Hk;
    const int N = rows_of((int64_t)max_q * a.G);
    const WsLayout w = ws_layout(D, N, sms);
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
    switch (D) {
    case 64: return launch_rows<64>(a, N, sms, nseq, stream);
    case 128: return launch_rows<128>(a, N, sms, nseq, stream);
    default: return launch_rows<256>(a, N, sms, nseq, stream);
    }
}

}  // extern "C"
