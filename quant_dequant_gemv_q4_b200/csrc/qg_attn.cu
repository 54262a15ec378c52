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
// Roles of a CTA's warps (one CTA an SM): a producer (bulk copies of 18 D bytes for each 16 places, those of
// neighbours in one, several tiles ahead), one or two warpgroups that unpack keys and as many for values, one for the
// softmax of each 32 query rows, and two warps that issue the matrix instructions, one for each product.  Key and
// value operands have buffers of a part of a tile (kSub), scores and weights of a tile, all handed over by mbarriers.
//
// What bounds it, at decode (N = 16), D = 256: issuing instructions.  A tile takes about 7450 warp instructions
// (unpacking two thirds of them) and 2600 cycles, 68% of the SM's issue slots, where its bytes would arrive in
// about 1660; a part of an item costs about 6000 cycles more (q in, the first reference, O out), which ragged
// batches and pages of few tiles feel.  200001 places of 4 heads: 69 us, 3.3 TB/s; 16 sequences of up to 16000:
// 53 us.  At D = 128 a tile has half the unpacking and takes about as long: 64 sequences of up to 6000 use 49% of the
// slots, their warps wait for what passes between the roles (101-105 us).  Two softmax warpgroups on alternate tiles, each with an O of its own,
// took 77, 58 and 100 us, two producers 70, 56 and 107: the instruction caches hold these loops only just, and
// what shortens one of them lengthens the others.  At N = 128 the softmax bounds it, a thread's 32 scores at a time:
// 1000 tokens on 7000, 425 us, 750 TFLOP/s, with 72 registers a thread and spills in the softmax.
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
constexpr int kHoleBar = 10;                    // named barriers 10, 11: the value warpgroups
constexpr int kMetas = 16;                      // tiles whose description is kept (more than any role lags)
constexpr int64_t kNoRow = INT64_MIN;           // no row of q or out (offsets of rows are negative where strides are)

// flags of a tile
constexpr int kFirst = 1;      // first of this CTA's part of its item
constexpr int kLast = 2;       // last of it
constexpr int kFromStart = 4;  // the part holds the item's first tile
constexpr int kComplete = 8;   // the part is the whole item
constexpr int kEdge = 16;      // some row does not see some place of the tile
constexpr int kHole = 32;      // some place of the tile is not there
constexpr int kNext = 64;      // (of a first tile) another part follows: `next`

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

// What the roles need to know of a tile, and of the part of an item after its own.
struct Item {
    int first, n, len, head, rt;
};
struct Meta {
    int flags, valid, pos, room;  // valid: blocks that are there; room: places down to the sequence's end
    Item item, next;
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
    static constexpr int kWork = N <= 32 ? 2 : 1;                // warpgroups for the keys, and for the values
    // operand buffers hold 1 / kSub of a tile; with two warpgroups there is one more than they fill at once
    static constexpr int kSub = D == 256 ? (N == 128 ? 4 : 2) : (N <= 32 ? 1 : 2);
    static constexpr int kBufs = N <= 32 ? 3 : 2;
    static constexpr int kMh = D >= 128 ? D / 128 : 1;           // M = 128 halves of O^T
    static constexpr int kKCols = D / 2 / kSub;                  // columns of a key buffer: D / kSub dimensions
    static constexpr int kVTok = kTile / kSub;                   // places of a value buffer
    static constexpr int kVCols = kVTok / 2;                     // columns of it in each half
    static constexpr int kSBufs = (D == 256 && N == 128) ? 1 : 2;
    static constexpr int kPBufs = (D == 256 && N == 128) ? 1 : 2;
    static constexpr int kSoft = N > 32 ? N / 32 : 1;            // softmax warpgroups
    static constexpr int kNS = N / kSoft;                        // query rows of each
    static constexpr int kWarps = 4 * (2 * kWork + kSoft) + 3;
    // tensor memory columns
    static constexpr int kK = 0, kV = kK + kBufs * kKCols, kS = kV + kBufs * kVCols * kMh, kO = kS + kSBufs * N;
    static constexpr int kCols = kO + kMh * N;
    static_assert(kCols <= 512, "tensor memory");
    // shared memory
    static constexpr int kTileBytes = kTileBlocks * F::kBlock;
    static constexpr int kStages = D == 256 ? (N >= 64 ? 3 : 4) : D == 128 ? (N == 128 ? 4 : 6) : 8;
    static constexpr int kQBufs = (D == 256 && N == 128) ? 1 : 2;
    static constexpr int kQ = kStages * kTileBytes;
    static constexpr int kQBytes = N * D * 2;
    static constexpr int kP = kQ + kQBufs * kQBytes;
    static constexpr int kPBytes = N * kTile * 2;
    static constexpr int kOutStride = D + 4;
    static constexpr int kOutRows = N <= 32 ? 16 : 8;            // rows of O that pass through shared memory at once
    static constexpr int kOutBytes = kSoft * kOutRows * kOutStride * 4;
    static constexpr int kPAll = kPBufs * kPBytes > kOutBytes ? kPBufs * kPBytes : kOutBytes;
    static constexpr int kBytes = kP + kPAll;
};

// Whether a call on this device has given up since qg_attn_kv4_device_error was last asked.
__device__ int g_gave_up;

// Giving up.  A wait that lasts longer than kWaitNs sets the call's error word and `gave_up`.  The producer, the only
// role whose waits end on that alone, then stops and sets `quiet` (as it does at its end in any case); the other roles
// wait on until `dead`, which is set once both are, and go through their remaining tiles without waiting.  The
// descriptions of the tiles no longer change by then, so the warps of a role take the same way through them and meet
// at its named barriers, which have no limit of their own.  What is computed is void; every address stays that of some
// tile that was described (a slot without one holds zeros: no rows).
struct Stop {
    int dead, gave_up, quiet;
};

template <int N> struct Small {
    uint64_t ring_full[8], ring_empty[8];
    uint64_t k_full[3], k_empty[3], v_full[3], v_empty[3], s_full[2], s_empty[2], p_full[2], p_empty[2], q_full[2];
    uint64_t o_full, o_empty;
    Meta meta[kMetas];
    Cursor found;
    int found_item;
    int64_t scan[2][32];
    int iscan[32];
    uint32_t tmem;
    uint64_t drained[2];  // the issuers' last products, after a wait that ran out
    Stop stop;
    int produced;         // tiles described so far
    alignas(16) float base[N];    // reference - kWeightShift
    alignas(16) int lim[2][N];    // last place that a row sees (of the parts of items in turn)
    int64_t orow[2][N];           // where a row of out starts, or kNoRow
    int64_t qrow[N];              // ... and of q
    float ref[N];
    float wred[4][N];             // by warp of the warpgroup
    float inv[N];
    float factor[N];
};

// Waits for a phase; false where it gives up.
template <bool PRODUCER = false> __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile Stop *stop, int *err)
{
    const uint32_t b = smem_u32(bar);
    if (mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        // (a try suspends the warp for a while only: keep what is issued between tries short)
#pragma unroll 1
        for (int i = 0; i < 8; ++i)
            if (mbar_try_wait(b, parity)) return true;
        if (PRODUCER ? stop->gave_up : stop->dead) return false;
        if (global_timer_ns() - t0 > kWaitNs) {
            stop->gave_up = 1;
            *err = 1;
            if (stop->quiet) stop->dead = 1;
        }
    }
}

// Waits until `need` tiles are described.
__device__ __forceinline__ void wait_described(int *produced, int need, volatile Stop *stop, int *err)
{
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        int v;
        asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(produced)) : "memory");
        if (v >= need || stop->dead) return;
        if (global_timer_ns() - t0 > kWaitNs) {
            stop->gave_up = 1;
            *err = 1;
            if (stop->quiet) stop->dead = 1;
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
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(16) Small<N> sm;
    static_assert(C::kBytes + sizeof(Small<N>) <= 227 * 1024, "shared memory of a block");
    static_assert(offsetof(Small<N>, base) % 16 == 0 && offsetof(Small<N>, lim) % 16 == 0, "read four at a time");
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (warp-uniform)
    const int cta = blockIdx.x, grid = gridDim.x;
    constexpr int kProducer = C::kWarps - 3, kIssuer = C::kWarps - 2;  // (and the second products' issuer)

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&sm.ring_full[i]), 1);
            mbar_init(smem_u32(&sm.ring_empty[i]), 8 * C::kWork);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(smem_u32(&sm.k_full[i]), 4);
            mbar_init(smem_u32(&sm.k_empty[i]), 1);
            mbar_init(smem_u32(&sm.v_full[i]), 4);
            mbar_init(smem_u32(&sm.v_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sm.s_full[i]), 1);
            mbar_init(smem_u32(&sm.s_empty[i]), 4 * C::kSoft);
            mbar_init(smem_u32(&sm.p_full[i]), 4 * C::kSoft);
            mbar_init(smem_u32(&sm.p_empty[i]), 1);
            mbar_init(smem_u32(&sm.q_full[i]), 4 * C::kSoft);
        }
        mbar_init(smem_u32(&sm.o_full), 1);
        mbar_init(smem_u32(&sm.o_empty), 4 * C::kSoft);
        mbar_init(smem_u32(&sm.drained[0]), 1);
        mbar_init(smem_u32(&sm.drained[1]), 1);
        mbar_init_fence();
        sm.stop = {0, 0, 0};
        sm.produced = 0;
    }
    for (int i = threadIdx.x; i < (int)(sizeof(sm.meta) / 4); i += C::kWarps * 32) reinterpret_cast<int *>(sm.meta)[i] = 0;
    // Tensor memory is taken only when the kernels before are done, and the kernels after may start only when
    // it is taken: neither then holds it while it waits for the other.
    pdl_wait();
    if (warp == kIssuer) tmem_alloc(smem_u32(&sm.tmem), 512);
    if (cta == 0 && threadIdx.x == 0) *a.err = 0;

    // ---- the run of tiles of this CTA: the tiles of all sequences, then the sequence its first one is in
    const int threads = C::kWarps * 32;
    int64_t total = 0;
    Seq mine = {};       // this thread's sequence of the last round, and the tiles of one of its heads
    int64_t mine_units = 0;
    for (int s = threadIdx.x; s < a.nseq; s += threads) {
        mine = load_seq<N>(a, s);
        mine_units = head_units<N>(a, mine);
        total += mine_units * a.Hk;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) sm.scan[0][warp] = total;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
    total = 0;
    for (int w = 0; w < C::kWarps; ++w) total += sm.scan[0][w];
    const int64_t per = (total + grid - 1) / grid;
    const int64_t begin = per * cta < total ? per * cta : total;
    const int64_t end = begin + per < total ? begin + per : total;
    const int count = __shfl_sync(0xffffffffu, (int)(end - begin), 0);
    if (count == 0) {
        if (threadIdx.x == 0 && !a.by_item) a.cut[cta] = make_int4(0, 0, 0, 0);
        if (cta == 0 && a.by_item)
            for (int i = threadIdx.x; i < grid; i += threads) a.cut[i] = make_int4(0, 0, 0, 0);
    } else {
        int64_t base = 0;
        int items = 0;
        for (int s0 = 0; s0 < a.nseq; s0 += threads) {
            const int s = s0 + threadIdx.x;
            if (a.nseq > threads) {  // (else the first pass has left it)
                mine = {};
                mine_units = 0;
                if (s < a.nseq) {
                    mine = load_seq<N>(a, s);
                    mine_units = head_units<N>(a, mine);
                }
                if (s0 > 0) __syncthreads();  // the sums of the round before have been read
            }
            const int64_t u = mine_units * a.Hk;
            const int it = mine.tiles * a.Hk;
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
            if (lane == 31) {
                sm.scan[1][warp] = up;
                sm.iscan[warp] = itp;
            }
            __syncthreads();
            int64_t before = base + up - u;
            int ibefore = items + itp - it;
            for (int w = 0; w < C::kWarps; ++w) {
                if (w < warp) {
                    before += sm.scan[1][w];
                    ibefore += sm.iscan[w];
                }
                base += sm.scan[1][w];
                items += sm.iscan[w];
            }
            if (begin >= before && begin < before + u) {
                Cursor c;
                c.q = mine;
                c.s = s;
                int64_t rest = begin - before;
                c.head = (int)(rest / mine_units);
                rest -= c.head * mine_units;
                c.rt = 0;
                c.units = item_units<N>(a, mine, 0);
                while (rest >= c.units) {
                    rest -= c.units;
                    c.units = item_units<N>(a, mine, ++c.rt);
                }
                c.unit = (int)rest;
                sm.found = c;
                sm.found_item = ibefore + c.head * mine.tiles + c.rt;
            }
        }
        // the join looks at every entry that the argument sizes allow for
        if (cta == 0 && a.by_item)
            for (int i = items + (int)threadIdx.x; i < grid; i += threads) a.cut[i] = make_int4(0, 0, 0, 0);
        __syncthreads();
    }

    volatile Stop *const stop = &sm.stop;
    if (warp == kProducer) {
        // ---- copies and descriptions of the tiles
        Cursor c = sm.found;
        int item = sm.found_item;
        bool any_cut = false, from_start = false;
        const int page_blocks = a.page / kKvBlock;
        // page of block 8 unit + lane of the cursor's item (up to 31 blocks past the sequence's last: their places may
        // pass 2^31), -1 past its end
        auto look_up = [&](const Cursor &k, int unit) -> int {
            const int blk = unit * kTileBlocks + lane;
            return (int64_t)blk * kKvBlock < k.q.len ? a.table[(int64_t)k.s * a.width + blk / page_blocks] : -1;
        };
        int ahead = 0, pages = -1, pages_next = -1;
        for (int i = 0; i < count; ++i) {
            const int st = i % C::kStages;
            const bool free = i < C::kStages || wait<true>(&sm.ring_empty[st], ((i / C::kStages) & 1) ^ 1, stop, a.err);
            if (!__all_sync(0xffffffffu, free)) break;
            const int pos = c.unit * kTile;
            const bool first = i == 0 || c.unit == 0;
            if (first) from_start = c.unit == 0;
            const bool whole_end = c.unit + 1 == c.units;
            const bool last = whole_end || i + 1 == count;
            const bool complete = whole_end && from_start;
            // the pages of the tile's blocks: looked up for four tiles of an item at a time, the next four while
            // these are copied (a look-up takes as long as half a tile)
            if (first || c.unit == ahead) {
                if (first) ahead = c.unit;
                pages = first ? look_up(c, ahead) : pages_next;
                ahead += 4;
                pages_next = ahead < c.units ? look_up(c, ahead) : -1;
            }
            const int64_t pg = __shfl_sync(0xffffffffu, pages, (c.unit - (ahead - 4)) * kTileBlocks + (lane & 7));
            const bool ok = lane < kTileBlocks && pg >= 0 && pg < a.pages;
            const uint32_t valid = __ballot_sync(0xffffffffu, ok);
            const uint32_t bar = smem_u32(&sm.ring_full[st]);
            // one copy for each run of neighbouring blocks of a page
            const int in_page = (int)((uint32_t)(c.unit * kTileBlocks + lane) % (uint32_t)page_blocks);
            const int64_t blk = (pg * a.Hk + c.head) * page_blocks + in_page;
            const uint32_t heads = __ballot_sync(0xffffffffu, ok && (lane == 0 || in_page == 0));
            if ((heads >> lane) & 1) {
                // down to the next run, or the last block that is there (a run has no gaps: one page)
                const uint32_t later = heads & ~((2u << lane) - 1);
                const uint32_t rest = later ? (1u << (__ffs(later) - 1)) - 1 : 0xffffffffu;
                const int run = __popc(valid & rest & ~((1u << lane) - 1));
                bulk_g2s_plain(smem_u32(smem + st * C::kTileBytes + lane * F::kBlock), a.cache + blk * F::kBlock, run * F::kBlock, bar);
            }
            __syncwarp();
            if (lane == 0) {
                Meta &m = sm.meta[i % kMetas];
                const int left = c.units - c.unit - 1;
                const int tok0 = (int)((uint32_t)(c.rt * N) / (uint32_t)a.G);  // the row tile's first query token
                int flags = (first ? kFirst : 0) | (last ? kLast : 0) | (from_start ? kFromStart : 0) | (complete ? kComplete : 0);
                if (valid != (1 << kTileBlocks) - 1 || pos + kTile > c.q.len) flags |= kHole | kEdge;
                if (pos + kTile > c.q.len - c.q.n + tok0 + 1) flags |= kEdge;
                if (first) {
                    m.item = {c.q.first, c.q.n, c.q.len, c.head, c.rt};
                    if (i + left + 1 < count) {
                        Cursor n = c;
                        next_item<N>(a, n);
                        m.next = {n.q.first, n.q.n, n.q.len, n.head, n.rt};
                        flags |= kNext;
                    }
                }
                m.flags = flags;
                m.valid = valid;
                m.pos = pos;
                m.room = c.q.len - pos;
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
            if (++c.unit == c.units) {
                next_item<N>(a, c);
                ++item;
            }
        }
        if (lane == 0) {
            __threadfence_block();
            stop->quiet = 1;
            if (count > 0 && !a.by_item && !any_cut) a.cut[cta] = make_int4(0, 0, 0, 0);
        }
    } else if (warp >= kIssuer) {
        // ---- the matrix instructions: a warp for the scores and one for the weighted sums, so that neither waits
        // for the other's operands; a warp stays together, an elected lane issues
        constexpr uint32_t kIdesc1 = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
        constexpr uint32_t kIdesc2 = kIdesc1 | (1u << 16);  // B (the weights) with the query rows contiguous
        int seg = 0;  // parts of items begun
        if (warp == kIssuer) {
            const uint32_t qa = smem_u32(smem + C::kQ);
            uint32_t qb = qa;
            for (int i = 0; i < count; ++i) {
                const int sb = i % C::kSBufs;
                wait_described(&sm.produced, i + 1, stop, a.err);
                if (__shfl_sync(0xffffffffu, sm.meta[i % kMetas].flags, 0) & kFirst) {
                    wait(&sm.q_full[seg % C::kQBufs], (seg / C::kQBufs) & 1, stop, a.err);
                    qb = qa + (seg % C::kQBufs) * C::kQBytes;
                    ++seg;
                }
                if (i >= C::kSBufs) wait(&sm.s_empty[sb], ((i / C::kSBufs) & 1) ^ 1, stop, a.err);
                for (int h = 0; h < C::kSub; ++h) {
                    const int u = i * C::kSub + h, b = u % C::kBufs;
                    wait(&sm.k_full[b], (u / C::kBufs) & 1, stop, a.err);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < D / C::kSub / 16; ++k) {
                        const int step = h * (D / C::kSub / 16) + k;
                        umma_f16_ts_elect(tmem + C::kS + sb * N, tmem + C::kK + b * C::kKCols + 8 * k,
                                          umma_desc_none(qb + step * 32 * N, 16 * N, 128), kIdesc1, step > 0);
                    }
                    umma_commit_elect(smem_u32(&sm.k_empty[b]));
                }
                umma_commit_elect(smem_u32(&sm.s_full[sb]));
            }
        } else {
            const uint32_t pa = smem_u32(smem + C::kP);
            for (int i = 0; i < count; ++i) {
                const int pb = i % C::kPBufs;
                wait_described(&sm.produced, i + 1, stop, a.err);
                const int flags = __shfl_sync(0xffffffffu, sm.meta[i % kMetas].flags, 0);
                if (flags & kFirst) {
                    if (seg > 0) wait(&sm.o_empty, (seg - 1) & 1, stop, a.err);
                    ++seg;
                }
                wait(&sm.p_full[pb], (i / C::kPBufs) & 1, stop, a.err);
                for (int h = 0; h < C::kSub; ++h) {
                    const int u = i * C::kSub + h, b = u % C::kBufs;
                    wait(&sm.v_full[b], (u / C::kBufs) & 1, stop, a.err);
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < C::kVTok / 16; ++k)
#pragma unroll
                        for (int mh = 0; mh < C::kMh; ++mh)
                            umma_f16_ts_elect(tmem + C::kO + mh * N, tmem + C::kV + (b * C::kMh + mh) * C::kVCols + 8 * k,
                                              umma_desc_none(pa + pb * C::kPBytes + (h * (C::kVTok / 16) + k) * 256, 128, 16 * kTile), kIdesc2,
                                              !((flags & kFirst) && h == 0 && k == 0));
                    umma_commit_elect(smem_u32(&sm.v_empty[b]));
                }
                umma_commit_elect(smem_u32(&sm.p_empty[pb]));
                if (flags & kLast) umma_commit_elect(smem_u32(&sm.o_full));
            }
        }
    } else if (warp < 4 * C::kWork) {
        // ---- keys: one place a thread; of two warpgroups, each takes every other buffer
        const int wk = C::kWork > 1 ? warp >> 2 : 0;
        const int t = (warp & 3) * 32 + lane;
        const int blk = t / kKvBlock, tok = t % kKvBlock;
        // offsets in a tile of this place's first chunk and scales: a chunk's number is xored in, since rows
        // of chunks are aligned to their size
        const int code_at = blk * F::kBlock + tok * F::kCodeRow + ((kv4_swizzle(tok) & F::kChunkMask) << 4);
        const int scale_at = blk * F::kBlock + F::kCodes + tok * F::kGroups * 4;
        static_assert(F::kBlock % F::kCodeRow == 0 && C::kTileBytes % F::kCodeRow == 0, "rows of chunks are aligned");
        constexpr int kChunks = D / 32 / C::kSub;  // of a buffer
        constexpr int kPer = N > 32 && kChunks > 1 ? 2 : 1;
        for (int i = 0; i < count; ++i) {
            const int st = i % C::kStages;
            wait(&sm.ring_full[st], (i / C::kStages) & 1, stop, a.err);
            const uint8_t *kb = smem + st * C::kTileBytes;
#pragma unroll 1
            for (int h = (wk + i * C::kSub) % C::kWork; h < C::kSub; h += C::kWork) {
                const int u = i * C::kSub + h, b = u % C::kBufs;
                if (u >= C::kBufs) {
                    wait(&sm.k_empty[b], ((u / C::kBufs) & 1) ^ 1, stop, a.err);
                    tc_fence_after();
                }
                const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + C::kK + b * C::kKCols;
                // Short loops: with few query rows four warps of a scheduler unpack, in two loops that ought to
                // stay in its instruction cache (unrolled twice, 200001 places took 72 us instead of 69).
#pragma unroll 1
                for (int c = 0; c < kChunks; c += kPer) {
                    const int ch = h * kChunks + c;
                    const uint32_t sc = *reinterpret_cast<const uint32_t *>(kb + scale_at + (ch >> 1) * 4);
                    uint32_t x[4 * kPer], r[16 * kPer];
#pragma unroll
                    for (int y = 0; y < kPer; ++y) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(kb + (code_at ^ ((ch + y) << 4)));
                        x[4 * y] = v.x, x[4 * y + 1] = v.y, x[4 * y + 2] = v.z, x[4 * y + 3] = v.w;
                    }
                    const __half2 d = __low2half2(as_h2(sc)), m = __high2half2(as_h2(sc));
#pragma unroll
                    for (int e = 0; e < 4 * kPer; ++e) {
                        const uint32_t x8 = x[e] >> 8;
                        r[4 * e] = dequant_lo(x[e], d, m);
                        r[4 * e + 1] = dequant_hi(x[e], d, m);
                        r[4 * e + 2] = dequant_lo(x8, d, m);
                        r[4 * e + 3] = dequant_hi(x8, d, m);
                    }
                    TmemWrite32<16 * kPer>::run(to + 16 * c, r);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.k_full[b]));
            }
            if (lane == 0) mbar_arrive(smem_u32(&sm.ring_empty[st]));
        }
    } else if (warp < 8 * C::kWork) {
        // ---- values: 64 (D = 256) or 32 dimensions a warp, four nibbles of two places a register; of two
        // warpgroups, each takes every other buffer
        const int w = warp & 3;
        const int wv = C::kWork > 1 ? (warp >> 2) - 2 : 0;
        constexpr int kStep = D == 256 ? 16 : 32;  // places of one ldmatrix
        constexpr int kBatch = N > 32 && C::kVTok >= 32 ? 32 : kStep;  // places written at once (a short loop, as for the keys)
        const bool idle = D == 64 && w >= 2;       // lanes 64 .. 127 of O^T hold nothing
        const int group = D == 256 ? w : D == 128 ? w >> 1 : 0;
        // where this lane reads within a step: the row it addresses (a 16-byte chunk of a place), and the
        // (d, m) of its two places of each eight
        const int at = D == 256 ? (lane >> 4) * 8 + (lane & 7) : lane;
        const int chunk = D == 256 ? 2 * w + ((lane >> 3) & 1) : w & F::kChunkMask;
        const int tok = at % kKvBlock;
        const int code_at = (at / kKvBlock) * F::kBlock + tok * F::kCodeRow + ((chunk ^ (kv4_swizzle(tok) & F::kChunkMask)) << 4);
        const int scale_at = F::kCodes + (2 * (lane & 3) * F::kGroups + group) * 4;
        const uint32_t lanes = tmem + ((uint32_t)(w * 32) << 16) + C::kV;
        for (int i = 0; i < count; ++i) {
            const int st = i % C::kStages;
            wait(&sm.ring_full[st], (i / C::kStages) & 1, stop, a.err);
            const Meta &m = sm.meta[i % kMetas];
            if (m.flags & kHole) {
                // places that are not there hold anything, NaN among it: this warpgroup zeroes the scales of its own
                // places, a thread a place
                const int pl = w * 32 + lane;
                if ((C::kWork == 1 || (i * C::kSub + pl / C::kVTok) % 2 == wv) && (!((m.valid >> (pl / kKvBlock)) & 1) || pl >= m.room))
                    for (int g = 0; g < F::kGroups; ++g)
                        *reinterpret_cast<uint32_t *>(smem + st * C::kTileBytes + (pl / kKvBlock) * F::kBlock + F::kPart + F::kCodes +
                                                      ((pl % kKvBlock) * F::kGroups + g) * 4) = 0;
                fence_proxy_async_smem();  // the stage is overwritten by a bulk copy (the async proxy) later on
                bar_sync(kHoleBar + wv, 128);
            }
#pragma unroll 1
            for (int h = (wv + i * C::kSub) % C::kWork; h < C::kSub; h += C::kWork) {
                const int u = i * C::kSub + h, b = u % C::kBufs;
                const uint8_t *vb = smem + st * C::kTileBytes + F::kPart + h * (C::kVTok / kKvBlock) * F::kBlock;
                if (u >= C::kBufs) {
                    wait(&sm.v_empty[b], ((u / C::kBufs) & 1) ^ 1, stop, a.err);
                    tc_fence_after();
                }
                if (!idle) {
#pragma unroll 1
                    for (int p = 0; p < C::kVTok; p += kBatch) {
                        // the operand's registers: D = 256, by nibble, (chunk 2w, 2w + 1) of each 8 places;
                        // else by pair of nibbles, (nibble 2q, 2q + 1) of each 8 places
                        uint32_t r[D == 256 ? 4 : 2][kBatch / 4];
#pragma unroll
                        for (int z = 0; z < kBatch / kStep; ++z, vb += (kStep / kKvBlock) * F::kBlock) {
                            uint32_t x[4];
                            ldmatrix_x4_trans(smem_u32(vb + code_at), x);
                            __half2 dd[kStep / 8], mm[kStep / 8];
#pragma unroll
                            for (int e = 0; e < kStep / 8; ++e) {
                                const uint8_t *sp = vb + scale_at + (e >> 1) * F::kBlock + (e & 1) * 8 * F::kGroups * 4;
                                const uint32_t s0 = *reinterpret_cast<const uint32_t *>(sp);
                                const uint32_t s1 = *reinterpret_cast<const uint32_t *>(sp + F::kGroups * 4);
                                dd[e] = as_h2(__byte_perm(s0, s1, 0x5410));
                                mm[e] = as_h2(__byte_perm(s0, s1, 0x7632));
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int g = D == 256 ? e >> 1 : e;
                                const uint32_t x8 = x[e] >> 8;
                                const uint32_t v[4] = {dequant_lo(x[e], dd[g], mm[g]), dequant_hi(x[e], dd[g], mm[g]),
                                                       dequant_lo(x8, dd[g], mm[g]), dequant_hi(x8, dd[g], mm[g])};
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    if constexpr (D == 256)
                                        r[j][4 * z + e] = v[j];
                                    else
                                        r[j >> 1][8 * z + 2 * e + (j & 1)] = v[j];
                                }
                            }
                        }
                        const uint32_t col = lanes + b * C::kMh * C::kVCols + p / 2;
                        if constexpr (D == 256) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                TmemWrite16<kBatch / 8>::run(col + ((uint32_t)(16 * (j & 1)) << 16) + (j >> 1) * C::kVCols, r[j]);
                        } else {
#pragma unroll
                            for (int q = 0; q < 2; ++q) TmemWrite16<kBatch / 8>::run(col + ((uint32_t)(16 * q) << 16), r[q]);
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
        constexpr int kVec = D / 8;              // 16-byte pieces of a row of q
        const int wg = (warp - 8 * C::kWork) >> 2;  // softmax warpgroup
        const int n0 = wg * NS;                  // its first query row
        const int w = warp & 3;                  // tensor-memory quadrant
        const int t = w * 32 + lane;
        const int bar_id = 1 + wg;
        constexpr int kAllBar = 1 + C::kSoft;
        const uint32_t quad = tmem + ((uint32_t)(w * 32) << 16);
        float *stage = reinterpret_cast<float *>(smem + C::kP) + wg * C::kOutRows * C::kOutStride;
        float sum[NS];
        int seg = 0;
        // q of a part of an item into its buffer, with what each row sees and where it goes; k index in the
        // order that the codes are unpacked in; rows that are not there zero
        auto stage_q = [&](const Item &m, int which) {
            const int qb = which % C::kQBufs;
            if (t < NS) {
                const uint32_t row = (uint32_t)(m.rt * N + n0 + t);
                const int tok = (int)(row / (uint32_t)a.G);
                const bool ok = tok < m.n;
                const int64_t tt = m.first + tok, hh = m.head * a.G + (int)(row - (uint32_t)tok * (uint32_t)a.G);
                sm.lim[which & 1][n0 + t] = ok ? m.len - m.n + tok : -1;
                sm.orow[which & 1][n0 + t] = ok ? tt * a.out.st + hh * a.out.sh : kNoRow;
                sm.qrow[n0 + t] = ok ? tt * a.q.st + hh * a.q.sh : kNoRow;
            }
            bar_sync(bar_id, 128);
            constexpr int kBatch = NS * kVec / 128 < 4 ? NS * kVec / 128 : 4;
#pragma unroll 1
            for (int x0 = t; x0 < NS * kVec; x0 += 128 * kBatch) {
                uint32_t v[kBatch][4];
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {
                    const int x = x0 + 128 * y;
                    const int n = n0 + (x >> 1) % NS, g = 2 * (x / (2 * NS)) + (x & 1);  // two pieces of a row side by side
                    const int64_t at = sm.qrow[n];
                    v[y][0] = v[y][1] = v[y][2] = v[y][3] = 0;
                    if (at != kNoRow) {
                        const __half *qp = static_cast<const __half *>(a.q.p) + at;
                        if (a.q.vec > 1) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(qp + 8 * g);
                            v[y][0] = u.x, v[y][1] = u.y, v[y][2] = u.z, v[y][3] = u.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                v[y][e] = as_u32(__halves2half2(qp[(8 * g + 2 * e) * a.q.sd], qp[(8 * g + 2 * e + 1) * a.q.sd]));
                        }
                    }
                }
#pragma unroll
                for (int y = 0; y < kBatch; ++y) {
                    const int x = x0 + 128 * y;
                    const int n = n0 + (x >> 1) % NS, g = 2 * (x / (2 * NS)) + (x & 1);
                    *reinterpret_cast<uint4 *>(smem + C::kQ + qb * C::kQBytes + g * 16 * N + (n >> 3) * 128 + (n & 7) * 16) =
                        make_uint4(__byte_perm(v[y][0], v[y][2], 0x5410), __byte_perm(v[y][0], v[y][2], 0x7632),
                                   __byte_perm(v[y][1], v[y][3], 0x5410), __byte_perm(v[y][1], v[y][3], 0x7632));
                }
            }
            fence_proxy_async_smem();
            bar_sync(bar_id, 128);
            if (lane == 0) mbar_arrive(smem_u32(&sm.q_full[qb]));
        };
        if (count > 0) {
            wait_described(&sm.produced, 1, stop, a.err);
            stage_q(sm.meta[0].item, 0);
        }
        Item next = {};
        bool has_next = false;
        int flags = 0;
        for (int i = 0; i < count; ++i) {
            const int sb = i % C::kSBufs, pb = i % C::kPBufs;
            wait(&sm.s_full[sb], (i / C::kSBufs) & 1, stop, a.err);
            tc_fence_after();
            const Meta &m = sm.meta[i % kMetas];
            flags = m.flags;
            const bool first = flags & kFirst;
            if (first) {
                next = m.next;
                has_next = flags & kNext;
#pragma unroll
                for (int n = 0; n < NS; ++n) sum[n] = 0.0f;
            }
            const int pos = m.pos + t;
            const bool there = ((m.valid >> (t / kKvBlock)) & 1) && t < m.room;
            float x[NS];
            // this place's scores, less the rows' references; -inf where a row does not see the place
            auto load = [&](bool less) {
                TmemRead<NS>::run(quad + C::kS + sb * N + n0, x);
#pragma unroll
                for (int n = 0; n < NS; n += 4) {
                    float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (less) b = *reinterpret_cast<const float4 *>(&sm.base[n0 + n]);
                    x[n] = fmaf(x[n], a.scale_log2, -b.x);
                    x[n + 1] = fmaf(x[n + 1], a.scale_log2, -b.y);
                    x[n + 2] = fmaf(x[n + 2], a.scale_log2, -b.z);
                    x[n + 3] = fmaf(x[n + 3], a.scale_log2, -b.w);
                }
                if (flags & kEdge) {
#pragma unroll
                    for (int n = 0; n < NS; n += 4) {
                        const int4 l = *reinterpret_cast<const int4 *>(&sm.lim[seg & 1][n0 + n]);
                        if (!there || pos > l.x) x[n] = -INFINITY;
                        if (!there || pos > l.y) x[n + 1] = -INFINITY;
                        if (!there || pos > l.z) x[n + 2] = -INFINITY;
                        if (!there || pos > l.w) x[n + 3] = -INFINITY;
                    }
                }
            };
            load(!first);
            bool move = first;
            if (!first) {
                float over = x[0];
#pragma unroll
                for (int n = 1; n < NS; ++n) over = fmaxf(over, x[n]);
                move = over > kMoveMax + kWeightShift;
            }
            if (bar_or(bar_id, 128, move)) {
                // the rows' maxima over the 128 places; O and the sums follow the reference
                if (!first) load(false);
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    const int top = __reduce_max_sync(0xffffffffu, float_order(x[n]));
                    if (lane == (n & 31)) sm.wred[w][n0 + n] = order_float(top);
                }
                bar_sync(bar_id, 128);
                if (t < NS) {
                    const float old = first ? -INFINITY : sm.ref[n0 + t];
                    float top = old;
#pragma unroll
                    for (int y = 0; y < 4; ++y) top = fmaxf(top, sm.wred[y][n0 + t]);
                    if (sm.lim[seg & 1][n0 + t] < 0) top = fmaxf(top, 0.0f);  // a row that sees nothing stays out of this
                    sm.ref[n0 + t] = top;
                    // a row that has seen nothing yet moves at its first score
                    sm.base[n0 + t] = top == -INFINITY ? -1e30f : top - kWeightShift;
                    sm.factor[n0 + t] = top == -INFINITY ? 1.0f : ex2(old - top);
                }
                bar_sync(bar_id, 128);
                if (!first) {
#pragma unroll
                    for (int n = 0; n < NS; ++n) sum[n] *= sm.factor[n0 + n];
                    // every product before this tile is in O
                    wait(&sm.p_empty[(i - 1) % C::kPBufs], ((i - 1) / C::kPBufs) & 1, stop, a.err);
                    tc_fence_after();
#pragma unroll 1
                    for (int y = 0; y < C::kMh * NS; y += 16) {
                        const uint32_t at = quad + C::kO + (y / NS) * N + n0 + y % NS;
                        float o[16];
                        uint32_t r[16];
                        TmemRead<16>::run(at, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[e] * sm.factor[n0 + y % NS + e]);
                        TmemWrite32<16>::run(at, r);
                    }
                    tmem_wait_st();
                }
                load(true);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.s_empty[sb]));
            if (i >= C::kPBufs) wait(&sm.p_empty[pb], ((i / C::kPBufs) & 1) ^ 1, stop, a.err);
            uint8_t *pp = smem + C::kP + pb * C::kPBytes + (n0 >> 3) * (16 * kTile) + (t >> 3) * 128 + (t & 7) * 16;
#pragma unroll
            for (int n = 0; n < NS; n += 8) {
                float e[8];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    e[y] = ex2(x[n + y]);
                    sum[n + y] += e[y];
                }
                *reinterpret_cast<uint4 *>(pp + (n >> 3) * (16 * kTile)) =
                    make_uint4(pack_h2(e[0], e[1]), pack_h2(e[2], e[3]), pack_h2(e[4], e[5]), pack_h2(e[6], e[7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.p_full[pb]));
            // q of the next part: in its own buffer while this part runs (the first products of the part before
            // this one are done: their scores came before this tile's), or when this part's are done
            if (C::kQBufs > 1 ? first && has_next : (flags & kLast) && has_next) {
                if (C::kQBufs == 1 && C::kSoft > 1) bar_sync(kAllBar, 128 * C::kSoft);
                stage_q(next, seg + 1);
            }
            if (flags & kLast) {
                // ---- the sums over the places
#pragma unroll
                for (int c = 0; c < NS; c += 16) {
                    float v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = sum[c + e];
                    const float r = reduce_scatter<16>(v, lane);
                    if (lane < 16) sm.wred[w][n0 + c + lane] = r;
                }
                bar_sync(bar_id, 128);
                const int slot = 2 * cta + ((flags & kFromStart) ? 1 : 0);
                const bool complete = flags & kComplete;
                if (t < NS) {
                    const int n = n0 + t;
                    const float den = (sm.wred[0][n] + sm.wred[1][n]) + (sm.wred[2][n] + sm.wred[3][n]);
                    sm.inv[n] = complete ? (den > 0.0f ? 1.0f / den : 0.0f) : 1.0f;
                    if (!complete) a.stat[(int64_t)slot * N + n] = make_float2(sm.ref[n], den);
                }
                wait(&sm.o_full, seg & 1, stop, a.err);
                tc_fence_after();
                bar_sync(bar_id, 128);
                // ---- O, some rows at a time through shared memory (the weights' buffers are free now)
                // (loops kept rolled: this code is seldom in the instruction caches)
#pragma unroll 1
                for (int c = 0; c < NS; c += C::kOutRows) {
#pragma unroll 1
                    for (int z = 0; z < C::kMh * C::kOutRows; z += 8) {
                        const int mh = z / C::kOutRows, c8 = z % C::kOutRows;
                        float o[8];
                        TmemRead<8>::run(quad + C::kO + mh * N + n0 + c + c8, o);
                        float *to = stage + c8 * C::kOutStride + o_dim<D>(t, mh);
                        if (D > 64 || t < 64) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) to[e * C::kOutStride] = o[e] * sm.inv[n0 + c + c8 + e];
                        }
                    }
                    bar_sync(bar_id, 128);
#pragma unroll 1
                    for (int y = t; y < C::kOutRows * kVec; y += 128) {
                        const int e = y / kVec, g = y % kVec;
                        const int64_t at = sm.orow[seg & 1][n0 + c + e];
                        const float4 v0 = *reinterpret_cast<const float4 *>(stage + e * C::kOutStride + 8 * g);
                        const float4 v1 = *reinterpret_cast<const float4 *>(stage + e * C::kOutStride + 8 * g + 4);
                        if (at == kNoRow) continue;
                        if (!complete) {
                            float *dst = a.part + ((int64_t)slot * N + n0 + c + e) * D + 8 * g;
                            *reinterpret_cast<float4 *>(dst) = v0;
                            *reinterpret_cast<float4 *>(dst + 4) = v1;
                        } else {
                            __half *dst = static_cast<__half *>(a.out.p) + at + 8 * g * a.out.sd;
                            const uint4 h = make_uint4(pack_h2(v0.x, v0.y), pack_h2(v0.z, v0.w), pack_h2(v1.x, v1.y), pack_h2(v1.z, v1.w));
                            if (a.out.vec > 1) {
                                *reinterpret_cast<uint4 *>(dst) = h;
                            } else {
                                const uint32_t hh[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    dst[2 * x * a.out.sd] = __low2half(as_h2(hh[x]));
                                    dst[(2 * x + 1) * a.out.sd] = __high2half(as_h2(hh[x]));
                                }
                            }
                        }
                    }
                    if (c + C::kOutRows < NS) bar_sync(bar_id, 128);
                }
                tc_fence_before();
                // no warpgroup writes weights over another's staging area
                if (C::kSoft > 1)
                    bar_sync(kAllBar, 128 * C::kSoft);
                else
                    bar_sync(bar_id, 128);
                if (lane == 0) mbar_arrive(smem_u32(&sm.o_empty));
                ++seg;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (stop->gave_up) {
        if (threadIdx.x == 0) g_gave_up = 1;
        // copies and products in flight end before shared and tensor memory are given up
        if (warp == kProducer)
            for (int st = 0; st < C::kStages && st < sm.produced; ++st)
                (void)mbar_wait_bounded(smem_u32(&sm.ring_full[st]), ((sm.produced - 1 - st) / C::kStages) & 1);
        if (warp >= kIssuer) {
            umma_commit_elect(smem_u32(&sm.drained[warp - kIssuer]));
            (void)mbar_wait_bounded(smem_u32(&sm.drained[warp - kIssuer]), 0);
        }
        __syncthreads();
    }
    if (warp == kIssuer) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The items that were cut between CTAs: out = sum_i 2^(ref_i - ref) O_i / sum_i 2^(ref_i - ref) sum_i,
// in a fixed order.  One block takes RB rows of one item; D / 4 threads share a row's dimensions and the
// rest of its threads the parts.
constexpr int kMostParts = 1024;  // an item has at most one part a CTA

template <int D, int N, int RB> __global__ void __launch_bounds__(512) attn_kv4_join_kernel(const AttnArgs a)
{
    constexpr int TX = D / 4;            // threads across a row
    constexpr int TY = 512 / (TX * RB);  // threads that share its parts
    static_assert(TY >= 1, "a row's threads fit the block");
    __shared__ float4 acc[RB][TY][TX];
    __shared__ float factor[RB][kMostParts / (RB > 1 ? 4 : 1)];
    __shared__ float den[RB];
    pdl_launch_dependents();
    pdl_wait();
    const int4 c = a.cut[blockIdx.x];
    const int gave_up = *a.err;  // (cuts and parts may be missing then)
    if ((c.w == 0) | (gave_up != 0)) return;
    const int head = c.y & 0xffff, cta = c.y >> 16;
    const int x = threadIdx.x % TX, y = threadIdx.x / TX % TY, rl = threadIdx.x / (TX * TY);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Seq q = load_seq<N>(a, c.x);
    auto slot = [&](int i) -> int64_t { return i ? 2 * (cta + i) : 2 * cta + 1; };
    // a warp a row: the reference of all parts, each part's factor, the sum
    if (warp < RB) {
        const int r = blockIdx.y * RB + warp;
        float top = -INFINITY;
        for (int i = lane; i < c.w; i += 32) top = fmaxf(top, a.stat[slot(i) * N + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float l = 0.0f;
        for (int i = lane; i < c.w; i += 32) {
            const float2 st = a.stat[slot(i) * N + r];
            const float f = st.x == -INFINITY ? 0.0f : ex2(st.x - top);
            factor[warp][i] = f;
            l = fmaf(st.y, f, l);
        }
        l = warp_sum(l);
        if (lane == 0) den[warp] = l;
    }
    __syncthreads();
    const int r = blockIdx.y * RB + rl;
    const uint32_t row = (uint32_t)(c.z * N + r);
    const int tok = (int)(row / (uint32_t)a.G);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (tok < q.n) {
#pragma unroll 8
        for (int i = y; i < c.w; i += TY) {
            const float f = factor[rl][i];
            const float4 u = *reinterpret_cast<const float4 *>(a.part + (slot(i) * N + r) * D + 4 * x);
            v.x = fmaf(u.x, f, v.x);
            v.y = fmaf(u.y, f, v.y);
            v.z = fmaf(u.z, f, v.z);
            v.w = fmaf(u.w, f, v.w);
        }
    }
    if (TY > 1) {
        acc[rl][y][x] = v;
        __syncthreads();
        if (y != 0) return;
        for (int i = 1; i < TY; ++i) {
            const float4 u = acc[rl][i][x];
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
    }
    if (tok >= q.n) return;
    const float inv = den[rl] > 0.0f ? 1.0f / den[rl] : 0.0f;
    const float w[4] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv};
    store_dims<4>(a.out, q.first + tok, head * a.G + (int)(row - (uint32_t)tok * (uint32_t)a.G), 4 * x, w);
}

// Query rows of an item: the fewest columns that hold what a sequence has (by the caller's max_q), so that
// few rows leave tensor time and shared memory to the copies; many rows share each unpacked tile.  With 16, 32, 64 and
// 128 columns, 12 rows on 200001 places took 69, 87, 89 and 136 us, 48 rows on 4 x 30000 places 112, 106, 69 and 103,
// and 6000 rows on 8000 places 881, 586, 316 and 272.
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
    if (cuda_status(cudaGetDevice(&dev)) != QG_OK) return QG_ERR_CUDA;
    if (dev >= 64 || !(raised.load() >> dev & 1)) {
        if (cuda_status(cudaFuncSetAttribute(attn_kv4_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, N>::kBytes)) != QG_OK)
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
        return launch_pdl(attn_kv4_join_kernel<D, N, 1>, dim3((unsigned)items, N), dim3(512), 0, stream, a);
    return launch_pdl(attn_kv4_join_kernel<D, N, 4>, dim3(grid, N / 4), dim3(512), 0, stream, a);
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
    if (T * (Hq / Hk) > 0x7fffffff - 256) return QG_ERR_SHAPE;
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
    if (sms > kMostParts / 4) return QG_ERR_SHAPE;  // (no such device)
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

int qg_attn_kv4_device_error(void *stream, int *flag)
{
    if (!flag) return QG_ERR_NULL;
    *flag = 0;
    void *p = nullptr;
    int v = 0;
    if (cuda_status(cudaGetSymbolAddress(&p, g_gave_up)) != QG_OK ||
        cuda_status(cudaStreamSynchronize(static_cast<cudaStream_t>(stream))) != QG_OK ||
        cuda_status(cudaMemcpy(&v, p, sizeof(v), cudaMemcpyDeviceToHost)) != QG_OK)
        return QG_ERR_CUDA;
    if (v != 0 && cuda_status(cudaMemset(p, 0, sizeof(v))) != QG_OK) return QG_ERR_CUDA;
    *flag = v;
    return QG_OK;
}

}  // extern "C"
