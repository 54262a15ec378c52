// qg_sample.cu -- one token a row from its logits and a given random number (qg_sample).  Declaration
// and contract: include/qg.h.
//
// With z = logit / temperature, in descending order (equal logits: the lower index first):
//   top-k keeps the first k; top-p keeps, of those, each token before which less than p of their weight
//   w = exp(z - z_max) lies; min-p drops weights below min_p; the token is the first in the vocabulary's
//   order whose running weight exceeds u times the kept weight.
// Each filter keeps a prefix of the descending order, so the kept tokens are those above a logit and the
// first few equal to it: a cut.
//
// One thread-block cluster takes a row and keeps it in its shared memory (up to sixteen CTAs, so 248,320
// logits are read once), and the passes over the row run on chip.  The row is never sorted:
//   1. the largest logit;
//   2. a histogram of counts over bins linear in z, 64 a factor of two, and (for top-p) the weights' sum in fp32;
//   3. the bins in which the cut lies: exactly known for the k-th token; for top-p, since a bin's weights
//      are within a factor 2^(1/64) of each other, the weight below a bin is bounded on both sides by the
//      counts, which leaves two or three bins.  If the tokens down to the last of these are at most 1024,
//      they are gathered in one CTA, sorted, filtered and chosen from;
//   4. otherwise only the tokens of those bins are gathered, and counted (or weighed) in finer and finer bins, with
//      the exact weight above them, which gives the cut (should they be too many for a list, over the row itself);
//   5. the token is found from the running sums in index order: from those of 4, a thread's consecutive logits each,
//      and the listed tokens above the cut, or by another pass where that does not do (min-p, ties at the cut).
//
// Weights are whole multiples of 2^-44 of the largest (64-bit integers): their sums do not depend on the order
// of the additions, so a call gives the same token every time.  A weight is off by about 2^-30 of itself
// (Row::weight), in either direction, and by half of 2^-44 at most from its rounding to a whole number, of which
// those below 2^-45 lose all.  The choice is that of the exact formula but for u (or a filter's border) within
// 2^-30 + V 2^-45 of a border: 1e-9 where the weights in the sums are large, 3e-8 (half a step of u next to 1) for a
// million of the smallest.  64-bit exponentials instead (exact to 2^-45) took 113 cycles of a scheduler for 32 of them.
//
// What bounds it is the chain of stages, most of them short and run once, 32 warps wide: about 55,000 cycles for a row
// of 151936 (32 us; its bytes would take 0.1), of which the passes over the row are 12,000, the list's sorts 4,000 to
// 9,000, and the rest sums and barriers of the block and the cluster, and code that no cache holds yet.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <mutex>

#include "qg_kv4.cuh"

namespace {

using namespace qg;
namespace cg = cooperative_groups;

constexpr int kThreads = 1024;  // (with 512, 16 x 248320 took a quarter longer)
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 4096;
constexpr int kPer = kBins / kThreads;  // bins of a thread
constexpr float kBinStep = 0.98922801319397548f;  // 2^(-1/64)
constexpr float kDeepest = 45.9f;  // the bins go down to 2^-45.9 of the largest weight (from 2^-45 on weights are 0)
constexpr int kList = 2 * kThreads;
constexpr double kOne = 17592186044416.0;  // the largest weight, 2^44
typedef unsigned long long u64;
constexpr int64_t kMostLogits = (1 << 20) - 1;  // so many weights of 2^44 fit 64 bits
constexpr int kMostCtas = 16;
constexpr double kRough = 4294967296.0;  // the largest weight in the rough sum
constexpr int64_t kMostRows = 16 * 65535;       // rows_kernel's grid

struct SampleArgs {
    const float *x;
    int64_t V, rs, es;  // strides in elements
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *token;
    int64_t per;  // logits of a CTA
};

struct Shared {
    alignas(16) unsigned count[kBins];
    alignas(16) unsigned total[kBins];  // of the cluster
    u64 list[kList];  // key << 32 | ~index (the cluster's, in its first CTA)
    u64 own[kList];   // the CTA's part of the list; weights of finer histograms
    unsigned table[64];  // 2^(i / 64) in 2^-30
    // exchanged over the cluster
    float top;
    int64_t best;
    unsigned listed, klo, khi, cut_key, cut_ties, cta_ties;
    u64 cta_weight, cta_total, cta_rough;
    // the CTA's own
    unsigned own_listed, own_at;
    u64 scan_w[kWarps];
    unsigned scan_c[kWarps];
    float scan_f[2][kWarps];
    int bin[2];
    unsigned before[2], in_bin;
    u64 fine_before;
};

// logits in an order-preserving integer form
__device__ __forceinline__ unsigned key_of(float x)
{
    const unsigned b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float of_key(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }

__device__ __forceinline__ float clean(float x)
{
    x += 0.0f;                      // -0 and +0 are equal
    return x != x ? -INFINITY : x;  // NaN is never chosen
}

// (kept out of line: code that is seldom run costs those passes that would have to be fetched around it)
__device__ __noinline__ bool at_least_exact(double t, double min_p) { return exp2(t) >= min_p; }

// A CTA's part of a row; RESIDENT: in shared memory.
template <bool RESIDENT> struct Row {
    const float *x;  // in global memory otherwise
    int64_t es;
    const float *slice;
    const unsigned *table;
    bool infinite;  // the largest logit is +inf: those count as 0, all others as -inf
    int n;
    float xmax;
    double c, zc;  // log2(e) / temperature, and the largest logit times it
    float ch, cl;  // c as the sum of two floats

    __device__ __forceinline__ float get(int i) const
    {
        float v;
        if constexpr (RESIDENT)
            v = slice[i];
        else
            v = clean(x[i * es]);
        return !infinite ? v : v == INFINITY ? 0.0f : -INFINITY;
    }
    // f(i, x) for the CTA's logits
    template <typename F> __device__ __forceinline__ void each(F f) const
    {
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += kThreads) f(i, get(i));
    }
    // The weight in whole 2^-44, without a branch, and the bin of the histogram.
    // t = (xmax - x) c is formed as a sum of two floats (the difference and the product with their rounding
    // errors: about 2^-46 of t).  With n = 64 t rounded, which is the bin (monotone in x), t = n / 64 + r and
    // |r| <= 1/128: 2^-t = 2^-q 2^(j/64) e^y, y = -r ln 2; a table, and the Taylor series of e^y - 1 to the third
    // power in fp32 (2^-24 of at most 0.0055; the fourth power is below 4e-11), multiplied in 62 bits and rounded.
    __device__ __forceinline__ u64 weight(float x, int *bin) const
    {
        const float d = xmax - x;
        const float v = d - xmax;
        const float dl = (xmax - (d - v)) - (x + v);
        const float t0 = d * ch;
        const float t = fminf(t0, kDeepest);
        const float tl = fmaf(d, ch, -t0) + fmaf(d, cl, dl * ch);  // (NaN at -inf)
        const float m = fmaf(t, 64.0f, 12582912.0f);  // 1.5 * 2^23: the sum's low bits are 64 t, rounded
        const int n64 = __float_as_int(m) - 0x4b400000;
        const float y = (fmaf(m - 12582912.0f, -1.0f / 64.0f, t) + tl) * -0.693147180559945f;
        const float e = y * fmaf(y, fmaf(y, 1.0f / 6.0f, 0.5f), 1.0f);
        const int q = (n64 + 63) >> 6;
        const unsigned factor = 0x80000000u + (unsigned)__float2int_rn(e * 2147483648.0f);
        *bin = n64;
        const u64 w = ((u64)table[(q << 6) - n64] * factor + (1ull << (16 + q))) >> (17 + q);
        return t0 < kDeepest ? w : 0;  // (deeper, y is of no matter)
    }
    __device__ __forceinline__ u64 weight(float x) const
    {
        int b;
        return weight(x, &b);
    }
    __device__ __forceinline__ int bin(float x) const
    {
        return __float_as_int(fmaf(fminf((xmax - x) * ch, kDeepest), 64.0f, 12582912.0f)) - 0x4b400000;
    }
    __device__ __forceinline__ float rough(float x) const { return exp2f(-fminf((xmax - x) * ch, kDeepest)); }
    // whether the weight is at least min_p (decided in 64 bits where it is close)
    __device__ __forceinline__ bool at_least(float x, u64 w, double min_p) const
    {
        if (x == xmax) return true;
        const double least = min_p * kOne;
        if (fabs((double)w - least) > least * 1e-6 + 2.0) return (double)w > least;
        return at_least_exact(fma((double)x, c, -zc), min_p);
    }
};

// What a block does once it does 32 warps wide, eight cycles an instruction: sums over a warp are single reductions
// (of 64 bits three, by 24 bits), and prefixes come for counts and for weights apart.
__device__ __forceinline__ unsigned warp_total(unsigned v) { return __reduce_add_sync(0xffffffffu, v); }
__device__ __forceinline__ u64 warp_total(u64 v)
{
    const unsigned a = warp_total((unsigned)v & 0xffffffu), b = warp_total((unsigned)(v >> 24) & 0xffffffu), c = warp_total((unsigned)(v >> 48));
    return ((u64)c << 48) + ((u64)b << 24) + a;
}
__device__ __forceinline__ float warp_total(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename T> __device__ __forceinline__ T warp_incl(T v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

// Sum of w over the block.
__device__ __noinline__ u64 block_sum(Shared &s, u64 w)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    w = warp_total(w);
    __syncthreads();
    if (lane == 0) s.scan_w[warp] = w;
    __syncthreads();
    return warp_total(lane < kWarps ? s.scan_w[lane] : 0ull);
}

// Exclusive prefix over the block's threads, and the total.
template <typename T> struct Scan {
    T before, all;
};
template <typename T> __device__ __forceinline__ Scan<T> scan_over(T *parts, T v)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T incl = warp_incl(v, lane);
    __syncthreads();
    if (lane == 31) parts[warp] = incl;
    __syncthreads();
    const T part = lane < kWarps ? parts[lane] : T(0);
    return {incl - v + warp_total(lane < warp ? part : T(0)), warp_total(part)};
}
__device__ __noinline__ Scan<unsigned> block_scan(Shared &s, unsigned c) { return scan_over(s.scan_c, c); }
__device__ __noinline__ Scan<u64> block_scan(Shared &s, u64 w) { return scan_over(s.scan_w, w); }

// Sum of a CTA's value over the cluster: each warp fetches the CTAs' values with one load.
template <typename T> __device__ __forceinline__ T over_cluster(cg::cluster_group &cl, Shared &s, T Shared::*field)
{
    const unsigned lane = threadIdx.x & 31;
    return warp_total(lane < cl.num_blocks() ? cl.map_shared_rank(&s, lane)->*field : T(0));
}

// Descending sort of one 64-bit value a thread (bitonic: exchanges within a warp by shuffles, between warps
// through shared memory); m values, the others 0.  Warps past the power of two that holds m take no part.
__device__ __noinline__ u64 block_sort(u64 v, u64 *buf, int m)
{
    const int t = threadIdx.x;
    int size = 32;
    while (size < m) size <<= 1;
    if (t < size) {
#pragma unroll 1
        for (int k = 2; k <= size; k <<= 1)
#pragma unroll 1
            for (int j = k >> 1; j > 0; j >>= 1) {
                u64 o;
                if (j >= 32) {
                    asm volatile("bar.sync 1, %0;" ::"r"(size) : "memory");
                    buf[t] = v;
                    asm volatile("bar.sync 1, %0;" ::"r"(size) : "memory");
                    o = buf[t ^ j];
                } else {
                    o = __shfl_xor_sync(0xffffffffu, v, j);
                }
                const bool low = (t & j) == 0, down = (t & k) == 0;
                v = (low == down) == (v > o) ? v : o;
            }
    }
    __syncthreads();
    return v;
}

// The cluster's histogram, kPer bins a thread.  Each CTA adds up its share of the bins and hands the sums to
// all (every CTA reading every histogram took four times as long with sixteen).
__device__ __forceinline__ void cluster_counts(cg::cluster_group &cl, Shared &s, unsigned (&c)[kPer])
{
    const unsigned n = cl.num_blocks();
    cl.sync();  // all histograms are whole
    if (n > 1) {
        const unsigned share = (kBins + n - 1) / n, end = min((cl.block_rank() + 1) * share, (unsigned)kBins);
        for (unsigned at = cl.block_rank() * share + threadIdx.x; at < end; at += kThreads) {
            unsigned sum = 0;
#pragma unroll 4
            for (unsigned r = 0; r < n; ++r) sum += cl.map_shared_rank(&s, r)->count[at];
#pragma unroll 4
            for (unsigned r = 0; r < n; ++r) cl.map_shared_rank(&s, r)->total[at] = sum;
        }
        cl.sync();
    }
    const uint4 *from = reinterpret_cast<const uint4 *>(&(n > 1 ? s.total : s.count)[kPer * threadIdx.x]);
#pragma unroll
    for (int j = 0; j < kPer; j += 4) {
        const uint4 v = from[j / 4];
        c[j] = v.x, c[j + 1] = v.y, c[j + 2] = v.z, c[j + 3] = v.w;
    }
}

// The bin in which the k-th token lies, with the tokens before it and in it.  Returns the number of all.
__device__ unsigned find_count(Shared &s, const unsigned (&c)[kPer], unsigned k)
{
    unsigned sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += c[j];
    const Scan<unsigned> z = block_scan(s, sum);
    unsigned cb = z.before;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (cb < k && cb + c[j] >= k) {
            s.bin[0] = s.bin[1] = kPer * threadIdx.x + j;
            s.before[0] = cb;
            s.in_bin = c[j];
        }
        cb += c[j];
    }
    __syncthreads();
    return z.all;
}

// The bins between which the cut of top-p lies: the first whose lower bound, and the first whose upper bound,
// of the weight after it is at most `tail`.  s.before[0]: tokens before the first, s.before[1]: down to the
// last of them (of all tokens, `c`; the weights are those of `kept` of them).  The bounds' margin of 2e-4
// covers the bins' borders, these sums and the one in `tail`, all in fp32 (of at most 2^10 logits a thread).
// A tail of weights below 2^-32 is off by more than that margin as whole numbers of 2^-44; the cut may then lie past the
// last of these bins (all of them are kept) or before the first (none), by less than the tail weighs.
// The same sum is rounded differently by two neighbouring threads, so both may see a border between their bins, or
// neither: of several the outermost bins are taken, by atomics, so that every CTA of a cluster, from the same
// counts, takes the same ones (how many cluster barriers it meets depends on them), and of none all bins.
__device__ void find_share(Shared &s, const unsigned (&c)[kPer], const unsigned (&kept)[kPer], float tail)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b0 = kPer * threadIdx.x;
    // a bin holds t within half a bin of b / 64; the last one that is used everything deeper
    float edge = exp2f(-((float)b0 - 0.5f) / 64.0f), h = 0.0f, l = 0.0f;
    float hi[kPer], lo[kPer];  // weight of a bin, at most and at least
    unsigned sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        hi[j] = (float)kept[j] * edge * 1.0002f;
        edge *= kBinStep;
        lo[j] = b0 + j >= 2937 ? 0.0f : (float)kept[j] * edge * 0.9998f;
        h += hi[j];
        l += lo[j];
        sum += c[j];
    }
    // of the bins after the thread's
    float hs = h, ls = l;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, hs, o), y = __shfl_down_sync(0xffffffffu, ls, o);
        if (lane + o < 32) {
            hs += x;
            ls += y;
        }
    }
    if (lane == 0) {
        s.scan_f[0][warp] = hs;
        s.scan_f[1][warp] = ls;
    }
    float after_h = __shfl_down_sync(0xffffffffu, hs, 1), after_l = __shfl_down_sync(0xffffffffu, ls, 1);
    if (lane == 31) after_h = after_l = 0.0f;
    const Scan<unsigned> z = block_scan(s, sum);
    unsigned cb = z.before;
    if (threadIdx.x == 0) {
        s.bin[0] = kBins;
        s.bin[1] = -1;
    }
    const bool later = lane > warp && lane < kWarps;
    after_h += warp_total(later ? s.scan_f[0][lane] : 0.0f);
    after_l += warp_total(later ? s.scan_f[1][lane] : 0.0f);
    __syncthreads();
    // up through the thread's bins: the weight after bin j, and after the bin before it
#pragma unroll
    for (int j = kPer - 1; j >= 0; --j) {
        const bool first = b0 + j == 0;
        if (after_l <= tail && (first || after_l + lo[j] > tail)) atomicMin(&s.bin[0], b0 + j);
        if (after_h <= tail && (first || after_h + hi[j] > tail)) atomicMax(&s.bin[1], b0 + j);
        after_l += lo[j];
        after_h += hi[j];
    }
    __syncthreads();
    const int from = s.bin[0] < kBins ? s.bin[0] : 0, to = s.bin[1] >= 0 ? s.bin[1] : kBins - 1;
    __syncthreads();  // (read everywhere)
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (b0 + j == from) {
            s.bin[0] = from;
            s.before[0] = cb;
        }
        cb += c[j];
        if (b0 + j == to) {
            s.bin[1] = to;
            s.before[1] = cb;
        }
    }
    __syncthreads();
}

// The cut of a share among the m listed tokens, with `above` before them: s.cut_key and s.cut_ties (all: kAll).
// Their weights are added up over finer and finer bins of their keys (a sort of 1024 took 19,600 cycles, a round of
// this takes 3,000, and there are two or three), until the bin in which the running weight reaches the target has
// one key.
constexpr unsigned kAll = 0xffffffffu;
template <bool RESIDENT> __device__ __noinline__ void cut_of_list(Shared &s, const Row<RESIDENT> &r, int m, u64 above, double target)
{
    u64 *bins = reinterpret_cast<u64 *>(s.count);  // (the histogram has been read)
    const int tid = threadIdx.x;
    unsigned key[kList / kThreads], lo = 0xffffffffu, hi = 0;
#pragma unroll
    for (int j = 0; j < kList / kThreads; ++j) {
        const int at = tid + j * kThreads;
        key[j] = at < m ? (unsigned)(s.list[at] >> 32) : 0;  // (no token has key 0)
        if (key[j]) {
            lo = min(lo, key[j]);
            hi = max(hi, key[j]);
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if ((tid & 31) == 0) {
        atomicMin(&s.klo, lo);
        atomicMax(&s.khi, hi);
    }
    __syncthreads();
    lo = s.klo;
    hi = s.khi;
    for (;;) {
        const int shift = hi - lo >= (unsigned)kThreads ? 22 - __clz(hi - lo) : 0;
        bins[tid] = 0;
        if (tid == 0) s.bin[0] = -1;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kList / kThreads; ++j)
            if (key[j] >= lo && key[j] <= hi) {
                const u64 w = r.weight(of_key(key[j]));
                if (w) atomicAdd(&bins[(hi - key[j]) >> shift], w);
            }
        __syncthreads();
        const u64 w = bins[tid];
        const Scan<u64> z = block_scan(s, w);
        if (w && (double)(above + z.before) < target && !((double)(above + z.before + w) < target)) {
            s.bin[0] = tid;
            s.fine_before = z.before;
        }
        __syncthreads();
        const int b = s.bin[0];
        if (b < 0) {  // (in the first round only) none of the list is kept, or all of it
            if (tid == 0) {
                s.cut_key = (double)above < target ? lo : hi;
                s.cut_ties = (double)above < target ? kAll : above ? 0 : 1;  // (p of 0: the first token alone)
            }
            break;
        }
        above += s.fine_before;
        hi -= (unsigned)b << shift;
        const unsigned width = (1u << shift) - 1;
        lo = hi - lo < width ? lo : hi - width;
        if (lo == hi) {
            // the fewest ties whose weight reaches the target
            unsigned n = 0;
#pragma unroll
            for (int j = 0; j < kList / kThreads; ++j) n += key[j] == lo;
            const unsigned equal = block_scan(s, n).all;
            if (tid == 0) {
                const double need = ceil((target - (double)above) / (double)r.weight(of_key(lo)));
                s.cut_key = lo;
                s.cut_ties = need < (double)equal ? (need < 1.0 ? 1u : (unsigned)need) : kAll;  // (all: no need to count them)
            }
            break;
        }
        __syncthreads();  // (the bins have been read)
    }
    __syncthreads();
}

template <bool RESIDENT> __global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs a)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared &s = *reinterpret_cast<Shared *>(dyn);
    float *slice = reinterpret_cast<float *>(dyn + sizeof(Shared));
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), C = cl.num_blocks();
    const int64_t row = blockIdx.x / C;
    const int lane = threadIdx.x & 31, tid = threadIdx.x;

    for (int b = tid; b < kBins; b += kThreads) s.count[b] = 0;
    if (tid < 64) s.table[tid] = __double2uint_rn(exp2(tid / 64.0) * 1073741824.0);
    if (tid == 0) {
        s.best = INT64_MAX;
        s.listed = s.own_listed = 0;
        s.klo = 0xffffffffu;
        s.khi = 0;
    }
    pdl_launch_dependents();
    pdl_wait();

    // ---- the row into shared memory, and its largest logit
    const int64_t base = (int64_t)rank * a.per;
    const int n = (int)(base < a.V ? (a.V - base < a.per ? a.V - base : a.per) : 0);
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    const int64_t k_arg = a.top_k ? a.top_k[row] : 0;
    const double p_arg = a.top_p ? (double)a.top_p[row] : 1.0;
    double mp = a.min_p ? (double)a.min_p[row] : 0.0;
    const double u = a.u[row] < 0.0f ? 0.0 : (double)a.u[row];
    const float *x = a.x + row * a.rs + base * a.es;
    float top = -INFINITY;
    {
        int i = tid;
        constexpr int U = 8;
        for (; i + (U - 1) * kThreads < n; i += U * kThreads) {
            float v[U];
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = x[(i + (int64_t)j * kThreads) * a.es];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const float y = clean(v[j]);
                if (RESIDENT) slice[i + j * kThreads] = y;
                top = fmaxf(top, y);
            }
        }
        for (; i < n; i += kThreads) {
            const float y = clean(x[i * a.es]);
            if (RESIDENT) slice[i] = y;
            top = fmaxf(top, y);
        }
    }
    auto warp_max = [](float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    };
    top = warp_max(top);
    if (lane == 0) s.scan_f[0][tid >> 5] = top;
    __syncthreads();
    top = warp_max(lane < kWarps ? s.scan_f[0][lane] : -INFINITY);
    if (tid == 0) s.top = top;
    cl.sync();
    top = warp_max(lane < C ? cl.map_shared_rank(&s, lane)->top : -INFINITY);
    if (top == -INFINITY) {  // nothing to choose from
        if (rank == 0 && tid == 0) a.token[row] = -1;
        cl.sync();
        return;
    }
    const unsigned k = k_arg > 0 && k_arg < a.V ? (unsigned)k_arg : 0;  // 0: all
    const bool by_p = p_arg < 1.0;
    const double p = p_arg > 0.0 ? p_arg : 0.0;
    const bool infinite = top == INFINITY;
    if (infinite) top = 0.0f;
    Row<RESIDENT> r{x, a.es, slice, s.table, infinite, n, top, 0.0, 0.0, 0.0f, 0.0f};

    if (!(t > 0.0f) || k == 1 || mp > 1.0) {
        // the lowest index of the largest logit
        int64_t best = INT64_MAX;
        for (int i = tid; i < n && best == INT64_MAX; i += kThreads)
            if (r.get(i) == top) best = base + i;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int64_t b = __shfl_xor_sync(0xffffffffu, best, o);
            best = b < best ? b : best;
        }
        if (lane == 0 && best != INT64_MAX) atomicMin(reinterpret_cast<long long *>(&s.best), (long long)best);
        cl.sync();
        if (rank == 0 && tid == 0) {
            for (int c = 0; c < C; ++c) {
                const int64_t b = cl.map_shared_rank(&s, c)->best;
                best = b < best ? b : best;
            }
            a.token[row] = (int32_t)best;
        }
        cl.sync();
        return;
    }
    r.c = 1.4426950408889634074 / (double)fmaxf(t, FLT_MIN);  // (finite in fp32)
    r.zc = (double)top * r.c;
    r.ch = (float)r.c;
    r.cl = (float)(r.c - (double)r.ch);

    // kept: the tokens above cut_key, and the first cut_ties equal to it
    // the logits of a thread where order counts: consecutive, an odd number of them, so that the threads' reads fall
    // in different banks
    const int seg = ((n + kThreads - 1) / kThreads) | 1;
    const int i0 = min(n, tid * seg), i1 = min(n, i0 + seg);
    u64 above_mine = 0;   // weight of the thread's logits in the bins above the cut's
    bool listed = false;  // ... and the kept tokens of the cut's bins are those of the list from cut_key up
    unsigned cut_key = 0, cut_ties = kAll;
    if (k || by_p) {
        u64 all_w = 0;      // the share's total
        float rough = 0.0f;  // of all weights, in fp32 (all that finding the bins takes)
        r.each([&](int, float x) {
            if (x != -INFINITY) {
                atomicAdd(&s.count[r.bin(x)], 1u);
                rough += r.rough(x);
            }
        });
        if (!k) {
            const u64 w = block_sum(s, (u64)(rough * kRough));
            if (tid == 0) s.cta_rough = w;
        }
        unsigned c[kPer], kept_c[kPer];  // tokens of a bin, and those of the first k
        cluster_counts(cl, s, c);
        float tail = 0.0f;
        if (!k) tail = (float)((1.0 - p) * (double)over_cluster(cl, s, &Shared::cta_rough) * (1.0 / kRough));
#pragma unroll
        for (int j = 0; j < kPer; ++j) kept_c[j] = c[j];

        // Two cuts at most: the k-th token, and then (unless the list of all that can be kept settles it) the
        // share of the first k's weight.
        for (int pass = k ? 0 : 1; pass < 2; ++pass) {
            const bool share = pass == 1;
            if (share && !by_p) break;
            unsigned before, reach;  // tokens before the bins of the cut, and down to the last of them
            if (share) {
                find_share(s, c, kept_c, k ? (float)((1.0 - p) * (double)all_w * (1.0 / kOne)) : tail);
                before = s.before[0];
                reach = s.before[1];
                if (mp > 0.0) {
                    // A token of weight min_p lies within a bin of `least`: where the share's cut is deeper than that, it
                    // changes nothing, and where it is higher, min-p does not.
                    const int least = (int)(-64.0f * log2f((float)mp));
                    if (min(s.bin[0], s.bin[1]) > least + 1) break;
                    if (max(s.bin[0], s.bin[1]) < least - 1) mp = 0.0;
                }
            } else {
                if (find_count(s, c, k) < k) {
                    // fewer than k: no cut by the count
                    if (by_p) {
                        u64 w = 0;
                        r.each([&](int, float x) { w += r.weight(x); });
                        w = block_sum(s, w);
                        if (tid == 0) s.cta_weight = w;
                        cl.sync();
                        all_w = over_cluster(cl, s, &Shared::cta_weight);
                        cl.sync();
                    }
                    continue;
                }
                before = s.before[0];
                reach = before + s.in_bin;
            }
            const bool whole = reach <= kThreads;  // all that can be kept is a list that can be sorted
            const int b0 = whole ? 0 : min(s.bin[0], s.bin[1]), b1 = s.bin[1];
            const bool listable = whole || reach - before <= (unsigned)(share ? kList : kThreads);
            Shared *first = cl.map_shared_rank(&s, 0);
            // The tokens of those bins: into the list, or their least and largest key; for a share also the weight of
            // those above them and (after a cut by the count it is known, and the tokens below that are not in it)
            // of all.  The weights go by the threads' segments, for the choice to use.
            const bool weigh = share && !(k && whole);
            u64 above = 0, total = 0;
            unsigned klo = 0xffffffffu, khi = 0;
#pragma unroll 1
            for (int i = weigh ? i0 : tid; i < (weigh ? i1 : n); i += weigh ? 1 : kThreads) {
                const float x = r.get(i);
                int b;
                if (weigh) {
                    const u64 w = r.weight(x, &b);
                    total += w;
                    above += b < b0 ? w : 0;
                } else {
                    b = r.bin(x);
                }
                if (b < b0 || b > b1 || x == -INFINITY) continue;
                const unsigned key = key_of(x);
                klo = min(klo, key);
                khi = max(khi, key);
                if (listable) {
                    const unsigned at = atomicAdd(&s.own_listed, 1u);
                    if (at < kList) s.own[at] = (u64)key << 32 | (0xffffffffu - (unsigned)(base + i));
                }
            }
            if (weigh) {
                above_mine = above;
                above = block_sum(s, above);
                total = block_sum(s, total);
                if (tid == 0) {
                    s.cta_weight = above;
                    s.cta_total = total;
                }
            }
            if (listable) {
                __syncthreads();
                // a CTA's tokens go to the list together: one remote addition, not one a token
                const unsigned found = min(s.own_listed, (unsigned)kList);
                if (tid == 0) s.own_at = found ? atomicAdd(&first->listed, found) : 0;
                __syncthreads();
                for (unsigned e = tid; e < found; e += kThreads)
                    if (s.own_at + e < kList) first->list[s.own_at + e] = s.own[e];
                cl.sync();
                if (rank == 0) {
                    if (weigh) {
                        above = over_cluster(cl, s, &Shared::cta_weight);
                        if (!k) all_w = over_cluster(cl, s, &Shared::cta_total);
                    }
                    const int m = (int)min(s.listed, (unsigned)kList);
                    if (share && !whole) {
                        cut_of_list(s, r, m, above, p * (double)all_w);
                    } else {
                        const bool mine = tid < m;
                        const u64 e = block_sort(mine ? s.list[tid] : 0, s.list, m);
                        const unsigned key = (unsigned)(e >> 32);
                        const u64 w = mine ? r.weight(of_key(key)) : 0;
                        bool keep = mine;
                        if (whole) {
                            if (k) keep = keep && (unsigned)tid < k;
                            if (by_p) {
                                const Scan<u64> z = block_scan(s, keep ? w : 0ull);
                                keep = keep && (tid == 0 || (double)z.before < p * (double)(share ? all_w : z.all));
                            }
                            if (mp > 0.0) keep = keep && r.at_least(of_key(key), w, mp);
                            // the kept tokens by their index, lowest first
                            const int kept = __syncthreads_count(keep);
                            const u64 f = block_sort(keep ? e << 32 | key : 0, s.list, kept);
                            const u64 fw = tid < kept ? r.weight(of_key((unsigned)f)) : 0;
                            const Scan<u64> z = block_scan(s, fw);
                            const double target = u * (double)z.all;
                            const u64 upto = z.before + fw;
                            const bool last = !((double)z.all > target);  // u of 1 or more, or NaN: the last kept token
                            if (fw && (last ? upto == z.all : (double)upto > target && !((double)z.before > target)))
                                a.token[row] = (int32_t)(0xffffffffu - (unsigned)(f >> 32));
                        } else {
                            keep = keep && before + tid < k;
                            const int kept = __syncthreads_count(keep);
                            // the last kept one and how many equal to it are kept (none: the cut is above the list)
                            if (tid == (kept ? kept - 1 : 0)) s.cut_key = key;
                            __syncthreads();
                            const unsigned ties = __syncthreads_count(keep && key == s.cut_key);
                            const unsigned equal = __syncthreads_count(mine && key == s.cut_key);
                            if (tid == 0) s.cut_ties = ties == equal ? kAll : ties;
                        }
                    }
                }
                cl.sync();
                if (whole) return;
                cut_key = first->cut_key;
                cut_ties = first->cut_ties;
                listed = weigh && cut_ties == kAll && !(mp > 0.0);
            } else {
                // too many tokens next to the cut: finer and finer histograms over the keys lo .. hi of those bins
                klo = __reduce_min_sync(0xffffffffu, klo);
                khi = __reduce_max_sync(0xffffffffu, khi);
                if (lane == 0) {
                    atomicMin(&s.klo, klo);
                    atomicMax(&s.khi, khi);
                }
                cl.sync();
                if (weigh) {
                    above = over_cluster(cl, s, &Shared::cta_weight);
                    if (!k) all_w = over_cluster(cl, s, &Shared::cta_total);
                }
                const double target = share ? p * (double)all_w : 0.0;
                u64 done_w = above;
                unsigned done_c = before;
                unsigned lo = __reduce_min_sync(0xffffffffu, lane < C ? cl.map_shared_rank(&s, lane)->klo : 0xffffffffu);
                unsigned hi = __reduce_max_sync(0xffffffffu, lane < C ? cl.map_shared_rank(&s, lane)->khi : 0u);
                for (;;) {
                    int shift = 0;
                    while (((hi - lo) >> shift) >= (unsigned)kThreads) ++shift;
                    cl.sync();
                    s.count[tid] = 0;
                    s.own[tid] = 0;
                    __syncthreads();
                    r.each([&](int, float x) {
                        const unsigned ky = key_of(x);
                        if (ky < lo || ky > hi) return;
                        const int b = (int)((hi - ky) >> shift);
                        atomicAdd(&s.count[b], 1u);
                        if (share) {
                            const u64 w = r.weight(x);
                            if (w) atomicAdd(&s.own[b], w);
                        }
                    });
                    if (tid == 0) s.bin[0] = -1;
                    cl.sync();
                    unsigned fc = 0;
                    u64 fw = 0;
#pragma unroll 4
                    for (int q = 0; q < C; ++q) {
                        const Shared *o = cl.map_shared_rank(&s, q);
                        fc += o->count[tid];
                        fw += o->own[tid];
                    }
                    const unsigned cb = block_scan(s, fc).before;
                    const u64 wb = block_scan(s, fw).before;
                    const bool here = share ? fc && (double)(done_w + wb) < target && !((double)(done_w + wb + fw) < target)
                                            : done_c + cb < k && done_c + cb + fc >= k;
                    if (here) {
                        s.bin[0] = tid;
                        s.before[0] = cb;
                        s.fine_before = wb;
                    }
                    __syncthreads();
                    const int b = s.bin[0];
                    if (b < 0) {  // (in the first round only, as in cut_of_list) all of these bins' tokens are kept, or none
                        const bool all = share && (double)done_w < target;
                        cut_key = all ? lo : done_c ? hi : key_of(top);  // (p of 0: the first token alone)
                        cut_ties = all ? kAll : done_c ? 0 : 1;
                        break;
                    }
                    done_c += s.before[0];
                    done_w += s.fine_before;
                    const unsigned nhi = hi - ((unsigned)b << shift);
                    const unsigned width = (1u << shift) - 1;
                    lo = nhi - lo < width ? lo : nhi - width;
                    hi = nhi;
                    if (lo == hi) {
                        cut_key = lo;
                        if (share) {
                            // the fewest ties whose weight reaches the target
                            const u64 w1 = r.weight(of_key(cut_key));
                            const double need = w1 ? ceil((target - (double)done_w) / (double)w1) : 1.0;
                            cut_ties = need < 1.0 ? 1u : need < 4294967295.0 ? (unsigned)need : kAll;
                        } else {
                            cut_ties = k - done_c;
                        }
                        break;
                    }
                }
            }
            cl.sync();  // the cut has been read everywhere: the list and the bounds may be used again
            if (listed) break;  // (a share's cut is the last)
            if (tid == 0) {
                s.listed = s.own_listed = 0;
                s.klo = 0xffffffffu;
                s.khi = 0;
            }
            if (!share && by_p) {
                // the weight of the first k, and their counts in the bins
                const float xc = of_key(cut_key);
                const int bc = r.bin(xc);
                u64 w = 0;
                unsigned in = 0;  // of the cut's bin, above the cut (all the ties are kept: with them)
                r.each([&](int, float x) {
                    const unsigned ky = key_of(x);
                    if (ky > cut_key || (ky == cut_key && cut_ties == kAll)) {
                        w += r.weight(x);
                        in += r.bin(x) == bc;
                    }
                });
                const unsigned in_all = block_scan(s, in).all;
                w = block_sum(s, w);
                if (tid == 0) {
                    s.cta_weight = w;
                    s.cta_ties = in_all;
                }
                cl.sync();
                const unsigned extra = cut_ties == kAll ? 0 : cut_ties;
                all_w = over_cluster(cl, s, &Shared::cta_weight) + (u64)extra * r.weight(xc);
                const unsigned kept_in = over_cluster(cl, s, &Shared::cta_ties) + extra;
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int b = kPer * tid + j;
                    kept_c[j] = b < bc ? c[j] : b == bc ? kept_in : 0;
                }
                cl.sync();
            }
        }
    }

    // ---- the choice, in index order
    unsigned ties_before = 0;
    if (cut_ties != kAll) {  // which of the tokens equal to the cut are kept depends on those before them
        unsigned ties = 0;
        for (int i = i0; i < i1; ++i) ties += key_of(r.get(i)) == cut_key;
        const Scan<unsigned> z = block_scan(s, ties);
        ties_before = z.before;
        if (tid == 0) s.cta_ties = z.all;
        cl.sync();
        for (int q = 0; q < rank; ++q) ties_before += cl.map_shared_rank(&s, q)->cta_ties;
    }
    // its weight, 0 if it is not kept; `earlier`: tokens equal to the cut before it
    auto kept_weight = [&](float x, unsigned earlier) -> u64 {
        const unsigned ky = key_of(x);
        const u64 w = r.weight(x);
        const bool in = x != -INFINITY && (ky > cut_key || (ky == cut_key && earlier < cut_ties)) && (!(mp > 0.0) || r.at_least(x, w, mp));
        return in ? w : 0;
    };
    u64 mine = 0;
    unsigned seen = ties_before;
    if (listed) {
        s.list[tid] = 0;
        __syncthreads();
        for (unsigned at = tid; at < s.own_listed; at += kThreads) {
            const u64 e = s.own[at];
            if ((unsigned)(e >> 32) >= cut_key)
                atomicAdd(&s.list[(unsigned)(0xffffffffu - (unsigned)e - base) / (unsigned)seg], r.weight(of_key((unsigned)(e >> 32))));
        }
        __syncthreads();
        mine = above_mine + s.list[tid];
    } else {
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            const float x = r.get(i);
            mine += kept_weight(x, seen);
            seen += key_of(x) == cut_key;
        }
    }
    const Scan<u64> z = block_scan(s, mine);
    if (tid == 0) s.cta_weight = z.all;
    cl.sync();
    const u64 theirs = lane < C ? cl.map_shared_rank(&s, lane)->cta_weight : 0;
    const u64 before = z.before + warp_total(lane < rank ? theirs : 0ull), all_w = warp_total(theirs);
    const double target = u * (double)all_w;
    const bool last = !((double)all_w > target);  // u of 1 or more, or NaN: the last kept token
    const bool here = mine && (last ? before + mine == all_w : (double)(before + mine) > target && !((double)before > target));
    // the thread whose logits hold the token hands them to its warp, a logit a lane
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
        const int from = __ffs(who) - 1;
        u64 run = __shfl_sync(0xffffffffu, before, from);
        seen = __shfl_sync(0xffffffffu, ties_before, from);
        const int e0 = __shfl_sync(0xffffffffu, i0, from), e1 = __shfl_sync(0xffffffffu, i1, from);
        for (int e = e0; e < e1; e += 32) {
            const int i = e + lane;
            const float x = i < e1 ? r.get(i) : -INFINITY;
            const unsigned equal = __ballot_sync(0xffffffffu, i < e1 && key_of(x) == cut_key);
            const u64 w = i < e1 ? kept_weight(x, seen + __popc(equal & ((1u << lane) - 1))) : 0;
            const u64 upto = run + warp_incl(w, lane);
            const unsigned hit = __ballot_sync(0xffffffffu, w && (last ? upto == all_w : (double)upto > target));
            if (hit) {
                if (lane == __ffs(hit) - 1) a.token[row] = (int32_t)(base + i);
                break;
            }
            run = __shfl_sync(0xffffffffu, upto, 31);
            seen += __popc(equal);
        }
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
}

// Rows side by side (a GEMV's [V][B]) to rows one after another: 64 x 16 tiles through shared memory.
__global__ void __launch_bounds__(256) rows_kernel(const float *x, float *y, int64_t rows, int64_t V, int64_t rs, int64_t es)
{
    __shared__ float tile[16][65];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t v0 = (int64_t)blockIdx.x * 64, r0 = (int64_t)blockIdx.y * 16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int e = threadIdx.x + 256 * j;
        const int64_t r = r0 + (e & 15), v = v0 + (e >> 4);
        if (r < rows && v < V) tile[e & 15][e >> 4] = x[r * rs + v * es];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int e = threadIdx.x + 256 * j;
        const int64_t r = r0 + (e >> 6), v = v0 + (e & 63);
        if (r < rows && v < V) y[r * V + v] = tile[e >> 6][e & 63];
    }
}

// Clusters of 1 to 16 CTAs that the current device holds side by side (a CTA takes a multiprocessor; the
// multiprocessors of a cluster lie in one of the chip's partitions, so fewer than their number suggests), and its
// shared memory for a block.
struct Card {
    int optin;
    int side_by_side[kMostCtas + 1];  // 0: a size that it does not take
};

int look_at_card(Card *out)
{
    static std::atomic<int> known[64];
    static Card cards[64];
    static std::mutex lock;
    int dev = 0;
    if (cuda_status(cudaGetDevice(&dev)) != QG_OK || dev >= 64) return QG_ERR_CUDA;
    if (!known[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> hold(lock);
        Card c = {};
        if (cuda_status(cudaDeviceGetAttribute(&c.optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != QG_OK) return QG_ERR_CUDA;
        for (auto kernel : {sample_kernel<true>, sample_kernel<false>})
            if (cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, c.optin)) != QG_OK ||
                cuda_status(cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != QG_OK)
                return QG_ERR_CUDA;
        for (int C = 1; C <= kMostCtas; ++C) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(C);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = c.optin;
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = C;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            if (cuda_status(cudaOccupancyMaxActiveClusters(&c.side_by_side[C], sample_kernel<true>, &cfg)) != QG_OK) c.side_by_side[C] = 0;
        }
        if (c.side_by_side[1] < 1) return QG_ERR_CUDA;
        cards[dev] = c;
        known[dev].store(1, std::memory_order_release);
    }
    *out = cards[dev];
    return QG_OK;
}

// CTAs of a row's cluster.  A row takes about as long as 41000 logits of a CTA, 700 for each CTA of the cluster and then
// a CTA's share (of a share that does not fit the shared memory 1.7 times as long; 1000 logits take 0.5 us); rows that
// find no room side by side wait.  Shares are not cut below 8192 logits.  Top-p of one row of 151936 took 142, 85, 41,
// 34, 31 and 32 us with 1, 2, 4, 6, 8 and 16 CTAs (the first two not resident); of 8 rows 41, 45, 33 and 62 with 4, 6, 8
// and 16; of 16 rows 42, 36, 62 and 93; of 64 rows of 50257 63, 34, 54 and 122 with 1, 2, 4 and 8; of 4 rows of 32000 35,
// 28, 24, 23 and 27 with 1, 2, 4, 8 and 16.
int cluster_of(const Card &card, int64_t rows, int64_t V)
{
    int best = 1;
    double least = 0;
    for (int C = 1; C <= kMostCtas && (C == 1 || V > (int64_t)(C - 1) * 8192); ++C) {
        const int64_t side = card.side_by_side[C], per = (V + C - 1) / C;
        if (side < 1) continue;
        const bool resident = per <= (card.optin - (int)sizeof(Shared)) / 4;
        const double cost = (double)((rows + side - 1) / side) * (41000.0 + 700.0 * C + (double)per * (resident ? 1.0 : 1.7));
        if (C == 1 || cost < least) {
            best = C;
            least = cost;
        }
    }
    return best;
}

}  // namespace

extern "C" {

size_t qg_sample_workspace(int64_t rows, int64_t V, int64_t elem_stride)
{
    // rows that do not stand one after another are set out so first: a cluster reads its row alone, and of
    // rows side by side it would fetch a whole sector for each logit
    if (rows < 2 || V < 1 || elem_stride == 1 || rows > kMostRows || V > kMostLogits) return 0;
    return (size_t)rows * (size_t)V * sizeof(float);
}

int qg_sample(const float *logits, int64_t rows, int64_t V, int64_t row_stride, int64_t elem_stride,
              const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
              const float *u, int32_t *token, void *workspace, size_t workspace_bytes, void *stream)
{
    if (rows < 0 || V < 1 || V > kMostLogits || rows > kMostRows) return QG_ERR_SHAPE;
    if (rows == 0) return QG_OK;
    if (!logits || !token || !u) return QG_ERR_NULL;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(temperature) |
                           reinterpret_cast<uintptr_t>(top_k) | reinterpret_cast<uintptr_t>(top_p) |
                           reinterpret_cast<uintptr_t>(min_p) | reinterpret_cast<uintptr_t>(u) |
                           reinterpret_cast<uintptr_t>(token) | reinterpret_cast<uintptr_t>(workspace);
    if (bits % 4) return QG_ERR_ALIGN;
    const size_t need = qg_sample_workspace(rows, V, elem_stride);
    if (workspace && workspace_bytes < need) return QG_ERR_SCRATCH;
    Card card;
    if (const int rc = look_at_card(&card); rc != QG_OK) return rc;
    SampleArgs a = {};
    a.x = logits;
    a.rs = row_stride;
    a.es = elem_stride;
    if (need && workspace) {
        const int rc = launch_pdl(rows_kernel, dim3((unsigned)((V + 63) / 64), (unsigned)((rows + 15) / 16)), dim3(256), 0, stream,
                                  logits, static_cast<float *>(workspace), rows, V, row_stride, elem_stride);
        if (rc != QG_OK) return rc;
        a.x = static_cast<const float *>(workspace);
        a.rs = V;
        a.es = 1;
    }
    const int C = cluster_of(card, rows, V);
    a.V = V;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.token = token;
    a.per = (V + C - 1) / C;
    const bool resident = a.per <= (card.optin - (int)sizeof(Shared)) / 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared) + (resident ? (size_t)a.per * 4 : 0);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&cfg, resident ? sample_kernel<true> : sample_kernel<false>, a));
}

}  // extern "C"
