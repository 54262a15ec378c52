// qg_sample.cu -- one token a row from its logits and a given random number (qg_sample).  Declaration
// and contract: include/qg.h.
//
// With z = logit / temperature, in descending order (equal logits: the lower index first):
//   top-k keeps the first k; top-p keeps, of those, the shortest prefix whose share of their weight
//   w = exp(z - z_max) reaches p; min-p drops weights below min_p; the token is the first in the
//   vocabulary's order whose running weight exceeds u times the kept weight.
//
// One thread-block cluster takes a row and keeps it in its shared memory (up to eight CTAs, so 248,320
// logits are read once from HBM), so the passes over the row run on chip.  The row is never sorted:
//   1. the largest logit;
//   2. a histogram (counts, and weights where they are needed) over bins linear in the logit, which
//      spread the bulk of a vocabulary over many bins; all CTAs add up the cluster's histograms over
//      distributed shared memory and find the bin in which the k-th token or the p-th share falls;
//   3. if the tokens down to that bin are few (kList), they are gathered in one CTA, where each
//      thread compares one token with all others and so knows its rank, the weight before it and its
//      running weight in index order: filters and choice follow at once;
//   4. otherwise the cut (a logit and how many of the tokens equal to it stay) is found in that bin
//      alone, by lists or finer histograms, and a pass in index order finds the token.
//
// Weights are whole multiples of 2^-44 of the largest (64-bit integers from 64-bit exponentials): their
// sums do not depend on the order of the additions, atomic ones among them, so a call gives the same
// token every time; and with errors of 2^-45 a weight the choice is that of the exact formula but for
// u within about 1e-9 of a border.
#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "qg_kv4.cuh"

namespace {

using namespace qg;
namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kList = 1024;
constexpr int kMaxCluster = 8;
constexpr double kWeightOne = 17592186044416.0;  // 2^44
typedef unsigned long long u64;

struct SampleArgs {
    const float *x;
    int64_t V, rs, es;  // strides in elements
    const float *temperature, *top_p, *min_p, *u;
    const int32_t *top_k;
    int32_t *token;
    int64_t per;   // logits of a CTA
    int resident;  // the CTA's logits stand in shared memory
};

struct Shared {
    u64 weight[kBins];
    unsigned count[kBins];
    u64 lw[kList];
    float lx[kList];
    int64_t li[kList];
    // exchanged over the cluster
    float top;
    int64_t best;
    unsigned listed;
    u64 cta_weight;
    unsigned cta_ties;
    unsigned klo, khi;
    // results of the CTA's own searches
    u64 scan_w[32];
    unsigned scan_c[32];
    int bin;
    unsigned before_c, in_bin;
    u64 before_w, total_w;
    unsigned cut_key, cut_ties;
    double cut_u;
    int64_t pick;
};

// logits in an order-preserving integer form; -inf (and NaN) lowest
__device__ __forceinline__ unsigned key_of(float x)
{
    const unsigned b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float clean(float x)
{
    x += 0.0f;                          // -0 and +0 are equal
    return x != x ? -INFINITY : x;      // NaN is never chosen
}

struct Row {
    const SampleArgs &a;
    const float *slice;
    int64_t row, base;
    int n;
    double inv_t, zmax;
    float xmax;

    __device__ __forceinline__ float get(int i) const
    {
        return a.resident ? slice[i] : clean(a.x[row * a.rs + (base + i) * a.es]);
    }
    __device__ __forceinline__ double ratio(float x) const
    {
        if (x == xmax) return 1.0;
        return exp((double)x * inv_t - zmax);  // 0 for -inf, and below +inf
    }
    __device__ __forceinline__ u64 weight(float x) const { return __double2ull_rn(ratio(x) * kWeightOne); }
};

template <typename T> __device__ __forceinline__ T warp_incl(T v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
    }
    return v;
}

// Exclusive prefix over the block's threads of (c, w), and the totals.
__device__ __forceinline__ void block_scan(Shared &s, unsigned c, u64 w, unsigned *c_before, u64 *w_before, unsigned *c_all, u64 *w_all)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned ci = warp_incl(c, lane);
    const u64 wi = warp_incl(w, lane);
    __syncthreads();
    if (lane == 31) {
        s.scan_c[warp] = ci;
        s.scan_w[warp] = wi;
    }
    __syncthreads();
    if (warp == 0) {
        const unsigned cw = warp_incl(s.scan_c[lane], lane);
        const u64 ww = warp_incl(s.scan_w[lane], lane);
        s.scan_c[lane] = cw;
        s.scan_w[lane] = ww;
    }
    __syncthreads();
    *c_before = ci - c + (warp ? s.scan_c[warp - 1] : 0);
    *w_before = wi - w + (warp ? s.scan_w[warp - 1] : 0);
    *c_all = s.scan_c[31];
    *w_all = s.scan_w[31];
}

// Adds up the cluster's histograms and finds the bin where the cumulative count reaches want_c (by
// weight: where the cumulative weight first reaches want_w).  Every CTA finds the same.
__device__ void find_bin(cg::cluster_group &cl, Shared &s, bool by_weight, unsigned want_c, double share, u64 want_w)
{
    cl.sync();  // all histograms are whole
    constexpr int PB = kBins / kThreads;
    unsigned c[PB];
    u64 w[PB];
    unsigned cs = 0;
    u64 ws = 0;
#pragma unroll
    for (int b = 0; b < PB; ++b) {
        c[b] = 0;
        w[b] = 0;
        for (unsigned r = 0; r < cl.num_blocks(); ++r) {
            const Shared *o = cl.map_shared_rank(&s, r);
            c[b] += o->count[threadIdx.x * PB + b];
            w[b] += o->weight[threadIdx.x * PB + b];
        }
        cs += c[b];
        ws += w[b];
    }
    unsigned cb, ca;
    u64 wb, wa;
    block_scan(s, cs, ws, &cb, &wb, &ca, &wa);
    // `share` >= 0: the wanted weight is that share of all
    const double target = share >= 0.0 ? share * (double)wa : (double)want_w;
    if (threadIdx.x == 0) s.bin = -1;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < PB; ++b) {
        const bool here = by_weight ? ((double)wb < target && (double)(wb + w[b]) >= target)
                                    : (cb < want_c && cb + c[b] >= want_c);
        if (here) {
            s.bin = threadIdx.x * PB + b;
            s.before_c = cb;
            s.before_w = wb;
            s.in_bin = c[b];
        }
        cb += c[b];
        wb += w[b];
    }
    if (threadIdx.x == 0) s.total_w = wa;
    cl.sync();  // the histograms may be cleared
}

__device__ __forceinline__ void clear_hist(Shared &s)
{
    for (int b = threadIdx.x; b < kBins; b += kThreads) {
        s.count[b] = 0;
        s.weight[b] = 0;
    }
}

// Bins of the first histogram: linear in the logit, 64 a unit of z.
struct LinearBins {
    float xmax, scale;
    __device__ __forceinline__ int operator()(float x) const
    {
        if (x == xmax) return 0;
        const float d = (xmax - x) * scale;  // monotone in x
        return d < (float)(kBins - 1) ? (int)d : kBins - 1;
    }
};

__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs a)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    Shared &s = *reinterpret_cast<Shared *>(dyn);
    float *slice = reinterpret_cast<float *>(dyn + sizeof(Shared));
    cg::cluster_group cl = cg::this_cluster();
    const int rank = cl.block_rank(), C = cl.num_blocks();
    const int64_t row = blockIdx.x / C;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();

    const int64_t base = (int64_t)rank * a.per;
    const int n = (int)(base < a.V ? (a.V - base < a.per ? a.V - base : a.per) : 0);
    Row r{a, slice, row, base, n, 0.0, 0.0, 0.0f};

    // ---- the row into shared memory, and its largest logit
    if (threadIdx.x == 0) {
        s.top = -INFINITY;
        s.best = INT64_MAX;
        s.listed = 0;
    }
    clear_hist(s);
    float top = -INFINITY;
    {
        const float *x = a.x + row * a.rs + base * a.es;
        if (a.resident) {
            const int full = n / (4 * kThreads) * (4 * kThreads);
            for (int i = threadIdx.x; i < full; i += 4 * kThreads) {
                float v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = x[(i + (int64_t)j * kThreads) * a.es];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float y = clean(v[j]);
                    slice[i + j * kThreads] = y;
                    top = fmaxf(top, y);
                }
            }
            for (int i = full + threadIdx.x; i < n; i += kThreads) {
                const float y = clean(x[i * a.es]);
                slice[i] = y;
                top = fmaxf(top, y);
            }
        } else {
            for (int i = threadIdx.x; i < n; i += kThreads) top = fmaxf(top, clean(x[i * a.es]));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    __shared__ float warp_top[32];
    if (lane == 0) warp_top[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 32; ++w) top = fmaxf(top, warp_top[w]);
        s.top = top;
    }
    cl.sync();
    top = -INFINITY;
    for (int c = 0; c < C; ++c) top = fmaxf(top, cl.map_shared_rank(&s, c)->top);
    r.xmax = top;
    if (top == -INFINITY) {  // nothing to choose from
        if (rank == 0 && threadIdx.x == 0) a.token[row] = -1;
        cl.sync();
        return;
    }
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = !(t > 0.0f);
    const int64_t k_arg = a.top_k ? a.top_k[row] : 0;
    const unsigned k = k_arg > 0 && k_arg < a.V ? (unsigned)k_arg : 0;  // 0: all
    const double p_arg = a.top_p ? (double)a.top_p[row] : 1.0;
    const bool by_p = p_arg < 1.0;
    const double p = p_arg > 0.0 ? p_arg : 0.0;
    const double mp = a.min_p ? (double)a.min_p[row] : 0.0;
    const double u = a.u ? (double)a.u[row] : 0.0;

    if (greedy || k == 1) {
        // the lowest index of the largest logit
        int64_t best = INT64_MAX;
        for (int i = threadIdx.x; i < n && best == INT64_MAX; i += kThreads)
            if (r.get(i) == top) best = base + i;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int64_t b = __shfl_xor_sync(0xffffffffu, best, o);
            best = b < best ? b : best;
        }
        if (lane == 0 && best != INT64_MAX) atomicMin(reinterpret_cast<long long *>(&s.best), (long long)best);
        cl.sync();
        if (rank == 0 && threadIdx.x == 0) {
            for (int c = 0; c < C; ++c) {
                const int64_t b = cl.map_shared_rank(&s, c)->best;
                best = b < best ? b : best;
            }
            a.token[row] = (int32_t)best;
        }
        cl.sync();
        return;
    }
    r.inv_t = 1.0 / (double)t;
    r.zmax = (double)top * r.inv_t;

    unsigned cut_key = 0, cut_ties = 0xffffffffu;  // kept: above cut_key, and the first cut_ties equal to it
    if (k || by_p) {
        // ---- histogram linear in the logit
        const bool weigh = by_p;
        const LinearBins bins{top, 64.0f / t};
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const float x = r.get(i);
            if (x == -INFINITY) continue;
            const int b = bins(x);
            atomicAdd(&s.count[b], 1u);
            if (weigh) {
                const u64 w = r.weight(x);
                if (w) atomicAdd(&s.weight[b], w);
            }
        }
        // the deepest bin that can hold a kept token: of the k-th, or of the p-th share of everything
        // (a share of the first k's weight is reached no later)
        if (k)
            find_bin(cl, s, false, k, -1.0, 0);
        else
            find_bin(cl, s, true, 0, p, 0);
        // fewer than k tokens, or p = 0 (the first token alone): all of a row, or its first bin
        const bool all = s.bin < 0 && k;
        if (s.bin < 0 && !k && threadIdx.x == 0) {
            s.bin = 0;
            s.before_c = 0;
            s.before_w = 0;
            unsigned c0 = 0;
            for (int c = 0; c < C; ++c) c0 += cl.map_shared_rank(&s, c)->count[0];
            s.in_bin = c0;
        }
        cl.sync();
        const int bin = s.bin;
        const unsigned reach = s.before_c + s.in_bin;
        if (!all && reach <= kList) {
            // ---- everything that can be kept, in one list
            Shared *first = cl.map_shared_rank(&s, 0);
            for (int i = threadIdx.x; i < n; i += kThreads) {
                const float x = r.get(i);
                if (x == -INFINITY || bins(x) > bin) continue;
                const unsigned at = atomicAdd(&first->listed, 1u);
                if (at < kList) {
                    first->lx[at] = x;
                    first->li[at] = base + i;
                    first->lw[at] = r.weight(x);
                }
            }
            cl.sync();
            if (rank == 0) {
                const int m = (int)(s.listed < kList ? s.listed : kList);
                const int i = threadIdx.x;
                const bool mine = i < m;
                const float xi = mine ? s.lx[i] : 0.0f;
                const int64_t ii = mine ? s.li[i] : 0;
                const u64 wi = mine ? s.lw[i] : 0;
                unsigned rk = 0;
                u64 before = 0;
                if (mine)
                    for (int j = 0; j < m; ++j) {
                        const float xj = s.lx[j];
                        if (xj > xi || (xj == xi && s.li[j] < ii)) {
                            ++rk;
                            before += s.lw[j];
                        }
                    }
                bool keep = mine && (k == 0 || rk < k);
                unsigned cb, ca;
                u64 wb, wa;
                if (by_p) {
                    u64 total = s.total_w;
                    if (k) {
                        block_scan(s, 0, keep ? wi : 0, &cb, &wb, &ca, &wa);
                        total = wa;
                    }
                    keep = keep && (rk == 0 || (double)before < p * (double)total);
                }
                if (mp > 0.0) keep = keep && (rk == 0 || r.ratio(xi) >= mp);
                const u64 kw = keep ? wi : 0;
                block_scan(s, 0, kw, &cb, &wb, &ca, &wa);
                if (mine) s.lw[i] = kw;
                if (threadIdx.x == 0) s.best = -1;
                __syncthreads();
                u64 upto = 0;  // running weight in index order, this token included
                if (kw) {
                    for (int j = 0; j < m; ++j)
                        if (s.li[j] <= ii) upto += s.lw[j];
                    const double target = u * (double)wa;
                    // u of 1 or more (or NaN) takes the last kept token
                    if (((double)upto > target && !((double)(upto - kw) > target)) || (upto == wa && !((double)wa > target)))
                        a.token[row] = (int32_t)ii;
                }
            }
            cl.sync();
            return;
        }
        // ---- a cut within the row.  First by count, then by weight among those.
        u64 kept_w = s.total_w;
        for (int pass = 0; pass < 2; ++pass) {
            const bool by_weight = pass == 1;
            if (by_weight ? !by_p : (k == 0 || all)) continue;
            if (by_weight && k && !all) {
                // the weight of the first k tokens
                u64 w = 0;
                for (int i = threadIdx.x; i < n; i += kThreads) {
                    const float x = r.get(i);
                    if (x != -INFINITY && key_of(x) > cut_key) w += r.weight(x);
                }
                unsigned cb, ca;
                u64 wb, wa;
                block_scan(s, 0, w, &cb, &wb, &ca, &wa);
                if (threadIdx.x == 0) s.cta_weight = wa;
                cl.sync();
                kept_w = 0;
                for (int c = 0; c < C; ++c) kept_w += cl.map_shared_rank(&s, c)->cta_weight;
                const unsigned kb = cut_key & 0x80000000u ? cut_key & 0x7fffffffu : ~cut_key;
                kept_w += (u64)cut_ties * r.weight(__uint_as_float(kb));
                cl.sync();
            }
            const double target = by_weight ? p * (double)kept_w : 0.0;
            // finer and finer histograms over keys lo .. hi, the tokens above hi counted before
            unsigned lo = key_of(-INFINITY) + 1, hi = key_of(top);
            unsigned done_c = 0;
            u64 done_w = 0;
            for (;;) {
                int shift = 0;
                while (((hi - lo) >> shift) >= (unsigned)kBins) ++shift;
                clear_hist(s);
                __syncthreads();
                for (int i = threadIdx.x; i < n; i += kThreads) {
                    const unsigned ky = key_of(r.get(i));
                    if (ky < lo || ky > hi) continue;
                    const int b = (int)((hi - ky) >> shift);
                    atomicAdd(&s.count[b], 1u);
                    if (by_weight) {
                        const u64 w = r.weight(r.get(i));
                        if (w) atomicAdd(&s.weight[b], w);
                    }
                }
                const u64 want_w = target > (double)done_w ? (u64)ceil(target - (double)done_w) : 0;
                find_bin(cl, s, by_weight, k - done_c, -1.0, want_w);
                const int b = s.bin;
                if (b < 0) {
                    // no weight is wanted: the first token alone (or rounding at the last): the largest key
                    cut_key = want_w == 0 ? key_of(top) : lo;
                    cut_ties = want_w == 0 ? 1 : 0xffffffffu;
                    break;
                }
                done_c += s.before_c;
                done_w += s.before_w;
                const unsigned nhi = hi - ((unsigned)b << shift);
                const unsigned width = (1u << shift) - 1;
                const unsigned nlo = nhi - lo < width ? lo : nhi - width;
                hi = nhi;
                lo = nlo;
                __syncthreads();
                if (lo == hi) {
                    cut_key = lo;
                    if (by_weight) {
                        const unsigned kb = cut_key & 0x80000000u ? cut_key & 0x7fffffffu : ~cut_key;
                        const u64 w1 = r.weight(__uint_as_float(kb));
                        // the fewest ties whose weight reaches the target
                        u64 m = w1 ? (u64)ceil((target - (double)done_w) / (double)w1) : 1;
                        if (m < 1) m = 1;
                        cut_ties = (unsigned)(m < 0xffffffffu ? m : 0xffffffffu);
                    } else {
                        cut_ties = k - done_c;
                    }
                    break;
                }
            }
        }
    }

    // ---- the choice, in index order: each thread takes consecutive logits (an odd number of them, so
    // that the threads' reads fall in different banks)
    const int seg = ((n + kThreads - 1) / kThreads) | 1;
    const int i0 = min(n, (int)threadIdx.x * seg), i1 = min(n, i0 + seg);
    unsigned ties = 0;
    for (int i = i0; i < i1; ++i) ties += key_of(r.get(i)) == cut_key;
    unsigned ties_before, ca;
    u64 wb, wa;
    block_scan(s, ties, 0, &ties_before, &wb, &ca, &wa);
    if (threadIdx.x == 0) s.cta_ties = ca;
    cl.sync();
    for (int c = 0; c < rank; ++c) ties_before += cl.map_shared_rank(&s, c)->cta_ties;
    auto kept_weight = [&](float x, unsigned &seen) -> u64 {
        const unsigned ky = key_of(x);
        if (x == -INFINITY || ky < cut_key) return 0;
        if (ky == cut_key && seen++ >= cut_ties) return 0;
        const double q = r.ratio(x);
        if (mp > 0.0 && q < mp && x != top) return 0;
        return __double2ull_rn(q * kWeightOne);
    };
    u64 mine = 0;
    unsigned seen = ties_before;
    for (int i = i0; i < i1; ++i) mine += kept_weight(r.get(i), seen);
    unsigned cb;
    block_scan(s, 0, mine, &cb, &wb, &ca, &wa);
    if (threadIdx.x == 0) s.cta_weight = wa;
    cl.sync();
    u64 before = wb, all_w = 0;
    for (int c = 0; c < C; ++c) {
        const u64 w = cl.map_shared_rank(&s, c)->cta_weight;
        if (c < rank) before += w;
        all_w += w;
    }
    const double target = u * (double)all_w;
    const bool last = !((double)all_w > target);  // u of 1 or more, or NaN: the last kept token
    const bool here = last ? mine && before + mine == all_w
                           : (double)(before + mine) > target && !((double)before > target);
    if (mine && here) {
        u64 run = before;
        seen = ties_before;
        for (int i = i0; i < i1; ++i) {
            const u64 w = kept_weight(r.get(i), seen);
            run += w;
            if (w && (last ? run == all_w : (double)run > target)) {
                a.token[row] = (int32_t)(base + i);
                break;
            }
        }
    }
    cl.sync();  // no CTA leaves while another reads its shared memory
}

}  // namespace

extern "C" int qg_sample(const float *logits, int64_t rows, int64_t V, int64_t row_stride, int64_t elem_stride,
                         const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                         const float *u, int32_t *token, void *stream)
{
    if (rows < 0 || V < 1 || V > 0x7fffffff || rows > 0x7fffffff / kMaxCluster) return QG_ERR_SHAPE;
    if (rows == 0) return QG_OK;
    if (!logits || !token || !u) return QG_ERR_NULL;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(temperature) |
                           reinterpret_cast<uintptr_t>(top_k) | reinterpret_cast<uintptr_t>(top_p) |
                           reinterpret_cast<uintptr_t>(min_p) | reinterpret_cast<uintptr_t>(u) | reinterpret_cast<uintptr_t>(token);
    if (bits % 4) return QG_ERR_ALIGN;
    int dev = 0, optin = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess)
        return QG_ERR_CUDA;
    const int64_t room = (optin - (int)sizeof(Shared) - 1024) / 4;  // logits of a CTA
    int C = 1;
    while (C < kMaxCluster && V > (int64_t)C * 8192) C *= 2;
    SampleArgs a = {};
    a.x = logits;
    a.V = V;
    a.rs = row_stride;
    a.es = elem_stride;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.token = token;
    a.per = (V + C - 1) / C;
    a.resident = a.per <= room;
    const size_t smem = sizeof(Shared) + (a.resident ? (size_t)a.per * 4 : 0);
    static std::atomic<uint64_t> raised{0};
    if (dev >= 64 || !(raised.load() >> dev & 1)) {
        if (cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin - 1024) != cudaSuccess)
            return QG_ERR_CUDA;
        if (dev < 64) raised.fetch_or(uint64_t(1) << dev);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, sample_kernel, a) == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}
