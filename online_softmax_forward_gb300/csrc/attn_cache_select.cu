// attn_cache_select.cu -- which pages of a sequence each query attends to.
//
// For query row i, kv head h (its group's G query heads) and page p:
//     score(p) = k_scale[p] * max_g sum_c max(q_gc * lo_pc, q_gc * hi_pc),
// lo and hi being the smallest and largest key code of each channel of the
// page: an upper bound of every q . k in it, from 2 d bytes a page instead of
// page * d.  The page of the query's last visible key is always taken, then
// the highest scores, ties to the lowest page.
//
// With q split into its positive and negative part the sum is one product of
// length 2 d, [q+ q-] . [hi lo]: eight heads and eight pages at a time on
// mma.m16n8k16, in the fp16 form of attn_cache_fwd.cu (a power of two per row of
// q, codes exact).  A cluster of CTAs shares the pages of one (sequence, kv
// head, query) and writes its scores into the first CTA's shared memory, which
// finds the cut by a histogram of 1024 bins, then among the pages of the cut's bin,
// and writes the list.
//
// The fp32 scores carry a bound on their error.  A page whose score is further
// from the cut than that is decided by it; the few others are summed again in
// fp64, where the products of a 16-bit q and an 8-bit code (at most 19 bits) add
// up exactly unless they span more than 2^27, so the choice does not depend on
// the order of a sum.  (fp64 for every page would cost more than the reading:
// this GPU has 1/64 the fp64 rate.)  Pages marked by a NaN scale score infinity and do not
// widen the bound.  More than 256 pages near the cut (equal keys, a q that is not finite) are
// all summed in fp64 and cut by a radix search: 1.6 ms for 4095 pages that tie, 30 us for 4096
// pages without such ties.
//
// Bound: by waits.  With the attention over the choice, 32 of 512 pages for 64 units
// take 26 us and 96 of 4096 for 16 units 34 us, 13 and 22 us of it here, where the
// bounds alone would be read in 1 to 3 us: lengths, table, bounds, scores, histogram
// and list follow one another.  Three kernels in its place (scores, cut, list) took 50
// and 75 us for the pair, a bisection in place of the histogram 49.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_internal.h"
#include "cache_codec.cuh"
#include "cache_index.h"
#include "cache_mma.cuh"

namespace attn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
constexpr int kGroups = 2;  // groups of eight pages a warp loads at once

struct SelectArgs {
    const void *q;  // [B][Hkv * G][Sq][d]
    const uint8_t *bounds;
    const float *k_scale;
    const int32_t *table, *lens, *counts;
    int32_t *pages;  // [B][Hkv][Sq][n]
    double *exact;   // [B][Hkv][Sq][max_pages]: fp64 scores of the pages near the cut
    int B, Hkv, G, Sq, page, n_pages, max_pages, n, causal, cluster, cluster_shift;
    FastDiv by_queries, by_heads;
    int *status;
};

// fp32 value as an integer of the same order.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
}

// Score of a page whose scale is NaN, above all others whatever q is: it is attended to, so that
// the NaN shows.  ordered(infinity).
constexpr uint32_t kMarked = 0xff800000u;
// The same order for doubles.
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);  // -0 as 0
    return u >> 63 ? ~u : u | (uint64_t)1 << 63;
}

// `local` (a shared memory address) in the cluster's first CTA.
__device__ __forceinline__ uint32_t in_first_cta(uint32_t local) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(local));
    return r;
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sum of the threads' numbers before this one's; `warps` is not in use.
__device__ __forceinline__ int block_scan(int x, int *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warps[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) incl += w < warp ? warps[w] : 0;
    return incl - x;
}

// Exact score of a page, in fp64: eight lanes per head, four heads at a time.
template <int D, int FMT, int DT>
__device__ double exact_score(const SelectArgs &a, int b, int hk, int i, int phys) {
    const int lane = threadIdx.x & 31, sub = lane >> 3, c0 = (lane & 7) * (D / 8);
    double best = -INFINITY;
    if (phys < 0 || phys >= a.n_pages) return best;
    const int64_t ph = (int64_t)phys * a.Hkv + hk;
    const uint8_t *lo = a.bounds + (size_t)ph * 2 * D + c0, *hi = lo + D;
#pragma unroll 1
    for (int h0 = 0; h0 < a.G; h0 += 4) {
        const int h = min(h0 + sub, a.G - 1);  // a head twice changes no maximum
        const size_t qi = (((size_t)b * a.Hkv * a.G + hk * a.G + h) * a.Sq + i) * D + c0;
        const bool there = in_bounds(qi + D / 8 <= (size_t)a.B * a.Hkv * a.G * a.Sq * D, a.status);
        double x[4] = {};
#pragma unroll
        for (int c = 0; c < D / 8; c += 8) {
            float q8[8], l8[8], h8[8];
            codec::load8<DT>(a.q, there ? qi + c : 0, q8);
            const uint2 lw = *reinterpret_cast<const uint2 *>(lo + c);
            const uint2 hw = *reinterpret_cast<const uint2 *>(hi + c);
            codec::decode4<FMT>(lw.x, l8); codec::decode4<FMT>(lw.y, l8 + 4);
            codec::decode4<FMT>(hw.x, h8); codec::decode4<FMT>(hw.y, h8 + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e & 3] = fma((double)q8[e], (double)(q8[e] < 0.f ? l8[e] : h8[e]), x[e & 3]);
        }
        double y = (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        best = (y > best || y != y) ? y : best;
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        const double y = __shfl_xor_sync(0xffffffffu, best, o);
        best = (y > best || y != y) ? y : best;
    }
    best *= a.k_scale[ph];
    return best != best ? INFINITY : best;  // a NaN is attended to, so that it shows
}

// One cluster per (b, hk, i).  Dynamic shared memory: scores [max_pages], then
// the list of pages near the cut [max_pages].
template <int D, int FMT, int DT>
__global__ void __launch_bounds__(kThreads, 2) cache_select_kernel(const SelectArgs a) {
    using U = Unpack<FMT>;
    constexpr int QS = D / 16;
    extern __shared__ __align__(16) uint32_t key[];  // ordered scores, later 1 for a page that is in
    __shared__ int wsum[kWarps], s_near, s_in, s_open, s_bin;
    __shared__ int hist[kBins];
    __shared__ double s_exact[kThreads];
    // largest scale (infinity: leave it to fp64), largest and smallest score, by warp and by CTA
    __shared__ uint32_t w_top[3][kWarps], s_top[3][kMaxCluster];
    const int64_t unit = blockIdx.x >> a.cluster_shift;
    const int rank = (int)(blockIdx.x & (a.cluster - 1));
    const uint32_t head_of = (uint32_t)unit / a.by_queries;
    const int i = (int)((uint32_t)unit - head_of * a.Sq);
    const int b = (int)(head_of / a.by_heads);
    const int hk = (int)(head_of - (uint32_t)b * a.Hkv);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, t4 = lane & 3;
    if (!in_bounds(b < a.B && hk < a.Hkv && i < a.Sq, a.status)) return;  // the whole cluster
    const int len0 = a.lens[b], cnt0 = a.counts ? a.counts[b] : a.Sq;
    const int len = clamp_len(len0, a.max_pages, a.page);
    const int cnt = min(max(cnt0, 0), a.Sq);
    if ((len != len0 || cnt != cnt0) && t == 0) atomicOr(a.status, kStatusTable);
    const int vis = (int)(((int64_t)visible_keys(len, cnt, i, a.causal) + a.page - 1) / a.page);
    int32_t *out = a.pages + unit * a.n;
    if (vis <= a.n) {  // every page, for the whole cluster
        if (rank == 0)
            for (int j = t; j < a.n; j += kThreads) out[j] = j < vis ? j : -1;
        return;
    }
    cluster_arrive();  // all CTAs of the cluster run before anyone writes to the first
    const int m = vis - 1;       // pages that compete
    const int k = a.n - 1;       // places for them
    const int32_t *table = a.table + (int64_t)b * a.max_pages;

    // ---- scores of this CTA's pages
    const int slice = ((m + a.cluster - 1) / a.cluster + 7) / 8 * 8;
    const int p0 = rank * slice, p1 = min(m, p0 + slice);
    const uint32_t first_key = in_first_cta((uint32_t)__cvta_generic_to_shared(key));
    for (int h = t; h < kBins; h += kThreads) hist[h] = 0;
    if (t == 0) s_near = s_in = s_open = 0;
    float mass = 0.f, scale_top = 0.f;
    uint32_t high = 0, low = 0xffffffffu;
    bool odd = false;
    for (int g0 = 0; g0 < a.G; g0 += 8) {
        // rows: heads g0 + g.  k steps 0 .. QS - 1 hold the positive parts of channels
        // 4s .. 4s + 3 of the lane's D/4, the others the negative ones
        uint32_t qa[2][QS][4];
        float back, sum = 0.f;
        {
            float f[D / 4];
            if (g0 + g < a.G) {
                const size_t at = (((size_t)b * a.Hkv * a.G + hk * a.G + g0 + g) * a.Sq + i) * D + t4 * (D / 4);
#pragma unroll
                for (int e = 0; e < D / 4; e += 8) codec::load8<DT>(a.q, at + e, f + e);
            } else {
#pragma unroll
                for (int e = 0; e < D / 4; ++e) f[e] = 0.f;
            }
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < D / 4; ++e) {
                amax = fmaxf(amax, fabsf(f[e]));
                sum += fabsf(f[e]);
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float mul;
            row_power(amax, mul, back);
#pragma unroll
            for (int s = 0; s < QS; ++s)
#pragma unroll
                for (int side = 0; side < 2; ++side) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // a NaN stays in both parts
                        const float v = f[4 * s + e];
                        y[e] = ((side ? v > 0.f : v < 0.f) ? 0.f : v) * mul;
                    }
                    uint32_t *x = qa[side][s];
                    x[0] = pack_f16(y[0], y[1]);
                    x[2] = pack_f16(y[2], y[3]);
                    x[1] = x[3] = 0;
                    if constexpr (DT == 0) {  // rows 8 .. 15: what fp16 leaves of an fp32 q
                        const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&x[0]));
                        const float2 w = __half22float2(*reinterpret_cast<const __half2 *>(&x[2]));
                        x[1] = pack_f16(y[0] - u.x, y[1] - u.y);
                        x[3] = pack_f16(y[2] - w.x, y[3] - w.y);
                    }
                }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        mass = (sum > mass || sum != sum) ? sum : mass;
        if (g0 == 0) cluster_wait();
        int next[kGroups];  // pages of the table, asked for a step ahead
        auto look = [&](int base) {
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const int p = base + 8 * j + g;
                next[j] = p < p1 && in_bounds(p < a.max_pages, a.status) ? table[p] : -1;
            }
        };
        constexpr int kStride = kThreads / 4 * kGroups;
        look(p0 + warp * 8 * kGroups);
#pragma unroll 1
        for (int base = p0 + warp * 8 * kGroups; base < p1; base += kStride) {
            uint4 lo[kGroups][D / 64], hi[kGroups][D / 64];
            float sc[kGroups];
            int phys[kGroups];
#pragma unroll
            for (int j = 0; j < kGroups; ++j) phys[j] = next[j];
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const bool in = phys[j] >= 0 && phys[j] < a.n_pages;
                if (base + 8 * j + g < p1 && !in && t4 == 0) atomicOr(a.status, kStatusTable);
                const int64_t ph = in ? (int64_t)phys[j] * a.Hkv + hk : 0;
                const uint4 *src = reinterpret_cast<const uint4 *>(a.bounds + (size_t)ph * 2 * D + t4 * (D / 4));
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    lo[j][c] = in ? src[c] : make_uint4(0, 0, 0, 0);
                    hi[j][c] = in ? src[D / 16 + c] : make_uint4(0, 0, 0, 0);
                }
                sc[j] = in ? a.k_scale[ph] : 0.f;
            }
            look(base + kStride);
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                float s0[4] = {}, s1[4] = {};
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const uint32_t hw[4] = {hi[j][c].x, hi[j][c].y, hi[j][c].z, hi[j][c].w};
                    const uint32_t lw[4] = {lo[j][c].x, lo[j][c].y, lo[j][c].z, lo[j][c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t b0, b1;
                        const uint32_t *x = qa[0][c * 4 + e], *y = qa[1][c * 4 + e];
                        U::quad(hw[e], b0, b1);
                        mma16816(s0, x[0], x[1], x[2], x[3], b0, b1);
                        U::quad(lw[e], b0, b1);
                        mma16816(s1, y[0], y[1], y[2], y[3], b0, b1);
                    }
                }
                scale_top = fmaxf(scale_top, sc[j]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // page 2 t4 + c of the group, head g0 + g
                    float x = (s0[c] + s1[c]) + (s0[2 + c] + s1[2 + c]);
                    x = x != x ? INFINITY : x * back;
                    if (g0 + g >= a.G) x = -INFINITY;
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
                    const int from = (2 * t4 + c) * 4;
                    const float s = __shfl_sync(0xffffffffu, sc[j], from);
                    const int ok = __shfl_sync(0xffffffffu, phys[j], from);
                    const int p = base + 8 * j + 2 * t4 + c;
                    if (g == 0 && p < p1 && in_bounds(p < a.max_pages, a.status)) {
                        x *= s;
                        uint32_t y = s == s ? ordered(x) : kMarked;
                        if (ok < 0 || ok >= a.n_pages) {  // outside the pool: scores lowest
                            y = ordered(-INFINITY);
                        } else if (s == s) {
                            // what is not finite leaves the decision to fp64
                            if (!(fabsf(x) <= 3.402823466e38f)) odd = true;
                            high = max(high, y), low = min(low, y);
                        }
                        const uint32_t at = first_key + p * 4;
                        if (g0 == 0) st_cluster(at, y);
                        else asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(at), "r"(y) : "memory");
                    }
                }
            }
        }
    }
    // the largest scale bounds every page's error
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        scale_top = fmaxf(scale_top, __shfl_xor_sync(0xffffffffu, scale_top, o));
        const float y = __shfl_xor_sync(0xffffffffu, mass, o);
        mass = (y > mass || y != y) ? y : mass;
    }
    odd = __any_sync(0xffffffffu, odd);
    high = __reduce_max_sync(0xffffffffu, high);
    low = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) {
        w_top[0][warp] = odd ? 0x7f800000u : __float_as_uint(scale_top);
        w_top[1][warp] = high;
        w_top[2][warp] = low;
    }
    __syncthreads();
    if (t < 3) {
        uint32_t x = w_top[t][0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) x = t < 2 ? max(x, w_top[t][w]) : min(x, w_top[t][w]);
        st_cluster(in_first_cta((uint32_t)__cvta_generic_to_shared(&s_top[t][rank])), x);
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;

    // ---- the cut, in the first CTA
    uint32_t top = 0;
    for (int r = 0; r < a.cluster; ++r) {
        top = max(top, s_top[0][r]);
        high = max(high, s_top[1][r]);
        low = min(low, s_top[2][r]);
    }
    // |error| of a score: 2 QS <= 16 sums of 16 products and 3 of sums, each off by at
    // most 2^-22 of what sum |q| * code has reached, two fp32 products and q's 22
    // bits: below 2^-18 * sum |q| * largest code * scale, twice that of a difference; where
    // that is next to nothing, scores lose bits below fp32's normal numbers
    constexpr float kTop = FMT == ATTN_CACHE_E4M3 ? 448.f : 128.f;
    float eps = (kTop * mass) * (0x1p-17f * __uint_as_float(top));
    if (eps < 0x1p-100f) eps = 0x1p-100f;
    const float least = unordered(low), per_bin = kBins / (unordered(high) - least);
    // pages whose score may be that of the last place: every one, or those of the
    // n-th score's bin and of the bins within eps of it
    int bin_lo = 0, bin_hi = kBins - 1;
    const bool binned = k > 0 && eps <= 1e37f && per_bin > 0.f && per_bin <= 1e37f;
    // not decreasing with the score
    auto bin_of = [&](float x) { return (int)fminf(fmaxf((x - least) * per_bin, 0.f), kBins - 1.f); };
    if (binned) {
#pragma unroll 4
        for (int p = t; p < m; p += kThreads) atomicAdd(&hist[bin_of(unordered(key[p]))], 1);
        __syncthreads();
        // thread t: bins kBins - 1 - 4 t down
        int c[4], sum = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += c[e] = hist[kBins - 1 - 4 * t - e];
        int above = block_scan(sum, wsum);
        if (above < k && k <= above + sum) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (above < k && k <= above + c[e]) s_bin = kBins - 1 - 4 * t - e;
                above += c[e];
            }
        }
        __syncthreads();
        const int bin = s_bin;
        // one bin for the place in the bin, one for the rounding of (x - least) * per_bin
        const float reach = eps * per_bin + 2.f;
        bin_lo = (int)fmaxf(bin - reach, 0.f);
        bin_hi = (int)fminf(bin + reach, kBins - 1.f);
    }
    static_assert(kBins == 4 * kThreads, "four bins a thread");
    int *near = reinterpret_cast<int *>(key + a.max_pages);
    // q or every scale is 0: all scores are, but a marked page's
    bool equal = top == 0 || (mass == 0.f && top < 0x7f800000u);
    if (equal) {
        int marked = 0;
        for (int p = t; p < m; p += kThreads) marked |= key[p] == kMarked;
        equal = !__syncthreads_or(marked);
    }
    int n_in = 0;
#pragma unroll 4
    for (int p = t; p < m; p += kThreads) {
        const int bin = binned ? bin_of(unordered(key[p])) : bin_lo;
        const bool in = equal ? p < k : bin > bin_hi && k > 0;
        if (!in && !equal && k > 0 && bin >= bin_lo) near[atomicAdd(&s_near, 1)] = p;
        else key[p] = in ? 1 : 0;
        n_in += in;
    }
    n_in = __reduce_add_sync(0xffffffffu, n_in);
    if (lane == 0) atomicAdd(&s_in, n_in);
    __syncthreads();
    const int near_n = s_near, places = k - s_in;  // at least one place if there is a near page
    // Up to kThreads of them are settled among themselves first: `sure` beat a page whatever the
    // errors, `may` might.  More would take too long pair by pair (4095 pages that tie: 12 ms)
    const bool pairs = near_n <= kThreads;
    double *exact = pairs ? s_exact : a.exact + unit * a.max_pages;
    constexpr uint32_t kOpen = 2, kTie = 4;
    if (pairs) {
        int sure = 0, may = 0;
        if (t < near_n) {
            const float x = unordered(key[near[t]]);
            for (int o = 0; o < near_n; ++o) {
                const float y = unordered(key[near[o]]);
                sure += y > x + eps;
                may += !(y < x - eps);  // itself among them
            }
        }
        // 1: in, 0: out.  The scores are still read by others
        const uint32_t fate = may - 1 < places ? 1 : sure >= places ? 0 : kOpen;
        if (t < near_n && fate == kOpen) s_open = 1;
        const int settled = __reduce_add_sync(0xffffffffu, t < near_n && fate == 1);
        __syncthreads();
        if (lane == 0) atomicAdd(&s_in, settled);
        if (t < near_n) key[near[t]] = fate;
        __syncthreads();
    }
    int want = k - s_in;  // places for the open ones
    if (!pairs || s_open) {
#pragma unroll 1
        for (int j = warp; j < near_n; j += kWarps) {
            const int p = near[j];
            if (pairs && key[p] != kOpen) continue;  // the same for the whole warp
            const double x = exact_score<D, FMT, DT>(a, b, hk, i, table[p]);
            if (lane == 0 && in_bounds(j < (pairs ? kThreads : a.max_pages), a.status)) exact[j] = x;
        }
        __syncthreads();
        if (pairs) {
            bool in = false;
            if (t < near_n && key[near[t]] == kOpen) {
                const double x = s_exact[t];
                int place = 0;
                for (int o = 0; o < near_n; ++o)
                    if (key[near[o]] == kOpen) place += s_exact[o] > x || (s_exact[o] == x && near[o] < near[t]);
                in = place < want;
            }
            __syncthreads();
            if (in) key[near[t]] = 1;
        } else {  // the cut, by eight bits of the scores' order at a time
            uint64_t cut = 0, known = 0;
#pragma unroll 1
            for (int shift = 56; shift >= 0; shift -= 8) {
                hist[t] = 0;
                __syncthreads();
                for (int j = t; j < near_n; j += kThreads) {
                    const uint64_t u = ordered(exact[j]);
                    if ((u & known) == cut) atomicAdd(&hist[u >> shift & 255], 1);
                }
                __syncthreads();
                const int c = hist[255 - t], above = block_scan(c, wsum);
                if (above < want && want <= above + c) {
                    s_bin = 255 - t;
                    s_in = above;
                }
                __syncthreads();
                cut |= (uint64_t)s_bin << shift;
                known |= (uint64_t)255 << shift;
                want -= s_in;  // of those that share the bits known so far
            }
            for (int j = t; j < near_n; j += kThreads) {
                const uint64_t u = ordered(exact[j]);
                key[near[j]] = u > cut ? 1 : u < cut ? 0 : kTie;  // the lowest `want` ties are in
            }
        }
    }
    __syncthreads();
    // ascending order; the last visible page closes the list.  A thread takes a stretch of
    // pages, of odd length so that the threads' reads fall into different banks
    const int per = (m + kThreads - 1) / kThreads | 1;
    const int p_end = min(m, (t + 1) * per);
    if (!pairs) {
        int ties = 0;
        for (int p = t * per; p < p_end; ++p) ties += key[p] == kTie;
        ties = block_scan(ties, wsum);
        for (int p = t * per; p < p_end; ++p)
            if (key[p] == kTie) key[p] = ties++ < want;
        __syncthreads();
    }
    int mine = 0;
    for (int p = t * per; p < p_end; ++p) mine += (int)(key[p] & 1);
    int at = block_scan(mine, wsum);
    for (int p = t * per; p < p_end; ++p)
        if (key[p] & 1) {
            if (in_bounds(at < k, a.status)) out[at] = p;
            ++at;
        }
    if (t == 0) out[k] = m;
}

template <int D, int FMT, int DT>
int launch_select_t(SelectArgs &a, int sms, cudaStream_t stream) {
    const int64_t units = (int64_t)a.B * a.Hkv * a.Sq;
    // CTAs per unit: up to eight while they fit the GPU at two an SM and have 64 pages each
    a.cluster_shift = 0;
    while (1 << a.cluster_shift < kMaxCluster && units << (a.cluster_shift + 1) <= 2 * sms &&
           128 << a.cluster_shift <= a.max_pages)
        ++a.cluster_shift;
    a.cluster = 1 << a.cluster_shift;
    a.by_queries = fast_div((uint32_t)a.Sq);
    a.by_heads = fast_div((uint32_t)a.Hkv);
    auto kern = cache_select_kernel<D, FMT, DT>;
    if (!set_smem_limit_once(reinterpret_cast<const void *>(kern), kMaxSelectPages * 8)) return ATTN_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)a.max_pages * 8;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)a.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, (const SelectArgs)a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

template <int D, int FMT>
int launch_select_q(SelectArgs &a, int dtype, int sms, cudaStream_t stream) {
    if (dtype == ATTN_F32) return launch_select_t<D, FMT, 0>(a, sms, stream);
    if (dtype == ATTN_BF16 || dtype == ATTN_BF16_OUT_F32) return launch_select_t<D, FMT, 1>(a, sms, stream);
    return launch_select_t<D, FMT, 2>(a, sms, stream);
}

}  // namespace

int launch_cache_select(const attn_cache &c, const void *q, const int32_t *table, int max_pages,
                        const int32_t *lens, const int32_t *counts, int32_t *pages, int n_select,
                        int B, int H, int Sq, int causal, int dtype, void *workspace,
                        cudaStream_t stream) {
    SelectArgs a = {q, (const uint8_t *)c.k_bounds, c.k_scale, table, lens, counts, pages,
                    reinterpret_cast<double *>(workspace), B, c.H_kv, H / c.H_kv, Sq, c.page,
                    c.n_pages, max_pages, n_select, causal, 1, 0, {}, {}, status_word_device_ptr()};
    if (!a.status) return ATTN_ERR_CUDA;
    const int sms = device_sm_count();
    if (sms <= 0) return ATTN_ERR_CUDA;
    if (c.d == 64)
        return c.format == ATTN_CACHE_E4M3 ? launch_select_q<64, ATTN_CACHE_E4M3>(a, dtype, sms, stream)
                                           : launch_select_q<64, ATTN_CACHE_I8>(a, dtype, sms, stream);
    return c.format == ATTN_CACHE_E4M3 ? launch_select_q<128, ATTN_CACHE_E4M3>(a, dtype, sms, stream)
                                       : launch_select_q<128, ATTN_CACHE_I8>(a, dtype, sms, stream);
}

}  // namespace attn
