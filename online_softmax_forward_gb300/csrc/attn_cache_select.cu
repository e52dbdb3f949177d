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
// finds the cut by bisection and writes the list.
//
// The fp32 scores carry a bound on their error.  A page whose score is further
// from the cut than that is decided by it; the few others are summed again in
// fp64, where the products of a 16-bit q and an 8-bit code (at most 19 bits) add
// up exactly unless they span more than 2^27, so the choice does not depend on
// the order of a sum.  (fp64 for every page would cost more than the reading:
// this GPU has 1/64 the fp64 rate.)
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
constexpr int kGroups = 4;  // groups of eight pages a warp loads at once

struct SelectArgs {
    const void *q;  // [B][Hkv * G][Sq][d]
    const uint8_t *bounds;
    const float *k_scale;
    const int32_t *table, *lens, *counts;
    int32_t *pages;  // [B][Hkv][Sq][n]
    double *exact;   // [B][Hkv][Sq][max_pages]: fp64 scores of the pages near the cut
    int B, Hkv, G, Sq, page, n_pages, max_pages, n, causal, cluster;
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

// Exclusive prefix sum of one flag per thread; *total gets the block's sum.
__device__ __forceinline__ int block_scan(int x, int *warps, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t m = __ballot_sync(0xffffffffu, x != 0);
    __syncthreads();  // `warps` may still be read from the last call
    if (lane == 0) warps[warp] = __popc(m);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warps[w];
        all += warps[w];
    }
    *total = all;
    return before + __popc(m & ((1u << lane) - 1));
}

// One cluster per (b, hk, i).  Dynamic shared memory: keys [max_pages], then
// the list of pages near the cut [max_pages].
template <int D, int FMT, int DT>
__global__ void __launch_bounds__(kThreads) cache_select_kernel(const SelectArgs a) {
    using U = Unpack<FMT>;
    constexpr int QS = D / 16;
    extern __shared__ __align__(16) uint32_t key[];
    __shared__ int wsum[2][kWarps], s_near;
    __shared__ uint32_t wmin[2][kWarps], s_top[kMaxCluster];
    const int64_t unit = blockIdx.x / a.cluster;
    const int rank = (int)(blockIdx.x - unit * a.cluster);
    const int i = (int)(unit % a.Sq);
    const int hk = (int)(unit / a.Sq % a.Hkv);
    const int b = (int)(unit / a.Sq / a.Hkv);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, g = lane >> 2, t4 = lane & 3;
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
    float mass = 0.f, scale_top = 0.f;
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
#pragma unroll 1
        for (int base = p0 + warp * 8 * kGroups; base < p1; base += kThreads / 4 * kGroups) {
            uint4 lo[kGroups][D / 64], hi[kGroups][D / 64];
            float sc[kGroups];
            int phys[kGroups];
#pragma unroll
            for (int j = 0; j < kGroups; ++j) {
                const int p = base + 8 * j + g;
                phys[j] = p < p1 ? table[p] : -1;
            }
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
                        // what is not finite leaves the decision to fp64; a page outside the
                        // pool scores lowest
                        if (!(fabsf(x) <= 3.402823466e38f)) odd = true;
                        if (ok < 0 || ok >= a.n_pages) x = -INFINITY;
                        const uint32_t at = first_key + p * 4;
                        if (g0 == 0) st_cluster(at, ordered(x));
                        else asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(at), "r"(ordered(x)) : "memory");
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
    if (lane == 0) wmin[0][warp] = odd ? 0x7f800000u : __float_as_uint(scale_top);
    __syncthreads();
    if (t == 0) {
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = max(top, wmin[0][w]);
        st_cluster(in_first_cta((uint32_t)__cvta_generic_to_shared(&s_top[rank])), top);
        if (rank == 0) s_near = 0;
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;

    // ---- the cut, in the first CTA
    uint32_t top = 0;
    for (int r = 0; r < a.cluster; ++r) top = max(top, s_top[r]);
    // |error| of a score: 2 QS + 2 <= 18 additions of partial sums, each off by at
    // most 2^-22 of sum |q| * code, two fp32 products and q's 22 bits: below
    // 2^-17 * sum |q| * largest code * scale
    constexpr float kTop = FMT == ATTN_CACHE_E4M3 ? 448.f : 128.f;
    const float eps = 0x1p-17f * kTop * mass * __uint_as_float(top);
    float cut_lo = -INFINITY, cut_hi = INFINITY;  // decided above cut_hi: in; below cut_lo: out
    if (k > 0 && eps <= 3.402823466e38f) {
        // the k-th largest key: the largest v that at least k keys reach, by bisection;
        // done as soon as exactly k do, v then being the smallest of them
        uint32_t v = 0, most = 0xffffffffu;  // at least k keys >= v; fewer than k > most
        int buf = 0;
        while (v < most) {
            const uint32_t mid = v + ((most - v) >> 1) + 1;
            int n = 0;
            uint32_t low = 0xffffffffu;
            for (int p = t; p < m; p += kThreads) {
                const uint32_t x = key[p];
                if (x >= mid) {
                    ++n;
                    low = min(low, x);
                }
            }
            n = __reduce_add_sync(0xffffffffu, n);
            low = __reduce_min_sync(0xffffffffu, low);
            if (lane == 0) {
                wsum[buf][warp] = n;
                wmin[buf][warp] = low;
            }
            __syncthreads();
            n = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                n += wsum[buf][w];
                low = min(low, wmin[buf][w]);
            }
            buf ^= 1;
            if (n >= k) {
                v = low;  // the smallest key that reaches mid
                if (n == k) break;
            } else {
                most = mid - 1;
            }
        }
        const float T = unordered(v);
        cut_lo = T - 2.f * eps;
        cut_hi = T + 2.f * eps;
        // a bound that rounds back to T would decide equal scores
        if (!(cut_lo < T)) cut_lo = T;
        if (!(cut_hi > T)) cut_hi = T;
    }
    // pages above the cut are in, those near it are listed
    int *near = reinterpret_cast<int *>(key + a.max_pages);
    int n_in = 0;
    for (int p = t; p < m; p += kThreads) {
        const float x = unordered(key[p]);
        const bool in = k > 0 && x > cut_hi;
        if (k > 0 && !in && !(x < cut_lo)) near[atomicAdd(&s_near, 1)] = p;
        key[p] = in ? 1 : 0;
        n_in += in;
    }
    n_in = __reduce_add_sync(0xffffffffu, n_in);
    __syncthreads();
    if (lane == 0) wsum[0][warp] = n_in;
    __syncthreads();
    int sure = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sure += wsum[0][w];
    const int near_n = s_near, places = k - sure;
    if (near_n <= places) {
        for (int j = t; j < near_n; j += kThreads) key[near[j]] = 1;
    } else {
        double *exact = a.exact + unit * a.max_pages;
#pragma unroll 1
        for (int j = warp; j < near_n; j += kWarps) {
            const int phys = table[near[j]];
            double best = -INFINITY;
            if (phys >= 0 && phys < a.n_pages) {
                const int64_t ph = (int64_t)phys * a.Hkv + hk;
                const uint8_t *lo = a.bounds + (size_t)ph * 2 * D, *hi = lo + D;
                const double s = a.k_scale[ph];
#pragma unroll 1
                for (int h = 0; h < a.G; ++h) {
                    const size_t qi = (((size_t)b * a.Hkv * a.G + hk * a.G + h) * a.Sq + i) * D;
                    double x = 0.0;
                    for (int c = lane * 8; c < D; c += 256) {
                        float q8[8], l8[8], h8[8];
                        codec::load8<DT>(a.q, qi + c, q8);
                        const uint2 lw = *reinterpret_cast<const uint2 *>(lo + c);
                        const uint2 hw = *reinterpret_cast<const uint2 *>(hi + c);
                        codec::decode4<FMT>(lw.x, l8); codec::decode4<FMT>(lw.y, l8 + 4);
                        codec::decode4<FMT>(hw.x, h8); codec::decode4<FMT>(hw.y, h8 + 4);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            x = fma((double)q8[e], (double)(q8[e] < 0.f ? l8[e] : h8[e]), x);
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                    best = (x > best || x != x) ? x : best;
                }
                best *= s;
                if (best != best) best = INFINITY;  // a NaN is attended to, so that it shows
            }
            if (lane == 0) exact[j] = best;
        }
        __syncthreads();
        for (int j = t; j < near_n; j += kThreads) {
            const double x = exact[j];
            const int p = near[j];
            int place = 0;
            for (int o = 0; o < near_n; ++o)
                place += exact[o] > x || (exact[o] == x && near[o] < p);
            if (place < places) key[p] = 1;
        }
    }
    __syncthreads();
    // ascending order; the last visible page closes the list
    int done = 0;
    for (int base = 0; base < m; base += kThreads) {
        const int p = base + t;
        const int in = p < m ? (int)key[p] : 0;
        int n;
        const int at = done + block_scan(in, wsum[0], &n);
        if (in && in_bounds(at < k, a.status)) out[at] = p;
        done += n;
    }
    if (t == 0) out[k] = m;
}

template <int D, int FMT, int DT>
int launch_select_t(SelectArgs &a, int sms, cudaStream_t stream) {
    const int64_t units = (int64_t)a.B * a.Hkv * a.Sq;
    // CTAs per unit: up to eight while they fit the GPU at two an SM and have 64 pages each
    a.cluster = 1;
    while (a.cluster < kMaxCluster && units * a.cluster * 2 <= 2 * sms && a.cluster * 2 * 64 <= a.max_pages)
        a.cluster *= 2;
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
                    c.n_pages, max_pages, n_select, causal, 1, status_word_device_ptr()};
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
