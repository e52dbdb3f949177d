// attn_cache_select.cu -- which pages of a sequence each query attends to.
//
// For query row i, kv head h (its group's G query heads) and page p:
//     score(p) = k_scale[p] * max_g sum_c max(q_gc * lo_pc, q_gc * hi_pc),
// lo and hi being the smallest and largest key code of each channel of the
// page: an upper bound of every q . k in it, from 2 d bytes a page instead of
// page * d.  The page of the query's last visible key is always taken, then
// the highest scores, ties to the lowest page.
//
// Scores are summed in fp32 with a bound on their error.  A page whose score
// is further from the cut than that is decided by it; the few others are
// summed again in fp64, where the products of a 16-bit q and an 8-bit code
// (at most 19 bits) add up exactly unless they span more than 2^27, so the
// choice does not depend on the order of a sum.  (fp64 for every page would
// cost more than the reading: this GPU has 1/64 the fp64 rate.)
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_internal.h"
#include "cache_codec.cuh"
#include "cache_index.h"

namespace attn {
namespace {

struct SelectArgs {
    const void *q;  // [B][Hkv * G][Sq][d]
    const uint8_t *bounds;
    const float *k_scale;
    const int32_t *table, *lens, *counts;
    int32_t *pages;  // [B][Hkv][Sq][n]
    float *scores;   // [B][Hkv][Sq][max_pages]
    float *mass;     // [B][Hkv][Sq]: max over the group of sum |q|
    double *exact;   // [B][Hkv][Sq][max_pages]: fp64 scores of the pages near the cut
    int B, Hkv, G, Sq, page, n_pages, max_pages, n, causal;
    int *status;
};

constexpr int kScoreThreads = 256;
constexpr int kScorePages = 128;   // pages per CTA of the score kernel
constexpr int kSelectThreads = 256;

__device__ __forceinline__ float warp_sum_f(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Pages visible to query i of sequence b.
__device__ __forceinline__ int visible_pages(const SelectArgs &a, int b, int i) {
    const int len0 = a.lens[b], cnt0 = a.counts ? a.counts[b] : a.Sq;
    const int len = clamp_len(len0, a.max_pages, a.page);
    const int cnt = min(max(cnt0, 0), a.Sq);
    if ((len != len0 || cnt != cnt0) && threadIdx.x == 0) atomicOr(a.status, kStatusTable);
    const int keys = visible_keys(len, cnt, i, a.causal);
    return (int)(((int64_t)keys + a.page - 1) / a.page);
}

// Physical page, or -1 (reported) for an entry outside the pool.
__device__ __forceinline__ int page_of(const SelectArgs &a, int b, int lp) {
    const int phys = a.table[(int64_t)b * a.max_pages + lp];
    if (phys < 0 || phys >= a.n_pages) {
        atomicOr(a.status, kStatusTable);
        return -1;
    }
    return phys;
}

// grid (units, page chunks); 16 channels per lane, D / 16 lanes per page.
template <int D, int FMT, int DT>
__global__ void __launch_bounds__(kScoreThreads) cache_score_kernel(const SelectArgs a) {
    constexpr int L = D / 16;       // lanes per page
    constexpr int PPW = 32 / L;     // pages per warp step
    extern __shared__ float sq[];   // [G][D] positive parts, then [G][D] negative parts
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t unit = blockIdx.x;  // (b, hk, i)
    const int i = (int)(unit % a.Sq);
    const int hk = (int)(unit / a.Sq % a.Hkv);
    const int b = (int)(unit / a.Sq / a.Hkv);
    const int vis = visible_pages(a, b, i);
    const int p0 = blockIdx.y * kScorePages;
    if (vis <= a.n || p0 >= vis - 1) return;  // every page is taken, or none of these is scored
    float *pos = sq, *neg = sq + a.G * D;
    for (int t = threadIdx.x; t < a.G * (D / 8); t += kScoreThreads) {
        const int g = t / (D / 8), c = t % (D / 8) * 8;
        float f[8];
        codec::load8<DT>(a.q, (((size_t)b * a.Hkv * a.G + hk * a.G + g) * a.Sq + i) * D + c, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {  // written so that a NaN stays in both parts
            pos[g * D + c + e] = f[e] < 0.f ? 0.f : f[e];
            neg[g * D + c + e] = f[e] > 0.f ? 0.f : f[e];
        }
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane / L, l = lane % L;
    if (blockIdx.y == 0 && warp == 0) {
        float most = 0.f;
        for (int g = 0; g < a.G; ++g) {
            float s = 0.f;
            for (int c = lane; c < D; c += 32) s += pos[g * D + c] - neg[g * D + c];
            s = warp_sum_f(s);
            most = (s > most || s != s) ? s : most;
        }
        if (lane == 0) a.mass[unit] = most;
    }
    const int p1 = min(p0 + kScorePages, vis - 1);
    for (int base = p0 + warp * PPW; base < p1; base += kScoreThreads / 32 * PPW) {
        const int lp = base + sub;
        float best = -INFINITY, s = 0.f;
        int phys = -1;
        if (lp < p1) phys = page_of(a, b, lp);
        uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
        if (phys >= 0) {
            const int64_t ph = (int64_t)phys * a.Hkv + hk;
            const uint4 *src = reinterpret_cast<const uint4 *>(a.bounds + (size_t)ph * 2 * D) + l;
            lo = src[0];
            hi = src[L];
            s = a.k_scale[ph];
        }
        float fl[16], fh[16];
        codec::decode4<FMT>(lo.x, fl); codec::decode4<FMT>(lo.y, fl + 4);
        codec::decode4<FMT>(lo.z, fl + 8); codec::decode4<FMT>(lo.w, fl + 12);
        codec::decode4<FMT>(hi.x, fh); codec::decode4<FMT>(hi.y, fh + 4);
        codec::decode4<FMT>(hi.z, fh + 8); codec::decode4<FMT>(hi.w, fh + 12);
        for (int g = 0; g < a.G; ++g) {
            const float4 *qp = reinterpret_cast<const float4 *>(pos + g * D + l * 16);
            const float4 *qn = reinterpret_cast<const float4 *>(neg + g * D + l * 16);
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float4 u = qp[e], w = qn[e];
                x = fmaf(u.x, fh[4 * e], fmaf(w.x, fl[4 * e], x));
                x = fmaf(u.y, fh[4 * e + 1], fmaf(w.y, fl[4 * e + 1], x));
                x = fmaf(u.z, fh[4 * e + 2], fmaf(w.z, fl[4 * e + 2], x));
                x = fmaf(u.w, fh[4 * e + 3], fmaf(w.w, fl[4 * e + 3], x));
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            best = (x > best || x != x) ? x : best;
        }
        // a page outside the pool scores lowest
        if (lp < p1 && l == 0 && in_bounds(lp < a.max_pages, a.status))
            a.scores[unit * a.max_pages + lp] = phys >= 0 ? best * s : -INFINITY;
    }
}

// fp32 value as an integer of the same order.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? u & 0x7fffffffu : ~u);
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
    for (int w = 0; w < kSelectThreads / 32; ++w) {
        if (w < warp) before += warps[w];
        all += warps[w];
    }
    *total = all;
    return before + __popc(m & ((1u << lane) - 1));
}

// One CTA per (b, hk, i).  Shared memory: keys [max_pages], then the list of
// pages near the cut [max_pages].
template <int D, int FMT, int DT>
__global__ void __launch_bounds__(kSelectThreads) cache_select_kernel(const SelectArgs a) {
    extern __shared__ __align__(16) uint8_t sm[];
    __shared__ int hist[256], wsum[kSelectThreads / 32];
    __shared__ int s_bin, s_left, s_near;
    __shared__ uint32_t s_top;
    const int64_t unit = blockIdx.x;
    const int i = (int)(unit % a.Sq);
    const int hk = (int)(unit / a.Sq % a.Hkv);
    const int b = (int)(unit / a.Sq / a.Hkv);
    const int vis = visible_pages(a, b, i);
    int32_t *out = a.pages + unit * a.n;
    const int t = threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (vis <= a.n) {
        for (int j = t; j < a.n; j += kSelectThreads) out[j] = j < vis ? j : -1;
        return;
    }
    double *exact = a.exact + unit * a.max_pages;                         // [max_pages]
    uint32_t *key = reinterpret_cast<uint32_t *>(sm);                     // [max_pages]
    int *near = reinterpret_cast<int *>(key + a.max_pages);               // [max_pages]
    const int m = vis - 1;       // pages that compete
    const int k = a.n - 1;       // places for them
    if (t == 0) {
        s_near = 0;
        s_top = 0;
    }
    __syncthreads();
    const float *sc = a.scores + unit * a.max_pages;
    // the largest scale bounds every page's error; a score that is not
    // finite leaves the whole decision to fp64
    float scale_top = 0.f;
    bool odd = false;
    for (int p = t; p < m; p += kSelectThreads) {
        const float x = sc[p];
        key[p] = ordered(x);
        const int phys = a.table[(int64_t)b * a.max_pages + p];
        if (phys >= 0 && phys < a.n_pages) {
            const float s = a.k_scale[(int64_t)phys * a.Hkv + hk];
            if (!(fabsf(x) <= 3.402823466e38f) || s != s) odd = true;
            scale_top = fmaxf(scale_top, s);
        }
    }
    atomicMax(&s_top, odd ? 0x7f800000u : __float_as_uint(scale_top));
    __syncthreads();
    // |error| <= 2^-24 * (16 + 4 additions) * sum |q| * top * scale, and the
    // rounding of the last product; 24 covers both
    constexpr float kTop = FMT == ATTN_CACHE_E4M3 ? 448.f : 128.f;
    const float eps = 24.f * 5.9604645e-8f * kTop * a.mass[unit] * __uint_as_float(s_top);

    float cut_lo = -INFINITY, cut_hi = INFINITY;  // decided above cut_hi: in; below cut_lo: out
    if (k == 0) {
        cut_lo = INFINITY;
    } else if (eps <= 3.402823466e38f) {
        // the k-th largest key, 8 bits at a time
        uint32_t prefix = 0, mask = 0;
        int left = k;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int h = t; h < 256; h += kSelectThreads) hist[h] = 0;
            __syncthreads();
            for (int p = t; p < m; p += kSelectThreads)
                if ((key[p] & mask) == prefix) atomicAdd(&hist[(key[p] >> shift) & 255], 1);
            __syncthreads();
            if (t < 32) {  // lane t: bins 255 - 8 t down to 248 - 8 t
                int c[8], sum = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum += c[e] = hist[255 - 8 * t - e];
                int incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, o);
                    if (t >= o) incl += y;
                }
                int above = incl - sum;
                if (above < left && left <= incl) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (above < left && left <= above + c[e]) {
                            s_bin = 255 - 8 * t - e;
                            s_left = left - above;
                            above = 1 << 30;
                        } else {
                            above += c[e];
                        }
                    }
                }
            }
            __syncthreads();
            prefix |= (uint32_t)s_bin << shift;
            mask |= 255u << shift;
            left = s_left;
        }
        const float T = unordered(prefix);
        cut_lo = T - 2.f * eps;
        cut_hi = T + 2.f * eps;
        // a bound that rounds back to T would decide equal scores
        if (!(cut_lo < T)) cut_lo = T;
        if (!(cut_hi > T)) cut_hi = T;
    }
    // pages above the cut are in, those near it are listed
    int sure = 0;
    for (int base = 0; base < m; base += kSelectThreads) {
        const int p = base + t;
        const float x = p < m ? unordered(key[p]) : 0.f;
        const bool in = p < m && k > 0 && x > cut_hi;
        const bool close = p < m && k > 0 && !in && !(x < cut_lo);
        if (close) {
            const int at = atomicAdd(&s_near, 1);
            near[at] = p;
        }
        int n;
        block_scan(in, wsum, &n);
        sure += n;
        __syncthreads();
        if (p < m) key[p] = in ? 1 : 0;
    }
    __syncthreads();
    const int near_n = s_near, places = k - sure;
    if (near_n <= places) {
        for (int j = t; j < near_n; j += kSelectThreads) key[near[j]] = 1;
    } else {
        const int warp = t >> 5, lane = t & 31;
        for (int j = warp; j < near_n; j += kSelectThreads / 32) {
            const int phys = a.table[(int64_t)b * a.max_pages + near[j]];
            double best = -INFINITY;
            if (phys >= 0 && phys < a.n_pages) {
                const int64_t ph = (int64_t)phys * a.Hkv + hk;
                const uint8_t *lo = a.bounds + (size_t)ph * 2 * D, *hi = lo + D;
                const double s = a.k_scale[ph];
                for (int g = 0; g < a.G; ++g) {
                    const size_t qi = (((size_t)b * a.Hkv * a.G + hk * a.G + g) * a.Sq + i) * D;
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
        for (int j = t; j < near_n; j += kSelectThreads) {
            const double x = exact[j];
            const int p = near[j];
            int rank = 0;
            for (int o = 0; o < near_n; ++o)
                rank += exact[o] > x || (exact[o] == x && near[o] < p);
            if (rank < places) key[p] = 1;
        }
    }
    __syncthreads();
    // ascending order; the last visible page closes the list
    int done = 0;
    for (int base = 0; base < m; base += kSelectThreads) {
        const int p = base + t;
        const int in = p < m ? (int)key[p] : 0;
        int n;
        const int at = done + block_scan(in, wsum, &n);
        if (in && in_bounds(at < k, a.status)) out[at] = p;
        done += n;
    }
    if (t == 0) out[k] = m;
}

template <int D, int FMT, int DT>
int launch_select_t(const SelectArgs &a, cudaStream_t stream) {
    const int64_t units = (int64_t)a.B * a.Hkv * a.Sq;
    const int chunks = (a.max_pages + kScorePages - 1) / kScorePages;
    auto score = cache_score_kernel<D, FMT, DT>;
    auto select = cache_select_kernel<D, FMT, DT>;
    const int smem1 = 2 * a.G * D * 4;
    const int smem2 = a.max_pages * 8;
    if (!set_smem_limit_once(reinterpret_cast<const void *>(score), 2 * kMaxSelectGroup * D * 4) ||
        !set_smem_limit_once(reinterpret_cast<const void *>(select), kMaxSelectPages * 8))
        return ATTN_ERR_LAUNCH;
    score<<<dim3((unsigned)units, (unsigned)chunks), kScoreThreads, smem1, stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)units);
    cfg.blockDim = dim3(kSelectThreads);
    cfg.dynamicSmemBytes = (size_t)smem2;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, select, a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

template <int D, int FMT>
int launch_select_q(const SelectArgs &a, int dtype, cudaStream_t stream) {
    if (dtype == ATTN_F32) return launch_select_t<D, FMT, 0>(a, stream);
    if (dtype == ATTN_BF16 || dtype == ATTN_BF16_OUT_F32) return launch_select_t<D, FMT, 1>(a, stream);
    return launch_select_t<D, FMT, 2>(a, stream);
}

}  // namespace

int launch_cache_select(const attn_cache &c, const void *q, const int32_t *table, int max_pages,
                        const int32_t *lens, const int32_t *counts, int32_t *pages, int n_select,
                        int B, int H, int Sq, int causal, int dtype, void *workspace,
                        cudaStream_t stream) {
    const int64_t units = (int64_t)B * c.H_kv * Sq;
    double *exact = reinterpret_cast<double *>(workspace);
    float *scores = reinterpret_cast<float *>(exact + units * max_pages);
    SelectArgs a = {q, (const uint8_t *)c.k_bounds, c.k_scale, table, lens, counts, pages, scores,
                    scores + units * max_pages, exact, B, c.H_kv, H / c.H_kv, Sq, c.page, c.n_pages,
                    max_pages, n_select, causal, status_word_device_ptr()};
    if (!a.status) return ATTN_ERR_CUDA;
    if (c.d == 64)
        return c.format == ATTN_CACHE_E4M3 ? launch_select_q<64, ATTN_CACHE_E4M3>(a, dtype, stream)
                                           : launch_select_q<64, ATTN_CACHE_I8>(a, dtype, stream);
    return c.format == ATTN_CACHE_E4M3 ? launch_select_q<128, ATTN_CACHE_E4M3>(a, dtype, stream)
                                       : launch_select_q<128, ATTN_CACHE_I8>(a, dtype, stream);
}

}  // namespace attn
