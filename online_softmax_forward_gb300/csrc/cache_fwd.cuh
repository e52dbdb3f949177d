// cache_fwd.cuh -- what the attention kernels over the cache share: their
// arguments, where a tile lies among the sequences, and the rows of a unit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "attn_internal.h"
#include "cache_codec.cuh"
#include "cache_index.h"

namespace attn {

struct FwdArgs {
    const void *q;
    void *o;
    float *lse;
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *table, *lens, *counts, *pages;
    float *hold;      // [warp][R][D]: state of the unit a warp's range begins inside of, if more follows
    float *po, *pl;   // states of the CTAs' shared units by slot: [slot][R][D], [slot][R] (log2)
    int4 *tail;       // [CTA]: the unit that runs over the end of a CTA's range
    int B, Hkv, G, Sq, page, n_pages, max_pages, n_sel, causal;
    int nseg, rows, nrb;  // row groups of a (sequence, kv head), rows of one, row blocks of one
    int units;            // of a sequence: Hkv * nseg * nrb
    int dtype, workers;
    int one_each;         // a CTA per unit, and no state left for a second kernel
    FastDiv by_units, by_per, by_nrb, by_group;  // per = nseg * nrb
    float sl2;  // scale * log2(e)
    int *status;
};

// attn_cache_tc.cu: the 128-row kernel.  a: every field but the workspace's and
// those of the row blocks.
int launch_cache_tc(FwdArgs &a, int d, int format, void *workspace, cudaStream_t stream);

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Sequence lengths as tile counts, summed: prefix[b] tiles before sequence b.
// For a block of THREADS; warp_sums [THREADS / 32].
template <int THREADS>
__device__ __forceinline__ void scan_lengths(const FwdArgs &a, int kt, int *prefix, int *warp_sums) {
    const int per = (a.B + THREADS - 1) / THREADS;
    const int b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
        const int len0 = a.lens[b], cnt = a.counts ? a.counts[b] : a.Sq;
        const int len = clamp_len(len0, a.max_pages, a.page);
        if ((len != len0 || cnt < 0 || cnt > a.Sq) && blockIdx.x == 0)
            atomicOr(a.status, kStatusTable);
        const int n = (int)(((int64_t)len + kt - 1) / kt);
        prefix[b + 1] = n;  // turned into a sum below
        sum += n;
    }
    int incl = sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int at = incl - sum;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) at += w < warp ? warp_sums[w] : 0;
    for (int b = b0; b < b1; ++b) prefix[b + 1] = at += prefix[b + 1];
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
}

// Where tile x lies.
__device__ __forceinline__ Place place_of(const FwdArgs &a, const int *prefix, int tpu, int64_t x) {
    Place p;
    if (a.pages) {
        const int64_t n = quotient(x, tpu);
        p.b = (int)quotient(n, a.units);
        p.unit = (int)(n - (int64_t)p.b * a.units);
        p.n = tpu;
        p.t = (int)(x - n * tpu);
        return p;
    }
    const int y = (uint64_t)x >> 31 ? (int)(x / a.units) : (int)((uint32_t)x / a.by_units);
    int lo = 0, hi = a.B - 1;  // the last b with prefix[b] <= y
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= y) lo = mid; else hi = mid - 1;
    }
    const int64_t in = x - (int64_t)prefix[lo] * a.units;
    p.b = lo;
    p.n = prefix[lo + 1] - prefix[lo];
    p.unit = (int)quotient(in, p.n);
    p.t = (int)(in - (int64_t)p.unit * p.n);
    return p;
}

struct Unit {
    int b, hk, seg, rb;
};
__device__ __forceinline__ Unit unit_at(const FwdArgs &a, int b, int unit) {
    Unit u;
    u.b = b;
    u.hk = (int)((uint32_t)unit / a.by_per);
    const int in = unit - u.hk * a.nseg * a.nrb;
    u.seg = (int)((uint32_t)in / a.by_nrb);
    u.rb = in - u.seg * a.nrb;
    return u;
}

// Query and head of row r of a unit; false past the group's rows.
template <int R>
__device__ __forceinline__ bool row_of(const FwdArgs &a, const Unit &u, int r, int &i, int &h) {
    const int row = u.rb * R + r;
    const int q = a.pages ? u.seg : (int)((uint32_t)row / a.by_group);
    i = q;
    h = u.hk * a.G + (a.pages ? row : row - q * a.G);
    return row < a.rows;
}

// Elements [i, i + N) of q as fp32.
template <int N>
__device__ __forceinline__ void load_q(const FwdArgs &a, size_t i, float *f) {
    if (a.dtype == ATTN_F32) {
#pragma unroll
        for (int e = 0; e < N; e += 8) codec::load8<0>(a.q, i + e, f + e);
    } else if (a.dtype == ATTN_BF16 || a.dtype == ATTN_BF16_OUT_F32) {
#pragma unroll
        for (int e = 0; e < N; e += 8) codec::load8<1>(a.q, i + e, f + e);
    } else {
#pragma unroll
        for (int e = 0; e < N; e += 8) codec::load8<2>(a.q, i + e, f + e);
    }
}

// The bounds-checking build: is the row of q of this head and query there?
__device__ __forceinline__ bool q_row(const FwdArgs &a, const Unit &u, int h, int i) {
    return in_bounds(u.b < a.B && h < a.Hkv * a.G && i < a.Sq, a.status);
}

// Eight consecutive outputs.
__device__ __forceinline__ void store_o8(const FwdArgs &a, size_t i, const float *f) {
    if (a.dtype == ATTN_BF16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&h);
        }
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.o) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if (a.dtype == ATTN_F16) {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.o) + i) =
            make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
    } else {
        float4 *p = reinterpret_cast<float4 *>(reinterpret_cast<float *>(a.o) + i);
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// `top` before the first key: any visible score is above it by more than the
// range of exp2, so that its weight comes out infinite and sets the references.
constexpr float kUnset = -3.0e38f;

// One output.
__device__ __forceinline__ void store_o(const FwdArgs &a, size_t i, float x) {
    if (a.dtype == ATTN_BF16) reinterpret_cast<__nv_bfloat16 *>(a.o)[i] = __float2bfloat16_rn(x);
    else if (a.dtype == ATTN_F16) reinterpret_cast<__half *>(a.o)[i] = __float2half_rn(x);
    else reinterpret_cast<float *>(a.o)[i] = x;
}

// Row of o and lse that row r of a unit is; false past the group's rows.
template <int R>
__device__ __forceinline__ bool out_row(const FwdArgs &a, const Unit &u, int r, size_t &row) {
    int i, h;
    if (!row_of<R>(a, u, r, i, h)) return false;
    row = ((size_t)u.b * a.Hkv * a.G + h) * a.Sq + i;
    return in_bounds(i < a.Sq && h < a.Hkv * a.G && u.b < a.B, a.status);
}
// Factor of the weights that join the states of kCacheMaxCtas CTAs: their sum of the largest
// values is finite.
constexpr float kFits = 0x1p-8f;
constexpr float kLn2 = 0.69314718055994530942f;

}  // namespace attn
