// attn_bwd.cu -- backward pass: the plan, the kernel of the row statistics and
// the one that adds the splits (attn_bwd.h has the mathematics).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <algorithm>

#include "attn_bwd.h"

namespace attn {

bool bwd_plan(const Problem &call, BwdPlan *plan) {
    Problem p = call;
    plan->off = call.Skv - call.Sq;
    plan->wrap = 0;
    if (p.group > 1 && (!p.causal || (p.Sq <= kStatTile && plan->off >= 0)) && (int64_t)p.group * p.Sq <= kMaxBwdRows) {
        p.H /= p.group;
        p.Sq *= p.group;
        p.group = 1;
        if (p.causal) plan->wrap = call.Sq;
    }
    plan->p = p;
    if (p.Sq > kMaxBwdRows || p.Skv > kMaxBwdRows) return false;
    const bool f32 = p.dtype == ATTN_F32, f16 = p.dtype == ATTN_F16 || p.dtype == ATTN_F16_OUT_F32;
    const int64_t bh = p.bh(), bhk = p.bh_kv();
    // the sizes below are products of these; anything near 2^62 bytes is refused first
    const double est = 4.0 * kScaleRows * kMaxBwdSplits * ((double)bh * (p.Sq + 128.0) + (double)bhk * (p.Skv + 128.0)) *
                       (p.d + 2.0);
    if (est > 4.0e18) return false;
    // rows of a unit's own tile and of the tiles it walks over
    const int step = f32 ? 64 : 128;
    auto tiles = [](int n, int tile) { return (n + tile - 1) / tile; };
    auto units_of = [&](int tile) { return (double)bhk * tiles(p.Skv, tile) + (double)bh * tiles(p.Sq, tile); };
    plan->tile = step;
    // fp32: smaller units while they do not fill the places of two CTAs an SM
    if (f32)
        while (plan->tile > 16 && units_of(plan->tile) < 1.5 * kBwdSms) plan->tile /= 2;
    plan->nq = tiles(p.Sq, plan->tile);
    plan->nk = tiles(p.Skv, plan->tile);
    plan->ns_kv = plan->ns_q = 1;
    // Costs in products of a step: a kv unit makes four a step, a q unit three.  A unit
    // longer than three quarters of an SM's share of everything would be what the
    // launch waits for, so it is cut; but not below eight steps, where the partial sums
    // and their kernel cost more than they give.
    const double len_kv = 4.0 * p.group * tiles(p.Sq, step), len_q = 3.0 * tiles(p.Skv, step);
    const double share = ((double)bhk * plan->nk * len_kv + (double)bh * plan->nq * len_q) / kBwdSms *
                         (p.causal && call.Sq == call.Skv ? 0.5 : 1.0);
    // dS sums to zero over a row's keys and is largest where these are few, so that there its
    // rounding to 16 bits is most of what dq and dk are wrong by, and in a causal call it is
    // large beside the gradients of the later rows (8192 tokens in bf16: one element of dq
    // wrong by 0.44 of dq's root mean square, now 0.17).  Steps of query tiles whose first row
    // sees at most kFewKeys keys therefore take dS in two parts, with one product more.  Where
    // there are no more keys in all, P is in two parts too (2 heads of 128 keys 7.0 us in
    // any form; 1024 heads of 100 keys 43.6 -> 51 us); in the first tile of a causal call that
    // would cost the issuing warp of all steps another test (8192 tokens 5 %).  The rule goes
    // by positions alone, so that no row's precision depends on what else is in the batch.
    plan->few = 0;
    if (p.Skv <= kFewKeys) plan->few = plan->nq;
    else if (plan->wrap) plan->few = plan->off < kFewKeys ? plan->nq : 0;  // every tile may hold a first position
    else if (p.causal && plan->off < kFewKeys) plan->few = std::min(plan->nq, (kFewKeys - 1 - plan->off) / kStatTile + 1);
    if (f32) plan->few = 0;
    const double least = 32.0;
    const double goal = share * 0.75 > least ? share * 0.75 : least;
    auto cut = [&](double len) {
        const double n = ceil(len / goal);
        return n < 1 ? 1 : n > kMaxBwdSplits ? kMaxBwdSplits : (int)n;
    };
    plan->ns_kv = cut(len_kv);
    plan->ns_q = cut(len_q);
    // The units with the longer walks start first, so that the last ones are short (fp32, 2 x
    // 8 heads of 40 queries to 2000 keys, d = 64: 70 -> 45 us; 77 queries of 32768 keys, 32
    // heads in bf16: 178 -> 167 us).
    plan->q_first = len_q / plan->ns_q > len_kv / plan->ns_kv;
    const double units = (double)bhk * plan->nk * plan->ns_kv + (double)bh * plan->nq * plan->ns_q;
    if (units > (double)(INT32_MAX / 2)) return false;
    plan->n_units = (int64_t)units;
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    plan->off_stats = f32 ? 0 : 256;  // fp32 units compute the statistics themselves
    const size_t stat_tiles = (size_t)bh * tiles(p.Sq, kStatTile);
    plan->off_max = plan->off_stats + (f32 ? 0 : up(stat_tiles * (f16 ? kScaleRows : 2) * kStatTile * 4));
    plan->off_max_v = plan->off_max + (f16 ? up(stat_tiles * 2 * 4) : 0);
    const size_t maxima = (f16 ? up(stat_tiles * 2 * 4) + up((size_t)bhk * tiles(p.Skv, kStatTile) * 4) : 0);
    // bf16 leaves this room unused; workspaces keep their least size
    plan->off_part_kv = plan->off_max + (f32 ? 0 : std::max(maxima, up(kMaximaBytes)));
    plan->off_part_q = plan->off_part_kv +
                       (plan->ns_kv > 1 ? up((size_t)plan->ns_kv * bhk * p.Skv * p.d * 2 * 4) : 0);
    plan->bytes = plan->off_part_q + (plan->ns_q > 1 ? up((size_t)plan->ns_q * bh * p.Sq * p.d * 4) : 0);
    return true;
}

namespace {

constexpr int kPreThreads = 256;
constexpr int kSumThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }  // of o
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }

template <typename T, int N>
struct alignas(16) Row {
    T e[N];
};

struct PreParams {
    const void *o, *dout, *v;
    const float *lse, *dlse;
    float *stats;
    float *max_q, *max_v;   // fp16: [tiles][2] largest |do| and |D|, [v_tiles] largest |v|
    unsigned *counter;      // of the units, set to 0
    int64_t tiles, v_tiles; // blocks of statistics, tiles of v
    int Sq, tiles_per_head, Skv, v_tiles_per_head;
    float add;              // to nl (fp16: P is kept times 2^add)
    int *status;
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, s));
    return x;
}

// Row statistics.  D / E lanes share a row (E elements of do in 16 bytes), four rows at
// a time with all loads first; what bounds it is reading o and do once (32 heads of
// 8192 rows of 128 in bf16, 135 MB: 24 us, 5.6 TB/s).
//
// fp16 (kScale): a CTA takes whole tiles, so that it can join their largest norms (attn_bwd.h),
// and then tiles of v.
template <typename TD, typename TO, int D, bool kScale>
__global__ void __launch_bounds__(kPreThreads) bwd_stats_kernel(const PreParams p) {
    constexpr int E = 16 / sizeof(TD), L = D / E;  // elements of a lane, lanes of a row
    constexpr int R = 32 / L;                      // rows of a warp
    constexpr int U = 4;                           // rows of a lane group, all loads first
    constexpr int kGroups = kStatTile / (R * U);   // times a warp reads, in a tile
    constexpr int kWarps = kPreThreads / 32;
    constexpr int kPer = kScale ? kScaleRows : 2;
    static_assert(L >= 1 && L <= 32 && kStatTile % (R * U) == 0, "lanes");
    const int lane = threadIdx.x & 31, sub = lane % L, rw = lane / L;
    if (blockIdx.x == 0 && threadIdx.x == 0) p.counter[0] = 0u;
    // the next kernel may be set up on SMs that this one leaves free; it waits for the results
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    [[maybe_unused]] float big_do = 0.f, big_d = 0.f;
    auto group = [&](int64_t tile, int g) {
        const int in_tile = g * (R * U) + rw;
        const int64_t bh = tile / p.tiles_per_head;
        const int row0 = (int)(tile - bh * p.tiles_per_head) * kStatTile + in_tile;
        Row<TD, E> x[U];
        Row<TO, E> y[U];
        float l[U], dl[U];
        constexpr int kWords = sizeof(y[0]) / 16;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const size_t r = (size_t)bh * p.Sq + row0 + u * R, at = r * D + sub * E;
            l[u] = -INFINITY;
            dl[u] = 0.f;
            if (row0 + u * R < p.Sq) {
                if (sub == 0) {
                    l[u] = p.lse[r];
                    if (p.dlse) dl[u] = p.dlse[r];
                }
                *reinterpret_cast<uint4 *>(&x[u]) = *reinterpret_cast<const uint4 *>((const TD *)p.dout + at);
#pragma unroll
                for (int i = 0; i < kWords; ++i)
                    reinterpret_cast<uint4 *>(&y[u])[i] = reinterpret_cast<const uint4 *>((const TO *)p.o + at)[i];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int row = row0 + u * R;
            float dot = 0.f, sq = 0.f, nl = -INFINITY, nd = 0.f;
            if (row < p.Sq) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    dot = fmaf(to_f(x[u].e[i]), to_f(y[u].e[i]), dot);
                    if constexpr (kScale) sq = fmaf(to_f(x[u].e[i]), to_f(x[u].e[i]), sq);
                }
            }
#pragma unroll
            for (int s = L / 2; s > 0; s >>= 1) {
                dot += __shfl_xor_sync(0xffffffffu, dot, s);
                if constexpr (kScale) sq += __shfl_xor_sync(0xffffffffu, sq, s);
            }
            if (sub != 0) continue;
            float norm = 0.f;
            if (row < p.Sq) {
                // a row that sees no key has P = 0, and no D that P would be multiplied with
                nl = l[u] == -INFINITY ? -INFINITY : fmaf(l[u], -1.4426950408889634f, p.add);
                nd = l[u] == -INFINITY ? 0.f : dl[u] - dot;
                if (kScale && l[u] != -INFINITY) {
                    norm = sqrtf(sq);
                    if (norm < INFINITY && fabsf(nd) < INFINITY) {  // false for NaN, too
                        big_do = fmaxf(big_do, norm);
                        big_d = fmaxf(big_d, fabsf(nd));
                    }
                }
            }
            float *st = p.stats + (size_t)tile * kPer * kStatTile + in_tile + u * R;
            if (in_bounds(tile < p.tiles && in_tile + u * R < kStatTile, p.status)) {
                st[0] = nl;
                st[kStatTile] = nd;
                if constexpr (kScale) st[2 * kStatTile] = norm;
            }
        }
    };
    if constexpr (!kScale) {
        const int64_t warp = ((int64_t)blockIdx.x * kPreThreads + threadIdx.x) >> 5;
        const int64_t warps = (int64_t)gridDim.x * kPreThreads >> 5;
        for (int64_t w = warp; w < p.tiles * kGroups; w += warps) group(w / kGroups, (int)(w % kGroups));
    } else {
        __shared__ float part[2][kWarps];
        const int warp = threadIdx.x >> 5;
        for (int64_t item = blockIdx.x; item < p.tiles + p.v_tiles; item += gridDim.x) {
            big_do = big_d = 0.f;
            const bool of_v = item >= p.tiles;
            if (!of_v) {
                for (int g = warp; g < kGroups; g += kWarps) group(item, g);
            } else {
                const int64_t tile = item - p.tiles, slice = tile / p.v_tiles_per_head;
                const int row0 = (int)(tile - slice * p.v_tiles_per_head) * kStatTile;
                constexpr int kTimes = kStatTile / (kWarps * R);
                Row<TD, E> x[kTimes];
#pragma unroll
                for (int i = 0; i < kTimes; ++i) {
                    const int row = row0 + (i * kWarps + warp) * R + rw;
                    *reinterpret_cast<uint4 *>(&x[i]) = make_uint4(0, 0, 0, 0);
                    if (row < p.Skv)
                        *reinterpret_cast<uint4 *>(&x[i]) = *reinterpret_cast<const uint4 *>(
                            (const TD *)p.v + ((size_t)slice * p.Skv + row) * D + sub * E);
                }
#pragma unroll
                for (int i = 0; i < kTimes; ++i) {
                    float sq = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) sq = fmaf(to_f(x[i].e[e]), to_f(x[i].e[e]), sq);
#pragma unroll
                    for (int s = L / 2; s > 0; s >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, s);
                    if (sq < INFINITY) big_do = fmaxf(big_do, sqrtf(sq));
                }
            }
            big_do = warp_max(big_do);
            big_d = warp_max(big_d);
            if (lane == 0) {
                part[0][warp] = big_do;
                part[1][warp] = big_d;
            }
            __syncthreads();
            if (threadIdx.x < 2) {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) x = fmaxf(x, part[threadIdx.x][i]);
                if (!of_v) {
                    p.max_q[2 * item + threadIdx.x] = x;
                } else if (threadIdx.x == 0) {
                    p.max_v[item - p.tiles] = x;
                }
            }
            __syncthreads();
        }
    }
}

struct SumParams {
    const float *part[3];  // [splits][n] each; null: nothing to add
    void *out[3];
    int64_t n[3];          // elements
    int splits[3];
    int type;              // of the gradients: 0 fp32, 1 bf16, 2 fp16
};

// Adds the splits of dk, dv and dq in order; four elements a thread.
__global__ void __launch_bounds__(kSumThreads) bwd_sum_kernel(const SumParams p) {
    const int j = blockIdx.y;
    if (!p.part[j]) return;
    const int64_t n4 = p.n[j] / 4;
    const int64_t stride = (int64_t)gridDim.x * kSumThreads;
    for (int64_t i = (int64_t)blockIdx.x * kSumThreads + threadIdx.x; i < n4; i += stride) {
        const float4 *src = reinterpret_cast<const float4 *>(p.part[j]) + i;
        float4 a = *src;
        for (int s = 1; s < p.splits[j]; ++s) {
            const float4 b = src[s * n4];
            a.x += b.x;
            a.y += b.y;
            a.z += b.z;
            a.w += b.w;
        }
        if (p.type == 0) {
            reinterpret_cast<float4 *>(p.out[j])[i] = a;
        } else {
            uint2 w;
            if (p.type == 1) {
                *reinterpret_cast<__nv_bfloat162 *>(&w.x) = __floats2bfloat162_rn(a.x, a.y);
                *reinterpret_cast<__nv_bfloat162 *>(&w.y) = __floats2bfloat162_rn(a.z, a.w);
            } else {
                *reinterpret_cast<__half2 *>(&w.x) = __floats2half2_rn(a.x, a.y);
                *reinterpret_cast<__half2 *>(&w.y) = __floats2half2_rn(a.z, a.w);
            }
            reinterpret_cast<uint2 *>(p.out[j])[i] = w;
        }
    }
}

template <typename TD, typename TO, int D, bool kScale>
int launch_stats(const PreParams &p, cudaStream_t stream) {
    constexpr int R = 32 / (D * (int)sizeof(TD) / 16);
    const int64_t warps = p.tiles * (kStatTile / R / 4);
    int64_t grid = kScale ? p.tiles + p.v_tiles : (warps + kPreThreads / 32 - 1) / (kPreThreads / 32);
    const int64_t most = kScale ? 1 << 20 : kPreBlocks;
    if (grid > most) grid = most;
    bwd_stats_kernel<TD, TO, D, kScale><<<(unsigned)grid, kPreThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

template <int D>
int stats_16(const PreParams &p, int dtype, cudaStream_t stream) {
    switch (dtype) {
    case ATTN_BF16: return launch_stats<__nv_bfloat16, __nv_bfloat16, D, false>(p, stream);
    case ATTN_BF16_OUT_F32: return launch_stats<__nv_bfloat16, float, D, false>(p, stream);
    case ATTN_F16: return launch_stats<__half, __half, D, true>(p, stream);
    default: return launch_stats<__half, float, D, true>(p, stream);
    }
}

}  // namespace

int launch_bwd(const BwdArgs &a, const BwdPlan &plan, cudaStream_t stream) {
    const Problem &p = plan.p;
    uint8_t *ws = (uint8_t *)a.workspace;
    const bool f16 = p.dtype == ATTN_F16 || p.dtype == ATTN_F16_OUT_F32;
    PreParams r{};
    r.o = a.o;
    r.dout = a.dout;
    r.v = a.v;
    r.lse = a.lse;
    r.dlse = a.dlse;
    r.counter = (unsigned *)ws;
    r.stats = (float *)(ws + plan.off_stats);
    r.max_q = (float *)(ws + plan.off_max);
    r.max_v = (float *)(ws + plan.off_max_v);
    r.tiles_per_head = (p.Sq + kStatTile - 1) / kStatTile;
    r.tiles = p.bh() * r.tiles_per_head;
    r.v_tiles_per_head = (p.Skv + kStatTile - 1) / kStatTile;
    r.v_tiles = p.bh_kv() * r.v_tiles_per_head;
    r.Sq = p.Sq;
    r.Skv = p.Skv;
    r.add = f16 ? (float)kBwdP16Log2 : 0.f;
    r.status = status_word_device_ptr();
    if (!r.status) return ATTN_ERR_CUDA;
    int st = ATTN_OK;
    if (p.dtype != ATTN_F32)
        st = p.d == 64 ? stats_16<64>(r, p.dtype, stream) : stats_16<128>(r, p.dtype, stream);
    if (st != ATTN_OK) return st;
    st = p.dtype == ATTN_F32 ? launch_bwd_f32(a, plan, stream) : launch_bwd_tc(a, plan, stream);
    if (st != ATTN_OK || (plan.ns_kv == 1 && plan.ns_q == 1)) return st;
    SumParams s{};
    int64_t most = 0;
    auto add = [&](int j, const float *part, void *out, int64_t n, int splits) {
        s.part[j] = part;
        s.out[j] = out;
        s.n[j] = n;
        s.splits[j] = splits;
        if (n > most) most = n;
    };
    if (plan.ns_kv > 1) {
        const int64_t n = p.bh_kv() * p.Skv * p.d;
        const float *kv = (const float *)(ws + plan.off_part_kv);
        add(0, kv, a.dk, n, plan.ns_kv);
        add(1, kv + (size_t)plan.ns_kv * n, a.dv, n, plan.ns_kv);
    }
    if (plan.ns_q > 1)
        add(2, (const float *)(ws + plan.off_part_q), a.dq, p.bh() * p.Sq * p.d, plan.ns_q);
    s.type = elem_bytes_out(p.dtype) == 4 ? 0 : f16 ? 2 : 1;
    int64_t grid = (most / 4 + kSumThreads - 1) / kSumThreads;
    if (grid > 8 * kBwdSms) grid = 8 * kBwdSms;
    bwd_sum_kernel<<<dim3((unsigned)grid, 3), kSumThreads, 0, stream>>>(s);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // namespace attn
