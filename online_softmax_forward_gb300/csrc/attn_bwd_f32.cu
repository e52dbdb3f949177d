// attn_bwd_f32.cu -- fp32 backward pass of attention on CUDA cores (attn_bwd.h
// has the formulas and the two kinds of units).
//
// A CTA of 256 threads runs one unit: tiles X1, X2 of 16 R rows stay in shared
// memory, tiles Y1, Y2 of 64 rows stream through it (kv unit: X = k, v and Y =
// q, do; q unit: X = q, do and Y = k, v).  Each step makes
//     T1 = X1 Y1^T, T2 = X2 Y2^T   (R x 4 results a thread, 16 bytes a load)
//     P = exp2(scale log2(e) T1 + nl), dS = P (T2 + nd)
//     A2 += dS Y1, and in a kv unit A1 += P Y2   (R rows x D / 16 channels a thread)
// with P and dS passed through shared memory between the two.  The row
// statistics are computed where do is loaded (o is read once more for each kv
// unit, which costs less than a kernel of its own), so that a small problem is
// one launch.  What bounds it is the FP32 FMA rate: rows are padded so that
// no load meets a bank twice.  R (attn_bwd.cu) is the largest of 4, 2 and 1
// that gives enough units to fill the GPU: 4 has the most FMAs a load.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_bwd.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kT = 64;        // rows of a Y tile
constexpr int kThreads = 256;

template <int D, int R>
struct Cfg {
    static constexpr int kX = 16 * R;  // rows of an X tile
    static constexpr int kLd = D + 4;
    static constexpr int kLdP = kX + 8;  // row stride of P and dS
    static constexpr int kOffY = 2 * kX * kLd;
    static constexpr int kOffP = kOffY + 2 * kT * kLd;
    static constexpr int kOffStat = kOffP + 2 * kT * kLdP;
    static constexpr int kSmemBytes = (kOffStat + 2 * kT) * 4;
    // CTAs an SM that shared memory allows, two at most
    static constexpr int kCtas = 2 * kSmemBytes + 2048 <= 233472 ? 2 : 1;
    static constexpr int kW = D >= 64 ? 4 : D / 16;  // channels of a load of the sums
    static constexpr int kNC = D / (16 * kW);
};

struct Params {
    const float *q, *k, *v, *dout, *o;
    const float *lse, *dlse;
    float *dk, *dv, *dq;  // gradients, or the splits' partial sums
    int BH, BHk, group, Sq, Skv, causal;
    int off, wrap;   // of BwdPlan
    int nq, nk;      // X tiles of a slice: query rows, keys
    int yq;          // Y tiles of query rows of a slice
    int ns_kv, ns_q;
    float scale_log2, scale;
    int *status;
};

template <int W>
struct alignas(4 * W) Floats {
    float e[W];
};

// N rows of a [rows, D] slice from row r0 on; rows behind the last one are zero.
template <int D, int N>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int r0, int rows, int *status) {
    constexpr int V = D / 4;
#pragma unroll
    for (int t = threadIdx.x; t < N * V; t += kThreads) {
        const int r = t / V, c = (t % V) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < rows && in_bounds(r0 + r >= 0 && c + 4 <= D, status))
            x = *reinterpret_cast<const float4 *>(src + (size_t)(r0 + r) * D + c);
        *reinterpret_cast<float4 *>(dst + r * (D + 4) + c) = x;
    }
}

// The same for rows of do, with their statistics: nl = -lse log2(e) (-inf for a row
// without a key, and behind the last one) and nd = dlse - rowsum(o do).
template <int D, int N>
__device__ __forceinline__ void load_do(float *dst, float *nl, float *nd, const Params &p, int slice, int r0) {
    constexpr int V = D / 4;  // lanes of a row
    static_assert(N * V % 32 == 0, "whole warps");
    const size_t s = (size_t)slice * p.Sq;
#pragma unroll
    for (int t = threadIdx.x; t < N * V; t += kThreads) {
        const int r = t / V, c = (t % V) * 4, row = r0 + r;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        float dot = 0.f;
        const bool live = row < p.Sq && in_bounds(slice < p.BH, p.status);
        if (live) {
            x = *reinterpret_cast<const float4 *>(p.dout + (s + row) * D + c);
            const float4 y = *reinterpret_cast<const float4 *>(p.o + (s + row) * D + c);
            dot = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, x.w * y.w)));
        }
        *reinterpret_cast<float4 *>(dst + r * (D + 4) + c) = x;
#pragma unroll
        for (int m = V / 2; m > 0; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
        if (t % V == 0) {
            const float l = live ? p.lse[s + row] : -INFINITY;
            nl[r] = l == -INFINITY ? -INFINITY : l * -1.4426950408889634f;
            nd[r] = live ? (p.dlse ? p.dlse[s + row] : 0.f) - dot : 0.f;
        }
    }
}

// T[i][j] = X[tx + 16 i] . Y[ty + 16 j]
template <int D, int R>
__device__ __forceinline__ void product(const float *X, const float *Y, int tx, int ty, float (&T)[R][4]) {
    constexpr int LD = D + 4;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) T[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 x[R], y[4];
#pragma unroll
        for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const float4 *>(X + (tx + 16 * i) * LD + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4 *>(Y + (ty + 16 * j) * LD + c);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                T[i][j] = fmaf(x[i].x, y[j].x, T[i][j]);
                T[i][j] = fmaf(x[i].y, y[j].y, T[i][j]);
                T[i][j] = fmaf(x[i].z, y[j].z, T[i][j]);
                T[i][j] = fmaf(x[i].w, y[j].w, T[i][j]);
            }
    }
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, Cfg<D, R>::kCtas)
attn_bwd_f32_kernel(const Params p) {
    using C = Cfg<D, R>;
    constexpr int LD = C::kLd, LP = C::kLdP, W = C::kW, NC = C::kNC, X = C::kX;
    extern __shared__ __align__(16) float sm[];
    float *X1 = sm, *X2 = sm + X * LD, *Y1 = sm + C::kOffY, *Y2 = Y1 + kT * LD;
    float *Ps = sm + C::kOffP, *Ds = Ps + kT * LP;
    float *nls = sm + C::kOffStat, *nds = nls + kT;  // of the query rows of Y or of X
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tx = (warp & 1) * 8 + (lane & 7), ty = (warp >> 1) * 4 + (lane >> 3);

    // the unit: kv units first, longest first where the call is causal
    const int n_kv = p.BHk * p.nk * p.ns_kv;
    const bool kv = (int)blockIdx.x < n_kv;
    int u = kv ? (int)blockIdx.x : (int)blockIdx.x - n_kv;
    const int slices = kv ? p.BHk : p.BH, ns = kv ? p.ns_kv : p.ns_q;
    int tile = u / (slices * ns);
    u -= tile * slices * ns;
    const int zx = u / ns, split = u - zx * ns;
    if (!kv && p.causal) tile = p.nq - 1 - tile;
    const int x0 = tile * X;
    const bool skips = p.causal && !p.wrap;  // whole tiles that the mask leaves out
    const int first = kv && skips ? max(0, x0 - p.off) / kT : 0;
    int per;  // steps of a head
    if (kv) {
        per = p.yq - first;
    } else {
        const int end = skips ? min(p.Skv, min(x0 + X, p.Sq) + p.off) : p.Skv;
        per = end > 0 ? (end + kT - 1) / kT : 0;
    }
    const int64_t steps = (int64_t)per * (kv ? p.group : 1);
    const int t0 = (int)(steps * split / ns), n = (int)(steps * (split + 1) / ns) - t0;
    const int skip = per > 0 ? t0 / per : 0;
    int y = first + t0 - skip * per;
    int zy = kv ? zx * p.group + skip : zx / p.group;
    const int xrows = kv ? p.Skv : p.Sq, yrows = kv ? p.Sq : p.Skv;
    if (!in_bounds(zx < slices && x0 < xrows, p.status)) return;

    float a1[R][NC][W], a2[R][NC][W];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < W; ++e) a1[i][c][e] = a2[i][c][e] = 0.f;

    if (n > 0) {
        const size_t s = (size_t)zx * xrows * D;
        load_tile<D, X>(X1, (kv ? p.k : p.q) + s, x0, xrows, p.status);
        if (kv)
            load_tile<D, X>(X2, p.v + s, x0, xrows, p.status);
        else
            load_do<D, X>(X2, nls, nds, p, zx, x0);
    }
    for (int step = 0; step < n; ++step) {
        const int y0 = y * kT;
        if (step > 0) __syncthreads();  // the previous step's reads of Y, P and dS are done
        const size_t s = (size_t)zy * yrows * D;
        if (in_bounds(zy < (kv ? p.BH : p.BHk) && y0 < yrows, p.status)) {
            load_tile<D, kT>(Y1, (kv ? p.q : p.k) + s, y0, yrows, p.status);
            if (kv)
                load_do<D, kT>(Y2, nls, nds, p, zy, y0);
            else
                load_tile<D, kT>(Y2, p.v + s, y0, yrows, p.status);
        }
        __syncthreads();
        float T1[R][4], T2[R][4];
        product<D, R>(X1, Y1, tx, ty, T1);
        product<D, R>(X2, Y2, tx, ty, T2);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int xi = tx + 16 * i, yi = ty + 16 * j;
                const int qi = kv ? y0 + yi : x0 + xi, kj = kv ? x0 + xi : y0 + yi;
                const int pos = p.wrap ? qi % p.wrap : qi;
                const bool seen = kj < p.Skv && (!p.causal || kj <= pos + p.off);
                const float l = nls[kv ? yi : xi], d = nds[kv ? yi : xi];
                const float pr = seen ? ptx::ex2_approx(fmaf(T1[i][j], p.scale_log2, l)) : 0.f;
                if (kv) Ps[yi * LP + xi] = pr;
                Ds[yi * LP + xi] = seen ? pr * (T2[i][j] + d) : 0.f;
            }
        __syncthreads();
        // rows R ty .. of X, channels tx W + 16 W c
#pragma unroll 4
        for (int r = 0; r < kT; ++r) {
            const Floats<R> ds = *reinterpret_cast<const Floats<R> *>(Ds + r * LP + R * ty);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const Floats<W> b = *reinterpret_cast<const Floats<W> *>(Y1 + r * LD + tx * W + 16 * W * c);
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int e = 0; e < W; ++e) a2[i][c][e] = fmaf(ds.e[i], b.e[e], a2[i][c][e]);
            }
            if (kv) {
                const Floats<R> pr = *reinterpret_cast<const Floats<R> *>(Ps + r * LP + R * ty);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const Floats<W> b = *reinterpret_cast<const Floats<W> *>(Y2 + r * LD + tx * W + 16 * W * c);
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int e = 0; e < W; ++e) a1[i][c][e] = fmaf(pr.e[i], b.e[e], a1[i][c][e]);
                }
            }
        }
        ++y;
        if (kv && y == p.yq) {
            y = first;
            ++zy;
        }
    }

    const size_t part = (size_t)split * slices * xrows;
    const size_t extent = (size_t)ns * slices * xrows * D;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int row = x0 + R * ty + i;
        if (row >= xrows) continue;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            const size_t g = (part + (size_t)zx * xrows + row) * D + tx * W + 16 * W * c;
            if (!in_bounds(g + W <= extent, p.status)) continue;
            Floats<W> o;
#pragma unroll
            for (int e = 0; e < W; ++e) o.e[e] = a2[i][c][e] * p.scale;
            *reinterpret_cast<Floats<W> *>((kv ? p.dk : p.dq) + g) = o;
            if (kv) {
#pragma unroll
                for (int e = 0; e < W; ++e) o.e[e] = a1[i][c][e];
                *reinterpret_cast<Floats<W> *>(p.dv + g) = o;
            }
        }
    }
}

template <int D, int R>
int launch_r(const Params &p, int64_t units, cudaStream_t stream) {
    if (!set_smem_limit_once(reinterpret_cast<const void *>(attn_bwd_f32_kernel<D, R>), Cfg<D, R>::kSmemBytes))
        return ATTN_ERR_LAUNCH;
    attn_bwd_f32_kernel<D, R><<<(unsigned)units, kThreads, Cfg<D, R>::kSmemBytes, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

template <int D>
int launch_d(const Params &p, const BwdPlan &plan, cudaStream_t stream) {
    switch (plan.tile) {
    case 64: return launch_r<D, 4>(p, plan.n_units, stream);
    case 32: return launch_r<D, 2>(p, plan.n_units, stream);
    default: return launch_r<D, 1>(p, plan.n_units, stream);
    }
}

}  // namespace

int launch_bwd_f32(const BwdArgs &a, const BwdPlan &plan, cudaStream_t stream) {
    const Problem &pr = plan.p;
    uint8_t *ws = (uint8_t *)a.workspace;
    Params p{};
    p.q = (const float *)a.q;
    p.k = (const float *)a.k;
    p.v = (const float *)a.v;
    p.dout = (const float *)a.dout;
    p.o = (const float *)a.o;
    p.lse = a.lse;
    p.dlse = a.dlse;
    p.BH = (int)pr.bh();
    p.BHk = (int)pr.bh_kv();
    p.group = pr.group;
    p.Sq = pr.Sq;
    p.Skv = pr.Skv;
    p.causal = pr.causal;
    p.off = plan.off;
    p.wrap = plan.wrap;
    p.nq = plan.nq;
    p.nk = plan.nk;
    p.ns_kv = plan.ns_kv;
    p.ns_q = plan.ns_q;
    p.yq = (pr.Sq + kT - 1) / kT;
    p.scale_log2 = pr.scale * 1.4426950408889634f;
    p.scale = pr.scale;
    p.status = status_word_device_ptr();
    if (!p.status) return ATTN_ERR_CUDA;
    float *part_kv = (float *)(ws + plan.off_part_kv);
    p.dk = plan.ns_kv > 1 ? part_kv : (float *)a.dk;
    p.dv = plan.ns_kv > 1 ? part_kv + (size_t)plan.ns_kv * pr.bh_kv() * pr.Skv * pr.d : (float *)a.dv;
    p.dq = plan.ns_q > 1 ? (float *)(ws + plan.off_part_q) : (float *)a.dq;
    switch (pr.d) {
    case 16: return launch_d<16>(p, plan, stream);
    case 32: return launch_d<32>(p, plan, stream);
    case 64: return launch_d<64>(p, plan, stream);
    case 128: return launch_d<128>(p, plan, stream);
    default: return ATTN_ERR_INVALID_ARG;
    }
}

}  // namespace attn
