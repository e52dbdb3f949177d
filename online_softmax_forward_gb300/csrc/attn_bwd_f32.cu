// attn_bwd_f32.cu -- fp32 backward pass of attention on CUDA cores (attn_bwd.h
// has the formulas and the two kinds of units).
//
// A CTA of 256 threads runs one unit: tiles X1, X2 of 64 rows stay in shared
// memory, tiles Y1, Y2 of 64 rows stream through it (kv unit: X = k, v and Y =
// q, do; q unit: X = q, do and Y = k, v).  Each step makes
//     T1 = X1 Y1^T, T2 = X2 Y2^T   (4 x 4 results a thread, 16 bytes a load)
//     P = exp2(scale log2(e) T1 + nl), dS = P (T2 + nd)
//     A2 += dS Y1, and in a kv unit A1 += P Y2   (4 rows x D / 16 channels a thread)
// with P and dS passed through shared memory between the two.  What bounds it
// is the FP32 FMA rate: 16-byte loads feed eight FMAs each in both parts, and
// rows are padded so that no load meets a bank twice.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_bwd.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kT = 64;        // rows of every tile
constexpr int kThreads = 256;
constexpr int kLdP = 72;      // row stride of P and dS

template <int D>
struct Cfg {
    static constexpr int kLd = D + 4;
    static constexpr int kTile = kT * kLd;
    static constexpr int kSmemBytes = (4 * kTile + 2 * kT * kLdP) * 4;
    static constexpr int kW = D >= 64 ? 4 : D / 16;  // channels of a load of the sums
    static constexpr int kNC = D / (16 * kW);
};

struct Params {
    const float *q, *k, *v, *dout;
    const float *stats;
    float *dk, *dv, *dq;  // gradients, or the splits' partial sums
    int BH, BHk, group, Sq, Skv, causal;
    int nq, nk, ns_kv, ns_q, stat_tiles;
    float scale_log2, scale;
    int *status;
};

template <int W>
struct alignas(4 * W) Floats {
    float e[W];
};

// 64 rows of a [rows, D] slice from row r0 on; rows behind the last one are zero.
template <int D>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int r0, int rows, int *status) {
    constexpr int V = D / 4;
#pragma unroll
    for (int t = threadIdx.x; t < kT * V; t += kThreads) {
        const int r = t / V, c = (t % V) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r0 + r < rows && in_bounds(r0 + r >= 0 && c + 4 <= D, status))
            x = *reinterpret_cast<const float4 *>(src + (size_t)(r0 + r) * D + c);
        *reinterpret_cast<float4 *>(dst + r * (D + 4) + c) = x;
    }
}

// T[i][j] = X[tx + 16 i] . Y[ty + 16 j]
template <int D>
__device__ __forceinline__ void product(const float *X, const float *Y, int tx, int ty, float (&T)[4][4]) {
    constexpr int LD = D + 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) T[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] = *reinterpret_cast<const float4 *>(X + (tx + 16 * i) * LD + c);
            y[i] = *reinterpret_cast<const float4 *>(Y + (ty + 16 * i) * LD + c);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                T[i][j] = fmaf(x[i].x, y[j].x, T[i][j]);
                T[i][j] = fmaf(x[i].y, y[j].y, T[i][j]);
                T[i][j] = fmaf(x[i].z, y[j].z, T[i][j]);
                T[i][j] = fmaf(x[i].w, y[j].w, T[i][j]);
            }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
attn_bwd_f32_kernel(const Params p) {
    using C = Cfg<D>;
    constexpr int LD = C::kLd, W = C::kW, NC = C::kNC;
    extern __shared__ __align__(16) float sm[];
    float *X1 = sm, *X2 = sm + C::kTile, *Y1 = sm + 2 * C::kTile, *Y2 = sm + 3 * C::kTile;
    float *Ps = sm + 4 * C::kTile, *Ds = Ps + kT * kLdP;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tx = (warp & 1) * 8 + (lane & 7), ty = (warp >> 1) * 4 + (lane >> 3);
    const int off = p.Skv - p.Sq;

    // the unit: kv units first, longest first where the call is causal
    const int n_kv = p.BHk * p.nk * p.ns_kv;
    const bool kv = (int)blockIdx.x < n_kv;
    int u = kv ? (int)blockIdx.x : (int)blockIdx.x - n_kv;
    const int slices = kv ? p.BHk : p.BH, ns = kv ? p.ns_kv : p.ns_q;
    int tile = u / (slices * ns);
    u -= tile * slices * ns;
    const int zx = u / ns, split = u - zx * ns;
    if (!kv && p.causal) tile = p.nq - 1 - tile;
    const int x0 = tile * kT;
    const int first = kv && p.causal ? max(0, x0 - off) / kT : 0;
    int per;  // steps of a head
    if (kv) {
        per = p.nq - first;
    } else {
        const int end = p.causal ? min(p.Skv, min(x0 + kT, p.Sq) + off) : p.Skv;
        per = end > 0 ? (end + kT - 1) / kT : 0;
    }
    const int64_t steps = (int64_t)per * (kv ? p.group : 1);
    const int t0 = (int)(steps * split / ns), n = (int)(steps * (split + 1) / ns) - t0;
    const int skip = per > 0 ? t0 / per : 0;
    int y = first + t0 - skip * per;
    int zy = kv ? zx * p.group + skip : zx / p.group;
    const int xrows = kv ? p.Skv : p.Sq, yrows = kv ? p.Sq : p.Skv;
    if (!in_bounds(zx < slices && x0 < xrows, p.status)) return;

    if (n > 0) {
        const size_t s = (size_t)zx * xrows * D;
        load_tile<D>(X1, (kv ? p.k : p.q) + s, x0, xrows, p.status);
        load_tile<D>(X2, (kv ? p.v : p.dout) + s, x0, xrows, p.status);
    }
    float a1[4][NC][W], a2[4][NC][W];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < W; ++e) a1[i][c][e] = a2[i][c][e] = 0.f;

    auto stat = [&](int slice, int row, float &nl, float &nd) {
        const float *s = p.stats + ((size_t)slice * p.stat_tiles + row / kStatTile) * 2 * kStatTile + row % kStatTile;
        nl = -INFINITY;
        nd = 0.f;
        if (row < p.Sq && in_bounds(slice < p.BH, p.status)) {
            nl = s[0];
            nd = s[kStatTile];
        }
    };
    float nl[4], nd[4];  // of this thread's four query rows
    if (!kv) {
#pragma unroll
        for (int i = 0; i < 4; ++i) stat(zx, x0 + tx + 16 * i, nl[i], nd[i]);
    }

    for (int step = 0; step < n; ++step) {
        const int y0 = y * kT;
        __syncthreads();  // the previous step's reads of Y, P and dS are done
        const size_t s = (size_t)zy * yrows * D;
        if (in_bounds(zy < (kv ? p.BH : p.BHk) && y0 < yrows, p.status)) {
            load_tile<D>(Y1, (kv ? p.q : p.k) + s, y0, yrows, p.status);
            load_tile<D>(Y2, (kv ? p.dout : p.v) + s, y0, yrows, p.status);
        }
        if (kv) {
#pragma unroll
            for (int i = 0; i < 4; ++i) stat(zy, y0 + ty + 16 * i, nl[i], nd[i]);
        }
        __syncthreads();
        float T1[4][4], T2[4][4];
        product<D>(X1, Y1, tx, ty, T1);
        product<D>(X2, Y2, tx, ty, T2);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int xr = x0 + tx + 16 * i, yr = y0 + ty + 16 * j;
                const int qi = kv ? yr : xr, kj = kv ? xr : yr;
                const bool seen = kj < p.Skv && (!p.causal || kj <= qi + off);
                const float l = kv ? nl[j] : nl[i], dd = kv ? nd[j] : nd[i];
                const float pr = seen ? ptx::ex2_approx(fmaf(T1[i][j], p.scale_log2, l)) : 0.f;
                if (kv) Ps[(ty + 16 * j) * kLdP + tx + 16 * i] = pr;
                Ds[(ty + 16 * j) * kLdP + tx + 16 * i] = seen ? pr * (T2[i][j] + dd) : 0.f;
            }
        __syncthreads();
        // rows 4 ty .. 4 ty + 3 of X, channels tx W + 16 W c
#pragma unroll 4
        for (int r = 0; r < kT; ++r) {
            const float4 ds = *reinterpret_cast<const float4 *>(Ds + r * kLdP + 4 * ty);
            const float dsv[4] = {ds.x, ds.y, ds.z, ds.w};
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const Floats<W> b = *reinterpret_cast<const Floats<W> *>(Y1 + r * LD + tx * W + 16 * W * c);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < W; ++e) a2[i][c][e] = fmaf(dsv[i], b.e[e], a2[i][c][e]);
            }
            if (kv) {
                const float4 pr = *reinterpret_cast<const float4 *>(Ps + r * kLdP + 4 * ty);
                const float prv[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const Floats<W> b = *reinterpret_cast<const Floats<W> *>(Y2 + r * LD + tx * W + 16 * W * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < W; ++e) a1[i][c][e] = fmaf(prv[i], b.e[e], a1[i][c][e]);
                }
            }
        }
        ++y;
        if (kv && y == p.nq) {
            y = first;
            ++zy;
        }
    }

    const size_t part = (size_t)split * slices * xrows;
    const size_t extent = (size_t)ns * slices * xrows * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = x0 + 4 * ty + i;
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

template <int D>
int launch_d(const Params &p, int64_t units, cudaStream_t stream) {
    if (!set_smem_limit_once(reinterpret_cast<const void *>(attn_bwd_f32_kernel<D>), Cfg<D>::kSmemBytes))
        return ATTN_ERR_LAUNCH;
    attn_bwd_f32_kernel<D><<<(unsigned)units, kThreads, Cfg<D>::kSmemBytes, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // namespace

int launch_bwd_f32(const BwdArgs &a, const Problem &pr, const BwdPlan &plan, cudaStream_t stream) {
    uint8_t *ws = (uint8_t *)a.workspace;
    Params p{};
    p.q = (const float *)a.q;
    p.k = (const float *)a.k;
    p.v = (const float *)a.v;
    p.dout = (const float *)a.dout;
    p.stats = (const float *)(ws + plan.off_stats);
    p.BH = (int)pr.bh();
    p.BHk = (int)pr.bh_kv();
    p.group = pr.group;
    p.Sq = pr.Sq;
    p.Skv = pr.Skv;
    p.causal = pr.causal;
    p.nq = plan.nq;
    p.nk = plan.nk;
    p.ns_kv = plan.ns_kv;
    p.ns_q = plan.ns_q;
    p.stat_tiles = (pr.Sq + kStatTile - 1) / kStatTile;
    p.scale_log2 = pr.scale * 1.4426950408889634f;
    p.scale = pr.scale;
    p.status = status_word_device_ptr();
    if (!p.status) return ATTN_ERR_CUDA;
    float *part_kv = (float *)(ws + plan.off_part_kv);
    p.dk = plan.ns_kv > 1 ? part_kv : (float *)a.dk;
    p.dv = plan.ns_kv > 1 ? part_kv + (size_t)plan.ns_kv * pr.bh_kv() * pr.Skv * pr.d : (float *)a.dv;
    p.dq = plan.ns_q > 1 ? (float *)(ws + plan.off_part_q) : (float *)a.dq;
    switch (pr.d) {
    case 16: return launch_d<16>(p, plan.n_units, stream);
    case 32: return launch_d<32>(p, plan.n_units, stream);
    case 64: return launch_d<64>(p, plan.n_units, stream);
    case 128: return launch_d<128>(p, plan.n_units, stream);
    default: return ATTN_ERR_INVALID_ARG;
    }
}

}  // namespace attn
