// attn_bwd_f32.cu -- fp32 backward pass of attention (attn_bwd.h has the
// formulas and the two kinds of units).
//
// A CTA of 256 threads runs one unit: tiles X1, X2 of 16 R rows stay in shared
// memory, tiles Y1, Y2 of 64 rows stream through it (kv unit: X = k, v and Y =
// q, do; q unit: X = q, do and Y = k, v).  Each step makes
//     T1 = X1 Y1^T, T2 = X2 Y2^T
//     P = exp2(scale log2(e) T1 + nl), dS = P (T2 + nd)
//     A2 += dS Y1, and in a kv unit A1 += P Y2
// A warp owns 16 rows of X and its share of the 64 columns.
//
//  * Products.  fp32 FMAs are bound by what shared memory delivers to registers
//    (4 x 4 results a thread: 22 TFLOP/s of 74), so the products run on the tensor
//    cores, each fp32 number as the sum of two tf32 ones, hi (rounded to 11
//    bits) and lo = x - hi: x y = hi hi + hi lo + lo hi, wrong by 2^-21 of |x y| at
//    most for numbers of 2^-112 to 2^128 - 2^116.  (Larger ones round to an infinity, and
//    of smaller ones lo is no normal number and counts as 0.  Bounding hi by the largest
//    tf32 number, one more instruction a split, cost 5 to 10 %.)  mma.sync: its
//    fragments come from plain fp32 tiles of any width and stay in registers; tcgen05
//    would want both parts of every tile in shared memory, which two tiles of 64 rows fill.
//  * P and dS never leave registers: the accumulator of T holds columns 2 t, 2 t +
//    1 where the left operand of A wants k = t, t + 4, which is only another
//    order of the summed rows, so Y's rows are read in that order.
//  * The tensor cores' sums round towards zero.  T adds its large products (hi hi)
//    apart from the small ones, 64 channels at a time (one sum over 128: error 1.06e-6 in
//    place of 0.85e-6, 186 us in place of 190): 8 such roundings at most; the small ones' sum
//    takes 2 for each 8 channels, of numbers 2^-11 as large.  A's sums of a step start at
//    zero and are added to the unit's in fp32: 12 roundings at most.
//  * The next step's tiles are copied while this one's are multiplied (two stages).
//  * The row statistics are computed where do has come (o is read once more for
//    each kv unit, which costs less than a kernel of its own), so that a small
//    problem is one launch.
//  * The loads of T's products are ldmatrix, and up to 32 rows X is split into its parts
//    once, beside itself (8 heads of 512: 49.7 -> 46.3 us; 64 rows would leave room for
//    one CTA an SM). Products of one part follow each other over the column tiles, so
//    that none waits for the one before it.
// R (attn_bwd.cu) is the largest of 4, 2 and 1 that gives enough units to fill the
// GPU; the 8 / R warps that share rows add their sums at the end, in order.
//
// What bounds it: the tensor cores' tf32 rate (300 TFLOP/s measured for mma.sync, 100
// for three products), 54 to 58 % busy, and the loads and splits between
// their instructions.  8 heads of 512 x 512, d = 64: 46 us (as FP32 FMAs 90); 64 heads of
// 1000 x 1000, 16 kv heads, causal: 578 us, 35 TFLOP/s of the five products.
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
    static constexpr int kX = 16 * R;      // rows of an X tile
    static constexpr int kWY = 8 / R;      // warps that share rows of X
    static constexpr int kN = kT / kWY / 8;  // 8-column tiles of T a warp
    static constexpr int kLd = D + 4;
    // X is held as its two parts, X1, X2 (hi) and behind them their lo
    static constexpr bool kParts = R <= 2;
    static constexpr int kOffY = (kParts ? 4 : 2) * kX * kLd;
    static constexpr int kStage = 2 * kT * kLd;  // Y1 and Y2; two stages
    static constexpr int kOffStat = kOffY + 2 * kStage;
    static constexpr int kSmemBytes = (kOffStat + 3 * kT) * 4;
    // CTAs an SM: the sums of 128 channels take the registers of a whole one
    static constexpr int kCtas = D <= 64 ? 2 : 1;
    static_assert(8 * 16 * D <= kStage, "the warps' sums fit where Y was");
};

struct Params {
    const float *q, *k, *v, *dout, *o;
    const float *lse, *dlse;
    float *dk, *dv, *dq;  // gradients, or the splits' partial sums
    int BH, BHk, group, Sq, Skv, causal;
    int off, wrap;   // of BwdPlan
    int nq, nk;      // X tiles of a slice: query rows, keys
    int yq;          // Y tiles of query rows of a slice
    int ns_kv, ns_q, q_first;
    float scale_log2, scale;
    int *status;
};

// x = hi + lo, hi with 11 significant bits (to nearest), lo what is left
struct Split {
    uint32_t hi, lo;
};
__device__ __forceinline__ Split split(float x) {
    Split r;
    r.hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    r.lo = __float_as_uint(x - __uint_as_float(r.hi));
    return r;
}

// c += a b on 16 x 8 by 8 x 8 tiles (tf32: the lower 13 bits of a and b are not read).
// Thread l, g = l / 4, t = l mod 4: a at rows g, g + 8, k = t (a[0], a[1]) and t + 4 (a[2],
// a[3]); b at k = t, t + 4, column g; c at rows g (c[0], c[1]), g + 8, columns 2 t, 2 t + 1.
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// N rows of a [rows, D] slice from row r0 on, asynchronously; rows before `from_row` and
// behind the last one are zero.
template <int D, int N>
__device__ __forceinline__ void load_tile(float *dst, const float *src, int r0, int from_row, int rows, int *status) {
    constexpr int V = D / 4;
#pragma unroll
    for (int t = threadIdx.x; t < N * V; t += kThreads) {
        const int r = t / V, c = (t % V) * 4;
        const bool live = r0 + r >= from_row && r0 + r < rows && in_bounds(r0 + r >= 0 && c + 4 <= D, status);
        const float *from = live ? src + (size_t)(r0 + r) * D + c : src;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_addr(dst + r * (D + 4) + c)),
                     "l"(from), "r"(live ? 16 : 0)
                     : "memory");
    }
}

// What the statistics of N query rows need beside do, on its way in registers: o, and
// (thread r, row r) lse and dlse.
template <int D, int N>
struct StatRows {
    static constexpr int V = D / 4, K = (N * V + kThreads - 1) / kThreads;
    float4 o[K];
    float lse, dlse;

    __device__ __forceinline__ void load(const Params &p, int slice, int r0) {
        const size_t s = (size_t)slice * p.Sq;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int t = threadIdx.x + i * kThreads, row = r0 + t / V;
            o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < N * V && row < p.Sq && in_bounds(slice < p.BH, p.status))
                o[i] = *reinterpret_cast<const float4 *>(p.o + (s + row) * D + (t % V) * 4);
        }
        const int row = r0 + threadIdx.x;
        lse = -INFINITY;
        dlse = 0.f;
        if (threadIdx.x < N && row < p.Sq && in_bounds(slice < p.BH, p.status)) {
            lse = p.lse[s + row];
            if (p.dlse) dlse = p.dlse[s + row];
        }
    }
    // nl = -lse log2(e) (-inf for a row without a key, and behind the last one), nd =
    // -rowsum(o do) and, apart, dlse; `dout` are the rows of do in shared memory
    __device__ __forceinline__ void finish(const float *dout, float *nl, float *nd, float *dl) const {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int t = threadIdx.x + i * kThreads;
            if (N * V % kThreads != 0 && t >= N * V) break;  // whole warps
            const float4 x = *reinterpret_cast<const float4 *>(dout + t / V * (D + 4) + (t % V) * 4);
            float dot = fmaf(x.x, o[i].x, fmaf(x.y, o[i].y, fmaf(x.z, o[i].z, x.w * o[i].w)));
#pragma unroll
            for (int m = V / 2; m > 0; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
            if (t % V == 0) nd[t / V] = -dot;
        }
        if (threadIdx.x < N) {
            nl[threadIdx.x] = lse == -INFINITY ? -INFINITY : lse * -1.4426950408889634f;
            dl[threadIdx.x] = dlse;
        }
    }
};

// 8 x 4 blocks of 32-bit numbers: thread l gets row l / 4, column l mod 4 of each; thread l
// names row l mod 8 of block l / 8.
__device__ __forceinline__ void load_blocks(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void load_blocks(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
}

// T = X Y^T for 16 rows of X and 8 N rows of Y; kLo: how far behind X's hi its lo is, or
// 0 where X is whole.
template <int D, int N, int kLo>
__device__ __forceinline__ void product(const float *X, const float *Y, int lane, float (&T)[N][4]) {
    constexpr int LD = D + 4, J = N > 1 ? 2 : 1;  // column tiles of one load
    constexpr int kSum = D < 64 ? D : 64;         // channels of one sum of the tensor cores
    static_assert(D <= 2 * kSum, "two sums at most");
    const uint32_t xa = ptx::smem_addr(X + (lane & 15) * LD + (lane >> 4) * 4);
    const uint32_t ya = ptx::smem_addr(Y + ((lane & 7) + (N > 1 ? lane >> 4 << 3 : 0)) * LD + (lane >> 3 & 1) * 4);
    float small[N][4];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) T[j][e] = small[j][e] = 0.f;
    auto channels = [&](float (&big)[N][4], int k0) {  // kSum of them from k0 on
#pragma unroll 2
        for (int k = k0; k < k0 + kSum; k += 8) {
            Split a[4], b[N][2];
            uint32_t x[4], xl[4];
            load_blocks(x, xa + k * 4);
            if constexpr (kLo > 0) load_blocks(xl, xa + (kLo + k) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (kLo > 0) a[e] = Split{x[e], xl[e]};
                else a[e] = split(__uint_as_float(x[e]));
            }
#pragma unroll
            for (int j = 0; j < N; j += J) {
                uint32_t y[2 * J];
                load_blocks(y, ya + (8 * j * LD + k) * 4);
#pragma unroll
                for (int e = 0; e < 2 * J; ++e) b[j + e / 2][e & 1] = split(__uint_as_float(y[e]));
            }
#pragma unroll
            for (int j = 0; j < N; ++j) mma(small[j], a[0].lo, a[1].lo, a[2].lo, a[3].lo, b[j][0].hi, b[j][1].hi);
#pragma unroll
            for (int j = 0; j < N; ++j) mma(big[j], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[j][0].hi, b[j][1].hi);
#pragma unroll
            for (int j = 0; j < N; ++j) mma(small[j], a[0].hi, a[1].hi, a[2].hi, a[3].hi, b[j][0].lo, b[j][1].lo);
        }
    };
    channels(T, 0);
    if constexpr (D > kSum) {
        float big[N][4];
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) big[j][e] = 0.f;
        channels(big, kSum);
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) T[j][e] += big[j][e];
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) T[j][e] += small[j][e];
}

// A += W Y for 16 rows of W (8 N columns, as `product` leaves them) and all channels of
// 8 N rows of Y.
template <int D, int N>
__device__ __forceinline__ void accumulate(float (&A)[D / 8][4], const float (&W)[N][4], const float *Y, int g, int t) {
    constexpr int LD = D + 4, M = D / 8 < 4 ? D / 8 : 4;  // channel tiles at a time
    Split w[N][4];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[j][e] = split(W[j][e]);
#pragma unroll
    for (int m0 = 0; m0 < D / 8; m0 += M) {
        float c[M][4];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) c[m][e] = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            Split b[M][2];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                // columns 2 t and 2 t + 1 of W stand where k = t and t + 4 do
                const float *y = Y + (8 * j + 2 * t) * LD + 8 * (m0 + m) + g;
                b[m][0] = split(y[0]);
                b[m][1] = split(y[LD]);
            }
#pragma unroll
            for (int m = 0; m < M; ++m)
                mma(c[m], w[j][0].lo, w[j][2].lo, w[j][1].lo, w[j][3].lo, b[m][0].hi, b[m][1].hi);
#pragma unroll
            for (int m = 0; m < M; ++m)
                mma(c[m], w[j][0].hi, w[j][2].hi, w[j][1].hi, w[j][3].hi, b[m][0].lo, b[m][1].lo);
#pragma unroll
            for (int m = 0; m < M; ++m)
                mma(c[m], w[j][0].hi, w[j][2].hi, w[j][1].hi, w[j][3].hi, b[m][0].hi, b[m][1].hi);
        }
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) A[m0 + m][e] += c[m][e];
    }
}

template <int D, int R>
__global__ void __launch_bounds__(kThreads, Cfg<D, R>::kCtas)
attn_bwd_f32_kernel(const Params p) {
    using C = Cfg<D, R>;
    constexpr int LD = C::kLd, X = C::kX, N = C::kN;
    extern __shared__ __align__(16) float sm[];
    float *X1 = sm, *X2 = sm + X * LD, *Ys = sm + C::kOffY;
    float *nls = sm + C::kOffStat, *nds = nls + kT, *dls = nds + kT;  // of the query rows of Y or of X
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int xw = warp % R * 16, yw = warp / R * (8 * N);  // first row and column of the warp

    // the unit: the kind of BwdPlan::q_first first, longest first where the call is causal
    const int n_kv = p.BHk * p.nk * p.ns_kv, n_q = p.BH * p.nq * p.ns_q;
    const bool kv = p.q_first ? (int)blockIdx.x >= n_q : (int)blockIdx.x < n_kv;
    int u = (int)blockIdx.x - (kv ? (p.q_first ? n_q : 0) : (p.q_first ? 0 : n_kv));
    const int slices = kv ? p.BHk : p.BH, ns = kv ? p.ns_kv : p.ns_q;
    int tile = u / (slices * ns);
    u -= tile * slices * ns;
    const int zx = u / ns, cut = u - zx * ns;
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
    const int t0 = (int)(steps * cut / ns), n = (int)(steps * (cut + 1) / ns) - t0;
    const int skip = per > 0 ? t0 / per : 0;
    int y = first + t0 - skip * per;
    int zy = kv ? zx * p.group + skip : zx / p.group;
    const int xrows = kv ? p.Skv : p.Sq, yrows = kv ? p.Sq : p.Skv;
    // query rows that see no key read as zeros: their P is 0, which would not make 0 of an infinity
    const int blind = p.causal && p.off < 0 ? -p.off : 0, x_from = kv ? 0 : blind, y_from = kv ? blind : 0;
    if (!in_bounds(zx < slices && x0 < xrows, p.status)) return;

    float a1[D / 8][4], a2[D / 8][4];
#pragma unroll
    for (int m = 0; m < D / 8; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) a1[m][e] = a2[m][e] = 0.f;

    // Y1 and Y2 of a step into stage `st`, and what their statistics need
    StatRows<D, kT> rows;
    auto load_y = [&](int st, int zy, int y0) {
        const size_t s = (size_t)zy * yrows * D;
        float *Y = Ys + st * C::kStage;
        if (in_bounds(zy < (kv ? p.BH : p.BHk) && y0 < yrows, p.status)) {
            load_tile<D, kT>(Y, (kv ? p.q : p.k) + s, y0, y_from, yrows, p.status);
            load_tile<D, kT>(Y + kT * LD, (kv ? p.dout : p.v) + s, y0, y_from, yrows, p.status);
            if (kv) rows.load(p, zy, y0);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (n > 0) {
        const size_t s = (size_t)zx * xrows * D;
        load_tile<D, X>(X1, (kv ? p.k : p.q) + s, x0, x_from, xrows, p.status);
        load_tile<D, X>(X2, (kv ? p.v : p.dout) + s, x0, x_from, xrows, p.status);
        load_y(0, zy, y * kT);
        if (!kv) {
            StatRows<D, X> mine;
            mine.load(p, zx, x0);
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
            mine.finish(X2, nls, nds, dls);
        }
        if constexpr (C::kParts) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncthreads();
            for (int i = threadIdx.x; i < 2 * X * (D / 4); i += kThreads) {
                uint4 *at = reinterpret_cast<uint4 *>(X1 + i / (D / 4) * LD + i % (D / 4) * 4);
                const uint4 x = *at;
                const Split a = split(__uint_as_float(x.x)), b = split(__uint_as_float(x.y)),
                            c = split(__uint_as_float(x.z)), d = split(__uint_as_float(x.w));
                *at = make_uint4(a.hi, b.hi, c.hi, d.hi);
                at[2 * X * LD / 4] = make_uint4(a.lo, b.lo, c.lo, d.lo);
            }
        }
    }
    for (int step = 0; step < n; ++step) {
        const int y0 = y * kT;
        float *Y1 = Ys + (step & 1) * C::kStage, *Y2 = Y1 + kT * LD;
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();  // this step's tiles are here, the other stage and the statistics are read
        if (kv) rows.finish(Y2, nls, nds, dls);
        ++y;
        if (kv && y == p.yq) {
            y = first;
            ++zy;
        }
        if (step + 1 < n) load_y((step + 1) & 1, zy, y * kT);
        float T1[N][4], T2[N][4];
        product<D, N, C::kParts ? 2 * X * LD : 0>(X1 + xw * LD, Y1 + yw * LD, lane, T1);
        product<D, N, C::kParts ? 2 * X * LD : 0>(X2 + xw * LD, Y2 + yw * LD, lane, T2);
        if (kv) __syncthreads();  // the statistics are written
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int xi = xw + g + 8 * (e >> 1), yi = yw + 8 * j + 2 * t + (e & 1);
                const int qi = kv ? y0 + yi : x0 + xi, kj = kv ? x0 + xi : y0 + yi;
                const int pos = p.wrap ? qi % p.wrap : qi;
                const bool seen = kj < p.Skv && (!p.causal || kj <= pos + p.off);
                const int si = kv ? yi : xi;
                const float l = nls[si], d = nds[si] + dls[si];
                const float pr = seen ? ptx::ex2_approx(fmaf(T1[j][e], p.scale_log2, l)) : 0.f;
                T1[j][e] = pr;
                T2[j][e] = seen ? pr * (T2[j][e] + d) : 0.f;
            }
        accumulate<D, N>(a2, T2, Y1 + yw * LD, g, t);
        if (kv) accumulate<D, N>(a1, T1, Y2 + yw * LD, g, t);
    }

    // The warps that share rows leave their sums where Y was, [warp's share][X][D], and
    // all threads add them in order.
    const size_t part = (size_t)cut * slices * xrows;
    const size_t extent = (size_t)ns * slices * xrows * D;
    auto write = [&](float (&a)[D / 8][4], float *dst, float scale) {
        __syncthreads();  // Y, or the sums before, are no longer read
        float *mine = Ys + ((warp / R) * X + xw + g) * D + 2 * t;
#pragma unroll
        for (int m = 0; m < D / 8; ++m) {
            *reinterpret_cast<float2 *>(mine + 8 * m) = make_float2(a[m][0], a[m][1]);
            *reinterpret_cast<float2 *>(mine + 8 * D + 8 * m) = make_float2(a[m][2], a[m][3]);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < X * D / 4; i += kThreads) {
            const int r = i / (D / 4), row = x0 + r;
            float4 o = *reinterpret_cast<const float4 *>(Ys + 4 * i);
#pragma unroll
            for (int w = 1; w < C::kWY; ++w) {
                const float4 b = *reinterpret_cast<const float4 *>(Ys + w * X * D + 4 * i);
                o = make_float4(o.x + b.x, o.y + b.y, o.z + b.z, o.w + b.w);
            }
            const size_t at = (part + (size_t)zx * xrows + row) * D + 4 * (i % (D / 4));
            if (row >= xrows || !in_bounds(at + 4 <= extent, p.status)) continue;
            *reinterpret_cast<float4 *>(dst + at) = make_float4(o.x * scale, o.y * scale, o.z * scale, o.w * scale);
        }
    };
    write(a2, kv ? p.dk : p.dq, p.scale);
    if (kv) write(a1, p.dv, 1.f);
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
    p.q_first = plan.q_first;
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
