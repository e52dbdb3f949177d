// attn_bwd_tc.cu -- bf16/fp16 backward pass of attention on the sm_103a tensor
// cores (attn_bwd.h has the formulas and the two kinds of units).
//
// Both kinds of units run through the same kernel, because they have the same
// shape.  A unit holds two tiles X1, X2 of 128 rows and streams pairs of tiles
// Y1, Y2 of 128 rows:
//     kv unit: X1 = k, X2 = v;  Y1 = q, Y2 = do, over the query tiles
//     q unit:  X1 = q, X2 = do; Y1 = k, Y2 = v,  over the key tiles
// and for each step
//     T1 = X1 Y1^T   (scores: P = exp2(scale log2(e) T1 + nl))
//     T2 = X2 Y2^T   (dP:     dS = P (T2 + nd))
//     A2 += dS Y1    (dk of a kv unit, dq of a q unit)
//     A1 += P Y2     (dv; kv units only)
// In a kv unit rows are keys, so that T1 and T2 come out as S^T and dP^T: P and
// dS are then already the left operands of the sums and go back into tensor
// memory where they came from, without a transposition and without touching
// shared memory.  Only the row statistics run along the columns there.
//
//  * Persistent grid, one CTA per SM, 12 warps; units are claimed from a
//    counter in the workspace, kv units of a group of heads first, longest
//    first, so that the CTAs running at any time share the tiles of a few heads
//    through L2 (32 heads of 8192 rows: 1.01 times the inputs read from DRAM).
//  * Warp 8 (producer) streams the tiles with TMA (128-byte swizzle) into a ring of
//    Y1 and one of Y2, and the statistics of a kv unit's query tile beside them.
//  * Warp 9 issues the tcgen05.mma (kind::f16, fp32 accumulate).  A kv unit's step
//    is A1(i), T1(i+1), A2(i), T2(i+1): while the first two run, the other
//    warps turn T2(i) into dS, while the last two run, T1(i+1) into P.  A q
//    unit has no A1, and T2 has two buffers: T1(i+1), T2(i+1) run before A2(i).
//  * Warps 0-3 and 4-7: columns 0-63 and 64-127 of T1 and T2, one thread per row
//    and half (32x32b loads; a 16x256b fragment would spare a kv unit's column
//    statistics their way through shared memory, but holds the read port of tensor
//    memory four times as long).  P stays in fp32 registers between the two; it is
//    rounded to 16 bits for A1 alone, and dS for A2 (as the tensor core takes 16-bit
//    operands; the sums are fp32).  fp16: P is kept times 2^14, and dS times a
//    power of two from the norms of do and v (attn_bwd.h), undone at the end; warp 10
//    joins a unit's norms from their tiles while its first products are on their way.
//    They also write a unit's sums: dv while the last A2 runs, then dk or dq.
//  * Tensor memory (512 columns): Cfg.  P and dS overwrite the first 32 columns of
//    each half of T1 and T2, the second parts (kTwo) the next 32.
//  * Every mbarrier wait is bounded, as in the forward kernel.
//
// What bounds it: at D = 128 and long walks the tensor cores.  32 heads of 8192
// tokens, causal, take 1053 us alone (tensor pipe busy 80 % of the clocks) and 1073 to
// 1098 us in a replayed graph with the row statistics: the seven products of whole tiles
// run at 1.78 to 1.86 PFLOP/s, near the rate that cuBLAS reaches on this GPU, 1.26 PFLOP/s
// of the five that a backward pass cannot do without.  (2.5 % less with kTwo = 0: the
// issuing warp's test stands between a wait and the product that others wait for.)  A step takes 2740 (kv) and 2060 (q) clocks in
// long walks, a unit's start and end about 4000 more, which is what 2 x 4001
// tokens (635 us, 1.03 PFLOP/s) and shorter calls lose.  At D = 64 the
// chain of exponentials and conversions is longer than the products: 1840 and 1400
// clocks a step of 1024 and 768.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <atomic>
#include <math.h>
#include <stdint.h>
#include <type_traits>

#include "attn_bwd.h"
#include "sm100_ptx.cuh"
#include "tc_common.cuh"
#include "tensor_map.h"

namespace attn {
namespace {

constexpr int kRows = 128;  // rows of every tile
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kScaleWarp = 10;  // fp16
constexpr int kThreads = 12 * 32;
constexpr int kComputeWarps = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int kSchedRing = 4;
constexpr int kSchedReaders = 9;  // issuer and 8 computing warps; fp16: and the warp of the scales
constexpr int kStatStages = 2;
constexpr int kLaunchRegs = 168;
constexpr int kComputeRegs = 224;
constexpr int kOtherRegs = 56;
static_assert(2 * 128 * kComputeRegs + 128 * kOtherRegs == kThreads * kLaunchRegs, "register split");
static_assert(kStatTile == kRows, "statistics of a tile");

template <int D>
struct Cfg {
    static_assert(D == 64 || D == 128, "head width");
    static constexpr int kChunks = D / 64;
    static constexpr int kChunkBytes = kRows * 128;  // one 64-channel column of a tile: 16 KB
    static constexpr int kTileBytes = kChunks * kChunkBytes;
    // Tensor-memory columns.  At D = 64 the sums leave room for two T1, so that a kv
    // unit's next scores need not wait for P to be consumed; a q unit has two T2, the
    // second one in place of A1 (D = 128) or of the second T1.
    static constexpr bool kTwoT1 = D == 64;
    static constexpr uint32_t kColT1b = 128, kColT2 = kTwoT1 ? 256 : 128, kColT2b = kTwoT1 ? 128 : 384;
    static constexpr uint32_t kColA2 = kTwoT1 ? 384 : 256, kColA1 = kTwoT1 ? 448 : 384;
    __device__ static constexpr uint32_t col_t1(int b) { return b ? kColT1b : 0u; }
    __device__ static constexpr uint32_t col_t2(int b) { return b ? kColT2b : kColT2; }
    // Rings of Y1 and of Y2.  A Y1 tile is held from T1 of its step until A2, six
    // products in both kinds of units, a Y2 tile for one or two; a tile takes about
    // three products' time to come (D = 128).  One ring of five made each wait for
    // the longer-held of the two (a q unit's step 2740 clocks, now 2060).
    static constexpr int kSlots1 = D == 128 ? 3 : 6;
    static constexpr int kSlots2 = D == 128 ? 2 : 4;
    static constexpr int kOffX = 0;  // X1, X2
    static constexpr int kOffY = 2 * kTileBytes;
    static constexpr int kOffStat = kOffY + (kSlots1 + kSlots2) * kTileBytes;
    __device__ static constexpr int slots(int t) { return t ? kSlots2 : kSlots1; }
    // slot of the n-th tile of Y_t, among all
    __device__ static __forceinline__ uint32_t slot(int t, uint32_t n) {
        return t ? kSlots1 + n % kSlots2 : n % kSlots1;
    }
    __device__ static __forceinline__ uint32_t round(int t, uint32_t n) { return n / (t ? kSlots2 : kSlots1); }
    static constexpr int kStatBytes = 2 * kStatTile * 4;
    static constexpr int kOffBar = kOffStat + kStatStages * kStatBytes;
    static constexpr int kSmemBytes = kOffBar + 896;
};
constexpr int kMaxSlots = 10;

struct Unit {
    int kind;   // 0: kv unit, 1: q unit, -2: no more units
    int zx, zy; // slice (batch, head) of X; of the first Y
    int x0;     // first row of X
    int y, n;   // first tile of Y, steps
    int first;  // kv unit: the first query tile of each head
    int split;
};

struct Bars {
    uint64_t x_full[2], x_empty[2];
    uint64_t y_full[kMaxSlots], y_empty[kMaxSlots];
    uint64_t st_full[kStatStages], st_empty[kStatStages];
    uint64_t t1_full[2], p_full[2];   // T1 computed; T1 read (q unit) or P written (kv unit)
    uint64_t t2_full[2], ds_full[2];  // T2 computed; dS written (of each buffer)
    uint64_t acc_full[2], acc_empty;  // A1 and A2 of a unit complete; both read
    uint64_t mma_done;
    uint64_t sched_full[kSchedRing], sched_empty[kSchedRing];
    uint64_t norm_full[kSchedRing];
    Unit sched_unit[kSchedRing];
    float norm[kSchedRing];  // fp16: a bound of the unit's |dS| (kv unit), the largest |v| (q unit)
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 896, "barrier block");

struct Params {
    const float *stats;
    const float *max_q, *max_v;  // fp16, of BwdPlan
    unsigned *counter;
    void *dk, *dv, *dq;               // gradients, or the splits' partial sums
    int BH, BHk, group, Sq, Skv, causal;
    int off, wrap, few;  // of BwdPlan
    int blind;           // first query rows of a head that see no key: behind tm_q's and tm_do's start
    int nq, nk, ns_kv, ns_q, q_first;
    int hg;       // kv slices per schedule group
    int n_units;
    int kv_f32, q_f32;  // fp32 output of dk and dv, of dq
    int wide;           // the outputs are 32-byte aligned
    float scale_log2, scale;
    int *status;
    unsigned long long timeout_ns;
};

// Unit u of the schedule: groups of hg kv slices; in a group first the kv units, then
// the q units (or the other way round, BwdPlan::q_first), longest first (causal: first key tiles, last query tiles).
__device__ __forceinline__ Unit decode_unit(int u, const Params &p) {
    Unit r;
    const int a_head = p.nk * p.ns_kv, b_head = p.group * p.nq * p.ns_q;
    const int per_group = p.hg * (a_head + b_head);
    const int g = u / per_group;
    int rem = u - g * per_group;
    const int heads = min(p.hg, p.BHk - g * p.hg);
    const bool skips = p.causal && !p.wrap;  // whole tiles that the mask leaves out
    const int n_first = heads * (p.q_first ? b_head : a_head);  // units of the kind that comes first
    const bool kv = p.q_first ? rem >= n_first : rem < n_first;
    if (rem >= n_first) rem -= n_first;
    if (kv) {
        const int width = heads * p.ns_kv;
        const int tile = rem / width;
        rem -= tile * width;
        const int head = rem / p.ns_kv;
        r.split = rem - head * p.ns_kv;
        r.kind = 0;
        r.zx = g * p.hg + head;
        r.x0 = tile * kRows;
        r.first = skips ? max(0, r.x0 - p.off) / kRows : 0;
        const int per = p.nq - r.first;  // query tiles of a head that see the tile
        const int64_t steps = (int64_t)per * p.group;
        const int t0 = (int)(steps * r.split / p.ns_kv), t1 = (int)(steps * (r.split + 1) / p.ns_kv);
        r.n = t1 - t0;
        const int skip = t0 / per;
        r.zy = r.zx * p.group + skip;
        r.y = r.first + t0 - skip * per;
    } else {
        const int width = heads * p.group * p.ns_q;
        int tile = rem / width;
        rem -= tile * width;
        const int head = rem / p.ns_q;
        r.split = rem - head * p.ns_q;
        if (p.causal) tile = p.nq - 1 - tile;
        r.kind = 1;
        r.zx = g * p.hg * p.group + head;
        r.zy = r.zx / p.group;
        r.x0 = tile * kRows;
        r.first = 0;
        const int end = skips ? min(p.Skv, min(r.x0 + kRows, p.Sq) + p.off) : p.Skv;
        const int steps = end > 0 ? (end + kRows - 1) / kRows : 0;
        const int t0 = (int)((int64_t)steps * r.split / p.ns_q), t1 = (int)((int64_t)steps * (r.split + 1) / p.ns_q);
        r.y = t0;
        r.n = t1 - t0;
    }
    return r;
}

// The next step's tile: key tiles in order; query tiles in order, head by head.
__device__ __forceinline__ void advance(const Unit &w, const Params &p, int &y, int &zy) {
    ++y;
    if (w.kind == 0 && y == p.nq) {
        y = w.first;
        ++zy;
    }
}

// fp16: what brings P dS' (P is kept times 2^14) to 2^14 at most where |dS'| <= most.
__device__ __forceinline__ float ds_scale_of(float most) {
    int e = 0;
    if (most > 0.f && most < INFINITY) e = max(-100, min(100, 13 - ilogbf(most)));
    return ldexpf(1.f, e - kBwdP16Log2);
}

template <bool kBF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (kBF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    } else {
        __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&h);
    }
}

__device__ __forceinline__ float4 ld_shared_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
}

// 32 bytes to global memory, as a whole sector where the address allows it.
__device__ __forceinline__ void st_global_v8(uint32_t *dst, const uint32_t *v, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]),
                     "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// One arrival for a whole warp, after what all its lanes did.
__device__ __forceinline__ void arrive_warp(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
}

// Untiled bulk copy into shared memory (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// What the rounding of x to `w` left, rounded itself.
template <bool kBF16>
__device__ __forceinline__ uint32_t pack_rest(float2 x, uint32_t w) {
    float2 h;
    if constexpr (kBF16) h = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else h = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return pack2<kBF16>(x.x - h.x, x.y - h.y);
}

// kTwo: what is held as the sum of two 16-bit numbers (BwdPlan::few).  0: nothing; 1: dS of the
// first p.few query tiles of each head; 2: P and dS throughout.
template <int D, bool kBF16, int kTwo>
__global__ void __launch_bounds__(kThreads, 1)
attn_bwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                   const Params p) {
    using C = Cfg<D>;
    constexpr int kSlots = C::kSlots1 + C::kSlots2;
    constexpr int kPer = kBF16 ? 2 : kScaleRows;  // numbers of a row's statistics
    // the tiles' swizzle needs 1024-byte alignment, which this declaration asks
    // for: there is no room to align by hand at D = 128
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars *bars = reinterpret_cast<Bars *>(smem + C::kOffBar);
    const uint32_t sX = ptx::smem_addr(smem + C::kOffX);
    const uint32_t sY = ptx::smem_addr(smem + C::kOffY);
    const uint32_t sStat = ptx::smem_addr(smem + C::kOffStat);
    if (sX & 1023) {  // never taken: the address is the same for every thread
        if (threadIdx.x == 0) atomicOr(p.status, kStatusTimeout);
        return;
    }

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const Watch watch{&bars->abort_flag, p.status, p.timeout_ns};
    auto bar = [&](uint64_t &b) { return ptx::smem_addr(&b); };

    // ---------------------------------------------------------------- setup
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(bar(bars->x_full[t]), 1);
            ptx::mbar_init(bar(bars->x_empty[t]), 1);
            ptx::mbar_init(bar(bars->t2_full[t]), 1);
            ptx::mbar_init(bar(bars->ds_full[t]), kComputeWarps);
            ptx::mbar_init(bar(bars->t1_full[t]), 1);
            ptx::mbar_init(bar(bars->p_full[t]), kComputeWarps);
        }
        for (int s = 0; s < kSlots; ++s) {
            ptx::mbar_init(bar(bars->y_full[s]), 1);
            ptx::mbar_init(bar(bars->y_empty[s]), 1);
        }
        for (int s = 0; s < kStatStages; ++s) {
            ptx::mbar_init(bar(bars->st_full[s]), 1);
            ptx::mbar_init(bar(bars->st_empty[s]), kComputeWarps);
        }
        for (int t = 0; t < 2; ++t) ptx::mbar_init(bar(bars->acc_full[t]), 1);
        ptx::mbar_init(bar(bars->acc_empty), kComputeWarps);
        ptx::mbar_init(bar(bars->mma_done), 1);
        for (int s = 0; s < kSchedRing; ++s) {
            ptx::mbar_init(bar(bars->sched_full[s]), 1);
            ptx::mbar_init(bar(bars->sched_empty[s]), kSchedReaders + (kBF16 ? 0 : 1));
            ptx::mbar_init(bar(bars->norm_full[s]), 1);
        }
        bars->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == kProducerWarp && lane == 0) {
        ptx::prefetch_tmap(&tm_q);
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
        ptx::prefetch_tmap(&tm_do);
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_addr(&bars->tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    // Launched while the kernel of the row statistics still runs: nothing of it, or of
    // what came before it, is read above.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);

    // The producer's k-th claim for a consumer warp, and the unit's norm where one is asked
    // for; false if the CTA is aborting.
    auto next_unit = [&](uint32_t &k, Unit &w, float *norm = nullptr) {
        const uint32_t s = k % kSchedRing;
        if (!__all_sync(0xffffffffu, watch.wait(bar(bars->sched_full[s]), (k / kSchedRing) & 1)))
            return false;
        const volatile Unit *su = &bars->sched_unit[s];
        w.kind = su->kind;
        w.zx = su->zx;
        w.zy = su->zy;
        w.x0 = su->x0;
        w.y = su->y;
        w.n = su->n;
        w.first = su->first;
        w.split = su->split;
        if (norm && w.kind >= 0) {
            if (!__all_sync(0xffffffffu, watch.wait(bar(bars->norm_full[s]), (k / kSchedRing) & 1))) return false;
            *norm = *(const volatile float *)&bars->norm[s];
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(bars->sched_empty[s]));
        ++k;
        return true;
    };

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer
        ptx::setmaxnreg_dec<kOtherRegs>();
        if (lane == 0) {
            uint32_t yn[2] = {0, 0}, xn[2] = {0, 0}, sn = 0;  // tiles of each Y and X, statistics loaded
            bool ok = true;
            auto stop = [&]() {
                *watch.abort_flag = 1;
                return false;
            };
            // rows from `row` on of slice z of q or do, or of k or v
            auto tile = [&](uint32_t dst, uint64_t &full, const CUtensorMap *tm, int row, int z, bool of_q) {
                if (!in_bounds(row >= 0 && row < (of_q ? p.Sq : p.Skv) && z >= 0 && z < (of_q ? p.BH : p.BHk), p.status))
                    return stop();
                ptx::mbar_arrive_expect_tx(bar(full), C::kTileBytes);
                for (int c = 0; c < C::kChunks; ++c)
                    ptx::tma_load_3d(dst + c * C::kChunkBytes, tm, bar(full), c * 64, of_q ? row - p.blind : row, z);
                return true;
            };
            auto load_x = [&](int t, const Unit &w) {
                if (!watch.wait(bar(bars->x_empty[t]), (xn[t] & 1) ^ 1)) return false;
                const CUtensorMap *tm = w.kind == 0 ? (t ? &tm_v : &tm_k) : (t ? &tm_do : &tm_q);
                if (!tile(sX + t * C::kTileBytes, bars->x_full[t], tm, w.x0, w.zx, w.kind != 0)) return false;
                ++xn[t];
                return true;
            };
            auto load_y = [&](int t, const Unit &w, int y, int zy) {
                const uint32_t s = C::slot(t, yn[t]);
                if (!watch.wait(bar(bars->y_empty[s]), (C::round(t, yn[t]) & 1) ^ 1)) return false;
                const CUtensorMap *tm = w.kind == 0 ? (t ? &tm_do : &tm_q) : (t ? &tm_v : &tm_k);
                if (!tile(sY + s * C::kTileBytes, bars->y_full[s], tm, y * kRows, zy, w.kind == 0)) return false;
                ++yn[t];
                return true;
            };
            auto load_stat = [&](int y, int zy) {
                const int s = sn % kStatStages;
                if (!watch.wait(bar(bars->st_empty[s]), ((sn / kStatStages) & 1) ^ 1)) return false;
                if (!in_bounds(y >= 0 && y < p.nq && zy >= 0 && zy < p.BH, p.status)) return stop();
                ptx::mbar_arrive_expect_tx(bar(bars->st_full[s]), C::kStatBytes);
                bulk_load(sStat + s * C::kStatBytes, p.stats + ((size_t)zy * p.nq + y) * kPer * kStatTile,
                          C::kStatBytes, bar(bars->st_full[s]));
                ++sn;
                return true;
            };
            unsigned claim = atomicAdd(p.counter, 1u);
            for (uint32_t k = 0; ok; ++k) {
                const uint32_t slot = k % kSchedRing;
                if (!watch.wait(bar(bars->sched_empty[slot]), ((k / kSchedRing) & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                Unit w{-2, 0, 0, 0, 0, 0, 0, 0};
                if (claim < (unsigned)p.n_units) w = decode_unit((int)claim, p);
                volatile Unit *su = &bars->sched_unit[slot];
                su->kind = w.kind;
                su->zx = w.zx;
                su->zy = w.zy;
                su->x0 = w.x0;
                su->y = w.y;
                su->n = w.n;
                su->first = w.first;
                su->split = w.split;
                ptx::mbar_arrive(bar(bars->sched_full[slot]));
                if (w.kind < 0) break;
                int y = w.y, zy = w.zy;
                for (int i = 0; i < w.n && ok; ++i) {
                    if (i == 0) ok = load_x(0, w);
                    ok = ok && load_y(0, w, y, zy);
                    if (w.kind == 0) ok = ok && load_stat(y, zy);
                    if (i == 0) ok = ok && load_x(1, w);
                    ok = ok && load_y(1, w, y, zy);
                    advance(w, p, y, zy);
                }
                if (ok) claim = atomicAdd(p.counter, 1u);
            }
            // teardown: every load this thread issued has landed
            for (int t = 0; t < 2; ++t)
                for (uint32_t s = 0; s < (uint32_t)C::slots(t) && s < yn[t]; ++s) {
                    const uint32_t last = s + ((yn[t] - 1 - s) / C::slots(t)) * C::slots(t);
                    watch.drain(bar(bars->y_full[C::slot(t, last)]), C::round(t, last) & 1);
                }
            for (uint32_t s = 0; s < (uint32_t)kStatStages && s < sn; ++s) {
                const uint32_t last = s + ((sn - 1 - s) / kStatStages) * kStatStages;
                watch.drain(bar(bars->st_full[s]), (last / kStatStages) & 1);
            }
            for (int t = 0; t < 2; ++t)
                if (xn[t] > 0) watch.drain(bar(bars->x_full[t]), (xn[t] - 1) & 1);
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        ptx::setmaxnreg_dec<kOtherRegs>();
        auto wait_all = [&](uint64_t &b, uint32_t parity) {
            return __all_sync(0xffffffffu, watch.wait(bar(b), parity));
        };
        constexpr uint32_t kIdescT = idesc_f16(kBF16, kRows, kRows, false);
        constexpr uint32_t kIdescA = idesc_f16(kBF16, kRows, D, true);
        const uint64_t dx = sdesc(sX, 16, 1024);
        const uint64_t dyk = sdesc(sY, 16, 1024);              // Y as [rows of the result's columns][channels]
        const uint64_t dyn = sdesc(sY, C::kChunkBytes, 1024);  // Y as [summed rows][channels of the result]
        uint32_t pos = 0;             // steps of the units before: tiles of Y1 and of Y2
        uint32_t xn = 0, un = 0;      // units begun, units whose sums were begun
        uint32_t pn[2] = {0, 0}, dn[2] = {0, 0};  // p_full and ds_full phases waited for
        bool ok = true;
        auto slot_full = [&](int t, uint32_t n) { return wait_all(bars->y_full[C::slot(t, n)], C::round(t, n) & 1); };
        auto free_slot = [&](int t, uint32_t n) { ptx::mma_commit_warp(bar(bars->y_empty[C::slot(t, n)])); };
        // T = X_t Y_t^T, Y_t its n-th tile
        auto issue_t = [&](uint32_t col, int t, uint32_t n) {
            const uint64_t da = dx + (uint64_t)((t * C::kTileBytes) >> 4);
            const uint64_t db = dyk + (uint64_t)((C::slot(t, n) * C::kTileBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4;
                ptx::mma_ss_warp(tmem + col, da + o, db + o, kIdescT, kk > 0 ? 1u : 0u);
            }
        };
        // A += (16-bit rows at column `col`) Y_t
        auto issue_a = [&](uint32_t acc, uint32_t col, int t, uint32_t n, bool add) {
            const uint64_t db = dyn + (uint64_t)((C::slot(t, n) * C::kTileBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kRows / 16; ++kk)
                ptx::mma_ts_warp(tmem + acc, tmem + col + (kk >> 2) * 64 + (kk & 3) * 8,
                                 db + (uint64_t)((kk * 16 * 128) >> 4), kIdescA, (add || kk > 0) ? 1u : 0u);
        };
        for (uint32_t k = 0; ok;) {
            Unit w;
            if (!next_unit(k, w)) { ok = false; break; }
            if (w.kind < 0) break;
            const int n = w.n;
            if (n == 0) continue;
            const bool kv = w.kind == 0;
            bool acc_free = false;
            auto need_acc = [&]() {  // the previous unit's sums have been read
                if (!acc_free && !wait_all(bars->acc_empty, (un & 1) ^ 1)) return false;
                acc_free = true;
                return true;
            };
            // T1 and T2 of step i
            auto t1 = [&](int i) {
                if (!slot_full(0, pos + i)) return false;
                ptx::tc_fence_after();
                const int b = C::kTwoT1 && kv ? i & 1 : 0;
                issue_t(C::col_t1(b), 0, pos + i);
                ptx::mma_commit_warp(bar(bars->t1_full[b]));
                if (i == n - 1) ptx::mma_commit_warp(bar(bars->x_empty[0]));
                return true;
            };
            auto t2 = [&](int i) {
                const int buf = kv ? 0 : i & 1;
                if (!slot_full(1, pos + i)) return false;
                if (!C::kTwoT1 && buf == 1 && !need_acc()) return false;
                ptx::tc_fence_after();
                issue_t(C::col_t2(buf), 1, pos + i);
                ptx::mma_commit_warp(bar(bars->t2_full[buf]));
                if (!kv) free_slot(1, pos + i);
                if (i == n - 1) ptx::mma_commit_warp(bar(bars->x_empty[1]));
                return true;
            };
            ok = wait_all(bars->x_full[0], xn & 1) && t1(0) && wait_all(bars->x_full[1], xn & 1) && t2(0);
            ++xn;
            int y = kv ? w.y : w.x0 / kRows, zy = w.zy;  // the step's query tile (kTwo 1)
            for (int i = 0; i < n && ok; ++i) {
                const bool two = kTwo == 2 || (kTwo == 1 && y < p.few);
                const int b1 = C::kTwoT1 && kv ? i & 1 : 0;
                if (C::kTwoT1 && kv && i + 1 < n && !t1(i + 1)) { ok = false; break; }
                // P(i) is written, or T1(i) read
                if (!wait_all(bars->p_full[b1], (b1 ? pn[1] : pn[0]) & 1)) { ok = false; break; }
                if (b1) ++pn[1]; else ++pn[0];
                if (kv) {
                    if (!need_acc()) { ok = false; break; }
                    ptx::tc_fence_after();
                    issue_a(C::kColA1, C::col_t1(b1), 1, pos + i, i > 0);
                    if constexpr (kTwo == 2) issue_a(C::kColA1, C::col_t1(b1) + 32, 1, pos + i, true);
                    free_slot(1, pos + i);
                    if (i == n - 1) ptx::mma_commit_warp(bar(bars->acc_full[0]));
                }
                if (i + 1 < n) {
                    if (!C::kTwoT1 || !kv) ok = t1(i + 1);
                    if (ok && !kv) ok = t2(i + 1);
                    if (!ok) break;
                }
                const int buf = kv ? 0 : i & 1;
                if (!wait_all(bars->ds_full[buf], (buf ? dn[1] : dn[0]) & 1) || !need_acc()) { ok = false; break; }
                if (buf) ++dn[1]; else ++dn[0];
                ptx::tc_fence_after();
                issue_a(C::kColA2, C::col_t2(buf), 0, pos + i, i > 0);
                if (two) issue_a(C::kColA2, C::col_t2(buf) + 32, 0, pos + i, true);
                free_slot(0, pos + i);
                if (kv && i + 1 < n) ok = t2(i + 1);
                if (kTwo == 1 && kv) advance(w, p, y, zy);
            }
            if (!ok) break;
            ptx::mma_commit_warp(bar(bars->acc_full[1]));
            ++un;
            pos += n;
        }
        ptx::mma_commit_warp(bar(bars->mma_done));
        watch.drain(bar(bars->mma_done), 0);
        __syncwarp();
    } else if (warp < kProducerWarp) {
        // ------------------------------------------------------------ P, dS, sums out
        ptx::setmaxnreg_inc<kComputeRegs>();
        const int half = warp >> 2;  // columns [64 half, 64 half + 64) of T1 and T2
        const int r = (warp & 3) * 32 + lane;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        float norm = 0.f, ds_scale = 1.f;  // fp16: of the unit, of this thread's row
        uint32_t n1[2] = {0, 0}, n2[2] = {0, 0}, sn = 0, an[2] = {0, 0};
        bool ok = true;

        // The steps of one unit, one row and 64 columns a thread.
        auto steps = [&](auto kind, const Unit &w) {
            constexpr bool KV = decltype(kind)::value;
            const int row = w.x0 + r;
            const int off = p.off;
            // q unit: this row's position, and the first key that a row of the tile may not see
            const int pos = p.wrap ? row % p.wrap : row;
            const int sees = KV ? 0 : min(p.Skv, p.causal ? pos + off + 1 : p.Skv);
            const int all_see = KV ? 0 : min(p.Skv, p.causal ? (p.wrap ? 0 : w.x0) + off + 1 : p.Skv);
            const float2 sc = make_float2(p.scale_log2, p.scale_log2);
            float rl = 0.f, rd = 0.f;  // q unit: nl and nd of this thread's row
            if constexpr (!KV) {
                const float *st = p.stats + ((size_t)w.zx * p.nq + w.x0 / kRows) * kPer * kStatTile + r;
                if (in_bounds(w.zx < p.BH && w.x0 / kRows < p.nq, p.status)) {
                    rl = st[0];
                    rd = st[kStatTile];
                    if constexpr (!kBF16) ds_scale = ds_scale_of(fmaf(st[2 * kStatTile], norm, fabsf(rd)));
                }
            } else if constexpr (!kBF16) {
                ds_scale = ds_scale_of(norm);
            }
            int y = w.y, zy = w.zy;
            auto one = [&](auto two, int i) {
                constexpr bool kRest = decltype(two)::value;  // dS in two parts
                const int y0 = y * kRows;
                const int stage = sn % kStatStages;
                [[maybe_unused]] const uint32_t st = sStat + stage * C::kStatBytes + half * 256;
                bool got = true;
                if constexpr (KV) got = watch.wait(bar(bars->st_full[stage]), (sn / kStatStages) & 1);
                const int b1 = C::kTwoT1 && KV ? i & 1 : 0;
                got = watch.wait(bar(bars->t1_full[b1]), (b1 ? n1[1] : n1[0]) & 1) && got;
                if (b1) ++n1[1]; else ++n1[0];
                if (!__all_sync(0xffffffffu, got)) return false;
                ptx::tc_fence_after();
                uint32_t a[2][32];
                const uint32_t tT1 = tl + C::col_t1(b1) + half * 64;
                ptx::tmem_ld32(tT1, a[0]);
                ptx::tmem_ld32(tT1 + 32, a[1]);
                ptx::tmem_wait_ld();
                reg_fence(a[0]);
                reg_fence(a[1]);
                if constexpr (!KV) {  // T1 is read: the next one may be written
                    ptx::tc_fence_before();
                    arrive_warp(bar(bars->p_full[b1]), lane);
                }
                const bool masked = KV ? p.causal && w.x0 + kRows - 1 > (p.wrap ? 0 : y0) + off : y0 + kRows > all_see;
                if (masked) {  // scores of pairs that do not see each other: -inf
                    if (KV && p.wrap) {
                        int at = (y0 + half * 64) % p.wrap;  // position of the query of column j
#pragma unroll
                        for (int j = 0; j < 64; ++j) {
                            if (row > at + off) a[j >> 5][j & 31] = __float_as_uint(-INFINITY);
                            if (++at == p.wrap) at = 0;
                        }
                    } else {
                        // columns visible to the row: from lo on, or below hi
                        const int lo = row - off - y0 - half * 64, hi = sees - y0 - half * 64;
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (KV ? j < lo : j >= hi) a[j >> 5][j & 31] = __float_as_uint(-INFINITY);
                    }
                }
                float2 pr[32];
                uint32_t pk[32], rest[kRest ? 32 : 1];
                // P = exp2(scores)
                auto weights = [&](int j) {
                    const uint32_t *s = &a[j >> 4][(2 * j) & 31];
                    float4 l = make_float4(rl, rl, rl, rl);
                    if constexpr (KV) l = ld_shared_v4(st + j * 8);
                    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[0]), __uint_as_float(s[1])), sc, make_float2(l.x, l.y));
                    const float2 z = __ffma2_rn(make_float2(__uint_as_float(s[2]), __uint_as_float(s[3])), sc, make_float2(l.z, l.w));
                    pr[j] = make_float2(ptx::ex2_approx(x.x), ptx::ex2_approx(x.y));
                    pr[j + 1] = make_float2(ptx::ex2_approx(z.x), ptx::ex2_approx(z.y));
                };
                if constexpr (KV) {
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        weights(j);
                        pk[j] = pack2<kBF16>(pr[j].x, pr[j].y);
                        pk[j + 1] = pack2<kBF16>(pr[j + 1].x, pr[j + 1].y);
                        if constexpr (kTwo == 2) {
                            rest[j] = pack_rest<kBF16>(pr[j], pk[j]);
                            rest[j + 1] = pack_rest<kBF16>(pr[j + 1], pk[j + 1]);
                        }
                    }
                    ptx::tmem_st32(tT1, pk);
                    if constexpr (kTwo == 2) ptx::tmem_st32(tT1 + 32, rest);
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before();
                    arrive_warp(bar(bars->p_full[b1]), lane);
                }
                const int buf = KV ? 0 : i & 1;
                got = watch.wait(bar(bars->t2_full[buf]), (buf ? n2[1] : n2[0]) & 1);
                if (buf) ++n2[1]; else ++n2[0];
                if (!__all_sync(0xffffffffu, got)) return false;
                ptx::tc_fence_after();
                const uint32_t tT2 = tl + C::col_t2(buf) + half * 64;
                uint32_t b[2][32];
                ptx::tmem_ld32(tT2, b[0]);
                ptx::tmem_ld32(tT2 + 32, b[1]);
                ptx::tmem_wait_ld();
                reg_fence(b[0]);
                reg_fence(b[1]);
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    if constexpr (!KV) weights(j);  // both tiles are here: exponentials and products mixed
                    const uint32_t *s = &b[j >> 4][(2 * j) & 31];
                    float4 l = make_float4(rd, rd, rd, rd);
                    if constexpr (KV) l = ld_shared_v4(st + kStatTile * 4 + j * 8);
                    float2 x = __fadd2_rn(make_float2(__uint_as_float(s[0]), __uint_as_float(s[1])), make_float2(l.x, l.y));
                    float2 z = __fadd2_rn(make_float2(__uint_as_float(s[2]), __uint_as_float(s[3])), make_float2(l.z, l.w));
                    if constexpr (!kBF16) {
                        x = __fmul2_rn(x, make_float2(ds_scale, ds_scale));
                        z = __fmul2_rn(z, make_float2(ds_scale, ds_scale));
                    }
                    x = __fmul2_rn(x, pr[j]);
                    z = __fmul2_rn(z, pr[j + 1]);
                    pk[j] = pack2<kBF16>(x.x, x.y);
                    pk[j + 1] = pack2<kBF16>(z.x, z.y);
                    if constexpr (kRest) {
                        rest[j] = pack_rest<kBF16>(x, pk[j]);
                        rest[j + 1] = pack_rest<kBF16>(z, pk[j + 1]);
                    }
                }
                ptx::tmem_st32(tT2, pk);
                if constexpr (kRest) ptx::tmem_st32(tT2 + 32, rest);
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                arrive_warp(bar(bars->ds_full[buf]), lane);
                if constexpr (KV) {
                    if (lane == 0) ptx::mbar_arrive(bar(bars->st_empty[stage]));
                    ++sn;
                }
                advance(w, p, y, zy);
                return true;
            };
            for (int i = 0; i < w.n; ++i) {
                if (kTwo == 1 && (KV ? y : w.x0 / kRows) < p.few) {
                    if (!one(std::bool_constant<(kTwo > 0)>{}, i)) return false;
                } else if (!one(std::bool_constant<kTwo == 2>{}, i)) {
                    return false;
                }
            }
            return true;
        };

        for (uint32_t k = 0; ok;) {
            Unit w;
            if (!next_unit(k, w, kBF16 ? nullptr : &norm)) { ok = false; break; }
            if (w.kind < 0) break;
            const bool kv = w.kind == 0;
            const int row = w.x0 + r;
            ok = kv ? steps(std::true_type{}, w) : steps(std::false_type{}, w);
            if (!ok) break;

            // ---- the unit's sums: dv (while A2 of the last step runs) and dk, or dq
            const int rows = kv ? p.Skv : p.Sq;
            const int64_t slices = kv ? p.BHk : p.BH;
            const bool f32 = kv ? p.kv_f32 : p.q_f32;
            const size_t part = (size_t)w.split * slices * rows;  // rows of the splits before
            const size_t extent = (size_t)slices * rows * (kv ? p.ns_kv : p.ns_q) * D;
            const size_t at = (part + (size_t)w.zx * rows + row) * D + half * (D / 2);
#pragma unroll 1
            for (int m = kv ? 0 : 1; m < 2; ++m) {  // 0: A1 (dv), 1: A2 (dk or dq)
                if (w.n > 0) {
                    const bool got = watch.wait(bar(bars->acc_full[m]), (m ? an[1] : an[0]) & 1);
                    if (m) ++an[1]; else ++an[0];
                    if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
                    ptx::tc_fence_after();
                }
                void *dst = m == 0 ? p.dv : kv ? p.dk : p.dq;
                const float f = m == 0 ? (kBF16 ? 1.f : 1.f / (1 << kBwdP16Log2))
                                       : (kBF16 ? p.scale : p.scale / (ds_scale * (1 << kBwdP16Log2)));
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t o[32];
                    __syncwarp();
                    if (w.n > 0) {
                        ptx::tmem_ld32(tl + (m == 0 ? C::kColA1 : C::kColA2) + half * (D / 2) + c * 32, o);
                        ptx::tmem_wait_ld();
                        reg_fence(o);
                        if (m == 1 && c == D / 64 - 1) {  // read: the next unit's sums may begin
                            ptx::tc_fence_before();
                            arrive_warp(bar(bars->acc_empty), lane);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                    }
                    const size_t g = at + c * 32;
                    if (row >= rows || !in_bounds(g + 32 <= extent, p.status)) continue;
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                    if (f32) {
                        uint32_t *d = reinterpret_cast<uint32_t *>(dst) + g;
#pragma unroll
                        for (int i = 0; i < 32; i += 8) st_global_v8(d + i, o + i, p.wide);
                    } else {
                        uint32_t *d = reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(dst) + g);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = pack2<kBF16>(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
#pragma unroll
                        for (int i = 0; i < 16; i += 8) st_global_v8(d + i, o + i, p.wide);
                    }
                }
            }
        }
    } else {
        // the other warps only give up their registers, but for fp16's norms
        ptx::setmaxnreg_dec<kOtherRegs>();
        if (!kBF16 && warp == kScaleWarp) {
            for (uint32_t k = 0;;) {
                const uint32_t s = k % kSchedRing;
                Unit w;
                if (!next_unit(k, w) || w.kind < 0) break;
                float a = 0.f, d = 0.f, v = 0.f;
                if (w.kind == 0) {
                    const int per = p.nq - w.first;
                    for (int i = lane; i < w.n; i += 32) {
                        const int t = w.y - w.first + i, head = w.zy + t / per, y = w.first + t % per;
                        if (!in_bounds(head < p.BH && y < p.nq, p.status)) break;
                        const float2 m = reinterpret_cast<const float2 *>(p.max_q)[(size_t)head * p.nq + y];
                        a = fmaxf(a, m.x);
                        d = fmaxf(d, m.y);
                    }
                    v = p.max_v[(size_t)w.zx * p.nk + w.x0 / kRows];
                } else {
                    for (int i = lane; i < w.n; i += 32) {
                        if (!in_bounds(w.zy < p.BHk && w.y + i < p.nk, p.status)) break;
                        v = fmaxf(v, p.max_v[(size_t)w.zy * p.nk + w.y + i]);
                    }
                }
                for (int m = 16; m > 0; m >>= 1) {
                    a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
                    d = fmaxf(d, __shfl_xor_sync(0xffffffffu, d, m));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
                }
                if (lane == 0) {
                    *(volatile float *)&bars->norm[s] = w.kind == 0 ? fmaf(a, v, d) : v;
                    ptx::mbar_arrive(bar(bars->norm_full[s]));
                }
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool kBF16, int kTwo>
int launch_typed(const BwdArgs &a, const Problem &pr, const BwdPlan &plan, cudaStream_t stream) {
    using C = Cfg<D>;
    // Rows that see no key have P = 0, which makes no 0 of an infinity that their do leaves in
    // dP: the maps of q and do start behind them, so that they read as zeros.  (Clearing dP
    // where it is read cost 4 % of every call.)
    const int blind = pr.causal && plan.off < 0 ? -plan.off : 0;
    const size_t skip = (size_t)blind * D * 2;
    CUtensorMap tq, tk, tv, td;
    if (!make_tile_map(&tq, (const uint8_t *)a.q + skip, kBF16, D, pr.Sq, pr.Sq - blind, pr.bh()) ||
        !make_tile_map(&tk, a.k, kBF16, D, pr.Skv, pr.Skv, pr.bh_kv()) ||
        !make_tile_map(&tv, a.v, kBF16, D, pr.Skv, pr.Skv, pr.bh_kv()) ||
        !make_tile_map(&td, (const uint8_t *)a.dout + skip, kBF16, D, pr.Sq, pr.Sq - blind, pr.bh()))
        return ATTN_ERR_CUDA;
    uint8_t *ws = (uint8_t *)a.workspace;
    Params p{};
    p.stats = (const float *)(ws + plan.off_stats);
    p.max_q = (const float *)(ws + plan.off_max);
    p.max_v = (const float *)(ws + plan.off_max_v);
    p.counter = (unsigned *)ws;
    p.BH = (int)pr.bh();
    p.BHk = (int)pr.bh_kv();
    p.group = pr.group;
    p.Sq = pr.Sq;
    p.Skv = pr.Skv;
    p.causal = pr.causal;
    p.off = plan.off;
    p.wrap = plan.wrap;
    p.few = plan.few;
    p.blind = blind;
    p.nq = plan.nq;
    p.nk = plan.nk;
    p.ns_kv = plan.ns_kv;
    p.ns_q = plan.ns_q;
    p.q_first = plan.q_first;
    p.n_units = (int)plan.n_units;
    p.scale_log2 = pr.scale * 1.4426950408889634f;
    p.scale = pr.scale;
    const int out_f32 = elem_bytes_out(pr.dtype) == 4;
    p.kv_f32 = out_f32 || plan.ns_kv > 1;
    p.q_f32 = out_f32 || plan.ns_q > 1;
    float *part_kv = (float *)(ws + plan.off_part_kv);
    p.dk = plan.ns_kv > 1 ? part_kv : a.dk;
    p.dv = plan.ns_kv > 1 ? part_kv + (size_t)plan.ns_kv * pr.bh_kv() * pr.Skv * D : a.dv;
    p.dq = plan.ns_q > 1 ? (void *)(ws + plan.off_part_q) : a.dq;
    p.wide = ((uintptr_t)p.dk | (uintptr_t)p.dv | (uintptr_t)p.dq) % 32 == 0;
    const int sms = device_sm_count();
    p.status = status_word_device_ptr();
    if (sms <= 0 || !p.status) return ATTN_ERR_CUDA;
    {
        // kv slices per group: about one and a half rounds of units, as equal groups where
        // that is possible; all slices otherwise, unless their tiles exceed what L2 holds
        const int64_t units = (int64_t)plan.nk * plan.ns_kv + (int64_t)pr.group * plan.nq * plan.ns_q;
        const int64_t h0 = (3 * sms / 2 + units - 1) / units;
        int64_t hg = h0 < 1 ? 1 : h0;
        while (hg < p.BHk && p.BHk % hg != 0) ++hg;
        const int64_t bytes = 4LL * D * (pr.bh() * pr.Sq + pr.bh_kv() * pr.Skv);
        if (hg >= p.BHk && bytes > (96LL << 20)) hg = h0;
        if (hg > p.BHk) hg = p.BHk;
        p.hg = (int)hg;
    }
    p.timeout_ns = watchdog_ns();
    auto kern = attn_bwd_tc_kernel<D, kBF16, kTwo>;
    // setmaxnreg needs exactly the registers it was planned for (see the forward kernel)
    static std::atomic<int> regs_ok{-1};
    int ok = regs_ok.load(std::memory_order_relaxed);
    if (ok < 0) {
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return ATTN_ERR_UNSUPPORTED_DEVICE;
        ok = (fa.numRegs == kLaunchRegs && fa.maxThreadsPerBlock >= kThreads) ? 1 : 0;
        regs_ok.store(ok, std::memory_order_relaxed);
    }
    if (!ok) return ATTN_ERR_LAUNCH;
    if (!set_smem_limit_once(reinterpret_cast<const void *>(kern), C::kSmemBytes)) return ATTN_ERR_LAUNCH;
    const int grid = (int)(plan.n_units < sms ? plan.n_units : sms);
    // starts its set-up before the row statistics are complete (see the kernel)
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    (void)cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, td, p);
    const cudaError_t e = cudaGetLastError();
    if (e == cudaErrorNoKernelImageForDevice || e == cudaErrorInvalidDeviceFunction)
        return ATTN_ERR_UNSUPPORTED_DEVICE;
    return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

template <int D, bool kBF16>
int launch_two(const BwdArgs &a, const Problem &pr, const BwdPlan &plan, cudaStream_t stream) {
    if (pr.Skv <= kFewKeys) return launch_typed<D, kBF16, 2>(a, pr, plan, stream);
    if (plan.few) return launch_typed<D, kBF16, 1>(a, pr, plan, stream);
    return launch_typed<D, kBF16, 0>(a, pr, plan, stream);
}

}  // namespace

int launch_bwd_tc(const BwdArgs &a, const BwdPlan &plan, cudaStream_t stream) {
    const Problem &p = plan.p;
    const bool bf16 = p.dtype == ATTN_BF16 || p.dtype == ATTN_BF16_OUT_F32;
    if (p.d == 128)
        return bf16 ? launch_two<128, true>(a, p, plan, stream) : launch_two<128, false>(a, p, plan, stream);
    if (p.d == 64)
        return bf16 ? launch_two<64, true>(a, p, plan, stream) : launch_two<64, false>(a, p, plan, stream);
    return ATTN_ERR_INVALID_ARG;
}

}  // namespace attn
