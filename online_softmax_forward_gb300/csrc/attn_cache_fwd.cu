// attn_cache_fwd.cu -- attention of a few query rows per sequence over the
// paged 8-bit cache, over all pages or over a list of pages per query.
//
//     s_j = scale * k_scale[page(j)] * (q . kcode_j)
//     o   = sum_j softmax_j(s) * v_scale[page(j)] * vcode_j
//
// Work.  A unit is (sequence, kv head, block of query rows): the G query heads
// of a kv head share its keys, so the rows of a block are (query, head of the
// group).  Its keys are walked in tiles of KT keys (a page, or 64 of its 128).
// All tiles of a call are numbered through and cut into equal contiguous
// ranges, one per warp (cache_index.h): ragged lengths and few sequences fill
// the GPU alike.  A warp writes the units it covers alone.  Of the units that
// several warps of a CTA share the states are joined in shared memory, and a
// second kernel joins the at most one unit that runs over the end of each CTA's
// range, with the online softmax's merge of states.
//
// Products.  The 8-bit codes are exact in fp16, so both products run on
// mma.m16n8k16 with fp32 accumulation and no dequantised tile exists
// anywhere: the page's scales multiply the scores and the page's share of o.
// A decode step is bound by reading the codes; of the 16 rows of the MMA few
// carry queries, which costs nothing that is scarce here.
//   8-row form: rows 0-7 are query rows, rows 8-15 the same rows' rounding
//     remainders: q = hi + lo (lo = 0 unless q is fp32) and p = hi + lo, so the
//     products are those of 22-bit numbers and fp32 outputs keep their digits.
//   16-row form (bf16 output, more than 8 rows): p is rounded once to fp16
//     (2^-12, against the output's 2^-9).
// q rows are first multiplied by a power of two that puts the row's largest
// magnitude in [2^14, 2^15): any fp32 or bf16 exponent then fits fp16.
//
// Softmax.  The sums l and o are kept relative to a reference `top` of the
// scores and, o, to a reference 2^11 / rv of the page scales, so the weight that
// enters the second product is p * v_scale * rv.  Both references move only when
// a step of 16 keys would pass fp16's range or a weight 2^4: one vote a step, no
// maximum across lanes and no rescaling in the others.
//
// Loads.  Each warp copies its own tiles into a ring of shared memory slots with
// 16-byte cp.async (a slot holds the codes of one tile's keys or values), all
// slots but the one in use in flight, and waits for nobody else.  The MMA's k
// index may name the channels in any order that q and k share, and its n index
// any channel of v: lane (g, t) = (lane / 4, lane % 4) reads D/4 consecutive
// bytes of key row g, and D/8 consecutive bytes of value rows 2t, 2t+1, 2t+8,
// 2t+9.  The 16-byte pieces of a row are swizzled so that both reads are free of
// bank conflicts.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_internal.h"
#include "cache_codec.cuh"
#include "cache_index.h"

namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = 24 * 1024;  // shared memory of each warp's tiles, later of its states
constexpr int kMinTiles = 1;  // tiles per worker when there are few

struct FwdArgs {
    const void *q;
    void *o;
    float *lse;
    const uint8_t *k, *v;
    const float *ks, *vs;
    const int32_t *table, *lens, *counts, *pages;
    float *hold;      // [warp][R][D]: state of the unit a warp's range begins inside of, if more follows
    float *po, *pl;   // states of the CTAs' shared units by slot: [slot][R][D], [slot][R] (log2)
    int4 *tail;       // [2 * CTA]: the unit that runs over the end of a CTA's range
    int B, Hkv, G, Sq, page, n_pages, max_pages, n_sel, causal;
    int nseg, rows, nrb;  // row groups of a (sequence, kv head), rows of one, row blocks of one
    int dtype, workers;
    float sl2;  // scale * log2(e)
    int *status;
};

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
__device__ __forceinline__ uint4 lds16(uint32_t p) {
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(p));
    return u;
}
__device__ __forceinline__ void sts16_zero(uint32_t p) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(p), "r"(0) : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t p) {
    uint2 u;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(p));
    return u;
}
// Byte offset of 16-byte piece c of row r in a slot.  D = 128: pieces are
// exchanged within a row by r & 7; D = 64: within a pair of rows (128 bytes) by
// the pair's number.
template <int D>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    if constexpr (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
    else return (uint32_t)((r >> 1) * 128 + ((((r & 1) * 4 + c) ^ ((r >> 1 & 3) * 2)) << 4));
}
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Codes as fp16 pairs, exact.  e4m3: one conversion a pair, as cheap as any
// integer instruction (2 clocks a warp and SM quarter; moving the bits into place
// by hand takes four).  int8: 0x6400 + u is the fp16 1024 + u, u = code + 128.
template <int FMT>
struct Unpack;
template <>
struct Unpack<ATTN_CACHE_E4M3> {
    // bytes (0, 1) and (2, 3) of w
    __device__ __forceinline__ static void quad(uint32_t w, uint32_t &lo, uint32_t &hi) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
    }
};
template <>
struct Unpack<ATTN_CACHE_I8> {
    __device__ __forceinline__ static uint32_t less1152(uint32_t w) {  // 1024 + u -> u - 128
        const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&w),
                                  __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    __device__ __forceinline__ static void quad(uint32_t w, uint32_t &lo, uint32_t &hi) {
        const uint32_t u = w ^ 0x80808080u;
        lo = less1152(__byte_perm(u, 0x64646464u, 0x4140));
        hi = less1152(__byte_perm(u, 0x64646464u, 0x4342));
    }
};

// Where a tile's unit lies.
struct Unit {
    int b, hk, seg, rb;
    int64_t begin, end;  // its tiles
};

// Sequence lengths as tile counts, summed: prefix[b] tiles before sequence b.
__device__ void scan_lengths(const FwdArgs &a, int kt, int64_t *prefix, int64_t *warp_sums) {
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = threadIdx.x * per, b1 = min(a.B, b0 + per);
    auto tiles = [&](int b) {
        const int len0 = a.lens[b], cnt = a.counts ? a.counts[b] : a.Sq;
        const int len = clamp_len(len0, a.max_pages, a.page);
        if ((len != len0 || cnt < 0 || cnt > a.Sq) && blockIdx.x == 0)
            atomicOr(a.status, kStatusTable);
        return ((int64_t)len + kt - 1) / kt;
    };
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += tiles(b);
    int64_t incl = sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    int64_t at = incl - sum;
    for (int w = 0; w < warp; ++w) at += warp_sums[w];
    for (int b = b0; b < b1; ++b) {
        prefix[b] = at;
        at += tiles(b);
    }
    if (b0 < a.B && b1 == a.B) prefix[a.B] = at;
}

// The unit that tile x belongs to.
__device__ __forceinline__ Unit unit_of(const FwdArgs &a, const int64_t *prefix, int64_t tpu, int64_t x) {
    Unit u;
    const int per = a.nseg * a.nrb;
    int64_t idx, first, len;  // unit within the sequence, the sequence's first tile, tiles per unit
    if (a.pages) {
        const int64_t n = x / tpu, units = (int64_t)a.Hkv * per;
        u.b = (int)(n / units);
        idx = n % units;
        first = u.b * units * tpu;
        len = tpu;
    } else {
        const int64_t units = (int64_t)a.Hkv * per, y = x / units;
        int lo = 0, hi = a.B - 1;  // the last b with prefix[b] <= y
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= y) lo = mid; else hi = mid - 1;
        }
        u.b = lo;
        first = prefix[lo] * units;
        len = prefix[lo + 1] - prefix[lo];
        idx = (x - first) / len;
    }
    u.begin = first + idx * len;
    u.end = u.begin + len;
    u.hk = (int)(idx / per);
    u.seg = (int)(idx % per / a.nrb);
    u.rb = (int)(idx % a.nrb);
    return u;
}

// Query and head of row r of a unit; false past the group's rows.
template <int R>
__device__ __forceinline__ bool row_of(const FwdArgs &a, const Unit &u, int r, int &i, int &h) {
    const int row = u.rb * R + r;
    if (row >= a.rows) return false;
    const int g = a.pages ? row : row % a.G;
    i = a.pages ? u.seg : row / a.G;
    h = u.hk * a.G + g;
    return true;
}

struct Tile {  // one key tile, held by one lane
    int at;    // tile of KT keys in the pool, -1: nothing to read
    int key0;  // its first key's position in the sequence
    float ks, vs;
};

template <int R, int KT>
__device__ __forceinline__ Tile find_tile(const FwdArgs &a, const int64_t *prefix, int64_t tpu, int64_t x) {
    Tile d;
    d.at = -1;
    d.key0 = 0;
    d.ks = d.vs = 0.f;
    const Unit u = unit_of(a, prefix, tpu, x);
    const int in_page = a.page / KT;
    const int64_t t = x - u.begin;
    const int len = clamp_len(a.lens[u.b], a.max_pages, a.page);
    const int cnt = a.counts ? min(max(a.counts[u.b], 0), a.Sq) : a.Sq;
    int lp = (int)(t / in_page);
    const int sub = (int)(t % in_page);
    if (a.pages) {
        const int64_t list = ((int64_t)u.b * a.Hkv + u.hk) * a.nseg + u.seg;
        lp = a.pages[list * a.n_sel + lp];
        if (lp < -1 || lp >= a.max_pages) atomicOr(a.status, kStatusTable);
        if (lp < 0 || lp >= a.max_pages) return d;
    }
    // the block's last query that is one of the sequence's sees the most keys
    int first, last, h;
    row_of<R>(a, u, 0, first, h);
    row_of<R>(a, u, min(a.rows - u.rb * R, R) - 1, last, h);
    last = min(last, cnt - 1);
    const int seen = last < first ? 0 : visible_keys(len, cnt, last, a.causal);
    const int64_t key0 = (int64_t)lp * a.page + sub * KT;
    if (key0 >= seen) return d;
    d.key0 = (int)key0;
    const int phys = a.table[(int64_t)u.b * a.max_pages + lp];
    if (phys < 0 || phys >= a.n_pages) {
        atomicOr(a.status, kStatusTable);
        return d;
    }
    const int64_t ph = (int64_t)phys * a.Hkv + u.hk;
    d.at = (int)(ph * in_page + sub);
    d.ks = a.ks[ph];
    d.vs = a.vs[ph];
    return d;
}

__device__ __forceinline__ void load_q8(const FwdArgs &a, size_t i, float *f) {
    if (a.dtype == ATTN_F32) codec::load8<0>(a.q, i, f);
    else if (a.dtype == ATTN_BF16 || a.dtype == ATTN_BF16_OUT_F32) codec::load8<1>(a.q, i, f);
    else codec::load8<2>(a.q, i, f);
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

// Row of o and lse that row r of a unit is; false past the group's rows.
template <int R>
__device__ __forceinline__ bool out_row(const FwdArgs &a, const Unit &u, int r, size_t &row) {
    int i, h;
    if (!row_of<R>(a, u, r, i, h)) return false;
    row = ((size_t)u.b * a.Hkv * a.G + h) * a.Sq + i;
    return in_bounds(i < a.Sq && h < a.Hkv * a.G && u.b < a.B, a.status);
}
constexpr float kLn2 = 0.69314718055994530942f;

// `top` before the first key: any visible score is above it by more than the
// range of exp2, so that its weight comes out infinite and sets the references.
constexpr float kUnset = -3.0e38f;

// One output.
__device__ __forceinline__ void store_o(const FwdArgs &a, size_t i, float x) {
    if (a.dtype == ATTN_BF16) reinterpret_cast<__nv_bfloat16 *>(a.o)[i] = __float2bfloat16_rn(x);
    else if (a.dtype == ATTN_F16) reinterpret_cast<__half *>(a.o)[i] = __float2half_rn(x);
    else reinterpret_cast<float *>(a.o)[i] = x;
}

// WIDE = 0: the 8-row form, 1: the 16-row form.
template <int D, int FMT, int WIDE, int KT>
__global__ void __launch_bounds__(kThreads, 1) cache_fwd_kernel(const FwdArgs a) {
    using U = Unpack<FMT>;
    constexpr int R = WIDE ? 16 : 8;
    constexpr int H = WIDE ? 2 : 1;    // query rows per lane: g, and g + 8 in the 16-row form
    constexpr int QS = D / 16;         // k steps of Q.K
    constexpr int VT = D / 8;          // output tiles of 8 channels
    constexpr int HALF = KT * D;       // bytes of a tile's keys, then its values
    constexpr int SLOT = 2 * HALF;
    constexpr int NS = kRing / SLOT < 8 ? kRing / SLOT : 8;
    static_assert(NS >= 3 && R * D * 4 <= kRing, "a warp's ring later holds a state");
    extern __shared__ __align__(128) uint8_t sm[];
    int64_t *prefix = reinterpret_cast<int64_t *>(sm + kWarps * kRing);  // [B + 1]
    __shared__ int64_t warp_sums[kWarps];
    __shared__ float s_lse[kWarps][2][R];
    __shared__ Unit s_unit[kWarps][2];
    __shared__ const float *s_keep[kWarps][2];
    __shared__ int64_t s_end[kWarps];   // past the warp's last tile
    __shared__ int s_has[kWarps];       // bit 0: a state of a unit begun before, bit 1: of one that goes on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int64_t tpu = a.pages ? (int64_t)a.n_sel * (a.page / KT) : 0;
    const int64_t units = (int64_t)a.Hkv * a.nseg * a.nrb;  // of one sequence
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int64_t total;
    if (a.pages) {
        total = a.B * units * tpu;
        // lengths and counts out of range are reported here for a page list
        if (blockIdx.x == 0)
            for (int b = threadIdx.x; b < a.B; b += kThreads) {
                const int len = a.lens[b], cnt = a.counts ? a.counts[b] : a.Sq;
                if (len != clamp_len(len, a.max_pages, a.page) || cnt < 0 || cnt > a.Sq)
                    atomicOr(a.status, kStatusTable);
            }
    } else {
        scan_lengths(a, KT, prefix, warp_sums);
        __syncthreads();
        total = prefix[a.B] * units;
        // sequences without a token have no tile: o = 0, lse = -inf
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            if (prefix[b] != prefix[b + 1]) continue;
            const size_t row0 = (size_t)b * a.Hkv * a.G * a.Sq, n = (size_t)a.Hkv * a.G * a.Sq;
            const float z[8] = {};
            for (size_t e = threadIdx.x; e < n * (D / 8); e += kThreads) store_o8(a, row0 * D + e * 8, z);
            if (a.lse)
                for (size_t e = threadIdx.x; e < n; e += kThreads) a.lse[row0 + e] = -INFINITY;
        }
    }
    const int64_t workers = worker_count(total, a.workers, kMinTiles);
    const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
    int64_t x0 = 0, x1 = 0;
    if (w < workers && total > 0) {
        x0 = worker_begin(w, total, workers);
        x1 = worker_begin(w + 1, total, workers);
    }
    if (lane == 0) {
        s_has[warp] = 0;
        s_end[warp] = x1;
    }

    // tiles x0 + 32 n + lane, and the next 32
    Tile cur = {-1, 0, 0.f, 0.f}, nxt = cur;
    if (x0 + lane < x1) cur = find_tile<R, KT>(a, prefix, tpu, x0 + lane);

    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm + warp * kRing);
    // tile j of the range into ring buffer `buf`; cur holds the tiles base .. base + 31
    auto issue = [&](int j, int buf, int n_tiles, int base) {
        const int held = j - base;  // < 64
        const int at = __shfl_sync(0xffffffffu, held < 32 ? cur.at : nxt.at, held & 31);
        if (j < n_tiles && at >= 0) {
            const size_t src = (size_t)at * HALF + lane * 16;
            const uint32_t dst = ring + buf * SLOT;
#pragma unroll
            for (int e = 0; e < HALF / 512; ++e) {
                const int c = e * 32 + lane;
                const uint32_t to = dst + swizzled<D>(c / (D / 16), c % (D / 16));
                cp_async16(to, a.k + src + e * 512);
                cp_async16(to + HALF, a.v + src + e * 512);
            }
        }
        cp_async_commit();
    };
    const int n_tiles = (int)(x1 - x0);
    int put = NS - 1, get = 0;  // ring buffers: next to fill, next to read
#pragma unroll 1
    for (int j = 0; j < NS - 1; ++j) issue(j, j, n_tiles, 0);

    int64_t x = x0;
    while (x < x1) {
        const Unit u = unit_of(a, prefix, tpu, x);
        const int64_t xe = u.end < x1 ? u.end : x1;
        const int len = clamp_len(a.lens[u.b], a.max_pages, a.page);
        const int cnt = a.counts ? min(max(a.counts[u.b], 0), a.Sq) : a.Sq;

        // query fragments: k step w holds channels 4w .. 4w + 3 of the lane's D/4 channels
        uint32_t qa[QS][4];
        float cq[H];
        int lim[H];
        int low = 0x7fffffff;  // fewest keys any row of the block sees
#pragma unroll
        for (int hh = 0; hh < H; ++hh) {
            float f[D / 4];
            int i, h;
            const bool real = row_of<R>(a, u, g + 8 * hh, i, h);
            lim[hh] = real ? visible_keys(len, cnt, i, a.causal) : 0;
            if (real) {
                const size_t at = (((size_t)u.b * a.Hkv * a.G + h) * a.Sq + i) * D + t * (D / 4);
#pragma unroll
                for (int e = 0; e < D / 4; e += 8) load_q8(a, at + e, f + e);
            } else {
#pragma unroll
                for (int e = 0; e < D / 4; ++e) f[e] = 0.f;
            }
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < D / 4; ++e) amax = fmaxf(amax, fabsf(f[e]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // 2^up puts amax in [2^14, 2^15); 0 and infinity stay as they are
            int up = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
            up = up > 126 ? 126 : up;
            if (amax == 0.f || !(amax <= 3.402823466e38f)) up = 0;
            const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
            cq[hh] = a.sl2 * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int s = 0; s < QS; ++s) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = f[4 * s + e] * mul;
                qa[s][hh] = pack_f16(y[0], y[1]);
                qa[s][hh + 2] = pack_f16(y[2], y[3]);
                if constexpr (!WIDE) {
                    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&qa[s][0]));
                    const float2 r = __half22float2(*reinterpret_cast<const __half2 *>(&qa[s][2]));
                    qa[s][1] = pack_f16(y[0] - p.x, y[1] - p.y);
                    qa[s][3] = pack_f16(y[2] - r.x, y[3] - r.y);
                }
            }
            if (real) low = min(low, lim[hh]);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, o));

        // l and acc relative to `top` and rv; the first key seen sets both
        float top[H], rv[H], l[H], acc[VT][4];
#pragma unroll
        for (int hh = 0; hh < H; ++hh) {
            top[hh] = kUnset;
            rv[hh] = 0x1p111f;
            l[hh] = 0.f;
        }
#pragma unroll
        for (int n = 0; n < VT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;

#pragma unroll 1
        for (; x < xe; ++x) {
            const int i = (int)(x - x0);
            if ((i & 31) == 0) {
                if (i > 0) cur = nxt;
                nxt.at = -1;
                if (x + 32 + lane < x1) nxt = find_tile<R, KT>(a, prefix, tpu, x + 32 + lane);
            }
            // the buffer read last is free again: every lane has passed its __syncwarp
            issue(i + NS - 1, put, n_tiles, i & ~31);
            put = put + 1 == NS ? 0 : put + 1;
            const int at = __shfl_sync(0xffffffffu, cur.at, i & 31);
            const int key0 = __shfl_sync(0xffffffffu, cur.key0, i & 31);
            const float ks = __shfl_sync(0xffffffffu, cur.ks, i & 31);
            const float vs = __shfl_sync(0xffffffffu, cur.vs, i & 31);
            const uint32_t kb = ring + get * SLOT, vb = kb + HALF;
            get = get + 1 == NS ? 0 : get + 1;
            if (at < 0) continue;
            cp_async_wait<NS - 1>();
            __syncwarp();
            if (FMT == ATTN_CACHE_E4M3 && key0 + KT > len) {
                // behind the sequence's last token a page may hold any code, NaN among
                // them, which a weight of 0 would not remove
                for (int c = lane; c < HALF / 16; c += 32)
                    if (key0 + c / (D / 16) >= len)
                        sts16_zero(vb + swizzled<D>(c / (D / 16), c % (D / 16)));
                __syncwarp();
            }
            float f[H], sv[H];
#pragma unroll
            for (int hh = 0; hh < H; ++hh) {
                f[hh] = ks * cq[hh];
                // a page no key of which the row sees adds nothing, not even its scale's NaN
                sv[hh] = key0 < lim[hh] ? vs : 0.f;
            }
#pragma unroll 1
            for (int k16 = 0; k16 < KT; k16 += 16) {
                float s[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float e0[4] = {}, e1[4] = {};  // two chains, for the latency
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 u4 = lds16(kb + k16 * D + swizzled<D>(n * 8 + g, t * (D / 64) + c));
                        const uint32_t words[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t b0, b1;
                            U::quad(words[e], b0, b1);
                            const int st = c * 4 + e;
                            mma16816((e & 1) ? e1 : e0, qa[st][0], qa[st][1], qa[st][2], qa[st][3], b0, b1);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] = e0[e] + e1[e];
                }
                float y[H][4], p[H][4], c[H];
                bool far = false;
#pragma unroll
                for (int hh = 0; hh < H; ++hh) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)  // hi and lo parts of q in the 8-row form
                        y[hh][e] = (WIDE ? s[e >> 1][2 * hh + (e & 1)] : s[e >> 1][e & 1] + s[e >> 1][2 + (e & 1)]) * f[hh];
                    if (key0 + k16 + 16 > low) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key0 + k16 + 8 * (e >> 1) + 2 * t + (e & 1) >= lim[hh]) y[hh][e] = -INFINITY;
                    }
                    c[hh] = sv[hh] * rv[hh];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[hh][e] = ex2(y[hh][e] - top[hh]);
                    const float most = fmaxf(fmaxf(p[hh][0], p[hh][1]), fmaxf(p[hh][2], p[hh][3]));
                    far = far || most > 16.f || most * c[hh] > 32768.f;
                }
                if (__any_sync(0xffffffffu, far)) {
                    // new references: the scores' maximum, and the page scale unless what o
                    // holds is larger by now
#pragma unroll
                    for (int hh = 0; hh < H; ++hh) {
                        float mx = fmaxf(fmaxf(y[hh][0], y[hh][1]), fmaxf(y[hh][2], y[hh][3]));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const float nt = fmaxf(top[hh], mx);
                        const float alpha = ex2(top[hh] - nt);  // 0 from kUnset
                        const float was = alpha * 2048.f / rv[hh];
                        const float nv = mx == -INFINITY ? rv[hh] : 2048.f / fmaxf(fmaxf(was, sv[hh]), 0x1p-100f);
                        const float to = alpha * (nv / rv[hh]);
                        l[hh] *= alpha;
#pragma unroll
                        for (int n = 0; n < VT; ++n) {
                            if constexpr (WIDE) {
                                acc[n][2 * hh] *= to;
                                acc[n][2 * hh + 1] *= to;
                            } else {
                                acc[n][0] *= to; acc[n][1] *= to; acc[n][2] *= to; acc[n][3] *= to;
                            }
                        }
                        top[hh] = nt;
                        rv[hh] = nv;
                        c[hh] = sv[hh] * nv;
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[hh][e] = ex2(y[hh][e] - nt);
                    }
                }
                uint32_t pa[4];
#pragma unroll
                for (int hh = 0; hh < H; ++hh) {
                    l[hh] += (p[hh][0] + p[hh][1]) + (p[hh][2] + p[hh][3]);
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float w0 = p[hh][2 * n] * c[hh], w1 = p[hh][2 * n + 1] * c[hh];
                        const uint32_t hi = pack_f16(w0, w1);
                        if constexpr (WIDE) {
                            pa[2 * n + hh] = hi;
                        } else {
                            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                            pa[2 * n] = hi;
                            pa[2 * n + 1] = pack_f16(w0 - b.x, w1 - b.y);
                        }
                    }
                }
                uint32_t r[4][D / 32];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = 2 * t + (e & 1) + ((e & 2) ? 8 : 0);
                    if constexpr (D == 128) {
                        const uint4 u4 = lds16(vb + k16 * D + swizzled<D>(row, g));
                        r[e][0] = u4.x; r[e][1] = u4.y; r[e][2] = u4.z; r[e][3] = u4.w;
                    } else {
                        const uint2 u2 = lds8(vb + k16 * D + swizzled<D>(row, g >> 1) + (g & 1) * 8);
                        r[e][0] = u2.x; r[e][1] = u2.y;
                    }
                }
#pragma unroll
                for (int q = 0; q < D / 32; ++q)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {  // bytes 2 hf and 2 hf + 1 of the four rows' words
                        uint32_t a0, a1, b0, b1;
                        U::quad(__byte_perm(r[0][q], r[1][q], hf ? 0x7362 : 0x5140), a0, a1);
                        U::quad(__byte_perm(r[2][q], r[3][q], hf ? 0x7362 : 0x5140), b0, b1);
                        mma16816(acc[4 * q + 2 * hf], pa[0], pa[1], pa[2], pa[3], a0, b0);
                        mma16816(acc[4 * q + 2 * hf + 1], pa[0], pa[1], pa[2], pa[3], a1, b1);
                    }
            }
            __syncwarp();  // the buffer may be filled again
        }

        // the unit's state: written if it is whole, else kept for the join.  The range's last unit
        // leaves it in the ring, which is not needed any more; a first unit that more follow, in
        // global memory.
        const bool whole = u.begin >= x0 && u.end <= x1;
        const bool before = u.begin < x0;
        float *keep = xe < x1 ? a.hold + w * R * D : reinterpret_cast<float *>(sm + warp * kRing);
        if (!in_bounds(w < (int64_t)gridDim.x * kWarps, a.status)) break;
        if (xe == x1) {
            cp_async_wait<0>();
            __syncwarp();
        }
#pragma unroll
        for (int hh = 0; hh < H; ++hh) {
            float sum = l[hh];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            // 0: no key was visible.  NaN scores alone leave `top` unset
            const float inv = sum == 0.f ? 0.f : 1.f / sum, unit = 1.f / rv[hh];
            const float lse2 = sum == 0.f ? -INFINITY : top[hh] + log2f(sum);
            const int r = g + 8 * hh;
            float f[D / 4];
#pragma unroll
            for (int n = 0; n < VT; ++n) {
                f[n] = (WIDE ? acc[n][2 * hh] : acc[n][0] + acc[n][2]) * inv * unit;
                f[VT + n] = (WIDE ? acc[n][2 * hh + 1] : acc[n][1] + acc[n][3]) * inv * unit;
            }
            if (whole) {
                size_t row;
                if (!out_row<R>(a, u, r, row)) continue;
#pragma unroll
                for (int e = 0; e < D / 4; e += 8) store_o8(a, row * D + t * (D / 4) + e, f + e);
                if (a.lse && t == 0) a.lse[row] = lse2 * kLn2;
            } else {
                float4 *p = reinterpret_cast<float4 *>(keep + r * D + t * (D / 4));
#pragma unroll
                for (int e = 0; e < D / 16; ++e) p[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                if (t == 0) s_lse[warp][before ? 0 : 1][r] = lse2;
            }
        }
        if (!whole && lane == 0) {
            s_unit[warp][before ? 0 : 1] = u;
            s_keep[warp][before ? 0 : 1] = keep;
            s_has[warp] |= before ? 1 : 2;
        }
    }
    __syncthreads();

    // Join the states of the CTA's shared units.  A group is a unit's pieces: a
    // state that goes on (or, from warp 0, one begun in an earlier CTA) and the
    // following warps' states of the same unit.  Each warp takes rows warp, warp + 8.
    int64_t X1 = 0;  // past the CTA's last tile
    for (int k = 0; k < kWarps; ++k) X1 = s_end[k] > X1 ? s_end[k] : X1;
    bool over = false;
    for (int first = 0; first < kWarps; ++first) {
#pragma unroll 1
        for (int side = first == 0 ? 0 : 1; side < 2; ++side) {
            if (!(s_has[first] & (1 << side))) continue;
            const Unit u = s_unit[first][side];
            int n = 1;  // pieces
            if (u.end > s_end[first])
                while (first + n < kWarps && (s_has[first + n] & 1) && s_unit[first + n][0].begin == u.begin) {
                    ++n;
                    if (u.end <= s_end[first + n - 1]) break;
                }
            const bool earlier = side == 0, later = u.end > X1;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (earlier ? 0 : 1);
            over = over || (later && !earlier);
            if (later && !earlier && threadIdx.x == 0) {
                const int last = (int)(worker_of(u.end - 1, total, workers) / kWarps);
                a.tail[2 * blockIdx.x] = make_int4(1, last, u.b, u.hk);
                a.tail[2 * blockIdx.x + 1] = make_int4(u.seg, u.rb, 0, 0);
            }
#pragma unroll 1
            for (int r = warp; r < R; r += kWarps) {
                float M = -INFINITY;
                for (int k = 0; k < n; ++k) M = fmaxf(M, s_lse[first + k][k == 0 ? side : 0][r]);
                const float top = M == -INFINITY ? 0.f : M;
                float L = 0.f, o[D / 32] = {};
                for (int k = 0; k < n; ++k) {
                    const int sd = k == 0 ? side : 0;
                    const float wt = ex2(s_lse[first + k][sd][r] - top);
                    const float *src = s_keep[first + k][sd] + r * D + lane;
                    L += wt;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) o[e] = fmaf(wt, src[32 * e], o[e]);
                }
                const float inv = L == 0.f ? 0.f : 1.f / L;
                const float lse2 = L == 0.f ? -INFINITY : top + log2f(L);
                if (earlier || later) {
                    if (!in_bounds(slot < 2 * (int64_t)gridDim.x, a.status)) continue;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) a.po[(slot * R + r) * D + lane + 32 * e] = o[e] * inv;
                    if (lane == 0) a.pl[slot * R + r] = lse2;
                } else {
                    size_t row;
                    if (!out_row<R>(a, u, r, row)) continue;
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) store_o(a, row * D + lane + 32 * e, o[e] * inv);
                    if (a.lse && lane == 0) a.lse[row] = lse2 * kLn2;
                }
            }
        }
    }
    if (!over && threadIdx.x == 0) a.tail[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
}

// Joins the states of the unit that runs over the end of CTA blockIdx.x's
// range: the CTA's own and those of the CTAs up to the one that holds the
// unit's end.  One CTA per (range end, row of the block).
template <int D, int R>
__global__ void __launch_bounds__(kThreads) cache_merge_kernel(const FwdArgs a) {
    __shared__ float wts[kCacheMaxCtas];
    __shared__ float red[kWarps];
    __shared__ float part[kWarps][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d0 = a.tail[2 * blockIdx.x];
    if (!d0.x) return;
    const int4 d1 = a.tail[2 * blockIdx.x + 1];
    Unit u;
    u.b = d0.z;
    u.hk = d0.w;
    u.seg = d1.x;
    u.rb = d1.y;
    const int r = blockIdx.y;
    size_t row;
    if (!out_row<R>(a, u, r, row)) return;
    const int n = d0.y - (int)blockIdx.x + 1;
    if (!in_bounds(n <= kCacheMaxCtas, a.status)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the owner's state lies in its second slot, the others' in their first
    auto slot = [&](int p) { return 2 * (int64_t)(blockIdx.x + p) + (p == 0 ? 1 : 0); };
    float M = -INFINITY;
    for (int p = threadIdx.x; p < n; p += kThreads) {
        wts[p] = a.pl[slot(p) * R + r];
        M = fmaxf(M, wts[p]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (lane == 0) red[warp] = M;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kWarps; ++k) M = fmaxf(M, red[k]);
    const float top = M == -INFINITY ? 0.f : M;
    // every warp sums all weights in the same order, and its own parts' o
    float L = 0.f;
    for (int p = lane; p < n; p += 32) L += ex2(wts[p] - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    constexpr int C = D / 32;
    float acc[C] = {};
#pragma unroll 4
    for (int p = warp; p < n; p += kWarps) {
        const float wt = ex2(wts[p] - top);
        const float *src = a.po + (slot(p) * R + r) * D + lane;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = fmaf(wt, src[32 * c], acc[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) part[warp][lane + 32 * c] = acc[c];
    __syncthreads();
    if (threadIdx.x < D) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) sum += part[k][threadIdx.x];
        store_o(a, row * D + threadIdx.x, sum * inv);
        if (a.lse && threadIdx.x == 0) a.lse[row] = L == 0.f ? -INFINITY : (top + log2f(L)) * kLn2;
    }
}

template <int D, int FMT, int WIDE, int KT>
int launch_fwd_t(const FwdArgs &a, unsigned grid, cudaStream_t stream) {
    constexpr int R = WIDE ? 16 : 8;
    auto fwd = cache_fwd_kernel<D, FMT, WIDE, KT>;
    constexpr size_t ring = (size_t)kWarps * kRing;
    if (!set_smem_limit_once(reinterpret_cast<const void *>(fwd), (int)(ring + (kMaxCacheBatch + 1) * 8)))
        return ATTN_ERR_LAUNCH;
    fwd<<<grid, kThreads, ring + (a.pages ? 0 : ((size_t)a.B + 1) * 8), stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, (unsigned)(a.rows < R ? a.rows : R));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, cache_merge_kernel<D, R>, a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

// Keys of a tile: at most 8 KB of keys and values, three of which a warp's ring
// holds, and no more than a page.
constexpr int tile_keys(int d, int page) {
    const int most = d == 128 ? 32 : 64;
    return page < most ? page : most;
}

template <int D, int FMT, int WIDE>
int launch_fwd_k(const FwdArgs &a, int kt, unsigned grid, cudaStream_t s) {
    if (kt == 16) return launch_fwd_t<D, FMT, WIDE, 16>(a, grid, s);
    if (kt == 32) return launch_fwd_t<D, FMT, WIDE, 32>(a, grid, s);
    return launch_fwd_t<D, FMT, WIDE, tile_keys(D, 64)>(a, grid, s);
}
template <int D, int FMT>
int launch_fwd_w(const FwdArgs &a, bool wide, int kt, unsigned grid, cudaStream_t s) {
    return wide ? launch_fwd_k<D, FMT, 1>(a, kt, grid, s) : launch_fwd_k<D, FMT, 0>(a, kt, grid, s);
}

}  // namespace

// The 16-row form where the output's own rounding hides the weights' and the
// rows do not fit eight.
static bool cache_wide(int rows, int dtype) { return dtype == ATTN_BF16 && rows > 8; }

// Workspace: the tails [2 * CTA], a state per warp, two per CTA and their lse.
size_t cache_fwd_workspace(int B, int H, int H_kv, int Sq, int d, int dtype, bool listed) {
    const int64_t rows = (int64_t)(H / H_kv) * (listed ? 1 : Sq);
    const size_t R = cache_wide((int)(rows > 16 ? 16 : rows), dtype) ? 16 : 8;
    return (size_t)kCacheMaxCtas * (32 + (kWarps + 2) * R * d * 4 + 2 * R * 4);
}

int launch_cache_fwd(const attn_cache &c, const void *q, void *o, float *lse, const int32_t *table,
                     int max_pages, const int32_t *lens, const int32_t *counts, const int32_t *pages,
                     int n_select, int B, int H, int Sq, int causal, float scale, int dtype,
                     void *workspace, cudaStream_t stream) {
    FwdArgs a = {};
    a.q = q; a.o = o; a.lse = lse;
    a.k = (const uint8_t *)c.k; a.v = (const uint8_t *)c.v;
    a.ks = c.k_scale; a.vs = c.v_scale;
    a.table = table; a.lens = lens; a.counts = counts; a.pages = pages;
    a.B = B; a.Hkv = c.H_kv; a.G = H / c.H_kv; a.Sq = Sq;
    a.page = c.page; a.n_pages = c.n_pages; a.max_pages = max_pages; a.n_sel = n_select;
    a.causal = causal; a.dtype = dtype;
    a.sl2 = scale * 1.4426950408889634f;
    a.nseg = pages ? Sq : 1;
    a.rows = pages ? a.G : a.G * Sq;
    const bool wide = cache_wide(a.rows, dtype);
    const int R = wide ? 16 : 8;
    a.nrb = (a.rows + R - 1) / R;
    const int64_t units = (int64_t)B * a.Hkv * a.nseg * a.nrb;  // at most B * H * Sq < 2^31
    a.status = status_word_device_ptr();
    if (!a.status) return ATTN_ERR_CUDA;
    const int kt = tile_keys(c.d, c.page);
    const int sms = device_sm_count();
    if (sms <= 0) return ATTN_ERR_CUDA;
    // as many CTAs as the longest possible lengths can give every warp a tile
    const double most = (double)units * (pages ? (double)n_select * c.page : (double)max_pages * c.page) / kt;
    int64_t ctas = most / kWarps < sms ? (int64_t)(most / kWarps) + 1 : sms;
    if (ctas > kCacheMaxCtas) ctas = kCacheMaxCtas;
    if (ctas > sms) ctas = sms;
    a.workers = (int)ctas * kWarps;
    a.tail = reinterpret_cast<int4 *>(workspace);
    a.hold = reinterpret_cast<float *>(a.tail + 2 * ctas);
    a.po = a.hold + (size_t)a.workers * R * c.d;
    a.pl = a.po + (size_t)2 * ctas * R * c.d;
    if (c.d == 64)
        return c.format == ATTN_CACHE_E4M3 ? launch_fwd_w<64, ATTN_CACHE_E4M3>(a, wide, kt, (unsigned)ctas, stream)
                                           : launch_fwd_w<64, ATTN_CACHE_I8>(a, wide, kt, (unsigned)ctas, stream);
    return c.format == ATTN_CACHE_E4M3 ? launch_fwd_w<128, ATTN_CACHE_E4M3>(a, wide, kt, (unsigned)ctas, stream)
                                       : launch_fwd_w<128, ATTN_CACHE_I8>(a, wide, kt, (unsigned)ctas, stream);
}

}  // namespace attn
