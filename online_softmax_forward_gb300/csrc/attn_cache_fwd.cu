// attn_cache_fwd.cu -- attention of a few query rows per sequence over the
// paged 8-bit cache, over all pages or over a list of pages per query.
//
//     s_j = scale * k_scale[page(j)] * (q . kcode_j)
//     o   = sum_j softmax_j(s) * v_scale[page(j)] * vcode_j
//
// Work.  A unit is (sequence, kv head, block of query rows): the G query heads
// of a kv head share its keys, so the rows of a block are (query, head of the
// group).  Its keys are walked in tiles of KT keys (32, or a page of 16).
// All tiles of a call are numbered through and cut into equal contiguous
// ranges, one per warp (cache_index.h): ragged lengths and few sequences fill
// the GPU alike.  A warp writes the units it covers alone.  Of the units that
// several warps of a CTA share the states are joined in shared memory, and a
// second kernel joins the at most one unit that runs over the end of each CTA's
// range, with the online softmax's merge of states.  Where units are few and of
// like length a CTA takes one each, and nothing is left to join (kSwitch).
//
// Products.  The 8-bit codes are exact in fp16, so both products run on
// mma.m16n8k16 with fp32 accumulation and no dequantised tile exists
// anywhere: the page's scales multiply the scores and the page's share of o.
// Keys and channels lie on the MMA's 16 rows and 8 query rows on its columns,
// S^T = K Q^T and O^T = V^T P^T, since a decode step has few queries: with the
// queries on the rows it takes twice the MMAs and twice the registers for o (4 x 32
// heads, 32k keys: 174 -> 171 us; one 1k sequence 11.1 -> 10.2 us).  P leaves
// the first product key by key and enters the second query by query: movmatrix
// turns it.  A warp takes up to two blocks of 8 rows, three at d = 64, which share
// the loads and conversions of the codes.
//   16-bit outputs: q is exact in fp16, p is rounded once to it (2^-12, as an
//     fp16 output is, or less than a bf16 one).
//   fp32 outputs: q = hi + lo and p = hi + lo in two products each, those of
//     22-bit numbers.
// q rows are first multiplied by a power of two that puts the row's largest
// magnitude in [2^14, 2^15): any fp32 or bf16 exponent then fits fp16.
//
// Softmax.  The sums l and o are kept relative to a reference `top` of the
// scores and, o, to a reference 2^11 / rv of weight times page scale, so the weight that
// enters the second product is p * v_scale * rv.  Both references move only when
// a step of 32 keys (a page of 16) would pass fp16's range or a weight 2^4: one vote, no
// maximum across lanes and no rescaling in the others.  The second follows what the row
// weighs most, not the largest page it sees: a page of huge values and no weight would
// push the other weights under fp16's normal numbers.  What is below 2^-25 of the
// largest weight times page scale keeps fewer bits, and nothing below 2^-36.
//
// Loads.  Each warp copies its own tiles into a ring of shared memory slots with
// 16-byte cp.async (a slot holds the codes of one tile's keys and values), all
// slots but the one in use in flight, and waits for nobody else.  (Tiles by TMA,
// with the swizzle in the tensor map, measured the same for 4 x 32 x 32k keys and
// cost the short calls a microsecond on the host.)  The MMA's k index may name the
// channels in any order that q and k share, and its row any channel of v: lane
// (g, t) = (lane / 4, lane % 4) reads D/4 consecutive bytes of key rows g and
// g + 8, and D/8 consecutive bytes of value rows 2t, 2t+1, 2t+8, 2t+9.  The 16-byte
// pieces of a row are swizzled so that both reads are free of bank conflicts.
//
// Bound: by the reading of the codes where they are many (4 x 32 heads, 32k keys,
// d = 128: 170 us, 6.3 TB/s, 93 % of the copy rate; the SMs do not get equal shares
// of the memory and the last ends 14 % after the mean), by waits in short calls
// (one sequence of 1000 tokens, 8 kv heads: 10 us, of which 3 for four steps of
// keys; the rest finds the tiles, loads q, joins, each a chain of cold loads and
// code).  From the last key to the end of a CTA, its barrier and join, the 32k-key call
// spends 10 000 clocks on average and the last CTA 5000.  8 warps of up to 240 registers; 12 warps, which one block's registers
// allow, measured 169 us and 9.9 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_internal.h"
#include "cache_fwd.cuh"
#include "cache_mma.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = 24 * 1024;  // shared memory of each warp's tiles, later of its states
// Tiles that a second unit and a second kernel cost a warp.  With 2, 5, 8, 12, 16 in us: five
// drafts of 16 sequences of up to 4096 tokens 33.5, 33.5, 31.9, 32.0, 29.8; one sequence of 1000
// tokens 10.6, 9.6, 9.6, 9.6, 9.6; selection and attention over 96 pages of 32 for 16 units
// 33.6, 33.4, 33.4, 40.9, 40.9
constexpr int kSwitch = 8;
// CTAs to a unit, on average, up to which the second kernel takes a row per warp.  A row per warp
// and a row per CTA: five drafts (20 rows) of 32 sequences of 2000 to 4096 tokens, 8 kv heads,
// 48.2 and 50.9 us; 64 ragged sequences 102.7 and 103.6; 4 of 32k (about five CTAs a unit) 42.9
// and 42.0; one of 32k and one kv head 44.1 and 13.4
constexpr int kFewShares = 3;

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
struct Tile {  // one key tile, held by one lane
    int at;    // tile of KT keys in the pool, -1: nothing to read
    int key0;  // its first key's position in the sequence
    float ks, vs;
};

// Quotients of normal numbers, to 2^-22; the divisor is at most 2^126.
__device__ __forceinline__ float ratio(float a, float b) { return __fdividef(a, b); }
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // an 8 x 8 tile of 16-bit numbers
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int R, int KT>
__device__ __forceinline__ Tile find_tile(const FwdArgs &a, const Place &p) {
    Tile d;
    d.at = -1;
    d.key0 = 0;
    d.ks = d.vs = 0.f;
    const int shift = 31 - __clz(a.page / KT);  // tiles of a page: a power of two
    int lp = p.t >> shift;
    const int sub = p.t & ((1 << shift) - 1);
    const Unit u = unit_at(a, p.b, p.unit);
    if (a.pages) {
        const int64_t list = ((int64_t)u.b * a.Hkv + u.hk) * a.nseg + u.seg;
        if (!in_bounds(list < (int64_t)a.B * a.Hkv * a.nseg && lp < a.n_sel, a.status)) return d;
        lp = a.pages[list * a.n_sel + lp];
        if (lp < -1 || lp >= a.max_pages) atomicOr(a.status, kStatusTable);
        if (lp < 0 || lp >= a.max_pages) return d;
    }
    if (!in_bounds(u.b < a.B && lp < a.max_pages, a.status)) return d;
    const int phys = a.table[(int64_t)u.b * a.max_pages + lp];
    const int len = clamp_len(a.lens[u.b], a.max_pages, a.page);
    const int cnt = a.counts ? min(max(a.counts[u.b], 0), a.Sq) : a.Sq;
    // the block's last query that is one of the sequence's sees the most keys
    int first, last, h;
    row_of<R>(a, u, 0, first, h);
    row_of<R>(a, u, min(a.rows - u.rb * R, R) - 1, last, h);
    last = min(last, cnt - 1);
    const int seen = last < first ? 0 : visible_keys(len, cnt, last, a.causal);
    const int64_t key0 = (int64_t)lp * a.page + sub * KT;
    if (key0 >= seen) return d;
    d.key0 = (int)key0;
    if (phys < 0 || phys >= a.n_pages) {
        atomicOr(a.status, kStatusTable);
        return d;
    }
    const int64_t ph = (int64_t)phys * a.Hkv + u.hk;
    if (!in_bounds(ph < (int64_t)a.n_pages * a.Hkv && sub < 1 << shift, a.status)) return d;
    d.at = (int)((ph << shift) + sub);
    d.ks = a.ks[ph];
    d.vs = a.vs[ph];
    return d;
}

// NB blocks of 8 query rows; FINE: q and the weights in 22 bits (NB = 1).
template <int D, int FMT, int NB, int FINE, int KT>
__global__ void __launch_bounds__(kThreads, 1) cache_fwd_kernel(const FwdArgs a) {
    using U = Unpack<FMT>;
    constexpr int R = NB * 8;
    constexpr int QS = D / 16;         // k steps of K.Q
    constexpr int VT = D / 16;         // output tiles of 16 channels
    static_assert(!FINE || NB == 1, "one block");
    constexpr int HALF = KT * D;       // bytes of a tile's keys, then its values
    constexpr int SLOT = 2 * HALF;
    constexpr int NS = kRing / SLOT < 8 ? kRing / SLOT : 8;
    static_assert(NS >= 3 && R * D * 4 <= kRing, "a warp's ring later holds a state");
    constexpr int STEP = KT < 32 ? KT : 32;  // keys of one softmax step
    constexpr int MT = STEP / 16;            // score tiles of 16 keys
    extern __shared__ __align__(128) uint8_t sm[];
    int *prefix = reinterpret_cast<int *>(sm + kWarps * kRing);  // [B + 1]
    __shared__ int warp_sums[kWarps];
    __shared__ float s_lse[kWarps][2][R];
    __shared__ const float *s_keep[kWarps][2];
    __shared__ int s_b[kWarps][2], s_unit[kWarps][2];  // the units of the warps' kept states
    __shared__ int s_has[kWarps];  // bit 0: a state of a unit begun before, 1: that unit goes on,
                                   // 2: a state of a unit begun here that goes on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int tpu = a.pages ? a.n_sel * (a.page / KT) : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    int64_t total = 0, workers = kWarps;
    int64_t x0 = 0;
    int w = warp, n_tiles = 0;  // this warp's range
    Place here = {0, 0, 0, 1};
    auto tiles = [&](int b) { return a.pages ? tpu : prefix[b + 1] - prefix[b]; };
    auto report = [&](int b) {  // a length or count out of range
        const int len = a.lens[b], cnt = a.counts ? a.counts[b] : a.Sq;
        if (len != clamp_len(len, a.max_pages, a.page) || cnt < 0 || cnt > a.Sq)
            atomicOr(a.status, kStatusTable);
    };
    auto share_unit = [&] {  // the warps' parts of the unit at `here`
        const int64_t share = worker_count(here.n, kWarps, 1);
        if (warp < share) {
            here.t = (int)worker_begin(warp, here.n, share);
            n_tiles = (int)worker_begin(warp + 1, here.n, share) - here.t;
        }
    };
    if (lane == 0) s_has[warp] = 0;
    if (a.one_each) {
        here.b = (int)((uint32_t)blockIdx.x / a.by_units);
        here.unit = blockIdx.x - here.b * a.units;
        if (!in_bounds(here.b < a.B, a.status)) return;
        if (here.unit == 0 && threadIdx.x == 0) report(here.b);
        here.n = a.pages ? tpu : (clamp_len(a.lens[here.b], a.max_pages, a.page) + KT - 1) / KT;
        share_unit();
        if (here.n == 0) {  // no token: o = 0, lse = -inf
            const Unit u = unit_at(a, here.b, here.unit);
            const float z[8] = {};
            for (int e = threadIdx.x; e < R * (D / 8); e += kThreads) {
                size_t row;
                if (!out_row<R>(a, u, e / (D / 8), row)) continue;
                store_o8(a, row * D + e % (D / 8) * 8, z);
                if (a.lse && e % (D / 8) == 0) a.lse[row] = -INFINITY;
            }
            return;
        }
    } else {
        if (a.pages) {
            total = (int64_t)a.B * a.units * tpu;
            if (blockIdx.x == 0)
                for (int b = threadIdx.x; b < a.B; b += kThreads) report(b);
        } else {
            scan_lengths<kThreads>(a, KT, prefix, warp_sums);
            total = (int64_t)prefix[a.B] * a.units;
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
        workers = worker_count(total, a.workers, 1);
        w += blockIdx.x * kWarps;
        const int64_t all = (int64_t)a.B * a.units;
        bool alone = false;  // a CTA takes one unit
        if (!a.pages && all <= gridDim.x) {
            int longest = 0;
            for (int b = threadIdx.x; b < a.B; b += kThreads) longest = max(longest, tiles(b));
            alone = !__syncthreads_or(longest > ((total + workers - 1) / workers + kSwitch) * kWarps);
        }
        if (alone) {
            if (blockIdx.x < all) {
                here.b = (int)((uint32_t)blockIdx.x / a.by_units);
                here.unit = blockIdx.x - here.b * a.units;
                here.n = tiles(here.b);
                share_unit();
            }
        } else if (w < workers && total > 0) {
            x0 = worker_begin(w, total, workers);
            n_tiles = (int)(worker_begin(w + 1, total, workers) - x0);
            here = place_of(a, prefix, tpu, x0);
        }
    }
    // lane: tile 32 k + lane of the range, and the one 32 further
    Place mine = here;
    Tile cur = {-1, 0, 0.f, 0.f}, nxt = cur;
    if (lane < n_tiles) {
        advance(mine, lane, a.units, tiles);
        cur = find_tile<R, KT>(a, mine);
    }

    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(sm + warp * kRing);
    // tile j of the range into ring buffer `buf`; cur holds the tiles base .. base + 31
    auto issue = [&](int j, int buf, int base) {
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
    int put = NS - 1, get = 0;  // ring buffers: next to fill, next to read
#pragma unroll 1
    for (int j = 0; j < NS - 1; ++j) issue(j, j, 0);

    int i = 0;  // tile of the range
    while (i < n_tiles) {
        const Unit u = unit_at(a, here.b, here.unit);
        if (!in_bounds(u.b < a.B && here.unit < a.units, a.status)) break;
        const int left = min(here.n - here.t, n_tiles - i);  // tiles of this unit in the range
        const int len = clamp_len(a.lens[u.b], a.max_pages, a.page);
        const int cnt = a.counts ? min(max(a.counts[u.b], 0), a.Sq) : a.Sq;

        // query fragments: k step w holds channels 4w .. 4w + 3 of the lane's D/4 channels of
        // row g of each block; the lane's scores, weights and sums are those of rows 2t, 2t + 1
        uint32_t qb[NB][QS][2], ql[FINE ? QS : 1][2];
        float2 cq[NB];
        int lim[NB][2];
        int low = 0x7fffffff;  // fewest keys any row of the block sees
        float fine[FINE ? D / 4 : 1];
        codec::Raw8<1> raw[FINE ? 1 : NB][D / 32];  // 16-bit q, loaded together
        int sees_all[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            int qi, h;
            const bool real = row_of<R>(a, u, nb * 8 + g, qi, h) && q_row(a, u, h, qi);
            sees_all[nb] = real ? visible_keys(len, cnt, qi, a.causal) : 0;
            if (real) low = min(low, sees_all[nb]);
            const size_t at = real ? (((size_t)u.b * a.Hkv * a.G + h) * a.Sq + qi) * D + t * (D / 4) : 0;
            if constexpr (FINE) {
                float *f = fine;
#pragma unroll
                for (int e = 0; e < D / 4; ++e) f[e] = 0.f;
                if (real) load_q<D / 4>(a, at, f);
            } else {
#pragma unroll
                for (int e = 0; e < D / 32; ++e) {
                    raw[nb][e].u[0] = make_uint4(0, 0, 0, 0);
                    if (real) raw[nb][e].load(a.q, at + 8 * e);
                }
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float f[D / 4];
            const int sees = sees_all[nb];
            if constexpr (FINE) {
#pragma unroll
                for (int e = 0; e < D / 4; ++e) f[e] = fine[e];
            } else {
#pragma unroll
                for (int e = 0; e < D / 32; ++e) {
                    if (a.dtype == ATTN_BF16) {
                        raw[nb][e].widen(f + 8 * e);
                    } else {
                        codec::Raw8<2> x;
                        x.u[0] = raw[nb][e].u[0];
                        x.widen(f + 8 * e);
                    }
                }
            }
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < D / 4; ++e) amax = fmaxf(amax, fabsf(f[e]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float mul, back;
            row_power(amax, mul, back);
            back *= a.sl2;
            cq[nb] = make_float2(__shfl_sync(0xffffffffu, back, t * 8), __shfl_sync(0xffffffffu, back, t * 8 + 4));
            lim[nb][0] = __shfl_sync(0xffffffffu, sees, t * 8);
            lim[nb][1] = __shfl_sync(0xffffffffu, sees, t * 8 + 4);
#pragma unroll
            for (int w4 = 0; w4 < QS; ++w4)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float y0 = f[4 * w4 + 2 * e] * mul, y1 = f[4 * w4 + 2 * e + 1] * mul;
                    qb[nb][w4][e] = pack_f16(y0, y1);
                    if constexpr (FINE) {
                        const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&qb[nb][w4][e]));
                        ql[w4][e] = pack_f16(y0 - p.x, y1 - p.y);
                    }
                }
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) low = min(low, __shfl_xor_sync(0xffffffffu, low, o));

        // l and acc relative to `top` and rv; the first key seen sets both
        float2 top[NB], rv[NB], l[NB];
        float acc[NB][VT][4];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            top[nb] = make_float2(kUnset, kUnset);
            rv[nb] = make_float2(0x1p123f, 0x1p123f);
            l[nb] = make_float2(0.f, 0.f);
#pragma unroll
            for (int n = 0; n < VT; ++n) acc[nb][n][0] = acc[nb][n][1] = acc[nb][n][2] = acc[nb][n][3] = 0.f;
        }

        const int stop = i + left;
#pragma unroll 1
        for (; i < stop; ++i) {
            if ((i & 31) == 0) {
                if (i > 0) cur = nxt;
                nxt.at = -1;
                if (i + 32 + lane < n_tiles) {
                    advance(mine, 32, a.units, tiles);
                    nxt = find_tile<R, KT>(a, mine);
                }
            }
            // the buffer read last is free again: every lane has passed its __syncwarp
            issue(i + NS - 1, put, i & ~31);
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
#pragma unroll 1
                for (int c = lane; c < HALF / 16; c += 32)
                    if (key0 + c / (D / 16) >= len)
                        sts16_zero(vb + swizzled<D>(c / (D / 16), c % (D / 16)));
                __syncwarp();
            }
#pragma unroll 1
            for (int step = 0; step < KT; step += STEP) {
                // two chains of products where one block alone would leave the MMAs waiting for
                // one another: halves of the channels, or q's parts
                constexpr int CH = NB == 1 ? 2 : 1;
                float s[NB * CH][MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
#pragma unroll
                    for (int n = 0; n < NB * CH; ++n) s[n][m][0] = s[n][m][1] = s[n][m][2] = s[n][m][3] = 0.f;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 x = lds16(kb + step * D + swizzled<D>(m * 16 + g, t * (D / 64) + c));
                        const uint4 y = lds16(kb + step * D + swizzled<D>(m * 16 + 8 + g, t * (D / 64) + c));
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t a0, a1, a2, a3;
                            U::quad(xs[e], a0, a2);
                            U::quad(ys[e], a1, a3);
                            const int st = c * 4 + e;
                            if constexpr (FINE) {
                                mma16816(s[0][m], a0, a1, a2, a3, qb[0][st][0], qb[0][st][1]);
                                mma16816(s[1][m], a0, a1, a2, a3, ql[st][0], ql[st][1]);
                            } else {
#pragma unroll
                                for (int n = 0; n < NB; ++n)
                                    mma16816(s[n + (CH - 1) * (e & 1)][m], a0, a1, a2, a3, qb[n][st][0], qb[n][st][1]);
                            }
                        }
                    }
                    if constexpr (CH == 2) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[0][m][e] += s[1][m][e];
                    }
                }
                const bool edge = key0 + step + STEP > low;  // some row does not see every key
                float2 p[NB][MT][2];  // weights of keys 16 m + g and 8 more, for both rows
                float2 c[NB];
                auto weights = [&](int nb) {
                    const float2 f = __fmul2_rn(cq[nb], make_float2(ks, ks));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            const float2 z = __ffma2_rn(make_float2(s[nb][m][2 * hf], s[nb][m][2 * hf + 1]), f,
                                                        make_float2(-top[nb].x, -top[nb].y));
                            p[nb][m][hf] = make_float2(ex2(z.x), ex2(z.y));
                        }
                    if (edge) {
                        const int at = key0 + step + g;
#pragma unroll
                        for (int m = 0; m < MT; ++m)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                if (m * 16 + hf * 8 >= lim[nb][0] - at) p[nb][m][hf].x = 0.f;
                                if (m * 16 + hf * 8 >= lim[nb][1] - at) p[nb][m][hf].y = 0.f;
                            }
                    }
                };
                bool far = false;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                    // a page no key of which the row sees adds nothing, not even its scale's NaN
                    c[nb] = __fmul2_rn(rv[nb], make_float2(key0 < lim[nb][0] ? vs : 0.f, key0 < lim[nb][1] ? vs : 0.f));
                    weights(nb);
                    float2 most = p[nb][0][0];
#pragma unroll
                    for (int e = 1; e < 2 * MT; ++e) {
                        most.x = fmaxf(most.x, p[nb][e >> 1][e & 1].x);
                        most.y = fmaxf(most.y, p[nb][e >> 1][e & 1].y);
                    }
                    // not <=: where c has overflowed beside weights of 0 the product is a NaN
                    far = far || fmaxf(most.x, most.y) > 16.f ||
                          !(most.x * c[nb].x <= 32768.f && most.y * c[nb].y <= 32768.f);
                }
                if (__any_sync(0xffffffffu, far)) {
                    // new references: the scores' maximum, and the largest weight times page scale
                    // unless what o holds is larger by now.  Returned: what o is to be multiplied by
                    auto moved = [&](float f, float sv, int seen, const float (&x)[2 * MT], float &top, float &rv,
                                     float &l, float &c) {
                        float mx = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 2 * MT; ++e)
                            if (!edge || 8 * e < seen) mx = fmaxf(mx, x[e] * f);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const float nt = fmaxf(top, mx);
                        const float alpha = ex2(top - nt);  // 0 from kUnset
                        const float was = ratio(alpha * 128.f, rv);  // a sixteenth, as `here`: finite for any scale
                        // Nothing but what the row weighs moves the reference of o: the page's scale
                        // times its largest weight.  Weights that are all 0 by now add nothing (but
                        // their scale's NaN); below 2^-112 the scale counts that much, so that c stays
                        // finite
                        const float e = ex2(mx - nt);
                        const float here = e > 0.f ? sv * fmaxf(e * 0x1p-4f, 0x1p-116f) : 0.f;
                        const float nv = mx == -INFINITY ? rv : ratio(128.f, fmaxf(fmaxf(was, here), 0x1p-116f));
                        const float to = alpha == 0.f ? 0.f : alpha * ratio(nv, rv);
                        l *= alpha;
                        top = nt;
                        rv = nv;
                        c = e > 0.f || sv != sv ? sv * nv : 0.f;
                        return to;
                    };
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        float x[2][2 * MT];
#pragma unroll
                        for (int e = 0; e < 4 * MT; ++e) x[e & 1][e >> 1] = s[nb][e >> 2][e & 3];
                        const int at = key0 + step + g;
                        float2 to;
                        to.x = moved(ks * cq[nb].x, key0 < lim[nb][0] ? vs : 0.f, lim[nb][0] - at, x[0], top[nb].x,
                                     rv[nb].x, l[nb].x, c[nb].x);
                        to.y = moved(ks * cq[nb].y, key0 < lim[nb][1] ? vs : 0.f, lim[nb][1] - at, x[1], top[nb].y,
                                     rv[nb].y, l[nb].y, c[nb].y);
#pragma unroll
                        for (int n = 0; n < VT; ++n) {
                            acc[nb][n][0] *= to.x;
                            acc[nb][n][1] *= to.y;
                            acc[nb][n][2] *= to.x;
                            acc[nb][n][3] *= to.y;
                        }
                        weights(nb);
                    }
                }
                uint32_t pb[NB][MT][2], pl[FINE ? MT : 1][2];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            l[nb] = __fadd2_rn(l[nb], p[nb][m][hf]);
                            const float2 w2 = __fmul2_rn(p[nb][m][hf], c[nb]);
                            const uint32_t hi = pack_f16(w2.x, w2.y);
                            pb[nb][m][hf] = transposed(hi);
                            if constexpr (FINE) {
                                const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                                pl[m][hf] = transposed(pack_f16(w2.x - b.x, w2.y - b.y));
                            }
                        }
#pragma unroll
                for (int st = 0; st < MT; ++st) {
                    uint32_t r[4][D / 32];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = st * 16 + 2 * t + (e & 1) + ((e & 2) ? 8 : 0);
                        if constexpr (D == 128) {
                            const uint4 u4 = lds16(vb + step * D + swizzled<D>(row, g));
                            r[e][0] = u4.x; r[e][1] = u4.y; r[e][2] = u4.z; r[e][3] = u4.w;
                        } else {
                            const uint2 u2 = lds8(vb + step * D + swizzled<D>(row, g >> 1) + (g & 1) * 8);
                            r[e][0] = u2.x; r[e][1] = u2.y;
                        }
                    }
#pragma unroll
                    for (int q = 0; q < D / 32; ++q)
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {  // bytes 2 hf and 2 hf + 1 of the four rows' words
                            uint32_t a0, a1, a2, a3;
                            U::quad(__byte_perm(r[0][q], r[1][q], hf ? 0x7362 : 0x5140), a0, a1);
                            U::quad(__byte_perm(r[2][q], r[3][q], hf ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb) {
                                float(&o4)[4] = acc[nb][2 * q + hf];
                                mma16816(o4, a0, a1, a2, a3, pb[nb][st][0], pb[nb][st][1]);
                                if constexpr (FINE) mma16816(o4, a0, a1, a2, a3, pl[st][0], pl[st][1]);
                            }
                        }
                }
            }
            __syncwarp();  // the buffer may be filled again
        }

        // the unit's state: written if it is whole, else kept for the join.  The range's last unit
        // leaves it in the ring, which is not needed any more; a first unit that more follow, in
        // global memory.
        const bool before = i == left && here.t > 0, after = here.t + left < here.n;
        float *keep = i < n_tiles ? a.hold + (size_t)w * R * D : reinterpret_cast<float *>(sm + warp * kRing);
        if (i == n_tiles) {
            cp_async_wait<0>();
            __syncwarp();
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float sum = x ? l[nb].y : l[nb].x;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                // 0: no key was visible.  NaN scores alone leave `top` unset
                const float inv = sum == 0.f ? 0.f : ratio(1.f, sum), unit = ratio(1.f, x ? rv[nb].y : rv[nb].x);
                const float lse2 = sum == 0.f ? -INFINITY : (x ? top[nb].y : top[nb].x) + log2f(sum);
                const int r = nb * 8 + 2 * t + x;
                float f[D / 8];  // channels g * D / 8 ...
#pragma unroll
                for (int n = 0; n < VT; ++n) {
                    f[2 * n] = acc[nb][n][x] * inv * unit;
                    f[2 * n + 1] = acc[nb][n][2 + x] * inv * unit;
                }
                if (!before && !after) {
                    size_t row;
                    if (!out_row<R>(a, u, r, row)) continue;
#pragma unroll
                    for (int e = 0; e < D / 8; e += 8) store_o8(a, row * D + g * (D / 8) + e, f + e);
                    if (a.lse && g == 0) a.lse[row] = lse2 * kLn2;
                } else if (in_bounds(w < (int)gridDim.x * kWarps, a.status)) {
                    float4 *p = reinterpret_cast<float4 *>(keep + r * D + g * (D / 8));
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) p[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    if (g == 0) s_lse[warp][before ? 0 : 1][r] = lse2;
                }
            }
        if ((before || after) && lane == 0) {
            const int side = before ? 0 : 1;
            s_b[warp][side] = here.b;
            s_unit[warp][side] = here.unit;
            s_keep[warp][side] = keep;
            s_has[warp] |= before ? (after ? 3 : 1) : 4;
        }
        if (i < n_tiles) advance(here, left, a.units, tiles);
    }
    __syncthreads();

    // Join the states of the CTA's shared units.  A unit's pieces are a state
    // that goes on (or, from warp 0, one begun in an earlier CTA) and the
    // following warps' states of units begun before, up to one that ends.  Each
    // warp takes rows warp, warp + 8; lane k holds piece k's weight.
    uint32_t heads = 0, goes = 0, tails = 0;  // by warp, from s_has
    {
        const int has = lane < kWarps ? s_has[lane] : 0;
        heads = __ballot_sync(0xffffffffu, has & 1);
        goes = __ballot_sync(0xffffffffu, has & 2);
        tails = __ballot_sync(0xffffffffu, has & 4);
    }
    if (!(tails | (heads & 1))) {  // nothing shared
        if (threadIdx.x == 0) a.tail[blockIdx.x] = make_int4(0, 0, 0, 0);
        return;
    }
    bool over = false;
#pragma unroll 1
    for (int g0 = heads & 1 ? -1 : __ffs(tails) - 1; g0 < kWarps;) {
        const int first = g0 < 0 ? 0 : g0, side = g0 < 0 ? 0 : 1;
        int n = 1;
        bool open = side ? true : (goes & 1);  // the unit goes on behind the pieces so far
        while (open && first + n < kWarps && (heads >> (first + n) & 1)) {
            open = goes >> (first + n) & 1;
            ++n;
        }
        const bool earlier = side == 0;
        const Unit u = unit_at(a, s_b[first][side], s_unit[first][side]);
        const int slot = 2 * blockIdx.x + (earlier ? 0 : 1);
        if (open && !earlier) {
            over = true;
            if (threadIdx.x == 0) {
                const int nt = tiles(u.b);
                const int64_t end = (a.pages ? (int64_t)u.b * a.units * nt : (int64_t)prefix[u.b] * a.units) +
                                    (int64_t)(s_unit[first][side] + 1) * nt;
                a.tail[blockIdx.x] = make_int4(1, (int)(worker_of(end - 1, total, workers) / kWarps), u.b,
                                               s_unit[first][side]);
            }
        }
#pragma unroll 1
        for (int r = warp; r < R; r += kWarps) {
            const float ls = lane < n ? s_lse[first + lane][lane == 0 ? side : 0][r] : -INFINITY;
            float M = ls;
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            const float base = M == -INFINITY ? 0.f : M;
            const float wt = ex2(ls - base);
            float L = wt;
#pragma unroll
            for (int o = 1; o < kWarps; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
            M = __shfl_sync(0xffffffffu, M, 0);
            L = __shfl_sync(0xffffffffu, L, 0);
            float o[D / 32] = {};  // of 2^-3 times the weights: a sum that the largest values fit
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float wk = __shfl_sync(0xffffffffu, wt, k) * 0x1p-3f;
                if (k >= n) continue;
                const float *src = s_keep[first + k][k == 0 ? side : 0] + r * D + lane;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) o[e] = fmaf(wk, src[32 * e], o[e]);
            }
            const float inv = L == 0.f ? 0.f : ratio(8.f, L);
            const float lse2 = L == 0.f ? -INFINITY : (M == -INFINITY ? 0.f : M) + log2f(L);
            if (earlier || open) {
                if (!in_bounds(slot < 2 * (int)gridDim.x, a.status)) continue;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) a.po[((size_t)slot * R + r) * D + lane + 32 * e] = o[e] * inv;
                if (lane == 0) a.pl[slot * R + r] = lse2;
            } else {
                size_t row;
                if (!out_row<R>(a, u, r, row)) continue;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) store_o(a, row * D + lane + 32 * e, o[e] * inv);
                if (a.lse && lane == 0) a.lse[row] = lse2 * kLn2;
            }
        }
        // the next state that goes on (this group's own is `first` or none)
        const uint32_t rest = tails >> first >> (side ? 1 : 0);
        if (!rest) break;
        g0 = first + (side ? 1 : 0) + __ffs(rest) - 1;
    }
    if (!over && threadIdx.x == 0) a.tail[blockIdx.x] = make_int4(0, 0, 0, 0);
}

static_assert(kCacheMaxCtas * kFits <= 1.f, "a sum of states that the largest values fit");

// Joins the states of the unit that runs over the end of CTA blockIdx.x's
// range: the CTA's own and those of the CTAs up to the one that holds the
// unit's end.  One CTA per (range end, row of the block).
template <int D, int R>
__global__ void __launch_bounds__(kThreads) cache_merge_kernel(const FwdArgs a) {
    __shared__ float wts[kCacheMaxCtas];
    __shared__ float red[kWarps];
    __shared__ float part[kWarps][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d0 = a.tail[blockIdx.x];
    if (!d0.x) return;
    const Unit u = unit_at(a, d0.z, d0.w);
    const int r = blockIdx.y;
    size_t row;
    if (!out_row<R>(a, u, r, row)) return;
    const int n = d0.y - (int)blockIdx.x + 1;
    if (!in_bounds(n >= 1 && n <= kCacheMaxCtas && blockIdx.x + n <= gridDim.x, a.status)) return;
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
        const float wt = ex2(wts[p] - top) * kFits;
        const float *src = a.po + (slot(p) * R + r) * D + lane;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = fmaf(wt, src[32 * c], acc[c]);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) part[warp][lane + 32 * c] = acc[c];
    __syncthreads();
    if (threadIdx.x < D) {
        const float inv = L == 0.f ? 0.f : ratio(1.f / kFits, L);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) sum += part[k][threadIdx.x];
        store_o(a, row * D + threadIdx.x, sum * inv);
        if (a.lse && threadIdx.x == 0) a.lse[row] = L == 0.f ? -INFINITY : (top + log2f(L)) * kLn2;
    }
}

// The same with a row per warp, for units that few CTAs share.
template <int D, int R>
__global__ void __launch_bounds__(kThreads) cache_merge_rows_kernel(const FwdArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d0 = a.tail[blockIdx.x];
    if (!d0.x) return;
    const Unit u = unit_at(a, d0.z, d0.w);
    const int lane = threadIdx.x & 31, r = blockIdx.y * kWarps + (threadIdx.x >> 5);
    size_t row;
    if (r >= R || !out_row<R>(a, u, r, row)) return;
    const int n = d0.y - (int)blockIdx.x + 1;
    if (!in_bounds(n >= 1 && n <= kCacheMaxCtas && blockIdx.x + n <= gridDim.x, a.status)) return;
    auto slot = [&](int p) { return 2 * (int64_t)(blockIdx.x + p) + (p == 0 ? 1 : 0); };
    float M = -INFINITY;
    for (int p = lane; p < n; p += 32) M = fmaxf(M, a.pl[slot(p) * R + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float top = M == -INFINITY ? 0.f : M;
    constexpr int C = D / 32;
    float L = 0.f, acc[C] = {};
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
        const float wt = ex2(a.pl[slot(p) * R + r] - top);
        const float *src = a.po + (slot(p) * R + r) * D + lane;
        L += wt;
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] = fmaf(wt * kFits, src[32 * c], acc[c]);
    }
    const float inv = L == 0.f ? 0.f : ratio(1.f / kFits, L);
#pragma unroll
    for (int c = 0; c < C; ++c) store_o(a, row * D + lane + 32 * c, acc[c] * inv);
    if (a.lse && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (top + log2f(L)) * kLn2;
}

template <int D, int FMT, int NB, int FINE, int KT>
int launch_fwd_t(const FwdArgs &a, unsigned grid, cudaStream_t stream) {
    constexpr int R = NB * 8;
    auto fwd = cache_fwd_kernel<D, FMT, NB, FINE, KT>;
    constexpr size_t ring = (size_t)kWarps * kRing;
    if (!set_smem_limit_once(reinterpret_cast<const void *>(fwd), (int)(ring + (kMaxCacheBatch + 1) * 4)))
        return ATTN_ERR_LAUNCH;
    fwd<<<grid, kThreads, ring + (a.pages ? 0 : ((size_t)a.B + 1) * 4), stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_LAUNCH;
    if (a.one_each) return ATTN_OK;
    cudaLaunchConfig_t cfg = {};
    const int rows = a.rows < R ? a.rows : R;
    const bool by_warp = (int64_t)a.B * a.units * kFewShares >= grid;
    cfg.gridDim = dim3(grid, by_warp ? (unsigned)(rows + kWarps - 1) / kWarps : (unsigned)rows);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, by_warp ? cache_merge_rows_kernel<D, R> : cache_merge_kernel<D, R>, a);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

// Keys of a tile: at most 8 KB of keys and values, three of which a warp's ring
// holds, and no more than a page.
constexpr int tile_keys(int page) { return page < 32 ? page : 32; }

template <int D, int FMT, int NB, int FINE>
int launch_fwd_k(const FwdArgs &a, int kt, unsigned grid, cudaStream_t s) {
    return kt == 16 ? launch_fwd_t<D, FMT, NB, FINE, 16>(a, grid, s) : launch_fwd_t<D, FMT, NB, FINE, 32>(a, grid, s);
}
template <int D>
constexpr int kMostBlocks = D == 64 ? 3 : 2;  // of 8 rows, in the registers of a warp
template <int D, int FMT>
int launch_fwd_n(const FwdArgs &a, int nb, bool fine, int kt, unsigned grid, cudaStream_t s) {
    if (fine) return launch_fwd_k<D, FMT, 1, 1>(a, kt, grid, s);
    if constexpr (kMostBlocks<D> == 3)
        if (nb == 3) return launch_fwd_k<D, FMT, 3, 0>(a, kt, grid, s);
    return nb == 2 ? launch_fwd_k<D, FMT, 2, 0>(a, kt, grid, s) : launch_fwd_k<D, FMT, 1, 0>(a, kt, grid, s);
}

}  // namespace

// fp32 outputs keep q and the weights in 22 bits.
static bool cache_fine(int dtype) { return dtype != ATTN_BF16 && dtype != ATTN_F16; }
// Blocks of 8 rows that a warp takes at once, which share the loads and conversions
// of the codes: as few units as the registers allow, of as few rows as cover them.
static int cache_blocks(int64_t rows, int dtype, int d) {
    const int64_t most = cache_fine(dtype) ? 1 : d == 64 ? kMostBlocks<64> : kMostBlocks<128>;
    const int64_t blocks = rows > 8 ? (rows + 7) / 8 : 1, units = (blocks + most - 1) / most;
    return (int)((blocks + units - 1) / units);
}

// Which kernel takes a call of 16-bit output over all pages.  The 128-row tcgen05
// kernel takes the same time for 9 rows as for 128; the one of this file is faster
// as long as its units leave SMs over or are small.  Times in us here and there,
// 8 kv heads, d = 128 (d = 64):
//      rows   2 x 4096 keys           16 x 4096               1 x 32768
//      32     20.6, 26.7 (17.4, 22.2) 56.9, 57.9 (44.1, 41.3) 36.3, 49.0 (27.1, 37.0)
//      48     24.0, 26.8 (22.1, 22.4) 74.3, 59.9 (58.4, 41.7) 43.7, 49.6 (35.0, 37.6)
//      64     26.5, 27.4 (25.8, 22.7) 92.1, 60.1 (72.3, 42.0) 50.7, 50.0 (42.0, 38.4)
//      96     30.8, 28.3 (28.5, 23.3) 126.9, 61.6 (90.7, 43.7) 67.3, 50.5 (49.4, 39.0)
// One rule for both widths: d = 64 would change over a few rows earlier (32 rows of 16 x 4096).
constexpr int64_t kTcRows = 33, kTcAlways = 65;
static bool cache_tc(int64_t rows, int64_t units, int sms, int dtype, bool listed) {
    return !listed && !cache_fine(dtype) && (rows >= kTcAlways || (rows >= kTcRows && units > sms));
}

// Workspace: the tails [CTA], a state per warp, two per CTA and their lse (the
// tcgen05 kernel: without the warps').  For any number of SMs.
size_t cache_fwd_workspace(int B, int H, int H_kv, int Sq, int d, int dtype, bool listed) {
    const int64_t rows = (int64_t)(H / H_kv) * (listed ? 1 : Sq);
    const size_t R = cache_blocks(rows, dtype, d) * 8;
    const size_t mma = (size_t)kCacheMaxCtas * (16 + (kWarps + 2) * R * d * 4 + 2 * R * 4);
    const size_t tc = (size_t)kCacheMaxCtas * (16 + 2 * 128 * (size_t)d * 4 + 2 * 128 * 4);
    if (cache_tc(rows, INT64_MAX, 0, dtype, listed)) return rows >= kTcAlways || tc > mma ? tc : mma;
    return mma;
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
    a.by_group = fast_div((uint32_t)a.G);
    a.status = status_word_device_ptr();
    if (!a.status) return ATTN_ERR_CUDA;
    const int sms = device_sm_count();
    if (sms <= 0) return ATTN_ERR_CUDA;
    const int nb = cache_blocks(a.rows, dtype, c.d), R = nb * 8;
    const bool fine = cache_fine(dtype);
    a.nrb = (a.rows + R - 1) / R;
    a.units = a.Hkv * a.nseg * a.nrb;
    const int64_t units = (int64_t)B * a.units;  // at most B * H * Sq < 2^31
    if (cache_tc(a.rows, units, sms, dtype, pages != nullptr)) return launch_cache_tc(a, c.d, c.format, workspace, stream);
    a.by_units = fast_div((uint32_t)a.units);
    a.by_per = fast_div((uint32_t)(a.nseg * a.nrb));
    a.by_nrb = fast_div((uint32_t)a.nrb);
    const int kt = tile_keys(c.page);
    // as many CTAs as the longest possible lengths can give every warp a tile
    const int room = sms < kCacheMaxCtas ? sms : kCacheMaxCtas;
    const double most = (double)units * (pages ? (double)n_select * c.page : (double)max_pages * c.page) / kt;
    int64_t ctas = most / kWarps < room ? (int64_t)(most / kWarps) + 1 : room;
    if (ctas > room) ctas = room;
    // A CTA for each unit, if that is not longer for a warp than its share of all the work by
    // more than what sharing a unit costs: by the number of listed pages or the longest possible
    // lengths, and then without the second kernel, or, in the kernel, by the lengths
    const int64_t longest = pages ? (int64_t)n_select * (c.page / kt) : ((int64_t)max_pages * c.page + kt - 1) / kt;
    const double share = pages ? (double)units * longest / ((double)room * kWarps) : 1;
    a.one_each = units <= room && longest <= (share + kSwitch) * kWarps;
    if (a.one_each) ctas = units;
    a.workers = (int)ctas * kWarps;
    a.tail = reinterpret_cast<int4 *>(workspace);
    a.hold = reinterpret_cast<float *>(a.tail + ctas);
    a.po = a.hold + (size_t)a.workers * R * c.d;
    a.pl = a.po + (size_t)2 * ctas * R * c.d;
    if (c.d == 64)
        return c.format == ATTN_CACHE_E4M3 ? launch_fwd_n<64, ATTN_CACHE_E4M3>(a, nb, fine, kt, (unsigned)ctas, stream)
                                           : launch_fwd_n<64, ATTN_CACHE_I8>(a, nb, fine, kt, (unsigned)ctas, stream);
    return c.format == ATTN_CACHE_E4M3 ? launch_fwd_n<128, ATTN_CACHE_E4M3>(a, nb, fine, kt, (unsigned)ctas, stream)
                                       : launch_fwd_n<128, ATTN_CACHE_I8>(a, nb, fine, kt, (unsigned)ctas, stream);
}

}  // namespace attn
