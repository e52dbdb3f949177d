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
//   16-row form (16-bit output, 9 to 16 rows; with a page list, any number above 8):
//     p is rounded once to fp16 (2^-12, as an fp16 output is, or less than a bf16 one).
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
#include "cache_fwd.cuh"
#include "cache_mma.cuh"
#include "sm100_ptx.cuh"

namespace attn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = 24 * 1024;  // shared memory of each warp's tiles, later of its states
constexpr int kMinTiles = 1;  // tiles per worker when there are few
constexpr int kOneEachTiles = 4 * kWarps;  // of a unit that one CTA takes

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
        lp = a.pages[list * a.n_sel + lp];
        if (lp < -1 || lp >= a.max_pages) atomicOr(a.status, kStatusTable);
        if (lp < 0 || lp >= a.max_pages) return d;
    }
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
    d.at = (int)((ph << shift) + sub);
    d.ks = a.ks[ph];
    d.vs = a.vs[ph];
    return d;
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
    constexpr int STEP = KT < 32 ? KT : 32;  // keys of one softmax step
    constexpr int NT = STEP / 8;             // score tiles of 8 keys
    constexpr int KS = STEP / 16;            // k steps of P.V
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
    if (lane == 0) s_has[warp] = 0;
    if (a.one_each) {
        here.b = (int)((uint32_t)blockIdx.x / a.by_units);
        here.unit = blockIdx.x - here.b * a.units;
        if (here.unit == 0 && threadIdx.x == 0) report(here.b);
        here.n = a.pages ? tpu : (clamp_len(a.lens[here.b], a.max_pages, a.page) + KT - 1) / KT;
        const int64_t share = worker_count(here.n, kWarps, 1);
        if (warp < share) {
            here.t = (int)worker_begin(warp, here.n, share);
            n_tiles = (int)worker_begin(warp + 1, here.n, share) - here.t;
        }
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
        workers = worker_count(total, a.workers, kMinTiles);
        w += blockIdx.x * kWarps;
        if (w < workers && total > 0) {
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
        const int left = min(here.n - here.t, n_tiles - i);  // tiles of this unit in the range
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
            int qi, h;
            const bool real = row_of<R>(a, u, g + 8 * hh, qi, h);
            lim[hh] = real ? visible_keys(len, cnt, qi, a.causal) : 0;
            if (real) {
                load_q<D / 4>(a, (((size_t)u.b * a.Hkv * a.G + h) * a.Sq + qi) * D + t * (D / 4), f);
                low = min(low, lim[hh]);
            } else {
#pragma unroll
                for (int e = 0; e < D / 4; ++e) f[e] = 0.f;
            }
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < D / 4; ++e) amax = fmaxf(amax, fabsf(f[e]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float mul, back;
            row_power(amax, mul, back);
            cq[hh] = a.sl2 * back;
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
                float s[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 u4 = lds16(kb + step * D + swizzled<D>(n * 8 + g, t * (D / 64) + c));
                        const uint32_t words[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t b0, b1;
                            U::quad(words[e], b0, b1);
                            const int st = c * 4 + e;
                            mma16816(s[n], qa[st][0], qa[st][1], qa[st][2], qa[st][3], b0, b1);
                        }
                    }
                }
                if constexpr (!WIDE) {  // hi and lo parts of q
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 x = __fadd2_rn(make_float2(s[n][0], s[n][1]), make_float2(s[n][2], s[n][3]));
                        s[n][0] = x.x;
                        s[n][1] = x.y;
                    }
                }
                const bool edge = key0 + step + STEP > low;  // some row does not see every key
                float2 p[H][NT];  // weights of keys 8 n + 2 t and the next
                float c[H];
                auto weights = [&](int hh) {
                    const float f = ks * cq[hh];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float2 z = __ffma2_rn(make_float2(s[n][2 * hh], s[n][2 * hh + 1]), make_float2(f, f),
                                                    make_float2(-top[hh], -top[hh]));
                        p[hh][n] = make_float2(ex2(z.x), ex2(z.y));
                    }
                    if (edge) {
                        const int seen = lim[hh] - (key0 + step + 2 * t);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (8 * n >= seen) p[hh][n].x = 0.f;
                            if (8 * n + 1 >= seen) p[hh][n].y = 0.f;
                        }
                    }
                };
                bool far = false;
#pragma unroll
                for (int hh = 0; hh < H; ++hh) {
                    // a page no key of which the row sees adds nothing, not even its scale's NaN
                    c[hh] = key0 < lim[hh] ? vs * rv[hh] : 0.f;
                    weights(hh);
                    float most = 0.f;
#pragma unroll
                    for (int n = 0; n < NT; ++n) most = ptx::max3(most, p[hh][n].x, p[hh][n].y);
                    far = far || most > 16.f || most * c[hh] > 32768.f;
                }
                if (__any_sync(0xffffffffu, far)) {
                    // new references: the scores' maximum, and the page scale unless what o
                    // holds is larger by now
#pragma unroll
                    for (int hh = 0; hh < H; ++hh) {
                        const float f = ks * cq[hh], sv = key0 < lim[hh] ? vs : 0.f;
                        const int seen = lim[hh] - (key0 + step + 2 * t);
                        float mx = -INFINITY;
#pragma unroll
                        for (int e = 0; e < 2 * NT; ++e)
                            if (!edge || 8 * (e >> 1) + (e & 1) < seen) mx = fmaxf(mx, s[e >> 1][2 * hh + (e & 1)] * f);
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        const float nt = fmaxf(top[hh], mx);
                        const float alpha = ex2(top[hh] - nt);  // 0 from kUnset
                        const float was = alpha * 2048.f / rv[hh];
                        const float nv = mx == -INFINITY ? rv[hh] : 2048.f / fmaxf(fmaxf(was, sv), 0x1p-100f);
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
                        c[hh] = sv * nv;
                        weights(hh);
                    }
                }
                uint32_t pa[KS][4];
#pragma unroll
                for (int hh = 0; hh < H; ++hh) {
                    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        sum = __fadd2_rn(sum, p[hh][n]);
                        const float2 w = __fmul2_rn(p[hh][n], make_float2(c[hh], c[hh]));
                        const uint32_t hi = pack_f16(w.x, w.y);
                        if constexpr (WIDE) {
                            pa[n / 2][(n & 1) * 2 + hh] = hi;
                        } else {
                            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                            pa[n / 2][(n & 1) * 2] = hi;
                            pa[n / 2][(n & 1) * 2 + 1] = pack_f16(w.x - b.x, w.y - b.y);
                        }
                    }
                    l[hh] += sum.x + sum.y;
                }
#pragma unroll
                for (int st = 0; st < KS; ++st) {
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
                            uint32_t a0, a1, b0, b1;
                            U::quad(__byte_perm(r[0][q], r[1][q], hf ? 0x7362 : 0x5140), a0, a1);
                            U::quad(__byte_perm(r[2][q], r[3][q], hf ? 0x7362 : 0x5140), b0, b1);
                            mma16816(acc[4 * q + 2 * hf], pa[st][0], pa[st][1], pa[st][2], pa[st][3], a0, b0);
                            mma16816(acc[4 * q + 2 * hf + 1], pa[st][0], pa[st][1], pa[st][2], pa[st][3], a1, b1);
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
            if (!before && !after) {
                size_t row;
                if (!out_row<R>(a, u, r, row)) continue;
#pragma unroll
                for (int e = 0; e < D / 4; e += 8) store_o8(a, row * D + t * (D / 4) + e, f + e);
                if (a.lse && t == 0) a.lse[row] = lse2 * kLn2;
            } else if (in_bounds(w < (int)gridDim.x * kWarps, a.status)) {
                float4 *p = reinterpret_cast<float4 *>(keep + r * D + t * (D / 4));
#pragma unroll
                for (int e = 0; e < D / 16; ++e) p[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                if (t == 0) s_lse[warp][before ? 0 : 1][r] = lse2;
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
#pragma unroll
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
            float o[D / 32] = {};
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float wk = __shfl_sync(0xffffffffu, wt, k);
                if (k >= n) continue;
                const float *src = s_keep[first + k][k == 0 ? side : 0] + r * D + lane;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) o[e] = fmaf(wk, src[32 * e], o[e]);
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
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
    if (!set_smem_limit_once(reinterpret_cast<const void *>(fwd), (int)(ring + (kMaxCacheBatch + 1) * 4)))
        return ATTN_ERR_LAUNCH;
    fwd<<<grid, kThreads, ring + (a.pages ? 0 : ((size_t)a.B + 1) * 4), stream>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_LAUNCH;
    if (a.one_each) return ATTN_OK;
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

// Query rows per kv head from which the 128-row tcgen05 kernel runs (16-bit
// outputs, all pages).
constexpr int64_t kTcRows = 33;
static bool cache_tc(int64_t rows, int dtype, bool listed) {
    return !listed && (dtype == ATTN_BF16 || dtype == ATTN_F16) && rows >= kTcRows;
}
// The 16-row form where the output's own rounding hides the weights' and the
// rows do not fit eight.
static bool cache_wide(int64_t rows, int dtype) {
    return (dtype == ATTN_BF16 || dtype == ATTN_F16) && rows > 8;
}

// Workspace: the tails [CTA], a state per warp, two per CTA and their lse (the
// tcgen05 kernel: without the warps').
size_t cache_fwd_workspace(int B, int H, int H_kv, int Sq, int d, int dtype, bool listed) {
    const int64_t rows = (int64_t)(H / H_kv) * (listed ? 1 : Sq);
    if (cache_tc(rows, dtype, listed))
        return (size_t)kCacheMaxCtas * (16 + 2 * 128 * (size_t)d * 4 + 2 * 128 * 4);
    const size_t R = cache_wide(rows, dtype) ? 16 : 8;
    return (size_t)kCacheMaxCtas * (16 + (kWarps + 2) * R * d * 4 + 2 * R * 4);
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
    if (cache_tc(a.rows, dtype, pages != nullptr)) return launch_cache_tc(a, c.d, c.format, workspace, stream);
    const bool wide = cache_wide(a.rows, dtype);
    const int R = wide ? 16 : 8;
    a.nrb = (a.rows + R - 1) / R;
    a.units = a.Hkv * a.nseg * a.nrb;
    const int64_t units = (int64_t)B * a.units;  // at most B * H * Sq < 2^31
    a.by_units = fast_div((uint32_t)a.units);
    a.by_per = fast_div((uint32_t)(a.nseg * a.nrb));
    a.by_nrb = fast_div((uint32_t)a.nrb);
    const int kt = tile_keys(c.d, c.page);
    const int sms = device_sm_count();
    if (sms <= 0) return ATTN_ERR_CUDA;
    // as many CTAs as the longest possible lengths can give every warp a tile
    const double most = (double)units * (pages ? (double)n_select * c.page : (double)max_pages * c.page) / kt;
    int64_t ctas = most / kWarps < sms ? (int64_t)(most / kWarps) + 1 : sms;
    if (ctas > kCacheMaxCtas) ctas = kCacheMaxCtas;
    if (ctas > sms) ctas = sms;
    // Few units of few tiles, by the longest possible lengths: a CTA each.  Four tiles a warp
    // take as long as one and the second kernel, which is then not launched (one sequence of
    // 1000 tokens, 8 kv heads: 11.1 us either way on the device, 17.1 and 14.5 us a call)
    const int longest = pages ? n_select * (c.page / kt) : (int)(((int64_t)max_pages * c.page + kt - 1) / kt);
    a.one_each = units <= ctas && longest <= kOneEachTiles;
    if (a.one_each) ctas = units;
    a.workers = (int)ctas * kWarps;
    a.tail = reinterpret_cast<int4 *>(workspace);
    a.hold = reinterpret_cast<float *>(a.tail + ctas);
    a.po = a.hold + (size_t)a.workers * R * c.d;
    a.pl = a.po + (size_t)2 * ctas * R * c.d;
    if (c.d == 64)
        return c.format == ATTN_CACHE_E4M3 ? launch_fwd_w<64, ATTN_CACHE_E4M3>(a, wide, kt, (unsigned)ctas, stream)
                                           : launch_fwd_w<64, ATTN_CACHE_I8>(a, wide, kt, (unsigned)ctas, stream);
    return c.format == ATTN_CACHE_E4M3 ? launch_fwd_w<128, ATTN_CACHE_E4M3>(a, wide, kt, (unsigned)ctas, stream)
                                       : launch_fwd_w<128, ATTN_CACHE_I8>(a, wide, kt, (unsigned)ctas, stream);
}

}  // namespace attn
