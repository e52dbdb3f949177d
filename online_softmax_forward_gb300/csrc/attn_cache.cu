// attn_cache.cu -- the paged 8-bit cache: quantising new keys and values into
// it (append) and reading them back (read).
//
// Layout: codes [n_pages][H_kv][page][d], one scale per (page, kv head), and
// for the keys the smallest and largest code of each channel per (page, kv
// head) as [2][d] codes.  A (page, head) block is one contiguous piece, so one
// CTA owns it: it alone decides the block's scale and no atomics are needed.
//
// Append, per block and tensor, with x the rows that land in it:
//     s  = max(s_old if the block holds older rows, pow2 scale of amax |x|)
//     codes of x = rn(x / s);  older codes = rn(code * s_old / s) when s grew
//     bounds = min / max (older bounds rounded the same way, codes of x)
// Rounding is monotone, so the bounds are the codes of the smallest and largest
// x of each channel, and no older row is read again for them.  Older rows are
// read only when the scale grows.  The new rows are read once: they wait in
// registers, as they lie in memory, until the block's scale is known.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_internal.h"
#include "cache_codec.cuh"
#include "cache_index.h"

namespace attn {
namespace {


struct AppendArgs {
    const void *x[2];   // new keys, values [B][Hkv][S][d]
    uint8_t *codes[2];  // [n_pages][Hkv][page][d]
    float *scale[2];    // [n_pages][Hkv]
    uint8_t *bounds;    // [n_pages][Hkv][2][d], keys only
    const int32_t *table, *pos, *counts;
    int B, S, Hkv, page, page_shift, n_pages, max_pages, touched;
    FastDiv by_heads, by_touched;
    int *status;
};

// Threads of a CTA: four rows each for pages up to 64.  With 256 threads for all, two
// prompts (8192 and 5462 tokens, 32 heads) take 142 us in pages of 16 (so 56) and 80 in
// pages of 32 (53), with d = 64 and int8 40 in pages of 64 (29).
template <int D, int MOST>
constexpr int kAppendThreads = MOST <= 64 ? MOST * D / 32 : 256;

// CTAs of an SM.  A CTA is a chain of waits (positions, rows, the block's maximum),
// which others hide: as many as leave each thread the registers for its rows.  The two
// prompts above, d = 128: bf16 52 us with eight of 32 registers (five: 71,
// before the instructions were fewer); fp32 83 us with four (five spill: 92, three:
// 112); fp32 with pages of 128 85 us with two, 94 with three.
template <int D, int DT, int MOST>
constexpr int kAppendCtasOf256 = DT != 0 ? (MOST == 128 ? 4 : 8) : D == 128 ? (MOST == 128 ? 2 : 4) : 4;
template <int D, int DT, int MOST>
constexpr int kAppendCtas = kAppendCtasOf256<D, DT, MOST> * (256 / kAppendThreads<D, MOST>) > 32
                                ? 32  // of an SM at most
                                : kAppendCtasOf256<D, DT, MOST> * (256 / kAppendThreads<D, MOST>);

// One CTA per (touched page of a sequence, kv head, keys or values).
// MOST: rows of the page, which registers hold.
// Bound by memory: 95 to 97 % of the copy rate in the case above.  It is also near the
// issue rate, so a page is found without divisions, and keys' ranges and values'
// magnitudes are kept as packed pairs of 16 bits until a warp's rows are joined.
template <int D, int FMT, int DT, int MOST>
__global__ void __launch_bounds__((kAppendThreads<D, MOST>), (kAppendCtas<D, DT, MOST>)) cache_append_kernel(const AppendArgs a) {
    constexpr int G = D / 8;               // 8-channel groups of a row: one per thread
    constexpr int T = kAppendThreads<D, MOST>;
    constexpr int RL = T / G;              // rows at a time
    constexpr int N = MOST / RL;
    constexpr int kW = T / 32;
    static_assert(T >= 2 * (D / 4), "the bounds' threads");
    using Range = codec::Range8<DT>;
    using Edge = typename std::conditional<DT == 0, float, uint16_t>::type;
    __shared__ uint32_t red[kW];
    __shared__ __align__(16) Edge edge[2][kW][D];  // smallest and largest by warp
    const int which = blockIdx.x & 1;
    const uint32_t page_of = (blockIdx.x >> 1) / a.by_heads;
    const int hk = (int)((blockIdx.x >> 1) - page_of * a.Hkv);
    const int b = (int)(page_of / a.by_touched);
    const int tp = (int)(page_of - (uint32_t)b * a.touched);
    if (!in_bounds(b < a.B && hk < a.Hkv, a.status)) return;
    const int pos = a.pos[b];
    int cnt = a.counts ? a.counts[b] : a.S;
    if (cnt < 0 || cnt > a.S || pos < 0) {  // nothing of this sequence is written
        if (threadIdx.x == 0) atomicOr(a.status, kStatusTable);
        return;
    }
    // Without rows the page at `pos` is not looked at either: it may be another's by now.
    if (cnt == 0) return;
    const int64_t end = (int64_t)pos + cnt;
    const int64_t lp = (pos >> a.page_shift) + (int64_t)tp;  // logical page
    const int64_t first = lp << a.page_shift;                // its first position
    if (first >= end) return;
    const int r0 = pos > first ? (int)(pos - first) : 0;                  // first new row
    const int r1 = end - first < a.page ? (int)(end - first) : a.page;    // past the last
    const void *xs = which ? a.x[1] : a.x[0];
    const int g = threadIdx.x % G, rl = threadIdx.x / G, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // row r of the page is row first + r - pos of x
    const size_t src = (((size_t)b * a.Hkv + hk) * a.S + (size_t)(first - pos + rl)) * D + g * 8;

    // the rows are asked for before the page that they go to
    codec::Raw8<DT> raw[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int r = rl + n * RL;
        const size_t i = src + n * (RL * D);
        if (r >= r0 && r < r1 && in_bounds(i + 8 <= (size_t)a.B * a.Hkv * a.S * D, a.status))
            raw[n].load(xs, i);
    }
    const int phys = lp < a.max_pages ? a.table[(int64_t)b * a.max_pages + lp] : -1;
    if (phys < 0 || phys >= a.n_pages) {  // the rows have no page: skipped and reported
        if (threadIdx.x == 0) atomicOr(a.status, kStatusTable);
        return;
    }
    const int64_t ph = (int64_t)phys * a.Hkv + hk;
    if (!in_bounds(ph < (int64_t)a.n_pages * a.Hkv && r1 <= a.page, a.status)) return;
    uint8_t *codes = (which ? a.codes[1] : a.codes[0]) + (ph << a.page_shift) * D;
    float *scale = (which ? a.scale[1] : a.scale[0]) + ph;
    const float before = r0 > 0 ? *scale : 0.f;
    uint32_t amax;  // as bits: a NaN's exceed infinity's
    if (which == 0 && a.bounds) {
        Range range;
        range.clear();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int r = rl + n * RL;
            if (r >= r0 && r < r1) range.add(raw[n]);
        }
#pragma unroll
        for (int o = G; o < 32; o <<= 1) range.join(o);  // the warp's rows
        amax = range.largest();
        if (lane < G) {
            constexpr int kE = 16 / sizeof(Edge);  // channels of a 16-byte store
#pragma unroll
            for (int e = 0; e < 8 / kE; ++e) {
                const uint32_t *l = range.lo + 4 * e, *h = range.hi + 4 * e;
                *reinterpret_cast<uint4 *>(&edge[0][warp][g * 8 + e * kE]) = make_uint4(l[0], l[1], l[2], l[3]);
                *reinterpret_cast<uint4 *>(&edge[1][warp][g * 8 + e * kE]) = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
    } else {
        uint32_t m[Range::kN] = {};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int r = rl + n * RL;
            if (r >= r0 && r < r1) Range::add_magnitudes(m, raw[n]);
        }
        amax = Range::largest(m);
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (lane == 0) red[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) amax = max(amax, red[w]);
    const float mine = codec::scale_for<FMT>(__uint_as_float(amax));
    const float now = (before != before || mine != mine) ? __int_as_float(0x7fc00000)
                                                         : fmaxf(before, mine);
    const float inv = codec::inverse_scale(now);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int r = rl + n * RL;
        if (r < r0 || r >= r1 || !in_bounds(((size_t)rl * D + g * 8) + n * (RL * D) + 8 <= (size_t)a.page * D, a.status)) continue;
        uint2 c = make_uint2(0, 0);
        if (inv > 0.f) {
            float f[8];
            raw[n].widen(f);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 y = __fmul2_rn(make_float2(f[e], f[e + 1]), make_float2(inv, inv));
                f[e] = y.x;
                f[e + 1] = y.y;
            }
            c.x = codec::encode4<FMT>(f[0], f[1], f[2], f[3]);
            c.y = codec::encode4<FMT>(f[4], f[5], f[6], f[7]);
        }
        *reinterpret_cast<uint2 *>(codes + (rl * D + g * 8) + n * (RL * D)) = c;
    }
    const bool grew = r0 > 0 && !(now == before);  // also when the block turned NaN
    const float ratio = now > 0.f ? before * inv : 0.f;
    if (grew) {  // the older rows under the larger scale
        for (int i = threadIdx.x; i < r0 * (D / 8); i += T) {
            if (!in_bounds((i + 1) * 8 <= a.page * D, a.status)) break;
            uint2 *p = reinterpret_cast<uint2 *>(codes) + i;
            uint2 c = *p;
            float f[8];
            codec::decode4<FMT>(c.x, f);
            codec::decode4<FMT>(c.y, f + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = ratio > 0.f ? f[e] * ratio : 0.f;
            c.x = codec::encode4<FMT>(f[0], f[1], f[2], f[3]);
            c.y = codec::encode4<FMT>(f[4], f[5], f[6], f[7]);
            *p = c;
        }
    }
    if (threadIdx.x == 0) *scale = now;
    // thread t: side t / (D / 4), four channels
    if (which == 0 && a.bounds && threadIdx.x < 2 * (D / 4)) {
        const int side = threadIdx.x / (D / 4), c4 = threadIdx.x % (D / 4);
        uint32_t *p = reinterpret_cast<uint32_t *>(a.bounds + ((size_t)ph * 2 + side) * D) + c4;
        constexpr int kV = DT == 0 ? 4 : 2;  // words of four channels
        uint32_t x[kV];
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            const uint32_t *y = reinterpret_cast<const uint32_t *>(&edge[side][w][c4 * 4]);
#pragma unroll
            for (int e = 0; e < kV; ++e)
                x[e] = w == 0 ? y[e] : side ? Range::most(x[e], y[e]) : Range::least(x[e], y[e]);
        }
        const uint32_t all[8] = {x[0], x[1], x[kV - 2], x[kV - 1], 0, 0, 0, 0};
        float f[8];
        Range::widen(all, f);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = inv > 0.f ? f[e] * inv : 0.f;
        if (r0 > 0) {
            float o[4];
            codec::decode4<FMT>(*p, o);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (grew) o[e] = ratio > 0.f ? o[e] * ratio : 0.f;
                f[e] = side ? fmaxf(f[e], o[e]) : fminf(f[e], o[e]);
            }
        }
        *p = codec::encode4<FMT>(f[0], f[1], f[2], f[3]);
    }
}

struct ReadArgs {
    const uint8_t *codes[2];
    const float *scale[2];
    void *out[2];  // [B][Hkv][S][d]
    const int32_t *table, *lens;
    int B, S, Hkv, page, page_shift, tile_shift, n_pages, max_pages, tiles;
    FastDiv by_heads, by_tiles;
    int *status;
};

constexpr int kReadThreads = 256;

// One CTA per (tile of a sequence, kv head, keys or values), a tile being 128 rows, or
// fewer, but a page at least, where that leaves SMs without work (a few short
// sequences: 4.3 us a page each, 6.5 us in tiles of 128).  16 codes a thread and step,
// 16-byte loads and stores; 4 codes for fp32, whose stores then lie side by side.
// Bound by memory: four contexts of 32k tokens, 8 kv heads, d = 128, to bf16 122 us,
// 97 % of the copy rate, with pages of 16 123 us (194 with a page to a CTA).
template <int D, int FMT, int DT>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const ReadArgs a) {
    constexpr int E = DT == 0 ? 4 : 16;  // codes of a step
    constexpr int G = D / E;
    __shared__ int64_t s_block[8];  // (page, kv head) blocks of the tile, -1: rows read as zero
    __shared__ float s_scale[8];
    const int which = blockIdx.x & 1;
    const uint32_t block_of = (blockIdx.x >> 1) / a.by_tiles;
    const int tile = (int)((blockIdx.x >> 1) - block_of * a.tiles);
    const int b = (int)(block_of / a.by_heads);
    const int hk = (int)(block_of - (uint32_t)b * a.Hkv);
    if (!in_bounds(b < a.B && hk < a.Hkv, a.status)) return;
    const int len0 = a.lens[b];
    const int len = clamp_len(len0, a.max_pages, a.page);
    if (len != len0 && threadIdx.x == 0) atomicOr(a.status, kStatusTable);
    const int64_t first = (int64_t)tile << a.tile_shift;
    const int rows = a.S - first < 1 << a.tile_shift ? (int)(a.S - first) : 1 << a.tile_shift;
    const int held = (int)max((int64_t)0, min((int64_t)rows, (int64_t)len - first));
    if (threadIdx.x < 1u << (a.tile_shift - a.page_shift)) {
        int64_t block = -1;
        const int64_t lp = (first >> a.page_shift) + threadIdx.x;
        if (((int)threadIdx.x << a.page_shift) < held && in_bounds(lp < a.max_pages, a.status)) {
            const int phys = a.table[(int64_t)b * a.max_pages + lp];
            if (phys < 0 || phys >= a.n_pages) atomicOr(a.status, kStatusTable);  // read as zero, reported
            else block = (int64_t)phys * a.Hkv + hk;
            if (!in_bounds(block < (int64_t)a.n_pages * a.Hkv, a.status)) block = -1;
        }
        s_block[threadIdx.x] = block;
        s_scale[threadIdx.x] = block < 0 ? 0.f : (which ? a.scale[1] : a.scale[0])[block];
    }
    __syncthreads();
    const uint8_t *codes = which ? a.codes[1] : a.codes[0];
    const size_t dst = (((size_t)b * a.Hkv + hk) * a.S + first) * D;
    void *out = which ? a.out[1] : a.out[0];
    for (int i = threadIdx.x; i < rows * G; i += kReadThreads) {
        const int r = i / G, in_page = r & (a.page - 1);
        const int64_t block = s_block[r >> a.page_shift];
        float f[E];
        if (r < held && block >= 0 && in_bounds(in_page * D + (i % G + 1) * E <= a.page * D, a.status)) {
            const float s = s_scale[r >> a.page_shift];
            const uint8_t *c = codes + ((block << a.page_shift) + in_page) * D + i % G * E;
            if constexpr (DT == 0) {
                codec::decode4<FMT>(*reinterpret_cast<const uint32_t *>(c), f);
            } else {
                const uint4 w = *reinterpret_cast<const uint4 *>(c);
                codec::decode4<FMT>(w.x, f);
                codec::decode4<FMT>(w.y, f + 4);
                codec::decode4<FMT>(w.z, f + 8);
                codec::decode4<FMT>(w.w, f + 12);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] *= s;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = 0.f;
        }
        const size_t at = dst + (size_t)i * E;
        if (!in_bounds(at + E <= (size_t)a.B * a.Hkv * a.S * D, a.status)) continue;
        if constexpr (DT == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = codec::clamped(f[e], 3.402823466e38f);
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(out) + at) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
            uint4 *p = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(out) + at);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                p[e] = make_uint4(codec::pack2_clamped<DT>(f[8 * e], f[8 * e + 1]),
                                  codec::pack2_clamped<DT>(f[8 * e + 2], f[8 * e + 3]),
                                  codec::pack2_clamped<DT>(f[8 * e + 4], f[8 * e + 5]),
                                  codec::pack2_clamped<DT>(f[8 * e + 6], f[8 * e + 7]));
        }
    }
}

int log2_of(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// f(integral constants D, FMT, DT) for the runtime values
template <template <int, int, int> class F, typename... A>
int dispatch(int d, int format, int dt, A... args) {
#define ATTN_CASE(DD, FF, TT) \
    if (d == DD && format == FF && dt == TT) return F<DD, FF, TT>::run(args...);
#define ATTN_CASES(FF) \
    ATTN_CASE(64, FF, 0) ATTN_CASE(64, FF, 1) ATTN_CASE(64, FF, 2) \
    ATTN_CASE(128, FF, 0) ATTN_CASE(128, FF, 1) ATTN_CASE(128, FF, 2)
    ATTN_CASES(ATTN_CACHE_E4M3)
    ATTN_CASES(ATTN_CACHE_I8)
#undef ATTN_CASES
#undef ATTN_CASE
    return ATTN_ERR_INVALID_ARG;
}

template <int D, int FMT, int DT>
struct RunAppend {
    static int run(const AppendArgs *a, unsigned grid, cudaStream_t s) {
        if (a->page == 16) cache_append_kernel<D, FMT, DT, 16><<<grid, kAppendThreads<D, 16>, 0, s>>>(*a);
        else if (a->page == 32) cache_append_kernel<D, FMT, DT, 32><<<grid, kAppendThreads<D, 32>, 0, s>>>(*a);
        else if (a->page == 64) cache_append_kernel<D, FMT, DT, 64><<<grid, kAppendThreads<D, 64>, 0, s>>>(*a);
        else cache_append_kernel<D, FMT, DT, 128><<<grid, kAppendThreads<D, 128>, 0, s>>>(*a);
        return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
    }
};
template <int D, int FMT, int DT>
struct RunRead {
    static int run(const ReadArgs *a, unsigned grid, cudaStream_t s) {
        cache_read_kernel<D, FMT, DT><<<grid, kReadThreads, 0, s>>>(*a);
        return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
    }
};

}  // namespace

int launch_cache_append(const attn_cache &c, const void *k, const void *v, const int32_t *table,
                        int max_pages, const int32_t *pos, const int32_t *counts, int B, int S,
                        int dtype, cudaStream_t stream) {
    const int64_t touched = touched_pages(S, c.page);
    const int64_t grid = (int64_t)B * c.H_kv * touched * 2;  // the caller checked it
    AppendArgs a = {{k, v}, {(uint8_t *)c.k, (uint8_t *)c.v}, {c.k_scale, c.v_scale},
                    (uint8_t *)c.k_bounds, table, pos, counts, B, S, c.H_kv, c.page, log2_of(c.page), c.n_pages,
                    max_pages, (int)touched, fast_div((uint32_t)c.H_kv), fast_div((uint32_t)touched),
                    status_word_device_ptr()};
    if (!a.status) return ATTN_ERR_CUDA;
    return dispatch<RunAppend>(c.d, c.format, dtype, (const AppendArgs *)&a, (unsigned)grid, stream);
}

int launch_cache_read(const attn_cache &c, const int32_t *table, int max_pages, const int32_t *lens,
                      void *k, void *v, int B, int S, int dtype, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return ATTN_ERR_CUDA;
    int shift = 7;
    auto tiles_of = [&](int sh) { return ((int64_t)S + (1 << sh) - 1) >> sh; };
    while (shift > log2_of(c.page) && (int64_t)B * c.H_kv * tiles_of(shift) * 2 < 8 * (int64_t)sms) --shift;
    const int64_t tiles = tiles_of(shift);
    const int64_t grid = (int64_t)B * c.H_kv * tiles * 2;
    ReadArgs a = {{(const uint8_t *)c.k, (const uint8_t *)c.v}, {c.k_scale, c.v_scale}, {k, v},
                  table, lens, B, S, c.H_kv, c.page, log2_of(c.page), shift, c.n_pages, max_pages, (int)tiles,
                  fast_div((uint32_t)c.H_kv), fast_div((uint32_t)tiles), status_word_device_ptr()};
    if (!a.status) return ATTN_ERR_CUDA;
    return dispatch<RunRead>(c.d, c.format, dtype, (const ReadArgs *)&a, (unsigned)grid, stream);
}

}  // namespace attn
