// attn_cache_tc.cu -- attention over the paged 8-bit cache for many query rows
// per kv head (prompt chunks, draft tokens), on tcgen05.
//
// The operation and the numbering of the work are those of attn_cache_fwd.cu.  A
// unit here is (sequence, kv head, block of 128 rows); its keys are walked in
// tiles of 128, and each CTA (one per SM) takes one contiguous range of tiles.
// With 128 rows the products are no longer free, and one conversion of the codes
// to fp16 serves all of them:
//
//   warps 8-10  load the codes of the keys and 11-13 those of the values, a tile
//               ahead in registers, convert them to fp16, exact, and write the
//               MMA's 128-byte-swizzled tiles into two rings of stages;
//   warps 0-3   softmax of the even tiles (t = 0), 4-7 of the odd ones (t = 1), a
//               thread per row: S_t out of tensor memory, the pages' scales
//               applied per 16 keys, P_t as fp16 over the first half of S_t;
//   warps 14-15 issue the products of t = 0 and 1, S_t = Q K_j^T and O_t += P_t V_j.
//
// The two warpgroups keep states of their own (top, rv, l and O_t, references moved
// only when 16 weights would pass 2^10 or fp16's range, as in attn_cache_fwd.cu), so
// that one exponentiates while the other's products run; they are joined when the
// unit ends.  P in fp16 is rounded by 2^-12, so this kernel serves the 16-bit
// outputs; what is below 2^-19 of a row's largest weight times page scale keeps fewer
// bits, and nothing below 2^-30.  A warp without a real row (few drafts, few heads)
// only keeps step.
//
// A tile's S, P and products go in halves of 64 keys.  Tensor memory (512 columns)
// is full with S_0 [0, 128), S_1 [128, 256), O_0 from 256 and O_1 from 256 + D, so
// P of a half lies over the first half of its S, and S_t(j + 2) of a half waits for
// the product that reads it; the other half keeps the tensor cores and the warps
// busy meanwhile, and 64 weights are what the registers of 16 warps hold.  Every
// wait is bounded, as in attn_tc.cu.
//
// Bound: 1024 rows on 4096 keys, 2 sequences of 8 kv heads, d = 128: 54 us, 32 % of the
// bf16 peak on 128 of the SMs, one unit each.  A tile takes 3400 clocks, of which the
// products need 1300; by a clock trace the products wait for keys 17 to 26 % and for
// weights 13 to 21 %, the converters are at work 80 % of the time (half of it converting,
// half looking up and fetching) and the softmax warps half of it, each a chain of loads,
// conversions and stores that waits for itself.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "attn_internal.h"
#include "cache_fwd.cuh"
#include "cache_mma.cuh"
#include "sm100_ptx.cuh"
#include "tc_common.cuh"

namespace attn {
namespace {

__device__ __forceinline__ uint4 ldg16(const uint8_t *p) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}

constexpr int R = 128;   // rows of a unit
constexpr int KT = 128;  // keys of a tile
constexpr int kConvertWarp0 = 8;  // 8 .. 10 keys, 11 .. 13 values
constexpr int kConverters = 3;
constexpr int kIssueWarp0 = 14;   // 14, 15
constexpr int kThreads = 16 * 32;
constexpr int kScaleRing = 8;       // tiles whose page scales are kept
constexpr int kScaleWords = 20;     // 8 of keys, 8 of values, the pieces that are missing; 16-byte steps
constexpr uint32_t kTmemCols = 512;
// What a second unit costs a CTA (its queries, the first scores, the join), in tiles:
// about 20 000 clocks against 3 400 a tile.  The chunk of the header, when it took 57 us
// with a unit per CTA: 64 with equal ranges.
constexpr int kSwitch = 6;
constexpr float kLargest = 1024.f;  // of 16 keys' sum of weights; 32 * 1024 fits fp16
constexpr float kBase = 32.f;       // weight times page scale times rv, at its largest after a move

struct Bars {
    uint64_t q_full, q_empty;
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [warpgroup][half of the tile]
    uint64_t o_empty, joined, mma_done[2];
    uint64_t sc_full[kScaleRing];
    uint32_t tmem_base;
    int abort_flag;
};

template <int D>
struct Cfg {
    static constexpr int kChunks = D / 64;
    static constexpr int kChunkBytes = 128 * 128;             // 64 channels of 128 rows, fp16
    static constexpr int kTile = kChunks * kChunkBytes;       // Q, K or V tile
    static constexpr int kKeyStages = D == 128 ? 2 : 4;
    static constexpr int kValueStages = D == 128 ? 3 : 4;
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kTile;
    static constexpr int kOffV = kOffK + kKeyStages * kTile;
    static constexpr int kOffScale = kOffV + kValueStages * kTile;       // [ring][words]
    static constexpr int kOffBack = kOffScale + kScaleRing * kScaleWords * 4;     // [2][128] fp32
    static constexpr int kOffState = kOffBack + 2 * R * 4;               // [2][2][3][128] fp32
    static constexpr int kOffBar = kOffState + 2 * 2 * 3 * R * 4;
    static constexpr int kOffPrefix = kOffBar + 512;
    static constexpr int kSmem = kOffPrefix + (kMaxCacheBatch + 1) * 4 + 1024;  // + alignment
};
static_assert(sizeof(Bars) <= 512, "barrier block");
static_assert(Cfg<128>::kSmem <= 227 * 1024 && Cfg<64>::kSmem <= 227 * 1024, "shared memory");

// A piece of a unit inside the CTA's range, the same for every role.
struct Piece {
    Unit u;
    int len, cnt;
    int t0, left;  // first tile of the unit, tiles in the range
    int live;      // of those, tiles that some row sees
};

struct TcArgs {
    FwdArgs f;
    unsigned long long timeout_ns;
};

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) cache_tc_kernel(const __grid_constant__ TcArgs args) {
    using C = Cfg<D>;
    using U = Unpack<FMT>;
    const FwdArgs &a = args.f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *bars = reinterpret_cast<Bars *>(sm + C::kOffBar);
    int *prefix = reinterpret_cast<int *>(sm + C::kOffPrefix);
    float *scales = reinterpret_cast<float *>(sm + C::kOffScale);
    float *backs = reinterpret_cast<float *>(sm + C::kOffBack);
    float *state = reinterpret_cast<float *>(sm + C::kOffState);
    __shared__ int warp_sums[kThreads / 32];
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const Watch watch{&bars->abort_flag, a.status, args.timeout_ns};
    auto bar = [&](uint64_t &b) { return ptx::smem_addr(&b); };
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        ptx::mbar_init(bar(bars->q_full), 256);
        ptx::mbar_init(bar(bars->q_empty), 2);
        for (int s = 0; s < 4; ++s) {
            ptx::mbar_init(bar(bars->k_full[s]), kConverters * 32);
            ptx::mbar_init(bar(bars->k_empty[s]), 1);
            ptx::mbar_init(bar(bars->v_full[s]), kConverters * 32);
            ptx::mbar_init(bar(bars->v_empty[s]), 1);
        }
        for (int t = 0; t < 2; ++t) {
            for (int h = 0; h < 2; ++h) {
                ptx::mbar_init(bar(bars->s_full[t][h]), 1);
                ptx::mbar_init(bar(bars->p_full[t][h]), 128);
                ptx::mbar_init(bar(bars->pv_done[t][h]), 1);
            }
            ptx::mbar_init(bar(bars->mma_done[t]), 1);
        }
        ptx::mbar_init(bar(bars->o_empty), 256);
        ptx::mbar_init(bar(bars->joined), 256);
        for (int s = 0; s < kScaleRing; ++s) ptx::mbar_init(bar(bars->sc_full[s]), 1);
        bars->abort_flag = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 0) {
        ptx::tmem_alloc(ptx::smem_addr(&bars->tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    scan_lengths<kThreads>(a, KT, prefix, warp_sums);
    const int64_t total = (int64_t)prefix[a.B] * a.units;
    // sequences without a token have no tile: o = 0, lse = -inf
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (prefix[b] != prefix[b + 1]) continue;
        const size_t row0 = (size_t)b * a.Hkv * a.G * a.Sq, n = (size_t)a.Hkv * a.G * a.Sq;
        const float z[8] = {};
        for (size_t e = threadIdx.x; e < n * (D / 8); e += kThreads) store_o8(a, row0 * D + e * 8, z);
        if (a.lse)
            for (size_t e = threadIdx.x; e < n; e += kThreads) a.lse[row0 + e] = -INFINITY;
    }
    auto tiles = [&](int b) { return prefix[b + 1] - prefix[b]; };
    const int64_t workers = worker_count(total, a.workers, 1);
    int64_t x0 = 0;
    int n_tiles = 0;
    Place start = {0, 0, 0, 1};
    // Equal ranges, or a unit each where that is no longer for the longest one
    int longest = 0;
    for (int b = threadIdx.x; b < a.B; b += kThreads) longest = max(longest, tiles(b));
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) warp_sums[threadIdx.x >> 5] = longest;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) longest = max(longest, warp_sums[w]);
    const int64_t all_units = (int64_t)a.B * a.units;
    const bool one_each = all_units <= gridDim.x && longest <= (total + workers - 1) / workers + kSwitch;
    int4 tail = make_int4(0, 0, 0, 0);  // the unit that runs over the end of the range, if it began in it
    if (one_each) {
        if (blockIdx.x < all_units) {
            start.b = blockIdx.x / a.units;
            start.unit = blockIdx.x - start.b * a.units;
            start.n = n_tiles = tiles(start.b);
        }
    } else if (blockIdx.x < workers && total > 0) {
        x0 = worker_begin(blockIdx.x, total, workers);
        n_tiles = (int)(worker_begin(blockIdx.x + 1, total, workers) - x0);
        start = place_of(a, prefix, 0, x0);
        const int64_t x1 = x0 + n_tiles;
        const Place p = place_of(a, prefix, 0, x1 - 1);
        const int64_t end = x1 - 1 - p.t + p.n;
        if (end > x1 && x1 - 1 - p.t >= x0)
            tail = make_int4(1, (int)worker_of(end - 1, total, workers), p.b, p.unit);
    }
    if (threadIdx.x == 0) a.tail[blockIdx.x] = tail;
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    const uint32_t sQ = ptx::smem_addr(sm + C::kOffQ), sK = ptx::smem_addr(sm + C::kOffK);
    const uint32_t sV = ptx::smem_addr(sm + C::kOffV);

    // the piece at `here` when `done` tiles of the range lie before it
    auto piece_at = [&](const Place &here, int done) {
        Piece p;
        p.u = unit_at(a, here.b, here.unit);
        p.len = clamp_len(a.lens[here.b], a.max_pages, a.page);
        p.cnt = a.counts ? min(max(a.counts[here.b], 0), a.Sq) : a.Sq;
        p.t0 = here.t;
        p.left = min(here.n - here.t, n_tiles - done);
        // the block's last query that is one of the sequence's sees the most keys
        int first, last, h;
        row_of<R>(a, p.u, 0, first, h);
        row_of<R>(a, p.u, min(a.rows - p.u.rb * R, R) - 1, last, h);
        last = min(last, p.cnt - 1);
        const int seen = last < first ? 0 : visible_keys(p.len, p.cnt, last, a.causal);
        p.live = max(0, min(p.left, (int)(((int64_t)seen + KT - 1) / KT) - p.t0));
        return p;
    };
    auto wait_all = [&](uint32_t b, uint32_t parity) {
        return __all_sync(0xffffffffu, watch.wait(b, parity));
    };
    if (warp >= kIssueWarp0) {
        // ------------------------------------------------------------ issuer of t's products
        const int t = warp - kIssueWarp0;
        uint32_t n = 0, qn = 0;   // tiles of t and units so far
        uint32_t slot = 0;        // live tiles before the unit
        bool ok = true;
        // half h of S_t of the tile-th live one of the range; `last`: of t's in the unit
        auto issue_s = [&](int h, uint32_t tile, bool last) {
            const uint32_t st = tile % C::kKeyStages;
            if (!wait_all(bar(bars->k_full[st]), (tile / C::kKeyStages) & 1)) return false;
            ptx::tc_fence_after();
            const uint64_t dq = sdesc(sQ, 16, 1024), dk = sdesc(sK + st * C::kTile + h * 64 * 128, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * C::kChunkBytes + (kk & 3) * 32) >> 4;
                ptx::mma_ss_warp(tmem + t * KT + h * 64, dq + off, dk + off, idesc_f16(false, R, 64, false), kk > 0 ? 1u : 0u);
            }
            ptx::mma_commit_warp(bar(bars->s_full[t][h]));
            if (h == 1) {
                ptx::mma_commit_warp(bar(bars->k_empty[st]));
                if (last) ptx::mma_commit_warp(bar(bars->q_empty));
            }
            return true;
        };
        // O_t += P_t V_j for half h; `first` tile: O_t is set, once the last unit's epilogue has
        // read it
        auto issue_pv = [&](int h, uint32_t tile, bool first) {
            const uint32_t st = tile % C::kValueStages;
            if (!wait_all(bar(bars->v_full[st]), (tile / C::kValueStages) & 1) ||
                !wait_all(bar(bars->p_full[t][h]), n & 1) ||
                (first && h == 0 && !wait_all(bar(bars->o_empty), (qn & 1) ^ 1)))
                return false;
            ptx::tc_fence_after();
            const uint64_t dv = sdesc(sV + st * C::kTile + h * 64 * 128, C::kChunkBytes, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                ptx::mma_ts_warp(tmem + 256 + t * D, tmem + t * KT + h * 64 + kk * 8,
                                 dv + (uint64_t)((kk * 16 * 128) >> 4), idesc_f16(false, R, D, true),
                                 (!first || h > 0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit_warp(bar(bars->pv_done[t][h]));
            if (h == 1) ptx::mma_commit_warp(bar(bars->v_empty[st]));
            return true;
        };
        Place here = start;
        for (int i = 0; i < n_tiles && ok;) {
            const Piece p = piece_at(here, i);
            if (p.live > 0) {
                ok = wait_all(bar(bars->q_full), qn & 1);
                if (ok && t >= p.live) ptx::mbar_arrive_warp(bar(bars->q_empty));  // a unit of one tile
                if (ok && t < p.live)
                    ok = issue_s(0, slot + t, t + 2 >= p.live) && issue_s(1, slot + t, t + 2 >= p.live);
                for (int j = t; j < p.live && ok; j += 2) {
                    // S_t of the next tile takes the place of P_t, half by half
                    const bool more = j + 2 < p.live, last = j + 4 >= p.live;
                    ok = issue_pv(0, slot + j, j < 2);
                    if (ok && more) ok = wait_all(bar(bars->pv_done[t][0]), n & 1) && issue_s(0, slot + j + 2, last);
                    ok = ok && issue_pv(1, slot + j, j < 2);
                    if (ok && more) ok = wait_all(bar(bars->pv_done[t][1]), n & 1) && issue_s(1, slot + j + 2, last);
                    ++n;
                }
                ++qn;
            }
            slot += p.live;
            i += p.left;
            if (i < n_tiles) advance(here, p.left, a.units, tiles);
        }
        // every MMA issued by this warp has completed before tensor memory is freed
        ptx::mma_commit_warp(bar(bars->mma_done[t]));
        watch.drain(bar(bars->mma_done[t]), 0);
        __syncwarp();
    } else if (warp >= kConvertWarp0) {
        // ------------------------------------------------------------ converters
        const bool values = warp >= kConvertWarp0 + kConverters;
        const int cw = warp - kConvertWarp0 - (values ? kConverters : 0);
        const int page_shift = 31 - __clz(a.page);
        // A warp's load covers 512 bytes, kRows rows of the tile: load e rows
        // (cw + 3 e) kRows on.  Row and 16-byte piece of a lane: for d = 128 the two halves of a
        // row are not written in the same quarter of the warp, whose lanes would meet in the same
        // banks
        constexpr int kRows = 512 / D, kIters = KT / kRows, N = (kIters + kConverters - 1) / kConverters;
        const int rl = D == 128 ? ((lane >> 2) & 1) + ((lane >> 4) << 1) : lane >> 2;
        const int ql = D == 128 ? (lane & 3) + ((lane >> 3) & 1) * 4 : lane & 3;
        const uint8_t *src = (values ? a.v : a.k) + rl * D + ql * 16;
        const uint32_t line = (values ? sV : sK) + (ql >> 2) * C::kChunkBytes + (cw * kRows + rl) * 128;
        // 16-byte places in the swizzled line: the row's bit 2 changes from load to load at d = 128
        const uint32_t in_line = (uint32_t)((ql & 3) * 2) ^ (uint32_t)((cw * kRows + rl) & 7);
        uint64_t *full = values ? bars->v_full : bars->k_full;
        uint64_t *empty = values ? bars->v_empty : bars->k_empty;
        const uint32_t stages = values ? C::kValueStages : C::kKeyStages;

        // the next tile to load: its piece and place in it
        Place here = start;
        Piece p;
        int i = 0, j = 0, slot = 0;
        int held0 = -4;  // `at` holds the places of the piece's tiles from this one on
        auto settle = [&] {  // to the first piece from here on that has a live tile
            while (i < n_tiles) {
                p = piece_at(here, i);
                if (p.live > 0) return;
                i += p.left;
                if (i < n_tiles) advance(here, p.left, a.units, tiles);
            }
        };
        // lane 8 k + s: 16-key piece s of tile held0 + k as a 16-row piece of the pool, -1: none.
        // Looked up for four tiles at a time, since each look waits for the table
        int at = -1;
        auto find = [&] {
            if (i < n_tiles && j < held0 + 4) return;
            held0 = j;
            at = -1;
            if (i >= n_tiles) return;
            const int tile = j + (lane >> 3), key = (p.t0 + tile) * KT + (lane & 7) * 16;
            if (tile < p.live && key < p.len && in_bounds(p.u.b < a.B && key >> page_shift < a.max_pages, a.status)) {
                const int phys = a.table[(int64_t)p.u.b * a.max_pages + (key >> page_shift)];
                if (phys < 0 || phys >= a.n_pages) atomicOr(a.status, kStatusTable);
                else at = ((phys * a.Hkv + p.u.hk) << (page_shift - 4)) + ((key & (a.page - 1)) >> 4);
                if (!in_bounds(at < ((int64_t)a.n_pages * a.Hkv) << (page_shift - 4), a.status)) at = -1;
            }
        };
        settle();
        find();
        uint4 raw[N];
        float scale = 0.f;   // lanes 0-7: of the tile's keys, 8-15: of its values, 16: `miss`
        uint32_t miss = 0;   // pieces of the tile that are not there
        int key0 = 0, len = 0, ring = 0;
        bool have = false;
        int seg[N];  // of the tile at (p, j): the pieces that this warp loads from
        auto places = [&] {
#pragma unroll
            for (int e = 0; e < N; ++e)
                seg[e] = __shfl_sync(0xffffffffu, at, (j - held0) * 8 + ((cw + kConverters * e) * kRows >> 4 & 7));
        };
        auto load = [&](int e) {
            const int row = (cw + kConverters * e) * kRows;
            if (row < KT && seg[e] >= 0) raw[e] = ldg16(src + (size_t)seg[e] * (16 * D) + (row & 15) * D);
        };
        // what was just loaded becomes the tile to convert; on to the next
        auto take = [&] {
            have = i < n_tiles;
            if (!have) return;
            const int first = (j - held0) * 8;
            miss = __ballot_sync(0xffffffffu, at < 0) >> first & 0xffu;
            if (warp == kConvertWarp0) {
                const int piece = __shfl_sync(0xffffffffu, at, first + (lane & 7));
                scale = lane == 16 ? __uint_as_float(miss) : 0.f;
                if (lane < 16 && piece >= 0) scale = (lane < 8 ? a.ks : a.vs)[piece >> (page_shift - 4)];
            }
            key0 = (p.t0 + j) * KT;
            len = p.len;
            ring = (slot + j) % kScaleRing;
            if (++j == p.live) {
                slot = (slot + p.live) % kScaleRing;
                j = 0;
                held0 = -4;
                i += p.left;
                if (i < n_tiles) advance(here, p.left, a.units, tiles);
                settle();
            }
            find();
        };
        places();
#pragma unroll
        for (int e = 0; e < N; ++e) load(e);
        take();
        uint32_t st = 0, lap = 0;
        while (have) {
            places();
            if (!__all_sync(0xffffffffu, watch.wait(bar(empty[st]), (lap & 1) ^ 1))) break;
            // behind the last token, or without a page, there are no values
            const int held = len - key0;
            const bool part = values && (held < KT || miss != 0);
            const uint32_t off = st * C::kTile;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                uint32_t h[8];
                U::quad(raw[e].x, h[0], h[1]);
                U::quad(raw[e].y, h[2], h[3]);
                U::quad(raw[e].z, h[4], h[5]);
                U::quad(raw[e].w, h[6], h[7]);
                load(e);
                const int row = (cw + kConverters * e) * kRows + rl;
                if (part && (row >= held || (miss >> (row >> 4 & 7) & 1))) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) h[k] = 0;
                }
                if (e < N - 1 || row < KT) {
                    const uint32_t to = line + off + e * (kConverters * kRows * 128);
                    const uint32_t in = in_line ^ (uint32_t)((e * kConverters * kRows) & 7);
                    ptx::st_shared_v4(to + (in << 4), h[0], h[1], h[2], h[3]);
                    ptx::st_shared_v4(to + ((in ^ 1) << 4), h[4], h[5], h[6], h[7]);
                }
            }
            if (warp == kConvertWarp0) {
                if (lane < 17) scales[ring * kScaleWords + lane] = scale;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(bars->sc_full[ring]));
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(bar(full[st]));
            if (++st == stages) {
                st = 0;
                ++lap;
            }
            take();
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        const int t = warp >> 2, wq = warp & 3, r = wq * 32 + lane;
        const uint32_t lanes = (uint32_t)(wq * 32) << 16;
        const uint32_t tS = tmem + lanes + t * KT, tO = tmem + lanes + 256 + t * D;
        uint32_t sn = 0, qn = 0, jn = 0;
        uint32_t slot = 0;  // live tiles before the unit
        bool ok = true;
        Place here = start;
        for (int i = 0; i < n_tiles && ok;) {
            const Piece p = piece_at(here, i);
            int qi, h;
            const bool real = row_of<R>(a, p.u, r, qi, h);
            const bool idle = !__any_sync(0xffffffffu, real);  // no row of this warp is one
            // rows past the block's see every token, so that only the last tile asks for a mask
            const int lim = real ? visible_keys(p.len, p.cnt, qi, a.causal) : p.len;
            const size_t at = real ? (((size_t)p.u.b * a.Hkv * a.G + h) * a.Sq + qi) * D : 0;
            float cq = 0.f;
            if (p.live > 0) {
                // Q: warp w of the eight takes rows 16 w .. 16 w + 15, D / 8 lanes a row, all
                // loaded before the first is used
                constexpr int LR = D / 8, PW = 32 / LR;  // lanes of a row, rows of a load
                float *back = backs + (qn & 1) * R;
                codec::Raw8<1> q[16 / PW];  // 16-bit of either type
                const int sub = lane / LR, piece = lane % LR;
#pragma unroll
                for (int e = 0; e < 16 / PW; ++e) {
                    int ri, rh;
                    q[e].u[0] = make_uint4(0, 0, 0, 0);
                    if (row_of<R>(a, p.u, warp * 16 + e * PW + sub, ri, rh) && q_row(a, p.u, rh, ri))
                        q[e].load(a.q, (((size_t)p.u.b * a.Hkv * a.G + rh) * a.Sq + ri) * D + piece * 8);
                }
                if (!__all_sync(0xffffffffu, watch.wait(bar(bars->q_empty), (qn & 1) ^ 1))) break;
#pragma unroll
                for (int e = 0; e < 16 / PW; ++e) {
                    float f[8];
                    if (a.dtype == ATTN_BF16) {
                        q[e].widen(f);
                    } else {
                        codec::Raw8<2> x;
                        x.u[0] = q[e].u[0];
                        x.widen(f);
                    }
                    float amax = fmaxf(ptx::max3(fabsf(f[0]), fabsf(f[1]), fabsf(f[2])),
                                       ptx::max3(fabsf(f[3]), fabsf(f[4]), ptx::max3(fabsf(f[5]), fabsf(f[6]), fabsf(f[7]))));
#pragma unroll
                    for (int o = 1; o < LR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
                    float mul, inv;
                    row_power(amax, mul, inv);
                    const int row = warp * 16 + e * PW + sub;
                    if (piece == 0) back[row] = inv;
                    ptx::st_shared_v4(sQ + (piece >> 3) * C::kChunkBytes + row * 128 +
                                          ((uint32_t)((piece & 7) ^ (row & 7)) << 4),
                                      pack_f16(f[0] * mul, f[1] * mul), pack_f16(f[2] * mul, f[3] * mul),
                                      pack_f16(f[4] * mul, f[5] * mul), pack_f16(f[6] * mul, f[7] * mul));
                }
                ptx::fence_proxy_async_smem();
                ptx::mbar_arrive(bar(bars->q_full));
                if (!__all_sync(0xffffffffu, watch.wait(bar(bars->q_full), qn & 1))) break;
                ++qn;
                cq = a.sl2 * back[r];
            }
            float top = kUnset, rv = 0x1p123f, l = 0.f;
            for (int j = t; j < p.live; j += 2) {
                const uint32_t ring = (slot + j) % kScaleRing, lap = (slot + j) / kScaleRing;
                ok = wait_all(bar(bars->sc_full[ring]), lap & 1);
                const float *ks = scales + ring * kScaleWords, *vs = ks + 8;
                const int key0 = (p.t0 + j) * KT;
                uint32_t miss = 0;
                bool edge = false;  // a row of this warp does not see every key
                if (ok && !idle) {
                    miss = __float_as_uint(ks[16]);
                    edge = __any_sync(0xffffffffu, miss != 0 || key0 + KT > lim);
                }
#pragma unroll 1
                for (int half = 0; half < 2 && ok; ++half) {
                    ok = wait_all(bar(bars->s_full[t][half]), sn & 1);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (!idle) {
                        const uint32_t tH = tS + half * 64;
                        uint32_t s0[32], s1[32];
                        ptx::tmem_ld32(tH, s0);
                        ptx::tmem_ld32(tH + 32, s1);
                        // four pieces of 16 keys, each of one page: the first key that the row does
                        // not see, and the values' scale.  A page no key of which the row sees adds
                        // nothing, not even its scale's NaN
                        int n[4];
                        float f[4], sv[4];
                        const float4 k4 = *reinterpret_cast<const float4 *>(ks + half * 4);
                        const float4 v4 = *reinterpret_cast<const float4 *>(vs + half * 4);
                        f[0] = k4.x * cq; f[1] = k4.y * cq; f[2] = k4.z * cq; f[3] = k4.w * cq;
                        sv[0] = v4.x; sv[1] = v4.y; sv[2] = v4.z; sv[3] = v4.w;
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            n[g] = 16;
                            if (edge) {
                                n[g] = (miss >> (half * 4 + g) & 1) ? 0 : lim - (key0 + half * 64 + g * 16);
                                if (n[g] <= 0) sv[g] = 0.f;
                            }
                        }
                        float all[4];  // sums of the weights of each 16
                        auto weights = [&] {  // of s0 and s1, in place
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const float2 f2 = make_float2(f[g], f[g]), t2 = make_float2(-top, -top);
                                float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                                uint32_t *s = (g < 2 ? s0 : s1) + (g & 1) * 16;
#pragma unroll
                                for (int e = 0; e < 16; e += 2) {
                                    float2 z = __ffma2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), f2, t2);
                                    z = make_float2(ptx::ex2_approx(z.x), ptx::ex2_approx(z.y));
                                    part[(e >> 1) & 1] = __fadd2_rn(part[(e >> 1) & 1], z);
                                    s[e] = __float_as_uint(z.x);
                                    s[e + 1] = __float_as_uint(z.y);
                                }
                                part[0] = __fadd2_rn(part[0], part[1]);
                                all[g] = part[0].x + part[0].y;
                            }
                            if (!edge) return;
#pragma unroll
                            for (int g = 0; g < 4; ++g) {  // again without what is not seen
                                uint32_t *s = (g < 2 ? s0 : s1) + (g & 1) * 16;
                                all[g] = 0.f;
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    if (e >= n[g]) s[e] = 0;
                                    all[g] += __uint_as_float(s[e]);
                                }
                            }
                        };
                        ptx::tmem_wait_ld();
                        reg_fence(s0);
                        reg_fence(s1);
                        // New references: the largest visible score, and the largest weight times page
                        // scale unless what O holds is larger by now.  A page whose weights are all 0
                        // by now says nothing of the second, and its share of O is 0 (or its scale's
                        // NaN); below 2^-112 a weight counts as that much, so that c stays finite.
                        // Returned: what O is to be multiplied by
                        auto refer = [&] {
                            float mx = -INFINITY, mg[4];
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const uint32_t *s = (g < 2 ? s0 : s1) + (g & 1) * 16;
                                float m = -INFINITY;
                                if (!edge) {
#pragma unroll
                                    for (int e = 0; e < 16; e += 2)
                                        m = ptx::max3(m, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                                } else {
#pragma unroll
                                    for (int e = 0; e < 16; ++e)
                                        if (e < n[g]) m = fmaxf(m, __uint_as_float(s[e]));
                                }
                                mg[g] = m == -INFINITY ? m : m * f[g];
                                mx = fmaxf(mx, mg[g]);
                            }
                            const float nt = fmaxf(top, mx);
                            const float alpha = ptx::ex2_approx(top - nt);  // 0 from kUnset
                            float held = fminf(alpha * kBase / rv, 3.402823466e38f);
#pragma unroll
                            for (int g = 0; g < 4; ++g) {
                                const float e = ptx::ex2_approx(mg[g] - nt);
                                if (e > 0.f) held = fmaxf(held, sv[g] * fmaxf(e, 0x1p-112f));
                                else if (sv[g] == sv[g]) sv[g] = 0.f;
                            }
                            const float nv = mx == -INFINITY ? rv : kBase / fmaxf(held, 0x1p-118f);
                            const float to = alpha == 0.f ? 0.f : alpha * (nv / rv);
                            l *= alpha;
                            top = nt;
                            rv = nv;
                            return to;
                        };
                        if (j < 2 && half == 0) refer();  // the unit's first references
                        weights();
                        float c[4] = {sv[0] * rv, sv[1] * rv, sv[2] * rv, sv[3] * rv};
                        const float most = fmaxf(fmaxf(all[0], all[1]), fmaxf(all[2], all[3]));
                        constexpr float kHeavy = kLargest * kBase;
                        // not <=: where c has overflowed beside weights of 0 the product is a NaN
                        const bool fits = all[0] * c[0] <= kHeavy && all[1] * c[1] <= kHeavy &&
                                          all[2] * c[2] <= kHeavy && all[3] * c[3] <= kHeavy;
                        if (__any_sync(0xffffffffu, most > kLargest || !fits)) {
                            ptx::tmem_ld32(tH, s0);
                            ptx::tmem_ld32(tH + 32, s1);
                            ptx::tmem_wait_ld();
                            reg_fence(s0);
                            reg_fence(s1);
                            const float to = refer();
#pragma unroll
                            for (int g = 0; g < 4; ++g) c[g] = sv[g] * rv;
                            weights();
                            // O_t holds the tiles before and this one's first half
                            if (j > 1 || half == 1) {
                                ok = half == 1 ? wait_all(bar(bars->pv_done[t][0]), sn & 1)
                                               : wait_all(bar(bars->pv_done[t][1]), (sn - 1) & 1);
                                ptx::tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D / 16; ++c) {
                                    uint32_t o[16];
                                    __syncwarp();
                                    ptx::tmem_ld16(tO + c * 16, o);
                                    ptx::tmem_wait_ld();
                                    reg_fence(o);
#pragma unroll
                                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * to);
                                    ptx::tmem_st16(tO + c * 16, o);
                                }
                            }
                        }
                        l += (all[0] + all[1]) + (all[2] + all[3]);
                        uint32_t pk[32];
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            const uint32_t *s = (g < 2 ? s0 : s1) + (g & 1) * 16;
                            const float2 c2 = make_float2(c[g], c[g]);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float2 x = __fmul2_rn(
                                    make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2);
                                pk[g * 8 + e] = pack_f16(x.x, x.y);
                            }
                        }
                        ptx::tmem_st32(tH, pk);  // over columns already taken
                        ptx::tmem_wait_st();
                    }
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(bar(bars->p_full[t][half]));
                }
                ++sn;
                if (!ok) break;
            }
            if (!ok) break;

            // ---- the unit's end: the two halves' states, each with half of the channels
            const int mine = (p.live - t + 1) / 2;  // tiles of this half
            if (mine > 0) {
                if (!wait_all(bar(bars->pv_done[t][0]), (sn - 1) & 1) ||
                    !wait_all(bar(bars->pv_done[t][1]), (sn - 1) & 1))
                    break;
            }
            float *own = state + ((jn & 1) * 2 + t) * 3 * R;
            own[r] = top;
            own[R + r] = rv;
            own[2 * R + r] = l;
            ptx::tc_fence_before();
            ptx::mbar_arrive(bar(bars->joined));
            const bool got = watch.wait(bar(bars->joined), jn & 1);
            if (!__all_sync(0xffffffffu, got)) break;
            ptx::tc_fence_after();
            const float *other = state + ((jn & 1) * 2 + (t ^ 1)) * 3 * R;
            ++jn;
            const float top2 = other[r], l2 = other[2 * R + r];
            const float base = fmaxf(top, top2);
            const float w1 = ptx::ex2_approx(top - base), w2 = ptx::ex2_approx(top2 - base);
            const float L = l * w1 + l2 * w2;  // 0: no key was visible
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const float lse2 = L == 0.f ? -INFINITY : base + log2f(L);
            // of this half's O and the other's, weight times inverse unit
            const float c1 = w1 * inv, u1 = 1.f / rv, c2 = w2 * inv, u2 = 1.f / other[R + r];
            const bool before = i == 0 && here.t > 0, after = here.t + p.left < here.n;
            const bool whole = !before && !after;
            const int sl = 2 * blockIdx.x + (before ? 0 : 1);
            const bool has2 = p.live - (t ^ 1) > 0;  // the other half had a tile
            if (!idle) {
#pragma unroll 1
                for (int c = t * (D / 2); c < (t + 1) * (D / 2); c += 32) {
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = 0.f;
                    if (mine > 0) {
                        uint32_t o[32];
                        ptx::tmem_ld32(tmem + lanes + 256 + t * D + c, o);
                        ptx::tmem_wait_ld();
                        reg_fence(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * c1 * u1;
                    }
                    if (has2) {
                        uint32_t o[32];
                        ptx::tmem_ld32(tmem + lanes + 256 + (t ^ 1) * D + c, o);
                        ptx::tmem_wait_ld();
                        reg_fence(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] += __uint_as_float(o[e]) * c2 * u2;
                    }
                    if (real && whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            if (in_bounds(at + c + e + 8 <= (size_t)a.B * a.Hkv * a.G * a.Sq * D, a.status))
                                store_o8(a, at + c + e, f + e);
                    } else if (real && in_bounds(sl < 2 * (int)gridDim.x, a.status)) {
                        // [D / 4][R][4]: a warp's store is one piece
                        float4 *d = reinterpret_cast<float4 *>(a.po + (size_t)sl * R * D) + (c / 4) * R + r;
#pragma unroll
                        for (int e = 0; e < 8; ++e) d[e * R] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    }
                    __syncwarp();  // the loads above are the whole warp's
                }
                if (t == 0 && real) {
                    if (!whole) {
                        if (in_bounds(sl < 2 * (int)gridDim.x, a.status)) a.pl[sl * R + r] = lse2;
                    }
                    else if (a.lse && in_bounds(at / D < (size_t)a.B * a.Hkv * a.G * a.Sq, a.status)) a.lse[at / D] = lse2 * kLn2;
                }
            }
            if (p.live > 0) {
                __syncwarp();
                ptx::tc_fence_before();
                ptx::mbar_arrive(bar(bars->o_empty));
            }
            slot += p.live;
            i += p.left;
            if (i < n_tiles) advance(here, p.left, a.units, tiles);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 0) ptx::tmem_dealloc(tmem, kTmemCols);
}

// Joins the states of the units that run over the CTAs' ends: eight rows a CTA,
// thread t four channels of row t % 8, so that a warp reads whole 128-byte lines
// of the states' [D / 4][R][4].
template <int D>
__global__ void __launch_bounds__(8 * D / 4) cache_tc_merge_kernel(const FwdArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d = a.tail[blockIdx.x];
    if (!d.x) return;
    const Unit u = unit_at(a, d.z, d.w);
    const int r = blockIdx.y * 8 + (threadIdx.x & 7), c4 = threadIdx.x >> 3;
    size_t row;
    if (!out_row<R>(a, u, r, row)) return;
    const int n = d.y - (int)blockIdx.x + 1;
    if (!in_bounds(n >= 1 && n <= kCacheMaxCtas && blockIdx.x + n <= gridDim.x, a.status)) return;
    auto slot = [&](int p) { return 2 * (size_t)(blockIdx.x + p) + (p == 0 ? 1 : 0); };
    float M = -INFINITY;
    for (int p = 0; p < n; ++p) M = fmaxf(M, a.pl[slot(p) * R + r]);
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, acc[4] = {};
#pragma unroll 4
    for (int p = 0; p < n; ++p) {
        const float wt = ptx::ex2_approx(a.pl[slot(p) * R + r] - base), w = wt * kFits;
        const float4 x = reinterpret_cast<const float4 *>(a.po + slot(p) * R * D)[c4 * R + r];
        L += wt;
        acc[0] = fmaf(w, x.x, acc[0]);
        acc[1] = fmaf(w, x.y, acc[1]);
        acc[2] = fmaf(w, x.z, acc[2]);
        acc[3] = fmaf(w, x.w, acc[3]);
    }
    const float inv = L == 0.f ? 0.f : 1.f / (kFits * L);
#pragma unroll
    for (int e = 0; e < 4; ++e) store_o(a, row * D + c4 * 4 + e, acc[e] * inv);
    if (a.lse && c4 == 0) a.lse[row] = L == 0.f ? -INFINITY : (base + log2f(L)) * kLn2;
}

template <int D, int FMT>
int launch_t(const FwdArgs &f, unsigned grid, cudaStream_t stream) {
    using C = Cfg<D>;
    auto kern = cache_tc_kernel<D, FMT>;
    if (!set_smem_limit_once(reinterpret_cast<const void *>(kern), C::kSmem)) return ATTN_ERR_LAUNCH;
    TcArgs args;
    args.f = f;
    args.timeout_ns = watchdog_ns();
    // the whole of shared memory for any batch, so that one CTA runs on an SM: tensor
    // memory has no room for two
    kern<<<grid, kThreads, C::kSmem, stream>>>(args);
    if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_LAUNCH;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, (unsigned)((f.rows < R ? f.rows : R) + 7) / 8);
    cfg.blockDim = dim3(8 * D / 4);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, cache_tc_merge_kernel<D>, f);
    return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // namespace

// a: every field but the workspace's and the row blocks'.
int launch_cache_tc(FwdArgs &a, int d, int format, void *workspace, cudaStream_t stream) {
    a.nrb = (a.rows + R - 1) / R;
    a.units = a.Hkv * a.nrb;
    a.by_units = fast_div((uint32_t)a.units);
    a.by_per = fast_div((uint32_t)a.nrb);
    a.by_nrb = a.by_per;
    const int sms = device_sm_count();
    const double most = (double)a.B * a.units * (((double)a.max_pages * a.page + KT - 1) / KT);
    int ctas = sms < kCacheMaxCtas ? sms : kCacheMaxCtas;
    if (most < ctas) ctas = (int)most;
    a.workers = ctas;
    a.tail = reinterpret_cast<int4 *>(workspace);
    a.po = reinterpret_cast<float *>(a.tail + ctas);
    a.pl = a.po + (size_t)2 * ctas * R * d;
    if (d == 64)
        return format == ATTN_CACHE_E4M3 ? launch_t<64, ATTN_CACHE_E4M3>(a, (unsigned)ctas, stream)
                                         : launch_t<64, ATTN_CACHE_I8>(a, (unsigned)ctas, stream);
    return format == ATTN_CACHE_E4M3 ? launch_t<128, ATTN_CACHE_E4M3>(a, (unsigned)ctas, stream)
                                     : launch_t<128, ATTN_CACHE_I8>(a, (unsigned)ctas, stream);
}

}  // namespace attn
