// cache_index.h -- index arithmetic of the paged 8-bit cache that the host,
// the kernels and the CPU tests share: which worker takes which key tiles,
// where a worker's partial results go, and which rows of a page a call
// touches.  Plain C++ (compiles without CUDA).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define ATTN_HD __host__ __device__ __forceinline__
#else
#define ATTN_HD inline
#endif

namespace attn {

// The total key tiles of a call, numbered 0 .. total - 1 in the order of the
// units they belong to, are cut into `workers` contiguous ranges: total / workers
// tiles each, the first total % workers of them one more.  worker_begin(w) is the
// first tile of worker w; worker_begin(workers) == total.
ATTN_HD int64_t quotient(int64_t a, int64_t b) {  // 64-bit division is long on the device
    return ((uint64_t)(a | b) >> 31) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
ATTN_HD int64_t worker_begin(int64_t w, int64_t total, int64_t workers) {
    const int64_t q = quotient(total, workers), r = total - q * workers;
    return w * q + (w < r ? w : r);
}
// The worker whose range holds tile x (0 <= x < total; total >= workers).
ATTN_HD int64_t worker_of(int64_t x, int64_t total, int64_t workers) {
    const int64_t q = quotient(total, workers), r = total - q * workers, longer = r * (q + 1);
    return x < longer ? quotient(x, q + 1) : r + quotient(x - longer, q);
}
// Workers that share `total` tiles: at least min_tiles each, at most `most`.
ATTN_HD int64_t worker_count(int64_t total, int64_t most, int64_t min_tiles) {
    const int64_t n = (total + min_tiles - 1) / min_tiles;
    return n < 1 ? 1 : (n < most ? n : most);
}
// Tokens a sequence's table row can address, and its length clamped to them.
ATTN_HD int64_t cache_capacity(int max_pages, int page) { return (int64_t)max_pages * page; }
ATTN_HD int clamp_len(int len, int max_pages, int page) {
    const int64_t cap = cache_capacity(max_pages, page);
    return len < 0 ? 0 : ((int64_t)len > cap ? (int)cap : len);
}
// Keys visible to query row i of a sequence that holds `len` tokens, the last
// `cnt` of which are the queries' own (causal), or all of them.
ATTN_HD int visible_keys(int len, int cnt, int i, int causal) {
    if (i >= cnt) return 0;
    if (!causal) return len;
    const int64_t n = (int64_t)len - cnt + i + 1;
    return n < 0 ? 0 : (n > len ? len : (int)n);
}
// Division of numbers below 2^31 by a number that the host knows: n / d =
// (high half of n * m, plus n) >> s with m = 2^32 (2^s - d) / d + 1, s the
// smallest power with 2^s >= d.
struct FastDiv {
    uint32_t d, m, s;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f = {d, 0, 0};
    while (((uint64_t)1 << f.s) < d) ++f.s;
    f.m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.s) - d)) / d + 1);
    return f;
}
ATTN_HD uint32_t operator/(uint32_t n, const FastDiv &f) {
#ifdef __CUDA_ARCH__
    return (__umulhi(n, f.m) + n) >> f.s;
#else
    return (uint32_t)((((uint64_t)n * f.m >> 32) + n) >> f.s);
#endif
}

// A tile's place: tile t of the n tiles of unit `unit` of sequence b.  Units of
// a sequence are numbered kv head, query (with a page list), row block.
struct Place {
    int b, unit, t, n;
};
// `by` tiles further.  tiles(b): tiles of a unit of sequence b; sequences
// without any are passed over.  The caller knows that the tile exists.
template <typename F>
ATTN_HD void advance(Place &p, int by, int units, F tiles) {
    p.t += by;
    while (p.t >= p.n) {
        p.t -= p.n;
        if (++p.unit == units) {
            p.unit = 0;
            do ++p.b; while ((p.n = tiles(p.b)) == 0);
        }
    }
}

// Largest number of pages that S consecutive tokens can touch.
ATTN_HD int64_t touched_pages(int64_t S, int page) { return S <= 0 ? 0 : (S + page - 2) / page + 1; }

}  // namespace attn
