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
ATTN_HD int64_t worker_begin(int64_t w, int64_t total, int64_t workers) {
    const int64_t q = total / workers, r = total - q * workers;
    return w * q + (w < r ? w : r);
}
// The worker whose range holds tile x (0 <= x < total; total >= workers).
ATTN_HD int64_t worker_of(int64_t x, int64_t total, int64_t workers) {
    const int64_t q = total / workers, r = total - q * workers, longer = r * (q + 1);
    return x < longer ? x / (q + 1) : r + (x - longer) / q;
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
// Largest number of pages that S consecutive tokens can touch.
ATTN_HD int64_t touched_pages(int64_t S, int page) { return S <= 0 ? 0 : (S + page - 2) / page + 1; }

}  // namespace attn
