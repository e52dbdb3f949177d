/*
 * attn.h -- C ABI of libattn.so: exact attention forward with online softmax
 * on NVIDIA GB300 (sm_103a).
 *
 * The operation (all three source pages compute it; they differ only in how
 * they tile it):
 *
 *   O[b,h,i,:] = sum_j softmax_j( scale * Q[b,h,i,:] . K[b,h,j,:] ) * V[b,h,j,:]
 *
 * over the keys j visible to query i, computed tile by tile: each query row
 * keeps a running maximum m, a normaliser l and an unnormalised accumulator a,
 * and both l and a are multiplied by exp(m_old - m_new) whenever a new key
 * tile raises the maximum, so that the full score matrix is never formed.
 *   - definition and dense reference: aiml.sh "verify-tiled-attention",
 *     function standard_attention (scale 1/sqrt(d), causal limit i+1);
 *     deepnotes "flash-attention-implemented-verified-and-measured",
 *     naive_attention on [B, H, S, d] tensors;
 *   - the tiled recurrence: aiml.sh "verify-tiled-attention",
 *     tiled_flash_attention; deepnotes ..., tiled_attention_online_softmax;
 *     huhohoo "tiled-online-softmax", section "Online normalization".
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout   q [B, H, Sq, d], k and v [B, H, Skv, d], o [B, H, Sq, d],
 *          lse [B, H, Sq]; all contiguous row-major, strides implied.
 *          q, k, v and o must be 16-byte aligned; lse 4-byte aligned.
 * causal   0 or 1.  Key j is visible to query i iff j <= i + (Skv - Sq)
 *          (bottom-right alignment; identical to the pages' j <= i when
 *          Sq == Skv).  A query row with no visible key gets o = 0 and
 *          lse = -inf.
 * scale    multiplies q . k.  scale <= 0 selects the pages' 1/sqrt(d); NaN or
 *          infinity is rejected.
 * lse      optional (NULL: not written).  Natural-log log-sum-exp of the
 *          scaled scores of each row, fp32.  Not on the pages; provided so a
 *          caller can merge partial results or compute a backward pass.
 * stream   a cudaStream_t (NULL = legacy default stream).  All work is
 *          enqueued on it asynchronously; no entry point synchronises except
 *          attn_check_status.  Device pointers must be valid on the current
 *          CUDA device.
 * Ownership  the caller owns every buffer.  The library keeps no per-call
 *          allocation; q, k and v are only read; o and lse must not overlap
 *          q, k or v (rejected) or each other.
 * Empty    B, H or Sq equal to 0 is a no-op returning ATTN_OK; Skv == 0 writes
 *          o = 0 and lse = -inf.
 * Errors   every entry point returns an attn_status; nothing aborts, exits or
 *          traps.  Invalid arguments are detected on the host before any
 *          launch.  attn_strerror() gives a message.
 */
#ifndef ATTN_GB300_ATTN_H
#define ATTN_GB300_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_ABI_VERSION 1

/* The library is built with hidden visibility; only the functions declared
 * with ATTN_API (this header's) are exported.  The test-only entry points
 * (attn_test.h) are exported by libattn_test.so alone. */
#if defined(__GNUC__) || defined(__clang__)
#define ATTN_API __attribute__((visibility("default")))
#else
#define ATTN_API
#endif

typedef enum attn_status {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1,        /* null/misaligned/overlapping pointer, bad size or dtype */
    ATTN_ERR_UNSUPPORTED_DEVICE = 2, /* current device is not compute capability 10.3 */
    ATTN_ERR_LAUNCH = 3,             /* a CUDA launch or copy failed */
    ATTN_ERR_TIMEOUT = 4,            /* a kernel's bounded wait expired (see attn_check_status) */
    ATTN_ERR_CUDA = 5,               /* another CUDA runtime/driver error */
    ATTN_ERR_SCRATCH_LIMIT = 6,      /* attn_fwd_splitkv_noalloc: problem exceeds its fixed scratch */
    ATTN_ERR_BOUNDS = 7,             /* bounds-checking build only: an index check failed and the
                                        access was skipped (see attn_check_status) */
    ATTN_ERR_TABLE = 8               /* a kernel read a block table or page list entry, a length or
                                        a count out of range; what it stands for was skipped (see
                                        attn_check_status) */
} attn_status;

typedef enum attn_dtype {
    ATTN_F32 = 0,          /* fp32 q/k/v/o; CUDA-core kernel, fp32 arithmetic */
    ATTN_BF16 = 1,         /* bf16 q/k/v/o; tensor-core kernel, fp32 accumulation */
    ATTN_F16 = 2,          /* fp16 q/k/v/o; tensor-core kernel, fp32 accumulation */
    ATTN_BF16_OUT_F32 = 3, /* bf16 q/k/v, fp32 o (no output rounding) */
    ATTN_F16_OUT_F32 = 4   /* fp16 q/k/v, fp32 o */
} attn_dtype;

/*
 * attn_fwd -- exact attention forward (the operation above).
 *
 * Supported head widths: ATTN_F32: d in {16, 32, 64, 128};
 * ATTN_BF16/F16 and their _OUT_F32 variants: d in {64, 128}.
 * ATTN_F32 runs the CUDA-core kernel with 32-row query blocks and 64-key
 * blocks (the key block of deepnotes "Correctness first"); the 16-bit types
 * run the tensor-core kernel with 128 x 128 tiles.
 * Requires a compute capability 10.3 device (GB300) for every dtype.
 *
 * CUDA graphs: the first call that uses a kernel variant on a device sets
 * up its per-device state (the kernel's shared-memory attribute, for the fp32
 * kernel its occupancy, the address of the status word); the variant follows
 * from dtype, d and the problem shape.  After that a call of the same shape
 * only enqueues one kernel on `stream` (two for attn_fwd_splitkv) and may be
 * captured into a CUDA graph; a replay reads whatever the captured pointers
 * hold at replay time.  Make one ordinary call of the shape before capturing.
 *
 * Work distribution (16-bit types): each launch of the tensor-core kernel
 * takes its work units from one of 256 device counters of the library,
 * chosen in turn, and returns that counter to zero when it ends.  At most
 * 256 such launches may therefore be in flight on one device at once, and a
 * CUDA graph containing the call must not be replayed concurrently with
 * itself (its replays share the counter captured with it).
 */
ATTN_API int attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
             int B, int H, int Sq, int Skv, int d, int causal, float scale,
             int dtype, void *stream);

/*
 * attn_fwd_gqa -- attn_fwd with kv heads that several query heads share: k and
 * v [B, H_kv, Skv, d], H_kv >= 1 and H >= 1 a multiple of it; query heads
 * h * H / H_kv .. (h + 1) * H / H_kv - 1 read kv head h.  The result is that
 * of attn_fwd on k and v with each head repeated, without the copies.
 * Everything else as attn_fwd (which is the case H_kv = H).
 */
ATTN_API int attn_fwd_gqa(const void *q, const void *k, const void *v, void *o, float *lse,
                 int B, int H, int H_kv, int Sq, int Skv, int d, int causal, float scale,
                 int dtype, void *stream);

/*
 * Backward pass
 * -------------
 * attn_bwd -- the gradients of a loss in q, k and v, given its gradients do in o
 * and (optionally) dlse in lse.  With the forward pass's o and lse,
 *   P  = exp(scale q k^T - lse) on the visible keys (0 elsewhere),
 *   dS = P * (do v^T - rowsum(o * do) + dlse),
 *   dq = scale dS k,   dk = scale dS^T q,   dv = P^T do,
 * dk and dv summed over the query heads that share a kv head.  The
 * probabilities are recomputed tile by tile (not on the source pages, which
 * stop at the forward pass; the tiles are theirs: aiml.sh
 * "verify-tiled-attention", tiled_flash_attention).
 *
 *   q, do  [B, H, Sq, d], k, v [B, H_kv, Skv, d] in dtype's input type;
 *   o      [B, H, Sq, d] in dtype's output type, lse [B, H, Sq] fp32: what
 *          attn_fwd (or _gqa, _splitkv) wrote for the same q, k, v, causal,
 *          scale and dtype.  Over a shard of the keys (causal = 0) they may be
 *          the merged o and lse of all shards: dk and dv are then the shard's,
 *          and the dq of the shards add up to the whole.
 *   dlse   [B, H, Sq] fp32 or NULL (zero)
 *   dq, dk, dv  as q, k, v, but in dtype's output type; all are written whole
 *   H >= 1 a multiple of H_kv >= 1; d, dtype, causal, scale as attn_fwd
 *   workspace  16-byte aligned scratch of attn_bwd_workspace_size bytes (NULL if
 *          that is 0).  Calls that may overlap on the GPU, replays of graphs
 *          among them, need workspaces of their own.
 * A row with lse = -inf (no visible key) contributes nothing and gets dq = 0,
 * whatever its o, do and dlse hold, as long as they are finite.  Skv == 0
 * writes dq = 0; Sq == 0 writes dk = dv = 0.  Infinities and NaN in a row of
 * q, k, v or do may reach every gradient of its 128-row tile, masked or not.
 * Arithmetic: fp32 sums.  16-bit types: P and dS are rounded to 16 bits as
 * operands of the products (dS of queries that see up to 128 keys, and P if
 * Skv <= 128, to twice as many bits).  fp16: after scaling by powers of two, P by
 * one for all, dS by one for each row of dq and one for each 128 rows of dk, from
 * the norms of what makes it, so that heads and sequences of very different do
 * share a call without loss; terms P (|do| |v| + |D|) of one sum that are less than
 * 2^-27 of the largest |do| |v| + |D| among the 128-row tiles it goes over lose bits.
 * fp32: each product of two numbers is wrong by 2^-21 of itself at most; numbers from
 * 2^128 - 2^116 on count as infinite, and what numbers below 2^-112 hold beyond their
 * first 11 bits may be lost.  Sums are made in a fixed order: equal calls give equal bits.
 * All arrays must be distinct; q, k, v, o, do and gradients 16-byte aligned.
 * Sq and Skv <= 2^31 - 1024.  CUDA graphs: as attn_fwd, without its limit on
 * launches in flight.
 * Two kernels (fp32: one), one more where few units share a long walk.
 */
ATTN_API int attn_bwd_workspace_size(int B, int H, int H_kv, int Sq, int Skv, int d, int causal,
                            int dtype, size_t *bytes);
ATTN_API int attn_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
             const void *do_, const float *dlse, void *dq, void *dk, void *dv, int B, int H,
             int H_kv, int Sq, int Skv, int d, int causal, float scale, int dtype,
             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Rotary positions
 * ----------------
 * attn_rotary -- turns pair i of the first `width` channels of each row by the
 * angle p * theta_i of its token's position p (before attn_fwd or
 * attn_cache_append; not on the source pages):
 *   (x, y) -> amplitude * (x cos a - y sin a, x sin a + y cos a);
 * transpose = 1 multiplies with the transposed matrices instead (angle -a,
 * the same amplitude): the gradient in the inputs, given the one in the outputs.
 * Channels from `width` on are copied.
 *
 *   q, k   rows of one or two tensors (k may be NULL) of dtype ATTN_F32,
 *          ATTN_BF16 or ATTN_F16: logically [B][H][S][d] with the strides (in
 *          elements, >= 0) of batch, head and token; channels are contiguous.
 *          `out` may be `in` with the same strides; otherwise no output may
 *          overlap an input (the positions and the angles too), the other output
 *          or itself: refused, but that strides with no order in common are tested
 *          for a few thousand combinations only.
 *   interleaved  0: pairs (i, i + width / 2); 1: pairs (2i, 2i + 1)
 *   turns  [width / 2] theta_i / (2 pi) as a 64-bit fraction of a turn per
 *          position (rounded theta_i / (2 pi) * 2^64, modulo 2^64)
 *   pos    int32: [B][S] if pos_per_token, else [B], the position of each
 *          sequence's first row, the others following; any values (they wrap
 *          at 32 bits)
 *   width  even, 2 .. d;  d even, <= 1024;  H <= 65536;  B * S < 2^31
 * fp32 arithmetic on the rows; the angle's error does not grow with the
 * position beyond 2^-64 turns of each.  One kernel.
 */
typedef struct attn_heads {
    const void *in;
    void *out;
    int H;
    int64_t in_stride[3], out_stride[3];
} attn_heads;

ATTN_API int attn_rotary(const attn_heads *q, const attn_heads *k, const uint64_t *turns, int width,
                int interleaved, float amplitude, int transpose, const int32_t *pos,
                int pos_per_token, int B, int S, int d, int dtype, void *stream);

/*
 * attn_validate -- the host-side argument check of attn_fwd, without any CUDA
 * call or launch.  Returns ATTN_OK or ATTN_ERR_INVALID_ARG.  Pointers are only
 * compared and tested for alignment, never dereferenced.
 */
ATTN_API int attn_validate(const void *q, const void *k, const void *v, const void *o,
                  const float *lse, int B, int H, int Sq, int Skv, int d,
                  int causal, float scale, int dtype);

/*
 * attn_fwd_staged -- attn_fwd on HOST buffers: copies q, k, v from host memory
 * to the caller's device buffers dq, dk, dv, runs attn_fwd into do_ / dlse,
 * and copies o (and lse when both lse_host and dlse are non-NULL) back to
 * host memory (one cudaMemcpyAsync per tensor, or per tensor and chunk).
 * Host buffers should be pinned for the copies to be asynchronous.  The call
 * returns after enqueueing; synchronise the stream before reading o_host.
 * Problems with at least 4 MiB of input are cut into up to 4 chunks of
 * (batch, head) slices, with shares 2 : 3 : 3.5 : 1.5 (small first and last
 * chunks, so the kernels start early and little is left after the last
 * copy in), that run on two streams the library creates once per device:
 * the copies of one chunk overlap the kernel of the other.  Those streams
 * start after the work queued on `stream` and `stream` waits for them, so the
 * call behaves as if everything ran on `stream`; concurrent staged calls on
 * one device share the two streams.  attn_shutdown releases them; call it
 * before a cudaDeviceReset that the process survives.
 * Sizes and dtype as attn_fwd; host pointers must not be NULL when their
 * tensor is non-empty.
 */
ATTN_API int attn_fwd_staged(const void *q_host, const void *k_host, const void *v_host,
                    void *o_host, float *lse_host, void *dq, void *dk, void *dv,
                    void *do_, float *dlse, int B, int H, int Sq, int Skv,
                    int d, int causal, float scale, int dtype, void *stream);

/*
 * Split-KV forward for a few query rows per head (decode)
 * --------------------------------------------------------
 * The keys of every (batch, head) are cut into n_splits contiguous ranges of
 * equal length (a multiple of 32 keys); each range is processed by its own
 * CTAs on CUDA cores (fp32 arithmetic for every input type), which write a
 * partial result -- the softmax-weighted average of the range's values and
 * the log-sum-exp of its scaled scores -- into `workspace`; attn_merge's
 * kernel then combines the partial results of every row.  The result is the
 * same operation as attn_fwd: only the order of the sums differs (the pages'
 * point that the tiling, here the split, changes nothing but rounding:
 * aiml.sh "verify-tiled-attention", tile-size sweep; huhohoo
 * "tiled-online-softmax", block size seven).
 */

/*
 * attn_splitkv_workspace_size -- bytes of the workspace attn_fwd_splitkv
 * needs: 4 * n_splits * B * H * Sq * (d + 1) (partial outputs
 * [n_splits][B*H][Sq][d] followed by partial lse [n_splits][B*H][Sq], fp32).
 * Host only.  d in {16, 32, 64, 128}; 1 <= n_splits <= 256.
 */
ATTN_API int attn_splitkv_workspace_size(int B, int H, int Sq, int d, int n_splits, size_t *bytes);

/*
 * attn_splitkv_plan -- the split count the library would pick on the current
 * device and, if workspace_bytes is not NULL, the workspace size for it.
 * The count minimises an estimate of the time: waves of CTAs over the
 * device's resident CTA slots times the 32-key tiles each warp walks plus a
 * fixed cost per CTA (about two tiles), with at least two tiles per warp in
 * each split.  Needs a compute capability 10.3 device.
 */
ATTN_API int attn_splitkv_plan(int B, int H, int Sq, int Skv, int d, int dtype, int *n_splits,
                      size_t *workspace_bytes);

/*
 * attn_fwd_splitkv -- attn_fwd computed by key splits.
 *
 * Arguments and layouts as attn_fwd, except:
 *   d          in {16, 32, 64, 128} for every dtype;
 *   Sq         <= 524280;
 *   n_splits   1 .. 256 (see attn_splitkv_plan); empty trailing splits are
 *              skipped;
 *   workspace  device memory of at least attn_splitkv_workspace_size bytes,
 *              16-byte aligned, owned by the caller and not overlapping any
 *              other argument; its contents are scratch (overwritten).
 *              May be NULL when Skv == 0.
 * Enqueues two kernels on `stream` (partial results, merge).  Returns
 * ATTN_ERR_INVALID_ARG for a missing, small, misaligned or overlapping
 * workspace; otherwise as attn_fwd.
 */
ATTN_API int attn_fwd_splitkv(const void *q, const void *k, const void *v, void *o, float *lse,
                     int B, int H, int Sq, int Skv, int d, int causal, float scale,
                     int dtype, int n_splits, void *workspace, size_t workspace_bytes,
                     void *stream);

/*
 * attn_fwd_splitkv_noalloc -- attn_fwd_splitkv for callers that must not
 * allocate memory.  No passage of the source pages corresponds to it: it is
 * an interface for code that cannot call cudaMalloc, for example code
 * running inside a custom allocator or a memory-pool callback, a runtime
 * that forbids allocation on its serving path, or a caller whose memory
 * budget is fixed in advance.
 *
 * Instead of a caller-provided workspace it uses a scratch array of
 * ATTN_NOALLOC_SCRATCH_BYTES (8 MiB) that is part of the library's device
 * image: every GPU on which the library is used holds it until the process
 * exits.  The call calls no allocating routine (no cudaMalloc, no library
 * allocator).
 *   - Size limit: the problem must fit, i.e.
 *     4 * n_splits * B * H * Sq * (d + 1) <= ATTN_NOALLOC_SCRATCH_BYTES
 *     (see attn_splitkv_workspace_size) whenever Skv > 0; otherwise
 *     ATTN_ERR_SCRATCH_LIMIT is returned before anything is launched.
 *   - Set-up on a device: the first call of ANY entry point on a device
 *     (with that device current) looks up the array's device address, which
 *     makes CUDA load the module holding it and reserve the 8 MiB there.  The
 *     first launch of each kernel variant may also make the driver load that
 *     kernel's code.  Both happen once per device; so, before entering code
 *     that must not allocate, make one call of this entry point on the
 *     device with the same dtype and head width (and before capturing a
 *     stream).  Later calls change nothing in the device's free memory.
 *   - Sharing: every call uses the same array, which keeps the contents of
 *     the last call.  Nothing in it needs to start at zero (each partial
 *     result is written before it is read), but calls that overlap on the GPU
 *     (different streams, or different host threads without ordering) race
 *     on it: order them, e.g. on one stream.
 * Other arguments, results and errors as attn_fwd_splitkv.
 */
#define ATTN_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)
ATTN_API int attn_fwd_splitkv_noalloc(const void *q, const void *k, const void *v, void *o, float *lse,
                             int B, int H, int Sq, int Skv, int d, int causal, float scale,
                             int dtype, int n_splits, void *stream);

/*
 * attn_merge -- combines partial attention results of the same query rows
 * over disjoint key sets (key splits, or key shards held by different
 * devices) into the result over the union of the keys.  Each partial result
 * is the state (m, l, a) of the online softmax in the form o_part = a / l,
 * lse_part = m + ln l; the merge is the update of huhohoo
 * "tiled-online-softmax" ("Online normalization") applied to whole states:
 *   M = max_p lse_p,  w_p = exp(lse_p - M),
 *   o = sum_p w_p o_p / sum_p w_p,  lse = M + ln(sum_p w_p).
 * A part with lse = -inf (no visible key) contributes nothing; a row whose
 * parts are all -inf gets o = 0 and lse = -inf.
 *
 *   n_parts    1 .. 4096;  rows 0 .. 2^31 - 1;  d >= 1
 *   o_parts    [n_parts][rows][d] fp32, device memory
 *   lse_parts  [n_parts][rows]    fp32, natural log
 *   o          [rows][d] of out_dtype: ATTN_F32, ATTN_BF16 or ATTN_F16
 *   lse        [rows] fp32, or NULL
 * fp32 arithmetic; asynchronous on `stream`.  Outputs must not overlap the
 * inputs or each other (ATTN_ERR_INVALID_ARG).
 */
ATTN_API int attn_merge(const float *o_parts, const float *lse_parts, int n_parts, int64_t rows, int d,
               void *o, float *lse, int out_dtype, void *stream);

/*
 * Paged 8-bit key/value cache
 * ---------------------------
 * The cache a decode step reads: a pool of pages that the caller owns.  A page
 * holds `page` consecutive tokens of one sequence, for every kv head, as 8-bit
 * codes; each (page, kv head) block of keys and of values has one scale, and
 * the value a code stands for is code * scale.  Not on the source pages; the
 * attention over it is the operation above on those values, computed tile by
 * tile (deepnotes "flash-attention-implemented-verified-and-measured",
 * tiled_attention_online_softmax), with a partial state per key range joined
 * as attn_merge does.
 *
 * Layout (all contiguous, device memory; codes and bounds 16-byte aligned):
 *   k, v            [n_pages][H_kv][page][d], 1 byte each
 *   k_scale, v_scale [n_pages][H_kv] fp32
 *   k_bounds        [n_pages][H_kv][2][d], 1 byte each: the smallest and the
 *                   largest key code of each channel.  May be NULL: then
 *                   attn_cache_append keeps none and attn_cache_select refuses.
 *   page in {16, 32, 64, 128}; d in {64, 128}; format one of attn_cache_format;
 *   n_pages * H_kv * page / 16 < 2^31; max_pages * page <= 2^31 - 1025.
 * Nothing in the pool needs to be initialised.
 *
 * Sequences  table [B][max_pages] int32 names the pages of each sequence in
 *   order: token j is row j % page of page table[b][j / page].  lens [B] (pos
 *   for append) is the number of tokens held; counts [B] (NULL: all rows) the
 *   rows of this call that are the sequence's, the first ones of its S (Sq)
 *   rows.  These arrays are device memory and only read, so a captured call
 *   follows them.  Entries of a row behind its last page are not read.
 *   A kernel that reads a needed page number outside 0 .. n_pages - 1, a
 *   length outside 0 .. max_pages * page or a count outside 0 .. S skips what
 *   it stands for (the length is clamped, the keys of a bad page count as
 *   absent, append writes nothing of a sequence with a bad count) and
 *   attn_check_status reports ATTN_ERR_TABLE.
 *
 * Scales  the smallest power of two s >= 2^-126 with amax <= top * s, amax the
 *   block's largest magnitude and top = 448 (e4m3) or 127 (int8); 0 for
 *   amax = 0.  Division by it is exact, so codes are x / s rounded once, to
 *   nearest, ties to even.  A NaN or an infinity makes the scale of its block
 *   NaN: everything read from that block and head is NaN until the page is
 *   started again at its first row.  attn_cache_read takes any scale, the
 *   others any finite scale >= 0 or NaN; pages that append continues must hold
 *   such powers of two.
 */
typedef enum attn_cache_format {
    ATTN_CACHE_E4M3 = 0, /* 4-bit exponent, 3-bit mantissa, no infinities; largest 448 */
    ATTN_CACHE_I8 = 1    /* -127 .. 127 */
} attn_cache_format;

typedef struct attn_cache {
    void *k, *v;
    float *k_scale, *v_scale;
    void *k_bounds;
    int n_pages, H_kv, page, d, format;
} attn_cache;

/*
 * attn_cache_append -- quantises counts[b] new tokens of each sequence behind
 * the pos[b] it holds.
 *
 *   k, v   [B][H_kv][S][d] of dtype ATTN_F32, ATTN_BF16 or ATTN_F16
 * A block that already holds rows of the sequence keeps them: its scale
 * becomes the larger of its own and the new rows', and when that grows the
 * older codes are rounded again under it.  pos[b] may lie before tokens
 * written earlier (they are overwritten; scale and bounds of a page that is
 * continued keep covering them).  Rows of a page behind the last new token are
 * left as they were.  A sequence with a count of 0 touches no page, and its
 * table row is not read.  No page may be written for two sequences, or for one
 * twice, in one call (its contents are then undefined).  The cache's arrays
 * must not overlap.  One kernel.
 */
ATTN_API int attn_cache_append(const attn_cache *cache, const void *k, const void *v,
                      const int32_t *table, int max_pages, const int32_t *pos,
                      const int32_t *counts, int B, int S, int dtype, void *stream);

/*
 * attn_cache_read -- the first S tokens of each sequence as k, v
 * [B][H_kv][S][d] of dtype ATTN_F32, ATTN_BF16 or ATTN_F16, for example for
 * attn_fwd.  Rows from lens[b] on are zero.  Values beyond the type's range
 * become its largest finite number.  One kernel.
 */
ATTN_API int attn_cache_read(const attn_cache *cache, const int32_t *table, int max_pages,
                    const int32_t *lens, void *k, void *v, int B, int S, int dtype, void *stream);

/*
 * attn_cache_select -- the pages each query attends to: for query row i and
 * kv head h, the page that holds the row's last visible key and the
 * n_select - 1 others with the highest
 *   score(p) = k_scale[p] * max over the query heads g of h of
 *              sum_c max(q_gc * lo_pc, q_gc * hi_pc)
 * (lo and hi from k_bounds), an upper bound of q . k over the page; equal
 * scores go to the lower page, a NaN scores highest.
 *
 *   q      [B][H][Sq][d] of an attn_dtype's input type; H a multiple of H_kv,
 *          at most 128 query heads per kv head
 *   pages  [B][H_kv][Sq][n_select] int32: page indices within the sequence (0
 *          its first page), ascending, then -1 where fewer are visible
 *   causal, counts as attn_fwd_cache;  max_pages and n_select <= 27648
 *   workspace  16-byte aligned scratch of attn_cache_select_workspace_size
 *          bytes, not overlapping any other argument
 *   B * H_kv * Sq < 2^28
 * The choice is that of exact sums (fp64 decides where fp32 does not).
 * One kernel.
 */
ATTN_API int attn_cache_select_workspace_size(int B, int H_kv, int Sq, int max_pages, size_t *bytes);
ATTN_API int attn_cache_select(const attn_cache *cache, const void *q, const int32_t *table,
                      int max_pages, const int32_t *lens, const int32_t *counts, int32_t *pages,
                      int n_select, int B, int H, int Sq, int causal, int dtype, void *workspace,
                      size_t workspace_bytes, void *stream);

/*
 * attn_fwd_cache -- attention of Sq query rows per sequence over its tokens in
 * the cache.
 *
 *   q, o   [B][H][Sq][d], lse [B][H][Sq] (NULL: not written), types as attn_fwd
 *          (every attn_dtype); H a multiple of H_kv, query heads
 *          h * H / H_kv .. of kv head h; B <= 4096; B * H * Sq < 2^31;
 *          B * max_pages * page / 16 < 2^31
 *   counts the last counts[b] of the lens[b] tokens are the queries' own:
 *          query i sits at position lens[b] - counts[b] + i.  Rows from
 *          counts[b] on see no key.
 *   causal key j is visible to query i iff j <= lens[b] - counts[b] + i (else
 *          every held token is); a row that sees no key gets o = 0, lse = -inf
 *   pages  NULL: all pages (n_select = 0).  Else [B][H_kv][Sq][n_select] with
 *          n_select <= 27648: query
 *          i of kv head h attends only to tokens of the listed pages (page
 *          indices within the sequence, as attn_cache_select gives them; -1 is
 *          skipped; a page listed twice counts twice).
 *   workspace  16-byte aligned scratch of attn_fwd_cache_workspace_size bytes
 *          (0 or n_select for its last argument), not overlapping any other
 *          argument.  Calls that may overlap on the GPU, replays of graphs
 *          among them, need workspaces of their own.
 * Arithmetic: exact products of codes and q (fp32 q: 22 bits of each row's
 * range; 16-bit q: down to 2^-31 of it), fp32 sums.  A weight times its page's v_scale keeps 22 bits for fp32
 * outputs and 11 for 16-bit ones, or is kept to 2^-36 of the row's largest
 * such product (16-bit outputs of many rows: 2^-30) where that is coarser.  A
 * weight below 2^-126 of the row's largest counts as 0.
 * Results do not depend on other sequences' contents, but the grouping of sums
 * (not their terms) follows all lengths of the call.  One or two kernels.
 */
ATTN_API int attn_fwd_cache_workspace_size(int B, int H, int H_kv, int Sq, int d, int dtype,
                                  int n_select, size_t *bytes);
ATTN_API int attn_fwd_cache(const attn_cache *cache, const void *q, void *o, float *lse,
                   const int32_t *table, int max_pages, const int32_t *lens,
                   const int32_t *counts, const int32_t *pages, int n_select, int B, int H,
                   int Sq, int causal, float scale, int dtype, void *workspace,
                   size_t workspace_bytes, void *stream);

/*
 * attn_check_status -- synchronises `stream`, then reads and clears the
 * library's device status word on the current device.  Returns
 * ATTN_ERR_BOUNDS if, in the bounds-checking build (libattn_checked.so,
 * compiled with ATTN_BOUNDS_CHECK), a kernel since the last check computed
 * a global-memory index or TMA coordinate outside its buffer (the access was
 * skipped, so the output is incomplete); ATTN_ERR_TIMEOUT if any tensor-core
 * kernel since the last check gave up a bounded wait (its output is then
 * incomplete); ATTN_ERR_TABLE if a cache kernel read a page number, length
 * or count out of range; ATTN_ERR_CUDA if the stream reports an error;
 * ATTN_OK otherwise.  The normal build never sets ATTN_ERR_BOUNDS.
 */
ATTN_API int attn_check_status(void *stream);

/*
 * attn_shutdown -- releases what the library created on the current device
 * and forgets what it cached about it.  It destroys the two streams and three
 * events of attn_fwd_staged, after waiting for those streams to finish.  It
 * clears the cached capability check, SM count and kernel shared-memory
 * limits, and the device addresses of the status word, of the no-alloc
 * scratch and of the tensor-core kernel's schedule counters.  Work the caller queued on its own streams is not waited for.
 * The next call on the device sets everything up again.  Call it before
 * cudaDeviceReset if the process goes on using the library, since a reset
 * invalidates those handles.  It must not run concurrently with other calls
 * on the same device.  Returns ATTN_OK, or ATTN_ERR_CUDA if destroying a
 * handle failed; the state is forgotten either way.  Not on the source
 * pages: resource management of this library.
 */
ATTN_API int attn_shutdown(void);

/* Human-readable text for an attn_status value (static storage). */
ATTN_API const char *attn_strerror(int status);

/* ATTN_ABI_VERSION of the loaded library. */
ATTN_API int attn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_GB300_ATTN_H */
