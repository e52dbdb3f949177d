// attn_bwd.h -- what the kernels of the backward pass share: the arguments, the
// plan of the work, and the layout of the workspace.
//
// From q, do [B, H, Sq, d], k, v [B, H_kv, Skv, d], o, lse of the forward pass
// and (optionally) the gradient of the lse:
//     P  = exp(scale q k^T - lse)        on the visible keys, recomputed
//     D  = rowsum(o * do) - dlse         (the softmax's and the lse's share)
//     dS = P * (do v^T - D)
//     dq = scale dS k,   dk = scale dS^T q,   dv = P^T do
// with dk and dv summed over the query heads that share a kv head.
//
// No sum is made by atomics, so results do not depend on the order in which
// CTAs run.  The work is cut into units of two kinds, each of which owns its
// outputs: a kv unit holds one tile of keys (k and v) and walks over the query
// tiles of all heads that share it; a q unit holds one tile of queries (q and
// do) and walks over the key tiles.  P and dP are therefore computed twice
// (seven products of a tile instead of five), which costs less than summing dq
// in global memory in a fixed order.  Where units are few and long, their
// walks are cut into splits that leave fp32 partial sums in the workspace,
// and a last kernel adds those in order.
//
// Both kinds need of each query row: nl = -lse log2(e) (-inf for a row that sees
// no key, so that its P is 0) and nd = -D.  For the 16-bit types a first kernel
// writes them as [B * H][query tiles of 128][2][128], rows behind Sq with nl =
// -inf, nd = 0; fp32 units compute them as they load do.
//
// fp16: dS is held in fp16 for the products with q and k, and its size follows that of
// do, which a loss scale or its absence, and the weight of a sequence or a token in the
// loss, move by orders of magnitude.  |dS| <= |do| |v| + |D|, so norms of the rows give a
// power of two that brings dS to 2^14 at most; it has to be one for all terms of a sum:
//     dq: one for each query row, from its |do| and |D| and the largest |v| of the key tiles
//         its unit walks over;
//     dk: one for each kv unit, from the largest |do| and |D| of the query tiles it walks
//         over and the largest |v| of its keys.
// So no head's precision depends on another's do.  The first kernel writes |do| of each row
// as a third number beside nl and nd (kScaleRows), and the largest values of each query tile
// and of each tile of v, which the units join.  Rows with an infinity or a NaN do not count.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "attn_internal.h"

namespace attn {

constexpr int kStatTile = 128;   // query rows of one block of row statistics
constexpr int kBwdSms = 152;     // the splits are planned for this many SMs
constexpr int kMaxBwdSplits = 64;
constexpr int kMaxBwdRows = INT32_MAX - 1023;  // of a head: ends of tiles fit 31 bits
constexpr int kFewKeys = 128;    // see BwdPlan::few
constexpr int kBwdP16Log2 = 14;  // fp16: P is kept times 2^14, so that small weights stay normal numbers
constexpr int kPreBlocks = 1216; // CTAs of the first kernel at most (bf16)
constexpr size_t kMaximaBytes = 3 * kPreBlocks * 4;
constexpr int kScaleRows = 3;    // fp16: numbers of a query row that the first kernel writes (bf16: 2)

struct BwdPlan {
    Problem p;          // the problem the kernels run, see below
    int off;            // key j is visible to the query at position i iff j <= i + off
    int wrap;           // 0, or query rows of a head, where p's rows are those of several heads
    int tile;           // rows of a unit's own tile
    int nq, nk;         // query and key tiles of that size
    int ns_kv, ns_q;    // splits of a kv unit and of a q unit
    bool q_first;       // q units come before kv units
    int few;            // 16-bit types: query tiles of a head, from the first on, with dS in two parts
    int64_t n_units;
    // fp16: off_max [B * H][query tiles][2] largest |do| and |D|, off_max_v [B * H_kv][key tiles] largest |v|
    size_t off_stats, off_max, off_max_v, off_part_kv, off_part_q, bytes;
};

struct BwdArgs {
    const void *q, *k, *v, *o, *dout;
    const float *lse, *dlse;
    void *dq, *dk, *dv;
    void *workspace;
};

// The plan follows from the sizes alone, so that the workspace does too.
// False if the problem is too large to number.
//
// The query heads that share a kv head lie one behind the other, so that their
// rows can be walked as the rows of one head (plan.p: H_kv heads of group * Sq
// rows), with fewer tiles left partly empty.  Without a causal mask this is
// always done; with one for up to a tile of queries and no more than there are keys,
// where a row's position is its number modulo Sq (longer ones would lose the key
// tiles that the mask leaves out; rows that see no key are the first of a head).
bool bwd_plan(const Problem &p, BwdPlan *plan);

// The kernels in order: row statistics (16-bit types), gradients, sum of the splits.
int launch_bwd(const BwdArgs &a, const BwdPlan &plan, cudaStream_t stream);
int launch_bwd_tc(const BwdArgs &a, const BwdPlan &plan, cudaStream_t stream);
int launch_bwd_f32(const BwdArgs &a, const BwdPlan &plan, cudaStream_t stream);

}  // namespace attn
