// Attention of drafted tokens over the paged MXFP4 cache.
//
//   o = sum_j 2^(c s_j - m) v_j / sum_j 2^(c s_j - m),  s_j = q . k_j,
//   c = scale * log2(e), over the visible tokens j, in one pass: m is a running
//   reference near the row's maximum, and o and the sum are scaled when it moves.
//
// A wave takes one key/value head and up to 16 * NR of the query rows that share it
// (drafts times q_heads / kv_heads), and walks its tokens 32 at a time.  The waves of
// a workgroup take HW neighbouring heads of the same tokens, and RG groups of rows,
// and stage the tokens together through LDS (Stage, copy_tile).
//
//   S^T = K Q^T on v_mfma_f32_16x16x32_bf16: lane (c = lane % 16, g = lane / 16)
//   reads the quarter g of token c's row (the order of a row's values among the
//   steps is free as long as Q is loaded alike), and widens it with its block scales
//   (exact in bf16).
//   The result leaves lane (c, g) with query row c and tokens 4g .. 4g+3, which
//   is what the B operand of O^T = V^T P^T takes if the token order within a
//   step is (g, tile, i): the weights never leave their lane.
//   V^T needs 8 tokens of one value per lane: a lane reads the same d/16 values
//   of its 8 tokens (16 lanes cover the row), widens each with its token's
//   scale, and pairs tokens with byte permutes.
//   O^T leaves lane (c, g) with d/4 consecutive values of row c.
//
// The reference m moves only when some score exceeds it by more than 2^8 (one
// ballot); until then no lane exchange is needed.  Weights are rounded to bf16
// for the second product (they enter it with V's 16-bit format); the rounded
// weights are what is summed, in fp32, by one more matrix instruction with ones.
//
// Work split: the batch's tiles of 32 tokens are laid end to end and cut into
// equal ranges, one per workgroup column, whatever the lengths; a sequence that
// a cut goes through leaves partial (m, sum, o) in the workspace, at most two
// per range, and a second kernel joins them in order.
//
// What bounds it: a token's keys and values are 2 * (d/2 + d/32) bytes, which HBM
// would give at 5 TB/s, and are read once for up to 64 query rows of a key/value head
// (16 at 256 values; more rows take more columns of workgroups, which read them
// again).  With one token to a sequence that is the bound.  With drafts, the
// instructions that widen FP4, turn V and take the exponentials cost more: at 32
// rows a head a step of 32 tokens takes a wave about 320 instructions, 34 of them
// matrix products.  Of the 169 us that the long contexts below take with their copies
// left out, leaving out a kind more saves: products 70, conversions 35, exponentials
// 33, turning V 15, the meeting of the waves 10.
// Heads of 128 values, over several cards: a call among others, and kernel + join
// traced one call after another, which add up to more:
//   64 sequences of 0 .. 8191 tokens, 8 drafts,
//     64 / 8 heads (287 MB)              112 .. 118 us, 2.5 TB/s   105 .. 120 + 13
//   4 of 90001 .. 131072, 16 drafts,
//     32 / 8 heads (524 MB)              183 .. 193 us, 2.8 TB/s   188 .. 225 + 10
//   the same, 64 / 8 heads, two columns         345 us
//   64 of 4096, 1 token, 64 / 8 heads (287 MB)   60 us, 4.8 TB/s         53 +  7
//   one of 100000, 1 token, 64 / 8 (109 MB)      32 us, 3.4 TB/s         24 +  8
//   one of 1500, 1 token, 64 / 8                 13 us, latency         8.8 + 5.2
// In what follows "first" and "second" case are the first two of these, by the
// kernels' least times.
// Tried and slower: each wave loading its head in the matrix core's layout (first
// case 128 us: half-line requests), 64 rows to a wave (154 us), three waves to a SIMD
// (151 us, spills), 64 tokens a step (117 us), 1 row tile of 16 to a wave (162 us).
// No faster: a tile's scores worked out beside the softmax of the one before (112 and
// 190 us), three tiles in flight (113 and 191 us).  Counters of the second case: the
// vector unit is issued to in 53% of the cycles (and holds exponentials longer), the
// matrix core busy in 30%; a wave issues 45% of its time, waits 28% for a unit and 27%
// for LDS and its workgroup.  30% of the LDS cycles are bank conflicts, in both cases,
// whose reads have not been told apart.
#include "attn_cache.h"

namespace fp4 {

size_t attn_tree_workspace_bytes(int drafts, int q_heads, int head_dim, int kv_heads) {
    const int rows = drafts * (q_heads / kv_heads);
    return part_bytes(((int64_t)2 << layout_of(rows, kv_heads, head_dim).shift) * kv_heads * ((rows + 15) / 16), head_dim);
}

hipError_t launch_attn_tree(const AttnTree& p, hipStream_t s) {
    const Layout l = layout_of(p.drafts * (p.q_heads / p.kv_heads), p.kv_heads, p.head_dim);
    const TreeArgs a = cache_args(p, l);
    return with_head_dim(p.head_dim, [&](auto d) {
        constexpr int D = decltype(d)::value;
        const hipError_t e = launch_walk<kTree, D>(a, l, (unsigned)l.columns, s);
        return e != hipSuccess ? e : launch_join<kTree, D>(a, 1, s);
    });
}

}  // namespace fp4
