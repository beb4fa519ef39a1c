// Attention over selected blocks of the paged MXFP4 cache.
//
// The walk of attn_tree.hip over other tokens: a drafted token's listed blocks stand
// one after another, as if they were the beginning of its sequence, and the tokens
// behind the last complete block and the drafted ones follow.  A wave takes the query
// heads of one drafted token that share a key/value head, each drafted token a column
// of workgroups of its own.  With one list for all heads the waves of a workgroup stage
// neighbouring heads of the same rows together; with a list for each, a workgroup has
// one head.
//
// What bounds it: latency for a few queries (lengths, list, page table and tiles are read
// one after another, and the join waits for the walk), HBM for many.  Calls among others
// on cold inputs, and kernel + join traced one call after another:
//   64 sequences, 64 blocks of 64 tokens each, 64 / 8
//     heads of 128 (290 MB)                            73 us, 4.0 TB/s     56 + 5
//   one, 32 blocks of 64 tokens, 64 / 8 heads of 128   13 us, latency       9 + 4
//   16, 4 drafts, 40 blocks of 32 tokens for each of
//     4 heads of 64, 20 / 4 (20 MB)             17 .. 18 us, latency      13 + 4
#include "attn_cache.h"

namespace fp4 {
namespace {

Layout blocks_layout(int drafts, int q_heads, int kv_heads, int head_dim, bool apart) {
    return layout_of(q_heads / kv_heads, kv_heads, head_dim, drafts, apart);
}

}  // namespace

int64_t attn_blocks_columns(int drafts, int q_heads, int kv_heads, int head_dim, int lists) {
    return blocks_layout(drafts, q_heads, kv_heads, head_dim, lists > 1).columns;
}

// The partial results, then span_pieces.
size_t attn_blocks_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads) {
    int shift = 0;
    for (bool apart : {false, true}) {
        const Layout l = blocks_layout(drafts, q_heads, kv_heads, head_dim, apart);
        shift = l.shift > shift ? l.shift : shift;
    }
    return part_bytes(((int64_t)2 << shift) * kv_heads * drafts * ((q_heads / kv_heads + 15) / 16), head_dim) +
           (size_t)batch * drafts * sizeof(int2);
}

hipError_t launch_attn_blocks(const AttnTree& p, hipStream_t s) {
    const Layout l = blocks_layout(p.drafts, p.q_heads, p.kv_heads, p.head_dim, p.lists > 1);
    TreeArgs a = cache_args(p, l);
    a.rows = a.group, a.row_tiles = (a.group + 15) / 16;
    a.ids = p.block_ids, a.select = p.n_select, a.lists = p.lists;
    a.span_pieces = reinterpret_cast<int2*>(a.part + part_bytes(((int64_t)2 << l.shift) * p.kv_heads * p.drafts * a.row_tiles, p.head_dim) /
                                                         sizeof(float));
    return with_head_dim(p.head_dim, [&](auto d) {
        constexpr int D = decltype(d)::value;
        const hipError_t e = launch_walk<kBlocks, D>(a, l, (unsigned)l.columns, s);
        return e != hipSuccess ? e : launch_join<kBlocks, D>(a, p.drafts, s);
    });
}

}  // namespace fp4
