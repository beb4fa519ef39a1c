// Attention of sequences that share prefixes over the paged MXFP4 cache.
//
// Softmax-weighted sums over two sets of tokens join exactly: with (m, l, o) of each,
// relative to its own reference m,
//   o = (2^(m1 - m) o1 + 2^(m2 - m) o2) / (2^(m1 - m) l1 + 2^(m2 - m) l2).
// So the prefix of a group of sequences is attended once, with the query rows of all of
// them, by the walk of attn_tree.hip (kPrefix): its keys and values are read and widened
// for up to 64 rows at a time, however many sequences there are.  The same walk takes
// every sequence's tokens behind the prefix (kOwn), and one join adds up the pieces of
// both.  The prefix is cut at whole tiles of 32 tokens; what is left of it goes with
// each sequence's own tokens, as all of a sequence does that is shorter than the prefix.
#include "attn_cache.h"

namespace fp4 {
namespace {

// The prefix's walk: as many rows to a workgroup as a group has on average, its spans of
// rows laid end to end, so that columns are heads alone.
Layout prefix_layout(int64_t batch, int drafts, int q_heads, int kv_heads, int head_dim, int groups) {
    const int64_t rows = batch * drafts * (q_heads / kv_heads) / groups;
    Layout l = layout_of((int)(rows > 65536 ? 65536 : rows < 1 ? 1 : rows), kv_heads, head_dim);
    l.columns = kv_heads / l.heads;
    l.shift = 3;
    while ((int64_t)l.columns * l.heads * l.groups << (l.shift + 1) <= kGridWaves) ++l.shift;
    return l;
}
int span_of(const Layout& l) { return 16 * l.nr * l.groups; }

int64_t prefix_tiles(const Layout& l, int64_t batch, int rows, int kv_heads, int groups) {
    return (((int64_t)2 << l.shift) * (span_of(l) / 16) + batch * rows / 16 + groups) * kv_heads;
}
int64_t own_tiles(const Layout& l, int64_t batch, int rows, int kv_heads) {
    return (((int64_t)2 << l.shift) + batch) * kv_heads * ((rows + 15) / 16);
}

}  // namespace

size_t attn_shared_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads, int groups) {
    const int rows = drafts * (q_heads / kv_heads);
    const size_t own = part_bytes(own_tiles(layout_of(rows, kv_heads, head_dim), batch, rows, kv_heads), head_dim);
    if (groups == 0) return own;
    return own + part_bytes(prefix_tiles(prefix_layout(batch, drafts, q_heads, kv_heads, head_dim, groups), batch, rows,
                                         kv_heads, groups), head_dim);
}

hipError_t launch_attn_shared(const AttnTree& p, hipStream_t s) {
    if (p.num_groups == 0) return launch_attn_tree(p, s);
    const int rows = p.drafts * (p.q_heads / p.kv_heads);
    const Layout l = layout_of(rows, p.kv_heads, p.head_dim);
    const Layout lp = prefix_layout(p.batch, p.drafts, p.q_heads, p.kv_heads, p.head_dim, p.num_groups);
    TreeArgs own = cache_args(p, l), pre = cache_args(p, lp);
    own.groups = pre.groups = p.groups;
    own.prefix_lens = pre.prefix_lens = p.prefix_lens;
    own.num_groups = pre.num_groups = p.num_groups;
    pre.part = reinterpret_cast<float*>(static_cast<char*>(p.ws) +
                                        part_bytes(own_tiles(l, p.batch, rows, p.kv_heads), p.head_dim));
    return with_head_dim(p.head_dim, [&](auto d) {
        constexpr int D = decltype(d)::value;
        hipError_t e = launch_walk<kPrefix, D>(pre, lp, (unsigned)lp.columns, s);
        if (e == hipSuccess) e = launch_walk<kOwn, D>(own, l, (unsigned)l.columns, s);
        return e != hipSuccess ? e : launch_join<kOwn, D>(own, {pre, span_of(lp)}, 1, s);
    });
}

}  // namespace fp4
