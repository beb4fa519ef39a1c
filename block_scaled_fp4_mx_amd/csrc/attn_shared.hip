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
//
// For many rows (attn_prefix_kernel) a workgroup takes 32 rows a wave of up to 8 waves.
// A tile of keys and values is widened to bf16 once for all of them, on its way from
// global memory through registers to LDS (a lane has one block of 32 codes and its
// scale), and the products are v_mfma_f32_32x32x16_bf16:
//   S^T = K Q^T: lane (c = lane % 32, h = lane / 32) ends with row c and tokens
//   8i + 4h .. 8i + 4h+3 of each 32, and the weights are the B operand of
//   O^T = V^T P^T as they stand, V^T by transposing LDS reads of 4 tokens of one value.
#include "attn_cache.h"

namespace fp4 {
namespace {

typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// A tile of keys and one of values in LDS, rows of D values without padding, 16-byte
// chunk x of row r at x ^ turn: key_turn keeps the 16 lanes that read one chunk of 16
// rows in different banks, value_turn the 4 rows of 64 bytes that half the lanes of a
// transposing read take.
template <int D, int W>
struct Wide {
    static constexpr int kRows = 32 * W;                     // query rows of a workgroup
    static constexpr int kTokens = 8192 / D;                 // keys of a tile
    static constexpr int kRow = 2 * D, kTile = kTokens * kRow;           // bytes
    static constexpr int kBlocks = kTokens * D / 32;         // of 32 codes, of the keys and of the values
    static constexpr int kItems = (2 * kBlocks + 64 * W - 1) / (64 * W);        // of a lane
    __device__ static constexpr int key_turn(int row) { return D == 64 ? (row >> 1) & 7 : row & 15; }
    __device__ static constexpr int value_turn(int row) { return D == 64 ? 4 * ((row >> 1) & 1) : 4 * (row & 3); }
};

template <int D, int W>
__global__ __launch_bounds__(64 * W, 2) void attn_prefix_kernel(const TreeArgs a) {
    using S = Wide<D, W>;
    constexpr int kRows = S::kRows, kTokens = S::kTokens, kSteps = D / 16, kOut = D / 32, kSub = kTokens / 32;
    constexpr int kBatch = kSteps < 8 ? kSteps : 8, kGroups = kTokens / 16;
    __shared__ __attribute__((aligned(16))) uint8_t tiles_lds[2 * 2 * S::kTile];        // keys, values; twice
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31, h = lane >> 5;
    const int head = __builtin_amdgcn_readfirstlane(blockIdx.y);

    Chunk<kPrefix> chunk = chunk_at<kPrefix>(a, 0, lane, 0, kRows);
    const int64_t total = all_tiles<kPrefix>(a, chunk, lane, 0, kRows);
    const int shift = shift_of(a, total);
    const int64_t lo = blockIdx.x * total >> shift, hi = (blockIdx.x + 1) * total >> shift;
    if (blockIdx.x >> shift || lo == hi) return;
    int64_t before = 0;
    while (before + (int64_t)chunk.all() <= lo) {
        before += chunk.all();
        chunk = chunk_at<kPrefix>(a, chunk.first + 64, lane, 0, kRows);
    }
    int group = chunk.first;
    {
        const int k = __popcll(__ballot(before + (int64_t)chunk.upto <= lo));
        if (k) before += chunk.read(chunk.upto, k - 1);
        group += k;
    }

    // This lane's blocks of a tile: its row, where they lie behind 16 rows' first one, and
    // where their four chunks go in LDS (chunk j at write ^ 16 j).
    int at_group[S::kItems];
    uint32_t code_at[S::kItems], scale_at[S::kItems], write[S::kItems];
#pragma unroll
    for (int i = 0; i < S::kItems; ++i) {
        const int item = (i * W + wave) * 64 + lane, row = item % S::kBlocks / (D / 32), block = item % (D / 32);
        const bool key = item < S::kBlocks;
        at_group[i] = item < 2 * S::kBlocks ? row / 16 : -1;
        code_at[i] = row % 16 * a.code_row + head * (D / 2) + block * 16;
        scale_at[i] = row % 16 * a.scale_row + head * (D / 32) + block;
        write[i] = (key ? 0 : S::kTile) + row * S::kRow + ((4 * block) ^ (key ? S::key_turn(row) : S::value_turn(row))) * 16;
    }
    // LDS offsets of this lane's reads: a step's keys (steps 8 on lie 256 bytes
    // further), and the values of each 32 (the fifth on 256 bytes further).
    constexpr int kTurns = kOut < 4 ? kOut : 4;
    uint32_t rk[kBatch], rv[kTurns];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) rk[i] = c * S::kRow + ((2 * i + h) ^ S::key_turn(c)) * 16;
    {
        const int r = 4 * h + (lane & 15) / 4, x = (2 * ((lane >> 4) & 1) + (lane & 3) / 2) ^ S::value_turn(r);
#pragma unroll
        for (int i = 0; i < kTurns; ++i) rv[i] = S::kTile + r * S::kRow + (x ^ (4 * i)) * 16 + (lane & 1) * 8;
    }

    int first = chunk.first;
    for (int64_t at = lo; at < hi;) {
        // Read again for every piece: a piece needs the registers.
        if (group - first == 64) first = group;
        if (at != lo || first != chunk.first) chunk = chunk_at<kPrefix>(a, first, lane, 0, kRows);
        const int at_lane = group - first;
        const int64_t cells = chunk.read(chunk.tiles, at_lane);
        if (cells == 0) {
            ++group;
            continue;
        }
        const int tiles = __builtin_amdgcn_readlane(chunk.per, at_lane), seen = __builtin_amdgcn_readlane(chunk.seen, at_lane);
        const int token0 = __builtin_amdgcn_readlane(chunk.token, at_lane);
        const int rows = __builtin_amdgcn_readlane(chunk.tokens, at_lane) * a.group;
        const int64_t span = cells >> 32 ? (at - before) / tiles : (int64_t)((uint32_t)(at - before) / (uint32_t)tiles);
        const int t0 = (int)(at - before - span * tiles), t1 = (int)min(hi - at + t0, (int64_t)tiles);
        const int32_t* table = a.table + (int64_t)(token0 / a.drafts) * a.max_pages;
        const int row0 = (int)span * kRows + 32 * wave, row = row0 + c;      // the wave's first query row, this lane's
        const bool live = row < rows, busy = row0 < rows;

        u32x4 q[kSteps];
        v16f o[kOut];
#pragma unroll
        for (int i = 0; i < kOut; ++i) o[i] = v16f{};
        float m = kFloor, sum[4] = {0.f, 0.f, 0.f, 0.f};     // sum: of the rounded weights, in four parts

        // The lanes hold the first cache rows of 64 runs of 16 tokens from run first_run on
        // (-1: none), worked out together.
        int first_run = -64, runs = 0;
        u32x4 code[S::kItems];
        uint32_t scale[S::kItems], valid = 0;
        auto load = [&](int t) {
            const int run = t * kGroups;
            if (run >= first_run + 64) {
                first_run = run;
                const int at_run = run + lane, per = a.page_size / 16, i = at_run / per;
                const int page = table[min(i, (int)a.max_pages - 1)];
                const bool there = at_run < seen / 16 && (uint32_t)page < (uint32_t)a.num_pages;
                runs = there ? page * a.page_size + (at_run - i * per) * 16 : -1;
            }
            valid = (uint32_t)(__ballot(runs >= 0) >> (run - first_run)) & ((1u << kGroups) - 1);
#pragma unroll
            for (int i = 0; i < S::kItems; ++i) {
                const int from = __shfl(runs, run - first_run + max(at_group[i], 0), 64);
                code[i] = u32x4{0, 0, 0, 0}, scale[i] = 127;
                if (at_group[i] >= 0 && from >= 0) {
                    const bool key = (i * W + wave) * 64 < S::kBlocks;           // a wave has one kind
                    code[i] = *reinterpret_cast<const u32x4*>((key ? a.kc : a.vc) + (int64_t)from * a.code_row + code_at[i]);
                    scale[i] = ((key ? a.ks : a.vs) + (int64_t)from * a.scale_row)[scale_at[i]];
                }
            }
        };
        auto store = [&](uint8_t* tile) {
#pragma unroll
            for (int i = 0; i < S::kItems; ++i) {
                if (at_group[i] < 0) continue;
                const float sc = __uint_as_float(scale[i] << 23);
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<u32x4*>(tile + (write[i] ^ (16 * j))) = widen8(code[i][j], sc);
            }
        };
        auto compute = [&](const uint8_t* tile, uint32_t runs_seen) {
            v16f s[kSub];
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                s[u] = v16f{};
#pragma unroll
                for (int b = 0; b < kSteps / kBatch; ++b) {
                    u32x4 kf[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        kf[i] = *reinterpret_cast<const u32x4*>(tile + rk[i] + 32 * u * S::kRow + 256 * b);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[i]),
                                                                       __builtin_bit_cast(bf16x8, q[b * kBatch + i]), s[u], 0, 0, 0);
                }
            }
            if (runs_seen != (1u << kGroups) - 1) {          // runs without a page, or behind the prefix
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[u][i] = runs_seen >> (2 * u + i / 8) & 1 ? s[u][i] : kNone;
            }
            float top = s[0][0];
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
            top *= a.scale2;
            if (__any(top > m + kSlack)) {
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float up = fmaxf(m, top);
                const float alpha = exp2_hw(m - up);
                m = up;
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] *= alpha;
#pragma unroll
                for (int i = 0; i < kOut; ++i) o[i] *= alpha;
            }
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                uint32_t p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[i] = pack2(exp2_hw(fmaf(s[u][2 * i], a.scale2, -m)), exp2_hw(fmaf(s[u][2 * i + 1], a.scale2, -m)));
                    sum[i & 3] = add_products(sum[i & 3], p[i], 0x3F803F80u);
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {                // 16 tokens
                    const bf16x8 pb = __builtin_bit_cast(bf16x8, u32x4{p[4 * w], p[4 * w + 1], p[4 * w + 2], p[4 * w + 3]});
#pragma unroll
                    for (int i = 0; i < kOut; ++i) {
                        const uint8_t* x = tile + rv[i % kTurns] + (32 * u + 16 * w) * S::kRow + 256 * (i / kTurns);
                        const v4s x0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(x));
                        const v4s x1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(x + 8 * S::kRow));
                        const bf16x8 va = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7));
                        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va, pb, o[i], 0, 0, 0);
                    }
                }
            }
        };
        // When the waves meet, tile t is in LDS and the other buffer is free: tile t + 1 goes
        // there from the registers, and tile t + 2 is asked for.
        load(t0);
        {
            const int r = live ? row : 0;
            const uint16_t* p = a.q + ((int64_t)token0 + r / a.group) * a.ld_q + ((int64_t)head * a.group + r % a.group) * D + 8 * h;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                q[s] = live ? *reinterpret_cast<const u32x4*>(p + 16 * s) ^ a.flip : u32x4{0, 0, 0, 0};
        }
        __syncthreads();                                     // the piece before has been read
        store(tiles_lds);
        uint32_t now = valid;
        if (t0 + 1 < t1) load(t0 + 1);
        // Of the two waves of a SIMD one widens before its products and one behind them, so
        // that the matrix core has work meanwhile.  One copy of the step, not one for each
        // buffer: at D = 256 two do not fit the registers.
        const bool early = wave < W / 2;
#pragma unroll 1
        for (int t = t0; t < t1; ++t) {
            const int buffer = ((t - t0) & 1) * 2 * S::kTile;
            __syncthreads();
            const uint32_t runs_seen = now;
            now = valid;
            auto widen = [&]() {
                if (t + 1 < t1) store(tiles_lds + (2 * S::kTile - buffer));
                if (t + 2 < t1) load(t + 2);
            };
            if (early) widen();
            if (busy) compute(tiles_lds + buffer, runs_seen);
            if (!early) widen();
        }

        float l = sum[0] + sum[1] + sum[2] + sum[3];
        l += __shfl_xor(l, 32, 64);
        if (row0 + (c & 16) < rows) {
            // As the walk's lanes hold a tile of 16 rows: value g * D/4 + k * D/16 + i of row c
            // at [i][g][c], component k.
            const int64_t slot = 2 * (int64_t)blockIdx.x + (at == lo ? 0 : 1);
            const PartPlace p = prefix_place(a, t0 == 0 && t1 == tiles, slot, tile_base(a, group), row0 + (c & 16), kRows, head);
            v4f* y = reinterpret_cast<v4f*>(a.part) + p.tile * (4 * D) + (c & 15);
            if constexpr (D == 128) {
#pragma unroll
                for (int i = 0; i < kOut; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[(4 * h + e) * 64 + i * 16] = v4f{o[i][e], o[i][4 + e], o[i][8 + e], o[i][12 + e]};
            } else if constexpr (D == 256) {
#pragma unroll
                for (int g = 0; g < 4; ++g)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            y[(8 * j + 4 * h + e) * 64 + g * 16] = v4f{o[2 * g][4 * j + e], o[2 * g][8 + 4 * j + e],
                                                                       o[2 * g + 1][4 * j + e], o[2 * g + 1][8 + 4 * j + e]};
            } else {
                // Components 0 and 2 are in the lower half of the wave, 1 and 3 in the upper: the
                // halves exchange values e and e + 2 and write one each.
#pragma unroll
                for (int i = 0; i < kOut; ++i)
#pragma unroll
                    for (int j = 0; j < 4; j += 2)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            v4f v;
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const float near = o[i][4 * (j + k) + e], far = o[i][4 * (j + k) + e + 2];
                                const float other = __shfl_xor(h ? near : far, 32, 64);
                                v[2 * k] = h ? other : near, v[2 * k + 1] = h ? far : other;
                            }
                            y[(e + 2 * h) * 64 + (2 * i + j / 2) * 16] = v;
                        }
            }
            float2* ml = reinterpret_cast<float2*>(a.part + p.stats * (16 * D));
            if (h == 0) ml[p.tile * 16 + (c & 15)] = make_float2(m, l);
        }
        at += t1 - t0;
        if (at - before == cells) before += cells, ++group;
    }
}

// How the prefix is attended: by the walk, with as many rows to a workgroup as a group
// has on average, or by attn_prefix_kernel.  Spans of rows are laid end to end, so that
// columns are heads alone.
struct PrefixLayout {
    Layout walk;
    int waves;                             // of attn_prefix_kernel; 0: the walk
    int span, shift;
};
PrefixLayout prefix_layout(int64_t batch, int drafts, int q_heads, int kv_heads, int head_dim, int groups) {
    const int64_t rows = batch * drafts * (q_heads / kv_heads) / groups;
    PrefixLayout l;
    l.walk = layout_of((int)(rows > 65536 ? 65536 : rows < 1 ? 1 : rows), kv_heads, head_dim);
    l.waves = rows > 128 || (head_dim == 256 && rows > 64) ? 8 : rows > 64 ? 4 : 0;
    l.span = l.waves ? 32 * l.waves : 16 * l.walk.nr * l.walk.groups;
    const int columns = l.waves ? kv_heads : kv_heads / l.walk.heads;
    const int waves = l.waves ? l.waves : l.walk.heads * l.walk.groups;
    l.shift = 3;
    while ((int64_t)columns * waves << (l.shift + 1) <= kGridWaves) ++l.shift;
    l.walk.shift = l.shift, l.walk.columns = columns;
    return l;
}

int64_t prefix_tiles(const PrefixLayout& l, int64_t batch, int rows, int kv_heads, int groups) {
    return (((int64_t)2 << l.shift) * (l.span / 16) + batch * rows / 16 + groups) * kv_heads;
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
    const PrefixLayout lp = prefix_layout(p.batch, p.drafts, p.q_heads, p.kv_heads, p.head_dim, p.num_groups);
    TreeArgs own = cache_args(p, l), pre = cache_args(p, lp.walk);
    own.groups = pre.groups = p.groups;
    own.prefix_lens = pre.prefix_lens = p.prefix_lens;
    own.num_groups = pre.num_groups = p.num_groups;
    pre.part = reinterpret_cast<float*>(static_cast<char*>(p.ws) +
                                        part_bytes(own_tiles(l, p.batch, rows, p.kv_heads), p.head_dim));
    return with_head_dim(p.head_dim, [&](auto d) {
        constexpr int D = decltype(d)::value;
        pre.prefix_tile = lp.waves ? Wide<D, 8>::kTokens : kTile;
        hipError_t e;
        if (lp.waves == 0) {
            e = launch_walk<kPrefix, D>(pre, lp.walk, (unsigned)lp.walk.columns, s);
        } else {
            const dim3 grid(1u << lp.shift, (unsigned)p.kv_heads);
            if (lp.waves == 8) {
                attn_prefix_kernel<D, 8><<<grid, 512, 0, s>>>(pre);
            } else {
                if constexpr (D < 256) attn_prefix_kernel<D, 4><<<grid, 256, 0, s>>>(pre);
            }
            e = hipGetLastError();
        }
        if (e == hipSuccess) e = launch_walk<kOwn, D>(own, l, (unsigned)l.columns, s);
        return e != hipSuccess ? e : launch_join<kOwn, D>(own, {pre, lp.span}, 1, s);
    });
}

}  // namespace fp4
