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
// For many rows (attend_prefix) a workgroup takes 32 rows a wave of up to 8 waves.
// A tile of keys and values is widened to bf16 once for all of them, on its way from
// global memory through registers to LDS (a lane has one block of 32 codes and its
// scale), and the products are v_mfma_f32_32x32x16_bf16:
//   S^T = K Q^T: lane (c = lane % 32, h = lane / 32) ends with row c and tokens
//   8i + 4h .. 8i + 4h+3 of each 32, and the weights are the B operand of
//   O^T = V^T P^T as they stand, V^T by transposing LDS reads of 4 tokens of one value.
//
// What bounds it: a prefix's bytes are few (51 MB for 64 samples of 16384 tokens, 10 us);
// products and softmax are 35 GFLOP (30 us at a library product's rate) and as many vector
// cycles.  A workgroup's tile of 64 tokens of 128 values (128 of 64) by 256 rows takes 2.55
// us, before which lie 2 to 4 us until the last workgroup starts, 2.8 us of reading lengths
// and bounds, and 4 us until the first tile is in LDS.  Calls among others, and kernel +
// join traced one call after another:
//   64 samples of 16384 tokens and up to 1024 own, 64 / 8 heads of 128     69 us   66 + 10
//   54 sessions over 6 prefixes of 1000 .. 9000, 3 drafts, 20 / 4 of 64    32 us   26 +  7
//   4 samples of 1500 tokens, 32 / 8 heads of 128 (by the walk)            16 us   12 +  5
//   32 samples of 16384 tokens and up to 1024 own, 32 / 4 heads of 256     79 us
// (the last one's floor is 15 us, and its kernel spills 37 vector registers).  By the counters of
// the samples the matrix cores are busy for 22% of the kernel and LDS for about as long, 27% of
// that in bank conflicts of the widened tiles' stores (512 cycles a tile: value_turn and
// key_turn serve the reads); a wave does a tile's scores, softmax and second product in turn, so
// little of this overlaps.
// Tried and slower: 4 waves to a workgroup (128 rows; 1 to 5%), the prefixes and the own
// tokens in two launches (68 against 65 us for the first one's kernels), a round of
// workgroups for each kind with the joins between.  Spans that fill fewer waves cost
// nearly as much as full ones: 48 sessions, with 120 rows to a group instead of 135, take
// 24 us, 72, with 180, 28, and 96, with 240, 32.
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
constexpr int kWideWaves = 8;              // of a workgroup that attends a prefix of many rows
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

// A group of a chunk, kept in LDS: a piece needs the registers, and reading the bounds and
// lengths again took each piece two round trips to memory.
struct Group {
    int per, seen, token, tokens;
    int64_t tiles;
};

// Workgroup (block_x, head) of the prefix's many rows.
template <int D, int W>
__device__ __forceinline__ void attend_prefix(const TreeArgs& a, uint8_t* tiles_lds, int block_x, int head, const Range<kPrefix>& range) {
    using S = Wide<D, W>;
    constexpr int kRows = S::kRows, kTokens = S::kTokens, kSteps = D / 16, kOut = D / 32, kSub = kTokens / 32;
    constexpr int kBatch = kSteps < 8 ? kSteps : 8, kGroups = kTokens / 16;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31, h = lane >> 5;

    const int64_t lo = range.lo, hi = range.hi;
    if (lo == hi) return;
    Chunk<kPrefix> chunk = range.chunk;
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

    __shared__ Group kept[64];
    int first = chunk.first;
    auto keep = [&]() {
        __syncthreads();                                     // the chunk before has been read
        if (wave == 0) kept[lane] = {chunk.per, chunk.seen, chunk.token, chunk.tokens, (int64_t)chunk.tiles};
        __syncthreads();
    };
    keep();
    for (int64_t at = lo; at < hi;) {
        if (group - first == 64) {
            first = group;
            chunk = chunk_at<kPrefix>(a, first, lane, 0, kRows);
            keep();
        }
        const Group& of = kept[group - first];
        const int64_t cells = scalar(of.tiles);
        if (cells == 0) {
            ++group;
            continue;
        }
        const int tiles = __builtin_amdgcn_readfirstlane(of.per), seen = __builtin_amdgcn_readfirstlane(of.seen);
        const int token0 = __builtin_amdgcn_readfirstlane(of.token);
        const int rows = __builtin_amdgcn_readfirstlane(of.tokens) * a.group;
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
                const float up = top > m + kSlack ? top : m;         // each row by its own scores alone
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
        // buffer: at D = 128 it takes 220 to 229 of 256 registers, at D = 256 it spills 37 (152
        // bytes of scratch a lane) as it is.
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
            const int64_t slot = 2 * (int64_t)block_x + (at == lo ? 0 : 1);
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
        if (head == 0 && threadIdx.x == 0)
            note_piece<kPrefix>(a, 2 * block_x + (at == lo ? 0 : 1), t0 == 0, t1 == tiles, group, token0, 0, span * kRows, kRows);
        at += t1 - t0;
        if (at - before == cells) before += cells, ++group;
    }
}

// Both kinds of work in one launch of workgroups that are all resident: the first ones
// take the sequences' own tokens, by the walk <NR, HW, RG>, the others the prefixes, by the
// same walk (W = 0) or attend_prefix, each kind as many as its tiles are of all.  (With a
// round of workgroups for each kind, 64 samples of 16384 tokens took 62 us.)
struct Split {
    int own_columns, prefix_columns;       // workgroups to a range
};
// Tile x * total / ranges, the same for all who ask.
__device__ __forceinline__ int64_t tile_at(int x, int64_t total, int ranges) {
    return x == ranges ? total : (int64_t)((double)x * (double)total / (double)ranges);
}
// Ranges of at most `most`, of kMinTiles tiles and more.
__device__ __forceinline__ int ranges_of(int64_t tiles, int64_t most) {
    return tiles == 0 ? 0 : (int)min(max(tiles / kMinTiles, (int64_t)1), max(most, (int64_t)1));
}
// What a tile of the own tokens costs a workgroup, of what one of the prefix does (heads of
// 128: 1.0 and 2.6 us).  Calls with 0.3, 0.37, 0.5 and 1:
//   64 samples of 16384 tokens, up to 1024 own, 64 / 8 heads of 128    70   69   73   81 us
//   the same, heads of 64                                             49   48   53   56
//   32 samples, 32 / 4 heads of 256 (tiles of 32 tokens both)          85   79   77   77
//   54 sessions, 20 / 4 heads of 64 | 128 | 256    32   32   34   36 | 44   42   43   46 | 97   93   91   96
constexpr double own_cost(int waves) { return waves ? 0.37 : 1.0; }

template <int D, int W>
constexpr int kPrefixLds = W ? 4 * Wide<D, W ? W : 1>::kTile : 0;    // keys and values, twice
template <int D, int W, int NR, int HW, int RG>
constexpr int kThreadsOf = W ? 64 * W : 64 * HW * RG;
template <int D, int W, int NR, int HW, int RG>
__global__ __launch_bounds__((kThreadsOf<D, W, NR, HW, RG>), D == 256 && W == 0 ? 1 : 2) void attn_shared_kernel(
    const TreeArgs pre, const TreeArgs own, const Split split) {
    constexpr int kLds = kPrefixLds<D, W> > kStaging<D, HW> ? kPrefixLds<D, W> : kStaging<D, HW>;
    constexpr int kSpan = W ? 32 * W : 16 * NR * RG;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
    const int lane = threadIdx.x & 63;
    Range<kOwn> mine{chunk_at<kOwn>(own, 0, lane, 0, 0), 0, 0};
    Range<kPrefix> shared{chunk_at<kPrefix>(pre, 0, lane, 0, kSpan), 0, 0};
    const int64_t own_total = all_tiles<kOwn>(own, mine.chunk, lane, 0, 0);
    const int64_t prefix_total = all_tiles<kPrefix>(pre, shared.chunk, lane, 0, kSpan);
    const double own_work = (double)own_total * split.own_columns * own_cost(W), work = own_work + (double)prefix_total * split.prefix_columns;
    if (work == 0) return;
    const int blocks = gridDim.x;
    // The prefix's share; the rest goes to the own tokens.
    const int prefix_ranges = min(
        ranges_of(prefix_total, (int64_t)((blocks - split.own_columns) * (1.0 - own_work / work)) / split.prefix_columns), pre.ranges);
    const int own_ranges = min(ranges_of(own_total, (blocks - prefix_ranges * split.prefix_columns) / split.own_columns), own.ranges);
    int i = blockIdx.x;
    if (i < own_ranges * split.own_columns) {
        if (W && __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) >= HW * RG) return;
        const int x = i % own_ranges;
        mine.lo = tile_at(x, own_total, own_ranges), mine.hi = tile_at(x + 1, own_total, own_ranges);
        walk<kOwn, D, NR, HW, RG>(own, lds, x, i / own_ranges, [&](int, int) { return mine; });
        return;
    }
    i -= own_ranges * split.own_columns;
    if (i >= prefix_ranges * split.prefix_columns) return;
    const int x = i / split.prefix_columns, y = i % split.prefix_columns;
    shared.lo = tile_at(x, prefix_total, prefix_ranges), shared.hi = tile_at(x + 1, prefix_total, prefix_ranges);
    if constexpr (W != 0)
        attend_prefix<D, W>(pre, lds, x, y, shared);
    else
        walk<kPrefix, D, NR, HW, RG>(pre, lds, x, y, [&](int, int) { return shared; });
}

// Joins the pieces of a sequence's own tokens and of its group's prefix: workgroup (x, y)
// takes 16 rows of a head (x) of sequence y, and of their values the kPer slices from kPer
// * z on.  The prefix's tiles of 16 rows begin elsewhere: each lane finds its row's.
template <int D, int kPer, int kTeams>
__global__ __launch_bounds__(64 * kPer * kTeams) void attn_shared_join_kernel(const TreeArgs a, const TreeArgs pre, int span) {
    constexpr int kTeam = 64 * kPer;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int b = blockIdx.y, row_tile = blockIdx.x % a.row_tiles, r0 = row_tile * 16, head = blockIdx.x / a.row_tiles;
    const int4 own = a.own_pieces[b];                         // not written for a sequence without drafted tokens
    const int rows = drafts_of(a, b) * a.group;
    if (r0 >= rows) return;
    const int first = own.x >> 1, last = own.y;
    const bool whole = first == last, shares = own.z >= 0;
    if (whole && !shares) return;                             // one piece: written already
    const int team = threadIdx.x / kTeam, part = threadIdx.x % kTeam, i = kPer * blockIdx.z + (part >> 6);

    Joined<D, kTeams> joined;
    if (shares) {
        // Rows of a group are below 2^31: 32-bit divisions.
        const uint32_t row = (uint32_t)(b - own.w) * (uint32_t)pre.rows + r0 + c, first_row = row - c;
        const bool live = r0 + c < rows;
        const uint32_t its_span = (live ? row : first_row) / (uint32_t)span;
        const int2 of = pre.span_pieces[(uint32_t)own.w * (uint32_t)pre.rows / (uint32_t)span + own.z + its_span];
        const int x0 = of.x >> 1, x1 = of.y, per_slot = span / 16;
        int most = x1 - x0;
#pragma unroll
        for (int n = 1; n < 16; n *= 2) most = max(most, __shfl_xor(most, n, 64));
        // Tiles of a piece, or of the group's uncut spans: from there on, the row's.
        const int64_t in_slot = (row - its_span * (uint32_t)span) / 16;
        const int64_t uncut = prefix_place(pre, true, 0, (int64_t)own.w * pre.rows / 16 + own.z, row / 16 * 16, span, head).tile;
        joined.add(pre.part, prefix_place(pre, false, 0, 0, 0, span, 0).stats, team, i, g, x0, live ? x1 : x0 - 1, most, (int)(row & 15),
                   [&](int x) {
                       const int64_t slot = x == x0 ? of.x : 2 * (int64_t)x;
                       return x0 == x1 ? uncut : (slot * per_slot + in_slot) * pre.kv_heads + head;
                   });
    }
    joined.add(a.part, part_place<kOwn>(a, whole, 0, b, 0, row_tile, head).stats, team, i, g, first, last, last - first, c, [&](int x) {
        return part_place<kOwn>(a, whole, x == first ? own.x : 2 * (int64_t)x, b, 0, row_tile, head).tile;
    });
    finish_join<D, kPer>(joined, team, part, i, lane, r0, rows, [&](int row) {
        return a.out + ((int64_t)b * a.drafts + row / a.group) * a.ld_out + ((int64_t)head * a.group + row % a.group) * D;
    });
}

// How the call is laid out, from its shapes alone.  The prefixes are attended by the walk,
// laid out for as many rows as a group has on average, or by attend_prefix; spans of rows
// are laid end to end, so that columns are heads alone.  Walk and attend_prefix, one group
// with up to 200 own tokens, 64 / 8 heads of 128 (32 / 4 of 256):
//   rows of the group                    16        32        64        96       128
//   prefix of 2000 tokens           17 | 18   19 | 18   22 | 22   24 | 22   26 | 23 us
//   of 16000                        24 | 29   28 | 29   32 | 33   43 | 36   41 | 40
//   of 2000, heads of 256           20 | 23   21 | 24   24 | 27   30 | 34   38 | 35
//   of 16000, heads of 256          28 | 39   42 | 41   51 | 46   72 | 61   74 | 62
// The average is over num_groups and the whole batch: the bounds are on the device.  Empty
// groups and sequences outside groups spoil it: the 64 samples above take 69 us alone, 83 as
// one of 8 groups of which the others are empty and 102 as one of 64; a group of two among 64
// sequences of 16384 tokens takes 221, the attention without groups 149.
struct SharedLayout {
    Layout own;
    int waves;                             // of attend_prefix; 0: the walk, laid out as own
    int span, prefix_columns, blocks;
    int own_ranges() const { return blocks / own.columns; }
    int prefix_ranges() const { return blocks / prefix_columns; }
};
// own_rows: of a sequence, rows: of a group.
SharedLayout shared_layout(int own_rows, int64_t rows, int kv_heads, int head_dim) {
    SharedLayout l;
    l.waves = rows <= 64 ? 0 : kWideWaves;
    l.own = layout_of(l.waves ? own_rows : (int)(rows < own_rows ? own_rows : rows), kv_heads, head_dim);
    const int own_span = 16 * l.own.nr * l.own.groups;
    l.own.columns = kv_heads / l.own.heads * ((own_rows + own_span - 1) / own_span);
    l.span = l.waves ? 32 * l.waves : own_span;
    l.prefix_columns = l.waves ? kv_heads : kv_heads / l.own.heads;
    // All resident where the columns allow it.
    l.blocks = kGridWaves / (l.waves ? l.waves : l.own.heads * l.own.groups);
    const int least = 2 * (l.own.columns + l.prefix_columns);
    if (l.blocks < least) l.blocks = least;
    return l;
}

int64_t own_tiles(const SharedLayout& l, int64_t batch, int rows, int kv_heads) {
    return (2 * (int64_t)l.own_ranges() + batch) * kv_heads * ((rows + 15) / 16);
}
int64_t prefix_tiles(const SharedLayout& l, int64_t batch, int rows, int kv_heads, int groups) {
    return (2 * (int64_t)l.prefix_ranges() * (l.span / 16) + batch * rows / 16 + groups) * kv_heads;
}
int64_t spans(const SharedLayout& l, int64_t batch, int rows, int groups) { return batch * rows / l.span + groups; }

}  // namespace

// In this order: own_pieces, span_pieces, the own tokens' partial results, the prefixes'.
// The largest of all layouts that up to 64 rows to a group (their row tiles change at 16
// and 32) and more may get, and of the attention without groups: each grows with the batch
// and the groups, so that a workspace serves every smaller step.
size_t attn_shared_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads, int groups) {
    size_t most = attn_tree_workspace_bytes(drafts, q_heads, head_dim, kv_heads);
    if (groups == 0) return most;
    const int rows = drafts * (q_heads / kv_heads);
    for (const int group_rows : {16, 32, 64, 65}) {
        const SharedLayout l = shared_layout(rows, group_rows, kv_heads, head_dim);
        const size_t bytes =
            (size_t)batch * sizeof(int4) + (size_t)((spans(l, batch, rows, groups) + 1) / 2) * sizeof(int4) +
            part_bytes(own_tiles(l, batch, rows, kv_heads) + prefix_tiles(l, batch, rows, kv_heads, groups), head_dim);
        most = bytes > most ? bytes : most;
    }
    return most;
}

hipError_t launch_attn_shared(const AttnTree& p, hipStream_t s) {
    if (p.num_groups == 0) return launch_attn_tree(p, s);
    const int rows = p.drafts * (p.q_heads / p.kv_heads);
    const SharedLayout l = shared_layout(rows, p.batch * rows / p.num_groups, p.kv_heads, p.head_dim);
    TreeArgs own = cache_args(p, l.own);
    own.groups = p.groups, own.prefix_lens = p.prefix_lens, own.num_groups = p.num_groups;
    own.own_pieces = static_cast<int4*>(p.ws);
    own.span_pieces = reinterpret_cast<int2*>(own.own_pieces + p.batch);
    own.part = reinterpret_cast<float*>(own.own_pieces + p.batch + (spans(l, p.batch, rows, p.num_groups) + 1) / 2);
    TreeArgs pre = own;
    pre.part = own.part + part_bytes(own_tiles(l, p.batch, rows, p.kv_heads), p.head_dim) / sizeof(float);
    own.ranges = l.own_ranges(), pre.ranges = l.prefix_ranges();
    const Split split{l.own.columns, l.prefix_columns};
    const unsigned blocks = (unsigned)l.blocks;
    return with_head_dim(p.head_dim, [&](auto d) {
        constexpr int D = decltype(d)::value, kW = kWideWaves;
        hipError_t e = with_layout<D>(l.own, [&](auto nr, auto hw, auto rg) {
            constexpr int kNR = decltype(nr)::value, kHW = decltype(hw)::value, kRG = decltype(rg)::value;
            pre.prefix_tile = l.waves ? Wide<D, kW>::kTokens : kTile;
            if (l.waves)
                attn_shared_kernel<D, kW, kNR, kHW, kRG><<<blocks, kThreadsOf<D, kW, kNR, kHW, kRG>, 0, s>>>(pre, own, split);
            else
                attn_shared_kernel<D, 0, kNR, kHW, kRG><<<blocks, kThreadsOf<D, 0, kNR, kHW, kRG>, 0, s>>>(pre, own, split);
            return hipGetLastError();
        });
        if (e != hipSuccess) return e;
        const unsigned row_tiles = (unsigned)(p.kv_heads * own.row_tiles);
        // Few rows, and so few workgroups: 16 waves to a slice, as in launch_join.
        if ((int64_t)row_tiles * p.batch * (D / 16) <= 512)
            attn_shared_join_kernel<D, 1, 16><<<dim3(row_tiles, (unsigned)p.batch, D / 16), 1024, 0, s>>>(own, pre, l.span);
        else
            attn_shared_join_kernel<D, D / 16, 1><<<dim3(row_tiles, (unsigned)p.batch), 4 * D, 0, s>>>(own, pre, l.span);
        return hipGetLastError();
    });
}

}  // namespace fp4
