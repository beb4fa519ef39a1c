// Attention over the paged MXFP4 cache: a wave's walk over its tokens, 32 at a time,
// and the split of the tokens of a batch over workgroups.  attn_tree.hip describes the
// kernel; attn_blocks.hip and attn_shared.hip run it over other tokens and rows.
#pragma once

#include <type_traits>

#include "fp4_internal.h"
#include "mma_core.h"

namespace fp4 {
namespace {

constexpr int kTile = 32;                  // tokens per step
// Tiles per range below which fewer ranges are used.  One token over 1500, kernel and
// join: 8.4 + 4.8 us; with 4, 12.2 + 4.0; with 1, 7.8 + 5.2, but over 8000 tokens
// 11.8 + 5.6 against 11.2 + 4.8.
constexpr int kMinTiles = 2;
// Waves of a full grid, two per SIMD (of which one fits at 256 values, where a wave
// takes 264 registers and more).  The long contexts above, with one row group, take
// 198 + 11 us; with 1024 waves 236 + 14, with 4096 228 + 20 (twice the partial results).
constexpr int kGridWaves = 2048;
constexpr float kSlack = 8.0f;             // scores may exceed the reference by 2^8
constexpr float kNone = -__builtin_inff();   // score of a hidden token
constexpr float kFloor = -3e38f;           // reference of a row that has seen nothing

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) uint8_t* lds_bytes;
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// What a workgroup's tokens and rows are.
enum Mode {
    kTree,       // a sequence's tokens; rows: its drafted tokens' heads
    kBlocks,     // its listed blocks, last incomplete block and drafted tokens; rows: one drafted token's heads
    kPrefix,     // the prefix of a group of sequences; rows: the heads of all their drafted tokens
    kOwn,        // a sequence's tokens behind its group's prefix; rows as in kTree
};

struct TreeArgs {
    const uint16_t* q;
    int64_t ld_q;
    const uint8_t *kc, *ks, *vc, *vs;
    int64_t num_pages;
    int page_size;
    int code_row, scale_row;               // bytes of a cache row
    const int32_t* table;
    int64_t max_pages;
    const int32_t *seq_lens, *draft_lens;
    const uint64_t* mask;
    int batch, drafts, group, kv_heads, rows;   // rows = drafts * group: query rows of a key/value head
    float scale2;                          // |scale| * log2(e), positive
    uint32_t flip;                         // sign bits of Q, set for a negative scale
    uint16_t* out;
    int64_t ld_out;
    // Partial results [2 * ranges][kv_heads][row tiles]: of 16 rows, the sums as the
    // lanes hold them ([D/16][64] of 4 values), then (m, sum) of each row.
    float* part;
    int row_tiles, shift, ranges;          // ranges: 1 << shift, or (kPrefix, kOwn) at most
    // kBlocks: lists [batch][drafts][lists][select] of blocks; the planes of workgroups
    // are the drafted tokens, and rows is one's, group.
    const int32_t* ids;
    int select, lists;
    // kPrefix, kOwn: group g is the sequences [groups[g], groups[g + 1]).  Pieces that
    // are not cut stand behind those of the ranges (slot 2 * ranges on): in kOwn by
    // sequence, in kPrefix by row tiles (tile_base).
    const int32_t *groups, *prefix_lens;
    int num_groups, prefix_tile;           // prefix_tile: tokens of a step of the prefix's walk
    // Where the pieces of a sequence's own tokens, or of a span of a group's rows, stand,
    // for the join: {first slot, last range, group or -1, its first sequence} by sequence, {first
    // slot, last range} by span_index (kBlocks: by sequence and drafted token).  The
    // workgroups that begin and end them write it.
    int4* own_pieces;
    int2* span_pieces;
};

__device__ __forceinline__ int drafts_of(const TreeArgs& a, int b) {
    return a.draft_lens ? min(max(a.draft_lens[b], 0), a.drafts) : a.drafts;
}

// Tokens of a sequence that can be seen at all: its committed and drafted ones,
// as far as the table's row goes (none in an empty pool).  Positions of a tile
// stay below 2^31.
__device__ __forceinline__ int tokens_of(const TreeArgs& a, int len, int drafts) {
    const int64_t n = (int64_t)len + drafts;
    return a.num_pages ? (int)min(min(n, a.max_pages * a.page_size), (int64_t)0x7FFFFFC0) : 0;
}

// Its tiles; a sequence with drafted tokens has at least one, so that its rows are written.
__device__ __forceinline__ uint32_t tiles_of(int seen, int drafts) {
    return drafts ? max((seen + kTile - 1) / kTile, 1) : 0;
}

// A value equal in all lanes, as a scalar (so that what follows from it is one too).
__device__ __forceinline__ int64_t scalar(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

// A value of the lanes that the DPP control word names, 0 where they have none.
template <int kControl, int kRows>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kControl, kRows, 0xF, false);
}
template <int kControl, int kRows>
__device__ __forceinline__ uint64_t moved(uint64_t v) {
    return (uint64_t)moved<kControl, kRows>((uint32_t)(v >> 32)) << 32 | moved<kControl, kRows>((uint32_t)v);
}
// Sum of the values of a lane and those before it (a tenth of the time of exchanges
// through LDS): within rows of 16 lanes, then the last lane of rows 0 and 2 into rows 1
// and 3, then that of row 1 into rows 2 and 3.
template <class T>
__device__ __forceinline__ T sum_upto(T v) {
    v += moved<0x111, 0xF>(v), v += moved<0x112, 0xF>(v), v += moved<0x114, 0xF>(v), v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);
    return v + moved<0x143, 0xC>(v);
}

__device__ __forceinline__ int prefix_of(const TreeArgs& a, int g) { return max(a.prefix_lens[g], 0); }
// Tokens of a prefix that are attended once for all: whole tiles, as far as the table's
// row goes.
__device__ __forceinline__ int shared_of(const TreeArgs& a, int prefix) { return tokens_of(a, prefix, 0) & ~(kTile - 1); }
// Sequence number i of the bounds of the groups, within the batch.
__device__ __forceinline__ int bound_of(const TreeArgs& a, int i) { return min(max(a.groups[i], 0), a.batch); }
// The row tiles (of 16 rows) before a group's, in an order of all groups' rows.
__device__ __forceinline__ int64_t tile_base(const TreeArgs& a, int g) {
    return (int64_t)bound_of(a, g) * a.rows / 16 + g;
}
__device__ __forceinline__ int64_t tile_base_end(const TreeArgs& a) {
    return (int64_t)a.batch * a.rows / 16 + a.num_groups;
}
// Of each lane's sequence b (ascending by lane): its group (-1: none), the group's first
// sequence and prefix.  The bounds are read 64 at a time, with the prefixes beside them,
// and searched by lane exchange.
struct Member {
    int group, first, prefix;
};
__device__ __forceinline__ Member member_of(const TreeArgs& a, int b, int lane) {
    int n = 0, first = 0, next = 0, prefix = 0;           // n: bounds up to b
    for (int j = 0; j <= a.num_groups; j += 64) {
        const int v = j + lane <= a.num_groups ? bound_of(a, j + lane) : 0x7FFFFFFF;
        const int p = j + lane < a.num_groups ? prefix_of(a, j + lane) : 0;
        int at = 0;
#pragma unroll
        for (int m = 32; m; m /= 2) at += __shfl(v, at + m - 1, 64) <= b ? m : 0;
        at += at == 63 && __shfl(v, 63, 64) <= b ? 1 : 0;
        const int from = max(at - 1, 0), first_here = __shfl(v, from, 64), prefix_here = __shfl(p, from, 64);
        const int next_here = __shfl(v, min(at, 63), 64);
        if (at == 0 && n == j) next = next_here;          // the bound behind the last one of the 64 before
        if (at) n = j + at, first = first_here, prefix = prefix_here, next = next_here;
        if (__all(at < 64)) break;
    }
    return n > 0 && n <= a.num_groups && first <= b && b < next ? Member{n - 1, first, prefix} : Member{-1, 0, 0};
}

// 64 sequences of the batch (kPrefix: groups) from first on, one to a lane, with the
// tiles of those up to a lane's own (fewer than 2^32: a sequence has fewer than 2^26).
// kPrefix counts a group's tiles once for each span of its rows.
template <Mode kMode>
struct Chunk {
    using Count = std::conditional_t<kMode == kPrefix, uint64_t, uint32_t>;
    int first, len, seen, drafts;
    int skip;                          // kBlocks: pages left out before the last incomplete one; kOwn: first tile
    int token, tokens;                 // kPrefix: of the rows; kOwn: the group and its first sequence
    int per;                           // kPrefix: tiles of a span
    Count tiles, upto;
    __device__ __forceinline__ static Count read(Count v, int k) {
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)v, k);
        if constexpr (kMode != kPrefix) return lo;
        return (Count)__builtin_amdgcn_readlane((uint32_t)((uint64_t)v >> 32), k) << (kMode == kPrefix ? 32 : 0) | lo;
    }
    __device__ __forceinline__ Count all() const { return read(upto, 63); }
};
// plane: kBlocks' drafted token; span: kPrefix's rows of a workgroup.
template <Mode kMode>
__device__ __forceinline__ Chunk<kMode> chunk_at(const TreeArgs& a, int first, int lane, int plane, int span) {
    Chunk<kMode> c;
    c.first = first;
    if constexpr (kMode == kPrefix) {
        const bool there = first + lane < a.num_groups;
        const int g = there ? first + lane : 0;
        c.token = bound_of(a, g);
        const int members = max(bound_of(a, g + 1) - c.token, 0);
        c.token *= a.drafts, c.tokens = members * a.drafts;
        c.len = c.seen = shared_of(a, prefix_of(a, g)), c.drafts = 0;
        c.per = (c.seen + a.prefix_tile - 1) / a.prefix_tile;
        c.tiles = there ? (uint64_t)(((int64_t)members * a.rows + span - 1) / span) * (uint32_t)c.per : 0;
    } else {
        const int b = min(first + lane, a.batch - 1);
        c.len = max(a.seq_lens[b], 0);
        c.drafts = drafts_of(a, b);
        if constexpr (kMode == kBlocks) {
            // The listed blocks stand before the rest of the sequence, as if they were all there is.
            const int full = c.len / a.page_size, n = min(full, a.select);
            c.skip = full - n;
            c.len -= c.skip * a.page_size;
            c.seen = a.num_pages && a.max_pages ? (int)min((int64_t)c.len + c.drafts, (int64_t)0x7FFFFFC0) : 0;
            c.tiles = first + lane < a.batch && plane < c.drafts ? tiles_of(c.seen, c.drafts) : 0;
        } else {
            c.seen = tokens_of(a, c.len, c.drafts);
            c.tiles = first + lane < a.batch ? tiles_of(c.seen, c.drafts) : 0;
            if constexpr (kMode == kOwn) {
                const Member x = member_of(a, b, lane);
                // A shorter sequence has its own table's rows, also of the tiles that it has whole.
                c.skip = c.len >= x.prefix ? shared_of(a, x.prefix) / kTile : 0;
                c.token = c.skip ? x.group : -1, c.tokens = c.skip ? x.first : 0;
                if (c.tiles) c.tiles = max((int)c.tiles - c.skip, 1);
            }
        }
    }
    c.upto = sum_upto(c.tiles);
    return c;
}

// All tiles of the batch; c: its first chunk.  Every workgroup of both kernels walks
// the lengths so, 64 sequences a step, and the join has workgroups for each sequence:
// the cost grows with the batch's square.  Sequences of 100 tokens, 1 token each: 64 of
// them 16 us, 256 26, 512 60, 1024 162, 4096 1980 (116 us of bytes).
template <Mode kMode>
__device__ __forceinline__ int64_t all_tiles(const TreeArgs& a, const Chunk<kMode>& c, int lane, int plane, int span) {
    int64_t n = c.all();
    const int items = kMode == kPrefix ? a.num_groups : a.batch;
    for (int b = 64; b < items; b += 64) n += chunk_at<kMode>(a, b, lane, plane, span).all();
    return scalar(n);
}

// The tiles are cut into 2^shift ranges: range x has those from x * tiles >> shift on.
__device__ __forceinline__ int shift_of(const TreeArgs& a, int64_t tiles) {
    int shift = a.shift;
    while (shift > 0 && tiles < (int64_t)kMinTiles << shift) --shift;
    return shift;
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

// Byte kByte of w (two E2M1 codes) times 2^(scale byte - 127), exact, as two bf16.
template <int kByte>
__device__ __forceinline__ uint32_t widen(uint32_t w, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, kByte));
}
__device__ __forceinline__ u32x4 widen8(uint32_t w, float scale) {
    return u32x4{widen<0>(w, scale), widen<1>(w, scale), widen<2>(w, scale), widen<3>(w, scale)};
}
// sum + the products of two pairs of bf16, in fp32.
__device__ __forceinline__ float add_products(float sum, uint32_t a, uint32_t b) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), sum, false);
}
// A block's scale from the aligned word that holds its byte: rotated so that the
// byte stands in the exponent's bits; widen looks at no others.
__device__ __forceinline__ float scale_of(uint32_t word, uint32_t turn) {
    return __uint_as_float(__builtin_amdgcn_alignbit(word, word, turn));
}
// Whether a block of this scale may hold values that are infinite in bf16 or no
// numbers: 4 * 2^126 is.
__device__ __forceinline__ bool is_huge(float scale) { return (__float_as_uint(scale) << 1) >> 24 >= 253; }
constexpr uint32_t kOnes = 0x7F7F7F7Fu;    // scales of 1

template <int N>
using Int = std::integral_constant<int, N>;

// A tile's place: the first cache row of its two halves (-1: no page).
struct Place {
    int row[2];
};

// A workgroup's staging of a tile in LDS: HW neighbouring heads of 32 tokens, a
// region for each.  Rows are read from global memory in 16-byte chunks, neighbouring
// lanes in neighbouring chunks of the heads' part of a row, straight into LDS: the
// memory behind is bound by requests, and whole 128-byte lines make the fewest (a
// head's part of a row alone is half a line at D = 128).  Every region gets 1/HW of the
// rows, of all heads:
//   keys    32 rows of HW * D/32 chunks; chunk x of a row at x ^ key_turn(row), so
//           that the 16 lanes that read one chunk of 16 rows meet different banks
//   values  8 runs of 4 rows: run 4h + i has tokens 16h + 4g + i, g = 0 .. 3, which
//           the four lane groups read together; head x of a row at x ^ value_turn(g),
//           which brings their parts into different banks
//   scales  the aligned words with a token's scale bytes, one plane of 32 key and
//           32 value words for each word of a token
template <int D, int HW>
struct Stage {
    static constexpr int kChunks = D / 32, kRow = HW * kChunks;          // chunks of a head, of a row
    static constexpr int kKeys = 16 * D, kValues = 16 * D, kWords = D == 256 ? 2 : 1;   // bytes, planes of a wave
    static constexpr int kBytes = kKeys + kValues + kWords * 256;
    static constexpr int kPlanes = HW * D >= 128 ? HW * D / 128 : 1;
    static constexpr int kItems = kChunks / 2;                           // copies of keys, and of values, per region
    __device__ static constexpr int key_turn(int row) {
        return kRow < 16 ? (row * kRow / 16) & (kRow - 1) : row & (kRow - 1) & 15;
    }
    __device__ static constexpr int value_turn(int g) { return HW >= 4 ? g : (g * HW) >> 2; }
};
constexpr int kStages = 3;                 // two tiles in flight behind the one in use

// Until at most kLeft of the wave's copies are outstanding.
template <int kLeft>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft) : "memory");
}
// LDS reads issued so far have returned, in all waves of the workgroup.
template <int kWaves>
__device__ __forceinline__ void meet() {
    if (kWaves > 1)
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// A lane's part in the copies and in the reads.
template <int D, int HW>
struct Lane {
    static constexpr int kItems = Stage<D, HW>::kItems;
    uint32_t key[kItems], value[kItems];                  // offsets of its chunks from 16 rows' first head
    const uint8_t* scale;                                 // its token's scale word, in row 0
    uint32_t read_key, read_value, read_ks, read_vs;      // LDS offsets
    uint32_t kturn, vturn[4];                             // turns that bring a scale byte into place
};
template <int D, int HW>
__device__ __forceinline__ Lane<D, HW> lane_of(const TreeArgs& a, int head0, int wave, int lane) {
    using S = Stage<D, HW>;
    constexpr int kRegion = kStages * S::kBytes, kShare = D / 32;        // a lane's bytes of a value row
    const int c = lane & 15, g = lane >> 4, first = head0 * (D / 32);
    Lane<D, HW> o;
#pragma unroll
    for (int k = 0; k < S::kItems; ++k) {
        const int slot = (wave * S::kItems + k) * 64 + lane, row = slot / S::kRow, at = slot % S::kRow;
        o.key[k] = row % 16 * a.code_row + head0 * (D / 2) + (at ^ S::key_turn(row % 16)) * 16;
        const int vg = row % 4, token = 4 * vg + row / 4 % 4;            // row: run * 4 + g
        o.value[k] = token * a.code_row + (head0 + (at / S::kChunks ^ S::value_turn(vg))) * (D / 2) + at % S::kChunks * 16;
    }
    const int row0 = c * a.scale_row + first;                            // of its token's scale bytes
    const int plane = wave * S::kWords % S::kPlanes;
    o.scale = (lane < 32 ? a.ks : a.vs) + (row0 & ~3) + 4 * plane;
    {
        const int at = (wave * S::kChunks + (D == 64 ? g / 2 : D == 128 ? g : 2 * g)) ^ S::key_turn(c);
        o.read_key = c / (32 / HW) * kRegion + (c % (32 / HW) * S::kRow + at) * 16 + (D == 64 ? g % 2 * 8 : 0);
    }
    o.read_value = S::kKeys + (g * S::kRow + (wave ^ S::value_turn(g)) * S::kChunks) * 16 + c * kShare;
    const int kblock = wave * (D / 32) + (D == 64 ? g / 2 : D == 128 ? g : 2 * g);
    const int vblock = wave * (D / 32) + c * (D / 16) / 32;
    auto plane_of = [&](int block) {                      // LDS offset of the plane with a head's scale block
        const int p = ((first & 3) + block) / 4;
        return p / S::kWords * kRegion + S::kKeys + S::kValues + p % S::kWords * 256;
    };
    // Words start at the row's aligned word; only D = 64 with an odd number of heads
    // has rows that do not start with one.
    o.read_ks = (D == 64 && HW == 1 ? S::kKeys + S::kValues : plane_of(kblock)) + c * 4;
    o.read_vs = (D == 64 && HW == 1 ? S::kKeys + S::kValues : plane_of(vblock)) + 128 + 4 * g * 4;
    o.kturn = (8 * ((row0 + kblock) & 3) + 9) & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o.vturn[j] = D == 64 && HW == 1 ? (8 * (((4 * g + j) * a.scale_row + first + vblock) & 3) + 9) & 31
                                        : (8 * ((first + vblock) & 3) + 9) & 31;
    return o;
}

// Starts a wave's copies of a tile into its head's region of the stage at lds (global
// memory to LDS, lane l's 16 or 4 bytes to M0 + offset + l * size); awaited by
// wait_copies: everything with RG = 1; with two waves to a head the first one's keys
// and scales, the second one's values.  Halves without a page read row 0 on (a row of
// the pool; hidden later).  Copies are one asm block behind one write of M0 (which
// needs a wait state); the instruction's offset, -4096 to 4095, counts on the global
// side as well, so each address is given less it.
template <int D, int HW, int RG>
__device__ __forceinline__ void copy_tile(const TreeArgs& a, const Place& p, const Lane<D, HW>& o, int hw, int rg, int lane,
                                          uint32_t lds) {
    const int row0 = max(p.row[0], 0), row1 = max(p.row[1], 0), mine = HW > 1 && hw < HW / 2 ? row0 : row1;
    const uint8_t* scale = o.scale + (uint64_t)(uint32_t)(lane & 16 ? row1 : row0) * (uint32_t)a.scale_row;
    if constexpr (D == 64) {                              // HW = 1: both halves in one instruction
        const uint64_t at = (uint64_t)(uint32_t)(HW == 1 && !(lane & 32) ? row0 : mine) * (uint32_t)a.code_row;
        const uint8_t *key = a.kc + at + o.key[0], *value = a.vc + at + o.value[0];
        if (RG == 1)
            asm volatile(
                "s_mov_b32 m0, %3\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, off\n\t"
                "global_load_lds_dwordx4 %1, off offset:1024\n\t"
                "global_load_lds_dword %2, off offset:2048" ::"v"(key),
                "v"(value - 1024), "v"(scale - 2048), "s"(lds)
                : "memory", "m0");
        else if (rg == 0)
            asm volatile(
                "s_mov_b32 m0, %2\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, off\n\t"
                "global_load_lds_dword %1, off offset:2048" ::"v"(key),
                "v"(scale - 2048), "s"(lds)
                : "memory", "m0");
        else
            asm volatile(
                "s_mov_b32 m0, %1\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, off offset:1024" ::"v"(value - 1024),
                "s"(lds)
                : "memory", "m0");
    } else {
        // HW = 1: the first half of the copies takes the tile's first half.
        const int64_t at0 = (int64_t)(HW == 1 ? row0 : mine) * a.code_row, at1 = HW == 1 ? (int64_t)row1 * a.code_row : at0;
        if constexpr (D == 128) {
            if (RG == 1)
                asm volatile(
                    "s_mov_b32 m0, %9\n\ts_nop 0\n\t"
                    "global_load_lds_dwordx4 %0, %4 offset:-1024\n\t"
                    "global_load_lds_dwordx4 %1, %5\n\t"
                    "global_load_lds_dwordx4 %2, %6 offset:1024\n\t"
                    "global_load_lds_dwordx4 %3, %7 offset:2048\n\t"
                    "global_load_lds_dword %8, off offset:3*1024" ::"v"(o.key[0]),
                    "v"(o.key[1]), "v"(o.value[0]), "v"(o.value[1]), "s"(a.kc + at0 + 1024), "s"(a.kc + at1),
                    "s"(a.vc + at0 - 1024), "s"(a.vc + at1 - 2048), "v"(scale - 3 * 1024), "s"(lds + 1024)
                    : "memory", "m0");
            else if (rg == 0)
                asm volatile(
                    "s_mov_b32 m0, %5\n\ts_nop 0\n\t"
                    "global_load_lds_dwordx4 %0, %2 offset:-1024\n\t"
                    "global_load_lds_dwordx4 %1, %3\n\t"
                    "global_load_lds_dword %4, off offset:3*1024" ::"v"(o.key[0]),
                    "v"(o.key[1]), "s"(a.kc + at0 + 1024), "s"(a.kc + at1), "v"(scale - 3 * 1024), "s"(lds + 1024)
                    : "memory", "m0");
            else
                asm volatile(
                    "s_mov_b32 m0, %4\n\ts_nop 0\n\t"
                    "global_load_lds_dwordx4 %0, %2 offset:1024\n\t"
                    "global_load_lds_dwordx4 %1, %3 offset:2048" ::"v"(o.value[0]),
                    "v"(o.value[1]), "s"(a.vc + at0 - 1024), "s"(a.vc + at1 - 2048), "s"(lds + 1024)
                    : "memory", "m0");
        } else {
            static_assert(D != 256 || RG == 1);
            asm volatile(
                "s_mov_b32 m0, %8\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, %4\n\t"
                "global_load_lds_dwordx4 %1, %5 offset:1024\n\t"
                "global_load_lds_dwordx4 %2, %6 offset:2048\n\t"
                "global_load_lds_dwordx4 %3, %7 offset:3*1024" ::"v"(o.key[0]),
                "v"(o.key[1]), "v"(o.key[2]), "v"(o.key[3]), "s"(a.kc + at0), "s"(a.kc + at0 - 1024),
                "s"(a.kc + at1 - 2048), "s"(a.kc + at1 - 3 * 1024), "s"(lds)
                : "memory", "m0");
            asm volatile(
                "s_mov_b32 m0, %10\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, %4 offset:-4096\n\t"
                "global_load_lds_dwordx4 %1, %5 offset:-3*1024\n\t"
                "global_load_lds_dwordx4 %2, %6 offset:-2048\n\t"
                "global_load_lds_dwordx4 %3, %7 offset:-1024\n\t"
                "global_load_lds_dword %8, off\n\t"
                "global_load_lds_dword %9, off offset:256" ::"v"(o.value[0]),
                "v"(o.value[1]), "v"(o.value[2]), "v"(o.value[3]), "s"(a.vc + at0 + 4096), "s"(a.vc + at0 + 3 * 1024),
                "s"(a.vc + at1 + 2048), "s"(a.vc + at1 + 1024), "v"(scale), "v"(scale + 4 - 256), "s"(lds + 8192)
                : "memory", "m0");
        }
    }
}

// Low (or high) halves of a and b: two tokens of one value.
template <bool kHigh>
__device__ __forceinline__ uint32_t pair(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, kHigh ? 0x07060302u : 0x05040100u);
}

// Where the sums of 16 rows of a piece stand, in tiles of 16 rows from a.part on, and
// how many tiles there are: the rows' (m, sum) stand behind them.
struct PartPlace {
    int64_t tile, stats;
};
// whole: a piece that no range cuts (kOwn; those of the others are written out).
template <Mode kMode>
__device__ __forceinline__ PartPlace part_place(const TreeArgs& a, bool whole, int64_t slot, int b, int plane, int row_tile,
                                                int head) {
    const int planes = kMode == kBlocks ? a.drafts : 1;
    const int64_t ranges = 2 * (int64_t)a.ranges, at = kMode == kOwn && whole ? ranges + b : slot;
    return {((at * a.kv_heads + head) * planes + plane) * a.row_tiles + row_tile,
            (ranges + (kMode == kOwn ? a.batch : 0)) * a.kv_heads * planes * a.row_tiles};
}
// The tile with row `row` (a multiple of 16) of a group whose tiles begin at tile0; a
// piece of a range has those of its span.
__device__ __forceinline__ PartPlace prefix_place(const TreeArgs& a, bool whole, int64_t slot, int64_t tile0, int64_t row,
                                                  int span, int head) {
    const int64_t ranges = 2 * (int64_t)a.ranges * (span / 16);
    const int64_t at = whole ? ranges + tile0 + row / 16 : slot * (span / 16) + row % span / 16;
    return {at * a.kv_heads + head, (ranges + tile_base_end(a)) * a.kv_heads};
}

// Place of a span of a group's rows in span_pieces (row: any of it).
__device__ __forceinline__ int64_t span_index(const TreeArgs& a, int group, int first_sequence, int64_t row, int span) {
    return (int64_t)first_sequence * a.rows / span + group + row / span;
}
// item: a sequence or a group; token, tokens: as its chunk has them (kBlocks: the drafted
// token); row: of the span.
template <Mode kMode>
__device__ __forceinline__ void note_piece(const TreeArgs& a, int slot, bool begins, bool ends, int item, int token, int tokens,
                                           int64_t row, int span) {
    if constexpr (kMode == kBlocks) {
        int2* to = a.span_pieces + ((int64_t)item * a.drafts + token);
        if (begins) to->x = slot;
        if (ends) to->y = slot >> 1;
    } else if constexpr (kMode == kOwn) {
        int4* to = a.own_pieces + item;
        if (begins) to->x = slot, to->z = token, to->w = tokens;
        if (ends) to->y = slot >> 1;
    } else {
        int2* to = a.span_pieces + span_index(a, item, token / a.drafts, row, span);
        if (begins) to->x = slot;
        if (ends) to->y = slot >> 1;
    }
}

// LDS of a workgroup's walk.
template <int D, int HW>
constexpr int kStaging = HW * kStages * Stage<D, HW>::kBytes;

// A workgroup's tiles, and the first 64 sequences (groups).
template <Mode kMode>
struct Range {
    Chunk<kMode> chunk;
    int64_t lo, hi;
};

// The walk of workgroup (block_x, block_y): column block_y, range block_x (range_at(plane,
// span) gives it).
template <Mode kMode, int D, int NR, int HW, int RG, class RangeAt>
__device__ __forceinline__ void walk(const TreeArgs& a, uint8_t* staging, int block_x, int block_y, RangeAt range_at) {
    constexpr int kSteps = D / 32, kOut = D / 16;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    using S = Stage<D, HW>;
    constexpr int kRegion = kStages * S::kBytes;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), groups = a.kv_heads / HW;
    const int hw = wave % HW, rg = RG == 1 ? 0 : wave / HW;
    const int head0 = __builtin_amdgcn_readfirstlane(block_y % groups) * HW, head = head0 + hw;
    constexpr int kSpan = 16 * NR * RG;                       // rows of a workgroup
    const int column = __builtin_amdgcn_readfirstlane(block_y / groups), spans = (a.rows + kSpan - 1) / kSpan;
    const int plane = kMode == kBlocks ? column / spans : 0;
    int r0 = ((kMode == kBlocks ? column - plane * spans : column) * RG + rg) * 16 * NR;
    const uint32_t lds = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_bytes)staging) + hw * kRegion;
    const Lane<D, HW> own = lane_of<D, HW>(a, head0, hw, lane);
    const Range<kMode> range = range_at(plane, kSpan);
    const int64_t lo = range.lo, hi = range.hi;
    if (lo == hi) return;
    Chunk<kMode> chunk = range.chunk;

    // The sequence that holds tile lo, and the tiles before it.
    int64_t before = 0;
    while (before + chunk.all() <= lo) {
        before += chunk.all();
        chunk = chunk_at<kMode>(a, chunk.first + 64, lane, plane, kSpan);
    }
    int b = chunk.first;
    {
        const int k = __popcll(__ballot((int64_t)(before + chunk.upto) <= lo));       // those that end by lo
        if (k) before += chunk.read(chunk.upto, k - 1);
        b += k;
    }

    for (int64_t at = lo; at < hi;) {
        if (b - chunk.first == 64) chunk = chunk_at<kMode>(a, b, lane, plane, kSpan);
        const int at_lane = b - chunk.first;
        const int64_t cells = chunk.read(chunk.tiles, at_lane);
        if (cells == 0) {
            ++b;
            continue;
        }
        int tiles = (int)cells, t0 = (int)(at - before);
        int64_t tile0 = 0;                                    // kPrefix: the row tiles before this span's
        if constexpr (kMode == kPrefix) {
            tiles = __builtin_amdgcn_readlane(chunk.per, at_lane);
            const int64_t span = (at - before) / tiles;
            t0 = (int)(at - before - span * tiles);
            r0 = (int)(span * RG + rg) * 16 * NR;
            tile0 = tile_base(a, b);
        }
        const int t1 = (int)min(hi - at + t0, (int64_t)tiles);
        const int len = __builtin_amdgcn_readlane(chunk.len, at_lane);
        const int seen = __builtin_amdgcn_readlane(chunk.seen, at_lane);
        const int nd = __builtin_amdgcn_readlane(chunk.drafts, at_lane);
        // kOwn: tile t of the piece is tile skip + t of the sequence.
        const int skip = kMode == kBlocks || kMode == kOwn ? __builtin_amdgcn_readlane(chunk.skip, at_lane) : 0;
        const int s0 = kMode == kOwn ? t0 + skip : t0, s1 = kMode == kOwn ? t1 + skip : t1;
        // kPrefix: all of a group see its first sequence's rows.
        const int row_token = kMode == kPrefix ? __builtin_amdgcn_readlane(chunk.token, at_lane) : b * a.drafts;
        const int row_tokens = kMode == kPrefix ? __builtin_amdgcn_readlane(chunk.tokens, at_lane) : nd;
        const int32_t* table = a.table + (int64_t)(kMode == kPrefix ? row_token / a.drafts : b) * a.max_pages;
        const int32_t* list = nullptr;
        if constexpr (kMode == kBlocks)
            list = a.ids + (((int64_t)b * a.drafts + plane) * a.lists + (a.lists > 1 ? head : 0)) * a.select;
        // Row r of the piece: its token behind row_token, its head in the group.
        auto token_of = [&](int r) { return kMode == kBlocks ? plane : r / a.group; };
        auto head_of = [&](int r) { return kMode == kBlocks ? r : r % a.group; };
        auto is_live = [&](int r) { return kMode == kBlocks ? r < a.group : r / a.group < row_tokens; };

        u32x4 q[NR][kSteps];
        uint64_t vis[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int row = r0 + 16 * n + c, t = token_of(row);
            const bool live = is_live(row);
            const uint16_t* x = a.q + ((int64_t)row_token + (live ? t : 0)) * a.ld_q +
                                ((int64_t)head * a.group + (live ? head_of(row) : 0)) * D + g * (D / 4);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                q[n][s] = live ? *reinterpret_cast<const u32x4*>(x + 8 * s) ^ a.flip : u32x4{0, 0, 0, 0};
            vis[n] = 0;
            if (kMode != kPrefix && live) {
                vis[n] = a.mask ? a.mask[(int64_t)b * a.drafts + t] : ~0ull >> (63 - t);
                if (nd < 64) vis[n] &= (1ull << nd) - 1;
            }
        }

        v4f o[NR][kOut];
        float m[NR];
        v4f sum[NR];                                          // of the rounded weights, all four alike
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            m[n] = kFloor, sum[n] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kOut; ++i) o[n][i] = v4f{0.f, 0.f, 0.f, 0.f};
        }

        // The lanes hold the cache rows of the next 64 halves of tiles (-1: no page),
        // worked out together once in 32 tiles and read by lane when their turn comes.
        int half_i = 2 * s0, first_half = half_i - 64, rows = 0;
        auto place = [&]() {
            if (half_i >= first_half + 64) {
                first_half = half_i;
                const int at = half_i + lane, per = a.page_size / 16, i = at / per;
                int at_page = i;
                if constexpr (kMode == kBlocks) {
                    const int complete = len / a.page_size + skip, n = complete - skip;
                    const int id = n ? list[min(i, n - 1)] : 0;
                    at_page = i >= n ? i + skip : (uint32_t)id < (uint32_t)complete ? id : (int)a.max_pages;
                }
                const int page = table[min(at_page, (int)a.max_pages - 1)];
                const bool there = at_page < a.max_pages && (uint32_t)page < (uint32_t)a.num_pages;
                rows = there ? page * a.page_size + (at - i * per) * 16 : -1;
            }
            Place p;
            p.row[0] = __builtin_amdgcn_readlane(rows, half_i - first_half);
            p.row[1] = __builtin_amdgcn_readlane(rows, half_i - first_half + 1);
            half_i += 2;
            return p;
        };
        bool any_apart = false;
        const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
        auto compute = [&](int t, const Place& here, uint32_t stage) {
            const uint8_t* mine = staging + stage;
            uint32_t kw[2][D / 32], kscale[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // Rows 16 on: HW/2 regions further, or in the only one.
                constexpr int kHalf = HW == 1 ? 16 * S::kRow * 16 : HW / 2 * kRegion;
                if constexpr (D == 64) {
                    const u32x2 x = *reinterpret_cast<const u32x2*>(mine + own.read_key + h * kHalf);
                    kw[h][0] = x[0], kw[h][1] = x[1];
                } else {
#pragma unroll
                    for (int i = 0; i < D / 128; ++i) {       // chunk 2g + 1 lies beside 2g
                        const u32x4 x = *reinterpret_cast<const u32x4*>(mine + (own.read_key ^ (16 * i)) + h * kHalf);
#pragma unroll
                        for (int w = 0; w < 4; ++w) kw[h][4 * i + w] = x[w];
                    }
                }
                kscale[h] = *reinterpret_cast<const uint32_t*>(mine + own.read_ks + 64 * h);
            }
            const int pos0 = t * kTile;
            const bool edge = pos0 + kTile > len || here.row[0] < 0 || here.row[1] < 0;     // some token is hidden
            v4f s[NR][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int n = 0; n < NR; ++n) s[n][h] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const float sc = scale_of(kscale[h], own.kturn + (D == 256 ? 8 * (i / 4) : 0));
                    const bf16x8 k = __builtin_bit_cast(bf16x8, widen8(kw[h][i], sc));
#pragma unroll
                    for (int n = 0; n < NR; ++n)
                        s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, __builtin_bit_cast(bf16x8, q[n][i]), s[n][h],
                                                                          0, 0, 0);
                }
            }
            u32x4 vscale[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) vscale[h] = *reinterpret_cast<const u32x4*>(mine + own.read_vs + 64 * h);
            if (edge) {
                bool apart = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int pos = pos0 + 16 * (j / 4) + 4 * g + j % 4, d = pos - len;
                    const bool there = (pos < seen) & (here.row[j / 4] >= 0);
                    // Whatever lies there, finite; blocks that may not be are added apart (2^-127 of them here).
                    const bool huge = there & (d >= 0) & is_huge(scale_of(vscale[j / 4][j % 4], own.vturn[j % 4]));
                    apart |= huge;
                    vscale[j / 4][j % 4] = huge ? 0u : there ? vscale[j / 4][j % 4] : kOnes;
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const bool see = there & ((d < 0) | ((uint32_t)(vis[n] >> (d & 63)) & 1u));
                        s[n][j / 4][j % 4] = see ? s[n][j / 4][j % 4] : kNone;
                    }
                }
                any_apart |= __any(apart);
            }
            float top[NR];
            bool rises = false;
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                top[n] = s[n][0][0];
#pragma unroll
                for (int j = 1; j < 8; ++j) top[n] = fmaxf(top[n], s[n][j / 4][j % 4]);
                rises |= top[n] * a.scale2 > m[n] + kSlack;
            }
            if (__any(rises)) {
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    float x = top[n] * a.scale2;
                    x = fmaxf(x, __shfl_xor(x, 16, 64));
                    x = fmaxf(x, __shfl_xor(x, 32, 64));
                    // kPrefix: the others' rows are those of other sequences, or nobody's; a row
                    // moves when its own scores rise, so that its bits are its own.
                    const float up = kMode == kPrefix && !(x > m[n] + kSlack) ? m[n] : fmaxf(m[n], x), alpha = exp2_hw(m[n] - up);
                    m[n] = up;
                    sum[n] *= alpha;
#pragma unroll
                    for (int i = 0; i < kOut; ++i) o[n][i] *= alpha;
                }
            }
            bf16x8 p[NR];
#pragma unroll
            for (int n = 0; n < NR; ++n) {
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = pack2(exp2_hw(fmaf(s[n][j / 2][2 * j % 4], a.scale2, -m[n])),
                                 exp2_hw(fmaf(s[n][j / 2][2 * j % 4 + 1], a.scale2, -m[n])));
                p[n] = __builtin_bit_cast(bf16x8, w);
                sum[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, p[n], sum[n], 0, 0, 0);
            }
            // V, a byte (two values) of the lane's 8 tokens at a time: widened, then
            // tokens paired per value.
            float scale[8];
            uint32_t vw[8][D == 256 ? 2 : 1];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                scale[j] = scale_of(vscale[j / 4][j % 4], own.vturn[j % 4]);
                const uint8_t* x = mine + own.read_value + j * HW / 8 * kRegion + j % (8 / HW) * 64 * S::kRow;
                if constexpr (D == 64) {
                    vw[j][0] = *reinterpret_cast<const uint16_t*>(x);
                } else if constexpr (D == 128) {
                    vw[j][0] = *reinterpret_cast<const uint32_t*>(x);
                } else {
                    const u32x2 y = *reinterpret_cast<const u32x2*>(x);
                    vw[j][0] = y[0], vw[j][1] = y[1];
                }
            }
            auto values = [&](auto byte_tag) {
                constexpr int kB = decltype(byte_tag)::value;
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = widen<kB % 4>(vw[j][kB / 4], scale[j]);
                const u32x4 lo = {pair<false>(w[0], w[1]), pair<false>(w[2], w[3]), pair<false>(w[4], w[5]), pair<false>(w[6], w[7])};
                const u32x4 hi = {pair<true>(w[0], w[1]), pair<true>(w[2], w[3]), pair<true>(w[4], w[5]), pair<true>(w[6], w[7])};
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    o[n][2 * kB] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, lo), p[n], o[n][2 * kB], 0, 0, 0);
                    o[n][2 * kB + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, hi), p[n], o[n][2 * kB + 1], 0, 0, 0);
                }
            };
            values(Int<0>()), values(Int<1>());
            if constexpr (D >= 128) values(Int<2>()), values(Int<3>());
            if constexpr (D == 256) values(Int<4>()), values(Int<5>()), values(Int<6>()), values(Int<7>());
        };
        if (seen > 0) {
            // Three stages and the places of their tiles take turns, by unrolling.  When
            // the waves meet, a tile's copies have landed in all regions, and the stage
            // of the tile before is free for the one after next.
            Place at_stage[kStages];
            auto start = [&](int k) {
                at_stage[k] = place();
                copy_tile<D, HW, RG>(a, at_stage[k], own, hw, rg, lane, lds + k * S::kBytes);
            };
            auto turn = [&](int t, auto tag) {
                constexpr int k = decltype(tag)::value;
                if (t + 1 >= s1)
                    wait_copies<0>();
                else if (RG == 1)
                    wait_copies<2 * S::kItems + S::kWords>();
                else if (rg == 0)
                    wait_copies<S::kItems + S::kWords>();
                else
                    wait_copies<S::kItems>();
                meet<HW * RG>();
                if (t + 2 < s1) start((k + 2) % kStages);
                compute(t, at_stage[k], k * S::kBytes);
            };
            start(0);
            if (s0 + 1 < s1) start(1);
            for (int t = s0; t < s1; t += 3) {
                turn(t, Int<0>());
                if (t + 1 < s1) turn(t + 1, Int<1>());
                if (t + 2 < s1) turn(t + 2, Int<2>());
            }
            meet<HW * RG>();                                  // before the next sequence's copies
        }
        // A weight of 0 does not hide an infinite value, so the drafted tokens' blocks
        // with such values are left out above and added here, to the rows that see them.
        if (kMode != kPrefix && any_apart) {
            constexpr int kScales = D == 256 ? 2 : 1;              // blocks that a lane's D/4 values lie in
            const int at_code = head * (D / 2) + g * (D / 8), at_scale = head * (D / 32) + (D == 64 ? g / 2 : kScales * g);
#pragma unroll 1
            for (int pos = max(s0 * kTile, len); pos < min(s1 * kTile, seen); ++pos) {
                const int at_page = pos / a.page_size + (kMode == kBlocks ? skip : 0), d = pos - len;
                if (kMode == kBlocks && at_page >= a.max_pages) break;
                const int page = table[at_page];
                if ((uint32_t)page >= (uint32_t)a.num_pages) continue;
                const int64_t cache_row = (int64_t)page * a.page_size + pos % a.page_size;
                const uint8_t* ks = a.ks + cache_row * a.scale_row + at_scale;
                const uint8_t* vs = a.vs + cache_row * a.scale_row + at_scale;
                const uint32_t* kc = reinterpret_cast<const uint32_t*>(a.kc + cache_row * a.code_row + at_code);
                const uint32_t* vc = reinterpret_cast<const uint32_t*>(a.vc + cache_row * a.code_row + at_code);
                float x[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n) x[n] = 0.f;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const u32x4 k = widen8(kc[i], __uint_as_float((uint32_t)ks[i / 4] << 23));
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            x[n] = add_products(x[n], k[j], q[n][i][j]);
                }
#pragma unroll
                for (int n = 0; n < NR; ++n) {
                    x[n] += __shfl_xor(x[n], 16, 64);
                    x[n] += __shfl_xor(x[n], 32, 64);
                    x[n] = bf16_lo(pack2(exp2_hw(fmaf(x[n], a.scale2, -m[n])), 0.f));
                }
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    const float scale = __uint_as_float((uint32_t)vs[i / 4] << 23);
                    const u32x4 v = widen8(vc[i], scale);
#pragma unroll
                    for (int n = 0; n < NR; ++n)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int at_o = (8 * i + j) % kOut, e = (8 * i + j) / kOut;
                            if (is_huge(scale) && (vis[n] >> (d & 63)) & 1)
                                o[n][at_o][e] = fmaf(x[n], j & 1 ? bf16_hi(v[j / 2]) : bf16_lo(v[j / 2]), o[n][at_o][e]);
                        }
                }
            }
        }

        const bool whole = t0 == 0 && t1 == tiles;
        const bool done = whole && (kMode == kTree || kMode == kBlocks || (kMode == kOwn && skip == 0));
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float l = sum[n][0];
            const int row = r0 + 16 * n + c;
            if (done) {
                if (!is_live(row)) continue;
                const float inv = l > 0.f ? 1.0f / l : 0.f;
                uint16_t* y = a.out + ((int64_t)row_token + token_of(row)) * a.ld_out +
                              ((int64_t)head * a.group + head_of(row)) * D + g * (D / 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {                 // D/16 consecutive values each
                    uint32_t w[kOut / 2];
#pragma unroll
                    for (int j = 0; j < kOut / 2; ++j) w[j] = pack2(o[n][2 * j][i] * inv, o[n][2 * j + 1][i] * inv);
#pragma unroll
                    for (int j = 0; j < kOut / 2; j += 2)
                        *reinterpret_cast<uint2*>(y + i * kOut + 2 * j) = make_uint2(w[j], w[j + 1]);
                }
            } else if (r0 + 16 * n < (kMode == kPrefix ? row_tokens * a.group : a.rows)) {
                const int64_t slot = 2 * (int64_t)block_x + (at == lo ? 0 : 1);
                const PartPlace p = kMode == kPrefix ? prefix_place(a, whole, slot, tile0, r0 + 16 * n, kSpan, head)
                                                     : part_place<kMode>(a, whole, slot, b, plane, (r0 >> 4) + n, head);
                v4f* y = reinterpret_cast<v4f*>(a.part) + p.tile * (4 * D) + lane;
#pragma unroll
                for (int i = 0; i < kOut; ++i) y[64 * i] = o[n][i];
                float2* ml = reinterpret_cast<float2*>(a.part + p.stats * (16 * D));
                if (g == 0) ml[p.tile * 16 + c] = make_float2(m[n], l);
            }
        }
        if constexpr (kMode == kBlocks) {
            if (block_y == plane * spans * groups && threadIdx.x == 0)
                note_piece<kMode>(a, 2 * block_x + (at == lo ? 0 : 1), t0 == 0, t1 == tiles, b, plane, 0, 0, kSpan);
        } else if constexpr (kMode == kOwn || kMode == kPrefix) {
            if (block_y == 0 && threadIdx.x == 0)
                note_piece<kMode>(a, 2 * block_x + (at == lo ? 0 : 1), t0 == 0, t1 == tiles, b,
                                  __builtin_amdgcn_readlane(chunk.token, at_lane), __builtin_amdgcn_readlane(chunk.tokens, at_lane), r0,
                                  kSpan);
        }
        at += t1 - t0;
        if (at - before == cells) before += cells, ++b;
    }
}

template <Mode kMode, int D, int NR, int HW, int RG>
__global__ __launch_bounds__(64 * HW * RG, D == 256 ? 1 : 2) void attn_walk_kernel(const TreeArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t staging[kStaging<D, HW>];
    walk<kMode, D, NR, HW, RG>(a, staging, blockIdx.x, blockIdx.y, [&](int plane, int span) {
        const int lane = threadIdx.x & 63;
        Range<kMode> r{chunk_at<kMode>(a, 0, lane, plane, span), 0, 0};
        const int64_t total = all_tiles<kMode>(a, r.chunk, lane, plane, span);
        const int shift = shift_of(a, total);
        if (blockIdx.x >> shift == 0) r.lo = blockIdx.x * total >> shift, r.hi = (blockIdx.x + 1) * total >> shift;
        return r;
    });
}

// A wave's part in joining partial results of 16 rows of one head: of their values slice
// i (the values i, i + D/16, ...), lane (c, g) those of row c in quarter g, 16 bytes as
// they were written.  kTeams teams take the pieces in turn; team order is the sum's.
template <int D, int kTeams>
struct Joined {
    float m = kFloor, l = 0.f;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    // Adds the pieces first .. last (most: last - first, the largest of the wave's lanes);
    // place(x): the tile of piece x, row: the lane's in it, stats_at: as PartPlace has it.
    template <class Place>
    __device__ __forceinline__ void add(const float* parts, int64_t stats_at, int team, int i, int g, int first, int last, int most,
                                        int row, Place place) {
        constexpr int kBatch = 8;
        const v4f* o = reinterpret_cast<const v4f*>(parts) + 64 * i + 16 * g + row;
        const float2* ml = reinterpret_cast<const float2*>(parts + stats_at * (16 * D)) + row;
#pragma unroll 1
        for (int x0 = first + team; x0 - first <= most; x0 += kBatch * kTeams) {
            float2 s[kBatch];
            v4f v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int x = x0 + k * kTeams;
                s[k] = make_float2(kFloor, 0.f);
                v[k] = v4f{0.f, 0.f, 0.f, 0.f};
                if (x <= last) {
                    const int64_t at = place(x);
                    s[k] = ml[at * 16];
                    v[k] = o[at * (4 * D)];
                }
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) top = fmaxf(top, s[k].x);
            const float keep = exp2_hw(m - top);
            m = top;
            l *= keep;
            acc *= keep;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float e = exp2_hw(s[k].x - top);
                l += s[k].y * e;
                acc += v[k] * e;
            }
        }
    }
};
// The teams' sums through LDS, and the rows r0 .. rows written where out_at(row) says; a
// team has kPer waves, wave part / 64 of it slice i.
template <int D, int kPer, int kTeams, class Out>
__device__ __forceinline__ void finish_join(Joined<D, kTeams>& j, int team, int part, int i, int lane, int r0, int rows, Out out_at) {
    constexpr int kTeam = 64 * kPer, kOut = D / 16;
    const int c = lane & 15, g = lane >> 4;
    __shared__ v4f sums[kTeams > 1 ? kTeam * kTeams : 1];
    __shared__ float2 stats[kTeams][16];
    if constexpr (kTeams > 1) {
        sums[threadIdx.x] = j.acc;
        if (part < 16) stats[team][part] = make_float2(j.m, j.l);
        __syncthreads();
        if (team == 0) {
            float top = kFloor;
#pragma unroll
            for (int k = 0; k < kTeams; ++k) top = fmaxf(top, stats[k][c].x);
            j.l = 0.f;
            j.acc = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kTeams; ++k) {
                const float e = exp2_hw(stats[k][c].x - top);
                j.l += stats[k][c].y * e;
                j.acc += sums[part + k * kTeam] * e;
            }
        }
    }
    const float inv = j.l > 0.f ? 1.0f / j.l : 0.f;
    if constexpr (kPer == kOut) {                             // whole rows go out through LDS in 16-byte parts
        __shared__ __attribute__((aligned(16))) uint16_t out_rows[16][D + 8];
#pragma unroll
        for (int k = 0; k < 4; ++k) out_rows[c][g * (D / 4) + k * kOut + i] = (uint16_t)pack2(j.acc[k] * inv, 0.f);
        __syncthreads();
        const int chunks = D / 8, r = threadIdx.x / chunks, at = threadIdx.x % chunks * 8;
        if (r < 16 && r0 + r < rows)
            *reinterpret_cast<uint4*>(out_at(r0 + r) + at) = *reinterpret_cast<const uint4*>(&out_rows[r][at]);
    } else if (team == 0 && r0 + c < rows) {
        uint16_t* y = out_at(r0 + c) + g * (D / 4) + i;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k * kOut] = (uint16_t)pack2(j.acc[k] * inv, 0.f);
    }
}

// Joins the partial results of the sequences that were cut: workgroup (x, y) takes
// 16 rows of a head (x; kBlocks: of a head's drafted token) of sequence y, and of their
// values the kPer slices from kPer * z on.
template <Mode kMode, int D, int kPer, int kTeams>
__global__ __launch_bounds__(64 * kPer * kTeams) void attn_join_kernel(const TreeArgs a) {
    constexpr int kTeam = 64 * kPer;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int b = blockIdx.y, row_tile = blockIdx.x % a.row_tiles, r0 = row_tile * 16;
    const int planes = kMode == kBlocks ? a.drafts : 1, at_plane = blockIdx.x / a.row_tiles;
    const int head = at_plane / planes, plane = at_plane - head * planes;
    int rows, first, last, first_slot;
    if constexpr (kMode == kBlocks) {
        const int2 pieces = a.span_pieces[(int64_t)b * a.drafts + plane];     // not written without drafted tokens
        rows = plane < drafts_of(a, b) ? a.group : 0;
        first = pieces.x >> 1, last = pieces.y, first_slot = pieces.x;
    } else {
        Chunk<kMode> chunk = chunk_at<kMode>(a, 0, lane, plane, 0);
        const int64_t total = all_tiles<kMode>(a, chunk, lane, plane, 0);
        const int shift = shift_of(a, total);
        int64_t before = 0;
        while (b - chunk.first >= 64) {
            before += chunk.all();
            chunk = chunk_at<kMode>(a, chunk.first + 64, lane, plane, 0);
        }
        const uint32_t tiles = chunk.read(chunk.tiles, b - chunk.first);
        rows = __builtin_amdgcn_readlane(chunk.drafts, b - chunk.first) * a.group;
        before += chunk.read(chunk.upto, b - chunk.first) - tiles;
        if (tiles == 0) return;
        // The ranges that hold its first and last tile: tile t lies in the last range
        // whose start, x * total >> shift, is at most t.
        first = (int)scalar((((before + 1) << shift) - 1) / total);
        last = (int)scalar((((before + tiles) << shift) - 1) / total);
        // The first piece is its range's second one unless the range starts with it.
        first_slot = 2 * first + ((first * total >> shift) == before ? 0 : 1);
    }
    if (r0 >= rows || first == last) return;                  // one piece: written already
    const int team = threadIdx.x / kTeam, part = threadIdx.x % kTeam, i = kPer * blockIdx.z + (part >> 6);

    Joined<D, kTeams> joined;
    joined.add(a.part, part_place<kMode>(a, false, 0, b, plane, row_tile, head).stats, team, i, g, first, last, last - first, c,
               [&](int x) {
                   return part_place<kMode>(a, false, x == first ? first_slot : 2 * (int64_t)x, b, plane, row_tile, head).tile;
               });
    finish_join<D, kPer>(joined, team, part, i, lane, r0, rows, [&](int row) {
        const int t = kMode == kBlocks ? plane : row / a.group, h = kMode == kBlocks ? row : row % a.group;
        return a.out + ((int64_t)b * a.drafts + t) * a.ld_out + ((int64_t)head * a.group + h) * D;
    });
}

// How the call is laid out, from its shapes alone.
struct Layout {
    int nr, heads, groups, columns, shift; // row tiles per wave, heads and row groups per workgroup, workgroups per range
};
// Two row tiles to a wave share the widened keys and values (the cases at the top,
// with one: 162 us and 284); at 256 values their sums do not fit the registers.  With
// more rows than that, two waves of a workgroup take one head's tokens and share the
// staged tiles.  A workgroup has at most 4 waves: the two cases take
//   4 heads, 1 row group    114 + 13 us,  201 + 12 us
//   2 heads, 2 row groups   113 + 13 us,  188 + 9 us
//   4 heads, 2 row groups   118 + 13 us,  193 + 9 us
//   1 head, 2 row groups    115 + 13 us,  195 + 10 us
// (2 heads, 4 row groups: 195 + 9 us; 8 heads, 1 row group: 119 + 13, 198 + 10).
// rows: of a key/value head; planes: of workgroups, each with its own tokens; apart: each
// head has tokens of its own.
inline Layout layout_of(int rows, int kv_heads, int head_dim, int planes = 1, bool apart = false) {
    Layout l;
    l.nr = rows > 16 && head_dim <= 128 ? 2 : 1;
    l.groups = rows > 16 * l.nr && head_dim <= 128 ? 2 : 1;
    l.heads = apart ? 1 : kv_heads % 4 == 0 && l.groups == 1 ? 4 : kv_heads % 2 == 0 ? 2 : 1;
    const int span = 16 * l.nr * l.groups;
    l.columns = kv_heads / l.heads * ((rows + span - 1) / span) * planes;
    // 2^shift ranges (at least 8, so that a range's workgroups meet on one XCD)
    l.shift = 3;
    while ((int64_t)l.columns * l.heads * l.groups << (l.shift + 1) <= kGridWaves) ++l.shift;
    return l;
}

// The instantiation of a kernel for a layout: f(row tiles, heads, row groups), as Int<>s.
template <int D, class F>
hipError_t with_layout(const Layout& l, F&& f) {
    auto with_heads = [&](auto nr, auto rg) {
        if constexpr (decltype(rg)::value == 1) {
            if (l.heads == 4) return f(nr, Int<4>(), rg);
        }
        return l.heads == 2 ? f(nr, Int<2>(), rg) : f(nr, Int<1>(), rg);
    };
    if constexpr (D <= 128) {
        if (l.nr == 2) return l.groups == 2 ? with_heads(Int<2>(), Int<2>()) : with_heads(Int<2>(), Int<1>());
    }
    return with_heads(Int<1>(), Int<1>());
}
template <class F>
hipError_t with_head_dim(int head_dim, F&& f) {
    switch (head_dim) {
        case 64: return f(Int<64>());
        case 128: return f(Int<128>());
        default: return f(Int<256>());
    }
}

// The walk, and the join of what it cut.
template <Mode kMode, int D>
hipError_t launch_walk(const TreeArgs& a, const Layout& l, unsigned columns, hipStream_t s) {
    return with_layout<D>(l, [&](auto nr, auto hw, auto rg) {
        constexpr int kNR = decltype(nr)::value, kHW = decltype(hw)::value, kRG = decltype(rg)::value;
        attn_walk_kernel<kMode, D, kNR, kHW, kRG><<<dim3(1u << l.shift, columns), 64 * kHW * kRG, 0, s>>>(a);
        return hipGetLastError();
    });
}
template <Mode kMode, int D>
hipError_t launch_join(const TreeArgs& a, int planes, hipStream_t s) {
    const unsigned row_tiles = (unsigned)(a.kv_heads * planes * a.row_tiles);
    // Many pieces of few rows (on average of the sequences, and so that all workgroups
    // are resident): 16 waves to a slice.  One sequence of 100000 tokens: 8 us, against
    // 37 with a wave to a slice; the 4 long contexts with 16 drafts: 16 us against 11.
    if (1 << a.shift >= 16 * a.batch && (int64_t)row_tiles * a.batch * (D / 16) <= 512)
        attn_join_kernel<kMode, D, 1, 16><<<dim3(row_tiles, (unsigned)a.batch, D / 16), 1024, 0, s>>>(a);
    else
        attn_join_kernel<kMode, D, D / 16, 1><<<dim3(row_tiles, (unsigned)a.batch), 4 * D, 0, s>>>(a);
    return hipGetLastError();
}

// What the entry points' arguments have in common.
inline TreeArgs cache_args(const AttnTree& p, const Layout& l) {
    TreeArgs a{};
    a.q = p.q, a.ld_q = p.ld_q, a.out = p.out, a.ld_out = p.ld_out;
    a.kc = p.cache.k_codes, a.ks = p.cache.k_scales, a.vc = p.cache.v_codes, a.vs = p.cache.v_scales;
    a.num_pages = p.cache.num_pages, a.page_size = (int)p.cache.page_size;
    a.code_row = (int)(p.cache.d / 2), a.scale_row = (int)(p.cache.d / 32);
    a.table = p.page_table, a.max_pages = p.max_pages;
    a.seq_lens = p.seq_lens, a.draft_lens = p.draft_lens, a.mask = p.tree_mask;
    a.batch = (int)p.batch, a.drafts = p.drafts, a.group = p.q_heads / p.kv_heads, a.kv_heads = p.kv_heads;
    a.rows = p.drafts * a.group;
    // Never 0: a hidden score is -inf and has to stay that when scaled.
    a.scale2 = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-37f);
    a.flip = p.scale < 0 ? 0x80008000u : 0u;
    a.part = static_cast<float*>(p.ws), a.row_tiles = (a.rows + 15) / 16, a.shift = l.shift, a.ranges = 1 << l.shift;
    return a;
}
// Bytes of tiles of 16 rows' sums and (m, sum).
inline size_t part_bytes(int64_t tiles, int head_dim) { return (size_t)tiles * 16 * (head_dim + 2) * sizeof(float); }

}  // namespace
}  // namespace fp4
