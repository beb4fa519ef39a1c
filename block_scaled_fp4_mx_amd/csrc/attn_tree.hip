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
    // Partial results [2 << shift][kv_heads][row tiles]: of 16 rows, the sums as the
    // lanes hold them ([D/16][64] of 4 values), then (m, sum) of each row.
    float* part;
    int row_tiles, shift;
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

// 64 sequences of the batch from first on, one to a lane, with the tiles of those
// up to a lane's own (fewer than 2^32: a sequence has fewer than 2^26).
struct Chunk {
    int first, len, seen, drafts;
    uint32_t tiles, upto;
    __device__ __forceinline__ uint32_t all() const { return __builtin_amdgcn_readlane(upto, 63); }
};
__device__ __forceinline__ Chunk chunk_at(const TreeArgs& a, int first, int lane) {
    const int b = min(first + lane, a.batch - 1);
    Chunk c;
    c.first = first;
    c.len = max(a.seq_lens[b], 0);
    c.drafts = drafts_of(a, b);
    c.seen = tokens_of(a, c.len, c.drafts);
    c.tiles = first + lane < a.batch ? tiles_of(c.seen, c.drafts) : 0;
    c.upto = c.tiles;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const uint32_t o = __shfl_up(c.upto, m, 64);
        if (lane >= m) c.upto += o;
    }
    return c;
}

// All tiles of the batch; c: its first chunk.  Every workgroup of both kernels walks
// the lengths so, 64 sequences a step, and the join has workgroups for each sequence:
// the cost grows with the batch's square.  Sequences of 100 tokens, 1 token each: 64 of
// them 16 us, 256 26, 512 60, 1024 162, 4096 1980 (116 us of bytes).
__device__ __forceinline__ int64_t all_tiles(const TreeArgs& a, const Chunk& c, int lane) {
    int64_t n = c.all();
    for (int b = 64; b < a.batch; b += 64) n += chunk_at(a, b, lane).all();
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

template <int D, int NR, int HW, int RG>
__global__ __launch_bounds__(64 * HW * RG, D == 256 ? 1 : 2) void attn_tree_kernel(const TreeArgs a) {
    constexpr int kSteps = D / 32, kOut = D / 16;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    using S = Stage<D, HW>;
    constexpr int kRegion = kStages * S::kBytes;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), groups = a.kv_heads / HW;
    const int hw = wave % HW, rg = RG == 1 ? 0 : wave / HW;
    const int head0 = __builtin_amdgcn_readfirstlane(blockIdx.y % groups) * HW, head = head0 + hw;
    const int r0 = (__builtin_amdgcn_readfirstlane(blockIdx.y / groups) * RG + rg) * 16 * NR;
    __shared__ __attribute__((aligned(16))) uint8_t staging[HW * kRegion];
    const uint32_t lds = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_bytes)(uint8_t*)staging) + hw * kRegion;
    const Lane<D, HW> own = lane_of<D, HW>(a, head0, hw, lane);
    Chunk chunk = chunk_at(a, 0, lane);
    const int64_t total = all_tiles(a, chunk, lane);
    const int shift = shift_of(a, total);
    const int64_t lo = blockIdx.x * total >> shift, hi = (blockIdx.x + 1) * total >> shift;
    if (blockIdx.x >> shift || lo == hi) return;

    // The sequence that holds tile lo, and the tiles before it.
    int64_t before = 0;
    while (before + chunk.all() <= lo) {
        before += chunk.all();
        chunk = chunk_at(a, chunk.first + 64, lane);
    }
    int b = chunk.first;
    {
        const int k = __popcll(__ballot((int64_t)(before + chunk.upto) <= lo));       // those that end by lo
        if (k) before += (uint32_t)__builtin_amdgcn_readlane(chunk.upto, k - 1);
        b += k;
    }

    for (int64_t at = lo; at < hi; ++b) {
        if (b - chunk.first == 64) chunk = chunk_at(a, b, lane);
        const int tiles = __builtin_amdgcn_readlane(chunk.tiles, b - chunk.first);
        if (tiles == 0) continue;
        const int t0 = (int)(at - before), t1 = (int)min(hi - before, (int64_t)tiles);
        const int len = __builtin_amdgcn_readlane(chunk.len, b - chunk.first);
        const int seen = __builtin_amdgcn_readlane(chunk.seen, b - chunk.first);
        const int nd = __builtin_amdgcn_readlane(chunk.drafts, b - chunk.first);
        const int32_t* table = a.table + (int64_t)b * a.max_pages;

        u32x4 q[NR][kSteps];
        uint64_t vis[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int row = r0 + 16 * n + c, t = row / a.group;
            const bool live = t < nd;
            const uint16_t* x = a.q + ((int64_t)b * a.drafts + (live ? t : 0)) * a.ld_q +
                                ((int64_t)head * a.group + row % a.group) * D + g * (D / 4);
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
                q[n][s] = live ? *reinterpret_cast<const u32x4*>(x + 8 * s) ^ a.flip : u32x4{0, 0, 0, 0};
            vis[n] = 0;
            if (live) {
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
        int half_i = 2 * t0, first_half = half_i - 64, rows = 0;
        auto place = [&]() {
            if (half_i >= first_half + 64) {
                first_half = half_i;
                const int at = half_i + lane, per = a.page_size / 16, i = at / per;
                const int page = table[min(i, (int)a.max_pages - 1)];
                const bool there = i < a.max_pages && (uint32_t)page < (uint32_t)a.num_pages;
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
                    const float up = fmaxf(m[n], x), alpha = exp2_hw(m[n] - up);
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
                if (t + 1 >= t1)
                    wait_copies<0>();
                else if (RG == 1)
                    wait_copies<2 * S::kItems + S::kWords>();
                else if (rg == 0)
                    wait_copies<S::kItems + S::kWords>();
                else
                    wait_copies<S::kItems>();
                meet<HW * RG>();
                if (t + 2 < t1) start((k + 2) % kStages);
                compute(t, at_stage[k], k * S::kBytes);
            };
            start(0);
            if (t0 + 1 < t1) start(1);
            for (int t = t0; t < t1; t += 3) {
                turn(t, Int<0>());
                if (t + 1 < t1) turn(t + 1, Int<1>());
                if (t + 2 < t1) turn(t + 2, Int<2>());
            }
            meet<HW * RG>();                                  // before the next sequence's copies
        }
        // A weight of 0 does not hide an infinite value, so the drafted tokens' blocks
        // with such values are left out above and added here, to the rows that see them.
        if (any_apart) {
            constexpr int kBlocks = D == 256 ? 2 : 1;              // that a lane's D/4 values lie in
            const int at_code = head * (D / 2) + g * (D / 8), at_scale = head * (D / 32) + (D == 64 ? g / 2 : kBlocks * g);
#pragma unroll 1
            for (int pos = max(t0 * kTile, len); pos < min(t1 * kTile, seen); ++pos) {
                const int page = table[pos / a.page_size], d = pos - len;
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
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float l = sum[n][0];
            const int row = r0 + 16 * n + c, t = row / a.group;
            if (whole) {
                if (t >= nd) continue;
                const float inv = l > 0.f ? 1.0f / l : 0.f;
                uint16_t* y = a.out + ((int64_t)b * a.drafts + t) * a.ld_out +
                              ((int64_t)head * a.group + row % a.group) * D + g * (D / 4);
#pragma unroll
                for (int i = 0; i < 4; ++i) {                 // D/16 consecutive values each
                    uint32_t w[kOut / 2];
#pragma unroll
                    for (int j = 0; j < kOut / 2; ++j) w[j] = pack2(o[n][2 * j][i] * inv, o[n][2 * j + 1][i] * inv);
#pragma unroll
                    for (int j = 0; j < kOut / 2; j += 2)
                        *reinterpret_cast<uint2*>(y + i * kOut + 2 * j) = make_uint2(w[j], w[j + 1]);
                }
            } else if (r0 + 16 * n < a.rows) {
                const int64_t slot = 2 * (int64_t)blockIdx.x + (at == lo ? 0 : 1);
                const int64_t rt = (slot * a.kv_heads + head) * a.row_tiles + r0 / 16 + n;
                v4f* y = reinterpret_cast<v4f*>(a.part) + rt * (4 * D) + lane;
#pragma unroll
                for (int i = 0; i < kOut; ++i) y[64 * i] = o[n][i];
                float2* ml = reinterpret_cast<float2*>(a.part + ((int64_t)2 << a.shift) * a.kv_heads * a.row_tiles * 16 * D);
                if (g == 0) ml[rt * 16 + c] = make_float2(m[n], l);
            }
        }
        at += t1 - t0;
        before += tiles;
    }
}

// Joins the partial results of the sequences that were cut: workgroup (x, y) takes
// 16 rows of a head (x) of sequence y, and of their values the kPer slices from
// kPer * z on (slice i: the values i, i + D/16, ...).  A wave reads a slice of a
// piece as it was written, 16 bytes a lane; kTeams of kPer waves take the pieces in
// turn, and their sums are joined through LDS in team order.
template <int D, int kPer, int kTeams>
__global__ __launch_bounds__(64 * kPer * kTeams) void attn_tree_join_kernel(const TreeArgs a) {
    constexpr int kTeam = 64 * kPer, kBatch = 8, kOut = D / 16;
    __shared__ v4f sums[kTeams > 1 ? kTeam * kTeams : 1];
    __shared__ float2 stats[kTeams][16];
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int b = blockIdx.y, head = blockIdx.x / a.row_tiles, r0 = blockIdx.x % a.row_tiles * 16;
    Chunk chunk = chunk_at(a, 0, lane);
    const int64_t total = all_tiles(a, chunk, lane);
    const int shift = shift_of(a, total);
    int64_t before = 0;
    while (b - chunk.first >= 64) {
        before += chunk.all();
        chunk = chunk_at(a, chunk.first + 64, lane);
    }
    const uint32_t tiles = __builtin_amdgcn_readlane(chunk.tiles, b - chunk.first);
    const int nd = __builtin_amdgcn_readlane(chunk.drafts, b - chunk.first);
    before += (uint32_t)__builtin_amdgcn_readlane(chunk.upto, b - chunk.first) - tiles;
    if (tiles == 0 || r0 >= nd * a.group) return;
    // The ranges that hold its first and last tile: tile t lies in the last range
    // whose start, x * total >> shift, is at most t.
    const int first = (int)scalar((((before + 1) << shift) - 1) / total);
    const int last = (int)scalar((((before + tiles) << shift) - 1) / total);
    if (first == last) return;                                // one piece: written already
    // The first piece is its range's second one unless the range starts with it.
    const int first_slot = 2 * first + ((first * total >> shift) == before ? 0 : 1);
    const int team = threadIdx.x / kTeam, part = threadIdx.x % kTeam, i = kPer * blockIdx.z + (part >> 6);
    const int64_t step = (int64_t)a.kv_heads * a.row_tiles;
    const v4f* o = reinterpret_cast<const v4f*>(a.part) + (int64_t)blockIdx.x * (4 * D) + 64 * i + lane;
    const float2* ml = reinterpret_cast<const float2*>(a.part + ((int64_t)2 << a.shift) * step * 16 * D) +
                       (int64_t)blockIdx.x * 16 + c;

    float m = kFloor, l = 0.f;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    for (int x0 = first + team; x0 <= last; x0 += kBatch * kTeams) {
        float2 s[kBatch];
        v4f v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int x = x0 + k * kTeams;
            s[k] = make_float2(kFloor, 0.f);
            v[k] = v4f{0.f, 0.f, 0.f, 0.f};
            if (x <= last) {
                const int64_t at = (x == first ? first_slot : 2 * (int64_t)x) * step;
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
    if constexpr (kTeams > 1) {
        sums[threadIdx.x] = acc;
        if (part < 16) stats[team][part] = make_float2(m, l);
        __syncthreads();
        if (team == 0) {
            float top = kFloor;
#pragma unroll
            for (int k = 0; k < kTeams; ++k) top = fmaxf(top, stats[k][c].x);
            l = 0.f;
            acc = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < kTeams; ++k) {
                const float e = exp2_hw(stats[k][c].x - top);
                l += stats[k][c].y * e;
                acc += sums[part + k * kTeam] * e;
            }
        }
    }
    const float inv = l > 0.f ? 1.0f / l : 0.f;
    auto out_at = [&](int row) {
        return a.out + ((int64_t)b * a.drafts + row / a.group) * a.ld_out + ((int64_t)head * a.group + row % a.group) * D;
    };
    if constexpr (kPer == kOut) {                             // whole rows go out through LDS in 16-byte parts
        __shared__ __attribute__((aligned(16))) uint16_t rows[16][D + 8];
#pragma unroll
        for (int k = 0; k < 4; ++k) rows[c][g * (D / 4) + k * kOut + i] = (uint16_t)pack2(acc[k] * inv, 0.f);
        __syncthreads();
        const int chunks = D / 8, r = threadIdx.x / chunks, at = threadIdx.x % chunks * 8;
        if (r < 16 && r0 + r < nd * a.group)
            *reinterpret_cast<uint4*>(out_at(r0 + r) + at) = *reinterpret_cast<const uint4*>(&rows[r][at]);
    } else if (team == 0 && r0 + c < nd * a.group) {
        uint16_t* y = out_at(r0 + c) + g * (D / 4) + i;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k * kOut] = (uint16_t)pack2(acc[k] * inv, 0.f);
    }
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
Layout layout_of(int drafts, int q_heads, int kv_heads, int head_dim) {
    const int rows = drafts * (q_heads / kv_heads);
    Layout l;
    l.nr = rows > 16 && head_dim <= 128 ? 2 : 1;
    l.groups = rows > 16 * l.nr && head_dim <= 128 ? 2 : 1;
    l.heads = kv_heads % 4 == 0 && l.groups == 1 ? 4 : kv_heads % 2 == 0 ? 2 : 1;
    const int span = 16 * l.nr * l.groups;
    l.columns = kv_heads / l.heads * ((rows + span - 1) / span);
    // 2^shift ranges (at least 8, so that a range's workgroups meet on one XCD)
    l.shift = 3;
    while ((int64_t)l.columns * l.heads * l.groups << (l.shift + 1) <= kGridWaves) ++l.shift;
    return l;
}

template <int D, int NR, int HW, int RG>
hipError_t launch(const TreeArgs& a, const Layout& l, hipStream_t s) {
    attn_tree_kernel<D, NR, HW, RG><<<dim3(1u << l.shift, (unsigned)l.columns), 64 * HW * RG, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned row_tiles = (unsigned)(a.kv_heads * a.row_tiles);
    // Many pieces of few rows (on average of the sequences, and so that all workgroups
    // are resident): 16 waves to a slice.  One sequence of 100000 tokens: 8 us, against
    // 37 with a wave to a slice; the 4 long contexts with 16 drafts: 16 us against 11.
    if (1 << l.shift >= 16 * a.batch && (int64_t)row_tiles * a.batch * (D / 16) <= 512)
        attn_tree_join_kernel<D, 1, 16><<<dim3(row_tiles, (unsigned)a.batch, D / 16), 1024, 0, s>>>(a);
    else
        attn_tree_join_kernel<D, D / 16, 1><<<dim3(row_tiles, (unsigned)a.batch), 4 * D, 0, s>>>(a);
    return hipGetLastError();
}
template <int D, int NR, int RG>
hipError_t launch(const TreeArgs& a, const Layout& l, hipStream_t s) {
    if constexpr (RG == 1) {
        if (l.heads == 4) return launch<D, NR, 4, RG>(a, l, s);
    }
    return l.heads == 2 ? launch<D, NR, 2, RG>(a, l, s) : launch<D, NR, 1, RG>(a, l, s);
}
template <int D>
hipError_t launch(const TreeArgs& a, const Layout& l, hipStream_t s) {
    if constexpr (D <= 128) {
        if (l.nr == 2) return l.groups == 2 ? launch<D, 2, 2>(a, l, s) : launch<D, 2, 1>(a, l, s);
    }
    return launch<D, 1, 1>(a, l, s);
}

}  // namespace

size_t attn_tree_workspace_bytes(int drafts, int q_heads, int head_dim, int kv_heads) {
    const Layout l = layout_of(drafts, q_heads, kv_heads, head_dim);
    const size_t row_tiles = (size_t)(drafts * (q_heads / kv_heads) + 15) / 16;
    return ((size_t)2 << l.shift) * kv_heads * row_tiles * 16 * (head_dim + 2) * sizeof(float);
}

hipError_t launch_attn_tree(const AttnTree& p, hipStream_t s) {
    const Layout l = layout_of(p.drafts, p.q_heads, p.kv_heads, p.head_dim);
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
    a.part = static_cast<float*>(p.ws), a.row_tiles = (a.rows + 15) / 16, a.shift = l.shift;
    switch (p.head_dim) {
        case 64: return launch<64>(a, l, s);
        case 128: return launch<128>(a, l, s);
        default: return launch<256>(a, l, s);
    }
}

}  // namespace fp4
