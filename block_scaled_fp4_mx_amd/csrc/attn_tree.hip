// Attention of drafted tokens over the paged MXFP4 cache.
//
//   o = sum_j 2^(c s_j - m) v_j / sum_j 2^(c s_j - m),  s_j = q . k_j,
//   c = scale * log2(e), over the visible tokens j, in one pass: m is a running
//   reference near the row's maximum, and o and the sum are scaled when it moves.
//
// Bound by HBM: a token's keys and values are 2 * (d/2 + d/32) bytes for all
// its heads and are read once for all query rows of a sequence.  A wave takes
// one key/value head and up to 16 * NR of the query rows that share it (drafts
// times q_heads / kv_heads), and walks its tokens 32 at a time without LDS or
// barriers: every operand is loaded in the layout the matrix core takes.
//
//   S^T = K Q^T on v_mfma_f32_16x16x32_bf16: lane (c = lane % 16, g = lane / 16)
//   loads the quarter g of token c's row, one load for all K steps (the order of
//   a row's values among the steps is free as long as Q is loaded alike), and
//   widens it with its block scales (exact in bf16).
//   The result leaves lane (c, g) with query row c and tokens 4g .. 4g+3, which
//   is what the B operand of O^T = V^T P^T takes if the token order within a
//   step is (g, tile, i): the weights never leave their lane.
//   V^T needs 8 tokens of one value per lane: a lane loads the same d/16 values
//   of its 8 tokens (16 lanes cover the row), widens each with its token's
//   scale, and pairs tokens with byte permutes.
//   O^T leaves lane (c, g) with d/4 consecutive values of row c.
//
// The reference m moves only when some score exceeds it by more than 2^8 (one
// ballot); until then no lane exchange is needed.  Weights are rounded to bf16
// for the second product (they enter it with V's 16-bit format); their sum is
// kept in fp32 from the unrounded weights.
//
// Work split: the batch's tiles of 32 tokens are laid end to end and cut into
// equal ranges, one per workgroup column, whatever the lengths; a sequence that
// a cut goes through leaves partial (m, sum, o) in the workspace, at most two
// per range, and a second kernel joins them in order.
#include <type_traits>

#include "fp4_internal.h"
#include "mma_core.h"

namespace fp4 {
namespace {

constexpr int kTile = 32;                  // tokens per step
constexpr int kMinTiles = 4;               // tiles per range below which fewer ranges are used
constexpr int kGridWaves = 2048;           // two per SIMD
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
    float* part;                           // [2 * ranges][kv_heads][rows][D] sums, then [..][2] (m, sum)
    int ranges;
};

__device__ __forceinline__ int drafts_of(const TreeArgs& a, int b) {
    return a.draft_lens ? min(max(a.draft_lens[b], 0), a.drafts) : a.drafts;
}

// Tokens of sequence b that can be seen at all: its committed and drafted ones,
// as far as the table's row goes (none in an empty pool).  Positions of a tile
// stay below 2^31.
__device__ __forceinline__ int tokens_of(const TreeArgs& a, int b) {
    const int64_t n = (int64_t)max(a.seq_lens[b], 0) + drafts_of(a, b);
    return a.num_pages ? (int)min(min(n, a.max_pages * a.page_size), (int64_t)0x7FFFFFC0) : 0;
}

// Tiles of sequence b; a sequence with drafted tokens has at least one, so that
// its rows are written.
__device__ __forceinline__ int tiles_of(const TreeArgs& a, int b) {
    if (b >= a.batch || drafts_of(a, b) == 0) return 0;
    return max((tokens_of(a, b) + kTile - 1) / kTile, 1);
}

// A value equal in all lanes, as a scalar (so that what follows from it is one too).
__device__ __forceinline__ int64_t scalar(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ int64_t wave_sum(int64_t v) {
#pragma unroll
    for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m, 64);
    return scalar(v);
}

// All tiles of the batch, and the ranges they are cut into.
__device__ __forceinline__ int64_t all_tiles(const TreeArgs& a, int lane) {
    int64_t n = 0;
    for (int b = lane; b < a.batch; b += 64) n += tiles_of(a, b);
    return wave_sum(n);
}
__device__ __forceinline__ int64_t used_ranges(const TreeArgs& a, int64_t tiles) {
    return min((int64_t)a.ranges, max((tiles + kMinTiles - 1) / kMinTiles, (int64_t)1));
}

// Tiles of the sequences before b (all lanes must call).
__device__ __forceinline__ int64_t tiles_before(const TreeArgs& a, int b, int lane) {
    int64_t n = 0;
    for (int i = lane; i < b; i += 64) n += tiles_of(a, i);
    return wave_sum(n);
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
// A block's scale from the aligned word that holds its byte: rotated so that the
// byte stands in the exponent's bits; widen looks at no others.
__device__ __forceinline__ float scale_of(uint32_t word, uint32_t turn) {
    return __uint_as_float(__builtin_amdgcn_alignbit(word, word, turn));
}
constexpr uint32_t kOnes = 0x7F7F7F7Fu;    // scales of 1

template <int N>
using Int = std::integral_constant<int, N>;

// A tile's place: the first cache row of its two halves (-1: no page).
struct Place {
    int row[2];
};

// A workgroup's staging of a tile in LDS: HW neighbouring heads of 32 tokens, one
// wave for each.  Rows are read from global memory in 16-byte chunks, neighbouring
// lanes in neighbouring chunks of the heads' part of a row, straight into LDS: the
// memory behind is bound by requests, and whole 128-byte lines make the fewest (a
// head's part of a row alone is half a line at D = 128).  Every wave copies 1/HW
// of the rows, of all heads, into a region of its own:
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
    static constexpr int kItems = kChunks / 2;                           // copies of keys, and of values, per wave
    static constexpr int kCopies = 2 * kItems + kWords;
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
template <int HW>
__device__ __forceinline__ void meet() {
    if (HW > 1)
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

// Starts a wave's copies of a tile into its region of the stage at lds (global
// memory to LDS, lane l's 16 or 4 bytes to M0 + offset + l * size); awaited by
// wait_copies.  Halves without a page read row 0 on (a row of the pool; hidden
// later).  A wave's copies are one asm block behind one write of M0 (which needs a
// wait state); the instruction's offset, -4096 to 4095, counts on the global side
// as well, so each address is given less it.
template <int D, int HW>
__device__ __forceinline__ void copy_tile(const TreeArgs& a, const Place& p, const Lane<D, HW>& o, int wave, int lane,
                                          uint32_t lds) {
    const int row0 = max(p.row[0], 0), row1 = max(p.row[1], 0), mine = HW > 1 && wave < HW / 2 ? row0 : row1;
    const uint8_t* scale = o.scale + (uint64_t)(uint32_t)(lane & 16 ? row1 : row0) * (uint32_t)a.scale_row;
    if constexpr (D == 64) {                              // HW = 1: both halves in one instruction
        const uint64_t at = (uint64_t)(uint32_t)(HW == 1 && !(lane & 32) ? row0 : mine) * (uint32_t)a.code_row;
        asm volatile(
            "s_mov_b32 m0, %3\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %0, off\n\t"
            "global_load_lds_dwordx4 %1, off offset:1024\n\t"
            "global_load_lds_dword %2, off offset:2048" ::"v"(a.kc + at + o.key[0]),
            "v"(a.vc + at + o.value[0] - 1024), "v"(scale - 2048), "s"(lds)
            : "memory", "m0");
    } else {
        // HW = 1: the first half of the copies takes the tile's first half.
        const int64_t at0 = (int64_t)(HW == 1 ? row0 : mine) * a.code_row, at1 = HW == 1 ? (int64_t)row1 * a.code_row : at0;
        if constexpr (D == 128) {
            asm volatile(
                "s_mov_b32 m0, %9\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, %4 offset:-1024\n\t"
                "global_load_lds_dwordx4 %1, %5\n\t"
                "global_load_lds_dwordx4 %2, %6 offset:1024\n\t"
                "global_load_lds_dwordx4 %3, %7 offset:2048\n\t"
                "global_load_lds_dword %8, off offset:3072" ::"v"(o.key[0]),
                "v"(o.key[1]), "v"(o.value[0]), "v"(o.value[1]), "s"(a.kc + at0 + 1024), "s"(a.kc + at1),
                "s"(a.vc + at0 - 1024), "s"(a.vc + at1 - 2048), "v"(scale - 3072), "s"(lds + 1024)
                : "memory", "m0");
        } else {
            asm volatile(
                "s_mov_b32 m0, %8\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, %4\n\t"
                "global_load_lds_dwordx4 %1, %5 offset:1024\n\t"
                "global_load_lds_dwordx4 %2, %6 offset:2048\n\t"
                "global_load_lds_dwordx4 %3, %7 offset:3072" ::"v"(o.key[0]),
                "v"(o.key[1]), "v"(o.key[2]), "v"(o.key[3]), "s"(a.kc + at0), "s"(a.kc + at0 - 1024),
                "s"(a.kc + at1 - 2048), "s"(a.kc + at1 - 3072), "s"(lds)
                : "memory", "m0");
            asm volatile(
                "s_mov_b32 m0, %10\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, %4 offset:-4096\n\t"
                "global_load_lds_dwordx4 %1, %5 offset:-3072\n\t"
                "global_load_lds_dwordx4 %2, %6 offset:-2048\n\t"
                "global_load_lds_dwordx4 %3, %7 offset:-1024\n\t"
                "global_load_lds_dword %8, off\n\t"
                "global_load_lds_dword %9, off offset:256" ::"v"(o.value[0]),
                "v"(o.value[1]), "v"(o.value[2]), "v"(o.value[3]), "s"(a.vc + at0 + 4096), "s"(a.vc + at0 + 3072),
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

template <int D, int NR, int HW>
__global__ __launch_bounds__(64 * HW, D == 256 || HW == 8 ? 1 : 2) void attn_tree_kernel(const TreeArgs a) {
    constexpr int kSteps = D / 32, kOut = D / 16;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    using S = Stage<D, HW>;
    constexpr int kRegion = kStages * S::kBytes;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), groups = a.kv_heads / HW;
    const int head0 = __builtin_amdgcn_readfirstlane(blockIdx.y % groups) * HW, head = head0 + wave;
    const int r0 = __builtin_amdgcn_readfirstlane(blockIdx.y / groups) * 16 * NR;
    __shared__ __attribute__((aligned(16))) uint8_t staging[HW * kRegion];
    const uint32_t lds =
        __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_bytes)(uint8_t*)staging) + wave * kRegion;
    const Lane<D, HW> own = lane_of<D, HW>(a, head0, wave, lane);
    const int64_t total = all_tiles(a, lane), ranges = used_ranges(a, total);
    if ((int64_t)blockIdx.x >= ranges || total == 0) return;
    const int64_t lo = scalar(blockIdx.x * total / ranges), hi = scalar((blockIdx.x + 1) * total / ranges);

    // The sequence that holds tile lo, and the tiles before it.
    int b = 0;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 64) {
        int64_t n = tiles_of(a, b0 + lane);
#pragma unroll
        for (int m = 1; m < 64; m *= 2) {
            const int64_t o = __shfl_up(n, m, 64);
            if (lane >= m) n += o;
        }
        const int64_t chunk = scalar(__shfl(n, 63, 64));
        if (before + chunk > lo) {
            const int k = __popcll(__ballot(before + n <= lo));       // sequences of this chunk that end by lo
            if (k) before += scalar(__shfl(n, k - 1, 64));
            b = b0 + k;
            break;
        }
        before += chunk;
    }
    b = __builtin_amdgcn_readfirstlane(b);

    for (int64_t at = lo; at < hi; ++b) {
        const int tiles = __builtin_amdgcn_readfirstlane(tiles_of(a, b));
        if (tiles == 0) continue;
        const int t0 = (int)(at - before), t1 = (int)min(hi - before, (int64_t)tiles);
        const int len = __builtin_amdgcn_readfirstlane(max(a.seq_lens[b], 0));
        const int seen = __builtin_amdgcn_readfirstlane(tokens_of(a, b));
        const int nd = __builtin_amdgcn_readfirstlane(drafts_of(a, b));
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
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int pos = pos0 + 16 * (j / 4) + 4 * g + j % 4, d = pos - len;
                    const bool there = (pos < seen) & (here.row[j / 4] >= 0);
                    vscale[j / 4][j % 4] = there ? vscale[j / 4][j % 4] : kOnes;      // whatever lies there, finite
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        const bool see = there & ((d < 0) | ((uint32_t)(vis[n] >> (d & 63)) & 1u));
                        s[n][j / 4][j % 4] = see ? s[n][j / 4][j % 4] : kNone;
                    }
                }
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
                copy_tile<D, HW>(a, at_stage[k], own, wave, lane, lds + k * S::kBytes);
            };
            auto turn = [&](int t, auto tag) {
                constexpr int k = decltype(tag)::value;
                if (t + 1 < t1)
                    wait_copies<S::kCopies>();
                else
                    wait_copies<0>();
                meet<HW>();
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
            meet<HW>();                                       // before the next sequence's copies
        }

        const bool whole = t0 == 0 && t1 == tiles;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const float l = sum[n][0];
            const int row = r0 + 16 * n + c, t = row / a.group;
            if (t >= nd) continue;
            if (whole) {
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
            } else {
                const int64_t slot = 2 * (int64_t)blockIdx.x + (at == lo ? 0 : 1);
                const int64_t at_row = (slot * a.kv_heads + head) * a.rows + row;
                float* y = a.part + at_row * D + g * (D / 4);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < kOut; j += 4)
                        *reinterpret_cast<float4*>(y + i * kOut + j) =
                            make_float4(o[n][j][i], o[n][j + 1][i], o[n][j + 2][i], o[n][j + 3][i]);
                if (g == 0) {
                    float* ml = a.part + 2 * (int64_t)a.ranges * a.kv_heads * a.rows * D + at_row * 2;
                    ml[0] = m[n], ml[1] = l;
                }
            }
        }
        at += t1 - t0;
        before += tiles;
    }
}

// Joins the partial results of the sequences that were cut.  A team of D/4 lanes
// takes a row (16 bytes a lane); kTeams of them share one, pieces dealt to them in
// turn, and their sums are joined through LDS in team order.  Workgroups of
// sequence y stride over its rows, so what the pieces are is found once for many.
template <int D, int kTeams, int kBlock>
__global__ __launch_bounds__(kBlock) void attn_tree_join_kernel(const TreeArgs a) {
    constexpr int kLanes = D / 4, kRows = kBlock / kLanes / kTeams, kBatch = 8;
    __shared__ float4 sums[kTeams > 1 ? kBlock : 1];
    __shared__ float2 stats[kTeams > 1 ? kBlock / kLanes : 1];
    const int lane = threadIdx.x & 63, b = blockIdx.y;
    const int64_t total = all_tiles(a, lane), ranges = used_ranges(a, total);
    const int tiles = __builtin_amdgcn_readfirstlane(tiles_of(a, b)), nd = drafts_of(a, b);
    if (tiles == 0) return;
    const int64_t before = tiles_before(a, b, lane);
    const int first = (int)scalar(((before + 1) * ranges - 1) / total);
    const int last = (int)scalar(((before + tiles) * ranges - 1) / total);
    if (first == last) return;                                // one piece: written already
    // The first piece is its range's second one unless the range starts with it.
    const int first_slot = 2 * first + (scalar(first * total / ranges) == before ? 0 : 1);
    const int all_rows = a.kv_heads * a.rows;
    const float* ml = a.part + 2 * (int64_t)a.ranges * all_rows * D;
    const int team = threadIdx.x / kLanes, part = team % kTeams, l4 = threadIdx.x % kLanes * 4;
    for (int r0 = blockIdx.x * kRows; r0 < all_rows; r0 += gridDim.x * kRows) {
        const int r = r0 + team / kTeams;
        const bool live = r < all_rows && r % a.rows / a.group < nd;
        float m = kFloor, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
        for (int x0 = first + part; live && x0 <= last; x0 += kBatch * kTeams) {
            float2 s[kBatch];
            float4 o[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int x = x0 + k * kTeams;
                s[k] = make_float2(kFloor, 0.f);
                o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (x <= last) {
                    const int64_t at = (int64_t)(x == first ? first_slot : 2 * x) * all_rows + r;
                    s[k] = *reinterpret_cast<const float2*>(ml + at * 2);
                    o[k] = *reinterpret_cast<const float4*>(a.part + at * D + l4);
                }
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) top = fmaxf(top, s[k].x);
            const float keep = exp2_hw(m - top);
            m = top;
            l *= keep;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] *= keep;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float e = exp2_hw(s[k].x - top);
                l += s[k].y * e;
                acc[0] += o[k].x * e, acc[1] += o[k].y * e, acc[2] += o[k].z * e, acc[3] += o[k].w * e;
            }
        }
        if constexpr (kTeams > 1) {
            sums[threadIdx.x] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (l4 == 0) stats[team] = make_float2(m, l);
            __syncthreads();
            if (part == 0) {
                float top = kFloor;
#pragma unroll
                for (int k = 0; k < kTeams; ++k) top = fmaxf(top, stats[team + k].x);
                l = acc[0] = acc[1] = acc[2] = acc[3] = 0.f;
#pragma unroll
                for (int k = 0; k < kTeams; ++k) {
                    const float e = exp2_hw(stats[team + k].x - top);
                    const float4 o = sums[threadIdx.x + k * kLanes];
                    l += stats[team + k].y * e;
                    acc[0] += o.x * e, acc[1] += o.y * e, acc[2] += o.z * e, acc[3] += o.w * e;
                }
            }
            __syncthreads();                                  // sums free for the next rows
        }
        if (live && part == 0) {
            const float inv = l > 0.f ? 1.0f / l : 0.f;
            const int row = r % a.rows, head = r / a.rows;
            uint16_t* y = a.out + ((int64_t)b * a.drafts + row / a.group) * a.ld_out +
                          ((int64_t)head * a.group + row % a.group) * D + l4;
            *reinterpret_cast<uint2*>(y) = make_uint2(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv));
        }
    }
}

template <int D, int kTeams, int kBlock>
void launch_join(const TreeArgs& a, hipStream_t s) {
    constexpr int kRows = kBlock / (D / 4) / kTeams;
    const int64_t need = ((int64_t)a.kv_heads * a.rows + kRows - 1) / kRows, most = 2048 * 256 / kBlock / a.batch;
    const unsigned x = (unsigned)(need < most ? need : most < 1 ? 1 : most);
    attn_tree_join_kernel<D, kTeams, kBlock><<<dim3(x, (unsigned)a.batch), kBlock, 0, s>>>(a);
}

// How the call is laid out, from its shapes alone.
struct Layout {
    int nr, waves, columns, ranges;        // row tiles per wave, waves (heads) per workgroup, workgroups per range
};
Layout layout_of(int drafts, int q_heads, int kv_heads, int head_dim) {
    const int rows = drafts * (q_heads / kv_heads);
    Layout l;
    l.nr = rows > 16 && head_dim <= 128 ? 2 : 1;
    l.waves = kv_heads % 8 == 0 && head_dim <= 128 ? 8 : kv_heads % 4 == 0 ? 4 : kv_heads % 2 == 0 ? 2 : 1;
    l.columns = kv_heads / l.waves * ((rows + 16 * l.nr - 1) / (16 * l.nr));
    // a multiple of 8, so that a range's workgroups meet on one XCD
    const int ranges = kGridWaves / (l.columns * l.waves) / 8 * 8;
    l.ranges = ranges < 8 ? 8 : ranges;
    return l;
}

template <int D, int NR, int HW>
hipError_t launch(const TreeArgs& a, const Layout& l, hipStream_t s) {
    attn_tree_kernel<D, NR, HW><<<dim3((unsigned)l.ranges, (unsigned)l.columns), 64 * HW, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // Pieces of a sequence on average: how many teams share a row.
    if (l.ranges >= 32 * a.batch)
        launch_join<D, 16, 1024>(a, s);
    else if (l.ranges >= 8 * a.batch)
        launch_join<D, 4, 256>(a, s);
    else
        launch_join<D, 1, 256>(a, s);
    return hipGetLastError();
}
template <int D, int NR>
hipError_t launch(const TreeArgs& a, const Layout& l, hipStream_t s) {
    if constexpr (D <= 128) {
        if (l.waves == 8) return launch<D, NR, 8>(a, l, s);
    }
    return l.waves == 4 ? launch<D, NR, 4>(a, l, s) : l.waves == 2 ? launch<D, NR, 2>(a, l, s) : launch<D, NR, 1>(a, l, s);
}

}  // namespace

size_t attn_tree_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads) {
    (void)batch;
    const Layout l = layout_of(drafts, q_heads, kv_heads, head_dim);
    return (size_t)2 * l.ranges * q_heads * drafts * (head_dim + 2) * sizeof(float);
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
    a.part = static_cast<float*>(p.ws), a.ranges = l.ranges;
    switch (p.head_dim) {
        case 64: return l.nr == 2 ? launch<64, 2>(a, l, s) : launch<64, 1>(a, l, s);
        case 128: return l.nr == 2 ? launch<128, 2>(a, l, s) : launch<128, 1>(a, l, s);
        default: return launch<256, 1>(a, l, s);
    }
}

}  // namespace fp4
