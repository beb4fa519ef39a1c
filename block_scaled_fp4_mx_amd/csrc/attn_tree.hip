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
constexpr int kWaves = 4;                  // at most, per workgroup
constexpr int kMinTiles = 4;               // tiles per range below which fewer ranges are used
constexpr int kWorkgroups = 512;           // two per CU: two waves per SIMD
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

// One wave's staging of a tile in LDS.  Rows are read from global memory in
// 16-byte chunks, neighbouring lanes in neighbouring chunks of a row, straight
// into LDS: the vector memory pipe is bound by requests, and loads in the matrix
// core's layout (a lane its own row) would cost it several times as many.
//   keys    32 rows of kChunks chunks; chunk x of row r at x ^ swizzle(r), so that
//           the 16 lanes that read one chunk of 16 rows meet different banks
//   values  8 runs of 64 lane shares (D/32 bytes): run 4h + i has, lane by lane,
//           what lane (c, g) needs of token 16h + 4g + i
//   scales  the aligned words with a token's scale bytes: 32 of the keys, 32 of
//           the values (twice for D = 256, whose heads have two words)
template <int D>
struct Stage {
    static constexpr int kChunks = D / 32;
    static constexpr int kKeys = 16 * D, kValues = 16 * D, kWords = D == 256 ? 2 : 1;
    static constexpr int kBytes = kKeys + kValues + kWords * 256;
    static constexpr int kCopies = D == 64 ? 3 : D == 128 ? 5 : 10;      // instructions to fill it
    __device__ static constexpr int swizzle(int row) { return (row * kChunks / 16) & (kChunks - 1); }
};
constexpr int kStages = 3;                 // two tiles in flight behind the one in use

// Until at most kLeft of the wave's copies are outstanding.
template <int kLeft>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLeft) : "memory");
}
// LDS reads issued so far have returned: their stage may be copied into.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// A lane's part in the copies and in the reads.
template <int D>
struct Lane {
    uint32_t key[D == 256 ? 2 : 1], value;                // offsets of its chunks within 16 rows
    const uint8_t* scale;                                 // its token's first scale word, in row 0
    uint32_t read_key, read_value, read_ks, read_vs;      // LDS offsets
    uint32_t kturn, vturn[4];                             // turns that bring a scale byte into place
};
template <int D>
__device__ __forceinline__ Lane<D> lane_of(const TreeArgs& a, int head, int lane) {
    using S = Stage<D>;
    constexpr int kC = S::kChunks;
    const int c = lane & 15, g = lane >> 4, col = head * (D / 2), scol = head * (D / 32);
    Lane<D> o;
#pragma unroll
    for (int i = 0; i < (D == 256 ? 2 : 1); ++i) {
        const int row = (i * 64 + lane) / kC % 16;
        o.key[i] = row * a.code_row + col + ((lane % kC) ^ S::swizzle(row)) * 16;
    }
    {
        const int share = lane * 16 / (D / 32);           // the lane whose share this chunk starts with
        const int run = share / 64, of = share % 64;      // run 4h + i; D = 64: also h
        o.value = (4 * (of / 16) + run % 4) * a.code_row + col + of % 16 * (D / 32);
    }
    const int first = c * a.scale_row + scol;
    o.scale = (lane < 32 ? a.ks : a.vs) + (first & ~3);
    o.read_key = D == 64 ? (c * kC + ((g / 2) ^ S::swizzle(c))) * 16 + g % 2 * 8
                         : (c * kC + ((D == 128 ? g : 2 * g) ^ S::swizzle(c))) * 16;
    o.read_value = S::kKeys + lane * (D / 32);
    o.read_ks = S::kKeys + S::kValues + (D == 256 ? g / 2 * 256 : 0) + c * 4;
    o.read_vs = S::kKeys + S::kValues + (D == 256 ? c / 8 * 256 : 0) + 128 + 4 * g * 4;
    const int kblock = D == 64 ? g / 2 : D == 128 ? g : 2 * g;
    o.kturn = (8 * ((first + kblock) & 3) + 9) & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int byte = (4 * g + j) * a.scale_row + scol + c * (D / 16) / 32;
        // Rows of 4 bytes or more a head keep the byte's place in its word.
        o.vturn[j] = D >= 128 && j ? o.vturn[0] : (8 * (byte & 3) + 9) & 31;
    }
    return o;
}

// Starts the copies of a tile into the stage at lds (global memory to LDS, lane
// l's 16 or 4 bytes to M0 + offset + l * size); awaited by wait_copies.  Halves
// without a page read row 0 on (a row of the pool; hidden later).  The copies of a
// tile are one asm block behind one write of M0 (which needs a wait state); the
// instruction's offset, -4096 to 4095, counts on the global side as well, so each
// address is given less it.
template <int D>
__device__ __forceinline__ void copy_tile(const TreeArgs& a, const Place& p, const Lane<D>& o, int lane, uint32_t lds) {
    const int row0 = max(p.row[0], 0), row1 = max(p.row[1], 0);
    const uint8_t* scale = o.scale + (uint64_t)(uint32_t)(lane & 16 ? row1 : row0) * (uint32_t)a.scale_row;
    if constexpr (D == 64) {                              // both halves in one instruction
        const uint64_t at = (uint64_t)(uint32_t)(lane & 32 ? row1 : row0) * (uint32_t)a.code_row;
        asm volatile(
            "s_waitcnt lgkmcnt(0)\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %0, off\n\t"
            "global_load_lds_dwordx4 %1, off offset:1024\n\t"
            "global_load_lds_dword %2, off offset:2048" ::"v"(a.kc + at + o.key[0]),
            "v"(a.vc + at + o.value - 1024), "v"(scale - 2048), "s"(lds)
            : "memory", "m0");
    } else {
        const int64_t at0 = (int64_t)row0 * a.code_row, at1 = (int64_t)row1 * a.code_row;
        if constexpr (D == 128) {
            asm volatile(
                "s_waitcnt lgkmcnt(0)\n\ts_mov_b32 m0, %7\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, %2 offset:-1024\n\t"
                "global_load_lds_dwordx4 %0, %3\n\t"
                "global_load_lds_dwordx4 %1, %4 offset:1024\n\t"
                "global_load_lds_dwordx4 %1, %5 offset:2048\n\t"
                "global_load_lds_dword %6, off offset:3072" ::"v"(o.key[0]),
                "v"(o.value), "s"(a.kc + at0 + 1024), "s"(a.kc + at1), "s"(a.vc + at0 - 1024), "s"(a.vc + at1 - 2048),
                "v"(scale - 3072), "s"(lds + 1024)
                : "memory", "m0");
        } else {
            const int64_t two = 2 * (int64_t)a.code_row;
            asm volatile(
                "s_waitcnt lgkmcnt(0)\n\ts_mov_b32 m0, %6\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, %2\n\t"
                "global_load_lds_dwordx4 %1, %3 offset:1024\n\t"
                "global_load_lds_dwordx4 %0, %4 offset:2048\n\t"
                "global_load_lds_dwordx4 %1, %5 offset:3072" ::"v"(o.key[0]),
                "v"(o.key[1]), "s"(a.kc + at0), "s"(a.kc + at0 - 1024), "s"(a.kc + at1 - 2048), "s"(a.kc + at1 - 3072), "s"(lds)
                : "memory", "m0");
            asm volatile(
                "s_mov_b32 m0, %6\n\ts_nop 0\n\t"
                "global_load_lds_dwordx4 %0, %1 offset:-4096\n\t"
                "global_load_lds_dwordx4 %0, %2 offset:-3072\n\t"
                "global_load_lds_dwordx4 %0, %3 offset:-2048\n\t"
                "global_load_lds_dwordx4 %0, %4 offset:-1024\n\t"
                "global_load_lds_dword %5, off\n\t"
                "global_load_lds_dword %7, off offset:256" ::"v"(o.value),
                "s"(a.vc + at0 + 4096), "s"(a.vc + at0 + two + 3072), "s"(a.vc + at1 + 2048), "s"(a.vc + at1 + two + 1024),
                "v"(scale), "s"(lds + 8192), "v"(scale + 4 - 256)
                : "memory", "m0");
        }
    }
}

// Low (or high) halves of a and b: two tokens of one value.
template <bool kHigh>
__device__ __forceinline__ uint32_t pair(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_perm(b, a, kHigh ? 0x07060302u : 0x05040100u);
}

template <int D, int NR>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void attn_tree_kernel(const TreeArgs a) {
    constexpr int kSteps = D / 32, kOut = D / 16;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int row_groups = (a.rows + 16 * NR - 1) / (16 * NR);
    const int unit = __builtin_amdgcn_readfirstlane(blockIdx.y * (blockDim.x >> 6) + (threadIdx.x >> 6));
    if (unit >= a.kv_heads * row_groups) return;
    const int head = __builtin_amdgcn_readfirstlane(unit % a.kv_heads);
    const int r0 = __builtin_amdgcn_readfirstlane(unit / a.kv_heads) * 16 * NR;

    using S = Stage<D>;
    __shared__ __attribute__((aligned(16))) uint8_t staging[kWaves][kStages * S::kBytes];
    const uint8_t* mine = staging[threadIdx.x >> 6];
    const uint32_t lds = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_bytes)(uint8_t*)mine);
    const Lane<D> own = lane_of<D>(a, head, lane);
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

        // Places the next 16 tokens at a time.  The lanes hold 64 page ids of the
        // row (one load per 64 pages), read by lane when their turn comes.
        int page_i = __builtin_amdgcn_readfirstlane(t0 * (kTile / 16) / (a.page_size / 16));
        int off = t0 * kTile - page_i * a.page_size;
        int pages = 0, first_page = page_i - 64;
        const int width = (int)a.max_pages;
        const uint32_t pool = (uint32_t)a.num_pages;
        const bool paired = a.page_size % kTile == 0;         // a tile's halves lie on one page
        auto row_of = [&]() {
            if (page_i >= first_page + 64) {
                first_page = page_i;
                const int i = page_i + lane;
                pages = table[min(i, width - 1)];
                if (i >= width) pages = -1;
            }
            const int page = __builtin_amdgcn_readlane(pages, page_i - first_page);
            return (uint32_t)page < pool ? page * a.page_size + off : -1;
        };
        auto advance = [&](int by) {
            off += by;
            const int wrap = off == a.page_size;
            off = wrap ? 0 : off;
            page_i += wrap;
        };
        auto place = [&]() {
            Place p;
            p.row[0] = row_of();
            if (paired) {
                p.row[1] = p.row[0] < 0 ? -1 : p.row[0] + 16;
                advance(32);
            } else {
                advance(16);
                p.row[1] = row_of();
                advance(16);
            }
            return p;
        };
        const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
        auto compute = [&](int t, const Place& here, uint32_t stage) {
            const uint8_t* lk = mine + stage + own.read_key;
            uint32_t kw[2][D / 32], kscale[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (D == 64) {
                    const u32x2 x = *reinterpret_cast<const u32x2*>(lk + h * 16 * S::kChunks * 16);
                    kw[h][0] = x[0], kw[h][1] = x[1];
                } else {
#pragma unroll
                    for (int i = 0; i < D / 128; ++i) {
                        const uint32_t at = i ? (own.read_key ^ 16) - own.read_key : 0;     // chunk 2g + 1 beside 2g
                        const u32x4 x = *reinterpret_cast<const u32x4*>(lk + (int32_t)at + h * 16 * S::kChunks * 16);
#pragma unroll
                        for (int w = 0; w < 4; ++w) kw[h][4 * i + w] = x[w];
                    }
                }
                kscale[h] = *reinterpret_cast<const uint32_t*>(mine + stage + own.read_ks + 64 * h);
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
            for (int h = 0; h < 2; ++h) vscale[h] = *reinterpret_cast<const u32x4*>(mine + stage + own.read_vs + 64 * h);
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
                const uint8_t* x = mine + stage + own.read_value + j * 2 * D;
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
            // Three stages and the places of their tiles take turns, by unrolling.
            Place at_stage[kStages];
            auto start = [&](int k) {
                at_stage[k] = place();
                copy_tile<D>(a, at_stage[k], own, lane, lds + k * S::kBytes);
            };
            auto turn = [&](int t, auto tag) {
                constexpr int k = decltype(tag)::value;
                if (t + 2 < t1) {
                    start((k + 2) % kStages);
                    wait_copies<2 * S::kCopies>();
                } else if (t + 1 < t1) {
                    wait_copies<S::kCopies>();
                } else {
                    wait_copies<0>();
                }
                compute(t, at_stage[k], k * S::kBytes);
            };
            start(0);
            if (t0 + 1 < t1) start(1);
            for (int t = t0; t < t1; t += 3) {
                turn(t, Int<0>());
                if (t + 1 < t1) turn(t + 1, Int<1>());
                if (t + 2 < t1) turn(t + 2, Int<2>());
            }
            wait_lds();                                       // before the next sequence's copies
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
    int nr, waves, columns, ranges;        // row tiles per wave, waves per workgroup, workgroups per range
};
Layout layout_of(int64_t batch, int drafts, int q_heads, int kv_heads, int head_dim) {
    const int rows = drafts * (q_heads / kv_heads);
    Layout l;
    l.nr = rows > 16 && head_dim <= 128 ? 2 : 1;
    const int units = kv_heads * ((rows + 16 * l.nr - 1) / (16 * l.nr));
    l.waves = units < kWaves ? units : kWaves;
    l.columns = (units + l.waves - 1) / l.waves;
    int64_t ranges = (int64_t)kWorkgroups * kWaves / ((int64_t)l.columns * l.waves);
    // a multiple of 8, so that a range's workgroups meet on one XCD
    ranges = ranges / 8 * 8;
    l.ranges = (int)(ranges < 8 ? 8 : ranges);
    (void)batch;
    return l;
}

template <int D, int NR>
hipError_t launch(const TreeArgs& a, const Layout& l, hipStream_t s) {
    attn_tree_kernel<D, NR><<<dim3((unsigned)l.ranges, (unsigned)l.columns), 64 * l.waves, 0, s>>>(a);
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

}  // namespace

size_t attn_tree_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads) {
    const Layout l = layout_of(batch, drafts, q_heads, kv_heads, head_dim);
    return (size_t)2 * l.ranges * q_heads * drafts * (head_dim + 2) * sizeof(float);
}

hipError_t launch_attn_tree(const AttnTree& p, hipStream_t s) {
    const Layout l = layout_of(p.batch, p.drafts, p.q_heads, p.kv_heads, p.head_dim);
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
