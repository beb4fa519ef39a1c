// Causal attention over packed prompts.
//
//   o_i = sum_{j<=i} 2^(c s_ij - m_i) v_j / sum_{j<=i} 2^(c s_ij - m_i),
//   s_ij = q_i . k_j,  c = scale * log2(e), in one pass over the keys.
//
// A workgroup of 4 waves (8 at D = 256) takes 32 consecutive rows a wave of one
// sequence and one query head, against tiles of kTokens keys and values in LDS, all
// on v_mfma_f32_32x32x16_bf16:
//   S^T = K Q^T: lane (c = lane % 32, h = lane / 32) ends with query row c and
//   tokens 8i + 4h .. 8i + 4h+3 of each 32, so a row's maximum and sum are lane
//   local but for one exchange, and the weights are the B operand of
//   O^T = V^T P^T as they stand (its token order is free as long as V^T is read
//   alike);
//   V^T: transposing LDS reads (ds_read_b64_tr_b16): 4 tokens of one value.
// The running reference m moves only when a score exceeds it by more than 2^8.
// Weights are rounded to bf16 for the second product (they enter it with V's
// 16-bit format); the rounded weights are what is summed, in fp32.
//
// Bound by the matrix core (4 D flop per visible pair and query head).  A call among
// others:
//   16384 rows, 32 / 4 heads of 128 values: 1.93 .. 2.05 ms from card to card, 1.07 ..
//   1.14 PFLOP/s (a large library product reaches 1.37); matrix cores busy 59% of the
//   cycles, at a clock that falls to 1.75 GHz under this load, the rest the exponentials
//   and sums, which two waves on a SIMD overlap in part.  Heads of 64: 1.12 ms, 0.99
//   PFLOP/s; of 256: 3.54 ms, 1.24 PFLOP/s;
//   4 prompts of 7676 rows in all, 64 / 8 heads: 292 .. 295 us, 0.84 PFLOP/s (traced one
//   call after another 290 .. 360), matrix cores busy 45%: a workgroup starts with a cold
//   query and first tile, and has 17 tiles on average to make up for it;
//   24 prompts of 3 .. 421 rows, 16 / 16 heads of 64: 13 us, one round of workgroups.
// Tried and slower or alike: tiles loaded through registers into padded LDS rows (2.41
// ms), interleaving the two halves' products, s_setprio around them.
#include "fp4_internal.h"
#include "mma_core.h"

namespace fp4 {
namespace {

// Waves of a workgroup, 32 query rows each.  8 waves (256 rows) at D = 256 keep two
// waves per SIMD in 256 registers (and 6 spilled ones), where 4 take 420; below, 4 and 8
// measured alike (16384 rows: 2.04 and 1.97 ms; four documents of 8k rows in all: 341
// and 357 us).
constexpr int waves_of(int head_dim) { return head_dim == 256 ? 8 : 4; }
constexpr float kSlack = 8.0f;
constexpr float kNone = -__builtin_inff();   // score of a hidden token
constexpr float kFloor = -3e38f;           // reference before the first tile

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

struct PromptArgs {
    const uint16_t *q, *k, *v;
    uint16_t* out;
    int64_t ld_q, ld_k, ld_v, ld_out;
    const int32_t* cu;
    int seqs, q_heads, group, tiles;       // tiles: workgroups per query head
    int64_t tokens;
    float scale2;                          // |scale| * log2(e), positive
    uint32_t flip;                         // sign bits of Q, set for a negative scale
};

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

typedef __attribute__((address_space(3))) uint8_t* lds_bytes;

// A tile of keys and one of values in LDS, rows of D values without padding.  They
// come straight from global memory (each of the W waves copies its share, 16 bytes
// a lane, 1 KiB an instruction), so rows are spread over the 64 banks by where a
// 16-byte chunk is put: chunk x of key row r at x ^ key_turn(r), which keeps the 16
// lanes that read one chunk of 16 rows apart, and of value row r at x ^
// value_turn(r), which does so for the 4 rows of 64 bytes that half the lanes of a
// transposing read take (256 bytes a cycle).
template <int D>
struct Shape {
    static constexpr int W = waves_of(D);
    static constexpr int kRows = 32 * W;                     // query rows of a workgroup
    static constexpr int kTokens = D == 256 ? 32 : 64;       // keys of a tile
    static constexpr int kRow = 2 * D, kTile = kTokens * kRow;           // bytes
    static constexpr int kCopies = kTile / 1024 / W;            // of keys, and of values, per wave
    static constexpr int kPerCopy = 1024 / kRow;             // rows
    __device__ static constexpr int key_turn(int row) { return D == 64 ? (row >> 1) & 7 : row & 15; }
    __device__ static constexpr int value_turn(int row) { return D == 64 ? 4 * ((row >> 1) & 1) : 4 * (row & 3); }
};

// A wave's copies of one tile, into LDS at keys and values; k and v: where the
// tile's first rows lie, less 1024 (kCopies - 1), which the lane offsets carry (the
// instruction's offset counts on both sides).  Awaited by wait_copies.
template <int kCopies>
__device__ __forceinline__ void copy_tile(const uint8_t* k, const uint8_t* v, const uint32_t* ko, const uint32_t* vo,
                                          uint32_t keys, uint32_t values) {
    if constexpr (kCopies == 1) {
        asm volatile(
            "s_mov_b32 m0, %4\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %0, %2\n\t"
            "s_mov_b32 m0, %5\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %1, %3" ::"v"(ko[0]),
            "v"(vo[0]), "s"(k), "s"(v), "s"(keys), "s"(values)
            : "memory", "m0");
    } else if constexpr (kCopies == 2) {
        asm volatile(
            "s_mov_b32 m0, %6\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %0, %4\n\t"
            "global_load_lds_dwordx4 %1, %4 offset:1024\n\t"
            "s_mov_b32 m0, %7\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %2, %5\n\t"
            "global_load_lds_dwordx4 %3, %5 offset:1024" ::"v"(ko[0]),
            "v"(ko[1]), "v"(vo[0]), "v"(vo[1]), "s"(k), "s"(v), "s"(keys), "s"(values)
            : "memory", "m0");
    } else {
        asm volatile(
            "s_mov_b32 m0, %10\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %0, %8\n\t"
            "global_load_lds_dwordx4 %1, %8 offset:1024\n\t"
            "global_load_lds_dwordx4 %2, %8 offset:2048\n\t"
            "global_load_lds_dwordx4 %3, %8 offset:3*1024\n\t"
            "s_mov_b32 m0, %11\n\ts_nop 0\n\t"
            "global_load_lds_dwordx4 %4, %9\n\t"
            "global_load_lds_dwordx4 %5, %9 offset:1024\n\t"
            "global_load_lds_dwordx4 %6, %9 offset:2048\n\t"
            "global_load_lds_dwordx4 %7, %9 offset:3*1024" ::"v"(ko[0]),
            "v"(ko[1]), "v"(ko[2]), "v"(ko[3]), "v"(vo[0]), "v"(vo[1]), "v"(vo[2]), "v"(vo[3]), "s"(k), "s"(v), "s"(keys),
            "s"(values)
            : "memory", "m0");
    }
}
// This wave's copies have landed and its LDS reads have returned, then all waves'.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// sum + the products of two pairs of bf16, in fp32.
__device__ __forceinline__ float add_products(float sum, uint32_t a, uint32_t b) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), sum, false);
}
__device__ __forceinline__ float add_pair(float sum, uint32_t pair) { return add_products(sum, pair, 0x3F803F80u); }

// First row of sequence s.  Its row tiles are numbered from row_of(s) / kRows + s
// on, which leaves every sequence enough of them and needs no table of lengths.
__device__ __forceinline__ int row_of(const PromptArgs& a, int s) {
    return min(max(a.cu[s], 0), (int)a.tokens);
}

template <int D>
__global__ __launch_bounds__(64 * waves_of(D), 2) void attn_prompt_kernel(const PromptArgs a) {
    using S = Shape<D>;
    constexpr int kRows = S::kRows, kTokens = S::kTokens, kSteps = D / 16, kOut = D / 32, kSub = kTokens / 32, kBatch = kSteps < 8 ? kSteps : 8;
    __shared__ __attribute__((aligned(16))) uint8_t tiles_lds[2 * 2 * S::kTile];        // keys, values; twice
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), c = lane & 31, h = lane >> 5;

    // Query heads of one key/value head meet on one XCD (workgroups are dealt to
    // the 8 XCDs in turn); late row tiles, which see the most keys, come first.
    int head, x;
    if (a.q_heads % 8 == 0) {
        const int per = a.q_heads / 8, i = blockIdx.x / 8;
        head = (int)(blockIdx.x % 8) * per + i % per;
        x = a.tiles - 1 - i / per;
    } else {
        head = blockIdx.x % a.q_heads;
        x = a.tiles - 1 - blockIdx.x / a.q_heads;
    }
    // The last sequence whose tiles start at or before x: 64 candidates at once, a
    // bound to a lane, after halving for larger batches.
    int lo = 0, hi = a.seqs;
    while (hi - lo > 64) {
        const int mid = (lo + hi) / 2;
        if (row_of(a, mid) / kRows + mid <= x)
            lo = mid;
        else
            hi = mid;
    }
    const int at = min(lo + lane, a.seqs);
    const int first = (int)row_of(a, at), behind = (int)row_of(a, min(at + 1, a.seqs));
    const int seq = __popcll(__ballot(lo + lane < hi && first / kRows + at <= x)) - 1;
    if (seq < 0) return;
    const int64_t start = __builtin_amdgcn_readlane(first, seq), end = __builtin_amdgcn_readlane(behind, seq);
    const int64_t q0 = (x - (start / kRows + lo + seq)) * kRows, len = end - start;
    if (q0 < 0 || q0 >= len) return;

    const int kv = head / a.group;
    const uint8_t* kg = reinterpret_cast<const uint8_t*>(a.k + start * a.ld_k + (int64_t)kv * D);
    const uint8_t* vg = reinterpret_cast<const uint8_t*>(a.v + start * a.ld_v + (int64_t)kv * D);
    const uint32_t lds = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(lds_bytes)tiles_lds);

    // Where this lane's chunks of a tile lie; rows behind the sequence are read as
    // its last one (hidden by the mask, and finite).
    uint32_t ko[S::kCopies], vo[S::kCopies];
    auto offsets = [&](int rows) {
#pragma unroll
        for (int i = 0; i < S::kCopies; ++i) {
            const int r = (wave * S::kCopies + i) * S::kPerCopy + lane / (D / 8), at = lane % (D / 8);
            const uint32_t pad = 1024 * (S::kCopies - 1 - i), from = min(r, rows - 1);
            ko[i] = from * (uint32_t)(2 * a.ld_k) + (at ^ S::key_turn(r)) * 16 + pad;
            vo[i] = from * (uint32_t)(2 * a.ld_v) + (at ^ S::value_turn(r)) * 16 + pad;
        }
    };
    offsets(kTokens);
    const int last_row = (int)min(q0 + kRows, len) - 1, tiles = last_row / kTokens + 1;
    const uint8_t* next_k = kg - 1024 * (S::kCopies - 1);    // the next tile to copy
    const uint8_t* next_v = vg - 1024 * (S::kCopies - 1);
    const int64_t step_k = 2 * kTokens * a.ld_k, step_v = 2 * kTokens * a.ld_v;
    auto copy = [&](int t) {
        const int left = (int)len - t * kTokens;
        if (left < kTokens) offsets(left);                   // the sequence's last tile
        const uint32_t at = lds + (t & 1) * 2 * S::kTile + wave * S::kCopies * 1024;
        copy_tile<S::kCopies>(next_k, next_v, ko, vo, at, at + S::kTile);
        next_k += step_k, next_v += step_v;
    };
    copy(0);

    const int row = (int)q0 + 32 * wave + c;                 // this lane's query row
    const bool live = row < len;
    u32x4 q[kSteps];
    {
        const uint16_t* p = a.q + (start + (live ? row : 0)) * a.ld_q + (int64_t)head * D + 8 * h;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            q[s] = live ? *reinterpret_cast<const u32x4*>(p + 16 * s) : u32x4{0, 0, 0, 0};
            q[s] ^= a.flip;
        }
    }
    v16f o[kOut];
#pragma unroll
    for (int i = 0; i < kOut; ++i) o[i] = v16f{};
    float m = kFloor, sum[4] = {0.f, 0.f, 0.f, 0.f};         // sum: of the rounded weights, in four parts

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

    const int wave_first = (int)q0 + 32 * wave;
    bool apart = false;
    auto compute = [&](int t, const uint8_t* tile) {
        const int t0 = t * kTokens;
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
        if (t0 + kTokens - 1 > wave_first) {                 // the diagonal, in the wave's last tile
            // A weight of 0 does not hide a value that is infinite or no number.  The wave's
            // last tile holds its diagonal: if one of the tokens that some of its rows do
            // not see has such a value (a product with 0 tells), it is taken apart below.
            float odd = 0.f;
            for (int u = (wave_first - t0) / 32; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 32 * S::kRow / 1024; ++i) {
                    const u32x4 x = *reinterpret_cast<const u32x4*>(tile + S::kTile + 32 * u * S::kRow + 1024 * i + 16 * lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j) odd = add_products(odd, x[j], 0);
                }
            apart = __any(odd != 0.f);
            if (apart) return;
            const int d = row - t0;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    s[u][i] = 32 * u + 8 * (i / 4) + 4 * h + i % 4 > d ? kNone : s[u][i];
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
        // Every row sees token 0, so m is finite from the first tile on.
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = pack2(exp2_hw(fmaf(s[u][2 * i], a.scale2, -m)), exp2_hw(fmaf(s[u][2 * i + 1], a.scale2, -m)));
                sum[i & 3] = add_pair(sum[i & 3], p[i]);
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {                    // 16 tokens
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
    // When the waves meet, tile t is in LDS, and the other buffer is free.
    auto turn = [&](int t, const uint8_t* tile) {
        meet();
        if (t + 1 < tiles) copy(t + 1);
        if (t * kTokens <= wave_first + 31) compute(t, tile);    // else nothing of it is visible to the wave
    };
    int t = 0;
    for (; t + 2 <= tiles; t += 2) {
        turn(t, tiles_lds);
        turn(t + 1, tiles_lds + 2 * S::kTile);
    }
    if (t < tiles) turn(t, tiles_lds);

    if (apart) {                                             // one token at a time
#pragma unroll 1
        for (int token = wave_first / kTokens * kTokens; token <= min(wave_first + 31, (int)len - 1); ++token) {
            const uint8_t* x = kg + (int64_t)token * 2 * a.ld_k + 16 * h;
            float score = 0.f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const u32x4 w = *reinterpret_cast<const u32x4*>(x + 32 * s);
#pragma unroll
                for (int j = 0; j < 4; ++j) score = add_products(score, w[j], q[s][j]);
            }
            score += __shfl_xor(score, 32, 64);
            const bool see = token <= row;
            const float top = see ? score * a.scale2 : m, up = fmaxf(m, top), alpha = exp2_hw(m - up);
            const uint32_t weight = pack2(see ? exp2_hw(fmaf(score, a.scale2, -up)) : 0.f, 0.f);
            const float p = bf16_lo(weight);
            m = up;
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] *= alpha;
            sum[0] += h ? 0.f : p;
            const uint8_t* y = vg + (int64_t)token * 2 * a.ld_v + 8 * h;
#pragma unroll
            for (int i = 0; i < 4 * kOut; ++i) {
                const uint2 w = *reinterpret_cast<const uint2*>(y + 16 * i);
                const float v[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float old = o[i / 4][4 * (i % 4) + j] * alpha;
                    o[i / 4][4 * (i % 4) + j] = see ? fmaf(p, v[j], old) : old;
                }
            }
        }
    }

    float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    total += __shfl_xor(total, 32, 64);
    const float inv = 1.0f / total;
    // Lanes (c, 0) and (c, 1) hold alternate fours of values: they exchange a four of
    // every pair of eights, and each stores one eight.
    uint16_t* y = a.out + (start + row) * a.ld_out + (int64_t)head * D + 8 * h;
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            uint32_t w[2][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const auto x = __builtin_amdgcn_permlane32_swap(
                    pack2(o[i][4 * j + 2 * k] * inv, o[i][4 * j + 2 * k + 1] * inv),
                    pack2(o[i][4 * j + 4 + 2 * k] * inv, o[i][4 * j + 4 + 2 * k + 1] * inv), false, false);
                w[0][k] = x[0], w[1][k] = x[1];
            }
            if (live) *reinterpret_cast<uint4*>(y + 32 * i + 8 * j) = make_uint4(w[0][0], w[0][1], w[1][0], w[1][1]);
        }
}

}  // namespace

// Row tiles per query head: the tile numbers of attn_prompt_kernel.
int64_t attn_prompt_tiles(int64_t seqs, int64_t tokens, int head_dim) { return tokens / (32 * waves_of(head_dim)) + seqs; }

hipError_t launch_attn_prompt(const AttnPrompt& p, hipStream_t s) {
    PromptArgs a{};
    a.q = p.q, a.k = p.k, a.v = p.v, a.out = p.out;
    a.ld_q = p.ld_q, a.ld_k = p.ld_k, a.ld_v = p.ld_v, a.ld_out = p.ld_out;
    a.cu = p.cu_seqlens, a.seqs = (int)p.seqs, a.q_heads = p.q_heads, a.group = p.q_heads / p.kv_heads;
    a.tokens = p.tokens, a.tiles = (int)attn_prompt_tiles(p.seqs, p.tokens, p.head_dim);
    // Never 0: a hidden score is -inf and has to stay that when scaled.
    a.scale2 = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-37f);
    a.flip = p.scale < 0 ? 0x80008000u : 0u;
    const unsigned grid = (unsigned)((int64_t)a.tiles * p.q_heads);
    const unsigned threads = 64 * waves_of(p.head_dim);
    if (p.head_dim == 64)
        attn_prompt_kernel<64><<<grid, threads, 0, s>>>(a);
    else if (p.head_dim == 128)
        attn_prompt_kernel<128><<<grid, threads, 0, s>>>(a);
    else
        attn_prompt_kernel<256><<<grid, threads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fp4
