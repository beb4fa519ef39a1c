// Causal attention over packed prompts.
//
//   o_i = sum_{j<=i} 2^(c s_ij - m_i) v_j / sum_{j<=i} 2^(c s_ij - m_i),
//   s_ij = q_i . k_j,  c = scale * log2(e), in one pass over the keys.
//
// Bound by the matrix core (4 D flop per visible pair and query head).  A
// workgroup of 4 waves takes 128 consecutive rows of one sequence and one query
// head; a wave takes 32 of them against tiles of kTokens keys in LDS, all on
// v_mfma_f32_32x32x16_bf16:
//   S^T = K Q^T: lane (c = lane % 32, h = lane / 32) ends with query row c and
//   tokens 8i + 4h .. 8i + 4h+3 of each 32, so a row's maximum and sum are lane
//   local but for one exchange, and the weights are the B operand of
//   O^T = V^T P^T as they stand (its token order is free as long as V^T is read
//   alike);
//   V^T: transposing LDS reads (ds_read_b64_tr_b16): 4 tokens of one value.
// The running reference m moves only when a score exceeds it by more than 2^8.
// Weights are rounded to bf16 for the second product; their sum stays fp32.
#include "fp4_internal.h"
#include "mma_core.h"

namespace fp4 {
namespace {

constexpr int kRows = 128;                 // query rows of a workgroup
constexpr int kThreads = 256;
constexpr float kSlack = 8.0f;
constexpr float kNone = -__builtin_inff();

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

template <int D>
struct Shape {
    static constexpr int kTokens = D == 256 ? 32 : 64;       // keys of a tile
    // Row pitches in LDS (bf16 values), off the multiples of the 64 banks so that
    // the rows that one instruction reads fall into different banks.
    static constexpr int kPitchK = D + 8;
    static constexpr int kPitchV = D + 16;
    static constexpr int kChunks = kTokens * D / 8 / kThreads;   // 16-byte chunks per lane and tile
};

// Sequences that start at or before tile x of the row tiles: tile numbers of
// sequence s run from cu[s] / kRows + s on, which leaves every sequence enough of
// them and needs no table of lengths.
__device__ __forceinline__ int64_t row_of(const PromptArgs& a, int s) {
    return min(max((int64_t)a.cu[s], (int64_t)0), a.tokens);
}

template <int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attn_prompt_kernel(const PromptArgs a) {
    using S = Shape<D>;
    constexpr int kTokens = S::kTokens, kSteps = D / 16, kOut = D / 32, kSub = kTokens / 32;
    __shared__ __attribute__((aligned(16))) uint16_t lk[2][kTokens * S::kPitchK];
    __shared__ __attribute__((aligned(16))) uint16_t lv[2][kTokens * S::kPitchV];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane & 31, h = lane >> 5;

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
    int lo = 0, hi = a.seqs - 1;
    while (lo < hi) {                                        // last sequence whose tiles start at or before x
        const int mid = (lo + hi + 1) / 2;
        if (row_of(a, mid) / kRows + mid <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int64_t start = row_of(a, lo), end = row_of(a, lo + 1);
    const int64_t q0 = (x - (start / kRows + lo)) * kRows, len = end - start;
    if (q0 < 0 || q0 >= len) return;

    const int kv = head / a.group;
    const uint16_t* kg = a.k + start * a.ld_k + (int64_t)kv * D;
    const uint16_t* vg = a.v + start * a.ld_v + (int64_t)kv * D;
    const int64_t row = q0 + 32 * wave + c;                  // this lane's query row
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
    float m = kNone, sum = 0.f;

    u32x4 sk[S::kChunks], sv[S::kChunks];
    auto fetch = [&](int64_t t0) {
#pragma unroll
        for (int i = 0; i < S::kChunks; ++i) {
            const int chunk = i * kThreads + threadIdx.x, r = chunk / (D / 8), col = chunk % (D / 8) * 8;
            const bool in = t0 + r < len;                    // behind the sequence: zeros, whatever lies there
            sk[i] = in ? *reinterpret_cast<const u32x4*>(kg + (t0 + r) * a.ld_k + col) : u32x4{0, 0, 0, 0};
            sv[i] = in ? *reinterpret_cast<const u32x4*>(vg + (t0 + r) * a.ld_v + col) : u32x4{0, 0, 0, 0};
        }
    };
    auto store = [&](int buf) {
#pragma unroll
        for (int i = 0; i < S::kChunks; ++i) {
            const int chunk = i * kThreads + threadIdx.x, r = chunk / (D / 8), col = chunk % (D / 8) * 8;
            *reinterpret_cast<u32x4*>(&lk[buf][r * S::kPitchK + col]) = sk[i];
            *reinterpret_cast<u32x4*>(&lv[buf][r * S::kPitchV + col]) = sv[i];
        }
    };

    const int64_t last_row = min(q0 + kRows, len) - 1;
    const int64_t wave_first = q0 + 32 * wave;
    const int tiles = (int)(last_row / kTokens) + 1;
    fetch(0);
    store(0);
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
        const int buf = t & 1;
        const int64_t t0 = (int64_t)t * kTokens;
        if (t + 1 < tiles) fetch(t0 + kTokens);
        if (t0 <= wave_first + 31) {                         // else nothing of this tile is visible to the wave
            v16f s[kSub];
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                s[u] = v16f{};
                const uint16_t* p = &lk[buf][(32 * u + c) * S::kPitchK + 8 * h];
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
                    s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(p + 16 * i)),
                        __builtin_bit_cast(bf16x8, q[i]), s[u], 0, 0, 0);
            }
            if (t0 + kTokens - 1 > wave_first) {             // the diagonal
                const int d = (int)(row - t0);
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (32 * u + 8 * (i / 4) + 4 * h + i % 4 > d) s[u][i] = kNone;
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
                const float alpha = up == m ? 1.0f : exp2_hw(m - up);
                m = up;
                sum *= alpha;
#pragma unroll
                for (int i = 0; i < kOut; ++i) o[i] *= alpha;
            }
            // Every row sees token 0, so m is finite from the first tile on.
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                uint32_t p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a0 = exp2_hw(fmaf(s[u][2 * i], a.scale2, -m));
                    const float a1 = exp2_hw(fmaf(s[u][2 * i + 1], a.scale2, -m));
                    sum += a0 + a1;
                    p[i] = pack2(a0, a1);
                }
#pragma unroll
                for (int w = 0; w < 2; ++w) {                // 16 tokens
                    const bf16x8 pb = __builtin_bit_cast(bf16x8, u32x4{p[4 * w], p[4 * w + 1], p[4 * w + 2], p[4 * w + 3]});
                    const uint16_t* base = &lv[buf][(32 * u + 16 * w + 4 * h + (lane & 15) / 4) * S::kPitchV +
                                                    16 * ((lane >> 4) & 1) + 4 * (lane & 3)];
#pragma unroll
                    for (int i = 0; i < kOut; ++i) {
                        const v4s x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(base + 32 * i));
                        const v4s y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(base + 32 * i + 8 * S::kPitchV));
                        const bf16x8 va = __builtin_bit_cast(bf16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
                        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(va, pb, o[i], 0, 0, 0);
                    }
                }
            }
        }
        if (t + 1 < tiles) store(buf ^ 1);
        __syncthreads();
    }

    sum += __shfl_xor(sum, 32, 64);
    if (!live) return;
    const float inv = 1.0f / sum;
    uint16_t* y = a.out + (start + row) * a.ld_out + (int64_t)head * D + 4 * h;
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint2*>(y + 32 * i + 8 * j) =
                make_uint2(pack2(o[i][4 * j] * inv, o[i][4 * j + 1] * inv), pack2(o[i][4 * j + 2] * inv, o[i][4 * j + 3] * inv));
}

}  // namespace

// Workgroups per query head: the tile numbers of attn_prompt_kernel.
int64_t attn_prompt_tiles(int64_t seqs, int64_t tokens) { return tokens / kRows + seqs; }

hipError_t launch_attn_prompt(const AttnPrompt& p, hipStream_t s) {
    PromptArgs a{};
    a.q = p.q, a.k = p.k, a.v = p.v, a.out = p.out;
    a.ld_q = p.ld_q, a.ld_k = p.ld_k, a.ld_v = p.ld_v, a.ld_out = p.ld_out;
    a.cu = p.cu_seqlens, a.seqs = (int)p.seqs, a.q_heads = p.q_heads, a.group = p.q_heads / p.kv_heads;
    a.tokens = p.tokens, a.tiles = (int)attn_prompt_tiles(p.seqs, p.tokens);
    // Never 0: a hidden score is -inf and has to stay that when scaled.
    a.scale2 = fmaxf(fabsf(p.scale) * 1.4426950408889634f, 1e-37f);
    a.flip = p.scale < 0 ? 0x80008000u : 0u;
    const unsigned grid = (unsigned)((int64_t)a.tiles * p.q_heads);
    if (p.head_dim == 64)
        attn_prompt_kernel<64><<<grid, kThreads, 0, s>>>(a);
    else if (p.head_dim == 128)
        attn_prompt_kernel<128><<<grid, kThreads, 0, s>>>(a);
    else
        attn_prompt_kernel<256><<<grid, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fp4
