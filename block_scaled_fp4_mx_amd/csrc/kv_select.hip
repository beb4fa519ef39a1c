// Selection of cache blocks by a cheap score.
//
//   s(t, n) = Q(q[t]) . E[page n],  the n_select complete blocks of largest s,
//   Q: MXFP4, E: one MXFP4 entry for every page of the pool.
//
// Scores: a wave takes 64 blocks of a sequence, 16 to a matrix instruction
// (v_mfma_scale_f32_16x16x128, entries times up to 16 drafted tokens), reading each
// entry once for all of them; lane (c = lane % 16, g = lane / 16) holds block g of a
// step's four blocks of 32 values of entry c, and quantizes the same block of query c
// for itself.  Scores go through the workspace, rows of blocks for each query.
//
// Selection: a workgroup takes one query.  Scores as ordered whole numbers, in
// registers; the threshold is found 8 bits at a time, by histograms of what still may
// hold it, from the highest bit in which the scores differ.  Its ties go to the lowest
// blocks: every wave has a run of neighbouring blocks, counts what it takes, and writes
// it in order behind what the waves before it take.  No order of atomics shows.
//
// Bound by latency: the entries of 64 contexts of 131072 tokens are 9 MB.
#include "fp4_internal.h"
#include "mma_core.h"
#include "quant_device.h"

namespace fp4 {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves, kHeld = 16;
constexpr int kTilesPerWave = 4, kScoreWaves = 4, kScoreSpan = 16 * kTilesPerWave * kScoreWaves;

struct SelectArgs {
    const uint16_t* q;
    int64_t ld_q;
    const uint8_t *codes, *scales;
    int64_t num_pages;
    int lists, dim;
    const int32_t* table;
    int64_t max_pages, pitch;              // pitch: of a query's scores in the workspace
    const int32_t *seq_lens, *draft_lens;
    int page_size, drafts;
    int select, n_first, n_recent;
    int32_t* ids;
    float* out_scores;                     // or NULL
    float* scores;
};

__device__ __forceinline__ int complete_blocks(const SelectArgs& a, int b) {
    return (int)min((int64_t)(max(a.seq_lens[b], 0) / a.page_size), a.max_pages);
}

// 32 values of one lane as a block: codes and the scale byte.
__device__ __forceinline__ uint4 quant32(const uint16_t* x, int& byte) {
    const uint4* p = reinterpret_cast<const uint4*>(x);
    uint32_t w[4][4], amax = 0, code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 v = p[i];
        w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
        amax = max(amax, mag_max8(w[i]));
    }
    byte = (int)mx_scale_byte(amax);
    const float sc = __uint_as_float((uint32_t)byte << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t c = 0;
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[i][0]), sc, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[i][1]), sc, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[i][2]), sc, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, w[i][3]), sc, 3);
        code[i] = c;
    }
    return make_uint4(code[0], code[1], code[2], code[3]);
}

// Workgroup (x, y, z): blocks from x * kScoreSpan on, list y, sequence z.  A block
// without a page gets no number, one whose score is none the lowest.
__global__ __launch_bounds__(64 * kScoreWaves) void select_scores_kernel(const SelectArgs a) {
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
    const int b = blockIdx.z, list = blockIdx.y;
    const int complete = complete_blocks(a, b);
    const int64_t n0 = (int64_t)blockIdx.x * kScoreSpan + wave * (16 * kTilesPerWave);
    if (n0 >= complete || a.num_pages == 0) return;
    const int page = n0 + lane < complete ? a.table[(int64_t)b * a.max_pages + n0 + lane] : -1;
    const int valid = (uint32_t)page < (uint32_t)a.num_pages ? page : -1;
    const int blocks = a.dim / 32, per_row = a.lists * blocks;
    for (int t0 = 0; t0 < a.drafts; t0 += 16) {
        v4f acc[kTilesPerWave];
#pragma unroll
        for (int k = 0; k < kTilesPerWave; ++k) acc[k] = v4f{0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < blocks; k0 += 4) {
            const bool in = k0 + g < blocks;
            uint4 q = make_uint4(0, 0, 0, 0);
            int q_scale = 127;
            if (in && t0 + c < a.drafts)
                q = quant32(a.q + ((int64_t)b * a.drafts + t0 + c) * a.ld_q + (int64_t)list * a.dim + (k0 + g) * 32, q_scale);
            uint4 e[kTilesPerWave];
            int e_scale[kTilesPerWave];
#pragma unroll
            for (int k = 0; k < kTilesPerWave; ++k) {
                const int row = max(__shfl(valid, 16 * k + c, 64), 0);
                e[k] = make_uint4(0, 0, 0, 0), e_scale[k] = 127;
                if (in) {
                    const int64_t at = (int64_t)row * per_row + list * blocks + k0 + g;
                    e[k] = reinterpret_cast<const uint4*>(a.codes)[at];
                    e_scale[k] = a.scales[at];
                }
            }
            const v8i qv = {(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < kTilesPerWave; ++k) {
                const v8i ev = {(int)e[k].x, (int)e[k].y, (int)e[k].z, (int)e[k].w, 0, 0, 0, 0};
                acc[k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ev, qv, acc[k], 4, 4, 0, e_scale[k], 0, q_scale);
            }
        }
        // Lane (c, g) has blocks 4g .. 4g + 3 of each tile for query c.
#pragma unroll
        for (int k = 0; k < kTilesPerWave; ++k) {
            float s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool there = __shfl(valid, 16 * k + 4 * g + i, 64) >= 0;
                s[i] = !there ? __builtin_nanf("") : acc[k][i] == acc[k][i] ? acc[k][i] + 0.0f : -__builtin_inff();
            }
            if (t0 + c < a.drafts && n0 + 16 * k < complete) {
                const int64_t row = ((int64_t)b * a.drafts + t0 + c) * a.lists + list;
                *reinterpret_cast<float4*>(a.scores + row * a.pitch + n0 + 16 * k + 4 * g) = make_float4(s[0], s[1], s[2], s[3]);
            }
        }
    }
}

// A score's place in the order of all: 0 no block, the last one a block that is taken
// before any other.
constexpr uint32_t kTaken = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t key_of(float s) {
    if (!(s == s)) return 0;
    const uint32_t u = __float_as_uint(s);
    return u >> 31 ? ~u : u | 0x80000000u;
}

// Workgroup x: query x (token and list).  kInRegisters: at most kThreads * kHeld blocks;
// otherwise the scores are read again where they are needed.
template <bool kInRegisters>
__global__ __launch_bounds__(kThreads) void select_blocks_kernel(const SelectArgs a) {
    __shared__ uint32_t hist[256], found[3];
    __shared__ int sums[kWaves][4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x;
    const int64_t token = row / a.lists;
    const int b = (int)(token / a.drafts), t = (int)(token - (int64_t)b * a.drafts);
    if (a.draft_lens && t >= a.draft_lens[b]) return;
    const int complete = a.num_pages ? complete_blocks(a, b) : 0;
    const float* scores = a.scores + row * a.pitch;
    // A wave's blocks: steps of 64 from start on.
    const int steps = (complete + kThreads - 1) / kThreads, start = wave * steps * 64;
    auto load = [&](int j) -> uint32_t {
        const int n = start + 64 * j + lane;
        if (j >= steps || n >= complete) return 0;
        const uint32_t k = key_of(scores[n]);
        return k && (n < a.n_first || n >= complete - a.n_recent) ? kTaken : k;
    };
    uint32_t held[kInRegisters ? kHeld : 1];
    if constexpr (kInRegisters) {
#pragma unroll
        for (int j = 0; j < kHeld; ++j) held[j] = load(j);
    }
    auto each = [&](auto f) {
        if constexpr (kInRegisters) {
#pragma unroll
            for (int j = 0; j < kHeld; ++j)
                if (j < steps) f(j, held[j]);
        } else {
            for (int j = 0; j < steps; ++j) f(j, load(j));
        }
    };

    int blocks = 0, taken = 0;
    uint32_t low = kTaken, high = 0;
    each([&](int, uint32_t k) {
        blocks += __popcll(__ballot(k != 0));
        taken += __popcll(__ballot(k == kTaken));
        if (k != 0 && k != kTaken) low = min(low, k), high = max(high, k);
    });
#pragma unroll
    for (int m = 1; m < 64; m *= 2) low = min(low, (uint32_t)__shfl_xor(low, m, 64)), high = max(high, (uint32_t)__shfl_xor(high, m, 64));
    if (lane == 0) sums[wave][0] = blocks, sums[wave][1] = taken, sums[wave][2] = (int)low, sums[wave][3] = (int)high;
    __syncthreads();
    blocks = taken = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        blocks += sums[w][0], taken += sums[w][1];
        low = min(low, (uint32_t)sums[w][2]), high = max(high, (uint32_t)sums[w][3]);
    }
    __syncthreads();

    // Blocks above the threshold are taken, and the first `ties` of those on it.
    uint32_t threshold = 0;
    int ties = 0;
    if (blocks > a.select) {
        int need = a.select - taken;
        if (need <= 0) {
            threshold = kTaken, ties = a.select;
        } else {
            // Scores less low; the threshold's bits from `bits` on are `prefix`.
            int bits = high > low ? 32 - __clz((int)(high - low)) : 0;
            uint32_t prefix = 0;
            threshold = low, ties = need;
            while (bits > 0) {
                const int shift = max(bits - 8, 0);
                if (threadIdx.x < 256) hist[threadIdx.x] = 0;
                __syncthreads();
                each([&](int, uint32_t k) {
                    const uint32_t d = k - low;
                    if (k != 0 && k != kTaken && (uint64_t)d >> bits == prefix) atomicAdd(&hist[d >> shift & 255], 1u);
                });
                __syncthreads();
                if (wave == 0) {                              // a lane has four digits, the last lane the highest
                    uint32_t own[4], above = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) own[i] = hist[4 * lane + i], above += own[i];
                    const uint32_t mine = above;
#pragma unroll
                    for (int m = 1; m < 64; m *= 2) {
                        const uint32_t o = __shfl_down(above, m, 64);
                        if (lane + m < 64) above += o;
                    }
                    above -= mine;                            // of the lanes behind
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        if (above < (uint32_t)need && above + own[i] >= (uint32_t)need)
                            found[0] = 4 * lane + i, found[1] = above, found[2] = own[i];
                        above += own[i];
                    }
                }
                __syncthreads();
                need -= (int)found[1];
                prefix = prefix << (bits - shift) | found[0];
                bits = shift;
                threshold = low + (prefix << shift), ties = need;
                if ((int)found[2] == need) {                  // all that begin so are taken
                    --threshold, ties = 0;
                    break;
                }
            }
        }
    }

    int above = 0, equal = 0;
    each([&](int, uint32_t k) {
        above += __popcll(__ballot(k > threshold));
        equal += __popcll(__ballot(k != 0 && k == threshold));
    });
    if (lane == 0) sums[wave][0] = above, sums[wave][1] = equal;
    __syncthreads();
    above = equal = 0;
    for (int w = 0; w < wave; ++w) above += sums[w][0], equal += sums[w][1];
    int at = above + min(equal, ties);
    const uint64_t before = (1ull << lane) - 1;
    int32_t* ids = a.ids + row * a.select;
    each([&](int j, uint32_t k) {
        const bool on = k != 0 && k == threshold;
        const uint64_t equals = __ballot(on);
        const bool take = k > threshold || (on && equal + __popcll(equals & before) < ties);
        const uint64_t takes = __ballot(take);
        if (take) {
            const int to = at + __popcll(takes & before), n = start + 64 * j + lane;
            ids[to] = n;
            if (a.out_scores) a.out_scores[row * a.select + to] = scores[n];
        }
        equal += __popcll(equals), at += __popcll(takes);
    });
    for (int i = min(blocks, a.select) + (int)threadIdx.x; i < a.select; i += kThreads) {
        ids[i] = -1;
        if (a.out_scores) a.out_scores[row * a.select + i] = -__builtin_inff();
    }
}

int64_t pitch_of(int64_t max_pages) { return (max_pages + 15) / 16 * 16; }

}  // namespace

size_t kv_select_workspace_bytes(int64_t batch, int drafts, int lists, int64_t max_pages) {
    return (size_t)batch * drafts * lists * pitch_of(max_pages) * sizeof(float);
}

hipError_t launch_kv_select(const KvSelect& p, hipStream_t s) {
    SelectArgs a{};
    a.q = p.q, a.ld_q = p.ld_q, a.codes = p.codes, a.scales = p.scales, a.num_pages = p.num_pages;
    a.lists = p.lists, a.dim = p.dim, a.table = p.page_table, a.max_pages = p.max_pages, a.pitch = pitch_of(p.max_pages);
    a.seq_lens = p.seq_lens, a.draft_lens = p.draft_lens, a.page_size = (int)p.page_size, a.drafts = p.drafts;
    a.select = p.n_select, a.n_first = p.n_first, a.n_recent = p.n_recent;
    a.ids = p.ids, a.out_scores = p.out_scores, a.scores = static_cast<float*>(p.ws);
    if (p.max_pages && p.num_pages) {
        const dim3 grid((unsigned)((p.max_pages + kScoreSpan - 1) / kScoreSpan), (unsigned)p.lists, (unsigned)p.batch);
        select_scores_kernel<<<grid, 64 * kScoreWaves, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const unsigned rows = (unsigned)(p.batch * p.drafts * p.lists);
    if (p.max_pages <= kThreads * kHeld)
        select_blocks_kernel<true><<<rows, kThreads, 0, s>>>(a);
    else
        select_blocks_kernel<false><<<rows, kThreads, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fp4
