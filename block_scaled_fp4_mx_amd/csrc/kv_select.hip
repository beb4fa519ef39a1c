// Selection of cache blocks by a cheap score.
//
//   s(t, n) = Q(q[t]) . E[page n],  the n_select complete blocks of largest s,
//   Q: MXFP4, E: one MXFP4 entry for every page of the pool.
//
// Scores (select_scores_kernel): a wave takes 64 blocks of a sequence, 16 to a matrix
// instruction (v_mfma_scale_f32_16x16x128, entries times up to 16 drafted tokens),
// reading each entry once for all of them; lane (c = lane % 16, g = lane / 16) holds
// block g of a step's four blocks of 32 values of entry c, and quantizes the same block
// of query c for itself.  Scores go through the workspace, rows of blocks for each query.
//
// Selection: a workgroup takes one query (select_one_kernel, with the scores in
// registers, which it works out itself where that is faster; select_blocks_kernel, for
// more than 8192 blocks).  The threshold is found among the scores, ties go to the lowest
// blocks, and what is taken is written in the blocks' order: no order of atomics shows.
//
// Bound by latency: the entries of 64 contexts of up to 131072 tokens are 5 MB.  A call
// among others, on cold inputs: 4 queries for each of these 12.0 us (13.4 with neighbouring
// queries on different XCDs); one query over 1562 blocks 8.3 us, of which 4 are the read of
// its 64-byte entries by one CU; 8 lists over 12 contexts 8.7 us (10.6).  One query in two
// launches: over 1562 blocks of 256 values 10.5 us, of 512 12.9; over 4096 of 128 12.8, 7812
// 13.9; over 10937, whose scores are read again at every step by one workgroup, 41.
#include "fp4_internal.h"
#include "mma_core.h"
#include "quant_device.h"

namespace fp4 {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
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
    int64_t first_row;                     // of a launch that selects from the scores in the workspace
};

__device__ __forceinline__ int complete_blocks(const SelectArgs& a, int b) {
    return (int)min((int64_t)(max(a.seq_lens[b], 0) / a.page_size), a.max_pages);
}

// 32 values of one lane as a block: codes and the scale byte.
__device__ __forceinline__ uint4 quant32(const uint4 (&x)[4], int& byte) {
    uint32_t w[4][4], amax = 0, code[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i][0] = x[i].x, w[i][1] = x[i].y, w[i][2] = x[i].z, w[i][3] = x[i].w;
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

// A score in the order of scores: without a number the lowest, -0 as 0.
__device__ __forceinline__ float ranked(float s) { return s == s ? s + 0.0f : -__builtin_inff(); }

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
            if (in && t0 + c < a.drafts) {
                const uint4* x = reinterpret_cast<const uint4*>(a.q + ((int64_t)b * a.drafts + t0 + c) * a.ld_q +
                                                                (int64_t)list * a.dim + (k0 + g) * 32);
                const uint4 raw[4] = {x[0], x[1], x[2], x[3]};
                q = quant32(raw, q_scale);
            }
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
                s[i] = there ? ranked(acc[k][i]) : __builtin_nanf("");
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

// The threshold that `need` of the blocks are above or on, by 8 bits of the score at a
// time from the highest in which two differ; each(f) calls f(step, key) for all of a
// thread's blocks.  Blocks above it are taken, and the first `ties` on it.
struct Threshold {
    uint32_t key;
    int ties;
};
template <class Each>
__device__ __forceinline__ Threshold threshold_by_bits(uint32_t low, uint32_t high, int need, uint32_t* hist, volatile uint32_t* found,
                                                       int wave, int lane, Each each) {
    // Scores less low; the threshold's bits from `bits` on are `prefix`.
    int bits = high > low ? 32 - __clz((int)(high - low)) : 0;
    uint32_t prefix = 0;
    Threshold t{low, need};
    while (bits > 0) {
        const int shift = max(bits - 8, 0);
        if (threadIdx.x < 256) hist[threadIdx.x] = 0;
        __syncthreads();
        each([&](int, uint32_t k) {
            const uint32_t d = k - low;
            if (k != 0 && k != kTaken && (uint64_t)d >> bits == prefix) atomicAdd(&hist[d >> shift & 255], 1u);
        });
        __syncthreads();
        if (wave == 0) {                                      // a lane has four digits, the last lane the highest
            uint32_t own[4], above = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) own[i] = hist[4 * lane + i], above += own[i];
            const uint32_t mine = above;
#pragma unroll
            for (int m = 1; m < 64; m *= 2) {
                const uint32_t o = __shfl_down(above, m, 64);
                if (lane + m < 64) above += o;
            }
            above -= mine;                                    // of the lanes behind
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
        t = {low + (prefix << shift), need};
        if ((int)found[2] == need) return {t.key - 1, 0};     // all that begin so are taken
    }
    return t;
}

// Workgroup x: query first_row + x (token and list), from its scores in the workspace,
// which are read again where they are needed.
__global__ __launch_bounds__(kThreads) void select_blocks_kernel(const SelectArgs a) {
    __shared__ uint32_t hist[256], found[3];
    __shared__ int sums[kWaves][4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = a.first_row + blockIdx.x;
    const int64_t token = row / a.lists;
    const int b = (int)(token / a.drafts), t = (int)(token - (int64_t)b * a.drafts);
    if (a.draft_lens && t >= a.draft_lens[b]) return;
    const int complete = a.num_pages ? complete_blocks(a, b) : 0;
    const float* scores = a.scores + row * a.pitch;
    // A wave's blocks: steps of 64 from start on.
    const int steps = (complete + kThreads - 1) / kThreads, start = wave * steps * 64;
    auto each = [&](auto f) {
        for (int j = 0; j < steps; ++j) {
            const int n = start + 64 * j + lane;
            const uint32_t k = n < complete ? key_of(scores[n]) : 0;
            f(j, k && (n < a.n_first || n >= complete - a.n_recent) ? kTaken : k);
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

    Threshold top{0, 0};
    if (blocks > a.select) {
        if (taken >= a.select)
            top = {kTaken, a.select};
        else
            top = threshold_by_bits(low, high, a.select - taken, hist, found, wave, lane, each);
    }

    int above = 0, equal = 0;
    each([&](int, uint32_t k) {
        above += __popcll(__ballot(k > top.key));
        equal += __popcll(__ballot(k != 0 && k == top.key));
    });
    if (lane == 0) sums[wave][0] = above, sums[wave][1] = equal;
    __syncthreads();
    above = equal = 0;
    for (int w = 0; w < wave; ++w) above += sums[w][0], equal += sums[w][1];
    int at = above + min(equal, top.ties);
    const uint64_t before = (1ull << lane) - 1;
    int32_t* ids = a.ids + row * a.select;
    each([&](int j, uint32_t k) {
        const bool on = k != 0 && k == top.key;
        const uint64_t equals = __ballot(on);
        const bool take = k > top.key || (on && equal + __popcll(equals & before) < top.ties);
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

// Moves between lanes, as the DPP control words name them; lanes without a source keep
// `none`.
template <int kControl, int kRows = 0xF>
__device__ __forceinline__ uint32_t moved(uint32_t v, uint32_t none) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, kControl, kRows, 0xF, false);
}
// Smallest (largest) of the wave's values, in all lanes: within 16 lanes, then over the
// four rows of 16.
template <bool kMax>
__device__ __forceinline__ uint32_t extreme(uint32_t v) {
    auto pick = [](uint32_t x, uint32_t y) { return kMax ? max(x, y) : min(x, y); };
    v = pick(v, moved<0xB1>(v, v));                           // lane ^ 1
    v = pick(v, moved<0x4E>(v, v));                           // lane ^ 2
    v = pick(v, moved<0x141>(v, v));                          // the mirrored lane of 8
    v = pick(v, moved<0x140>(v, v));                          // the mirrored lane of 16
    return pick(pick(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
                pick(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}
// Sum of the values of a lane and those before it.
__device__ __forceinline__ uint32_t sum_upto(uint32_t v) {
    v += moved<0x111>(v, 0), v += moved<0x112>(v, 0), v += moved<0x114>(v, 0), v += moved<0x118>(v, 0);
    v += moved<0x142, 0xA>(v, 0);                             // the last lane of rows 0 and 2 to rows 1 and 3
    return v + moved<0x143, 0xC>(v, 0);                       // that of row 1 to rows 2 and 3
}

// Both steps for one query in one workgroup of 16 waves, at most kSteps * 1024 blocks of
// entries of at most 128 values: scores stay in registers, a block to a lane.  The query
// stands in all 16 rows of the matrix instruction, so that every lane group has the
// scores of a tile's 16 blocks, and group g keeps tile g's.  The threshold lies in one of 256 equal parts between the
// lowest and the highest score; where no more than kNear blocks lie there, each of them
// counts those before it in the order of scores and blocks, otherwise it is found by
// bits.
//
// What it waits for is one read after another (lengths, page table, entries), each round
// trip to memory 0.7 to 1.2 us, and the meetings of the waves: so everything that is
// known at the start is asked for at once, and the entries of all steps together.
constexpr int kOneWaves = 16, kOneThreads = 64 * kOneWaves, kParts = 256, kNear = 64;
// Workgroups are dealt to the 8 XCDs in turn: each XCD takes neighbouring queries, which
// read the same entries (drafted tokens) or parts of the same lines (lists).
__device__ __forceinline__ int query_of(int block, int blocks) {
    const int xcd = block % 8;
    return blocks / 8 * xcd + min(xcd, blocks % 8) + block / 8;
}
// kFromScores: the scores are in the workspace already.
template <int kSteps, bool kFromScores>
__global__ __launch_bounds__(kOneThreads) void select_one_kernel(const SelectArgs a) {
    __shared__ __attribute__((aligned(16))) uint32_t hist[kParts];
    __shared__ uint32_t found[3], near_key[kNear], counts[kSteps * kOneWaves];
    __shared__ int near_block[kNear];
    __shared__ uint32_t all[5];                               // blocks, taken, lowest, highest, near
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = kFromScores ? a.first_row + blockIdx.x : query_of(blockIdx.x, gridDim.x);
    const int64_t token = row / a.lists;
    const int list = (int)(row - token * a.lists);
    const int b = (int)(token / a.drafts), t = (int)(token - (int64_t)b * a.drafts);
    // Step j of a wave: 64 blocks, the waves one after another.
    auto block_at = [&](int j) { return (j * kOneWaves + wave) * 64 + lane; };
    float score[kSteps];
    int page[kSteps];                                         // or what is negative without a block
    const int per_list = a.dim / 32, per_row = a.lists * per_list;
    const uint4* qp = reinterpret_cast<const uint4*>(a.q + token * a.ld_q + (int64_t)list * a.dim);
    uint4 raw[4];                                             // block g of the query
    if constexpr (kFromScores) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) score[j] = block_at(j) < a.pitch ? a.scores[row * a.pitch + block_at(j)] : 0.f;
    } else {
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
            page[j] = block_at(j) < a.max_pages && a.num_pages ? a.table[(int64_t)b * a.max_pages + block_at(j)] : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = g < per_list ? qp[4 * g + i] : make_uint4(0, 0, 0, 0);
    }
    if (threadIdx.x < kParts) hist[threadIdx.x] = 0;
    if (threadIdx.x < 5) all[threadIdx.x] = threadIdx.x == 2 ? kTaken : 0;
    const int complete = a.num_pages ? complete_blocks(a, b) : 0;
    if (a.draft_lens && t >= a.draft_lens[b]) return;
    const int steps = (complete + kOneThreads - 1) / kOneThreads;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        if constexpr (kFromScores)
            page[j] = block_at(j) < complete && score[j] == score[j] ? 0 : -1;
        else if (block_at(j) >= complete || (uint32_t)page[j] >= (uint32_t)a.num_pages)
            page[j] = -1;
    }
    if constexpr (!kFromScores) {
        uint4 e[kSteps][4];
        int e_scale[kSteps][4], q_scale;
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int from = max(__shfl(page[j], 16 * k + c, 64), 0);
                e[j][k] = make_uint4(0, 0, 0, 0), e_scale[j][k] = 127;
                if (g < per_list && j < steps) {
                    const int64_t at = (int64_t)from * per_row + list * per_list + g;
                    e[j][k] = reinterpret_cast<const uint4*>(a.codes)[at];
                    e_scale[j][k] = a.scales[at];
                }
            }
        const uint4 q = quant32(raw, q_scale);
        const v8i qv = {(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
            v4f acc[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const v8i ev = {(int)e[j][k].x, (int)e[j][k].y, (int)e[j][k].z, (int)e[j][k].w, 0, 0, 0, 0};
                acc[k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(qv, ev, v4f{0.f, 0.f, 0.f, 0.f}, 4, 4, 0, q_scale, 0,
                                                                         e_scale[j][k]);
            }
            score[j] = ranked(g < 2 ? (g == 0 ? acc[0][0] : acc[1][0]) : (g == 2 ? acc[2][0] : acc[3][0]));
        }
    }
    uint32_t key[kSteps];
    int blocks = 0, taken = 0;
    uint32_t low = kTaken, high = 0;
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
        const int n = block_at(j);
        key[j] = page[j] >= 0 ? (n < a.n_first || n >= complete - a.n_recent ? kTaken : key_of(score[j])) : 0;
        blocks += __popcll(__ballot(key[j] != 0));
        taken += __popcll(__ballot(key[j] == kTaken));
        if (key[j] != 0 && key[j] != kTaken) low = min(low, key[j]), high = max(high, key[j]);
    }
    low = extreme<false>(low), high = extreme<true>(high);
    __syncthreads();
    if (lane == 0 && blocks) {
        atomicAdd(&all[0], (uint32_t)blocks);
        if (taken) atomicAdd(&all[1], (uint32_t)taken);
        atomicMin(&all[2], low), atomicMax(&all[3], high);
    }
    __syncthreads();
    blocks = (int)all[0], taken = (int)all[1], low = all[2], high = all[3];

    // What is taken: above the threshold, and on it the first `ties`, or those of `mine`.
    Threshold top{0, 0};
    uint32_t mine = 0;                                        // a bit for each step
    const int need = a.select - taken;
    auto each = [&](auto f) {
#pragma unroll
        for (int j = 0; j < kSteps; ++j) f(j, key[j]);
    };
    auto value = [](uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); };
    if (blocks > a.select) {
        if (need <= 0) {
            top = {kTaken, a.select};
        } else {
            const float least = value(low), width = value(high) - least, per = (float)(kParts - 1) / width;
            bool by_bits = !(width > 0.f && width < __builtin_inff() && per < __builtin_inff());
            auto part_of = [&](float x) { return min((uint32_t)((x - least) * per), (uint32_t)kParts - 1); };
            if (!by_bits) {
                each([&](int j, uint32_t k) {
                    if (k != 0 && k != kTaken) atomicAdd(&hist[part_of(score[j])], 1u);
                });
                __syncthreads();
                if (wave == 0) {                              // a lane has four parts, lane 0 the highest
                    const uint4 own = *reinterpret_cast<const uint4*>(&hist[kParts - 4 - 4 * lane]);
                    const uint32_t sum = own.x + own.y + own.z + own.w;
                    uint32_t above = sum_upto(sum) - sum;
                    const uint32_t n[4] = {own.w, own.z, own.y, own.x};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (above < (uint32_t)need && above + n[i] >= (uint32_t)need)
                            found[0] = kParts - 1 - 4 * lane - i, found[1] = above, found[2] = n[i];
                        above += n[i];
                    }
                }
                __syncthreads();
                const uint32_t part = found[0];
                const int left = need - (int)found[1], there = (int)found[2];
                by_bits = there > kNear;
                if (!by_bits) {
                    top = {kTaken - 1, 0};                    // blocks that are taken before any other, and:
                    each([&](int j, uint32_t k) {
                        if (k == 0 || k == kTaken) return;
                        const uint32_t p = part_of(score[j]);
                        if (p > part || (p == part && there == left)) mine |= 1u << j;
                        if (p == part && there != left) {
                            const uint32_t to = atomicAdd(&all[4], 1u);
                            near_key[to] = k, near_block[to] = block_at(j);
                        }
                    });
                    if (there != left) {
                        __syncthreads();
                        each([&](int j, uint32_t k) {
                            if (k == 0 || k == kTaken || part_of(score[j]) != part) return;
                            int rank = 0;
                            for (int i = 0; i < there; ++i)
                                rank += near_key[i] > k || (near_key[i] == k && near_block[i] < block_at(j)) ? 1 : 0;
                            if (rank < left) mine |= 1u << j;
                        });
                    }
                }
            }
            if (by_bits) top = threshold_by_bits(low, high, need, hist, found, wave, lane, each);
        }
    }

    // Counts of each step of each wave, above the threshold and on it, 16 bits each (of at
    // most 8192 blocks), added up in the blocks' order.
    static_assert(kSteps * kOneThreads < 1 << 16);
    each([&](int j, uint32_t k) {
        const uint32_t above = __popcll(__ballot(k > top.key || (mine >> j & 1))), equal = __popcll(__ballot(k != 0 && k == top.key));
        if (lane == 0) counts[j * kOneWaves + wave] = equal << 16 | above;
    });
    __syncthreads();
    constexpr int kCounts = kSteps * kOneWaves;
    uint32_t first = sum_upto(lane < kCounts ? counts[lane] : 0), second = 0;
    if (kCounts > 64) second = sum_upto(counts[min(64 + lane, kCounts - 1)]) + __builtin_amdgcn_readlane(first, 63);
    const uint64_t before = (1ull << lane) - 1;
    int32_t* ids = a.ids + row * a.select;
    each([&](int j, uint32_t k) {
        const int i = j * kOneWaves + wave;                   // those before it
        const uint32_t upto = i == 0 ? 0 : i <= 64 ? __builtin_amdgcn_readlane(first, i - 1) : __builtin_amdgcn_readlane(second, i - 65);
        const int equal = (int)(upto >> 16), at = (int)(upto & 0xFFFFu) + min(equal, top.ties);
        const bool on = k != 0 && k == top.key;
        const bool take = k > top.key || (mine >> j & 1) || (on && equal + __popcll(__ballot(on) & before) < top.ties);
        const uint64_t takes = __ballot(take);
        if (take) {
            const int to = at + __popcll(takes & before);
            ids[to] = block_at(j);
            if (a.out_scores) a.out_scores[row * a.select + to] = score[j];
        }
    });
    for (int i = min(blocks, a.select) + (int)threadIdx.x; i < a.select; i += kOneThreads) {
        ids[i] = -1;
        if (a.out_scores) a.out_scores[row * a.select + i] = -__builtin_inff();
    }
}

// Queries of a launch: a grid has fewer than 2^32 threads.
constexpr int64_t kMostRows = 1 << 21;
static_assert(kMostRows * kOneThreads < (int64_t)1 << 32);

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
    const int64_t rows = p.batch * p.drafts * p.lists;
    // One launch where a workgroup has its query's entries in flight at once and a CU has
    // two workgroups of one step or one of two: one query over 500 blocks 6.6 us, in two
    // launches 8.7; 64 x 8 drafted tokens over 1000 11.5 and 12.7; 64 x 4 over 2000 12.8 and
    // 13.7, but 96 x 4 22.4 and 16.9; one over 4000, with more steps, 16.5 and 13.2.
    const bool one_step = p.max_pages <= kOneThreads;
    if (p.max_pages <= 2 * kOneThreads && p.dim <= 128 && rows <= (one_step ? 512 : 256)) {
        if (one_step)
            select_one_kernel<1, false><<<(unsigned)rows, kOneThreads, 0, s>>>(a);
        else
            select_one_kernel<2, false><<<(unsigned)rows, kOneThreads, 0, s>>>(a);
        return hipGetLastError();
    }
    if (p.num_pages && p.max_pages) {
        const dim3 grid((unsigned)((p.max_pages + kScoreSpan - 1) / kScoreSpan), (unsigned)p.lists, (unsigned)p.batch);
        select_scores_kernel<<<grid, 64 * kScoreWaves, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    for (; a.first_row < rows; a.first_row += kMostRows) {
        const unsigned n = (unsigned)(rows - a.first_row < kMostRows ? rows - a.first_row : kMostRows);
        if (p.max_pages <= 2 * kOneThreads)
            select_one_kernel<2, true><<<n, kOneThreads, 0, s>>>(a);
        else if (p.max_pages <= 8 * kOneThreads)
            select_one_kernel<8, true><<<n, kOneThreads, 0, s>>>(a);
        else
            select_blocks_kernel<<<n, kThreads, 0, s>>>(a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fp4
