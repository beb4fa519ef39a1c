// Rotation of queries and keys by their positions, with or without the head norms,
// and the append of keys and values to the paged MXFP4 cache, in one pass.
//
// For each query and key head x of head_dim values: y = x, or x * rsqrt(mean(x^2) +
// eps) * w; the first rot_dim values of y turned in pairs by the token's angles; one
// rounding to bf16.  Queries are stored so; keys, and values as they come, are
// quantized from bf16 in blocks of 32 into the cache row of the token's slot.  With
// norms the arithmetic is that of the head norm kernel and of the append, operation
// for operation, so the bytes are the same as from three calls; without them a turned
// value is one product and one fused multiply-add, y c -+ (y' s).
//
// Bound by HBM: a value of a query is read and written (4 bytes), one of a key or a
// value read and written as a code and its share of a scale (2.53 bytes); the keys
// never go to memory as bf16.  A lane owns 8 consecutive values, 4, 8, 16 or 32 lanes
// a head; a block of 32 is 4 neighbouring lanes, whose largest magnitude takes two
// quad exchanges.  A workgroup takes one token: its angles are read once.
//
// A call among others, 64 + 8 + 8 heads of 128 values: 8192 tokens (315 MB) 59 us, 5.3 TB/s,
// what a large copy reaches; 64 tokens 3.6 to 4.2 us, 3.2 of them the kernel, one round trip to
// memory.  4097 tokens of 20 + 4 + 4 heads of 96 (41 MB, a quarter of the lanes idle) 8.9 us,
// 4.6 TB/s.  With norms 73 us, 4.0 and 11.3.
#include "fp4_internal.h"
#include "quant_device.h"

namespace fp4 {
namespace {

constexpr int kThreads = 256;

struct Args {
    const uint16_t *q, *k, *v;
    uint16_t* qo;
    int64_t ldq, ldk, ldv, ldqo;
    const void *qw, *kw;              // [head_dim] bf16 or fp32, or NULL
    int w_f32;
    const float* cos_sin;
    const int32_t *positions, *slots;
    int64_t max_positions, capacity;
    uint8_t *kc, *ks, *vc, *vs;
    int q_heads, kv_heads, heads, head_dim, rot_dim;
    float eps, inv_dim;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
}

// 8 weights from element o on (ones without weights).
__device__ __forceinline__ void load_weights(const void* w, int w_f32, int o, float* f) {
    if (w == nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 1.0f;
    } else if (w_f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + o);
        const float4 a = p[0], b = p[1];
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + o), f);
    }
}

// kLanes lanes to a head, kHeads heads to each group of lanes (their loads are all in
// flight at once); heads in the order queries, keys, values.  Workgroup (x, y): token
// x, heads from y * kHeads * (256 / kLanes) on.
template <int kLanes, int kHeads, bool kInterleaved, bool kNorm>
__global__ __launch_bounds__(kThreads) void rope_append_kernel(const Args a) {
    constexpr int kGroups = kThreads / kLanes;
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const int half = a.rot_dim / 2, o = lane * 8;
    const float* angles = nullptr;
    if (a.rot_dim) {
        const int64_t pos = a.positions[t];
        if (pos < 0 || pos >= a.max_positions) return;                  // padding token (whole workgroup)
        angles = a.cos_sin + pos * a.rot_dim;
    }
    const bool own = o < a.head_dim;                                    // lanes past an uneven head hold zeros
    const bool turns = own && o < a.rot_dim;
    const int h0 = (int)blockIdx.y * kGroups * kHeads + group, keys_end = a.q_heads + a.kv_heads;

    uint4 x[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * kGroups;
        x[i] = make_uint4(0, 0, 0, 0);
        if (own && h < a.heads) {
            const uint16_t* p = h < a.q_heads  ? a.q + t * a.ldq + (int64_t)h * a.head_dim
                                : h < keys_end ? a.k + t * a.ldk + (int64_t)(h - a.q_heads) * a.head_dim
                                               : a.v + t * a.ldv + (int64_t)(h - keys_end) * a.head_dim;
            x[i] = *reinterpret_cast<const uint4*>(p + o);
        }
    }
    const int64_t slot = a.slots[t];
    // Angle i of a pair: half-split lanes need 8 of them, interleaved ones 4.
    constexpr int kAngles = kInterleaved ? 4 : 8;
    float c[kAngles], s[kAngles];
    const bool second = !kInterleaved && o >= half;                     // lane holds the b values
    if (turns) {
        const float* p = angles + (kInterleaved ? o / 2 : (second ? o - half : o));
#pragma unroll
        for (int i = 0; i < kAngles; i += 4) {
            const float4 u = *reinterpret_cast<const float4*>(p + i);
            const float4 w = *reinterpret_cast<const float4*>(p + half + i);
            c[i] = u.x, c[i + 1] = u.y, c[i + 2] = u.z, c[i + 3] = u.w;
            s[i] = w.x, s[i + 1] = w.y, s[i + 2] = w.z, s[i + 3] = w.w;
        }
    }
    const int peer = turns && !kInterleaved ? (second ? o - half : o + half) / 8 : lane;

#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * kGroups;
        const bool is_q = h < a.q_heads, is_v = h >= keys_end;
        const void* weights = is_q ? a.qw : a.kw;
        float y[8], r = 1.0f;
        unpack8(x[i], y);
        if constexpr (kNorm) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
            for (int m = 1; m < kLanes; m *= 2) ss += __shfl_xor(ss, m, kLanes);
            r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
            float w[8];
            if (own) load_weights(weights, a.w_f32, o, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = own ? y[j] * r * w[j] : 0.f;
        }
        if (kInterleaved) {
            if (turns) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = y[2 * j], q = y[2 * j + 1];
                    y[2 * j] = fmaf(p, c[j], -__fmul_rn(q, s[j]));
                    // The head norm kernel rounds the other product here.
                    y[2 * j + 1] = kNorm ? fmaf(p, s[j], __fmul_rn(q, c[j])) : fmaf(q, c[j], __fmul_rn(p, s[j]));
                }
            }
        } else if (a.rot_dim) {
            uint4 u;
            u.x = __shfl(x[i].x, peer, kLanes), u.y = __shfl(x[i].y, peer, kLanes);
            u.z = __shfl(x[i].z, peer, kLanes), u.w = __shfl(x[i].w, peer, kLanes);
            if (turns) {
                float z[8];
                unpack8(u, z);
                if constexpr (kNorm) {
                    float w[8];
                    load_weights(weights, a.w_f32, peer * 8, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) z[j] = z[j] * r * w[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float other = __fmul_rn(z[j], s[j]);
                    y[j] = fmaf(y[j], c[j], second ? other : -other);
                }
            }
        }
        if (!own || h >= a.heads) continue;
        if (is_q) {
            *reinterpret_cast<uint4*>(a.qo + t * a.ldqo + (int64_t)h * a.head_dim + o) =
                make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        } else if (slot >= 0 && slot < a.capacity) {
            uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, byte;
            if (!is_v) {
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = pack_bf16(y[2 * j], y[2 * j + 1]);
            }
            const uint32_t codes = mx_quant8(w, byte);
            // Place in the cache's rows: 8 values to a word of codes, 32 to a scale byte.
            const int64_t at = (slot * a.kv_heads + (h - (is_v ? keys_end : a.q_heads))) * (a.head_dim / 8) + lane;
            reinterpret_cast<uint32_t*>(is_v ? a.vc : a.kc)[at] = codes;
            if (lane % 4 == 0) (is_v ? a.vs : a.ks)[at / 4] = (uint8_t)byte;
        }
    }
}

template <int kLanes, int kHeads>
void launch(const Args& a, int64_t tokens, bool interleaved, bool norm, hipStream_t s) {
    constexpr int kSpan = kThreads / kLanes * kHeads;
    const dim3 grid((unsigned)tokens, (unsigned)((a.heads + kSpan - 1) / kSpan));
    if (interleaved && norm)
        rope_append_kernel<kLanes, kHeads, true, true><<<grid, kThreads, 0, s>>>(a);
    else if (interleaved)
        rope_append_kernel<kLanes, kHeads, true, false><<<grid, kThreads, 0, s>>>(a);
    else if (norm)
        rope_append_kernel<kLanes, kHeads, false, true><<<grid, kThreads, 0, s>>>(a);
    else
        rope_append_kernel<kLanes, kHeads, false, false><<<grid, kThreads, 0, s>>>(a);
}

template <int kLanes>
void launch(const Args& a, int64_t tokens, bool interleaved, bool norm, hipStream_t s) {
    constexpr int kGroups = kThreads / kLanes;
    const int slots = (a.heads + kGroups - 1) / kGroups;
    // Many tokens: the number of heads to a lane group that leaves the fewest groups without
    // one, the larger of two that leave as many (8192 tokens of 80 heads 59 us with five, 63
    // with one or two; 2048 of 48 heads 9.1 with three, 9.7 with one).  Few: two, so that
    // the heads spread over the CUs (512 tokens of 80 heads 5.6 us, 6.0 with five).
    int per = slots < 2 ? 1 : 2;
    if (slots >= 2 && tokens * a.heads >= (int64_t)kGroups * 4 * 1024) {
        int least = 1 << 30;
        for (int k = 2; k <= 5; ++k) {
            const int all = (a.heads + kGroups * k - 1) / (kGroups * k) * k;
            if (all <= least) least = all, per = k;
        }
    }
    switch (per) {
        case 1: return launch<kLanes, 1>(a, tokens, interleaved, norm, s);
        case 2: return launch<kLanes, 2>(a, tokens, interleaved, norm, s);
        case 3: return launch<kLanes, 3>(a, tokens, interleaved, norm, s);
        case 4: return launch<kLanes, 4>(a, tokens, interleaved, norm, s);
        default: return launch<kLanes, 5>(a, tokens, interleaved, norm, s);
    }
}

}  // namespace

hipError_t launch_kv_append_rope(const RopeAppend& p, hipStream_t s) {
    const int64_t capacity = p.cache.num_pages * p.cache.page_size;
    Args a{};
    a.q = p.q, a.k = p.k, a.v = p.v, a.qo = p.q_out;
    a.ldq = p.ld_q, a.ldk = p.ld_k, a.ldv = p.ld_v, a.ldqo = p.ld_qo;
    a.qw = p.q_weight, a.kw = p.k_weight, a.w_f32 = p.w_f32;
    a.cos_sin = p.cos_sin, a.positions = p.positions, a.slots = p.slots;
    a.max_positions = p.max_positions, a.capacity = capacity;
    a.kc = p.cache.k_codes, a.ks = p.cache.k_scales, a.vc = p.cache.v_codes, a.vs = p.cache.v_scales;
    a.q_heads = p.q_heads, a.kv_heads = p.kv_heads;
    a.heads = p.q_heads + (capacity ? (p.cache.v_codes ? 2 : 1) * p.kv_heads : 0);
    a.head_dim = p.head_dim, a.rot_dim = p.rot_dim;
    a.eps = p.eps, a.inv_dim = 1.0f / (float)p.head_dim;
    if (a.heads == 0) return hipSuccess;
    const int lanes = p.head_dim / 8;
    if (lanes <= 4)
        launch<4>(a, p.tokens, p.interleaved, p.norm, s);
    else if (lanes <= 8)
        launch<8>(a, p.tokens, p.interleaved, p.norm, s);
    else if (lanes <= 16)
        launch<16>(a, p.tokens, p.interleaved, p.norm, s);
    else
        launch<32>(a, p.tokens, p.interleaved, p.norm, s);
    return hipGetLastError();
}

}  // namespace fp4
