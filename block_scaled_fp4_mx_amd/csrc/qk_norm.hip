// Query/key head norms with the position rotation, in one pass.
//
// For each head x of head_dim values: y = x * rsqrt(mean(x^2) + eps) * w, then
// the first rot_dim values of y turned in pairs by the token's angles.  All of
// it is fp32; the bf16 result is the only rounding.
//
// Bound by HBM: every value is read and written once (4 bytes a value); a
// token's table row (4 * rot_dim bytes) is read once per workgroup and stays in
// registers for all its heads.  A lane owns 8 consecutive values (one 16-byte
// load and store); 2, 4, .. 32 lanes (head_dim / 8 rounded up to a power of
// two) own a head, so the sum of squares is a few lane exchanges and never
// touches LDS.  A half-split pair's other value lies rot_dim/16 lanes away: the
// raw input words are exchanged (4 words) and normalized again, which is less
// than exchanging 8 fp32 results.
//
// 72 heads of 128 values: 8192 tokens (306 MB) 71 us, 4.3 TB/s; 64 tokens 3.5 us, one
// round trip to memory.  4097 tokens of 24 heads of 96 values (39 MB, a quarter of the
// lanes idle) 10.5 us, 3.7 TB/s.
#include "fp4_internal.h"

namespace fp4 {
namespace {

constexpr int kThreads = 256;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

struct QkNormArgs {
    const uint16_t *q, *k;
    uint16_t *qo, *ko;
    int64_t ldq, ldk, ldqo, ldko;
    const void *qw, *kw;              // [head_dim] bf16 or fp32, or NULL
    int w_f32;
    const float* cos_sin;
    const int32_t* positions;
    int64_t max_positions;
    int q_heads, heads, head_dim, rot_dim;
    float eps, inv_dim;
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
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

// kLanes lanes to a head, kHeads heads to each group of lanes (their loads are
// all in flight at once).  Workgroup (x, y): token x, heads from
// y * kHeads * (256 / kLanes) on.
template <int kLanes, int kHeads, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(const QkNormArgs a) {
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
    const bool turned = own && o < a.rot_dim;
    const int h0 = (int)blockIdx.y * kGroups * kHeads + group;

    uint4 v[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * kGroups;
        v[i] = make_uint4(0, 0, 0, 0);
        if (own && h < a.heads) {
            const uint16_t* x = h < a.q_heads ? a.q + t * a.ldq + (int64_t)h * a.head_dim
                                              : a.k + t * a.ldk + (int64_t)(h - a.q_heads) * a.head_dim;
            v[i] = *reinterpret_cast<const uint4*>(x + o);
        }
    }
    // Angle i of a pair: half-split lanes need 8 of them, interleaved ones 4.
    constexpr int kAngles = kInterleaved ? 4 : 8;
    float c[kAngles], s[kAngles];
    const bool second = !kInterleaved && o >= half;                     // lane holds the b values
    if (turned) {
        const float* p = angles + (kInterleaved ? o / 2 : (second ? o - half : o));
#pragma unroll
        for (int i = 0; i < kAngles; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(p + i);
            const float4 y = *reinterpret_cast<const float4*>(p + half + i);
            c[i] = x.x, c[i + 1] = x.y, c[i + 2] = x.z, c[i + 3] = x.w;
            s[i] = y.x, s[i + 1] = y.y, s[i + 2] = y.z, s[i + 3] = y.w;
        }
    }
    const int peer = turned && !kInterleaved ? (second ? o - half : o + half) / 8 : lane;

#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
        const int h = h0 + i * kGroups;
        const bool is_q = h < a.q_heads;
        float x[8], y[8], w[8];
        unpack8(v[i], x);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
        for (int m = 1; m < kLanes; m *= 2) ss += __shfl_xor(ss, m, kLanes);
        const float r = rsqrtf(fmaf(ss, a.inv_dim, a.eps));
        const void* weights = is_q ? a.qw : a.kw;
        if (own) load_weights(weights, a.w_f32, o, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = own ? x[j] * r * w[j] : 0.f;
        if (kInterleaved) {
            if (turned) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float p = y[2 * j], q = y[2 * j + 1];
                    y[2 * j] = p * c[j] - q * s[j];
                    y[2 * j + 1] = q * c[j] + p * s[j];
                }
            }
        } else if (a.rot_dim) {
            uint4 u;
            u.x = __shfl(v[i].x, peer, kLanes), u.y = __shfl(v[i].y, peer, kLanes);
            u.z = __shfl(v[i].z, peer, kLanes), u.w = __shfl(v[i].w, peer, kLanes);
            if (turned) {
                float z[8], wz[8];
                unpack8(u, z);
                load_weights(weights, a.w_f32, peer * 8, wz);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float other = z[j] * r * wz[j];
                    y[j] = second ? y[j] * c[j] + other * s[j] : y[j] * c[j] - other * s[j];
                }
            }
        }
        if (own && h < a.heads) {
            uint16_t* out = is_q ? a.qo + t * a.ldqo + (int64_t)h * a.head_dim
                                 : a.ko + t * a.ldko + (int64_t)(h - a.q_heads) * a.head_dim;
            *reinterpret_cast<uint4*>(out + o) =
                make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        }
    }
}

template <int kLanes, int kHeads>
void launch(const QkNormArgs& a, int64_t tokens, bool interleaved, hipStream_t s) {
    constexpr int kSpan = kThreads / kLanes * kHeads;
    const dim3 grid((unsigned)tokens, (unsigned)((a.heads + kSpan - 1) / kSpan));
    if (interleaved)
        qk_norm_rope_kernel<kLanes, kHeads, true><<<grid, kThreads, 0, s>>>(a);
    else
        qk_norm_rope_kernel<kLanes, kHeads, false><<<grid, kThreads, 0, s>>>(a);
}

template <int kLanes>
void launch(const QkNormArgs& a, int64_t tokens, bool interleaved, hipStream_t s) {
    constexpr int kGroups = kThreads / kLanes;
    // Few tokens: one head to a lane group, so that the heads spread over the CUs (64
    // tokens of 72 heads: 3.6 us, 6.4 with five).  Else the number of 2 .. 5 that
    // leaves the fewest groups without a head, the larger of two that leave as many
    // (8192 tokens: 71 us with five, 87 with one; 97 with four, 56 of whose 128 are idle).
    int per = 1;
    if (tokens * a.heads >= (int64_t)kGroups * 4 * 1024) {
        int least = 1 << 30;
        for (int k = 2; k <= 5; ++k) {
            const int slots = (a.heads + kGroups * k - 1) / (kGroups * k) * k;
            if (slots <= least) least = slots, per = k;
        }
    }
    switch (per) {
        case 1: return launch<kLanes, 1>(a, tokens, interleaved, s);
        case 2: return launch<kLanes, 2>(a, tokens, interleaved, s);
        case 3: return launch<kLanes, 3>(a, tokens, interleaved, s);
        case 4: return launch<kLanes, 4>(a, tokens, interleaved, s);
        default: return launch<kLanes, 5>(a, tokens, interleaved, s);
    }
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNorm& p, hipStream_t s) {
    QkNormArgs a{};
    a.q = p.q, a.k = p.k, a.qo = p.q_out, a.ko = p.k_out;
    a.ldq = p.ld_q, a.ldk = p.ld_k, a.ldqo = p.ld_qo, a.ldko = p.ld_ko;
    a.qw = p.q_weight, a.kw = p.k_weight, a.w_f32 = p.w_f32;
    a.cos_sin = p.cos_sin, a.positions = p.positions, a.max_positions = p.max_positions;
    a.q_heads = p.q_heads, a.heads = p.q_heads + p.kv_heads;
    a.head_dim = p.head_dim, a.rot_dim = p.rot_dim;
    a.eps = p.eps, a.inv_dim = 1.0f / (float)p.head_dim;
    const int lanes = p.head_dim / 8;
    if (lanes <= 2)
        launch<2>(a, p.tokens, p.interleaved, s);
    else if (lanes <= 4)
        launch<4>(a, p.tokens, p.interleaved, s);
    else if (lanes <= 8)
        launch<8>(a, p.tokens, p.interleaved, s);
    else if (lanes <= 16)
        launch<16>(a, p.tokens, p.interleaved, s);
    else
        launch<32>(a, p.tokens, p.interleaved, s);
    return hipGetLastError();
}

}  // namespace fp4
