// C ABI of libfp4: argument validation and dispatch to the gfx950 kernels.
// Every check runs before the first HIP call, so a rejected call enqueues
// nothing; the library holds no state besides the per-thread error message.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "fp4_internal.h"

namespace {

thread_local char g_last_error[512] = "";

int fail(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return status;
}

int ok() {
    g_last_error[0] = '\0';
    return FP4_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int hip_status(hipError_t e, const char* what) {
    if (e != hipSuccess) return fail(FP4_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

#define FP4_REQUIRE(cond, status, ...) \
    do {                               \
        if (!(cond)) return fail(status, __VA_ARGS__); \
    } while (0)

#define FP4_PTR(p) FP4_REQUIRE((p) != nullptr, FP4_ERR_INVALID, "%s is NULL", #p); \
    FP4_REQUIRE(aligned16(p), FP4_ERR_ALIGN, "%s is not 16-byte aligned", #p)

// Scalars the kernels read (tensor scales, counters) need only natural alignment.
#define FP4_SCALAR_PTR(p) FP4_REQUIRE((p) != nullptr, FP4_ERR_INVALID, "%s is NULL", #p); \
    FP4_REQUIRE((reinterpret_cast<uintptr_t>(p) & 3u) == 0, FP4_ERR_ALIGN, "%s is not 4-byte aligned", #p)

int check_ld(int64_t ld, int64_t width, const char* name) {
    FP4_REQUIRE(ld >= width, FP4_ERR_INVALID, "%s (%lld) is smaller than the row width (%lld)", name,
                (long long)ld, (long long)width);
    FP4_REQUIRE(ld % 8 == 0, FP4_ERR_ALIGN, "%s (%lld) is not a multiple of 8", name, (long long)ld);
    return FP4_OK;
}

size_t nv_ws_bytes() { return 4096; }   // pass-1 partial maxima of the tensor amax (1024 words)

// The remap's and FP8 dequant's optional workspace: NULL (with 0 bytes) or at
// least fp4_scale_max_workspace_bytes(rows, k) bytes.
int check_scale_max_ws(const void* ws, size_t bytes, int64_t rows, int64_t k) {
    if (ws == nullptr) {
        FP4_REQUIRE(bytes == 0, FP4_ERR_WORKSPACE, "workspace is NULL but workspace_bytes=%zu", bytes);
        return FP4_OK;
    }
    const size_t need = fp4::scale_max_workspace_bytes(rows, k);
    FP4_REQUIRE(bytes >= need, FP4_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, bytes);
    return FP4_OK;
}

// Whether two arrays of `rows` rows (row pitch and width in bytes) share a byte.
// Rows of one pitch may interleave (columns of one fused array) without sharing any.
bool rows_overlap(const void* a, int64_t pitch_a, int64_t width_a, const void* b, int64_t pitch_b, int64_t width_b,
                  int64_t rows) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    const uintptr_t ea = pa + (uintptr_t)((rows - 1) * pitch_a + width_a);
    const uintptr_t eb = pb + (uintptr_t)((rows - 1) * pitch_b + width_b);
    if (pa >= eb || pb >= ea) return false;
    if (rows == 1 || pitch_a != pitch_b) return true;
    const uintptr_t pitch = (uintptr_t)pitch_a;
    const uintptr_t off = pb >= pa ? (pb - pa) % pitch : (pitch - (pa - pb) % pitch) % pitch;   // of b in a's rows
    return off < (uintptr_t)width_a || off + (uintptr_t)width_b > pitch;
}

// Whether a run of bytes shares one with an array of `rows` rows (it may lie between two rows).
bool run_overlaps(const void* a, int64_t pitch, int64_t width, int64_t rows, const void* run, uint64_t bytes) {
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pr = reinterpret_cast<uintptr_t>(run);
    const uintptr_t end = pa + (uintptr_t)((rows - 1) * pitch + width);
    if (bytes == 0 || pr >= end || pr + bytes <= pa) return false;
    if (pr <= pa) return true;
    const uintptr_t row = (pr - pa) / (uintptr_t)pitch, off = (pr - pa) % (uintptr_t)pitch;
    return off < (uintptr_t)width || (row + 1 < (uintptr_t)rows && off + bytes > (uintptr_t)pitch);
}

constexpr int64_t kMaxList = (int64_t)1 << 20;    // sequences of a batch, entries of a list of ids

int check_page_size(int64_t page_size) {
    FP4_REQUIRE(page_size > 0, FP4_ERR_INVALID, "page_size=%lld", (long long)page_size);
    FP4_REQUIRE(page_size % 16 == 0, FP4_ERR_SHAPE, "page_size=%lld is not a multiple of 16", (long long)page_size);
    return FP4_OK;
}

// A cache's sizes and arrays; an empty cache needs no arrays.
int check_cache(const fp4_kv_cache* cache, bool values_needed) {
    FP4_REQUIRE(cache != nullptr, FP4_ERR_INVALID, "cache is NULL");
    FP4_REQUIRE(cache->num_pages >= 0 && cache->d >= 0, FP4_ERR_INVALID, "negative size num_pages=%lld d=%lld",
                (long long)cache->num_pages, (long long)cache->d);
    if (int e = check_page_size(cache->page_size)) return e;
    FP4_REQUIRE(cache->d % 32 == 0, FP4_ERR_SHAPE, "d=%lld is not a multiple of 32", (long long)cache->d);
    FP4_REQUIRE(cache->d < (int64_t)1 << 31 && cache->num_pages < ((int64_t)1 << 31) / cache->page_size, FP4_ERR_SHAPE,
                "the cache is too large: num_pages=%lld of %lld rows, d=%lld (rows and d must be below 2^31)",
                (long long)cache->num_pages, (long long)cache->page_size, (long long)cache->d);
    if (cache->num_pages == 0 || cache->d == 0) return FP4_OK;
    FP4_PTR(cache->k_codes);
    FP4_PTR(cache->k_scales);
    FP4_REQUIRE((cache->v_codes == nullptr) == (cache->v_scales == nullptr), FP4_ERR_INVALID,
                "v_codes and v_scales must both be given or both be NULL");
    if (values_needed || cache->v_codes) {
        FP4_PTR(cache->v_codes);
        FP4_PTR(cache->v_scales);
    }
    return FP4_OK;
}

int check_pages(const fp4_kv_pages* pages) {
    FP4_REQUIRE(pages != nullptr, FP4_ERR_INVALID, "pages is NULL");
    FP4_REQUIRE(pages->batch >= 0 && pages->max_pages >= 0 && pages->num_pages >= 0, FP4_ERR_INVALID,
                "negative size batch=%lld max_pages=%lld num_pages=%lld", (long long)pages->batch,
                (long long)pages->max_pages, (long long)pages->num_pages);
    FP4_REQUIRE(pages->batch < kMaxList, FP4_ERR_SHAPE, "batch=%lld too large", (long long)pages->batch);
    FP4_REQUIRE(pages->max_pages < (int64_t)1 << 31 && pages->num_pages < (int64_t)1 << 31, FP4_ERR_SHAPE,
                "max_pages=%lld num_pages=%lld too large", (long long)pages->max_pages, (long long)pages->num_pages);
    if (pages->batch == 0) return FP4_OK;
    if (pages->max_pages) { FP4_SCALAR_PTR(pages->page_table); }
    FP4_SCALAR_PTR(pages->page_counts);
    FP4_SCALAR_PTR(pages->seq_lens);
    if (pages->num_pages) { FP4_SCALAR_PTR(pages->page_refs); }
    return FP4_OK;
}

int check_same_pool(const fp4_kv_cache* cache, const fp4_kv_pages* pages) {
    FP4_REQUIRE(cache->num_pages == pages->num_pages, FP4_ERR_INVALID, "the cache has %lld pages, page_refs %lld",
                (long long)cache->num_pages, (long long)pages->num_pages);
    return FP4_OK;
}

// The kernels work in powers of two, with scale * log2(e) in fp32.
int check_scale(float scale) {
    FP4_REQUIRE(std::fabs(scale) <= 0x1p127f, FP4_ERR_INVALID, "scale=%g is not finite or above 2^127", (double)scale);
    return FP4_OK;
}

// Head counts and head_dim of the attention entry points.
int check_heads(int q_heads, int kv_heads, int head_dim) {
    FP4_REQUIRE(q_heads > 0 && kv_heads > 0, FP4_ERR_INVALID, "q_heads=%d and kv_heads=%d must be positive", q_heads,
                kv_heads);
    FP4_REQUIRE(q_heads % kv_heads == 0 && q_heads <= 4096, FP4_ERR_SHAPE,
                "q_heads=%d is not a multiple of kv_heads=%d (or above 4096)", q_heads, kv_heads);
    FP4_REQUIRE(head_dim == 64 || head_dim == 128 || head_dim == 256, FP4_ERR_SHAPE, "head_dim=%d is not 64, 128 or 256",
                head_dim);
    return FP4_OK;
}

// reserved: by the slots of a reservation.
int kv_compact(const fp4_kv_cache* cache, const fp4_kv_pages* pages, const int32_t* accepted, int64_t max_accepted,
               const int32_t* accepted_lens, bool reserved, const int32_t* slots, int64_t max_new, void* stream,
               const char* what) {
    if (int e = check_cache(cache, false)) return e;
    if (int e = check_pages(pages)) return e;
    if (int e = check_same_pool(cache, pages)) return e;
    FP4_REQUIRE(!accepted || (max_accepted >= 0 && max_accepted <= 64), FP4_ERR_INVALID,
                "max_accepted=%lld outside [0, 64]", (long long)max_accepted);
    if (pages->batch == 0 || cache->num_pages == 0 || cache->d == 0) return ok();
    if (accepted) { FP4_SCALAR_PTR(accepted); }
    FP4_SCALAR_PTR(accepted_lens);
    if (reserved) {
        FP4_SCALAR_PTR(slots);
        if (max_new == 0) return ok();
    }
    return hip_status(fp4::launch_kv_compact(*cache, *pages, accepted, max_accepted, accepted_lens, slots, max_new,
                                             static_cast<hipStream_t>(stream)),
                      what);
}

}  // namespace

extern "C" {

int fp4_abi_version(void) { return 2; }

const char* fp4_status_string(int status) {
    switch (status) {
        case FP4_OK: return "ok";
        case FP4_ERR_INVALID: return "invalid argument";
        case FP4_ERR_SHAPE: return "unsupported shape";
        case FP4_ERR_ALIGN: return "misaligned pointer or leading dimension";
        case FP4_ERR_UNSUPPORTED: return "unsupported combination";
        case FP4_ERR_WORKSPACE: return "workspace missing or too small";
        case FP4_ERR_HIP: return "HIP runtime error";
        default: return "unknown status";
    }
}

const char* fp4_last_error(void) { return g_last_error; }

int fp4_quantize_mx(const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x,
                    uint8_t* codes, uint8_t* scales, void* stream) {
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    FP4_REQUIRE(k % 32 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 32", (long long)k);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(x_bf16);
    FP4_PTR(codes);
    FP4_PTR(scales);
    if (int e = check_ld(ld_x, k, "ld_x")) return e;
    return hip_status(fp4::launch_quantize_mx(static_cast<const uint16_t*>(x_bf16), rows, k, ld_x, codes,
                                              scales, static_cast<hipStream_t>(stream)),
                      "fp4_quantize_mx launch");
}

size_t fp4_quantize_nv_workspace_bytes(int64_t rows, int64_t k) {
    (void)rows;
    (void)k;
    return nv_ws_bytes();
}

int fp4_quantize_nv(const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x, uint8_t* codes,
                    uint8_t* scales, float* tensor_scale, int tensor_scale_is_input, void* workspace,
                    size_t workspace_bytes, void* stream) {
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    FP4_REQUIRE(k % 16 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 16", (long long)k);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(x_bf16);
    FP4_PTR(codes);
    FP4_PTR(scales);
    FP4_SCALAR_PTR(tensor_scale);
    if (int e = check_ld(ld_x, k, "ld_x")) return e;
    if (!tensor_scale_is_input) {
        FP4_REQUIRE(workspace != nullptr && workspace_bytes >= nv_ws_bytes(), FP4_ERR_WORKSPACE,
                    "workspace needs %zu bytes, got %zu", nv_ws_bytes(), workspace ? workspace_bytes : (size_t)0);
        FP4_REQUIRE(aligned16(workspace), FP4_ERR_ALIGN, "workspace is not 16-byte aligned");
    }
    return hip_status(fp4::launch_quantize_nv(static_cast<const uint16_t*>(x_bf16), rows, k, ld_x, codes, scales,
                                              tensor_scale, tensor_scale_is_input != 0,
                                              static_cast<uint32_t*>(workspace), static_cast<hipStream_t>(stream)),
                      "fp4_quantize_nv launch");
}

int fp4_quantize_nv_noalloc(const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x, uint8_t* codes,
                            uint8_t* scales, float* tensor_scale, int tensor_scale_is_input, void* stream) {
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    FP4_REQUIRE(k % 16 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 16", (long long)k);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(x_bf16);
    FP4_PTR(codes);
    FP4_PTR(scales);
    FP4_SCALAR_PTR(tensor_scale);
    if (int e = check_ld(ld_x, k, "ld_x")) return e;
    // The partial maxima need one word per pass-1 workgroup; the grid is capped
    // so that every shape fits the static array.
    FP4_REQUIRE(nv_ws_bytes() <= fp4::nv_scratch_bytes(), FP4_ERR_WORKSPACE,
                "the NV quantize needs %zu bytes of scratch, the static array holds %zu", nv_ws_bytes(),
                fp4::nv_scratch_bytes());
    return hip_status(fp4::launch_quantize_nv_noalloc(static_cast<const uint16_t*>(x_bf16), rows, k, ld_x, codes,
                                                      scales, tensor_scale, tensor_scale_is_input != 0,
                                                      static_cast<hipStream_t>(stream)),
                      "fp4_quantize_nv_noalloc launch");
}

size_t fp4_scale_max_workspace_bytes(int64_t rows, int64_t k) {
    return rows > 0 && k >= 32 ? fp4::scale_max_workspace_bytes(rows, k) : 0;
}

int fp4_remap_mx_to_nv(const uint8_t* codes, const uint8_t* scales_e8m0, int64_t rows, int64_t k,
                       uint8_t* scales_e4m3, float* tensor_scale, int32_t* n_inexact_blocks, void* workspace,
                       size_t workspace_bytes, void* stream) {
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    FP4_REQUIRE(k % 32 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 32", (long long)k);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(codes);
    FP4_PTR(scales_e8m0);
    FP4_PTR(scales_e4m3);
    FP4_SCALAR_PTR(tensor_scale);
    FP4_SCALAR_PTR(n_inexact_blocks);
    if (const int e = check_scale_max_ws(workspace, workspace_bytes, rows, k)) return e;
    return hip_status(fp4::launch_remap(codes, scales_e8m0, rows, k, scales_e4m3, tensor_scale, n_inexact_blocks,
                                        static_cast<uint8_t*>(workspace), static_cast<hipStream_t>(stream)),
                      "fp4_remap_mx_to_nv launch");
}

int fp4_dequant(fp4_format fmt, const uint8_t* codes, const uint8_t* scales, const float* tensor_scale,
                int64_t rows, int64_t k, void* out, fp4_dtype out_dtype, int64_t ld_out, void* stream) {
    FP4_REQUIRE(fmt == FP4_FMT_MX || fmt == FP4_FMT_NV, FP4_ERR_INVALID, "bad format %d", (int)fmt);
    FP4_REQUIRE(out_dtype == FP4_DT_BF16 || out_dtype == FP4_DT_F32, FP4_ERR_INVALID, "bad dtype %d", (int)out_dtype);
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    const int blk = fmt == FP4_FMT_MX ? 32 : 16;
    FP4_REQUIRE(k % blk == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of %d", (long long)k, blk);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(codes);
    FP4_PTR(scales);
    FP4_PTR(out);
    if (fmt == FP4_FMT_NV) { FP4_SCALAR_PTR(tensor_scale); }
    if (int e = check_ld(ld_out, k, "ld_out")) return e;
    return hip_status(fp4::launch_dequant(fmt, codes, scales, tensor_scale, rows, k, out, out_dtype == FP4_DT_F32,
                                          ld_out, static_cast<hipStream_t>(stream)),
                      "fp4_dequant launch");
}

int fp4_gemm(fp4_format fmt, const uint8_t* a_codes, const uint8_t* a_scales, const float* a_tensor_scale,
             const uint8_t* b_codes, const uint8_t* b_scales, const float* b_tensor_scale, int64_t m, int64_t n,
             int64_t k, void* c, fp4_dtype c_dtype, int64_t ldc, void* stream) {
    FP4_REQUIRE(fmt == FP4_FMT_MX || fmt == FP4_FMT_NV, FP4_ERR_INVALID, "bad format %d", (int)fmt);
    FP4_REQUIRE(c_dtype == FP4_DT_BF16 || c_dtype == FP4_DT_F32, FP4_ERR_INVALID, "bad dtype %d", (int)c_dtype);
    FP4_REQUIRE(m >= 0 && n >= 0 && k >= 0, FP4_ERR_INVALID, "negative size m=%lld n=%lld k=%lld", (long long)m,
                (long long)n, (long long)k);
    const int blk = fmt == FP4_FMT_MX ? 32 : 16;
    FP4_REQUIRE(k % blk == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of %d", (long long)k, blk);
    FP4_REQUIRE(m < (int64_t)65535 * 128, FP4_ERR_SHAPE, "m=%lld too large", (long long)m);
    if (m == 0 || n == 0) return ok();
    FP4_PTR(c);
    FP4_REQUIRE(ldc >= n, FP4_ERR_INVALID, "ldc (%lld) < n (%lld)", (long long)ldc, (long long)n);
    if (k > 0) {
        FP4_PTR(a_codes);
        FP4_PTR(a_scales);
        FP4_PTR(b_codes);
        FP4_PTR(b_scales);
    }
    if (fmt == FP4_FMT_NV) {
        FP4_SCALAR_PTR(a_tensor_scale);
        FP4_SCALAR_PTR(b_tensor_scale);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = fmt == FP4_FMT_MX
                       ? fp4::launch_gemm_mx(a_codes, a_scales, b_codes, b_scales, m, n, k, c, c_dtype == FP4_DT_F32, ldc, s)
                       : fp4::launch_gemm_nv(a_codes, a_scales, a_tensor_scale, b_codes, b_scales, b_tensor_scale, m, n,
                                             k, c, c_dtype == FP4_DT_F32, ldc, s);
    return hip_status(e, "fp4_gemm launch");
}

int fp4_kv_append_mx(const void* x_bf16, int64_t tokens, int64_t d, int64_t ld_x, const int32_t* slots,
                     uint8_t* cache_codes, uint8_t* cache_scales, int64_t capacity, void* stream) {
    FP4_REQUIRE(tokens >= 0 && d >= 0 && capacity >= 0, FP4_ERR_INVALID, "negative size tokens=%lld d=%lld capacity=%lld",
                (long long)tokens, (long long)d, (long long)capacity);
    FP4_REQUIRE(d % 32 == 0, FP4_ERR_SHAPE, "d=%lld is not a multiple of 32", (long long)d);
    if (tokens == 0 || d == 0 || capacity == 0) return ok();
    FP4_PTR(x_bf16);
    FP4_SCALAR_PTR(slots);
    FP4_PTR(cache_codes);
    FP4_PTR(cache_scales);
    if (int e = check_ld(ld_x, d, "ld_x")) return e;
    return hip_status(fp4::launch_kv_append(static_cast<const uint16_t*>(x_bf16), tokens, d, ld_x, slots, cache_codes,
                                            cache_scales, capacity, static_cast<hipStream_t>(stream)),
                      "fp4_kv_append_mx launch");
}

int fp4_fake_quant(fp4_format fmt, const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x, void* out,
                   fp4_dtype out_dtype, int64_t ld_out, float* tensor_scale, int tensor_scale_is_input, void* workspace,
                   size_t workspace_bytes, void* stream) {
    FP4_REQUIRE(fmt == FP4_FMT_MX || fmt == FP4_FMT_NV, FP4_ERR_INVALID, "bad format %d", (int)fmt);
    FP4_REQUIRE(out_dtype == FP4_DT_BF16 || out_dtype == FP4_DT_F32, FP4_ERR_INVALID, "bad dtype %d", (int)out_dtype);
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    const int blk = fmt == FP4_FMT_MX ? 32 : 16;
    FP4_REQUIRE(k % blk == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of %d", (long long)k, blk);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(x_bf16);
    FP4_PTR(out);
    if (int e = check_ld(ld_x, k, "ld_x")) return e;
    if (int e = check_ld(ld_out, k, "ld_out")) return e;
    {
        const uintptr_t xb = reinterpret_cast<uintptr_t>(x_bf16), ob = reinterpret_cast<uintptr_t>(out);
        const uintptr_t xe = xb + (uintptr_t)(((rows - 1) * ld_x + k) * 2);
        const uintptr_t oe = ob + (uintptr_t)(((rows - 1) * ld_out + k) * (out_dtype == FP4_DT_F32 ? 4 : 2));
        const bool overlap = xb < oe && ob < xe;
        const bool in_place = xb == ob && ld_x == ld_out && out_dtype == FP4_DT_BF16;
        FP4_REQUIRE(!overlap || in_place, FP4_ERR_INVALID, "out overlaps x without being x itself");
    }
    if (fmt == FP4_FMT_NV) {
        FP4_SCALAR_PTR(tensor_scale);
        if (!tensor_scale_is_input) {
            FP4_REQUIRE(workspace != nullptr && workspace_bytes >= nv_ws_bytes(), FP4_ERR_WORKSPACE,
                        "workspace needs %zu bytes, got %zu", nv_ws_bytes(), workspace ? workspace_bytes : (size_t)0);
            FP4_REQUIRE(aligned16(workspace), FP4_ERR_ALIGN, "workspace is not 16-byte aligned");
        }
    }
    return hip_status(fp4::launch_fake_quant(fmt, static_cast<const uint16_t*>(x_bf16), rows, k, ld_x, out,
                                             out_dtype == FP4_DT_F32, ld_out, tensor_scale, tensor_scale_is_input != 0,
                                             static_cast<uint32_t*>(workspace), static_cast<hipStream_t>(stream)),
                      "fp4_fake_quant launch");
}

int fp4_ste_backward(const void* grad, fp4_dtype grad_dtype, int64_t rows, int64_t k, int64_t ld_grad,
                     float* grad_master, int64_t ld_master, int accumulate, void* stream) {
    FP4_REQUIRE(grad_dtype == FP4_DT_BF16 || grad_dtype == FP4_DT_F32, FP4_ERR_INVALID, "bad dtype %d", (int)grad_dtype);
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    FP4_REQUIRE(k % 8 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 8", (long long)k);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(grad);
    FP4_PTR(grad_master);
    if (int e = check_ld(ld_grad, k, "ld_grad")) return e;
    if (int e = check_ld(ld_master, k, "ld_master")) return e;
    return hip_status(fp4::launch_ste_backward(grad, grad_dtype == FP4_DT_F32, rows, k, ld_grad, grad_master, ld_master,
                                               accumulate, static_cast<hipStream_t>(stream)),
                      "fp4_ste_backward launch");
}

int fp4_quantize_mxfp8(const void* x_bf16, int64_t rows, int64_t k, int64_t ld_x, uint8_t* codes8, uint8_t* scales,
                       void* stream) {
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    FP4_REQUIRE(k % 32 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 32", (long long)k);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(x_bf16);
    FP4_PTR(codes8);
    FP4_PTR(scales);
    if (int e = check_ld(ld_x, k, "ld_x")) return e;
    return hip_status(fp4::launch_quantize_mxfp8(static_cast<const uint16_t*>(x_bf16), rows, k, ld_x, codes8, scales,
                                                 static_cast<hipStream_t>(stream)),
                      "fp4_quantize_mxfp8 launch");
}

int fp4_mx_dequant_fp8(const uint8_t* codes, const uint8_t* scales_e8m0, int64_t rows, int64_t k,
                       uint8_t* values_e4m3, uint8_t* block_scales_e4m3, float* tensor_scale,
                       int32_t* n_inexact_blocks, void* workspace, size_t workspace_bytes, void* stream) {
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    FP4_REQUIRE(k % 32 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 32", (long long)k);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(codes);
    FP4_PTR(scales_e8m0);
    FP4_PTR(values_e4m3);
    FP4_SCALAR_PTR(tensor_scale);
    FP4_SCALAR_PTR(n_inexact_blocks);
    if (const int e = check_scale_max_ws(workspace, workspace_bytes, rows, k)) return e;
    return hip_status(fp4::launch_dequant_fp8(codes, scales_e8m0, rows, k, values_e4m3, block_scales_e4m3,
                                              tensor_scale, n_inexact_blocks, static_cast<uint8_t*>(workspace),
                                              static_cast<hipStream_t>(stream)),
                      "fp4_mx_dequant_fp8 launch");
}

int fp4_mx_to_mxfp8(const uint8_t* codes, int64_t rows, int64_t k, uint8_t* codes8, void* stream) {
    FP4_REQUIRE(rows >= 0 && k >= 0, FP4_ERR_INVALID, "negative size rows=%lld k=%lld", (long long)rows, (long long)k);
    FP4_REQUIRE(k % 32 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 32", (long long)k);
    if (rows == 0 || k == 0) return ok();
    FP4_PTR(codes);
    FP4_PTR(codes8);
    return hip_status(fp4::launch_mx_to_mxfp8(codes, rows, k, codes8, static_cast<hipStream_t>(stream)),
                      "fp4_mx_to_mxfp8 launch");
}

int fp4_gemm_w4a8(const uint8_t* a_codes8, const uint8_t* a_scales, const uint8_t* b_codes, const uint8_t* b_scales,
                  int64_t m, int64_t n, int64_t k, void* c, fp4_dtype c_dtype, int64_t ldc, void* stream) {
    FP4_REQUIRE(c_dtype == FP4_DT_BF16 || c_dtype == FP4_DT_F32, FP4_ERR_INVALID, "bad dtype %d", (int)c_dtype);
    FP4_REQUIRE(m >= 0 && n >= 0 && k >= 0, FP4_ERR_INVALID, "negative size m=%lld n=%lld k=%lld", (long long)m,
                (long long)n, (long long)k);
    FP4_REQUIRE(k % 32 == 0, FP4_ERR_SHAPE, "k=%lld is not a multiple of 32", (long long)k);
    FP4_REQUIRE(m < (int64_t)65535 * 128, FP4_ERR_SHAPE, "m=%lld too large", (long long)m);
    if (m == 0 || n == 0) return ok();
    FP4_PTR(c);
    FP4_REQUIRE(ldc >= n, FP4_ERR_INVALID, "ldc (%lld) < n (%lld)", (long long)ldc, (long long)n);
    if (k > 0) {
        FP4_PTR(a_codes8);
        FP4_PTR(a_scales);
        FP4_PTR(b_codes);
        FP4_PTR(b_scales);
    }
    return hip_status(fp4::launch_gemm_w4a8(a_codes8, a_scales, b_codes, b_scales, m, n, k, c, c_dtype == FP4_DT_F32,
                                            ldc, static_cast<hipStream_t>(stream)),
                      "fp4_gemm_w4a8 launch");
}

size_t fp4_moe_workspace_bytes(fp4_format fmt, int64_t tokens, int64_t hidden, int topk, int num_experts,
                               int64_t inter) {
    if (tokens < 0 || hidden <= 0 || topk < 1 || num_experts < 1 || inter <= 0) return 0;
    return fp4::moe_workspace_bytes(fmt, tokens, hidden, topk, num_experts, inter);
}

int fp4_moe_grouped_gemm(fp4_format fmt, const void* x_bf16, int64_t tokens, int64_t hidden,
                         const int32_t* topk_ids, const float* topk_weights, int topk, int num_experts,
                         int64_t inter, const uint8_t* w13_codes, const uint8_t* w13_scales,
                         const float* w13_tensor_scales, const uint8_t* w2_codes, const uint8_t* w2_scales,
                         const float* w2_tensor_scales, const float* act_tensor_scales, void* out_bf16,
                         void* workspace, size_t workspace_bytes, const fp4_moe_debug* dbg, void* stream) {
    FP4_REQUIRE(fmt == FP4_FMT_MX || fmt == FP4_FMT_NV, FP4_ERR_INVALID, "bad format %d", (int)fmt);
    FP4_REQUIRE(tokens >= 0, FP4_ERR_INVALID, "negative tokens");
    FP4_REQUIRE(topk >= 1 && topk <= 16, FP4_ERR_INVALID, "topk=%d outside [1, 16]", topk);
    FP4_REQUIRE(num_experts >= 1 && num_experts <= 1024, FP4_ERR_INVALID, "num_experts=%d outside [1, 1024]", num_experts);
    FP4_REQUIRE(hidden > 0 && inter > 0, FP4_ERR_INVALID, "hidden and inter must be positive");
    FP4_REQUIRE(hidden % 128 == 0 && inter % 128 == 0, FP4_ERR_SHAPE, "hidden=%lld and inter=%lld must be multiples of 128",
                (long long)hidden, (long long)inter);
    FP4_REQUIRE(tokens * topk < (int64_t)1 << 30 && fp4::moe_max_tiles(tokens, topk, num_experts) <= 65535,
                FP4_ERR_SHAPE, "tokens*topk=%lld too large", (long long)(tokens * topk));
    {
        // The grouped GEMM tiles address each operand with 32-bit byte offsets
        // from its base: the gathered activation rows (Q(x) by token, Q(h) by
        // routed slot; NV also their fp16 expansions) and one expert's weight
        // slab.  Each must stay below 2 GiB.
        const int64_t lim = (int64_t)1 << 31, S = tokens * topk;
        const int64_t act_x = fmt == FP4_FMT_NV ? tokens * hidden * 2 : tokens * (hidden / 2);
        const int64_t act_h = fmt == FP4_FMT_NV ? S * inter * 2 : S * (inter / 2);
        FP4_REQUIRE(act_x < lim && act_h < lim && inter * hidden < lim, FP4_ERR_SHAPE,
                    "operand too large for 32-bit tile offsets: activations %lld and %lld bytes, expert slab %lld "
                    "bytes (each must be below 2^31)",
                    (long long)act_x, (long long)act_h, (long long)(inter * hidden));
    }
    if (tokens == 0) return ok();
    FP4_PTR(x_bf16);
    FP4_SCALAR_PTR(topk_ids);
    FP4_SCALAR_PTR(topk_weights);
    FP4_PTR(w13_codes);
    FP4_PTR(w13_scales);
    FP4_PTR(w2_codes);
    FP4_PTR(w2_scales);
    FP4_PTR(out_bf16);
    if (fmt == FP4_FMT_NV) {
        FP4_SCALAR_PTR(w13_tensor_scales);
        FP4_SCALAR_PTR(w2_tensor_scales);
        FP4_SCALAR_PTR(act_tensor_scales);
    }
    const size_t need = fp4::moe_workspace_bytes(fmt, tokens, hidden, topk, num_experts, inter);
    FP4_REQUIRE(workspace != nullptr && workspace_bytes >= need, FP4_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
                need, workspace ? workspace_bytes : (size_t)0);
    FP4_REQUIRE(aligned16(workspace), FP4_ERR_ALIGN, "workspace is not 16-byte aligned");
    fp4::MoeArgs a{};
    a.fmt = fmt;
    a.x = static_cast<const uint16_t*>(x_bf16);
    a.tokens = tokens;
    a.hidden = hidden;
    a.inter = inter;
    a.ids = topk_ids;
    a.weights = topk_weights;
    a.topk = topk;
    a.num_experts = num_experts;
    a.w13c = w13_codes;
    a.w13s = w13_scales;
    a.w2c = w2_codes;
    a.w2s = w2_scales;
    a.w13ts = w13_tensor_scales;
    a.w2ts = w2_tensor_scales;
    a.act_ts = act_tensor_scales;
    a.out = static_cast<uint16_t*>(out_bf16);
    a.ws = workspace;
    a.ws_bytes = workspace_bytes;
    if (dbg) {
        a.dbg = *dbg;
        FP4_REQUIRE(aligned16(a.dbg.gate_up) && aligned16(a.dbg.h_bf16) && aligned16(a.dbg.h_codes) &&
                        aligned16(a.dbg.h_scales) && aligned16(a.dbg.y) && aligned16(a.dbg.gate_up_in) &&
                        aligned16(a.dbg.h_codes_in) && aligned16(a.dbg.h_scales_in),
                    FP4_ERR_ALIGN, "debug buffers must be 16-byte aligned");
        FP4_REQUIRE((a.dbg.h_codes_in == nullptr) == (a.dbg.h_scales_in == nullptr), FP4_ERR_INVALID,
                    "h_codes_in and h_scales_in must be given together");
    }
    return hip_status(fp4::launch_moe(a, static_cast<hipStream_t>(stream)), "fp4_moe_grouped_gemm launch");
}

int fp4_qk_norm_rope(const void* q, const void* k, int64_t tokens, int q_heads, int kv_heads, int head_dim,
                     int64_t ld_q, int64_t ld_k, const void* q_weight, const void* k_weight, fp4_dtype weight_dtype,
                     float eps, const float* cos_sin, int64_t max_positions, int rot_dim, int interleaved,
                     const int32_t* positions, void* q_out, int64_t ld_qo, void* k_out, int64_t ld_ko, void* stream) {
    FP4_REQUIRE(tokens >= 0 && q_heads >= 0 && kv_heads >= 0, FP4_ERR_INVALID,
                "negative size tokens=%lld q_heads=%d kv_heads=%d", (long long)tokens, q_heads, kv_heads);
    FP4_REQUIRE(weight_dtype == FP4_DT_BF16 || weight_dtype == FP4_DT_F32, FP4_ERR_INVALID, "bad dtype %d",
                (int)weight_dtype);
    FP4_REQUIRE(eps >= 0.0f && std::isfinite(eps), FP4_ERR_INVALID, "eps=%g is negative or not finite", (double)eps);
    FP4_REQUIRE(head_dim >= 16 && head_dim <= 256 && head_dim % 16 == 0, FP4_ERR_SHAPE,
                "head_dim=%d is not a multiple of 16 in [16, 256]", head_dim);
    FP4_REQUIRE(rot_dim >= 0 && rot_dim <= head_dim && rot_dim % 16 == 0, FP4_ERR_SHAPE,
                "rot_dim=%d is not a multiple of 16 in [0, head_dim=%d]", rot_dim, head_dim);
    FP4_REQUIRE(tokens < (int64_t)1 << 24, FP4_ERR_SHAPE, "tokens=%lld too large", (long long)tokens);
    FP4_REQUIRE(q_heads <= 65536 && kv_heads <= 65536, FP4_ERR_SHAPE, "q_heads=%d kv_heads=%d too large", q_heads,
                kv_heads);
    if (tokens == 0 || q_heads + kv_heads == 0) return ok();
    const int64_t wq = (int64_t)q_heads * head_dim, wk = (int64_t)kv_heads * head_dim;
    if (q_heads) {
        FP4_PTR(q);
        FP4_PTR(q_out);
        if (int e = check_ld(ld_q, wq, "ld_q")) return e;
        if (int e = check_ld(ld_qo, wq, "ld_qo")) return e;
    }
    if (kv_heads) {
        FP4_PTR(k);
        FP4_PTR(k_out);
        if (int e = check_ld(ld_k, wk, "ld_k")) return e;
        if (int e = check_ld(ld_ko, wk, "ld_ko")) return e;
    }
    if (q_heads == 0) q_weight = nullptr;
    if (kv_heads == 0) k_weight = nullptr;
    FP4_REQUIRE(aligned16(q_weight), FP4_ERR_ALIGN, "q_weight is not 16-byte aligned");
    FP4_REQUIRE(aligned16(k_weight), FP4_ERR_ALIGN, "k_weight is not 16-byte aligned");
    if (rot_dim) {
        FP4_PTR(cos_sin);
        FP4_SCALAR_PTR(positions);
        FP4_REQUIRE(max_positions >= 0, FP4_ERR_INVALID, "negative max_positions=%lld", (long long)max_positions);
    }
    if (q_heads) {
        FP4_REQUIRE((q_out == q && ld_qo == ld_q) || !rows_overlap(q_out, ld_qo * 2, wq * 2, q, ld_q * 2, wq * 2, tokens),
                    FP4_ERR_INVALID, "q_out overlaps q without being q itself");
    }
    if (kv_heads) {
        FP4_REQUIRE((k_out == k && ld_ko == ld_k) || !rows_overlap(k_out, ld_ko * 2, wk * 2, k, ld_k * 2, wk * 2, tokens),
                    FP4_ERR_INVALID, "k_out overlaps k without being k itself");
    }
    if (q_heads && kv_heads) {
        FP4_REQUIRE(!rows_overlap(q_out, ld_qo * 2, wq * 2, k, ld_k * 2, wk * 2, tokens), FP4_ERR_INVALID,
                    "q_out overlaps k");
        FP4_REQUIRE(!rows_overlap(k_out, ld_ko * 2, wk * 2, q, ld_q * 2, wq * 2, tokens), FP4_ERR_INVALID,
                    "k_out overlaps q");
        FP4_REQUIRE(!rows_overlap(q_out, ld_qo * 2, wq * 2, k_out, ld_ko * 2, wk * 2, tokens), FP4_ERR_INVALID,
                    "q_out overlaps k_out");
    }
    const uint64_t weight_bytes = (uint64_t)head_dim * (weight_dtype == FP4_DT_F32 ? 4 : 2);
    // Addresses end at 2^57: no table is longer.
    const uint64_t places = (uint64_t)(max_positions < (int64_t)1 << 45 ? max_positions : (int64_t)1 << 45);
    const struct {
        const char* name;
        const void* start;
        uint64_t bytes;
    } read[] = {{"q_weight", q_weight, q_weight ? weight_bytes : 0},
                {"k_weight", k_weight, k_weight ? weight_bytes : 0},
                {"cos_sin", cos_sin, rot_dim ? places * rot_dim * 4 : 0},
                {"positions", positions, rot_dim ? (uint64_t)tokens * 4 : 0}};
    for (const auto& r : read) {
        FP4_REQUIRE(!q_heads || !run_overlaps(q_out, ld_qo * 2, wq * 2, tokens, r.start, r.bytes), FP4_ERR_INVALID,
                    "q_out overlaps %s", r.name);
        FP4_REQUIRE(!kv_heads || !run_overlaps(k_out, ld_ko * 2, wk * 2, tokens, r.start, r.bytes), FP4_ERR_INVALID,
                    "k_out overlaps %s", r.name);
    }
    fp4::QkNorm p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.tokens = tokens;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.ld_q = ld_q;
    p.ld_k = ld_k;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.w_f32 = weight_dtype == FP4_DT_F32;
    p.eps = eps;
    p.cos_sin = cos_sin;
    p.max_positions = max_positions;
    p.rot_dim = rot_dim;
    p.interleaved = interleaved != 0;
    p.positions = positions;
    p.q_out = static_cast<uint16_t*>(q_out);
    p.ld_qo = ld_qo;
    p.k_out = static_cast<uint16_t*>(k_out);
    p.ld_ko = ld_ko;
    return hip_status(fp4::launch_qk_norm_rope(p, static_cast<hipStream_t>(stream)), "fp4_qk_norm_rope launch");
}

size_t fp4_kv_reserve_workspace_bytes(int64_t batch, int64_t num_pages) {
    return batch > 0 && num_pages >= 0 ? fp4::kv_reserve_workspace_bytes(batch, num_pages) : 0;
}

int fp4_kv_reserve(const fp4_kv_cache* cache, const fp4_kv_pages* pages, const int32_t* new_tokens, int32_t* slots,
                   int64_t max_new, int32_t* n_short, void* workspace, size_t workspace_bytes, void* stream) {
    if (int e = check_cache(cache, false)) return e;
    if (int e = check_pages(pages)) return e;
    if (int e = check_same_pool(cache, pages)) return e;
    FP4_REQUIRE(max_new >= 0, FP4_ERR_INVALID, "negative max_new=%lld", (long long)max_new);
    if (pages->batch == 0) return ok();
    FP4_SCALAR_PTR(new_tokens);
    FP4_SCALAR_PTR(n_short);
    if (max_new) { FP4_SCALAR_PTR(slots); }
    const size_t need = fp4::kv_reserve_workspace_bytes(pages->batch, pages->num_pages);
    FP4_REQUIRE(workspace != nullptr && workspace_bytes >= need, FP4_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
                need, workspace ? workspace_bytes : (size_t)0);
    FP4_REQUIRE(aligned16(workspace), FP4_ERR_ALIGN, "workspace is not 16-byte aligned");
    return hip_status(fp4::launch_kv_reserve(*cache, *pages, new_tokens, slots, max_new, n_short, workspace,
                                             static_cast<hipStream_t>(stream)),
                      "fp4_kv_reserve launch");
}

int fp4_kv_fork(const fp4_kv_pages* pages, const int32_t* pairs, int64_t n, int64_t page_size, void* stream) {
    if (int e = check_pages(pages)) return e;
    if (int e = check_page_size(page_size)) return e;
    FP4_REQUIRE(n >= 0, FP4_ERR_INVALID, "negative n=%lld", (long long)n);
    FP4_REQUIRE(n < kMaxList, FP4_ERR_SHAPE, "n=%lld too large", (long long)n);
    if (n == 0 || pages->batch == 0) return ok();
    FP4_SCALAR_PTR(pairs);
    return hip_status(fp4::launch_kv_fork(*pages, pairs, n, page_size, static_cast<hipStream_t>(stream)),
                      "fp4_kv_fork launch");
}

int fp4_kv_free(const fp4_kv_pages* pages, const int32_t* seqs, int64_t n, const int32_t* keep_lens, int64_t page_size,
                void* stream) {
    if (int e = check_pages(pages)) return e;
    if (int e = check_page_size(page_size)) return e;
    FP4_REQUIRE(n >= 0, FP4_ERR_INVALID, "negative n=%lld", (long long)n);
    FP4_REQUIRE(n < kMaxList, FP4_ERR_SHAPE, "n=%lld too large", (long long)n);
    if (n == 0 || pages->batch == 0) return ok();
    FP4_SCALAR_PTR(seqs);
    if (keep_lens) { FP4_SCALAR_PTR(keep_lens); }
    return hip_status(fp4::launch_kv_free(*pages, seqs, n, keep_lens, page_size, static_cast<hipStream_t>(stream)),
                      "fp4_kv_free launch");
}

int fp4_kv_compact(const fp4_kv_cache* cache, const fp4_kv_pages* pages, const int32_t* accepted, int64_t max_accepted,
                   const int32_t* accepted_lens, void* stream) {
    return kv_compact(cache, pages, accepted, max_accepted, accepted_lens, false, nullptr, 0, stream,
                      "fp4_kv_compact launch");
}

int fp4_kv_compact_reserved(const fp4_kv_cache* cache, const fp4_kv_pages* pages, const int32_t* accepted,
                            int64_t max_accepted, const int32_t* accepted_lens, const int32_t* slots, int64_t max_new,
                            void* stream) {
    FP4_REQUIRE(max_new >= 0, FP4_ERR_INVALID, "negative max_new=%lld", (long long)max_new);
    return kv_compact(cache, pages, accepted, max_accepted, accepted_lens, true, slots, max_new, stream,
                      "fp4_kv_compact_reserved launch");
}

int fp4_kv_copy_pages(const fp4_kv_cache* src, const fp4_kv_cache* dst, const int32_t* src_pages,
                      const int32_t* dst_pages, int64_t n, void* stream) {
    if (int e = check_cache(src, false)) return e;
    if (int e = check_cache(dst, false)) return e;
    FP4_REQUIRE(src->d == dst->d && src->page_size == dst->page_size, FP4_ERR_INVALID,
                "src has d=%lld page_size=%lld, dst d=%lld page_size=%lld", (long long)src->d, (long long)src->page_size,
                (long long)dst->d, (long long)dst->page_size);
    FP4_REQUIRE(n >= 0, FP4_ERR_INVALID, "negative n=%lld", (long long)n);
    if (n == 0 || src->num_pages == 0 || dst->num_pages == 0 || src->d == 0) return ok();
    FP4_REQUIRE((src->v_codes == nullptr) == (dst->v_codes == nullptr), FP4_ERR_INVALID,
                "one of src and dst has no values");
    FP4_REQUIRE(n < ((int64_t)1 << 24) / fp4::kv_copy_blocks(*src), FP4_ERR_SHAPE, "n=%lld pages too large for one call",
                (long long)n);
    FP4_SCALAR_PTR(src_pages);
    FP4_SCALAR_PTR(dst_pages);
    return hip_status(fp4::launch_kv_copy_pages(*src, *dst, src_pages, dst_pages, n, static_cast<hipStream_t>(stream)),
                      "fp4_kv_copy_pages launch");
}

size_t fp4_attn_tree_workspace_bytes(int64_t batch, int drafts, int q_heads, int head_dim, int kv_heads) {
    if (batch <= 0 || drafts < 1 || drafts > 64 || check_heads(q_heads, kv_heads, head_dim) != FP4_OK) return 0;
    return fp4::attn_tree_workspace_bytes(drafts, q_heads, head_dim, kv_heads);
}

int fp4_attn_tree_mx(const void* q, int64_t ld_q, const fp4_kv_cache* cache, const int32_t* page_table, int64_t max_pages,
                     const int32_t* seq_lens, const int32_t* draft_lens, const uint64_t* tree_mask, int64_t batch,
                     int drafts, int q_heads, int kv_heads, int head_dim, float scale, void* out, int64_t ld_out,
                     void* workspace, size_t workspace_bytes, void* stream) {
    if (int e = check_heads(q_heads, kv_heads, head_dim)) return e;
    if (int e = check_cache(cache, true)) return e;
    const int64_t width = (int64_t)q_heads * head_dim;
    FP4_REQUIRE(cache->d == (int64_t)kv_heads * head_dim, FP4_ERR_SHAPE, "the cache has d=%lld, kv_heads * head_dim is %lld",
                (long long)cache->d, (long long)kv_heads * head_dim);
    FP4_REQUIRE(drafts >= 1 && drafts <= 64, FP4_ERR_INVALID, "drafts=%d outside [1, 64]", drafts);
    FP4_REQUIRE(batch >= 0 && max_pages >= 0, FP4_ERR_INVALID, "negative size batch=%lld max_pages=%lld", (long long)batch,
                (long long)max_pages);
    FP4_REQUIRE(batch < 65536 && max_pages < (int64_t)1 << 31, FP4_ERR_SHAPE, "batch=%lld or max_pages=%lld too large",
                (long long)batch, (long long)max_pages);
    if (int e = check_scale(scale)) return e;
    if (batch == 0) return ok();
    FP4_PTR(q);
    FP4_PTR(out);
    if (int e = check_ld(ld_q, width, "ld_q")) return e;
    if (int e = check_ld(ld_out, width, "ld_out")) return e;
    if (max_pages) { FP4_SCALAR_PTR(page_table); }
    FP4_SCALAR_PTR(seq_lens);
    FP4_REQUIRE((reinterpret_cast<uintptr_t>(draft_lens) & 3u) == 0, FP4_ERR_ALIGN, "draft_lens is not 4-byte aligned");
    FP4_REQUIRE((reinterpret_cast<uintptr_t>(tree_mask) & 7u) == 0, FP4_ERR_ALIGN, "tree_mask is not 8-byte aligned");
    FP4_REQUIRE(!rows_overlap(out, ld_out * 2, width * 2, q, ld_q * 2, width * 2, batch * drafts), FP4_ERR_INVALID,
                "out overlaps q");
    const size_t need = fp4::attn_tree_workspace_bytes(drafts, q_heads, head_dim, kv_heads);
    FP4_REQUIRE(workspace != nullptr && workspace_bytes >= need, FP4_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
                need, workspace ? workspace_bytes : (size_t)0);
    FP4_REQUIRE(aligned16(workspace), FP4_ERR_ALIGN, "workspace is not 16-byte aligned");
    fp4::AttnTree p{};
    p.q = static_cast<const uint16_t*>(q);
    p.ld_q = ld_q;
    p.cache = *cache;
    p.page_table = page_table;
    p.max_pages = max_pages;
    p.seq_lens = seq_lens;
    p.draft_lens = draft_lens;
    p.tree_mask = tree_mask;
    p.batch = batch;
    p.drafts = drafts;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.scale = scale;
    p.out = static_cast<uint16_t*>(out);
    p.ld_out = ld_out;
    p.ws = workspace;
    return hip_status(fp4::launch_attn_tree(p, static_cast<hipStream_t>(stream)), "fp4_attn_tree_mx launch");
}

int fp4_attn_prompt(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int64_t seqs, int64_t tokens,
                    int q_heads, int kv_heads, int head_dim, int64_t ld_q, int64_t ld_k, int64_t ld_v, float scale,
                    void* out, int64_t ld_out, void* stream) {
    if (int e = check_heads(q_heads, kv_heads, head_dim)) return e;
    FP4_REQUIRE(seqs >= 0 && tokens >= 0, FP4_ERR_INVALID, "negative size seqs=%lld tokens=%lld", (long long)seqs,
                (long long)tokens);
    FP4_REQUIRE(tokens < (int64_t)1 << 30 && seqs < kMaxList, FP4_ERR_SHAPE, "tokens=%lld or seqs=%lld too large",
                (long long)tokens, (long long)seqs);
    FP4_REQUIRE(fp4::attn_prompt_tiles(seqs, tokens, head_dim) < ((int64_t)1 << 23) / q_heads, FP4_ERR_SHAPE,
                "tokens=%lld, seqs=%lld and q_heads=%d give too many row tiles (2^23)", (long long)tokens, (long long)seqs,
                q_heads);
    if (int e = check_scale(scale)) return e;
    if (seqs == 0 || tokens == 0) return ok();
    const int64_t wq = (int64_t)q_heads * head_dim, wk = (int64_t)kv_heads * head_dim;
    FP4_PTR(q);
    FP4_PTR(k);
    FP4_PTR(v);
    FP4_PTR(out);
    FP4_SCALAR_PTR(cu_seqlens);
    if (int e = check_ld(ld_q, wq, "ld_q")) return e;
    if (int e = check_ld(ld_k, wk, "ld_k")) return e;
    if (int e = check_ld(ld_v, wk, "ld_v")) return e;
    if (int e = check_ld(ld_out, wq, "ld_out")) return e;
    FP4_REQUIRE(ld_k < (int64_t)1 << 24 && ld_v < (int64_t)1 << 24, FP4_ERR_SHAPE, "ld_k=%lld or ld_v=%lld too large (2^24)",
                (long long)ld_k, (long long)ld_v);
    FP4_REQUIRE(!rows_overlap(out, ld_out * 2, wq * 2, q, ld_q * 2, wq * 2, tokens), FP4_ERR_INVALID, "out overlaps q");
    FP4_REQUIRE(!rows_overlap(out, ld_out * 2, wq * 2, k, ld_k * 2, wk * 2, tokens), FP4_ERR_INVALID, "out overlaps k");
    FP4_REQUIRE(!rows_overlap(out, ld_out * 2, wq * 2, v, ld_v * 2, wk * 2, tokens), FP4_ERR_INVALID, "out overlaps v");
    fp4::AttnPrompt p{};
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.cu_seqlens = cu_seqlens;
    p.seqs = seqs;
    p.tokens = tokens;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.head_dim = head_dim;
    p.ld_q = ld_q;
    p.ld_k = ld_k;
    p.ld_v = ld_v;
    p.scale = scale;
    p.out = static_cast<uint16_t*>(out);
    p.ld_out = ld_out;
    return hip_status(fp4::launch_attn_prompt(p, static_cast<hipStream_t>(stream)), "fp4_attn_prompt launch");
}

}  // extern "C"
