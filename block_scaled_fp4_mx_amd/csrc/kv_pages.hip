// Pages of the MXFP4 cache: reserving (with copy on write), forking, freeing,
// committing drafted rows, and copying whole pages.
//
// A page holds page_size consecutive rows, so its codes and its scales are each
// one contiguous run of bytes whose start is 16-byte aligned (page_size is a
// multiple of 16); a page copy is four plain copies.  Which page a sequence gets
// is decided by prefix sums over the sequences and over the free pages in
// ascending order, never by the order in which workgroups arrive, so equal
// states give equal tables.  The only atomics are integer counts.
//
// All but copy_pages are bound by latency: a launch and two to four round trips to
// memory.  64 sequences of 200 .. 4096 tokens in pages of 64 rows of 1024 values, 8
// new tokens each: free 3.0 us, plan 6.3 (7.0 with the references asked for after the
// sequences' needs), apply 2.5 .. 3.2, compact 5.6 (7.7 with one array read after
// another), by a reservation's slots 6.2.  16 sequences forked into 8 each: fork 4.2;
// apply 4.7 where each child copies its last page (6.3 with one workgroup to a sequence
// instead of 8).
#include "fp4_internal.h"

namespace fp4 {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kScanPages = 8;               // page references per lane and round of the free-page scan
constexpr int kThreads = 256;
constexpr int kReserveSplit = 8;            // workgroups per sequence that carry out a reservation
constexpr int kCopyUnits = 4;               // 16-byte units per lane of a page copy
constexpr int kMoveUnits = 8;               // units per lane and round of a row move

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// Reservation of one sequence, from the plan to its execution.
struct Plan {
    int32_t first;      // index of its first page in the list of taken pages
    int32_t need;       // new pages behind the table row's used entries
    int32_t count;      // used entries before the call
    int32_t source;     // its last page, if others hold it too (taken page `first` gets its rows), else -1
};

struct ReserveWs {
    int32_t* refused;   // one word: 1 = the pool or a table row is too small
    Plan* plan;         // [batch]
    int32_t* taken;     // [num_pages] the pages handed out, ascending
};

__host__ __device__ inline ReserveWs reserve_ws(void* ws, int64_t batch) {
    uint8_t* p = static_cast<uint8_t*>(ws);
    return ReserveWs{reinterpret_cast<int32_t*>(p), reinterpret_cast<Plan*>(p + 16),
                     reinterpret_cast<int32_t*>(p + 16 + batch * (int64_t)sizeof(Plan))};
}

__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {       // inclusive
#pragma unroll
    for (int m = 1; m < 64; m *= 2) {
        const int64_t o = __shfl_up(v, m, 64);
        if (lane >= m) v += o;
    }
    return v;
}

// Exclusive prefix of v over the workgroup; the sums of v and w over all threads in
// `total` and `total_w`.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t w, int64_t* sums, int64_t& total, int64_t& total_w) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t in = wave_scan(v, lane);
    const int64_t in_w = __any(w != 0) ? wave_scan(w, lane) : 0;
    __syncthreads();                                                       // sums free again
    if (lane == 63) sums[wave] = in, sums[kPlanWaves + wave] = in_w;
    __syncthreads();
    int64_t before = 0, all = 0, all_w = 0;
#pragma unroll 4
    for (int i = 0; i < kPlanWaves; ++i) {
        before += i < wave ? sums[i] : 0;
        all += sums[i];
        all_w += sums[kPlanWaves + i];
    }
    total = all;
    total_w = all_w;
    return before + in - v;
}

__device__ __forceinline__ int32_t held_pages(const fp4_kv_pages& t, int64_t b) {
    return (int32_t)min((int64_t)max(t.page_counts[b], 0), t.max_pages);
}

// One workgroup: what each sequence needs (in order), then the free pages in
// ascending order up to that many.  The reference counts of a 32768-page pool
// are 128 KiB, so one workgroup's read of them is short, and it stops at the
// last page needed.  A pool of a million pages costs the same while low ones are free,
// and 0.6 ms where only its last 4096 are.
__global__ __launch_bounds__(kPlanThreads) void reserve_plan_kernel(fp4_kv_pages t, const int32_t* new_tokens,
                                                                    int64_t page_size, int32_t* n_short, ReserveWs ws) {
    __shared__ int64_t sums[2 * kPlanWaves];
    // References of this lane's pages of a round; the first round's are on their way
    // while the sequences' needs are worked out.
    int32_t refs[kScanPages];
    auto load_refs = [&](int64_t q) {
#pragma unroll
        for (int i = 0; i < kScanPages; ++i) refs[i] = q + i < t.num_pages ? t.page_refs[q + i] : 1;
    };
    load_refs((int64_t)threadIdx.x * kScanPages);
    int64_t want_all = 0, over_all = 0;
    for (int64_t b0 = 0; b0 < t.batch; b0 += kPlanThreads) {
        const int64_t b = b0 + threadIdx.x;
        int64_t want = 0, over = 0;
        Plan p{0, 0, 0, -1};
        if (b < t.batch) {
            const int64_t len = max(t.seq_lens[b], 0), add = max(new_tokens[b], 0);
            p.count = held_pages(t, b);
            if (add > 0) {
                const int64_t pages = (len + add + page_size - 1) / page_size, last = len / page_size;
                over = max(pages - t.max_pages, (int64_t)0);
                p.need = (int32_t)max(min(pages, t.max_pages) - p.count, (int64_t)0);
                if (len % page_size && last < p.count) {
                    const int32_t page = t.page_table[b * t.max_pages + last];
                    if (page >= 0 && page < t.num_pages && t.page_refs[page] > 1) p.source = page;
                }
                want = p.need + (p.source >= 0);
            }
        }
        int64_t chunk, chunk_over;
        const int64_t first = want_all + block_scan(want, over, sums, chunk, chunk_over);
        want_all += chunk;
        over_all += chunk_over;
        p.first = (int32_t)min(first, (int64_t)0x7FFFFFFF);               // past the pool only in a refused call
        if (b < t.batch) ws.plan[b] = p;
    }
    int64_t found = 0;
    for (int64_t q0 = 0; q0 < t.num_pages && found < want_all; q0 += kPlanThreads * kScanPages) {
        const int64_t q = q0 + (int64_t)threadIdx.x * kScanPages;
        if (q0) load_refs(q);
        uint32_t free_bits = 0;
#pragma unroll
        for (int i = 0; i < kScanPages; ++i) free_bits |= refs[i] == 0 ? 1u << i : 0u;
        int64_t chunk, none;
        int64_t rank = found + block_scan(__popc(free_bits), 0, sums, chunk, none);
        for (; free_bits && rank < want_all; ++rank, free_bits &= free_bits - 1)
            ws.taken[rank] = (int32_t)(q + __ffs(free_bits) - 1);
        found += chunk;
    }
    if (threadIdx.x == 0) {
        const int64_t missing = over_all + max(want_all - found, (int64_t)0);
        *n_short = (int32_t)min(missing, (int64_t)0x7FFFFFFF);
        *ws.refused = missing > 0;
    }
}

// Bytes [0, bytes) from src to dst (both 16-byte aligned), by `threads` threads.
__device__ __forceinline__ void copy_bytes(const uint8_t* src, uint8_t* dst, int64_t bytes, int64_t thread,
                                           int64_t threads) {
    const int64_t units = bytes / 16;
    for (int64_t u = thread; u < units; u += threads)
        reinterpret_cast<uint4*>(dst)[u] = reinterpret_cast<const uint4*>(src)[u];
    for (int64_t i = units * 16 + thread; i < bytes; i += threads) dst[i] = src[i];
}

// Carries the plan out: kReserveSplit workgroups per sequence share the row
// copy and the slots; the first one also updates the table, the count and the
// references.  Nothing that one of them writes is read by another: the page of
// a slot comes from the plan, or from table entries that stay as they are.
__global__ __launch_bounds__(kThreads) void reserve_apply_kernel(fp4_kv_cache c, fp4_kv_pages t,
                                                                 const int32_t* new_tokens, int32_t* slots,
                                                                 int64_t max_new, ReserveWs ws) {
    const int64_t b = blockIdx.x, ps = c.page_size;
    const int64_t tid = (int64_t)blockIdx.y * kThreads + threadIdx.x, threads = (int64_t)gridDim.y * kThreads;
    const Plan p = ws.plan[b];
    const int64_t len = max(t.seq_lens[b], 0), add = *ws.refused ? 0 : max(new_tokens[b], 0), last = len / ps;
    const int32_t* taken = ws.taken + p.first;
    const int copied = p.source >= 0;
    int32_t* row = t.page_table + b * t.max_pages;
    for (int64_t j = tid; j < max_new; j += threads) {
        int64_t slot = -1;
        if (j < add) {
            const int64_t pos = len + j, i = pos / ps;
            const int64_t page = i >= p.count ? taken[copied + i - p.count] : copied && i == last ? taken[0] : row[i];
            if (page >= 0 && page < t.num_pages) slot = page * ps + pos % ps;
        }
        slots[b * max_new + j] = (int32_t)slot;
    }
    if (add == 0) return;
    if (blockIdx.y == 0) {
        for (int i = threadIdx.x; i < p.need; i += kThreads) {
            const int32_t page = taken[copied + i];
            row[p.count + i] = page;
            t.page_refs[page] = 1;
        }
        if (threadIdx.x == 0) {
            t.page_counts[b] = p.count + p.need;
            if (copied) {
                row[last] = taken[0];
                t.page_refs[taken[0]] = 1;
                atomicSub(t.page_refs + p.source, 1);
            }
        }
    }
    if (!copied) return;
    const int64_t rows = len % ps, cb = c.d / 2, sb = c.d / 32;
    const int64_t from = (int64_t)p.source * ps, to = (int64_t)taken[0] * ps;
    copy_bytes(c.k_codes + from * cb, c.k_codes + to * cb, rows * cb, tid, threads);
    copy_bytes(c.k_scales + from * sb, c.k_scales + to * sb, rows * sb, tid, threads);
    if (c.v_codes) {
        copy_bytes(c.v_codes + from * cb, c.v_codes + to * cb, rows * cb, tid, threads);
        copy_bytes(c.v_scales + from * sb, c.v_scales + to * sb, rows * sb, tid, threads);
    }
}

// One workgroup per pair.  No workgroup reads what another writes: a pair whose
// source is a target of the call, or whose target an earlier pair names, does nothing.
__global__ __launch_bounds__(kThreads) void fork_kernel(fp4_kv_pages t, const int32_t* pairs, int64_t n,
                                                        int64_t page_size) {
    const int64_t i = blockIdx.x;
    const int32_t from = pairs[2 * i], to = pairs[2 * i + 1];
    if (from < 0 || from >= t.batch || to < 0 || to >= t.batch) return;
    bool clash = from == to;
    for (int64_t j = threadIdx.x; j < n; j += kThreads) {
        const int32_t other = pairs[2 * j + 1];
        clash |= other == from || (j < i && other == to);
    }
    if (__syncthreads_or(clash)) return;
    if (t.page_counts[to] != 0) return;
    const int64_t len = max(t.seq_lens[from], 0);
    const int64_t count = min((len + page_size - 1) / page_size, (int64_t)held_pages(t, from));
    for (int64_t p = threadIdx.x; p < count; p += kThreads) {
        const int32_t page = t.page_table[from * t.max_pages + p];
        t.page_table[to * t.max_pages + p] = page;
        if (page >= 0 && page < t.num_pages) atomicAdd(t.page_refs + page, 1);
    }
    __syncthreads();                                          // every wave has read the target's count
    if (threadIdx.x == 0) {
        t.page_counts[to] = (int32_t)count;
        t.seq_lens[to] = (int32_t)min(len, count * page_size);
    }
}

// One workgroup per listed sequence; of an id listed twice the first entry acts.
__global__ __launch_bounds__(kThreads) void free_kernel(fp4_kv_pages t, const int32_t* seqs, const int32_t* keep_lens,
                                                        int64_t page_size) {
    const int64_t i = blockIdx.x;
    const int32_t b = seqs[i];
    if (b < 0 || b >= t.batch) return;
    bool earlier = false;
    for (int64_t j = threadIdx.x; j < i; j += kThreads) earlier |= seqs[j] == b;
    if (__syncthreads_or(earlier)) return;
    const int64_t count = held_pages(t, b);
    const int64_t len = min((int64_t)max(t.seq_lens[b], 0), keep_lens ? (int64_t)max(keep_lens[i], 0) : (int64_t)0);
    const int64_t kept = min((len + page_size - 1) / page_size, count);
    int32_t* row = t.page_table + (int64_t)b * t.max_pages;
    for (int64_t p = kept + threadIdx.x; p < count; p += kThreads) {
        const int32_t page = row[p];
        row[p] = -1;
        if (page >= 0 && page < t.num_pages) atomicSub(t.page_refs + page, 1);
    }
    __syncthreads();                                          // every wave has read the count and the length
    if (threadIdx.x == 0) {
        t.page_counts[b] = (int32_t)kept;
        t.seq_lens[b] = (int32_t)min(len, kept * page_size);
    }
}

// The rows of one or two arrays (key and value codes, or scales) in units of T, and
// their way through registers: units u0 .. u0 + w of n rows.  from/to: rows in LDS,
// -1 = none.
template <typename T>
struct Rows {
    uint8_t *a, *b;                          // b: NULL for one array
    int64_t bytes;                           // of a row
    int per, all;                            // units of an array's row, of both
    __device__ Rows(uint8_t* x, uint8_t* y, int64_t row_bytes)
        : a(x), b(y), bytes(row_bytes), per((int)(row_bytes / sizeof(T))), all(y ? 2 * per : per) {}
    __device__ __forceinline__ T* at(int64_t row, int u) const {
        return reinterpret_cast<T*>((u < per ? a : b) + row * bytes) + (u < per ? u : u - per);
    }
    __device__ __forceinline__ int width(int n) const { return min(kThreads * kMoveUnits / n, all); }   // n <= 64: at least 32
    __device__ __forceinline__ void gather(T* v, int u0, int w, int n, const int64_t* from) const {
#pragma unroll
        for (int k = 0; k < kMoveUnits; ++k) {
            const int item = k * kThreads + threadIdx.x, i = item / w;
            if (k * kThreads < w * n && item < w * n && from[i] >= 0) v[k] = *at(from[i], u0 + item - i * w);
        }
    }
    __device__ __forceinline__ void scatter(const T* v, int u0, int w, int n, const int64_t* from, const int64_t* to) const {
#pragma unroll
        for (int k = 0; k < kMoveUnits; ++k) {
            const int item = k * kThreads + threadIdx.x, i = item / w;
            if (k * kThreads < w * n && item < w * n && from[i] >= 0) *at(to[i], u0 + item - i * w) = v[k];
        }
    }
};

// All reads of a unit of the rows before its writes; as a rule (8 rows of 4096 values,
// 64 of 512) everything is read before one meeting of the waves.
template <typename T>
__device__ __forceinline__ void move_rows(const fp4_kv_cache& c, const int64_t* from, const int64_t* to, int n) {
    const Rows<u32x4> codes(c.k_codes, c.v_codes, c.d / 2);
    const Rows<T> scales(c.k_scales, c.v_scales, c.d / 32);
    const int cw = codes.width(n), sw = scales.width(n);
    u32x4 v[kMoveUnits];
    T s[kMoveUnits];
    for (int u = 0, x = 0; u < codes.all || x < scales.all; u += cw, x += sw) {
        const int nu = max(min(cw, codes.all - u), 0), nx = max(min(sw, scales.all - x), 0);
        if (nu) codes.gather(v, u, nu, n, from);
        if (nx) scales.gather(s, x, nx, n, from);
        __syncthreads();
        if (nu) codes.scatter(v, u, nu, n, from, to);
        if (nx) scales.scatter(s, x, nx, n, from, to);
    }
}

// Cache row of a position below the sequence's held pages, and its page; -1: no page of the pool.
__device__ __forceinline__ int64_t row_of(const fp4_kv_pages& t, int64_t b, int64_t pos, int64_t ps, int64_t& page) {
    page = t.page_table[b * t.max_pages + pos / ps];
    return page >= 0 && page < t.num_pages ? page * ps + pos % ps : -1;
}

// One workgroup per sequence: moves the accepted rows (kept in registers between
// the reads and the writes), then grows the length.  With the slots of a reservation
// it commits tokens up to the first whose slot is not its position's row: slots of a
// refused reservation are -1, and those of one that has been committed, or whose page
// has been copied or let go since, are other rows.  They are also what tells of a
// short pool: the table alone cannot, the rest of a last page looks like reserved rows.
__global__ __launch_bounds__(kThreads) void compact_kernel(fp4_kv_cache c, fp4_kv_pages t, const int32_t* accepted,
                                                           int64_t max_accepted, const int32_t* accepted_lens,
                                                           const int32_t* slots, int64_t max_new) {
    __shared__ int64_t from[64], to[64];
    __shared__ int32_t granted;
    const int64_t b = blockIdx.x, ps = c.page_size;
    const int64_t len = max(t.seq_lens[b], 0), room = max(held_pages(t, b) * ps - len, (int64_t)0);
    int64_t n = max(accepted_lens[b], 0);
    if (accepted) n = min(n, max_accepted);
    n = min(n, room);
    if (slots) {
        n = min(n, max_new);
        if (threadIdx.x == 0) granted = (int32_t)n;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < n; i += kThreads) {
            int64_t page;
            const int64_t row = row_of(t, b, len + i, ps, page);
            if (row < 0 || slots[b * max_new + i] != row) {
                atomicMin(&granted, (int32_t)i);
                break;
            }
        }
        __syncthreads();
        n = granted;
    }
    if (n == 0) return;
    if (accepted) {
        // The page of the first uncommitted row may be shared by forks since the rows
        // were reserved: it is written unless another holder's tokens reach that far, or
        // that holder commits in this call too.  Only one of them can have reserved rows
        // there (a reservation copies a shared page), so the call is in error and neither
        // writes.  A holder that commits counts by its accepted_lens and its first slot,
        // which stay as they are: its length is written by its own workgroup meanwhile.
        const int64_t last = len / ps;
        const int32_t first_page = len % ps ? t.page_table[b * t.max_pages + last] : -1;
        bool alone = true;
        if (first_page >= 0 && first_page < t.num_pages && t.page_refs[first_page] > 1) {
            bool seen = false;
            for (int64_t o = threadIdx.x; o < t.batch; o += kThreads)
                seen |= o != b && last < held_pages(t, o) && t.page_table[o * t.max_pages + last] == first_page &&
                        ((accepted_lens[o] > 0 && (!slots || slots[o * max_new] >= 0)) || t.seq_lens[o] > len);
            alone = !__syncthreads_or(seen);
        }
        if (threadIdx.x < 64) {
            int64_t row[2] = {-1, -1};
            const int64_t i = threadIdx.x, a = i < n ? accepted[b * max_accepted + i] : -1;
            if (a >= 0 && a < room && a != i) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    int64_t page;
                    const int64_t r = row_of(t, b, len + (k ? i : a), ps, page);
                    if (r >= 0 && (k == 0 || (page == first_page ? alone : t.page_refs[page] == 1))) row[k] = r;
                }
                if (slots && (a >= max_new || slots[b * max_new + a] != row[0])) row[0] = -1;
            }
            from[i] = row[1] < 0 ? -1 : row[0];
            to[i] = row[1];
        }
        __syncthreads();
        if (c.d % 128 == 0)
            move_rows<uint32_t>(c, from, to, (int)n);
        else
            move_rows<uint8_t>(c, from, to, (int)n);
    }
    __syncthreads();                                          // every wave has read the length
    if (threadIdx.x == 0) t.seq_lens[b] = (int32_t)(len + n);
}

// Whole pages: kThreads * kCopyUnits units of one pair to a workgroup; a pair's
// units run through key codes, key scales, value codes, value scales.  Bound by
// HBM; neither side is read again soon, so loads and stores pass the caches by.
// 8192 pages of 64 rows of 1024 values (1.14 GB read and written): 223 us, 5.1 TB/s;
// 234 us with plain loads and stores, 338 us with those and 8 units to a lane.
__global__ __launch_bounds__(kThreads) void copy_pages_kernel(fp4_kv_cache src, fp4_kv_cache dst,
                                                              const int32_t* src_pages, const int32_t* dst_pages,
                                                              uint32_t blocks_per_pair) {
    const uint32_t i = blockIdx.x / blocks_per_pair, part = blockIdx.x % blocks_per_pair;
    const int64_t a = src_pages[i], b = dst_pages[i];
    if (a < 0 || a >= src.num_pages || b < 0 || b >= dst.num_pages) return;
    const int64_t cu = src.page_size * (src.d / 32), su = src.page_size * (src.d / 32) / 16;   // 16-byte units
    const int64_t total = (cu + su) * (src.v_codes ? 2 : 1);
    const int64_t u0 = (int64_t)part * kThreads * kCopyUnits + threadIdx.x;
    u32x4 v[kCopyUnits], *to[kCopyUnits];
#pragma unroll
    for (int k = 0; k < kCopyUnits; ++k) {
        int64_t u = u0 + (int64_t)k * kThreads;
        if (u >= total) continue;
        const bool val = u >= cu + su;
        if (val) u -= cu + su;
        const bool scale = u >= cu;
        if (scale) u -= cu;
        const uint8_t* s = scale ? (val ? src.v_scales : src.k_scales) : (val ? src.v_codes : src.k_codes);
        uint8_t* d = scale ? (val ? dst.v_scales : dst.k_scales) : (val ? dst.v_codes : dst.k_codes);
        const int64_t n = scale ? su : cu;
        v[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(s) + a * n + u);
        to[k] = reinterpret_cast<u32x4*>(d) + b * n + u;
    }
#pragma unroll
    for (int k = 0; k < kCopyUnits; ++k)
        if (u0 + (int64_t)k * kThreads < total) __builtin_nontemporal_store(v[k], to[k]);
}

}  // namespace

size_t kv_reserve_workspace_bytes(int64_t batch, int64_t num_pages) {
    return (size_t)(16 + batch * (int64_t)sizeof(Plan) + num_pages * 4);
}

hipError_t launch_kv_reserve(const fp4_kv_cache& c, const fp4_kv_pages& t, const int32_t* new_tokens, int32_t* slots,
                             int64_t max_new, int32_t* n_short, void* ws, hipStream_t s) {
    const ReserveWs w = reserve_ws(ws, t.batch);
    reserve_plan_kernel<<<1, kPlanThreads, 0, s>>>(t, new_tokens, c.page_size, n_short, w);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    reserve_apply_kernel<<<dim3((unsigned)t.batch, kReserveSplit), kThreads, 0, s>>>(c, t, new_tokens, slots, max_new, w);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const fp4_kv_pages& t, const int32_t* pairs, int64_t n, int64_t page_size, hipStream_t s) {
    fork_kernel<<<(unsigned)n, kThreads, 0, s>>>(t, pairs, n, page_size);
    return hipGetLastError();
}

hipError_t launch_kv_free(const fp4_kv_pages& t, const int32_t* seqs, int64_t n, const int32_t* keep_lens,
                          int64_t page_size, hipStream_t s) {
    free_kernel<<<(unsigned)n, kThreads, 0, s>>>(t, seqs, keep_lens, page_size);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const fp4_kv_cache& c, const fp4_kv_pages& t, const int32_t* accepted,
                             int64_t max_accepted, const int32_t* accepted_lens, const int32_t* slots, int64_t max_new,
                             hipStream_t s) {
    compact_kernel<<<(unsigned)t.batch, kThreads, 0, s>>>(c, t, accepted, max_accepted, accepted_lens, slots, max_new);
    return hipGetLastError();
}

// Workgroups of one copied page; the caller keeps n times it within a grid.
int64_t kv_copy_blocks(const fp4_kv_cache& c) {
    const int64_t cu = c.page_size * (c.d / 32), su = cu / 16, total = (cu + su) * (c.v_codes ? 2 : 1);
    return (total + kThreads * kCopyUnits - 1) / (kThreads * kCopyUnits);
}

hipError_t launch_kv_copy_pages(const fp4_kv_cache& src, const fp4_kv_cache& dst, const int32_t* src_pages,
                                const int32_t* dst_pages, int64_t n, hipStream_t s) {
    const int64_t per = kv_copy_blocks(src);
    copy_pages_kernel<<<(unsigned)(n * per), kThreads, 0, s>>>(src, dst, src_pages, dst_pages, (uint32_t)per);
    return hipGetLastError();
}

}  // namespace fp4
