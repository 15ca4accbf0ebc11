// sm_103a page tables and cache writes (afx_kv_tables, afx_kv_write).
//
// The cache of keys and values is a pool of pages of P tokens; a request's
// cached tokens 0 .. len-1 live in the pages of its row of the block table.
//
// kv_tables_kernel turns old and new lengths into page moves and a slot for
// every new token.  With p(x) = ceil(x / P), request r takes
// max(0, p(new) - p(old)) pages or gives back max(0, p(old) - p(new)); the
// exclusive sums of those counts, in request order, place every page:
// growth page j is the (M-1-j)-th page given back while j < M (M pages come
// back in all), then the free stack from its top.  No page is read from
// where the same call writes one, so all of it runs in one kernel: every
// CTA computes the sums over all requests for itself (8 bytes a request,
// from L2) into shared memory and then takes its share of the tokens and
// pages, finding a token's request by bisection of the sums.
// Bound: latency (a launch, the lengths, the sums, a bisection, the table, the
// store); the 8 bytes a new token written come to less.  4096 requests with a
// new prompt for one in ten (300,000 new tokens): 16 us alone with cold caches;
// one step of 8 requests: 7 us, less than a call takes the host.
//
// kv_write_kernel copies each new token's keys and values into its slot:
// 2 * heads * dim elements read and written once, 16 bytes a lane and four
// loads in flight a lane.  Bound: HBM bandwidth: 32,701 tokens of 8 heads of
// 128, 268 MB moved, in 42 us a call, 6.3 TB/s; one step of 64 tokens 3 us alone.
#include "afx_serving.cuh"

namespace afx {
namespace serve {
namespace {

constexpr int kTabThreads = 1024;
constexpr uint32_t kMaxRequests = AFX_KV_MAX_REQUESTS;

struct TablesArgs {
    const int32_t *old_len, *new_len;
    int32_t* table;
    int32_t* stack;
    const int32_t* count;
    int32_t* count_out;
    int32_t *starts, *slots, *positions;
    int32_t* status;
    uint32_t n, cols, n_pages, max_tokens, shift;  // P = 1 << shift
    uint32_t wide;  // slots and positions are 16-byte aligned
};

struct Sums {
    uint64_t add, grow, drop;
};

// Exclusive sums of v over the CTA's threads; *total gets the sums.
__device__ Sums block_exclusive(Sums v, Sums* total) {
    __shared__ Sums warp_sums[kTabThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t a = __shfl_up_sync(0xFFFFFFFFu, inc.add, d), g = __shfl_up_sync(0xFFFFFFFFu, inc.grow, d),
                       f = __shfl_up_sync(0xFFFFFFFFu, inc.drop, d);
        if (lane >= d) {
            inc.add += a;
            inc.grow += g;
            inc.drop += f;
        }
    }
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    Sums w = lane < (static_cast<int>(blockDim.x) >> 5) ? warp_sums[lane] : Sums{0, 0, 0};
    const Sums own = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t a = __shfl_up_sync(0xFFFFFFFFu, w.add, d), g = __shfl_up_sync(0xFFFFFFFFu, w.grow, d),
                       f = __shfl_up_sync(0xFFFFFFFFu, w.drop, d);
        if (lane >= d) {
            w.add += a;
            w.grow += g;
            w.drop += f;
        }
    }
    *total = Sums{__shfl_sync(0xFFFFFFFFu, w.add, 31), __shfl_sync(0xFFFFFFFFu, w.grow, 31), __shfl_sync(0xFFFFFFFFu, w.drop, 31)};
    const uint64_t before_add = __shfl_sync(0xFFFFFFFFu, w.add - own.add, warp), before_grow = __shfl_sync(0xFFFFFFFFu, w.grow - own.grow, warp),
                   before_drop = __shfl_sync(0xFFFFFFFFu, w.drop - own.drop, warp);
    return Sums{before_add + inc.add - v.add, before_grow + inc.grow - v.grow, before_drop + inc.drop - v.drop};
}

// The last r with first[r] <= x (first[0] = 0, nondecreasing, n entries):
// the request that item x of a count with those exclusive sums belongs to.
__device__ __forceinline__ uint32_t owner(const uint32_t* first, uint32_t n, uint32_t x) {
    uint32_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) >> 1;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

struct PageMoves {
    const TablesArgs& a;
    const uint32_t *t0, *g0, *d0;
    uint32_t count, grow, drop;

    __device__ uint32_t pages(uint32_t len) const { return (len >> a.shift) + ((len & ((1u << a.shift) - 1)) != 0); }
    // the f-th page given back
    __device__ int32_t freed(uint32_t f) const {
        const uint32_t r = owner(d0, a.n, f);
        return a.table[static_cast<uint64_t>(r) * a.cols + pages(a.new_len[r]) + (f - d0[r])];
    }
    // the j-th page handed out
    __device__ int32_t taken(uint32_t j) const {
        return j < drop ? freed(drop - 1 - j) : a.stack[count - 1 - (j - drop)];
    }
};

__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const TablesArgs a) {
    extern __shared__ uint32_t sums[];
    uint32_t* t0 = sums;
    uint32_t* g0 = t0 + a.n + 1;
    uint32_t* d0 = g0 + a.n + 1;
    const uint32_t page_mask = (1u << a.shift) - 1;
    const uint64_t max_len = static_cast<uint64_t>(a.cols) << a.shift;
    wait_for_earlier();
    let_next_start();
    const int32_t have = *a.count;
    const uint32_t threads = blockDim.x, per = ceil_div(a.n, threads);
    const uint32_t r0 = min(a.n, threadIdx.x * per), r1 = min(a.n, r0 + per);

    Sums mine{0, 0, 0};
    int32_t bad = 0;
    for (uint32_t r = r0; r < r1; ++r) {
        const int32_t o = a.old_len[r], w = a.new_len[r];
        if (o < 0 || w < 0 || static_cast<uint64_t>(o) > max_len || static_cast<uint64_t>(w) > max_len) {
            bad = AFX_DEV_BAD_LENGTH;
            continue;
        }
        const uint32_t po = (o >> a.shift) + ((o & page_mask) != 0), pw = (w >> a.shift) + ((w & page_mask) != 0);
        mine.add += w > o ? w - o : 0;
        mine.grow += pw > po ? pw - po : 0;
        mine.drop += po > pw ? po - pw : 0;
    }
    Sums total;
    Sums at = block_exclusive(mine, &total);
    // all of it or nothing: a call that cannot be served changes no page
    if (total.add > a.max_tokens) bad |= AFX_DEV_BAD_LENGTH;
    if (have < 0 || static_cast<uint32_t>(have) > a.n_pages || have + total.drop > a.n_pages + total.grow)
        bad |= AFX_DEV_BAD_LENGTH;  // the count is not one of this pool, or pages came back twice
    else if (total.grow > have + total.drop)
        bad |= AFX_DEV_NO_PAGES;
    const bool refused = __syncthreads_or(bad) != 0;
    if (bad && blockIdx.x == 0) raise(a.status, bad);
    const uint32_t gid = blockIdx.x * threads + threadIdx.x, stride = gridDim.x * threads;
    if (refused) {
        for (uint32_t i = gid; i <= a.n; i += stride) a.starts[i] = 0;
        for (uint32_t i = gid; i < a.max_tokens; i += stride) a.slots[i] = a.positions[i] = -1;
        if (gid == 0) *a.count_out = have;
        return;
    }
    for (uint32_t r = r0; r < r1; ++r) {
        const int32_t o = a.old_len[r], w = a.new_len[r];
        const uint32_t po = (o >> a.shift) + ((o & page_mask) != 0), pw = (w >> a.shift) + ((w & page_mask) != 0);
        t0[r] = static_cast<uint32_t>(at.add);
        g0[r] = static_cast<uint32_t>(at.grow);
        d0[r] = static_cast<uint32_t>(at.drop);
        at.add += w > o ? w - o : 0;
        at.grow += pw > po ? pw - po : 0;
        at.drop += po > pw ? po - pw : 0;
    }
    __syncthreads();
    const uint32_t n_add = static_cast<uint32_t>(total.add), n_grow = static_cast<uint32_t>(total.grow),
                   n_drop = static_cast<uint32_t>(total.drop);
    const PageMoves mv{a, t0, g0, d0, static_cast<uint32_t>(have), n_grow, n_drop};

    if (gid == 0) *a.count_out = static_cast<int32_t>(have + n_drop - n_grow);
    for (uint32_t i = gid; i <= a.n; i += stride) a.starts[i] = static_cast<int32_t>(i < a.n ? t0[i] : n_add);
    for (uint32_t j = gid; j < n_grow; j += stride) {
        const uint32_t r = owner(g0, a.n, j);
        const int32_t page = mv.taken(j);
        if (page < 0 || static_cast<uint32_t>(page) >= a.n_pages) raise(a.status, AFX_DEV_BAD_PAGE);
        a.table[static_cast<uint64_t>(r) * a.cols + mv.pages(a.old_len[r]) + (j - g0[r])] = page;
    }
    bool wrong = false;  // an id outside the pool comes back; told at the end, where nothing waits for it
    for (uint32_t f = gid; f + n_grow < n_drop; f += stride) {
        const int32_t page = mv.freed(f);
        wrong |= static_cast<uint32_t>(page) >= a.n_pages;
        a.stack[have + f] = page;
    }
    // four tokens a thread: their request is looked up once, their page where it changes
    for (uint32_t t = 4 * gid; t < a.max_tokens; t += 4 * stride) {
        int32_t slot[4], pos[4];
        uint32_t r = t < n_add ? owner(t0, a.n, t) : 0, held = 0, seen_col = UINT32_MAX;
        int32_t page = -1;
        bool load = true;
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            slot[j] = pos[j] = -1;
            if (t + j >= n_add) continue;
            while (r + 1 < a.n && t0[r + 1] <= t + j) {
                ++r;
                load = true;
            }
            if (load) {
                held = a.old_len[r];
                load = false;
                seen_col = UINT32_MAX;
            }
            const uint32_t at_pos = held + (t + j - t0[r]), col = at_pos >> a.shift;
            if (col != seen_col) {
                // a page the request already has is in its row; a new one is
                // being written there by another thread, so it is worked out
                const uint32_t first_new = mv.pages(held);
                page = col < first_new ? a.table[static_cast<uint64_t>(r) * a.cols + col] : mv.taken(g0[r] + col - first_new);
                seen_col = col;
                if (page < 0 || static_cast<uint32_t>(page) >= a.n_pages) raise(a.status, AFX_DEV_BAD_PAGE);
            }
            pos[j] = static_cast<int32_t>(at_pos);
            if (page >= 0 && static_cast<uint32_t>(page) < a.n_pages)
                slot[j] = static_cast<int32_t>((static_cast<uint32_t>(page) << a.shift) | (at_pos & page_mask));
        }
        if (a.wide && t + 4 <= a.max_tokens) {
            *reinterpret_cast<int4*>(a.slots + t) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            *reinterpret_cast<int4*>(a.positions + t) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                if (t + j < a.max_tokens) {
                    a.slots[t + j] = slot[j];
                    a.positions[t + j] = pos[j];
                }
        }
    }
    if (wrong) raise(a.status, AFX_DEV_BAD_PAGE);
}

struct WriteArgs {
    const uint8_t* src[2];
    uint8_t* dst[2];
    const int32_t* slots;
    int32_t* status;
    uint64_t src_token, src_head;                  // bytes
    uint64_t dst_page, dst_token, dst_head;        // bytes
    uint32_t n_tokens, heads, row_bytes, shift, n_slots;
};

constexpr int kWriteThreads = 256;

// V: the bytes a lane moves at once (16, or 2 where the source's address or
// strides are not multiples of 16).
template <typename V>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const WriteArgs a) {
    wait_for_earlier();
    let_next_start();
    const uint32_t per_row = a.row_bytes / sizeof(V), per_token = per_row * a.heads;
    const uint64_t units = static_cast<uint64_t>(a.n_tokens) * per_token;
    const uint64_t step = static_cast<uint64_t>(gridDim.x) * kWriteThreads;
    constexpr int kAtOnce = 2;  // of keys and of values each
    for (uint64_t u0 = static_cast<uint64_t>(blockIdx.x) * kWriteThreads + threadIdx.x; u0 < units; u0 += kAtOnce * step) {
        V v[kAtOnce][2];
        uint64_t to[kAtOnce];
        bool real[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const uint64_t u = u0 + i * step;
            real[i] = u < units;
            if (!real[i]) continue;
            const uint32_t t = static_cast<uint32_t>(u / per_token), in = static_cast<uint32_t>(u - static_cast<uint64_t>(t) * per_token);
            const uint32_t h = in / per_row, c = in - h * per_row;
            const int32_t slot = __ldg(a.slots + t);
            const uint64_t from = t * a.src_token + h * a.src_head + c * sizeof(V);
#pragma unroll
            for (int p = 0; p < 2; ++p) v[i][p] = __ldg(reinterpret_cast<const V*>(a.src[p] + from));
            if (slot >= 0 && static_cast<uint32_t>(slot) >= a.n_slots) raise(a.status, AFX_DEV_BAD_PAGE);
            real[i] = slot >= 0 && static_cast<uint32_t>(slot) < a.n_slots;  // negative: padding
            to[i] = (static_cast<uint32_t>(slot) >> a.shift) * a.dst_page +
                    (static_cast<uint32_t>(slot) & ((1u << a.shift) - 1)) * a.dst_token + h * a.dst_head + c * sizeof(V);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
            if (real[i]) {
#pragma unroll
                for (int p = 0; p < 2; ++p) *reinterpret_cast<V*>(a.dst[p] + to[i]) = v[i][p];
            }
    }
}

bool page_shift(uint32_t page_tokens, uint32_t* shift) {
    for (uint32_t s = 4; s <= 8; ++s)
        if (page_tokens == 1u << s) {
            *shift = s;
            return true;
        }
    return false;
}

}  // namespace

afx_status check_cache(const afx_kv_cache* c, uint32_t* shift) {
    if (!c) return afx_fail(AFX_E_ARG, "null cache description", 0);
    if (c->format != AFX_FMT_BF16 && c->format != AFX_FMT_FP16)
        return afx_fail(AFX_E_ARG, "the cache holds BF16 or FP16", 0);
    if (!page_shift(c->page_tokens, shift))
        return afx_fail(AFX_E_ARG, "pages hold 16, 32, 64, 128 or 256 tokens", 0);
    if (c->head_dim != 64 && c->head_dim != 128) return afx_fail(AFX_E_ARG, "heads have 64 or 128 elements", 0);
    if (c->kv_heads == 0 || c->kv_heads > 1024) return afx_fail(AFX_E_ARG, "1 to 1024 key/value heads", 0);
    if (c->n_pages == 0 || static_cast<uint64_t>(c->n_pages) * c->page_tokens > INT32_MAX)
        return afx_fail(AFX_E_ARG, "a pool holds 1 page or more and fewer than 2^31 tokens", 0);
    if (c->page_stride % 8 || c->token_stride % 8 || c->head_stride % 8)
        return afx_fail(AFX_E_ARG, "cache strides must be multiples of 8 elements", 0);
    if (c->token_stride < c->head_dim || (c->kv_heads > 1 && c->head_stride < c->head_dim) ||
        (c->n_pages > 1 && c->page_stride < c->head_dim))
        return afx_fail(AFX_E_ARG, "cache strides must not be smaller than a head", 0);
    if (!device_ptr(c->k_dev, 16) || !device_ptr(c->v_dev, 16))
        return afx_fail(AFX_E_ARG, "the cache must be 16-byte aligned device memory", 0);
    return AFX_OK;
}

}  // namespace serve
}  // namespace afx

using namespace afx::serve;

extern "C" afx_status afx_kv_tables(uint32_t page_tokens, uint32_t n_pages, const int32_t* old_len_dev,
                                    const int32_t* new_len_dev, uint32_t n_requests, int32_t* table_dev,
                                    uint32_t table_cols, int32_t* free_pages_dev,
                                    const int32_t* free_count_dev, int32_t* free_count_out_dev, int32_t* starts_dev,
                                    int32_t* slots_dev, int32_t* positions_dev, uint32_t max_tokens,
                                    afx_stream_t stream, int32_t* status_dev) {
    TablesArgs a{};
    if (!page_shift(page_tokens, &a.shift)) return afx_fail(AFX_E_ARG, "pages hold 16, 32, 64, 128 or 256 tokens", 0);
    if (n_requests == 0 || n_requests > kMaxRequests) return afx_fail(AFX_E_ARG, "1 to 16384 requests", 0);
    if (n_pages == 0 || static_cast<uint64_t>(n_pages) * page_tokens > INT32_MAX)
        return afx_fail(AFX_E_ARG, "a pool holds 1 page or more and fewer than 2^31 tokens", 0);
    if (table_cols == 0 || static_cast<uint64_t>(table_cols) * page_tokens > INT32_MAX)
        return afx_fail(AFX_E_ARG, "a table row holds 1 page or more and fewer than 2^31 tokens", 0);
    if (max_tokens > INT32_MAX) return afx_fail(AFX_E_ARG, "max_tokens must be below 2^31", 0);
    if (!device_ptr(old_len_dev, 4) || !device_ptr(new_len_dev, 4) || !device_ptr(table_dev, 4) ||
        !device_ptr(free_pages_dev, 4) || !device_ptr(free_count_dev, 4) || !device_ptr(free_count_out_dev, 4) ||
        !device_ptr(starts_dev, 4) || (max_tokens && (!device_ptr(slots_dev, 4) || !device_ptr(positions_dev, 4))) ||
        (status_dev && !device_ptr(status_dev, 4)))
        return afx_fail(AFX_E_ARG, "the arrays must be device memory", 0);
    if (free_count_out_dev == free_count_dev)
        return afx_fail(AFX_E_ARG, "the free count is read and written at different places", 0);
    a.old_len = old_len_dev;
    a.new_len = new_len_dev;
    a.table = table_dev;
    a.stack = free_pages_dev;
    a.count = free_count_dev;
    a.count_out = free_count_out_dev;
    a.starts = starts_dev;
    a.slots = slots_dev;
    a.positions = positions_dev;
    a.status = status_dev;
    a.n = n_requests;
    a.cols = table_cols;
    a.n_pages = n_pages;
    a.max_tokens = max_tokens;
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    a.wide = !((reinterpret_cast<uintptr_t>(slots_dev) | reinterpret_cast<uintptr_t>(positions_dev)) & 15u);
    // a thread a request (the sums over fewer threads cost less), and enough CTAs for four tokens a thread
    uint32_t threads = (n_requests + 31) / 32 * 32;
    threads = threads < 128 ? 128 : threads > kTabThreads ? kTabThreads : threads;
    const uint32_t want = ceil_div(ceil_div(max_tokens, 4) + n_requests, threads);
    const uint32_t grid = want < 1 ? 1 : want > static_cast<uint32_t>(sms) ? sms : want;
    const size_t smem = 3 * sizeof(uint32_t) * (static_cast<size_t>(n_requests) + 1);
    AFX_SERVE_TRY(cudaFuncSetAttribute(kv_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(3 * sizeof(uint32_t) * (kMaxRequests + 1))),
                  "cudaFuncSetAttribute");
    AFX_SERVE_TRY(launch_early(kv_tables_kernel, grid, threads, smem, reinterpret_cast<cudaStream_t>(stream), a), "kv_tables_kernel launch");
    return AFX_OK;
}

extern "C" afx_status afx_kv_write(const afx_kv_cache* cache, const void* k_dev, const void* v_dev,
                                   uint64_t token_stride, uint64_t head_stride, const int32_t* slots_dev,
                                   uint32_t n_tokens, afx_stream_t stream, int32_t* status_dev) {
    WriteArgs a{};
    const afx_status st = check_cache(cache, &a.shift);
    if (st != AFX_OK) return st;
    if (n_tokens == 0) return AFX_OK;
    if (n_tokens > INT32_MAX) return afx_fail(AFX_E_ARG, "too many tokens", 0);
    if (!device_ptr(k_dev, 2) || !device_ptr(v_dev, 2) || !device_ptr(slots_dev, 4) ||
        (status_dev && !device_ptr(status_dev, 4)))
        return afx_fail(AFX_E_ARG, "keys, values and slots must be device memory", 0);
    a.src[0] = static_cast<const uint8_t*>(k_dev);
    a.src[1] = static_cast<const uint8_t*>(v_dev);
    a.dst[0] = static_cast<uint8_t*>(cache->k_dev);
    a.dst[1] = static_cast<uint8_t*>(cache->v_dev);
    a.slots = slots_dev;
    a.status = status_dev;
    a.src_token = 2 * token_stride;
    a.src_head = 2 * head_stride;
    a.dst_page = 2 * cache->page_stride;
    a.dst_token = 2 * cache->token_stride;
    a.dst_head = 2 * cache->head_stride;
    a.n_tokens = n_tokens;
    a.heads = cache->kv_heads;
    a.row_bytes = 2 * cache->head_dim;
    a.n_slots = cache->n_pages * cache->page_tokens;
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    const bool wide = !((reinterpret_cast<uintptr_t>(k_dev) | reinterpret_cast<uintptr_t>(v_dev) | a.src_token | a.src_head) & 15u);
    const uint64_t units = static_cast<uint64_t>(n_tokens) * a.heads * (a.row_bytes / (wide ? 16u : 2u));
    const uint64_t want = (units + kWriteThreads - 1) / kWriteThreads, most = static_cast<uint64_t>(sms) * 8;
    const uint32_t grid = static_cast<uint32_t>(want < most ? want : most);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    AFX_SERVE_TRY(wide ? launch_early(kv_write_kernel<uint4>, grid, kWriteThreads, 0, s, a)
                       : launch_early(kv_write_kernel<unsigned short>, grid, kWriteThreads, 0, s, a),
                  "kv_write_kernel launch");
    return AFX_OK;
}
