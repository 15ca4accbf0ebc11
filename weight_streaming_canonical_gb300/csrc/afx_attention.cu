// sm_103a attention over paged keys and values for a batch that shares a
// long prefix (afx_attention_workspace, afx_attention_plan, afx_attention).
//
// Row (t, h) of the queries sees the prefix, common to the batch, and its
// own request's cached tokens up to its position.  With s = scale * q.k,
//     out = sum_j softmax(s)_j v_j,   lse = log sum_j e^(s_j).
// Two key sets A, B with running maxima m, sums l = sum e^(s - m) and
// weighted values o join as m = max(m_A, m_B), l = l_A e^(m_A - m) + l_B
// e^(m_B - m), and o likewise.  So the prefix is one problem for the whole
// batch: all tokens' rows of a key/value head (the "packed" rows, token by
// token, the G = q_heads / kv_heads heads of a token next to one another)
// against one copy of its keys, read once a row tile instead of once a
// request; each request's own tokens are a second, small problem; and long
// key ranges are cut into pieces that run side by side.  All of it is a
// list of items (a tile of packed rows x a range of keys) that one plan
// kernel writes a step (the lengths are on the GPU, and every layer of the
// step uses the same list), one attention kernel works off and one join
// kernel puts together in a fixed order.
#include "afx_serving.cuh"

namespace afx {
namespace serve {

afx_status check_cache(const afx_kv_cache* c, uint32_t* shift);  // afx_kv.cu

namespace {

constexpr uint32_t kPlanThreads = 1024;
constexpr uint32_t kMaxRequests = AFX_KV_MAX_REQUESTS;
constexpr uint32_t kRows = 16;         // packed rows of an item
constexpr uint32_t kKeyAlign = 64;     // item key ranges start at multiples of this
constexpr uint32_t kMinKeys = 256;     // keys of an item, at least, where a range is cut
constexpr uint32_t kTargetUnits = 1216;  // items x heads that the cuts aim at

// The key names what the plan was made for: a workspace that holds no plan,
// or that of another description, is refused instead of read.
struct PlanHead {
    uint32_t n_items, n_groups, n_tokens, n_prefix_groups;
    uint64_t key;
};

// A tile of packed rows of one source: its pieces' results start at
// part_row, piece s at part_row + s * rows.
struct Group {
    uint32_t part_row, n_pieces, rows, pad;
};

struct Item {
    int32_t request;        // -1: the prefix
    uint32_t row0, rows;    // packed rows of the source
    uint32_t key0, key1;    // keys of the source
    uint32_t part_row;      // where the results of its rows go
    uint32_t token0;        // first token of the source
    int32_t seen;           // token i of the source sees keys below seen + i + 1 (prefix: all)
};

struct Layout {
    uint64_t token_request, request_group, groups, items, part_ml, part_o, total;
    uint32_t max_groups, max_items, max_rows;
};

struct AttnArgs {
    const void *k, *v;
    uint64_t page_stride, token_stride, head_stride;  // elements
    const int32_t *table, *prefix_table, *starts, *lens;
    const void* q;
    void* out;
    float* lse;
    uint64_t q_token, q_head, out_token, out_head;  // elements
    uint8_t* ws;
    int32_t* status;
    Layout L;
    uint32_t table_cols, n_requests, n_tokens, prefix_len, group, kv_heads, shift, n_pages, q_wide;
    float scale_log2;
    uint64_t plan_key;
};

__host__ __device__ inline uint64_t up(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }

// Keys that the last token of packed rows [row0, row0 + rows) sees.
__device__ __forceinline__ uint32_t visible(int32_t seen, uint32_t last_row, uint32_t group) {
    const int64_t v = static_cast<int64_t>(seen) + last_row / group + 1;
    return v > 0 ? static_cast<uint32_t>(v) : 0u;
}

// ---- the plan ----------------------------------------------------------------------

__device__ uint64_t block_sum_exclusive(uint64_t v, uint64_t* total, uint64_t* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t o = __shfl_up_sync(0xFFFFFFFFu, inc, d);
        if (lane >= d) inc += o;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    uint64_t before = 0, all = 0;
    for (uint32_t w = 0; w < kPlanThreads / 32; ++w) {
        const uint64_t s = scratch[w];
        if (static_cast<int>(w) < warp) before += s;
        all += s;
    }
    *total = all;
    return before + inc - v;
}

// One CTA.  A request's rows are cut into groups of kRows; every group's
// keys are cut into pieces of `piece` keys, chosen so that all pieces x heads come
// to about kTargetUnits (enough to fill the GPU, and a bound on the
// workspace), but not below kMinKeys.
__global__ void __launch_bounds__(kPlanThreads) attention_plan_kernel(const AttnArgs a) {
    __shared__ uint64_t scratch[kPlanThreads / 32];
    PlanHead* head = reinterpret_cast<PlanHead*>(a.ws);
    int32_t* token_request = reinterpret_cast<int32_t*>(a.ws + a.L.token_request);
    uint32_t* request_group = reinterpret_cast<uint32_t*>(a.ws + a.L.request_group);
    Group* groups = reinterpret_cast<Group*>(a.ws + a.L.groups);
    Item* items = reinterpret_cast<Item*>(a.ws + a.L.items);
    const uint32_t R = a.n_requests, G = a.group;
    const uint32_t per = ceil_div(R, kPlanThreads);
    const uint32_t r0 = min(R, threadIdx.x * per), r1 = min(R, r0 + per);
    const uint64_t max_len = static_cast<uint64_t>(a.table_cols) << a.shift;

    // the lengths have to make sense before anything is addressed by them
    bool bad = false;
    uint64_t keys = 0;
    if (threadIdx.x == 0 && a.starts[0] != 0) bad = true;
    for (uint32_t r = r0; r < r1; ++r) {
        const int32_t s = a.starts[r], e = a.starts[r + 1], len = a.lens[r];
        if (s < 0 || e < s || static_cast<uint32_t>(e) > a.n_tokens || len < 0 || static_cast<uint64_t>(len) > max_len) {
            bad = true;
            continue;
        }
        const uint32_t rows = static_cast<uint32_t>(e - s) * G;
        for (uint32_t row = 0; row < rows; row += kRows)
            keys += visible(len - (e - s), min(rows, row + kRows) - 1, G);
    }
    const bool refused = __syncthreads_or(bad) != 0;
    if (refused) {
        if (threadIdx.x == 0) {
            raise(a.status, AFX_DEV_BAD_LENGTH);
            *head = PlanHead{0, 0, 0, 0, a.plan_key};
        }
        return;
    }
    const uint32_t n_tokens = a.starts[R];
    const uint32_t prefix_rows = a.prefix_len ? n_tokens * G : 0;
    const uint32_t prefix_groups = ceil_div(prefix_rows, kRows);
    uint64_t total_keys;
    block_sum_exclusive(keys, &total_keys, scratch);
    total_keys += static_cast<uint64_t>(prefix_groups) * a.prefix_len;
    const uint64_t units = kTargetUnits / a.kv_heads ? kTargetUnits / a.kv_heads : 1;
    const uint64_t want = up((total_keys + units - 1) / units, kKeyAlign);
    const uint32_t piece = static_cast<uint32_t>(want < kMinKeys ? kMinKeys : want < (1u << 31) ? want : 1u << 31);

    // the prefix: every group has the same pieces
    const uint32_t prefix_pieces = ceil_div(a.prefix_len, piece);
    for (uint32_t g = threadIdx.x; g < prefix_groups; g += kPlanThreads) {
        const uint32_t row0 = g * kRows, rows = min(kRows, prefix_rows - row0);
        groups[g] = Group{row0 * prefix_pieces, prefix_pieces, rows, 0};
    }
    for (uint32_t i = threadIdx.x; i < prefix_groups * prefix_pieces; i += kPlanThreads) {
        // piece by piece, so that the groups that read the same keys run together
        const uint32_t s = i / prefix_groups, g = i % prefix_groups;
        const uint32_t row0 = g * kRows, rows = min(kRows, prefix_rows - row0);
        items[i] = Item{-1, row0, rows, s * piece, min(a.prefix_len, (s + 1) * piece), row0 * prefix_pieces + s * rows, 0, 0};
    }

    // the requests' own tokens
    uint64_t n_groups = 0, n_items = 0, n_rows = 0;
    for (uint32_t r = r0; r < r1; ++r) {
        const uint32_t s = a.starts[r], e = a.starts[r + 1];
        const int32_t seen = a.lens[r] - static_cast<int32_t>(e - s);
        const uint32_t rows = (e - s) * G;
        for (uint32_t row = 0; row < rows; row += kRows) {
            const uint32_t n = min(kRows, rows - row), pieces = ceil_div(visible(seen, row + n - 1, G), piece);
            ++n_groups;
            n_items += pieces;
            n_rows += static_cast<uint64_t>(pieces) * n;
        }
    }
    uint64_t all_groups, all_items, all_rows;
    uint32_t g = static_cast<uint32_t>(block_sum_exclusive(n_groups, &all_groups, scratch)) + prefix_groups;
    uint32_t it = static_cast<uint32_t>(block_sum_exclusive(n_items, &all_items, scratch)) + prefix_groups * prefix_pieces;
    uint32_t pr = static_cast<uint32_t>(block_sum_exclusive(n_rows, &all_rows, scratch)) + prefix_rows * prefix_pieces;
    for (uint32_t r = r0; r < r1; ++r) {
        const uint32_t s = a.starts[r], e = a.starts[r + 1];
        const int32_t seen = a.lens[r] - static_cast<int32_t>(e - s);
        const uint32_t rows = (e - s) * G;
        request_group[r] = g;
        for (uint32_t row = 0; row < rows; row += kRows) {
            const uint32_t n = min(kRows, rows - row), end = visible(seen, row + n - 1, G), pieces = ceil_div(end, piece);
            groups[g++] = Group{pr, pieces, n, 0};
            for (uint32_t p = 0; p < pieces; ++p, pr += n)
                items[it++] = Item{static_cast<int32_t>(r), row, n, p * piece, min(end, (p + 1) * piece), pr, s, seen};
        }
        for (uint32_t t = s; t < e; ++t) token_request[t] = static_cast<int32_t>(r);
    }
    if (threadIdx.x == 0)
        *head = PlanHead{prefix_groups * prefix_pieces + static_cast<uint32_t>(all_items),
                         prefix_groups + static_cast<uint32_t>(all_groups), n_tokens, prefix_groups, a.plan_key};
}

// ---- 16 packed rows x a range of keys ------------------------------------------------

template <typename T>
struct Mma;
template <>
struct Mma<__nv_bfloat16> {
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};
template <>
struct Mma<__half> {
    static __device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    }
    static __device__ __forceinline__ __half from(float x) { return __float2half_rn(x); }
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
    const uint32_t n = real ? 16u : 0u;  // 0: the 16 bytes are zeros, src is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

constexpr int kWarps = 4;
constexpr int kBlockKeys = 16;  // keys of one step of a warp; divides every page size
constexpr int kStages = 3;
// A row's reference maximum lags behind by up to this many powers of two:
// exact all the same (numerator and denominator use the same reference), it
// saves scaling the sums on every small rise; p stays below 2^8, which both
// 16-bit types hold.
constexpr float kLag = 8.0f;

template <int D>
constexpr size_t rows16_smem() {
    return static_cast<size_t>(kWarps) * kStages * 2 * kBlockKeys * D * 2;
}

// The four warps of a CTA take every fourth block of 16 keys of the item,
// each with its own copies, maxima and sums, and meet once at the end.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) attention_rows16_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kChunks = D / 8;                     // 16-byte chunks of a key
    constexpr uint32_t kTile = kBlockKeys * D * 2;     // bytes of a block's keys
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const PlanHead head = *reinterpret_cast<const PlanHead*>(a.ws);
    if (head.key != a.plan_key) {
        if (threadIdx.x == 0) raise(a.status, AFX_DEV_BAD_PLAN);
        return;
    }
    const Item* items = reinterpret_cast<const Item*>(a.ws + a.L.items);
    float* part_o = reinterpret_cast<float*>(a.ws + a.L.part_o);
    float2* part_ml = reinterpret_cast<float2*>(a.ws + a.L.part_ml);
    const T* q = static_cast<const T*>(a.q);
    const T* kp = static_cast<const T*>(a.k);
    const T* vp = static_cast<const T*>(a.v);
    uint8_t* mine = smem + warp * (kStages * 2 * kTile);
    const uint32_t mine_addr = smem_addr(mine);
    const uint32_t page_mask = (1u << a.shift) - 1;

    for (uint32_t unit = blockIdx.x; unit < head.n_items * a.kv_heads; unit += gridDim.x) {
        const Item it = items[unit / a.kv_heads];
        const uint32_t h = unit % a.kv_heads;
        const int32_t* pages = it.request < 0 ? a.prefix_table : a.table + static_cast<uint64_t>(it.request) * a.table_cols;

        // the queries as A fragments: rows lane / 4 and lane / 4 + 8
        uint32_t qf[D / 16][4];
        uint32_t limit[2];  // keys the row sees
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t i = lane / 4 + half * 8, row = it.row0 + i;
            const bool live = i < it.rows;
            limit[half] = it.request < 0 || !live ? UINT32_MAX : visible(it.seen, row, a.group);
            const T* src = q + (it.token0 + row / a.group) * a.q_token + (h * a.group + row % a.group) * a.q_head + (lane % 4) * 2;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t v = 0;
                    if (live) {
                        const T* s = src + ks * 16 + kk * 8;
                        if (a.q_wide)
                            v = *reinterpret_cast<const uint32_t*>(s);
                        else
                            v = *reinterpret_cast<const uint16_t*>(s) |
                                static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(s + 1)) << 16;
                    }
                    qf[ks][kk * 2 + half] = v;
                }
        }
        const uint32_t min_limit = it.request < 0 ? UINT32_MAX : visible(it.seen, it.row0, a.group);

        const uint32_t n_blocks = ceil_div(it.key1 - it.key0, kBlockKeys);
        const uint32_t n_mine = n_blocks > static_cast<uint32_t>(warp) ? ceil_div(n_blocks - warp, kWarps) : 0;
        int32_t page_of = 0;  // lane l: the page of this warp's block base + l
        auto issue = [&](uint32_t i) {
            if (i < n_mine) {
                if (i % 32 == 0) {  // 32 blocks' pages at a time
                    const uint32_t key = it.key0 + (warp + kWarps * (i + lane)) * kBlockKeys;
                    page_of = i + lane < n_mine ? pages[key >> a.shift] : 0;
                    if (page_of < 0 || static_cast<uint32_t>(page_of) >= a.n_pages) {
                        raise(a.status, AFX_DEV_BAD_PAGE);
                        page_of = 0;
                    }
                }
                const uint32_t key = it.key0 + (warp + kWarps * i) * kBlockKeys;
                const uint64_t page = static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, page_of, i % 32));
                const uint64_t base = page * a.page_stride + h * a.head_stride;
                const uint32_t buf = mine_addr + (i % kStages) * 2 * kTile;
#pragma unroll
                for (int c = 0; c < kBlockKeys * kChunks / 32; ++c) {
                    const uint32_t idx = c * 32 + lane, row = idx / kChunks, chunk = idx % kChunks;
                    const bool real = key + row < it.key1;  // past the range: zeros, whatever the page holds there
                    const uint64_t off = base + ((key + row) & page_mask) * a.token_stride + chunk * 8;
                    const uint32_t dst = buf + row * (D * 2) + ((chunk ^ (row & 7)) * 16);
                    copy16(dst, kp + off, real);
                    copy16(dst + kTile, vp + off, real);
                }
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        };

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][j] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) issue(s);
        for (uint32_t i = 0; i < n_mine; ++i) {
            issue(i + kStages - 1);
            asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const uint32_t buf = mine_addr + (i % kStages) * 2 * kTile;
            const uint32_t key = it.key0 + (warp + kWarps * i) * kBlockKeys;
            float s[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b[4];
                const uint32_t row = (lane / 16) * 8 + lane % 8, chunk = ks * 2 + ((lane / 8) & 1);
                ldmatrix4(b, buf + row * (D * 2) + ((chunk ^ (row & 7)) * 16));
                Mma<T>::mma(s[0], qf[ks], b[0], b[1]);
                Mma<T>::mma(s[1], qf[ks], b[2], b[3]);
            }
            const bool whole = key + kBlockKeys <= it.key1 && key + kBlockKeys <= min_limit;
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x = s[n][j] * a.scale_log2;
                    const uint32_t kk = key + n * 8 + (lane % 4) * 2 + (j & 1);
                    if (!whole && (kk >= it.key1 || kk >= limit[j >> 1])) x = -INFINITY;
                    s[n][j] = x;
                    top[j >> 1] = fmaxf(top[j >> 1], x);
                }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                top[half] = fmaxf(top[half], __shfl_xor_sync(0xFFFFFFFFu, top[half], 1));
                top[half] = fmaxf(top[half], __shfl_xor_sync(0xFFFFFFFFu, top[half], 2));
            }
            if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kLag || top[1] > m[1] + kLag)) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float next = fmaxf(m[half], top[half]);
                    const float f = next == -INFINITY ? 1.0f : exp2_approx(m[half] - next);
                    m[half] = next;
                    l[half] *= f;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][half * 2] *= f;
                        o[n][half * 2 + 1] *= f;
                    }
                }
            }
            const float ref[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[n][j] = exp2_approx(s[n][j] - ref[j >> 1]);
                    l[j >> 1] += s[n][j];
                }
            // the weights as A fragments, rounded to the cache's type for
            // the product with V (the sums above keep all their bits)
            const uint32_t p[4] = {Mma<T>::pack(s[0][0], s[0][1]), Mma<T>::pack(s[0][2], s[0][3]),
                                   Mma<T>::pack(s[1][0], s[1][1]), Mma<T>::pack(s[1][2], s[1][3])};
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                const uint32_t row = ((lane / 8) & 1) * 8 + lane % 8, chunk = n * 2 + lane / 16;
                ldmatrix4_t(b, buf + kTile + row * (D * 2) + ((chunk ^ (row & 7)) * 16));
                Mma<T>::mma(o[n * 2], p, b[0], b[1]);
                Mma<T>::mma(o[n * 2 + 1], p, b[2], b[3]);
            }
            __syncwarp();  // the buffer is read before it is filled again
        }
        asm volatile("cp.async.wait_group 0;\n" ::: "memory");
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 1);
            l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 2);
        }

        // the warps' sums meet: each scales its own to the common maximum
        __syncthreads();
        float* sm_ml = reinterpret_cast<float*>(smem);                       // [warp][16][2]
        float* sm_o = reinterpret_cast<float*>(smem) + kWarps * 16 * 2;      // [warp][16][D]
        static_assert(rows16_smem<D>() >= (kWarps * 16 * 2 + kWarps * 16 * D) * sizeof(float), "the sums fit the copies' space");
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = lane / 4 + half * 8;
            if (lane % 4 == 0) {
                sm_ml[(warp * 16 + row) * 2] = m[half];
                sm_ml[(warp * 16 + row) * 2 + 1] = l[half];
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
                *reinterpret_cast<float2*>(sm_o + (warp * 16 + row) * D + n * 8 + (lane % 4) * 2) =
                    make_float2(o[n][half * 2], o[n][half * 2 + 1]);
        }
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < it.rows * (D / 4); i += kWarps * 32) {
            const uint32_t row = i / (D / 4), c = i % (D / 4);
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_ml[(w * 16 + row) * 2]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float4 acc = make_float4(0, 0, 0, 0);
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2_approx(sm_ml[(w * 16 + row) * 2] - ref);
                const float4 x = *reinterpret_cast<const float4*>(sm_o + (w * 16 + row) * D + c * 4);
                sum += f * sm_ml[(w * 16 + row) * 2 + 1];
                acc.x += f * x.x;
                acc.y += f * x.y;
                acc.z += f * x.z;
                acc.w += f * x.w;
            }
            const uint64_t at = static_cast<uint64_t>(it.part_row + row) * a.kv_heads + h;
            *reinterpret_cast<float4*>(part_o + at * D + c * 4) = acc;
            if (c == 0) part_ml[at] = make_float2(top, sum);
        }
        __syncthreads();
    }
}

// ---- the join ------------------------------------------------------------------------

// One warp a row of the output: the pieces of its prefix group, then those
// of its request's group, in order.
template <typename T, int D>
__global__ void __launch_bounds__(128) attention_join_kernel(const AttnArgs a) {
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31;
    const uint32_t q_heads = a.kv_heads * a.group;
    const uint64_t w = static_cast<uint64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const PlanHead head = *reinterpret_cast<const PlanHead*>(a.ws);
    const uint32_t t = static_cast<uint32_t>(w / q_heads), qh = static_cast<uint32_t>(w % q_heads);
    if (head.key != a.plan_key || t >= head.n_tokens) return;
    const Group* groups = reinterpret_cast<const Group*>(a.ws + a.L.groups);
    const float* part_o = reinterpret_cast<const float*>(a.ws + a.L.part_o);
    const float2* part_ml = reinterpret_cast<const float2*>(a.ws + a.L.part_ml);
    const uint32_t r = reinterpret_cast<const int32_t*>(a.ws + a.L.token_request)[t];
    const uint32_t h = qh / a.group;
    const uint32_t row_p = t * a.group + qh % a.group;
    const uint32_t row_r = (t - a.starts[r]) * a.group + qh % a.group;
    Group src[2] = {Group{0, 0, 0, 0}, groups[reinterpret_cast<const uint32_t*>(a.ws + a.L.request_group)[r] + row_r / kRows]};
    const uint32_t in[2] = {row_p % kRows, row_r % kRows};
    if (head.n_prefix_groups) src[0] = groups[row_p / kRows];

    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        for (uint32_t p = lane; p < src[k].n_pieces; p += 32)
            top = fmaxf(top, part_ml[static_cast<uint64_t>(src[k].part_row + p * src[k].rows + in[k]) * a.kv_heads + h].x);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const float ref = top == -INFINITY ? 0.0f : top;
    float acc[kPer] = {}, sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll 4
        for (uint32_t p = 0; p < src[k].n_pieces; ++p) {
            const uint64_t at = static_cast<uint64_t>(src[k].part_row + p * src[k].rows + in[k]) * a.kv_heads + h;
            const float2 ml = part_ml[at];
            const float f = exp2_approx(ml.x - ref);
            sum += f * ml.y;
#pragma unroll
            for (int j = 0; j < kPer; ++j) acc[j] += f * part_o[at * D + lane * kPer + j];
        }
    // a row that sees no key: zeros, and the logarithm of an empty sum
    const float inv = sum > 0.0f ? 1.0f / sum : (top == -INFINITY ? 0.0f : 1.0f / sum);
    T* out = static_cast<T*>(a.out) + t * a.out_token + qh * a.out_head + lane * kPer;
#pragma unroll
    for (int j = 0; j < kPer; ++j) out[j] = Mma<T>::from(acc[j] * inv);
    if (a.lse && lane == 0)
        a.lse[static_cast<uint64_t>(t) * q_heads + qh] =
            top == -INFINITY ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
}

// ---- host side -----------------------------------------------------------------------

// Checks the description and lays the workspace out from it.
afx_status prepare(const afx_attention_args* d, AttnArgs* a) {
    if (!d) return afx_fail(AFX_E_ARG, "null attention description", 0);
    uint32_t shift = 0;
    const afx_status st = check_cache(&d->cache, &shift);
    if (st != AFX_OK) return st;
    const afx_kv_cache& c = d->cache;
    if (d->q_heads == 0 || d->q_heads % c.kv_heads || d->q_heads / c.kv_heads > 1024)
        return afx_fail(AFX_E_ARG, "q_heads must be a multiple of the cache's heads, at most 1024 times", 0);
    if (d->n_requests == 0 || d->n_requests > kMaxRequests) return afx_fail(AFX_E_ARG, "1 to 16384 requests", 0);
    if (d->n_tokens == 0 || static_cast<uint64_t>(d->n_tokens) * d->q_heads > INT32_MAX)
        return afx_fail(AFX_E_ARG, "n_tokens * q_heads must be from 1 to 2^31 - 1", 0);
    if (d->table_cols == 0 || static_cast<uint64_t>(d->table_cols) * c.page_tokens > INT32_MAX)
        return afx_fail(AFX_E_ARG, "a table row holds 1 page or more and fewer than 2^31 tokens", 0);
    if (d->prefix_len > INT32_MAX) return afx_fail(AFX_E_ARG, "prefix_len must be below 2^31", 0);
    if (!(d->scale > -INFINITY && d->scale < INFINITY)) return afx_fail(AFX_E_ARG, "scale must be finite", 0);
    if (!device_ptr(d->starts_dev, 4) || !device_ptr(d->lens_dev, 4) || !device_ptr(d->table_dev, 4) ||
        (d->prefix_len && !device_ptr(d->prefix_table_dev, 4)))
        return afx_fail(AFX_E_ARG, "starts, lens and tables must be device memory", 0);
    a->k = c.k_dev;
    a->v = c.v_dev;
    a->page_stride = c.page_stride;
    a->token_stride = c.token_stride;
    a->head_stride = c.head_stride;
    a->table = d->table_dev;
    a->prefix_table = d->prefix_table_dev;
    a->starts = d->starts_dev;
    a->lens = d->lens_dev;
    a->table_cols = d->table_cols;
    a->n_requests = d->n_requests;
    a->n_tokens = d->n_tokens;
    a->prefix_len = d->prefix_len;
    a->kv_heads = c.kv_heads;
    a->group = d->q_heads / c.kv_heads;
    a->shift = shift;
    a->n_pages = c.n_pages;
    a->scale_log2 = static_cast<float>(static_cast<double>(d->scale) * 1.4426950408889634074);
    // every group has one piece, and the cuts add at most kTargetUnits / kv_heads
    const uint64_t rows = static_cast<uint64_t>(d->n_tokens) * a->group;
    const uint64_t extra = kTargetUnits / c.kv_heads + 1;
    const uint64_t groups = 2 * ceil_div(static_cast<uint32_t>(rows), kRows) + d->n_requests + 1;
    Layout& L = a->L;
    L.max_groups = static_cast<uint32_t>(groups);
    L.max_items = static_cast<uint32_t>(groups + extra);
    L.max_rows = static_cast<uint32_t>(2 * rows + extra * kRows);
    uint64_t off = up(sizeof(PlanHead), 256);
    auto take = [&](uint64_t bytes) {
        const uint64_t at = off;
        off = up(off + bytes, 256);
        return at;
    };
    L.token_request = take(4ull * d->n_tokens);
    L.request_group = take(4ull * d->n_requests);
    L.groups = take(sizeof(Group) * groups);
    L.items = take(sizeof(Item) * static_cast<uint64_t>(L.max_items));
    L.part_ml = take(8ull * L.max_rows * c.kv_heads);
    L.part_o = take(4ull * L.max_rows * c.kv_heads * c.head_dim);
    L.total = off;
    uint64_t key = 0x61667850u;
    for (uint64_t v : {L.total, static_cast<uint64_t>(d->n_tokens), static_cast<uint64_t>(d->n_requests),
                       static_cast<uint64_t>(d->prefix_len), static_cast<uint64_t>(d->table_cols),
                       static_cast<uint64_t>(a->group), static_cast<uint64_t>(c.kv_heads), static_cast<uint64_t>(shift)})
        key = (key ^ v) * 0x9E3779B97F4A7C15ull + 1;
    a->plan_key = key;
    return AFX_OK;
}

afx_status bind_workspace(AttnArgs* a, void* ws, uint64_t bytes, int32_t* status) {
    if (bytes < a->L.total) return afx_fail(AFX_E_NOSPACE, "the attention workspace is smaller than afx_attention_workspace", 0);
    if (!device_ptr(ws, 256)) return afx_fail(AFX_E_ARG, "the workspace must be 256-byte aligned device memory", 0);
    if (status && !device_ptr(status, 4)) return afx_fail(AFX_E_ARG, "the status word must be device memory", 0);
    a->ws = static_cast<uint8_t*>(ws);
    a->status = status;
    return AFX_OK;
}

template <typename T, int D>
afx_status launch(const AttnArgs& a, cudaStream_t s) {
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    const size_t smem = rows16_smem<D>();
    AFX_SERVE_TRY(cudaFuncSetAttribute(attention_rows16_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem)),
                  "cudaFuncSetAttribute");
    attention_rows16_kernel<T, D><<<sms * 2, kWarps * 32, smem, s>>>(a);
    AFX_SERVE_TRY(cudaGetLastError(), "attention_rows16_kernel launch");
    const uint64_t warps = static_cast<uint64_t>(a.n_tokens) * a.kv_heads * a.group;
    attention_join_kernel<T, D><<<static_cast<uint32_t>((warps + 3) / 4), 128, 0, s>>>(a);
    AFX_SERVE_TRY(cudaGetLastError(), "attention_join_kernel launch");
    return AFX_OK;
}

}  // namespace
}  // namespace serve
}  // namespace afx

using namespace afx::serve;

extern "C" afx_status afx_attention_workspace(const afx_attention_args* args, uint64_t* bytes) {
    AttnArgs a{};
    if (!bytes) return afx_fail(AFX_E_ARG, "null pointer", 0);
    const afx_status st = prepare(args, &a);
    if (st != AFX_OK) return st;
    *bytes = a.L.total;
    return AFX_OK;
}

extern "C" afx_status afx_attention_plan(const afx_attention_args* args, void* workspace_dev, uint64_t workspace_bytes,
                                         afx_stream_t stream, int32_t* status_dev) {
    AttnArgs a{};
    afx_status st = prepare(args, &a);
    if (st == AFX_OK) st = bind_workspace(&a, workspace_dev, workspace_bytes, status_dev);
    if (st != AFX_OK) return st;
    attention_plan_kernel<<<1, kPlanThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(a);
    AFX_SERVE_TRY(cudaGetLastError(), "attention_plan_kernel launch");
    return AFX_OK;
}

extern "C" afx_status afx_attention(const afx_attention_args* args, const void* q_dev, uint64_t q_token_stride,
                                    uint64_t q_head_stride, void* out_dev, uint64_t out_token_stride,
                                    uint64_t out_head_stride, float* lse_dev, void* workspace_dev,
                                    uint64_t workspace_bytes, afx_stream_t stream, int32_t* status_dev) {
    AttnArgs a{};
    afx_status st = prepare(args, &a);
    if (st == AFX_OK) st = bind_workspace(&a, workspace_dev, workspace_bytes, status_dev);
    if (st != AFX_OK) return st;
    if (!device_ptr(q_dev, 2) || !device_ptr(out_dev, 2) || (lse_dev && !device_ptr(lse_dev, 4)))
        return afx_fail(AFX_E_ARG, "queries, outputs and lse must be device memory", 0);
    a.q = q_dev;
    a.out = out_dev;
    a.lse = lse_dev;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    a.q_wide = !((reinterpret_cast<uintptr_t>(q_dev) & 3u) || (q_token_stride & 1u) || (q_head_stride & 1u));
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf = args->cache.format == AFX_FMT_BF16, wide = args->cache.head_dim == 128;
    if (bf) return wide ? launch<__nv_bfloat16, 128>(a, s) : launch<__nv_bfloat16, 64>(a, s);
    return wide ? launch<__half, 128>(a, s) : launch<__half, 64>(a, s);
}
