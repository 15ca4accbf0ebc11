// sm_103a sampling of one token a row of logits (afx_sample).
//
// With z the logits (NaN counts as masked), m their maximum, T the
// temperature: y = (z - m) * (1 / T), w = e^y.  Tokens are ordered by z,
// descending, ties by index.  top-k keeps the first k; top-p keeps those
// whose preceding mass is below p times the mass top-k kept; min-p keeps
// w >= min_p; the drawn token is the first, by index, at which the running
// sum of the kept w exceeds u times their sum.
//
// Weights are summed as integers of 2^-44 (w <= 1 and 2^19 tokens at most,
// so every sum fits 63 bits): integer sums do not depend on their order, so
// the result does not depend on how a row is spread over CTAs, warps or
// atomics.
//
// A row belongs to a cluster of CTAs; each keeps a slice of it in shared
// memory, so the logits are read from memory once however many passes the
// choice takes:
//   1. load, maximum (ties: lowest index; at temperature 0 that is all);
//   2. top-k or top-p: a histogram of counts and masses over 1024 equal
//      steps of z between m and the last token with any mass, summed over
//      the cluster; the step where the count (the mass) is reached holds
//      the last token kept, which a pass over that step's tokens finds;
//   3. the kept mass of every warp's run, their running sums over the
//      cluster, and the run in which the aim falls, walked to the token.
// Bound: the read of the logits for many rows; for few rows the chain of
// cluster barriers.
#include <cooperative_groups.h>

#include "afx_serving.cuh"

namespace cg = cooperative_groups;

namespace afx {
namespace serve {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kBins = 1024;       // one a thread
constexpr uint32_t kListMax = 1024;    // tokens whose order is worked out pair by pair
constexpr uint32_t kMaxCluster = 16;
constexpr float kRange = 30.5f;        // e^-30.5 < 2^-44: no mass below m - 30.5 T
constexpr float kMassOne = 17592186044416.0f;  // 2^44

struct SampleArgs {
    const void* logits;
    uint64_t row_stride;  // elements
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    int32_t* tokens;
    float* logprobs;
    uint32_t vocab, slice, wide;
};

struct Shared {
    uint64_t mass[kBins];          // this CTA's histogram
    uint64_t all_mass[kBins];      // the cluster's
    uint64_t list[kListMax];       // on rank 0: tokens of one step
    uint64_t list_mass[kListMax];
    uint32_t count[kBins];
    uint32_t all_count[kBins];
    uint64_t scan[kWarps];
    uint32_t scan_count[kWarps];
    uint64_t best[kMaxCluster];    // every rank's maximum
    uint64_t lo[kMaxCluster], hi[kMaxCluster];  // every rank's smallest and largest key of a step
    uint64_t total[kMaxCluster];   // every rank's kept mass
    uint64_t threshold, kept_mass; // results of a selection
    uint64_t found_mass;
    uint32_t found_bin, found_count, list_n;
};

// The order of float32 as unsigned integers.
__device__ __forceinline__ uint32_t order_key(float z) {
    const uint32_t b = __float_as_uint(z);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// A token's place in the order: larger comes first; ties by lower index.
__device__ __forceinline__ uint64_t place(float z, uint32_t index) {
    return static_cast<uint64_t>(order_key(z)) << 32 | (0xFFFFFFFFu - index);
}

struct Row {
    float top, inv_t, step;  // m, 1 / T, bins a unit of z
    // y and w of a logit; w as an integer of 2^-44
    __device__ float scaled(float z) const { return z == top ? 0.0f : (z == -INFINITY ? -INFINITY : (z - top) * inv_t); }
    __device__ float weight(float z) const { return expf(scaled(z)); }
    __device__ uint64_t mass(float w) const { return static_cast<uint64_t>(w * kMassOne); }
    // 0 for the maximum, never smaller for a smaller z
    __device__ uint32_t bin(float z) const {
        if (z == top) return 0;
        const float b = (top - z) * step;
        return b < static_cast<float>(kBins - 1) ? static_cast<uint32_t>(b) : kBins - 1;
    }
};

__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const uint64_t o = __shfl_xor_sync(0xFFFFFFFFu, v, d);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}
__device__ __forceinline__ uint64_t warp_inclusive(uint64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const __nv_bfloat16* p) { return __bfloat162float(*p); }
template <>
__device__ __forceinline__ float load_logit<__half>(const __half* p) { return __half2float(*p); }

// NaN counts as masked; -0 and +0 are one value.
__device__ __forceinline__ float clean(float z) { return z != z ? -INFINITY : z + 0.0f; }

// The cluster's histogram of the tokens with lo <= place <= hi in the bins
// that bin_of gives, in every CTA's all_count and all_mass.
template <typename BinOf>
__device__ void histogram(cg::cluster_group& cluster, Shared& sh, const float* z, uint32_t n, uint32_t base, const Row& row,
                          uint64_t lo, uint64_t hi, BinOf bin_of) {
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    sh.count[threadIdx.x] = 0;
    sh.mass[threadIdx.x] = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t p = place(z[i], base + i);
        if (p < lo || p > hi) continue;
        const uint32_t b = bin_of(z[i], p);
        atomicAdd(&sh.count[b], 1u);
        const uint64_t w = row.mass(row.weight(z[i]));
        if (w) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[b]), static_cast<unsigned long long>(w));
    }
    cluster.sync();
    // rank r sums every ranks-th bin over the cluster and hands it to all
    for (uint32_t b = rank + ranks * (threadIdx.x / ranks), peer = threadIdx.x % ranks; b < kBins && threadIdx.x / ranks < ceil_div(kBins, ranks);
         b += ranks * (kThreads / ranks)) {
        uint32_t c = 0;
        uint64_t w = 0;
        for (uint32_t r = 0; r < ranks; ++r) {
            const Shared* other = cluster.map_shared_rank(&sh, r);
            c += other->count[b];
            w += other->mass[b];
        }
        Shared* to = cluster.map_shared_rank(&sh, peer);
        to->all_count[b] = c;
        to->all_mass[b] = w;
    }
    cluster.sync();
}

// The first bin at which the running count (by_mass: mass) from `before`
// reaches `aim`; found_count / found_mass: what runs before it.
__device__ void find_bin(Shared& sh, uint64_t before_count, uint64_t before_mass, uint64_t aim, bool by_mass) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t c = sh.all_count[threadIdx.x], w = sh.all_mass[threadIdx.x];
    const uint64_t ic = warp_inclusive(c), iw = warp_inclusive(w);
    __syncthreads();
    if (lane == 31) {
        sh.scan[warp] = iw;
        sh.scan_count[warp] = static_cast<uint32_t>(ic);
    }
    __syncthreads();
    uint64_t bc = before_count, bw = before_mass;
    for (int i = 0; i < warp; ++i) {
        bc += sh.scan_count[i];
        bw += sh.scan[i];
    }
    const uint64_t from = by_mass ? bw + iw - w : bc + ic - c, to = by_mass ? bw + iw : bc + ic;
    if (from < aim && to >= aim) {
        sh.found_bin = threadIdx.x;
        sh.found_count = static_cast<uint32_t>(bc + ic - c);
        sh.found_mass = bw + iw - w;
    }
    __syncthreads();
}

// The place of the last token kept when the order's first tokens are kept
// until their count (by_mass: mass) reaches aim, and the mass kept with it.
// The level-1 histogram (Row::bin over the whole row) is in all_count and
// all_mass.  aim is at least 1 and at most the row's count (mass).
__device__ void select(cg::cluster_group& cluster, Shared& sh, const float* z, uint32_t n, uint32_t base, const Row& row,
                       uint64_t aim, bool by_mass, uint64_t* threshold, uint64_t* kept) {
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    find_bin(sh, 0, 0, aim, by_mass);
    uint32_t bin = sh.found_bin;
    uint64_t before_count = sh.found_count, before_mass = sh.found_mass;
    uint32_t in_bin = sh.all_count[bin];
    uint64_t lo = 0, hi = ~uint64_t{0};
    bool by_bin = true;  // the step's tokens are those of level-1 bin `bin`, else those with lo <= place <= hi
    while (in_bin > kListMax) {
        if (by_bin) {  // the step's first and last places
            uint64_t a = ~uint64_t{0}, b = 0;
            for (uint32_t i = threadIdx.x; i < n; i += kThreads)
                if (row.bin(z[i]) == bin) {
                    const uint64_t p = place(z[i], base + i);
                    a = p < a ? p : a;
                    b = p > b ? p : b;
                }
            a = ~warp_max(~a);
            b = warp_max(b);
            __syncthreads();
            if (threadIdx.x % 32 == 0) {
                sh.list[threadIdx.x / 32] = a;
                sh.list_mass[threadIdx.x / 32] = b;
            }
            __syncthreads();
            if (threadIdx.x < 32) {
                a = ~warp_max(~sh.list[threadIdx.x]);
                b = warp_max(sh.list_mass[threadIdx.x]);
                if (threadIdx.x < ranks) {
                    Shared* to = cluster.map_shared_rank(&sh, threadIdx.x);
                    to->lo[rank] = a;
                    to->hi[rank] = b;
                }
            }
            cluster.sync();
            for (uint32_t r = 0; r < ranks; ++r) {
                if (r == 0 || sh.lo[r] < lo) lo = sh.lo[r];
                if (r == 0 || sh.hi[r] > hi) hi = sh.hi[r];
            }
            by_bin = false;
        }
        // [lo, hi] in up to 1024 equal steps of a power of two places
        const uint64_t span = hi - lo;
        const int shift = span >> 10 ? 64 - __clzll(static_cast<long long>(span >> 10)) : 0;
        histogram(cluster, sh, z, n, base, row, lo, hi, [&](float, uint64_t p) { return static_cast<uint32_t>((hi - p) >> shift); });
        find_bin(sh, before_count, before_mass, aim, by_mass);
        bin = sh.found_bin;
        before_count = sh.found_count;
        before_mass = sh.found_mass;
        in_bin = sh.all_count[bin];
        const uint64_t top = hi - (static_cast<uint64_t>(bin) << shift);
        const uint64_t width = (uint64_t{1} << shift) - 1;
        lo = top - lo > width ? top - width : lo;
        hi = top;
        cluster.sync();  // every rank has read its histogram before the next one is written
    }
    // the step's tokens, in any order, to rank 0
    Shared* zero = cluster.map_shared_rank(&sh, 0);
    if (rank == 0 && threadIdx.x == 0) sh.list_n = 0;
    cluster.sync();
    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        const uint64_t p = place(z[i], base + i);
        if (by_bin ? row.bin(z[i]) != bin : (p < lo || p > hi)) continue;
        const uint32_t at = atomicAdd(&zero->list_n, 1u);
        if (at < kListMax) {
            zero->list[at] = p;
            zero->list_mass[at] = row.mass(row.weight(z[i]));
        }
    }
    cluster.sync();
    if (rank == 0) {
        const uint32_t m = min(sh.list_n, kListMax);
        if (threadIdx.x < m) {
            const uint64_t p = sh.list[threadIdx.x], w = sh.list_mass[threadIdx.x];
            uint64_t ahead = before_count, mass = before_mass;
            for (uint32_t j = 0; j < m; ++j)
                if (sh.list[j] > p) {
                    ++ahead;
                    mass += sh.list_mass[j];
                }
            const uint64_t from = by_mass ? mass : ahead, to = by_mass ? mass + w : ahead + 1;
            if (from < aim && to >= aim)
                for (uint32_t r = 0; r < ranks; ++r) {
                    Shared* other = cluster.map_shared_rank(&sh, r);
                    other->threshold = p;
                    other->kept_mass = mass + w;
                }
        }
    }
    cluster.sync();
    *threshold = sh.threshold;
    *kept = sh.kept_mass;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    float* z = reinterpret_cast<float*>(raw + sizeof(Shared));
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t r = blockIdx.x / ranks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t base = min(a.vocab, rank * a.slice), n = min(a.vocab - base, a.slice);
    const T* src = static_cast<const T*>(a.logits) + r * a.row_stride + base;

    uint64_t best = 0;
    if (a.wide) {
        constexpr uint32_t kPer = 16 / sizeof(T);
        for (uint32_t i = threadIdx.x * kPer; i < n; i += kThreads * kPer) {
            if (i + kPer <= n) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + i));
                const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
                for (uint32_t j = 0; j < kPer; ++j) {
                    const float x = clean(static_cast<float>(e[j]));
                    z[i + j] = x;
                    const uint64_t p = place(x, base + i + j);
                    best = p > best ? p : best;
                }
            } else {
                for (uint32_t j = i; j < n; ++j) {
                    z[j] = clean(load_logit(src + j));
                    const uint64_t p = place(z[j], base + j);
                    best = p > best ? p : best;
                }
            }
        }
    } else {
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            z[i] = clean(load_logit(src + i));
            const uint64_t p = place(z[i], base + i);
            best = p > best ? p : best;
        }
    }
    best = warp_max(best);
    if (lane == 0) sh.scan[warp] = best;
    __syncthreads();
    if (warp == 0) {
        best = warp_max(sh.scan[lane]);
        if (lane < static_cast<int>(ranks)) cluster.map_shared_rank(&sh, lane)->best[rank] = best;
    }
    cluster.sync();
    for (uint32_t i = 0; i < ranks; ++i) best = (i == 0 || sh.best[i] > best) ? sh.best[i] : best;
    Row row;
    row.top = key_value(static_cast<uint32_t>(best >> 32));
    const float temp = a.temperature ? a.temperature[r] : 1.0f;
    if (row.top == -INFINITY || !(temp > 0.0f)) {  // nothing to draw from, or the maximum itself
        if (rank == 0 && threadIdx.x == 0) {
            const bool none = row.top == -INFINITY;
            a.tokens[r] = none ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
            if (a.logprobs) a.logprobs[r] = none ? -INFINITY : 0.0f;
        }
        return;  // the whole cluster: no rank reads another's memory any more
    }
    row.inv_t = 1.0f / temp;
    row.step = static_cast<float>(kBins) / (kRange * temp);

    const int32_t k = a.top_k ? a.top_k[r] : 0;
    const float p = a.top_p ? a.top_p[r] : 1.0f;
    const float min_p = a.min_p ? a.min_p[r] : 0.0f;
    const float least = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;
    const bool by_k = k > 0 && static_cast<uint32_t>(k) < a.vocab, by_p = p < 1.0f;
    uint64_t threshold = 0;  // places from here on are kept
    if (by_k || by_p) {
        histogram(cluster, sh, z, n, base, row, 0, ~uint64_t{0}, [&](float x, uint64_t) { return row.bin(x); });
        uint64_t kept = 0;
        const uint32_t mine_c = sh.all_count[threadIdx.x];
        const uint64_t mine_w = sh.all_mass[threadIdx.x];
        if (by_k) {
            select(cluster, sh, z, n, base, row, static_cast<uint64_t>(k), false, &threshold, &kept);
        } else {
            const uint64_t w = warp_sum(sh.all_mass[threadIdx.x]);
            if (lane == 0) sh.scan[warp] = w;
            __syncthreads();
            for (int i = 0; i < kWarps; ++i) kept += sh.scan[i];
            __syncthreads();
        }
        if (by_p) {
            const double aim = ceil(static_cast<double>(p) * static_cast<double>(kept));
            const uint64_t limit = aim >= 1.0 ? static_cast<uint64_t>(aim) : 1;
            sh.all_count[threadIdx.x] = mine_c;  // a selection may have refined the histogram
            sh.all_mass[threadIdx.x] = mine_w;
            __syncthreads();
            uint64_t t2, unused;
            select(cluster, sh, z, n, base, row, limit < kept ? limit : kept, true, &t2, &unused);
            threshold = t2 > threshold ? t2 : threshold;
        }
    }

    // the kept mass of every warp's run of the slice
    const uint32_t run = ceil_div(a.slice, kWarps), i0 = min(n, warp * run), i1 = min(n, i0 + run);
    auto kept_mass = [&](uint32_t i) -> uint64_t {
        if (i >= i1) return 0;
        const float x = z[i];
        if (place(x, base + i) < threshold) return 0;
        const float w = row.weight(x);
        return w >= least ? row.mass(w) : 0;
    };
    uint64_t mine = 0;
    for (uint32_t i = i0 + lane; i < i1; i += 32) mine += kept_mass(i);
    mine = warp_sum(mine);
    __syncthreads();
    if (lane == 0) sh.scan[warp] = mine;
    __syncthreads();
    uint64_t before = 0, slice_total = 0;
    for (int i = 0; i < kWarps; ++i) {
        const uint64_t s = sh.scan[i];
        if (i < warp) before += s;
        slice_total += s;
    }
    if (threadIdx.x < ranks) cluster.map_shared_rank(&sh, threadIdx.x)->total[rank] = slice_total;
    cluster.sync();
    uint64_t total = 0;
    for (uint32_t i = 0; i < ranks; ++i) {
        if (i < rank) before += sh.total[i];
        total += sh.total[i];
    }
    const double u = static_cast<double>(a.u[r]);
    const double scaled = u > 0.0 ? u * static_cast<double>(total) : 0.0;
    const uint64_t aim = scaled < static_cast<double>(total) ? min(static_cast<uint64_t>(scaled), total - 1) : total - 1;
    if (before <= aim && aim < before + mine) {  // the aim falls into this warp's run
        for (uint32_t i = i0; i < i1; i += 32) {
            const uint64_t w = kept_mass(i + lane), inc = warp_inclusive(w);
            const bool here = before + inc - w <= aim && aim < before + inc;
            if (here) {
                a.tokens[r] = static_cast<int32_t>(base + i + lane);
                if (a.logprobs)
                    a.logprobs[r] = row.scaled(z[i + lane]) - logf(static_cast<float>(total) * (1.0f / kMassOne));
            }
            before += __shfl_sync(0xFFFFFFFFu, inc, 31);
            if (before > aim) break;
        }
    }
}

template <typename T>
afx_status launch(const SampleArgs& a, uint32_t rows, uint32_t ranks, cudaStream_t s) {
    const size_t smem = sizeof(Shared) + static_cast<size_t>(a.slice) * sizeof(float);
    // the same for every call: calls on other threads set it too
    constexpr size_t most = sizeof(Shared) + AFX_SAMPLE_MAX_VOCAB / kMaxCluster * sizeof(float);
    AFX_SERVE_TRY(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most)),
                  "cudaFuncSetAttribute");
    AFX_SERVE_TRY(cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1),
                  "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(rows * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    AFX_SERVE_TRY(cudaLaunchKernelEx(&cfg, sample_kernel<T>, a), "sample_kernel launch");
    return AFX_OK;
}

}  // namespace
}  // namespace serve
}  // namespace afx

using namespace afx::serve;

extern "C" afx_status afx_sample(const void* logits_dev, uint32_t type, uint32_t rows, uint32_t vocab, uint64_t row_stride,
                                 const float* temperature_dev, const int32_t* top_k_dev, const float* top_p_dev,
                                 const float* min_p_dev, const float* u_dev, int32_t* tokens_dev, float* logprobs_dev,
                                 afx_stream_t stream) {
    if (type != AFX_LOGITS_F32 && type != AFX_LOGITS_BF16 && type != AFX_LOGITS_FP16)
        return afx_fail(AFX_E_ARG, "unknown logits type", 0);
    if (rows == 0) return AFX_OK;
    if (vocab == 0 || vocab > AFX_SAMPLE_MAX_VOCAB) return afx_fail(AFX_E_ARG, "a row has 1 to 524288 logits", 0);
    if (rows > 1u << 24 || (rows > 1 && row_stride < vocab))
        return afx_fail(AFX_E_ARG, "at most 2^24 rows, at least a row apart", 0);
    const uint32_t size = type == AFX_LOGITS_F32 ? 4 : 2;
    if (!device_ptr(logits_dev, size) || !device_ptr(u_dev, 4) || !device_ptr(tokens_dev, 4) ||
        (temperature_dev && !device_ptr(temperature_dev, 4)) || (top_k_dev && !device_ptr(top_k_dev, 4)) ||
        (top_p_dev && !device_ptr(top_p_dev, 4)) || (min_p_dev && !device_ptr(min_p_dev, 4)) ||
        (logprobs_dev && !device_ptr(logprobs_dev, 4)))
        return afx_fail(AFX_E_ARG, "the arrays must be device memory", 0);
    SampleArgs a{};
    a.logits = logits_dev;
    a.row_stride = row_stride;
    a.u = u_dev;
    a.temperature = temperature_dev;
    a.top_k = top_k_dev;
    a.top_p = top_p_dev;
    a.min_p = min_p_dev;
    a.tokens = tokens_dev;
    a.logprobs = logprobs_dev;
    a.vocab = vocab;
    const uint32_t ranks = vocab > 65536 ? 16 : vocab > 8192 ? 8 : 1;
    a.slice = ceil_div(ceil_div(vocab, ranks), 128) * 128;
    a.wide = !((reinterpret_cast<uintptr_t>(logits_dev) | (rows > 1 ? row_stride * size : 0)) & 15u);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (type == AFX_LOGITS_F32) return launch<float>(a, rows, ranks, s);
    if (type == AFX_LOGITS_BF16) return launch<__nv_bfloat16>(a, rows, ranks, s);
    return launch<__half>(a, rows, ranks, s);
}
