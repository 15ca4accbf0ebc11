// sm_103a sampling of one token a row of logits (afx_sample).
//
// With z the logits (NaN counts as masked), m their maximum, T the
// temperature (where above 0, at least 3e-39): y = (z - m) * (1 / T),
// w = e^y.  Tokens are ordered by z, descending, ties by index.  top-k keeps the first k; top-p keeps those
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
// choice takes.  Pass 1 gives every thread's and the row's maximum.  Then, by
// what the row asks for:
//   - temperature 0: the lowest index of the maximum;
//   - top-k up to 1024 (with or without top-p and min-p): the k-th largest of
//     the warps' (for larger k the threads') maxima bounds the k-th largest
//     logit from below, so the tokens from that bound on, a few more than k,
//     go to one CTA, which orders them and does the rest.  Only the threads
//     whose maximum reaches the bound look at their tokens again;
//   - no top-k, top-p 1: one pass of weights (min-p is a condition on each),
//     then the run of tokens in which the aim falls, walked to the token;
//   - top-p alone: the row's mass and the weight above two cuts in y, e^-4 and
//     e^-8, say how far down the boundary lies.  Where few tokens lie above a
//     cut, they go to one CTA at once; else a histogram of masses over equal
//     steps of z says which step the boundary is in, and the tokens of that
//     step, ordered in one CTA, give the last token kept;
//   - anything else, and rows where a list above is too long (thousands of
//     ties): a histogram of counts and masses refined until a list fits.
//
// Bound: for few rows the chain of cluster barriers and passes over shared
// memory; for many rows those passes' instructions.  151,936 tokens of
// float32, the kernel alone, caches cold: one row greedy 6 us, top-k 50 13,
// without cuts 17, top-p 0.9 at temperature 1 on logits with a flat tail 45;
// 512 rows, 311 MB, 118 (2.6 TB/s), 192, 221 and 615.
#include <cooperative_groups.h>

#include <utility>

#include "afx_serving.cuh"

namespace cg = cooperative_groups;

namespace afx {
namespace serve {
namespace {

constexpr int kThreads = 512;      // two CTAs an SM, where their tokens fit
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kBinBits = 9, kBins = 1u << kBinBits;  // one a thread
static_assert(kBins == kThreads, "a bin a thread");
constexpr uint32_t kListMax = 2048;    // tokens that one CTA sorts
constexpr uint32_t kPer = kListMax / kThreads;
constexpr uint32_t kTopMax = 1024;     // top-k that goes by the threads' maxima
constexpr uint32_t kMaxCluster = 16;
constexpr uint32_t kTooMany = 1u << 26;
constexpr uint32_t kShort = 256;       // tokens that are ordered pair by pair
constexpr int kCuts = 2;               // weights above e^-4 and e^-8 tell how far down top-p reaches
constexpr uint32_t kQueue = 160;       // tokens a warp has found and not yet dealt with: 31 and 128 more
constexpr float kRange = 30.5f;        // e^-30.5 < 2^-44: no mass below m - 30.5 T
constexpr float kMassOne = 17592186044416.0f;  // 2^44
constexpr float kMostF = 3.40282347e38f;       // the largest float32
constexpr float kLeastT = 3e-39f;              // 1 / T is finite from here on (the maximum's weight is e^(0 / T))

struct SampleArgs {
    const void* logits;
    uint64_t row_stride;  // elements
    const float *u, *temperature, *top_p, *min_p;
    const int32_t* top_k;
    int32_t* tokens;
    float* logprobs;
    uint32_t vocab, slice, run, wide;  // run: tokens of a warp
    uint32_t rows, ordered;
};

struct alignas(16) Shared {
    // a list is made when the histograms of masses have been used
    union {
        struct {
            uint64_t mass[kBins];      // this CTA's histogram
            uint64_t all_mass[kBins];  // the cluster's
        };
        uint64_t list[kListMax];       // on rank 0: tokens to be sorted
    };
    uint32_t count[kBins], coarse[kBins], fine[kBins];  // this CTA's counts, and masses in 2^-22 and 2^-44
    uint32_t all_count[kBins];         // the cluster's
    uint64_t scan[kWarps];
    uint32_t scan_count[kWarps];
    float top[kMaxCluster * kWarps];   // every warp's maximum, rank by rank
    uint64_t lo[kMaxCluster], hi[kMaxCluster];  // every rank's smallest and largest place of a step
    uint64_t part[kMaxCluster];        // every rank's mass above the steps
    uint64_t total[kMaxCluster];       // every rank's kept mass
    uint64_t threshold, kept_mass;     // results of a selection
    uint64_t found_mass;
    union {  // a warp's queue is empty when the others are used
        struct {
            uint64_t bins[kBins];      // masses by steps, of the cluster or of a list
            uint64_t short_key[kShort], short_mass[kShort];
        };
        uint16_t queue[kWarps][kQueue];
    };
    uint64_t found_key, found_before;
    uint32_t found_bin, found_count, list_n, first, short_n;
    float bound;
    float above[kCuts][kMaxCluster];   // every rank's weight above the cuts
};

static_assert(2 * (sizeof(Shared) + 19008 * sizeof(float) + 1024) <= 228 * 1024, "two CTAs an SM at 152,064 tokens over eight");

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
    // y and w of a logit (top is finite, inv_t above 0); w as an integer of 2^-44
    __device__ float scaled(float z) const { return (z - top) * inv_t; }
    __device__ float weight(float z) const { return expf(scaled(z)); }
    __device__ uint64_t mass(float w) const { return static_cast<uint64_t>(w * kMassOne); }
    // 0 for the maximum, never smaller for a smaller z
    __device__ uint32_t bin(float z) const {
        if (z == top) return 0;
        const float b = (top - z) * step;
        return b < static_cast<float>(kBins - 1) ? static_cast<uint32_t>(b) : kBins - 1;
    }
};

// A sum of weights as integers of 2^-44, without a conversion a weight: adding
// 2 leaves the weight's multiple of 2^-22 in the sum's last bits; what is
// left, at most 2^-23, added to 1.5 * 2^-21 and rounded down, leaves its
// multiple of 2^-44 there.  The bits are added up as they are and the
// constants taken off at the end (up to 1023 weights).
struct MassSum {
    uint32_t hi = 0, lo = 0, n = 0;
    static constexpr float kHi = 2.0f, kLo = 1.5f / 2097152.0f;
    __device__ __forceinline__ void add(float w) {
        const float t = __fadd_rn(w, kHi);
        hi += __float_as_uint(t);
        lo += __float_as_uint(__fadd_rd(__fsub_rn(w, __fsub_rn(t, kHi)), kLo));
        ++n;
    }
    __device__ __forceinline__ uint64_t total() const {
        const uint32_t h = hi - n * __float_as_uint(kHi);
        const int32_t l = static_cast<int32_t>(lo - n * __float_as_uint(kLo));
        return (static_cast<uint64_t>(h) << 22) + static_cast<uint64_t>(static_cast<int64_t>(l));
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

__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4]) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const __half* p, float (&x)[4]) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&v.x)), hi = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    x[0] = lo.x, x[1] = lo.y, x[2] = hi.x, x[3] = hi.y;
}

// NaN counts as masked (a maximum passes over it); -0 and +0 are one value.
__device__ __forceinline__ float clean(float z) { return fmaxf(z, -INFINITY) + 0.0f; }

// Sums the CTAs' histograms into every CTA's all_count (all_mass, or bins from
// coarse and fine), which
// nobody may be reading; before it, a cluster barrier behind the counting.
// Rank r sums the bins r, r + ranks, ...: a group of `ranks` lanes a bin, each lane reads one
// rank's count and hands the sum to one rank.
__device__ void combine(cg::cluster_group& cluster, Shared& sh, bool masses, bool parts = false) {
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t peer = threadIdx.x % ranks;
    Shared* other = cluster.map_shared_rank(&sh, peer);
    for (uint32_t b = rank + threadIdx.x / ranks * ranks; b < kBins; b += kThreads) {
        uint32_t c = other->count[b];
        if (parts && c > 1023) c = kTooMany;  // its parts may have wrapped
        uint64_t w = masses ? other->mass[b] : parts ? (static_cast<uint64_t>(other->coarse[b]) << 22) + other->fine[b] : 0;
        for (uint32_t d = 1; d < ranks; d <<= 1) {
            c += __shfl_xor_sync(0xFFFFFFFFu, c, d);
            if (masses || parts) w += __shfl_xor_sync(0xFFFFFFFFu, w, d);
        }
        other->all_count[b] = c;
        if (masses) other->all_mass[b] = w;
        if (parts) other->bins[b] = w;
    }
    cluster.sync();
}

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
    combine(cluster, sh, true);
}

// The first bin at which the running count (by_mass: mass) from `before`
// reaches `aim`; found_count / found_mass: what runs before it (masses: there
// is a histogram of them).
__device__ void find_bin(Shared& sh, uint64_t before_count, uint64_t before_mass, uint64_t aim, bool by_mass, bool masses = true) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t c = sh.all_count[threadIdx.x], w = masses ? sh.all_mass[threadIdx.x] : 0;
    const uint64_t ic = warp_inclusive(c), iw = warp_inclusive(w);
    __syncthreads();
    if (lane == 31) {
        sh.scan[warp] = iw;
        sh.scan_count[warp] = static_cast<uint32_t>(ic);
    }
    if (threadIdx.x == 0) sh.found_bin = kBins - 1;  // where the aim is not reached
    __syncthreads();
    uint64_t bc = before_count, bw = before_mass;
    for (int i = 0; i < warp; ++i) {
        bc += sh.scan_count[i];
        bw += sh.scan[i];
    }
    const uint64_t from = by_mass ? bw + iw - w : bc + ic - c, to = by_mass ? bw + iw : bc + ic;
    __syncthreads();
    if (from < aim && to >= aim) {
        sh.found_bin = threadIdx.x;
        sh.found_count = static_cast<uint32_t>(bc + ic - c);
        sh.found_mass = bw + iw - w;
    }
    __syncthreads();
}

// Exclusive running sums over the CTA's threads; *total gets the sum.
__device__ uint64_t block_exclusive(Shared& sh, uint64_t v, uint64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t inc = warp_inclusive(v);
    __syncthreads();
    if (lane == 31) sh.scan[warp] = inc;
    __syncthreads();
    const uint64_t run = warp_inclusive(lane < kWarps ? sh.scan[lane] : 0);
    *total = __shfl_sync(0xFFFFFFFFu, run, 31);
    const uint64_t before = warp ? __shfl_sync(0xFFFFFFFFu, run, warp - 1) : 0;
    return before + inc - v;
}

// Up to kShort elements are ordered by counting: several threads an element
// compare it with all others.
struct Element {
    uint32_t e, part, parts;  // this thread's element, and which part of the others it looks at
    __device__ explicit Element(uint32_t n) {
        uint32_t size = 64;
        while (size < n) size <<= 1;
        parts = kThreads / size;
        e = threadIdx.x / parts;
        part = threadIdx.x % parts;
    }
    __device__ uint64_t over_parts(uint64_t v) const {
        for (uint32_t d = 1; d < parts; d <<= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        return v;
    }
};

// Which of a list's elements (kPer a thread: key and mass, no two keys alike)
// is the last needed when they are taken by falling key until their mass,
// from `before` on, reaches aim; aim is reached by all of them.  found_key gets its key and found_before the mass
// before it.  bin_of: the step a key falls into, never smaller for a smaller key.
template <typename BinOf>
__device__ void reach(Shared& sh, const uint64_t (&key)[kPer], const uint64_t (&mass)[kPer], uint64_t before, uint64_t aim, BinOf bin_of) {
    __syncthreads();
    sh.bins[threadIdx.x] = 0;
    sh.count[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        sh.short_n = sh.found_bin = 0;
        sh.found_before = before;
    }
    __syncthreads();
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j)
        if (mass[j]) {
            const uint32_t b = bin_of(key[j]);
            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[b]), static_cast<unsigned long long>(mass[j]));
            atomicAdd(&sh.count[b], 1u);
        }
    __syncthreads();
    uint64_t all;
    const uint64_t mine = sh.bins[threadIdx.x], from = before + block_exclusive(sh, mine, &all);
    if (from < aim && aim <= from + mine) {
        sh.found_bin = threadIdx.x;
        sh.found_before = from;
    }
    __syncthreads();
    const uint32_t bin = sh.found_bin;
    uint32_t n = sh.count[bin];
    uint64_t lo = 0, hi = ~uint64_t{0};  // the step's keys that are meant
    auto meant = [&](uint32_t j) { return mass[j] && key[j] >= lo && key[j] <= hi && bin_of(key[j]) == bin; };
    while (n > kShort) {  // ties, mostly (16-bit logits have hundreds): steps of the keys themselves, from the first to the last
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        uint64_t least = ~uint64_t{0}, most = 0;
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j)
            if (meant(j)) {
                least = key[j] < least ? key[j] : least;
                most = key[j] > most ? key[j] : most;
            }
        least = ~warp_max(~least);
        most = warp_max(most);
        const uint64_t start = sh.found_before;
        __syncthreads();
        if (lane == 0) {
            sh.scan[warp] = ~least;
            sh.short_key[warp] = most;
        }
        sh.bins[threadIdx.x] = 0;
        sh.count[threadIdx.x] = 0;
        __syncthreads();
        least = ~warp_max(lane < kWarps ? sh.scan[lane] : 0);
        most = warp_max(lane < kWarps ? sh.short_key[lane] : 0);
        const uint64_t span = (most - least) >> kBinBits;
        const int shift = span ? 64 - __clzll(static_cast<long long>(span)) : 0;
#pragma unroll
        for (uint32_t j = 0; j < kPer; ++j)
            if (meant(j)) {
                const uint32_t b = static_cast<uint32_t>((most - key[j]) >> shift);
                atomicAdd(reinterpret_cast<unsigned long long*>(&sh.bins[b]), static_cast<unsigned long long>(mass[j]));
                atomicAdd(&sh.count[b], 1u);
            }
        __syncthreads();
        const uint64_t in_step = sh.bins[threadIdx.x], before_step = start + block_exclusive(sh, in_step, &all);
        if (before_step < aim && aim <= before_step + in_step) {
            sh.found_bin = threadIdx.x;
            sh.found_before = before_step;
        }
        __syncthreads();
        const uint64_t step = sh.found_bin;
        n = sh.count[step];  // fewer: the first and the last key are in two steps
        hi = most - (step << shift);
        lo = hi - least < (uint64_t{1} << shift) ? least : hi - ((uint64_t{1} << shift) - 1);
    }
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j)
        if (meant(j)) {
            const uint32_t at = atomicAdd(&sh.short_n, 1u);
            sh.short_key[at] = key[j];
            sh.short_mass[at] = mass[j];
        }
    __syncthreads();
    const Element el(n);
    const uint64_t own = el.e < n ? sh.short_key[el.e] : 0;
    uint64_t ahead = 0;
#pragma unroll 4
    for (uint32_t j = el.part; j < n; j += el.parts)
        if (sh.short_key[j] > own) ahead += sh.short_mass[j];
    ahead = sh.found_before + el.over_parts(ahead);
    __syncthreads();
    if (el.e < n && el.part == 0 && ahead < aim && aim <= ahead + sh.short_mass[el.e]) {
        sh.found_key = own;
        sh.found_before = ahead;
    }
    __syncthreads();
}

__device__ __forceinline__ float place_value(uint64_t p) { return key_value(static_cast<uint32_t>(p >> 32)); }

// Steps that just cover the list's n tokens, which may lie far below the row's
// maximum and close together: of z, or of the index where all have one z (in
// 16-bit logits hundreds do, and additions to one step take their turns).
struct ListSteps {
    Row row;
    bool ties;
    __device__ uint32_t of(uint64_t p) const {
        return row.bin(ties ? -static_cast<float>(0xFFFFFFFFu - static_cast<uint32_t>(p)) : place_value(p));
    }
};
__device__ ListSteps list_steps(Shared& sh, const uint64_t (&p)[kPer], uint32_t n) {
    uint64_t least = ~uint64_t{0}, most = 0;
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j)
        if (threadIdx.x + j * kThreads < n) {
            least = p[j] < least ? p[j] : least;
            most = p[j] > most ? p[j] : most;
        }
    least = ~warp_max(~least);
    most = warp_max(most);
    __syncthreads();
    if (threadIdx.x % 32 == 0) {
        sh.scan[threadIdx.x / 32] = ~least;
        sh.short_key[threadIdx.x / 32] = most;
    }
    __syncthreads();
    least = ~warp_max(threadIdx.x % 32 < kWarps ? sh.scan[threadIdx.x % 32] : 0);
    most = warp_max(threadIdx.x % 32 < kWarps ? sh.short_key[threadIdx.x % 32] : 0);
    ListSteps s;
    s.ties = least >> 32 == most >> 32;
    s.row.top = s.ties ? -static_cast<float>(0xFFFFFFFFu - static_cast<uint32_t>(most)) : place_value(most);
    s.row.inv_t = 1.0f;
    const float span = s.row.top - (s.ties ? -static_cast<float>(0xFFFFFFFFu - static_cast<uint32_t>(least)) : place_value(least));
    s.row.step = span > 0.0f && span < INFINITY ? static_cast<float>(kBins) / span : 1.0f;
    return s;
}

// Rank 0: list[0 .. n) holds the tokens around a boundary, before_count and
// before_mass what comes before them.  Every rank's threshold gets the place
// of the last token kept, kept_mass the mass kept with it.
__device__ void last_kept(cg::cluster_group& cluster, Shared& sh, Row row, uint32_t n, uint64_t before_count, uint64_t before_mass,
                          uint64_t aim, bool by_mass) {
    uint64_t p[kPer], w[kPer], mass[kPer];
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
        const uint32_t i = threadIdx.x + j * kThreads;
        p[j] = i < n ? sh.list[i] : 0;
        w[j] = i < n ? row.mass(row.weight(place_value(p[j]))) : 0;
        mass[j] = by_mass ? w[j] : i < n ? 1 : 0;
    }
    const ListSteps steps = list_steps(sh, p, n);
    reach(sh, p, mass, by_mass ? before_mass : before_count, aim, [&](uint64_t q) { return steps.of(q); });
    const uint64_t last = sh.found_key;
    uint64_t kept = 0, total;
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) kept += p[j] >= last ? w[j] : 0;
    block_exclusive(sh, kept, &total);
    if (threadIdx.x < cluster.num_blocks()) {
        Shared* other = cluster.map_shared_rank(&sh, threadIdx.x);
        other->threshold = last;
        other->kept_mass = before_mass + total;
    }
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
                sh.scan[threadIdx.x / 32] = a;
                sh.mass[threadIdx.x / 32] = b;  // between two histograms
            }
            __syncthreads();
            if (threadIdx.x < 32) {
                a = ~warp_max(threadIdx.x < kWarps ? ~sh.scan[threadIdx.x] : 0);
                b = warp_max(threadIdx.x < kWarps ? sh.mass[threadIdx.x] : 0);
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
        // [lo, hi] in up to kBins equal steps of a power of two places
        const uint64_t span = hi - lo;
        const int shift = span >> kBinBits ? 64 - __clzll(static_cast<long long>(span >> kBinBits)) : 0;
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
        if (at < kListMax) zero->list[at] = p;
    }
    cluster.sync();
    if (rank == 0) {
        last_kept(cluster, sh, row, min(sh.list_n, kListMax), before_count, before_mass, aim, by_mass);
    }
    cluster.sync();
    *threshold = sh.threshold;
    *kept = sh.kept_mass;
}

constexpr float kCutStep = 4.0f;
__device__ __forceinline__ constexpr float cut_weight(int c) {  // e^-4, e^-8
    constexpr float w[kCuts] = {0.0183156389f, 0.000335462628f};
    return w[c];
}

struct Want {  // a row's parameters
    uint32_t k;      // 0: no top-k
    float p, least;  // p >= 1: no top-p
    double u;
};

// floor(u * total), below total.
__device__ __forceinline__ uint64_t aim_of(double u, uint64_t total) {
    const double scaled = u > 0.0 ? u * static_cast<double>(total) : 0.0;
    return scaled < static_cast<double>(total) ? min(static_cast<uint64_t>(scaled), total - 1) : total - 1;
}
// ceil(p * mass), from 1 to mass: what has to be reached.
__device__ __forceinline__ uint64_t limit_of(float p, uint64_t mass) {
    const double aim = ceil(static_cast<double>(p) * static_cast<double>(mass));
    const uint64_t limit = aim >= 1.0 ? static_cast<uint64_t>(aim) : 1;
    return limit < mass ? limit : mass;
}

__device__ __forceinline__ void write_token(const SampleArgs& a, uint32_t r, const Row& row, uint32_t token, float z, uint64_t total) {
    a.tokens[r] = static_cast<int32_t>(token);
    if (a.logprobs) a.logprobs[r] = row.scaled(z) - logf(static_cast<float>(total) * (1.0f / kMassOne));
}

// list[0 .. n) holds all tokens that can be kept: the rest of the row's
// choice, by one CTA.  row_mass: what top-p is a share of, 0 for the mass of
// what top-k keeps.
__device__ void draw_from_list(const SampleArgs& a, uint32_t r, Shared& sh, Row row, const Want& want, uint32_t n, uint64_t row_mass) {
    const uint32_t k = want.k ? want.k : n;
    if (n <= kShort) {
        const Element el(n);
        const bool real = el.e < n, one = real && el.part == 0;
        const uint64_t mine = real ? sh.list[el.e] : 0;
        const float weight = real ? row.weight(place_value(mine)) : 0.0f;
        const uint64_t w = real ? row.mass(weight) : 0;
        if (one) sh.short_mass[el.e] = w;
        __syncthreads();
        uint64_t ahead = 0, before = 0, all, total;
#pragma unroll 4
        for (uint32_t j = el.part; j < n; j += el.parts)
            if (sh.list[j] > mine) {
                ++ahead;
                before += sh.short_mass[j];
            }
        ahead = el.over_parts(ahead);
        before = el.over_parts(before);
        const bool by_k = real && ahead < k;
        block_exclusive(sh, by_k && one ? w : 0, &all);
        const uint64_t limit = want.p < 1.0f ? limit_of(want.p, row_mass ? row_mass : all) : ~uint64_t{0};
        const uint64_t kept = by_k && before < limit && weight >= want.least ? w : 0;
        if (one) sh.bins[el.e] = kept;
        block_exclusive(sh, one ? kept : 0, &total);  // a barrier as well
        before = 0;
#pragma unroll 4
        for (uint32_t j = el.part; j < n; j += el.parts)  // lower indexes have larger low halves
            if (static_cast<uint32_t>(sh.list[j]) > static_cast<uint32_t>(mine)) before += sh.bins[j];
        before = el.over_parts(before);
        const uint64_t aim = aim_of(want.u, total);
        if (one && before <= aim && aim < before + kept)
            write_token(a, r, row, 0xFFFFFFFFu - static_cast<uint32_t>(mine), place_value(mine), total);
        return;
    }
    uint64_t p[kPer] = {}, mass[kPer], threshold = 0, sum = 0, all;
    auto weight = [&](uint32_t j) { return row.weight(place_value(p[j])); };
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
        const uint32_t i = threadIdx.x + j * kThreads;
        p[j] = i < n ? sh.list[i] : 0;
        mass[j] = i < n ? 1 : 0;
    }
    const ListSteps steps = list_steps(sh, p, n);
    auto step_of = [&](uint64_t q) { return steps.of(q); };
    if (n > k) {
        reach(sh, p, mass, 0, k, step_of);
        threshold = sh.found_key;
    }
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
        mass[j] = mass[j] && p[j] >= threshold ? row.mass(weight(j)) : 0;
        sum += mass[j];
    }
    block_exclusive(sh, sum, &all);
    if (want.p < 1.0f) {
        reach(sh, p, mass, 0, limit_of(want.p, row_mass ? row_mass : all), step_of);
        threshold = sh.found_key > threshold ? sh.found_key : threshold;
    }
    sum = 0;
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
        mass[j] = p[j] >= threshold && mass[j] && weight(j) >= want.least ? mass[j] : 0;
        sum += mass[j];
        p[j] = (p[j] & 0xFFFFFFFFu) << 32 | (p[j] >> 32);  // by index, the lowest first
    }
    uint64_t total;
    block_exclusive(sh, sum, &total);
    const uint32_t share = ceil_div(a.vocab, kBins);
    reach(sh, p, mass, 0, aim_of(want.u, total) + 1, [&](uint64_t q) { return (0xFFFFFFFFu - static_cast<uint32_t>(q >> 32)) / share; });
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j)
        if (mass[j] && p[j] == sh.found_key)
            write_token(a, r, row, 0xFFFFFFFFu - static_cast<uint32_t>(p[j] >> 32), key_value(static_cast<uint32_t>(p[j])), total);
}

// A warp's run of the slice is contiguous; a lane has four tokens at a time.
__device__ __forceinline__ uint32_t run_index(uint32_t run0, uint32_t i) { return run0 + i * 128 + (threadIdx.x & 31) * 4; }

// The row a cluster takes where not all run at once: of every kThreads rows
// the ones that take longest first (top-p over the whole row: more than three
// times as long as top-k, less at low temperatures), so that no long one
// starts when the others end: 512 rows of mixed parameters 273 us, 281
// without; 64 rows of BF16 54 and 62 (a call, caches flushed).
// The same in all CTAs of a cluster.  It costs a cluster 1 us, so only where
// there is a top-p.
__device__ uint32_t row_in_order(const SampleArgs& a, Shared& sh, uint32_t place) {
    const uint32_t window = place / kThreads * kThreads, row = window + threadIdx.x;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t kind = 4;
    if (row < a.rows) {
        const int32_t k = a.top_k ? __ldg(a.top_k + row) : 0;
        const float temp = a.temperature ? __ldg(a.temperature + row) : 1.0f;
        const bool whole = k > static_cast<int32_t>(kTopMax) || (k <= 0 && a.top_p && __ldg(a.top_p + row) < 1.0f);
        kind = !(temp > 0.0f) ? 3 : !whole ? 2 : temp < 1.0f ? 1 : 0;
    }
    uint32_t same = 0;
    uint64_t counts = 0;  // 16 bits a kind
#pragma unroll
    for (uint32_t c = 0; c < 4; ++c) {
        const uint32_t who = __ballot_sync(0xFFFFFFFFu, kind == c);
        if (kind == c) same = __popc(who & ((1u << lane) - 1));
        counts |= static_cast<uint64_t>(__popc(who)) << (16 * c);
    }
    if (lane == 0) sh.scan[warp] = counts;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const uint64_t c = sh.scan[w];
        if (w < warp) before += c;
        all += c;
    }
    const uint64_t first = all * 0x0001000100010000ull;  // sums of the kinds before each
    if (kind < 4 && ((first + before) >> (16 * kind) & 0xFFFFu) + same == place - window) sh.short_n = row;
    __syncthreads();
    return sh.short_n;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    float* z = reinterpret_cast<float*>(raw + sizeof(Shared));
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t base = min(a.vocab, rank * a.slice), n = min(a.vocab - base, a.slice);
    // this warp's run: a multiple of 128 tokens long, so that a lane's four are aligned
    const uint32_t run0 = min(n, warp * a.run), run1 = min(n, run0 + a.run);
    auto started = cluster.barrier_arrive();  // a rank's memory may be written once its CTA runs
    wait_for_earlier();
    let_next_start();
    uint32_t r = blockIdx.x / ranks;
    if (a.ordered) r = row_in_order(a, sh, r);
    const T* src = static_cast<const T*>(a.logits) + r * a.row_stride + base;

    // the row's parameters, under way with the logits
    float temp = a.temperature ? __ldg(a.temperature + r) : 1.0f;
    const int32_t top_k = a.top_k ? __ldg(a.top_k + r) : 0;
    const float top_p = a.top_p ? __ldg(a.top_p + r) : 1.0f, min_p = a.min_p ? __ldg(a.min_p + r) : 0.0f, u = __ldg(a.u + r);

    // pass 1: the slice into shared memory, NaN as minus infinity and -0 as 0; the thread's maximum
    float mine = -INFINITY;
    constexpr uint32_t kBatch = 5;  // loads in flight a lane
    uint32_t done = run0;
    if (a.wide)
        for (; done + kBatch * 128 <= run1; done += kBatch * 128) {
            float x[kBatch][4];
            const T* from = src + run_index(done, 0);
            float* to = z + run_index(done, 0);
#pragma unroll
            for (uint32_t j = 0; j < kBatch; ++j) load4(from + j * 128, x[j]);
#pragma unroll
            for (uint32_t j = 0; j < kBatch; ++j) {
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) x[j][c] = clean(x[j][c]);
                mine = fmaxf(mine, fmaxf(fmaxf(x[j][0], x[j][1]), fmaxf(x[j][2], x[j][3])));
                *reinterpret_cast<float4*>(to + j * 128) = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
            }
        }
    for (; done < run1; done += kBatch * 128) {
        float x[kBatch][4];
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) {
            const uint32_t at = run_index(done, j);
            if (a.wide && at + 4 <= run1) {
                load4(src + at, x[j]);
            } else {
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) x[j][c] = at + c < run1 ? load_logit(src + at + c) : -INFINITY;
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < kBatch; ++j) {
            const uint32_t at = run_index(done, j);
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) x[j][c] = clean(x[j][c]);
            mine = fmaxf(mine, fmaxf(fmaxf(x[j][0], x[j][1]), fmaxf(x[j][2], x[j][3])));
            if (at < run1) *reinterpret_cast<float4*>(z + at) = make_float4(x[j][0], x[j][1], x[j][2], x[j][3]);
        }
    }
    {
        float top = mine;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        float* warps = reinterpret_cast<float*>(sh.scan);
        if (lane == 0) warps[warp] = top;
        sh.count[threadIdx.x] = sh.coarse[threadIdx.x] = sh.fine[threadIdx.x] = 0;
        if (threadIdx.x == 0) {
            sh.list_n = 0;
            sh.first = 0xFFFFFFFFu;
        }
        __syncthreads();
        cluster.barrier_wait(std::move(started));
        // a warp's maximum to a rank: kWarps * ranks <= kThreads
        if (threadIdx.x < kWarps * ranks)
            cluster.map_shared_rank(&sh, threadIdx.x / kWarps)->top[rank * kWarps + threadIdx.x % kWarps] = warps[threadIdx.x % kWarps];
    }
    cluster.sync();
    Row row;
    row.top = -INFINITY;
    for (uint32_t i = lane; i < kWarps * ranks; i += 32) row.top = fmaxf(row.top, sh.top[i]);
#pragma unroll
    for (int d = 16; d; d >>= 1) row.top = fmaxf(row.top, __shfl_xor_sync(0xFFFFFFFFu, row.top, d));
    if (row.top == -INFINITY) {  // nothing to draw from
        if (rank == 0 && threadIdx.x == 0) {
            a.tokens[r] = -1;
            if (a.logprobs) a.logprobs[r] = -INFINITY;
        }
        return;  // the whole cluster: no rank reads another's memory any more
    }
    Shared* zero = cluster.map_shared_rank(&sh, 0);
    auto each = [&](auto&& f) {  // this thread's tokens
        uint32_t at = run_index(run0, 0), i = run0;
        for (; i + 128 <= run1; i += 128, at += 128) {
            const float4 v = *reinterpret_cast<const float4*>(z + at);
            f(at, v.x);
            f(at + 1, v.y);
            f(at + 2, v.z);
            f(at + 3, v.w);
        }
        for (uint32_t c = 0; c < 4 && at + c < run1; ++c) f(at + c, z[at + c]);
    };
    // f for the warp's tokens that pick takes, all at least low: they are collected first, so that the lanes work
    // together where only a few tokens are meant
    auto few = [&](float low, auto&& pick, auto&& f) {
        if (!__any_sync(0xFFFFFFFFu, mine >= low)) return;
        uint16_t* q = sh.queue[warp];
        uint32_t n_q = 0;
        for (uint32_t i = run0; i < run1; i += 128) {
            const uint32_t at = i + lane * 4;
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (at < run1) v = *reinterpret_cast<const float4*>(z + at);
            const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) {
                const bool take = at + c < run1 && pick(x[c]);
                const uint32_t taken = __ballot_sync(0xFFFFFFFFu, take);
                if (take) q[n_q + __popc(taken & ((1u << lane) - 1))] = static_cast<uint16_t>(at + c);
                n_q += __popc(taken);
            }
            __syncwarp();
            while (n_q >= 32) {
                n_q -= 32;
                const uint32_t j = q[n_q + lane];
                f(j, z[j]);
                __syncwarp();
            }
        }
        if (lane < static_cast<int>(n_q)) f(q[lane], z[q[lane]]);
        __syncwarp();
    };
    if (!(temp > 0.0f)) {  // the maximum itself
        if (mine == row.top)
            each([&](uint32_t i, float x) {
                if (x == row.top) atomicMin(&zero->first, base + i);
            });
        cluster.sync();
        if (rank == 0 && threadIdx.x == 0) {
            a.tokens[r] = static_cast<int32_t>(sh.first);
            if (a.logprobs) a.logprobs[r] = 0.0f;
        }
        return;
    }
    temp = fmaxf(temp, kLeastT);
    row.inv_t = temp == INFINITY ? 1.17549435e-38f : 1.0f / temp;  // not 0: masked logits stay minus infinity
    const bool infinite = row.top == INFINITY;
    if (infinite) {  // infinite logits share everything: as zeros among masked ones
        each([&](uint32_t i, float x) { z[i] = x == INFINITY ? 0.0f : -INFINITY; });
        mine = mine == INFINITY ? 0.0f : -INFINITY;
        row.top = 0.0f;
        __syncthreads();
    }
    row.step = fminf(static_cast<float>(kBins) / (kRange * temp), kMostF);  // the steps reach past kRange below T = 5e-38
    Want want;
    want.k = top_k > 0 && static_cast<uint32_t>(top_k) < a.vocab ? top_k : 0;
    want.p = top_p < 1.0f ? top_p : 1.0f;
    want.least = min_p > 0.0f ? fminf(min_p, 1.0f) : 0.0f;
    want.u = static_cast<double>(u);
    // a bound below every logit of the first `bins` steps, and of every token with mass
    auto lower_bound = [&](uint32_t bins) {
        const float span = __fmul_ru(__fdiv_ru(static_cast<float>(bins), row.step), 1.000002f);
        return __fsub_rd(row.top, span);
    };

    // the places of this row's tokens that `pick` takes, all at least low, into rank 0's list, if they fit: one
    // reservation a CTA
    auto push = [&](float low, auto&& pick) {
        uint32_t picked = 0;
        if (mine >= low)
            each([&](uint32_t, float x) { picked += pick(x); });
        uint64_t of_cta;
        uint32_t at = static_cast<uint32_t>(block_exclusive(sh, picked, &of_cta));
        if (threadIdx.x == 0) sh.short_n = of_cta ? atomicAdd(&zero->list_n, static_cast<uint32_t>(of_cta)) : 0;
        __syncthreads();
        at += sh.short_n;
        if (picked && sh.short_n + of_cta <= kListMax)
            each([&](uint32_t i, float x) {
                if (pick(x)) zero->list[at++] = place(x, base + i);
            });
        cluster.sync();
    };
    // after a push: draws from the list and tells whether the row is done
    auto draw = [&](uint64_t row_mass) {
        const uint32_t listed = zero->list_n;
        auto read = cluster.barrier_arrive();  // every rank has read it once this barrier is through
        if (listed <= kListMax && rank) return true;
        if (listed <= kListMax) draw_from_list(a, r, sh, row, want, listed, row_mass);
        cluster.barrier_wait(std::move(read));
        return listed <= kListMax;
    };
    uint64_t threshold = 0;  // places from here on are kept
    bool general = true;
    const uint32_t n_warps = kWarps * ranks;
    if (want.k && want.k <= kTopMax) {
        // the k-th largest of maxima of k groups or more: at least k tokens are as large
        float low;
        if (want.k <= n_warps - n_warps / 4 && !infinite) {
            // of the warps' (one without tokens has minus infinity): the warp whose it is tells every rank
            const float x = sh.top[rank * kWarps + warp];
            uint32_t larger = 0, as_large = 0;
#pragma unroll
            for (uint32_t i = 0; i < kMaxCluster * kWarps; i += 32)
                if (i < n_warps) {
                    const float y = i + lane < n_warps ? sh.top[i + lane] : -INFINITY;
                    larger += __popc(__ballot_sync(0xFFFFFFFFu, y > x));
                    as_large += __popc(__ballot_sync(0xFFFFFFFFu, i + lane < n_warps && y >= x));
                }
            if (larger < want.k && as_large >= want.k && lane < static_cast<int>(ranks)) cluster.map_shared_rank(&sh, lane)->bound = x;
            cluster.sync();
            low = fmaxf(sh.bound, lower_bound(kBins));
        } else {
            // of the threads' (with fewer maxima: all that have mass)
            if (mine > -INFINITY) atomicAdd(&sh.count[row.bin(mine)], 1u);
            cluster.sync();
            combine(cluster, sh, false);
            find_bin(sh, 0, 0, want.k, false, false);
            low = lower_bound(min(sh.found_bin + 1, kBins));
        }
        push(low, [&](float x) { return x >= low; });
        if (draw(0)) return;
    } else if (!want.k) {
        general = false;
        if (want.p < 1.0f) {
            // the row's mass
            MassSum sums;
            float cut[kCuts] = {};
            each([&](uint32_t, float x) {
                const float w = row.weight(x);
                sums.add(w);
#pragma unroll
                for (int c = 0; c < kCuts; ++c)
                    if (w > cut_weight(c)) cut[c] += w;
            });
            uint64_t slice_mass, all = 0;
            float* of_warps = reinterpret_cast<float*>(sh.bins);
#pragma unroll
            for (int c = 0; c < kCuts; ++c) {
#pragma unroll
                for (int d = 16; d; d >>= 1) cut[c] += __shfl_xor_sync(0xFFFFFFFFu, cut[c], d);
                if (lane == 0) of_warps[c * kWarps + warp] = cut[c];
            }
            block_exclusive(sh, sums.total(), &slice_mass);
            if (threadIdx.x < ranks) {
                Shared* other = cluster.map_shared_rank(&sh, threadIdx.x);
                other->total[rank] = slice_mass;
                for (int c = 0; c < kCuts; ++c) {
                    float sum = 0.0f;
                    for (int w = 0; w < kWarps; ++w) sum += of_warps[c * kWarps + w];
                    other->above[c][rank] = sum;
                }
            }
            cluster.sync();
            for (uint32_t i = 0; i < ranks; ++i) all += sh.total[i];
            // a cut above which there is more than top-p needs: if few tokens are there, they are all that matters
            int far = kCuts;
            for (int c = kCuts - 1; c >= 0; --c) {
                float sum = 0.0f;
                for (uint32_t i = 0; i < ranks; ++i) sum += sh.above[c][i];
                if (sum >= want.p * 1.0002f * static_cast<float>(all) * (1.0f / kMassOne)) far = c;
            }
            if (far < kCuts) {
                const float low = __fsub_rd(row.top, __fmul_ru(1.00001f * kCutStep * static_cast<float>(far + 1), temp));
                push(low, [&](float x) { return x >= low; });
                if (draw(all)) return;
                if (rank == 0 && threadIdx.x == 0) sh.list_n = 0;  // barriers follow before the next push
            }
            const uint64_t limit = limit_of(want.p, all);
            // Otherwise steps of z between the cut before that and that one.  Past the last cut: tokens of weight
            // below (1 - p) S / V have less than (1 - p) S together, so the limit is reached before them (half of it,
            // for the rounding of this float32 line)
            const float floor_w = fminf(0.5f * (1.0f - fmaxf(want.p, 0.0f)) * (static_cast<float>(all) * (1.0f / kMassOne)) / static_cast<float>(a.vocab), 0.5f);
            const float low = far < kCuts ? __fsub_rd(row.top, __fmul_ru(1.00001f * kCutStep * static_cast<float>(far + 1), temp))
                                          : fmaxf(lower_bound(kBins), __fsub_rd(row.top, __fmul_ru(-logf(fmaxf(floor_w, 1e-30f)), temp)));
            const float high = far ? fmaxf(low, row.top - kCutStep * static_cast<float>(far) * temp) : row.top;
            const float span = high - low, step = span > 0.0f && span < INFINITY ? static_cast<float>(kBins) / span : 1.0f;
            auto step_of = [&](float x) {  // of low <= x <= high
                const float b = (high - x) * step;
                return b < static_cast<float>(kBins - 1) ? static_cast<uint32_t>(b) : kBins - 1;
            };
            // the exact mass above the steps, and of each step in two parts of 22 bits (right for up to 1023 tokens)
            MassSum over;
            few(low, [&](float x) { return x >= low; }, [&](uint32_t, float x) {
                const float w = row.weight(x);
                if (x > high) {
                    over.add(w);
                } else {
                    const uint32_t b = step_of(x);
                    const uint64_t m = row.mass(w);
                    atomicAdd(&sh.count[b], 1u);
                    atomicAdd(&sh.coarse[b], static_cast<uint32_t>(m >> 22));
                    atomicAdd(&sh.fine[b], static_cast<uint32_t>(m) & 0x3FFFFFu);
                }
            });
            block_exclusive(sh, over.total(), &slice_mass);
            if (threadIdx.x < ranks) cluster.map_shared_rank(&sh, threadIdx.x)->part[rank] = slice_mass;
            cluster.sync();
            combine(cluster, sh, false, true);
            uint64_t above = 0, unused;
            for (uint32_t i = 0; i < ranks; ++i) above += sh.part[i];
            const uint64_t inside = sh.bins[threadIdx.x], from = above + block_exclusive(sh, inside, &unused);
            if (threadIdx.x == 0) sh.found_bin = kBins;
            __syncthreads();
            if (from < limit && limit <= from + inside) {
                sh.found_bin = threadIdx.x;
                sh.found_mass = from;
            }
            __syncthreads();
            // the tokens of the step where the limit is reached
            const uint32_t bin = sh.found_bin;
            const bool right = !__syncthreads_or(threadIdx.x <= bin && sh.all_count[threadIdx.x] >= kTooMany);
            const uint32_t listed = bin < kBins && right ? sh.all_count[bin] : kListMax + 1;
            if (listed <= kListMax) {
                above = sh.found_mass;
                push(low, [&](float x) { return x >= low && x <= high && step_of(x) == bin; });
                if (rank == 0) last_kept(cluster, sh, row, listed, 0, above, limit, true);
                cluster.sync();
                threshold = sh.threshold;
            } else {
                general = true;
            }
        }
    }
    if (general) {
        cluster.sync();  // the histograms and lists above are done with
        histogram(cluster, sh, z, n, base, row, 0, ~uint64_t{0}, [&](float x, uint64_t) { return row.bin(x); });
        uint64_t kept = 0;
        const uint32_t mine_c = sh.all_count[threadIdx.x];
        const uint64_t mine_w = sh.all_mass[threadIdx.x];
        if (want.k) {
            select(cluster, sh, z, n, base, row, want.k, false, &threshold, &kept);
        } else {
            block_exclusive(sh, mine_w, &kept);
        }
        if (want.p < 1.0f) {
            __syncthreads();
            sh.all_count[threadIdx.x] = mine_c;  // a selection may have refined the histogram
            sh.all_mass[threadIdx.x] = mine_w;
            __syncthreads();
            uint64_t t2, unused;
            select(cluster, sh, z, n, base, row, limit_of(want.p, kept), true, &t2, &unused);
            threshold = t2 > threshold ? t2 : threshold;
        }
    }

    // the kept mass of every warp's run
    const float low = threshold ? place_value(threshold) : lower_bound(kBins);
    auto kept_mass = [&](uint32_t i, float x) -> uint64_t {
        if (x < low || place(x, base + i) < threshold) return 0;
        const float w = row.weight(x);
        return w >= want.least ? row.mass(w) : 0;
    };
    MassSum sums;
    if (threshold == 0) {
        each([&](uint32_t, float x) {
            const float w = row.weight(x);
            sums.add(w >= want.least ? w : 0.0f);
        });
    } else {
        few(low, [&](float x) { return x >= low; }, [&](uint32_t i, float x) {
            if (place(x, base + i) < threshold) return;
            const float w = row.weight(x);
            sums.add(w >= want.least ? w : 0.0f);
        });
    }
    uint64_t mass = warp_sum(sums.total());
    __syncthreads();
    if (lane == 0) sh.scan[warp] = mass;
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
    const uint64_t aim = aim_of(want.u, total);
    if (before <= aim && aim < before + mass) {  // the aim falls into this warp's run
        for (uint32_t i = run0; i < run1; i += 32) {
            const uint32_t at = i + lane;
            const uint64_t w = at < run1 ? kept_mass(at, z[at]) : 0, inc = warp_inclusive(w);
            if (before + inc - w <= aim && aim < before + inc) write_token(a, r, row, base + at, z[at], total);
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
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
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
    // CTAs a row: as few as hold it in 32,640 tokens each (the barriers cost
    // less), more while the GPU has two CTAs an SM to give and 4096 tokens are left for each.  Two CTAs fit an SM up
    // to some 20,200 tokens each; with many rows, vocabularies that leave a CTA more have one
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    uint32_t ranks = 1;
    while (ranks < kMaxCluster &&
           (vocab / ranks > 32768 - 128 || (vocab / ranks > 4096 && static_cast<uint64_t>(rows) * ranks * 2 <= static_cast<uint64_t>(sms) * 2)))
        ranks *= 2;
    a.rows = rows;
    a.ordered = top_p_dev && rows > 1 && static_cast<uint64_t>(rows) * ranks > static_cast<uint64_t>(sms) * 2;
    a.slice = ceil_div(ceil_div(vocab, ranks), 128) * 128;
    a.run = ceil_div(a.slice, kWarps * 128) * 128;
    a.wide = !((reinterpret_cast<uintptr_t>(logits_dev) | (rows > 1 ? row_stride * size : 0)) & 15u);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (type == AFX_LOGITS_F32) return launch<float>(a, rows, ranks, s);
    if (type == AFX_LOGITS_BF16) return launch<__nv_bfloat16>(a, rows, ranks, s);
    return launch<__half>(a, rows, ranks, s);
}
