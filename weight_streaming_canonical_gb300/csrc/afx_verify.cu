// sm_103a verification of drafted tokens (afx_verify).
//
// Row t of a request decides on a draft d that was drawn from q_t; p_t is what
// afx_sample would draw from.  The draft stands with probability
// min(1, p_t(d) / q_t(d)): where u q_t(d) < p_t(d).  At the first row whose
// draft does not stand, the token is drawn from max(p_t - q_t, 0), which leaves
// tokens distributed as p_t: a token's chance is min(p, q) + (1 - sum min(p, q))
// max(p - q, 0) / sum max(p - q, 0) = p.
//
// Three kernels, a launch each, the first two one for each type of logits.
// verify_scan_kernel reads the rows that keep all their tokens or, at temperature 0, one: a part of a row a CTA, with a running
// maximum and sum, in one pass at the memory's rate.  Rows with top-k, top-p
// or min-p go to the sampling kernel without its draw (verify_record_kernel,
// afx_sample.cu), which records what they keep as the last place kept and the
// kept weights' sum, so that a token's share is its weight by the sum.  Both
// take all rows at once, although rows behind a refused draft turn out not to
// be needed: one after the other they would take as many passes as there are
// drafts.
//
// verify_kernel has a cluster a request: a thread a draft for the tests, then
// one pass over the row to draw from, whose masses, those of p or of
// max(p - q, 0), are summed as integers of 2^-44, chunk by chunk, so that the sums
// do not depend on their order; then the chunk in which the aim falls is read
// again.  A token that p does not keep needs no q, so that behind top-k or
// top-p few of the draft's logits are read.  Sums of the scan are of float32 and good
// for a test or a logarithm (accepted tokens of 151,936: off by 1.6e-7, root mean square; 1.6e-7 too with expf and sums
// held in two float32, for which 200 requests took 108 us instead of 97); a draw from
// differences of rows that keep all first sums their masses.
//
// Bound: with looked-up drafts and no cuts reading the rows, and the row to draw from once
// more: 200 requests of up to three drafts, 492 rows of 151,936, float32, 96 us; by
// itself on cold caches the scan takes 54 (5.6 TB/s) and the draws 53.  With top-k and top-p the records: 64
// requests of up to five drafts with their logits, BF16, 261 to 292 us by the inputs; by themselves
// 177 for the sampling kernel (barriers and passes over shared memory), 57 for the
// tests and draws, 25 for the scan.  One request of four drafts: 26 us, three kernels one after the other.
#include <cooperative_groups.h>

#include <type_traits>
#include <utility>

#include "afx_sample.cuh"

namespace cg = cooperative_groups;

namespace afx {
namespace serve {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kScanThreads = 256;
constexpr uint32_t kMostParts = 16;     // of a row
constexpr uint32_t kChunk = 512;        // tokens of a warp at a time
constexpr uint32_t kGroups = kChunk / 128;
constexpr uint32_t kMostChunks = AFX_SAMPLE_MAX_VOCAB / kWarps / kChunk;  // of a warp, one CTA a row

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

struct Part {  // of a row: its maximum, sum of e^((z - m) / T), lowest index of the maximum, infinite logits
    float top, sum;
    uint32_t first, infinite;
};

struct VerifyArgs {
    Side side[2];  // the target's, the drafts'
    Part* parts;   // [2 rows][n_parts]
    const int32_t *starts, *tokens;
    const float *u, *draw_u;
    int32_t *out_tokens, *counts;
    float* logprobs;
    int32_t* status;
    uint32_t n_requests, n_tokens, vocab, slice, run;
    uint32_t n_parts, part;
    uint32_t wide[2], scan_wide[2];  // rows are aligned for four tokens' loads, for 16 bytes'
};

// ---- one pass over rows that keep all ------------------------------------------------

// 16 bytes of logits
__device__ __forceinline__ void load_wide(const float* p, float (&x)[4]) { load4(p, x); }
__device__ __forceinline__ void load_wide(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
}
__device__ __forceinline__ void load_wide(const __half* p, float (&x)[8]) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ float exp2_approx(float x) {  // two last places off at most
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void join(Part& a, const Part& b, float inv_t) {
    const float top = fmaxf(a.top, b.top);
    if (top == -INFINITY) return;
    const float fa = a.top == top ? 1.0f : exp2_approx((a.top - top) * inv_t * 1.44269504f),
                fb = b.top == top ? 1.0f : exp2_approx((b.top - top) * inv_t * 1.44269504f);
    a.first = a.top < top ? b.first : b.top < top ? a.first : min(a.first, b.first);
    a.sum = a.sum * fa + b.sum * fb;
    a.top = top;
    a.infinite += b.infinite;
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads) verify_scan_kernel(const __grid_constant__ VerifyArgs a, const uint32_t row0) {
    constexpr uint32_t kPer = 16 / sizeof(T), kRuns = sizeof(T) == 4 ? 4 : 2;  // tokens a load, loads in flight
    __shared__ Part warps[kScanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_earlier();
    let_next_start();
    uint32_t r = row0 + blockIdx.y;
    const bool second = r >= a.n_tokens;
    const Side& side = a.side[second];
    const uint32_t record = r;
    if (second) r -= a.n_tokens;
    uint32_t request = 0;  // as many end by row r
    for (uint32_t i = 0; i < a.n_requests; i += kScanThreads)
        request += __syncthreads_count(i + threadIdx.x < a.n_requests && __ldg(a.starts + 1 + i + threadIdx.x) <= static_cast<int32_t>(r));
    if (request >= a.n_requests) return;
    const float t = temperature_of(side, request);
    if (t > 0.0f && !keeps_all(side, request, a.vocab)) return;
    if (second && draft_of(a.tokens, static_cast<int32_t>(r), min(__ldg(a.starts + 1 + request), static_cast<int32_t>(a.n_tokens)), a.vocab) < 0) return;
    const float inv_t = t > 0.0f ? inverse_temperature(t) : 1.0f;
    const uint32_t at0 = blockIdx.x * a.part, at1 = min(a.vocab, at0 + a.part);
    const T* z = static_cast<const T*>(side.logits) + r * side.row_stride;
    const bool wide = a.scan_wide[second];
    Part mine{-INFINITY, 0.0f, 0xFFFFFFFFu, 0};
    for (uint32_t i0 = at0; i0 < at1; i0 += kScanThreads * kPer * kRuns) {
        float x[kRuns][kPer];
#pragma unroll
        for (uint32_t j = 0; j < kRuns; ++j) {
            const uint32_t i = i0 + (j * kScanThreads + threadIdx.x) * kPer;
            if (wide && i + kPer <= at1) {
                load_wide(z + i, x[j]);
            } else {
#pragma unroll
                for (uint32_t c = 0; c < kPer; ++c) x[j][c] = i + c < at1 ? load_logit(z + i + c) : -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (uint32_t j = 0; j < kRuns; ++j)
#pragma unroll
            for (uint32_t c = 0; c < kPer; ++c) {
                x[j][c] = clean(x[j][c]);
                top = fmaxf(top, x[j][c]);
            }
        if (top == -INFINITY) continue;
        if (!(t > 0.0f)) {  // the maximum alone
            if (top > mine.top)
#pragma unroll
                for (uint32_t j = kRuns; j-- > 0;)
#pragma unroll
                    for (uint32_t c = kPer; c-- > 0;)
                        if (x[j][c] == top) mine.first = i0 + (j * kScanThreads + threadIdx.x) * kPer + c;
            mine.top = fmaxf(mine.top, top);
            continue;
        }
        if (top > mine.top) {
            mine.sum *= mine.top == -INFINITY || top == INFINITY ? 0.0f : exp2_approx((mine.top - top) * inv_t * 1.44269504f);
            mine.top = top;
        }
        if (mine.top == INFINITY) {  // these alone count from here on
#pragma unroll
            for (uint32_t j = 0; j < kRuns; ++j)
#pragma unroll
                for (uint32_t c = 0; c < kPer; ++c) mine.infinite += x[j][c] == INFINITY;
            continue;
        }
        float sum[4] = {};
#pragma unroll
        for (uint32_t j = 0; j < kRuns; ++j)
#pragma unroll
            for (uint32_t c = 0; c < kPer; ++c) sum[c % 4] += exp2_approx((x[j][c] - mine.top) * inv_t * 1.44269504f);
        mine.sum += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        Part o;
        o.top = __shfl_xor_sync(0xFFFFFFFFu, mine.top, d);
        o.sum = __shfl_xor_sync(0xFFFFFFFFu, mine.sum, d);
        o.first = __shfl_xor_sync(0xFFFFFFFFu, mine.first, d);
        o.infinite = __shfl_xor_sync(0xFFFFFFFFu, mine.infinite, d);
        join(mine, o, inv_t);
    }
    if (lane == 0) warps[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kScanThreads / 32; ++w) join(mine, warps[w], inv_t);
        a.parts[static_cast<uint64_t>(record) * a.n_parts + blockIdx.x] = mine;
    }
}

// What row r of a side keeps, recorded or from its parts.
struct Kind {  // of a request's rows of a side
    bool recorded, greedy;
    float inv_t;
    __device__ Kind(const Side& side, uint32_t request, uint32_t vocab) {
        const float t = temperature_of(side, request);
        const bool all = keeps_all(side, request, vocab);
        greedy = !(t > 0.0f);
        recorded = !greedy & !all;
        inv_t = greedy ? 1.0f : inverse_temperature(t);
    }
};
__device__ Kept kept_of(const VerifyArgs& a, int which, const Kind& kind, uint32_t r) {
    const Side& side = a.side[which];
    if (kind.recorded) return side.kept[r];
    const Part* parts = a.parts + (static_cast<uint64_t>(which) * a.n_tokens + r) * a.n_parts;
    Part all = parts[0];
    for (uint32_t i = 1; i < a.n_parts; ++i) join(all, parts[i], kind.inv_t);
    Kept k;
    k.infinite = all.top == INFINITY;
    k.top = k.infinite ? 0.0f : all.top;
    k.inv_t = kind.inv_t;
    k.least = 0.0f;
    k.threshold = kind.greedy ? place(k.top, all.first) : 0;
    const float sum = kind.greedy ? 1.0f : k.infinite ? static_cast<float>(all.infinite) : all.sum;
    k.total = all.top == -INFINITY ? 0 : static_cast<uint64_t>(static_cast<double>(sum) * kMassOne);
    return k;
}

// ---- the tests and the draw ------------------------------------------------------------

struct Shared {
    uint64_t chunks[kWarps][kMostChunks];  // masses
    uint64_t warps[2][kWarps];
    uint64_t total[3][2][kMaxCluster];     // every rank's masses, turn by turn
    int32_t first;
    uint16_t queue[kWarps][kChunk];        // tokens of a chunk that p keeps
};

__device__ __forceinline__ float log_share(const Kept& p, float z, uint64_t total) {
    return p.scaled(z) - logf(static_cast<float>(total) * (1.0f / kMassOne));
}

// What a side keeps of the row to draw from, with its order's last place as a
// logit and an index, and its weights' sum as the inverse to multiply with,
// held as the sum of two float32: rounded nearly always as the exact quotient.
struct Shares {
    float top, inv_t, least, low, inv_hi, inv_lo;
    uint32_t last, infinite;
    __device__ void set(const Kept& k) {
        top = k.top, inv_t = k.inv_t, least = k.least, infinite = k.infinite;
        low = k.threshold ? key_value(static_cast<uint32_t>(k.threshold >> 32)) : -INFINITY;
        last = k.threshold ? 0xFFFFFFFFu - static_cast<uint32_t>(k.threshold) : 0xFFFFFFFFu;
        inv_hi = 1.0f, inv_lo = 0.0f;
    }
    __device__ void divide_by(uint64_t total) {
        if (total == 0) return;
        // total / 2^44 as two float32; a step of Newton's method from the inverse of the first
        const float hi = static_cast<float>(total), lo = static_cast<float>(static_cast<int64_t>(total - static_cast<uint64_t>(hi)));
        const float t_hi = hi * (1.0f / kMassOne), t_lo = lo * (1.0f / kMassOne);
        inv_hi = __frcp_rn(t_hi);
        inv_lo = inv_hi * (fmaf(-inv_hi, t_hi, 1.0f) - inv_hi * t_lo);
    }
    __device__ __forceinline__ float value(float z) const {
        z = clean(z);
        return infinite ? (z == INFINITY ? 0.0f : -INFINITY) : z;
    }
    __device__ __forceinline__ bool keeps(float x, uint32_t i) const { return x > low || (x == low && i <= last); }
    // x as value() gives it; e^minus infinity is 0
    __device__ __forceinline__ float weight(float x, uint32_t i) const {
        const float w = expf((x - top) * inv_t);
        return keeps(x, i) && w >= least ? w : 0.0f;
    }
    __device__ __forceinline__ float share(float w) const { return fmaf(w, inv_hi, w * inv_lo); }
};

// four logits from i on, of tokens below end
template <typename T>
__device__ __forceinline__ void load_four(const T* row, bool wide, uint32_t i, uint32_t end, float (&x)[4]) {
    if (wide && i + 4 <= end) {
        load4(row + i, x);
    } else {
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) x[c] = i + c < end ? load_logit(row + i + c) : -INFINITY;
    }
}
template <typename P, typename Q>
__global__ void __launch_bounds__(kThreads, sizeof(P) + sizeof(Q) > 4 ? 2 : 3) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t r = blockIdx.x / ranks;
    const Side &target = a.side[0], &draft = a.side[1];
    auto started = cluster.barrier_arrive();  // a rank's memory may be written once its CTA runs
    // The scan's CTAs have all waited for the work before the call when this kernel starts, so the call's arguments are
    // there; what the scan and the records leave is waited for below
    if (a.n_tokens == 0) wait_for_earlier();
    const int32_t row0 = __ldg(a.starts + r), row1 = __ldg(a.starts + r + 1);
    const Kind p_kind(target, r, a.vocab), q_kind(draft, r, a.vocab);
    // all of the call or nothing: every CTA looks at all starts
    int bad = 0;
    for (uint32_t i = threadIdx.x; i <= a.n_requests; i += kThreads) {
        const int32_t s = __ldg(a.starts + i), before = i ? __ldg(a.starts + i - 1) : 0;
        bad |= s < before || s > static_cast<int32_t>(a.n_tokens) || (i == 0 && s != 0);
    }
    bad = __syncthreads_or(bad);
    cluster.barrier_wait(std::move(started));
    if (!bad && row0 + static_cast<int32_t>(threadIdx.x) + 1 < row1) {  // the first tests' logits are on their way
        const int32_t t = row0 + static_cast<int32_t>(threadIdx.x), d = draft_of(a.tokens, t, row1, a.vocab);
        if (d >= 0) {
            asm volatile("prefetch.global.L1 [%0];\n" ::"l"(static_cast<const P*>(target.logits) + t * target.row_stride + d));
            if (draft.logits) asm volatile("prefetch.global.L1 [%0];\n" ::"l"(static_cast<const Q*>(draft.logits) + t * draft.row_stride + d));
            asm volatile("prefetch.global.L1 [%0];\n" ::"l"(a.u + t));
        }
    }
    wait_for_earlier();
    let_next_start();
    if (bad || row0 == row1) {
        if (rank == 0 && threadIdx.x == 0) {
            a.counts[r] = 0;
            if (bad && r == 0) raise(a.status, AFX_DEV_BAD_LENGTH);
        }
        return;  // the whole cluster
    }
    auto z_of = [&](int32_t t, uint32_t i) { return clean(load_logit(static_cast<const P*>(target.logits) + t * target.row_stride + i)); };
    auto q_of = [&](int32_t t, uint32_t i) { return clean(load_logit(static_cast<const Q*>(draft.logits) + t * draft.row_stride + i)); };

    // the first row whose draft does not stand, or the last row
    const int32_t last = row1 - row0 - 1;
    int32_t stood = last;
    for (int32_t i0 = 0; i0 < last; i0 += kThreads) {
        const int32_t i = i0 + static_cast<int32_t>(threadIdx.x), t = row0 + i;
        if (threadIdx.x == 0) sh.first = last;
        __syncthreads();
        if (i < last) {
            const int32_t d = draft_of(a.tokens, t, row1, a.vocab);
            bool stands = d >= 0;
            if (stands) {
                const Kept p = kept_of(a, 0, p_kind, t);
                // u q < p, as products with the sums: of 64-bit numbers there are few units
                const double w = p.weight(p.value(z_of(t, d)), d);
                const double u = __ldg(a.u + t);
                if (draft.logits) {
                    const Kept q = kept_of(a, 1, q_kind, t);
                    const double other = q.total ? q.weight(q.value(q_of(t, d)), d) : 0.0f;
                    stands = u * other * static_cast<double>(p.total) < w * static_cast<double>(q.total ? q.total : 1);
                } else {
                    stands = u * static_cast<double>(p.total) < w * kMassOne;
                }
            }
            if (!stands) atomicMin(&sh.first, i);
        }
        __syncthreads();
        stood = sh.first;
        __syncthreads();
        if (stood < last) break;
    }
    const int32_t t = row0 + stood;
    const Kept kept = kept_of(a, 0, p_kind, t);
    const bool nothing = kept.top == -INFINITY, greedy = p_kind.greedy;
    if (rank == 0) {
        for (int32_t i = threadIdx.x; i <= last; i += kThreads) {
            if (i == stood && !nothing) continue;
            const uint32_t d = i < stood ? __ldg(a.tokens + row0 + i + 1) : 0;
            a.out_tokens[row0 + i] = i < stood ? static_cast<int32_t>(d) : -1;
            if (a.logprobs) {
                float l = i == stood ? -INFINITY : 0.0f;
                if (i < stood) {
                    const Kept k = kept_of(a, 0, p_kind, row0 + i);
                    l = log_share(k, k.value(z_of(row0 + i, d)), k.total);
                }
                a.logprobs[row0 + i] = l;
            }
        }
        if (threadIdx.x == 0) {
            a.counts[r] = nothing ? stood : stood + 1;
            if (greedy && !nothing) {  // the one token that p keeps, whatever q is
                a.out_tokens[t] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(kept.threshold));
                if (a.logprobs) a.logprobs[t] = 0.0f;
            }
        }
    }
    if (nothing || greedy) return;  // the whole cluster

    // the draw: from the weights of p, those of all but the draft, or the shares of p above those of q
    const int32_t refused = draft_of(a.tokens, t, row1, a.vocab);
    Shares p, q;
    p.set(kept);
    uint64_t p_total = kept.total, q_total = 0;
    bool both = false;
    uint32_t without = 0xFFFFFFFFu;
    if (refused >= 0 && draft.logits) {
        const Kept k = kept_of(a, 1, q_kind, t);
        q.set(k);
        q_total = k.total;
        both = q_total != 0;
    } else if (refused >= 0) {
        without = refused;
    }
    const uint32_t base = min(a.vocab, rank * a.slice), n = min(a.vocab - base, a.slice);
    const uint32_t run0 = base + min(n, warp * a.run), run1 = min(base + n, run0 + a.run);
    const P* z_row = static_cast<const P*>(target.logits) + t * target.row_stride;
    const Q* q_row = static_cast<const Q*>(draft.logits) + t * draft.row_stride;
    uint64_t before = 0, mine = 0, total = 0, q_sum = 0;
    uint32_t turn = 0;
    // From the masses of each chunk of this warp's run: of its run (mine), of the runs before it and of the row
    auto join_runs = [&](uint64_t of_run, uint64_t q_of_run) {
        __syncthreads();
        if (lane == 0) sh.warps[0][warp] = of_run, sh.warps[1][warp] = q_of_run;
        __syncthreads();
        uint64_t of_slice = 0, q_of_slice = 0;
        before = 0;
        for (uint32_t i = 0; i < kWarps; ++i) {
            if (i < warp) before += sh.warps[0][i];
            of_slice += sh.warps[0][i], q_of_slice += sh.warps[1][i];
        }
        if (threadIdx.x < ranks) {
            Shared* other = cluster.map_shared_rank(&sh, threadIdx.x);
            other->total[turn][0][rank] = of_slice, other->total[turn][1][rank] = q_of_slice;
        }
        cluster.sync();
        total = q_sum = 0;
        for (uint32_t i = 0; i < ranks; ++i) {
            if (i < rank) before += sh.total[turn][0][i];
            total += sh.total[turn][0][i];
            q_sum += sh.total[turn][1][i];
        }
        mine = of_run;
        ++turn;
    };
    auto sum_of_p = [&] {
        uint64_t of_run = 0;
        uint32_t k = 0;
        RawFour<P> raw[kGroups], next[kGroups];
        auto fetch = [&](uint32_t i0, RawFour<P>(&to)[kGroups]) {
#pragma unroll
            for (uint32_t j = 0; j < kGroups; ++j) to[j].load(z_row, a.wide[0], i0 + j * 128 + lane * 4, run1, -INFINITY);
        };
        fetch(run0, raw);
        const bool plain = p.low == -INFINITY && p.least == 0.0f && !p.infinite;
#pragma unroll 1
        for (uint32_t i0 = run0; i0 < run1; i0 += kChunk, ++k) {
            fetch(i0 + kChunk, next);
            uint64_t sum = 0;
            if (plain && without - i0 >= kChunk) {
                MassSum s;
#pragma unroll
                for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c) s.add(expf((clean(raw[j].get(c)) - p.top) * p.inv_t));
                sum = warp_sum(s.total());
            } else {
                bool any = false;
#pragma unroll
                for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c) any |= p.value(raw[j].get(c)) >= p.low;
                if (__any_sync(0xFFFFFFFFu, any)) {
                    MassSum s;
#pragma unroll
                    for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                        for (uint32_t c = 0; c < 4; ++c) {
                            const uint32_t i = i0 + j * 128 + lane * 4 + c;
                            s.add(i == without ? 0.0f : p.weight(p.value(raw[j].get(c)), i));
                        }
                    sum = warp_sum(s.total());
                }
            }
            if (lane == 0) sh.chunks[warp][k] = sum;
            of_run += sum;
#pragma unroll
            for (uint32_t j = 0; j < kGroups; ++j) raw[j] = next[j];
        }
        join_runs(of_run, 0);
    };
    // sums: the weights of p and of q, apart; otherwise the shares of p above those of q
    auto sum_of_both = [&](bool sums) {
        uint64_t of_run = 0, q_of_run = 0;
        uint32_t k = 0;
        const bool whole = sums || p.low == -INFINITY;  // all tokens are meant: both rows are read
        RawFour<P> raw[kGroups], next[kGroups];
        RawFour<Q> q_raw[kGroups], q_next[kGroups];
        auto fetch = [&](uint32_t i0, RawFour<P>(&to)[kGroups], RawFour<Q>(&q_to)[kGroups]) {
#pragma unroll
            for (uint32_t j = 0; j < kGroups; ++j) to[j].load(z_row, a.wide[0], i0 + j * 128 + lane * 4, run1, -INFINITY);
            if (whole)
#pragma unroll
                for (uint32_t j = 0; j < kGroups; ++j) q_to[j].load(q_row, a.wide[1], i0 + j * 128 + lane * 4, run1, -INFINITY);
        };
        fetch(run0, raw, q_raw);
#pragma unroll 1
        for (uint32_t i0 = run0; i0 < run1; i0 += kChunk, ++k) {
            uint64_t sum = 0, q_of_chunk = 0;
            if (i0 != run0)
#pragma unroll
                for (uint32_t j = 0; j < kGroups; ++j) raw[j] = next[j], q_raw[j] = q_next[j];
            fetch(i0 + kChunk, next, q_next);
            if (whole) {
                MassSum s, q_s;
#pragma unroll
                for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c) {
                        const uint32_t i = i0 + j * 128 + lane * 4 + c;
                        const float wp = p.weight(p.value(raw[j].get(c)), i), wq = q.weight(q.value(q_raw[j].get(c)), i);
                        s.add(sums ? wp : fmaxf(p.share(wp) - q.share(wq), 0.0f));
                        q_s.add(wq);
                    }
                sum = warp_sum(s.total());
                if (sums) q_of_chunk = warp_sum(q_s.total());
            } else {  // the tokens that p keeps are few: collected first, so that the lanes work together
                uint16_t* queue = sh.queue[warp];
                uint32_t n_q = 0;
#pragma unroll
                for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c) {
                        const bool take = p.value(raw[j].get(c)) >= p.low;
                        const uint32_t taken = __ballot_sync(0xFFFFFFFFu, take);
                        if (take) queue[n_q + __popc(taken & ((1u << lane) - 1))] = static_cast<uint16_t>(j * 128 + lane * 4 + c);
                        n_q += __popc(taken);
                    }
                __syncwarp();
                MassSum s;
                for (uint32_t e = lane; e < n_q; e += 32) {
                    const uint32_t i = i0 + queue[e];
                    const float wq = q.weight(q.value(load_logit(q_row + i)), i), wp = p.weight(p.value(load_logit(z_row + i)), i);
                    s.add(fmaxf(p.share(wp) - q.share(wq), 0.0f));
                }
                sum = n_q ? warp_sum(s.total()) : 0;
                __syncwarp();
            }
            if (lane == 0) sh.chunks[warp][k] = sum;
            of_run += sum, q_of_run += q_of_chunk;
        }
        join_runs(of_run, q_of_run);
    };
    if (both) {
        // sums of the scan, of float32, are summed anew
        const bool p_summed = p_kind.recorded, q_summed = q_kind.recorded || q_kind.greedy;
        if (!p_summed || !q_summed) {
            sum_of_both(true);
            if (!p_summed) p_total = total;
            if (!q_summed) q_total = q_sum;
        }
        p.divide_by(p_total), q.divide_by(q_total);
        sum_of_both(false);
        if (total == 0) {  // nothing is left over
            both = false;
            p.inv_hi = 1.0f, p.inv_lo = 0.0f;
        }
    }
    if (!both) {
        sum_of_p();
        if (total == 0 && without != 0xFFFFFFFFu) {
            without = 0xFFFFFFFFu;
            sum_of_p();
        }
        if (without == 0xFFFFFFFFu) p_total = total;
    }
    const uint64_t aim = aim_of(static_cast<double>(__ldg(a.draw_u + r)), total);
    if (!(before <= aim && aim < before + mine)) return;
    // the aim falls into this warp's run: its chunk, and the token in it
    uint32_t chunk = 0;
    __syncwarp();
    for (uint32_t k0 = 0; k0 < kMostChunks && k0 * kChunk < run1 - run0; k0 += 32) {
        const uint64_t m = (k0 + lane) * kChunk < run1 - run0 ? sh.chunks[warp][k0 + lane] : 0, inc = warp_inclusive(m);
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, before + inc - m <= aim && aim < before + inc);
        if (here) {
            const int of = __ffs(here) - 1;
            chunk = k0 + of;
            before += __shfl_sync(0xFFFFFFFFu, inc - m, of);
            break;
        }
        before += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
#pragma unroll 1
    for (uint32_t j = 0; j < kGroups; ++j) {
        const uint32_t i = run0 + chunk * kChunk + j * 128 + lane * 4;
        float x[4], y[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        load_four(z_row, a.wide[0], i, run1, x);
        if (both) load_four(q_row, a.wide[1], i, run1, y);
        uint64_t m[4], sum = 0;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            x[c] = p.value(x[c]);
            float w = i + c == without ? 0.0f : p.weight(x[c], i + c);
            if (both) w = fmaxf(p.share(w) - q.share(q.weight(q.value(y[c]), i + c)), 0.0f);
            m[c] = static_cast<uint64_t>(w * kMassOne);
            sum += m[c];
        }
        const uint64_t inc = warp_inclusive(sum);
        uint64_t at = before + inc - sum;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            if (at <= aim && aim < at + m[c]) {
                a.out_tokens[t] = static_cast<int32_t>(i + c);
                if (a.logprobs) a.logprobs[t] = log_share(kept, x[c], p_total);
            }
            at += m[c];
        }
        before += __shfl_sync(0xFFFFFFFFu, inc, 31);
    }
}

template <typename P, typename Q>
afx_status launch(const VerifyArgs& a, uint32_t ranks, cudaStream_t s) {
    AFX_SERVE_TRY(cudaFuncSetAttribute(verify_kernel<P, Q>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1), "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.n_requests * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    AFX_SERVE_TRY(cudaLaunchKernelEx(&cfg, verify_kernel<P, Q>, a), "verify_kernel launch");
    return AFX_OK;
}
template <typename P>
afx_status launch_draft(const VerifyArgs& a, uint32_t ranks, cudaStream_t s) {
    const uint32_t type = a.side[1].logits ? a.side[1].type : a.side[0].type;
    if (type == AFX_TYPE_F32) return launch<P, float>(a, ranks, s);
    if (type == AFX_TYPE_BF16) return launch<P, __nv_bfloat16>(a, ranks, s);
    return launch<P, __half>(a, ranks, s);
}

// `count` rows of both sides laid end to end, from `first` on, in grids of up to 65535 rows.
afx_status scan(const VerifyArgs& a, uint32_t type, uint64_t first, uint64_t count, cudaStream_t s) {
    constexpr uint64_t kGridRows = 65535;
    for (uint64_t r = 0; r < count; r += kGridRows) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(a.n_parts, static_cast<uint32_t>(count - r < kGridRows ? count - r : kGridRows));
        cfg.blockDim = dim3(kScanThreads);
        cfg.stream = s;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        const uint32_t row0 = static_cast<uint32_t>(first + r);
        AFX_SERVE_TRY(type == AFX_TYPE_F32    ? cudaLaunchKernelEx(&cfg, verify_scan_kernel<float>, a, row0)
                      : type == AFX_TYPE_BF16 ? cudaLaunchKernelEx(&cfg, verify_scan_kernel<__nv_bfloat16>, a, row0)
                                              : cudaLaunchKernelEx(&cfg, verify_scan_kernel<__half>, a, row0),
                      "verify_scan_kernel launch");
    }
    return AFX_OK;
}

uint64_t workspace_bytes_of(uint32_t n_tokens) {
    return (2 * (sizeof(Kept) + kMostParts * sizeof(Part)) * static_cast<uint64_t>(n_tokens) + 255) / 256 * 256 + 256;
}

bool sampling_ok(const afx_sampling& s) {
    return (!s.temperature_dev || device_ptr_here(s.temperature_dev, 4)) && (!s.top_k_dev || device_ptr_here(s.top_k_dev, 4)) &&
           (!s.top_p_dev || device_ptr_here(s.top_p_dev, 4)) && (!s.min_p_dev || device_ptr_here(s.min_p_dev, 4));
}

Side side_of(const void* logits, uint32_t type, uint64_t stride, const afx_sampling& s, Kept* kept) {
    Side d{};
    d.logits = logits;
    d.type = type;
    d.row_stride = stride;
    d.temperature = s.temperature_dev;
    d.top_k = s.top_k_dev;
    d.top_p = s.top_p_dev;
    d.min_p = s.min_p_dev;
    d.kept = kept;
    return d;
}

}  // namespace
}  // namespace serve
}  // namespace afx

using namespace afx::serve;

static_assert(AFX_TYPE_F32 == AFX_LOGITS_F32 && AFX_TYPE_BF16 == AFX_LOGITS_BF16 && AFX_TYPE_FP16 == AFX_LOGITS_FP16, "one list of types");

extern "C" afx_status afx_verify_workspace(uint32_t n_tokens, uint32_t n_requests, uint64_t* bytes) {
    if (!bytes) return afx_fail(AFX_E_ARG, "null size", 0);
    if (n_requests == 0 || n_requests > AFX_KV_MAX_REQUESTS || n_tokens > 1u << 24)
        return afx_fail(AFX_E_ARG, "1 to 16384 requests, at most 2^24 rows", 0);
    *bytes = workspace_bytes_of(n_tokens);
    return AFX_OK;
}

extern "C" afx_status afx_verify(const afx_verify_args* args, int32_t* out_tokens_dev, int32_t* counts_dev, float* logprobs_dev,
                                 void* workspace_dev, uint64_t workspace_bytes, afx_stream_t stream, int32_t* status_dev) {
    if (!args) return afx_fail(AFX_E_ARG, "null description", 0);
    const afx_verify_args& v = *args;
    if (v.type > AFX_TYPE_F32 || (v.draft_logits_dev && v.draft_type > AFX_TYPE_F32)) return afx_fail(AFX_E_ARG, "unknown logits type", 0);
    if (v.vocab == 0 || v.vocab > AFX_SAMPLE_MAX_VOCAB) return afx_fail(AFX_E_ARG, "a row has 1 to 524288 logits", 0);
    if (v.n_requests == 0 || v.n_requests > AFX_KV_MAX_REQUESTS || v.n_tokens > 1u << 24)
        return afx_fail(AFX_E_ARG, "1 to 16384 requests, at most 2^24 rows", 0);
    if (v.n_tokens > 1 && (v.row_stride < v.vocab || (v.draft_logits_dev && v.draft_row_stride < v.vocab)))
        return afx_fail(AFX_E_ARG, "rows of logits lie at least a row apart", 0);
    // no rows: counts of 0 all the same
    const uint32_t size = v.type == AFX_TYPE_F32 ? 4 : 2, draft_size = v.draft_type == AFX_TYPE_F32 ? 4 : 2;
    if (!device_ptr_here(v.starts_dev, 4) || !device_ptr_here(counts_dev, 4) || !device_ptr_here(v.draw_u_dev, 4) ||
        (v.n_tokens && (!device_ptr_here(v.logits_dev, size) || !device_ptr_here(v.tokens_dev, 4) || !device_ptr_here(v.u_dev, 4) || !device_ptr_here(out_tokens_dev, 4) ||
                        (logprobs_dev && !device_ptr_here(logprobs_dev, 4)) || (v.draft_logits_dev && !device_ptr_here(v.draft_logits_dev, draft_size)))) ||
        !sampling_ok(v.sampling) || (v.draft_logits_dev && !sampling_ok(v.draft_sampling)) || (status_dev && !device_ptr_here(status_dev, 4)))
        return afx_fail(AFX_E_ARG, "the arrays must be memory of the current device", 0);
    if (!device_ptr_here(workspace_dev, 256)) return afx_fail(AFX_E_ARG, "the workspace must be 256-byte aligned memory of the current device", 0);
    if (workspace_bytes < workspace_bytes_of(v.n_tokens)) return afx_fail(AFX_E_NOSPACE, "the workspace is smaller than afx_verify_workspace", 0);
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    VerifyArgs a{};
    Kept* kept = static_cast<Kept*>(workspace_dev);
    a.side[0] = side_of(v.logits_dev, v.type, v.row_stride, v.sampling, kept);
    // without drafts' logits their parameters mean nothing and have not been checked: the kernels, which read a side's by its
    // pointers, get none
    a.side[1] = side_of(v.draft_logits_dev, v.draft_type, v.draft_row_stride, v.draft_logits_dev ? v.draft_sampling : afx_sampling{}, kept + v.n_tokens);
    a.parts = reinterpret_cast<Part*>(kept + 2 * static_cast<uint64_t>(v.n_tokens));
    a.starts = v.starts_dev;
    a.tokens = v.tokens_dev;
    a.u = v.u_dev;
    a.draw_u = v.draw_u_dev;
    a.out_tokens = out_tokens_dev;
    a.counts = counts_dev;
    a.logprobs = logprobs_dev;
    a.status = status_dev;
    a.n_requests = v.n_requests;
    a.n_tokens = v.n_tokens;
    a.vocab = v.vocab;
    // A request's row over CTAs of more than 2048 tokens, up to twice as many as SMs in all, three times where drafts' logits are
    // read too (200 requests without: 96 us, 104 with the larger number; 96 requests of four drafts with, float32: 178 and 152)
    uint32_t ranks = 1;
    while (ranks < kMaxCluster && v.vocab / ranks > 4096 && static_cast<uint64_t>(v.n_requests) * ranks <= static_cast<uint64_t>(sms) * (v.draft_logits_dev ? 3 : 2)) ranks *= 2;
    a.slice = ceil_div(ceil_div(v.vocab, ranks), 128) * 128;
    a.run = ceil_div(a.slice, kWarps * kChunk) * kChunk;
    auto aligned = [&](const void* p, uint64_t stride, uint32_t bytes, uint32_t to) {
        return !((reinterpret_cast<uintptr_t>(p) | (v.n_tokens > 1 ? stride * bytes : 0)) & (to - 1));
    };
    a.wide[0] = aligned(v.logits_dev, v.row_stride, size, 4 * size);
    a.scan_wide[0] = aligned(v.logits_dev, v.row_stride, size, 16);
    a.wide[1] = v.draft_logits_dev && aligned(v.draft_logits_dev, v.draft_row_stride, draft_size, 4 * draft_size);
    a.scan_wide[1] = v.draft_logits_dev && aligned(v.draft_logits_dev, v.draft_row_stride, draft_size, 16);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (v.n_tokens) {
        // parts of rows: enough CTAs to fill the GPU several times over, with 1024 tokens or more each
        const uint64_t all = static_cast<uint64_t>(v.n_tokens) * (v.draft_logits_dev ? 2 : 1), want = (8ull * sms + all - 1) / all;
        a.n_parts = static_cast<uint32_t>(want > kMostParts ? kMostParts : want);
        a.part = ceil_div(ceil_div(v.vocab, a.n_parts), 1024) * 1024;
        a.n_parts = ceil_div(v.vocab, a.part);
        // the rows that keep all
        afx_status st = AFX_OK;
        if (!v.draft_logits_dev || v.draft_type == v.type) {
            st = scan(a, v.type, 0, all, s);
        } else {
            st = scan(a, v.type, 0, v.n_tokens, s);
            if (st == AFX_OK) st = scan(a, v.draft_type, v.n_tokens, v.n_tokens, s);
        }
        // the others, where there can be any
        const bool cuts = v.sampling.top_k_dev || v.sampling.top_p_dev || v.sampling.min_p_dev ||
                          (v.draft_logits_dev && (v.draft_sampling.top_k_dev || v.draft_sampling.top_p_dev || v.draft_sampling.min_p_dev));
        if (st == AFX_OK && cuts) st = launch_records(a.side[0], a.side[1], v.n_tokens, v.vocab, v.starts_dev, v.tokens_dev, v.n_requests, s);
        if (st != AFX_OK) return st;
    }
    if (v.type == AFX_TYPE_F32) return launch_draft<float>(a, ranks, s);
    if (v.type == AFX_TYPE_BF16) return launch_draft<__nv_bfloat16>(a, ranks, s);
    return launch_draft<__half>(a, ranks, s);
}
