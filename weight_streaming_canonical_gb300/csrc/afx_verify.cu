// sm_103a verification of drafted tokens (afx_verify).
//
// Row t of a request decides on a draft d that was drawn from q_t; p_t is what
// afx_sample would draw from.  The draft stands with probability
// min(1, p_t(d) / q_t(d)): where u q_t(d) < p_t(d).  At the first row whose
// draft does not stand, the token is drawn from max(p_t - q_t, 0), which leaves
// tokens distributed as p_t: a token's chance is min(p, q) + (1 - sum min(p, q))
// max(p - q, 0) / sum max(p - q, 0) = p.
//
// Up to three launches.  verify_scan_kernel reads the rows that keep all
// their tokens or, at temperature 0, one: a part of a row a CTA, with a running
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
// for a test or a logarithm; a draw from differences of rows that keep all
// first sums their masses.
#include <cooperative_groups.h>

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
    uint32_t wide[2];
};

// ---- one pass over rows that keep all ------------------------------------------------

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
    constexpr uint32_t kRuns = 8;  // of four tokens a thread, in flight
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
    const bool wide = a.wide[second];
    Part mine{-INFINITY, 0.0f, 0xFFFFFFFFu, 0};
    for (uint32_t i0 = at0; i0 < at1; i0 += kScanThreads * 4 * kRuns) {
        float x[kRuns][4];
#pragma unroll
        for (uint32_t j = 0; j < kRuns; ++j) {
            const uint32_t i = i0 + (j * kScanThreads + threadIdx.x) * 4;
            if (wide && i + 4 <= at1) {
                load4(z + i, x[j]);
            } else {
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) x[j][c] = i + c < at1 ? load_logit(z + i + c) : -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (uint32_t j = 0; j < kRuns; ++j)
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) {
                x[j][c] = clean(x[j][c]);
                top = fmaxf(top, x[j][c]);
            }
        if (top == -INFINITY) continue;
        if (!(t > 0.0f)) {  // the maximum alone
            if (top > mine.top)
#pragma unroll
                for (uint32_t j = kRuns; j-- > 0;)
#pragma unroll
                    for (uint32_t c = 4; c-- > 0;)
                        if (x[j][c] == top) mine.first = i0 + (j * kScanThreads + threadIdx.x) * 4 + c;
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
                for (uint32_t c = 0; c < 4; ++c) mine.infinite += x[j][c] == INFINITY;
            continue;
        }
        float sum[4] = {};
#pragma unroll
        for (uint32_t j = 0; j < kRuns; ++j)
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) sum[c] += exp2_approx((x[j][c] - mine.top) * inv_t * 1.44269504f);
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
__device__ Kept kept_of(const VerifyArgs& a, int which, uint32_t request, uint32_t r) {
    const Side& side = a.side[which];
    const float t = temperature_of(side, request);
    if (t > 0.0f && !keeps_all(side, request, a.vocab)) return side.kept[r];
    const Part* parts = a.parts + (static_cast<uint64_t>(which) * a.n_tokens + r) * a.n_parts;
    const float inv_t = t > 0.0f ? inverse_temperature(t) : 1.0f;
    Part all = parts[0];
    for (uint32_t i = 1; i < a.n_parts; ++i) join(all, parts[i], inv_t);
    Kept k;
    k.infinite = all.top == INFINITY;
    k.top = k.infinite ? 0.0f : all.top;
    k.inv_t = inv_t;
    k.least = 0.0f;
    k.threshold = t > 0.0f ? 0 : place(k.top, all.first);
    const float sum = !(t > 0.0f) ? 1.0f : k.infinite ? static_cast<float>(all.infinite) : all.sum;
    k.total = all.top == -INFINITY ? 0 : static_cast<uint64_t>(static_cast<double>(sum) * kMassOne);
    return k;
}

// ---- the tests and the draw ------------------------------------------------------------

struct Shared {
    uint64_t chunks[kWarps][kMostChunks];  // masses
    uint64_t warps[2][kWarps];
    uint64_t total[3][2][kMaxCluster];     // every rank's masses, turn by turn
    int32_t first;
};

__device__ __forceinline__ float log_share(const Kept& p, float z, uint64_t total) {
    return p.scaled(z) - logf(static_cast<float>(total) * (1.0f / kMassOne));
}

// x times a number held as the sum of two float32: the quotient by its inverse, rounded nearly always as the exact one is
struct Inverse {
    float hi, lo;
    __device__ explicit Inverse(uint64_t total) {
        const double inv = total ? static_cast<double>(kMassOne) / static_cast<double>(total) : 0.0;
        hi = static_cast<float>(inv);
        lo = static_cast<float>(inv - static_cast<double>(hi));
    }
    __device__ float times(float x) const { return fmaf(x, hi, x * lo); }
};

enum Weights { kOfTarget, kWithoutDraft, kLeftOver, kSums };  // kSums: those of p and of q, apart

template <typename P, typename Q>
struct Draw {
    const P* z_row;
    const Q* q_row;
    Kept p, q;
    float low;        // of p's tokens; minus infinity where all are kept
    bool p_all, q_all, z_wide, q_wide;
    int32_t refused;
    Inverse p_inv{0}, q_inv{0};

    // four logits from i on (of tokens below end)
    template <typename T>
    __device__ static void load(const T* row, bool wide, uint32_t i, uint32_t end, float (&x)[4]) {
        if (wide && i + 4 <= end) {
            load4(row + i, x);
        } else {
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) x[c] = i + c < end ? load_logit(row + i + c) : -INFINITY;
        }
    }
    __device__ static float weight(const Kept& k, bool all, float x, uint32_t i) {
        return all ? expf(k.scaled(x)) : k.weight(x, i);  // e^minus infinity is 0
    }
    // token i's mass, x and y its logits as value() gives them
    __device__ uint64_t mass(Weights w, uint32_t i, float x, float y) const {
        const float px = weight(p, p_all, x, i);
        if (w == kLeftOver) return static_cast<uint64_t>(fmaxf(p_inv.times(px) - q_inv.times(weight(q, q_all, y, i)), 0.0f) * kMassOne);
        if (w == kWithoutDraft && i == static_cast<uint32_t>(refused)) return 0;
        return static_cast<uint64_t>(px * kMassOne);
    }
    // this lane's logits of a chunk; false: no lane's can have mass
    __device__ bool chunk(Weights w, uint32_t i0, uint32_t end, float (&x)[kGroups][4], float (&y)[kGroups][4]) const {
        const uint32_t lane = threadIdx.x & 31;
        float most = -INFINITY;
#pragma unroll
        for (uint32_t j = 0; j < kGroups; ++j) load(z_row, z_wide, i0 + j * 128 + lane * 4, end, x[j]);
        if (w >= kLeftOver && p_all)  // most of q's are needed
#pragma unroll
            for (uint32_t j = 0; j < kGroups; ++j) load(q_row, q_wide, i0 + j * 128 + lane * 4, end, y[j]);
#pragma unroll
        for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) {
                x[j][c] = p.value(clean(x[j][c]));
                most = fmaxf(most, x[j][c]);
            }
        if (w != kSums && !__any_sync(0xFFFFFFFFu, most > -INFINITY && most >= low)) return false;
        if (w >= kLeftOver) {
            if (!p_all)
#pragma unroll
                for (uint32_t j = 0; j < kGroups; ++j) load(q_row, q_wide, i0 + j * 128 + lane * 4, end, y[j]);
#pragma unroll
            for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) y[j][c] = q.value(clean(y[j][c]));
        }
        return true;
    }
};

template <typename P, typename Q>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t r = blockIdx.x / ranks;
    const Side &target = a.side[0], &draft = a.side[1];
    auto started = cluster.barrier_arrive();  // a rank's memory may be written once its CTA runs
    wait_for_earlier();
    let_next_start();
    // all of the call or nothing: every CTA looks at all starts
    int bad = 0;
    for (uint32_t i = threadIdx.x; i <= a.n_requests; i += kThreads) {
        const int32_t s = __ldg(a.starts + i), before = i ? __ldg(a.starts + i - 1) : 0;
        bad |= s < before || s > static_cast<int32_t>(a.n_tokens) || (i == 0 && s != 0);
    }
    bad = __syncthreads_or(bad);
    const int32_t row0 = __ldg(a.starts + r), row1 = __ldg(a.starts + r + 1);
    cluster.barrier_wait(std::move(started));
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
                const Kept p = kept_of(a, 0, r, t);
                const double share = static_cast<double>(p.weight(p.value(z_of(t, d)), d)) * kMassOne / static_cast<double>(p.total);
                double other = 1.0;
                if (draft.logits) {
                    const Kept q = kept_of(a, 1, r, t);
                    other = q.total ? static_cast<double>(q.weight(q.value(q_of(t, d)), d)) * kMassOne / static_cast<double>(q.total) : 0.0;
                }
                stands = p.total && static_cast<double>(__ldg(a.u + t)) * other < share;
            }
            if (!stands) atomicMin(&sh.first, i);
        }
        __syncthreads();
        stood = sh.first;
        __syncthreads();
        if (stood < last) break;
    }
    const int32_t t = row0 + stood;
    Draw<P, Q> draw;
    draw.p = kept_of(a, 0, r, t);
    const bool nothing = draw.p.top == -INFINITY, greedy = !(temperature_of(target, r) > 0.0f);
    if (rank == 0) {
        for (int32_t i = threadIdx.x; i <= last; i += kThreads) {
            if (i == stood && !nothing) continue;
            const uint32_t d = i < stood ? __ldg(a.tokens + row0 + i + 1) : 0;
            a.out_tokens[row0 + i] = i < stood ? static_cast<int32_t>(d) : -1;
            if (a.logprobs) {
                float l = i == stood ? -INFINITY : 0.0f;
                if (i < stood) {
                    const Kept k = kept_of(a, 0, r, row0 + i);
                    l = log_share(k, k.value(z_of(row0 + i, d)), k.total);
                }
                a.logprobs[row0 + i] = l;
            }
        }
        if (threadIdx.x == 0) {
            a.counts[r] = nothing ? stood : stood + 1;
            if (greedy && !nothing) {  // the one token that p keeps, whatever q is
                a.out_tokens[t] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(draw.p.threshold));
                if (a.logprobs) a.logprobs[t] = 0.0f;
            }
        }
    }
    if (nothing || greedy) return;  // the whole cluster

    // the draw
    draw.refused = draft_of(a.tokens, t, row1, a.vocab);
    Weights weights = draw.refused < 0 ? kOfTarget : kWithoutDraft;
    draw.q = Kept{};
    if (draw.refused >= 0 && draft.logits) {
        draw.q = kept_of(a, 1, r, t);
        weights = draw.q.total ? kLeftOver : kOfTarget;
    }
    const uint32_t base = min(a.vocab, rank * a.slice), n = min(a.vocab - base, a.slice);
    const uint32_t run0 = base + min(n, warp * a.run), run1 = min(base + n, run0 + a.run);
    draw.z_row = static_cast<const P*>(target.logits) + t * target.row_stride;
    draw.q_row = static_cast<const Q*>(draft.logits) + t * draft.row_stride;
    draw.z_wide = a.wide[0], draw.q_wide = a.wide[1];
    draw.p_all = draw.p.threshold == 0 && draw.p.least == 0.0f, draw.q_all = draw.q.threshold == 0 && draw.q.least == 0.0f;
    draw.low = draw.p.threshold ? key_value(static_cast<uint32_t>(draw.p.threshold >> 32)) : -INFINITY;
    uint64_t before = 0, mine = 0, total = 0;
    uint32_t turn = 0;
    // the masses of every chunk of this warp's run, of its run (mine), of the runs before it and of the row
    auto sum_up = [&](Weights w) {
        uint64_t of_run[2] = {0, 0};
        uint32_t k = 0;
        for (uint32_t i0 = run0; i0 < run1; i0 += kChunk, ++k) {
            float x[kGroups][4], y[kGroups][4];
            uint64_t sum[2] = {0, 0};
            if (draw.chunk(w, i0, run1, x, y)) {
                if (w == kSums) {
                    MassSum s[2];
#pragma unroll
                    for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                        for (uint32_t c = 0; c < 4; ++c) {
                            const uint32_t i = i0 + j * 128 + lane * 4 + c;
                            s[0].add(draw.weight(draw.p, draw.p_all, x[j][c], i));
                            s[1].add(draw.weight(draw.q, draw.q_all, y[j][c], i));
                        }
                    sum[0] = s[0].total(), sum[1] = s[1].total();
                } else if (w != kLeftOver && draw.p_all) {
                    MassSum s;
#pragma unroll
                    for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                        for (uint32_t c = 0; c < 4; ++c) {
                            const float px = expf(draw.p.scaled(x[j][c]));
                            s.add(w == kWithoutDraft && i0 + j * 128 + lane * 4 + c == static_cast<uint32_t>(draw.refused) ? 0.0f : px);
                        }
                    sum[0] = s.total();
                } else {
#pragma unroll
                    for (uint32_t j = 0; j < kGroups; ++j)
#pragma unroll
                        for (uint32_t c = 0; c < 4; ++c)
                            if (x[j][c] > -INFINITY && x[j][c] >= draw.low) sum[0] += draw.mass(w, i0 + j * 128 + lane * 4 + c, x[j][c], y[j][c]);
                }
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) {
                sum[0] += __shfl_xor_sync(0xFFFFFFFFu, sum[0], d);
                if (w == kSums) sum[1] += __shfl_xor_sync(0xFFFFFFFFu, sum[1], d);
            }
            if (lane == 0) sh.chunks[warp][k] = sum[0];
            of_run[0] += sum[0], of_run[1] += sum[1];
        }
        __syncthreads();
        if (lane == 0) sh.warps[0][warp] = of_run[0], sh.warps[1][warp] = of_run[1];
        __syncthreads();
        uint64_t of_slice[2] = {0, 0};
        before = 0;
        for (uint32_t i = 0; i < kWarps; ++i) {
            if (i < warp) before += sh.warps[0][i];
            of_slice[0] += sh.warps[0][i], of_slice[1] += sh.warps[1][i];
        }
        if (threadIdx.x < ranks) {
            Shared* other = cluster.map_shared_rank(&sh, threadIdx.x);
            other->total[turn][0][rank] = of_slice[0], other->total[turn][1][rank] = of_slice[1];
        }
        cluster.sync();
        total = 0;
        uint64_t second = 0;
        for (uint32_t i = 0; i < ranks; ++i) {
            if (i < rank) before += sh.total[turn][0][i];
            total += sh.total[turn][0][i];
            second += sh.total[turn][1][i];
        }
        mine = of_run[0];
        ++turn;
        return second;
    };
    if (weights == kLeftOver) {
        uint64_t p_total = draw.p.total, q_total = draw.q.total;
        const bool q_summed = !(temperature_of(draft, r) > 0.0f) || !keeps_all(draft, r, a.vocab);
        const bool p_summed = !keeps_all(target, r, a.vocab);
        if (!p_summed || !q_summed) {
            const uint64_t second = sum_up(kSums);
            if (!p_summed) p_total = total;
            if (!q_summed) q_total = second;
        }
        draw.p_inv = Inverse(p_total), draw.q_inv = Inverse(q_total);
    }
    sum_up(weights);
    if (total == 0 && weights != kOfTarget) {  // nothing is left over
        weights = kOfTarget;
        sum_up(weights);
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
    float x[kGroups][4], y[kGroups][4];
    const uint32_t i0 = run0 + chunk * kChunk;
    draw.chunk(weights, i0, run1, x, y);
#pragma unroll
    for (uint32_t j = 0; j < kGroups; ++j) {
        uint64_t m[4], sum = 0;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            m[c] = x[j][c] > -INFINITY && x[j][c] >= draw.low ? draw.mass(weights, i0 + j * 128 + lane * 4 + c, x[j][c], y[j][c]) : 0;
            sum += m[c];
        }
        const uint64_t inc = warp_inclusive(sum);
        uint64_t at = before + inc - sum;
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            if (at <= aim && aim < at + m[c]) {
                a.out_tokens[t] = static_cast<int32_t>(i0 + j * 128 + lane * 4 + c);
                if (a.logprobs) a.logprobs[t] = log_share(draw.p, x[j][c], weights == kOfTarget ? total : draw.p.total);
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
    return (!s.temperature_dev || device_ptr(s.temperature_dev, 4)) && (!s.top_k_dev || device_ptr(s.top_k_dev, 4)) &&
           (!s.top_p_dev || device_ptr(s.top_p_dev, 4)) && (!s.min_p_dev || device_ptr(s.min_p_dev, 4));
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
    if (!device_ptr(v.starts_dev, 4) || !device_ptr(counts_dev, 4) || !device_ptr(v.draw_u_dev, 4) ||
        (v.n_tokens && (!device_ptr(v.logits_dev, size) || !device_ptr(v.tokens_dev, 4) || !device_ptr(v.u_dev, 4) || !device_ptr(out_tokens_dev, 4) ||
                        (logprobs_dev && !device_ptr(logprobs_dev, 4)) || (v.draft_logits_dev && !device_ptr(v.draft_logits_dev, draft_size)))) ||
        !sampling_ok(v.sampling) || (v.draft_logits_dev && !sampling_ok(v.draft_sampling)) || (status_dev && !device_ptr(status_dev, 4)))
        return afx_fail(AFX_E_ARG, "the arrays must be device memory", 0);
    if (!device_ptr(workspace_dev, 256)) return afx_fail(AFX_E_ARG, "the workspace must be 256-byte aligned device memory", 0);
    if (workspace_bytes < workspace_bytes_of(v.n_tokens)) return afx_fail(AFX_E_NOSPACE, "the workspace is smaller than afx_verify_workspace", 0);
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    VerifyArgs a{};
    Kept* kept = static_cast<Kept*>(workspace_dev);
    a.side[0] = side_of(v.logits_dev, v.type, v.row_stride, v.sampling, kept);
    a.side[1] = side_of(v.draft_logits_dev, v.draft_type, v.draft_row_stride, v.draft_sampling, kept + v.n_tokens);
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
    // a request's row over as many CTAs as there is room for two an SM, with 2048 tokens or more each
    uint32_t ranks = 1;
    while (ranks < kMaxCluster && v.vocab / ranks > 4096 && static_cast<uint64_t>(v.n_requests) * ranks <= static_cast<uint64_t>(sms)) ranks *= 2;
    a.slice = ceil_div(ceil_div(v.vocab, ranks), 128) * 128;
    a.run = ceil_div(a.slice, kWarps * kChunk) * kChunk;
    auto aligned = [&](const void* p, uint64_t stride, uint32_t bytes) {
        return !((reinterpret_cast<uintptr_t>(p) | (v.n_tokens > 1 ? stride * bytes : 0)) & (4 * bytes - 1));
    };
    a.wide[0] = aligned(v.logits_dev, v.row_stride, size);
    a.wide[1] = v.draft_logits_dev && aligned(v.draft_logits_dev, v.draft_row_stride, draft_size);
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
