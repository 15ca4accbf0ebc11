// sm_103a verification of drafted tokens (afx_verify).
//
// Row t of a request decides on a draft d that was drawn from q_t; p_t is what
// afx_sample would draw from.  The draft stands with probability
// min(1, p_t(d) / q_t(d)): where u q_t(d) < p_t(d).  At the first row whose
// draft does not stand, the token is drawn from max(p_t - q_t, 0), which leaves
// tokens distributed as p_t: a token's chance is min(p, q) + (1 - sum min(p, q))
// max(p - q, 0) / sum max(p - q, 0) = p.
//
// Two launches.  The first is the sampling kernel without its draw
// (verify_record_kernel, afx_sample.cu): for every row of the target and of the drafts what top-k,
// top-p and min-p keep, as the last place kept and the kept weights' sum, so
// that a token's share is its weight by the sum.  All rows at once, although
// rows behind a refused draft turn out not to be needed: one after the other they would take
// as many passes as there are drafts.  The second, verify_kernel, has a cluster
// a request: a thread a draft for the tests, then two passes over the row to draw from:
// the masses of max(p - q, 0) as integers of 2^-44, whose sums do not depend
// on their order, then the run of tokens in which the aim falls.  A token that
// p does not keep needs no q, so that behind top-k or top-p few of the draft's
// logits are read again.
#include <cooperative_groups.h>

#include <utility>

#include "afx_sample.cuh"

namespace cg = cooperative_groups;

namespace afx {
namespace serve {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct VerifyArgs {
    Side target, draft;
    const int32_t *starts, *tokens;
    const float *u, *draw_u;
    int32_t *out_tokens, *counts;
    float* logprobs;
    int32_t* status;
    uint32_t n_requests, n_tokens, vocab, slice, run;
    uint32_t wide, draft_wide;
};

struct Shared {
    uint64_t warps[kWarps];
    uint64_t total[2][kMaxCluster];  // every rank's mass: of the first choice of weights, of the second
    int32_t first;
};

template <typename P, typename Q>
struct Request {
    const VerifyArgs& a;
    __device__ float target(int32_t t, uint32_t i) const {
        return clean(load_logit(static_cast<const P*>(a.target.logits) + t * a.target.row_stride + i));
    }
    __device__ float draft(int32_t t, uint32_t i) const {
        return clean(load_logit(static_cast<const Q*>(a.draft.logits) + t * a.draft.row_stride + i));
    }
    // whether row t's draft d stands
    __device__ bool stands(int32_t t, uint32_t d) const {
        const Kept p = a.target.kept[t];
        const double share = static_cast<double>(p.weight(p.value(target(t, d)), d)) * kMassOne / static_cast<double>(p.total);
        double other = 1.0;
        if (a.draft.logits) {
            const Kept q = a.draft.kept[t];
            other = q.total ? static_cast<double>(q.weight(q.value(draft(t, d)), d)) * kMassOne / static_cast<double>(q.total) : 0.0;
        }
        return p.total && static_cast<double>(__ldg(a.u + t)) * other < share;
    }
    __device__ float log_share(const Kept& p, float z) const { return p.scaled(z) - logf(static_cast<float>(p.total) * (1.0f / kMassOne)); }
};

enum Weights { kOfTarget, kWithoutDraft, kLeftOver };

template <typename P, typename Q>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
    __shared__ Shared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const uint32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t r = blockIdx.x / ranks;
    const Request<P, Q> rq{a};
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

    // the first row whose draft does not stand, or the last row
    const int32_t last = row1 - row0 - 1;
    int32_t stood = last;
    for (int32_t i0 = 0; i0 < last; i0 += kThreads) {
        const int32_t i = i0 + threadIdx.x;
        if (threadIdx.x == 0) sh.first = last;
        __syncthreads();
        if (i < last) {
            const int32_t d = draft_of(a.tokens, row0 + i, row1, a.vocab);
            if (d < 0 || !rq.stands(row0 + i, d)) atomicMin(&sh.first, i);
        }
        __syncthreads();
        stood = sh.first;
        __syncthreads();
        if (stood < last) break;
    }
    const int32_t t = row0 + stood;
    const Kept p = a.target.kept[t];
    const bool nothing = p.top == -INFINITY;
    if (rank == 0) {
        for (int32_t i = threadIdx.x; i <= last; i += kThreads) {
            if (i == stood && !nothing) continue;
            const uint32_t d = i < stood ? __ldg(a.tokens + row0 + i + 1) : 0;
            a.out_tokens[row0 + i] = i < stood ? static_cast<int32_t>(d) : -1;
            if (a.logprobs) {
                float l = i == stood ? -INFINITY : 0.0f;
                if (i < stood) {
                    const Kept k = a.target.kept[row0 + i];
                    l = rq.log_share(k, k.value(rq.target(row0 + i, d)));
                }
                a.logprobs[row0 + i] = l;
            }
        }
        if (threadIdx.x == 0) a.counts[r] = nothing ? stood : stood + 1;
    }
    if (nothing) return;  // the whole cluster

    // the draw
    const int32_t refused = draft_of(a.tokens, t, row1, a.vocab);
    Kept q{};
    if (refused >= 0 && a.draft.logits) q = a.draft.kept[t];
    Weights weights = refused < 0 ? kOfTarget : !a.draft.logits ? kWithoutDraft : q.total ? kLeftOver : kOfTarget;
    const float p_total = static_cast<float>(p.total) * (1.0f / kMassOne), q_total = static_cast<float>(q.total) * (1.0f / kMassOne);
    const float low = key_value(static_cast<uint32_t>(p.threshold >> 32));  // NaN where all are kept
    const uint32_t base = min(a.vocab, rank * a.slice), n = min(a.vocab - base, a.slice);
    const uint32_t run0 = min(n, warp * a.run), run1 = min(n, run0 + a.run);
    const P* z_row = static_cast<const P*>(a.target.logits) + t * a.target.row_stride;
    const Q* q_row = static_cast<const Q*>(a.draft.logits) + t * a.draft.row_stride;
    // token i's mass, x and y its logits
    auto mass_of = [&](uint32_t i, float x, float y) -> uint64_t {
        const float w = p.weight(x, i);
        if (weights == kOfTarget) return static_cast<uint64_t>(w * kMassOne);
        if (weights == kWithoutDraft) return i == static_cast<uint32_t>(refused) ? 0 : static_cast<uint64_t>(w * kMassOne);
        return static_cast<uint64_t>(fmaxf(__fdiv_rn(w, p_total) - __fdiv_rn(q.weight(y, i), q_total), 0.0f) * kMassOne);
    };
    uint64_t before = 0, mine = 0, total = 0;
    for (int turn = 0; turn < 2; ++turn) {
        uint64_t sum = 0;
        for (uint32_t i = run0 + lane * 4; i < run1 + lane * 4; i += 128) {  // whole warps
            float x[4];
            if (a.wide && i + 4 <= run1) {
                load4(z_row + base + i, x);
            } else {
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) x[c] = i + c < run1 ? load_logit(z_row + base + i + c) : -INFINITY;
            }
            bool any = false;
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) {
                x[c] = p.value(clean(x[c]));
                any |= x[c] > -INFINITY && !(x[c] < low);
            }
            if (!__any_sync(0xFFFFFFFFu, any)) continue;
            float y[4] = {};
            if (weights == kLeftOver) {
                if (a.draft_wide && i + 4 <= run1) {
                    load4(q_row + base + i, y);
                } else {
#pragma unroll
                    for (uint32_t c = 0; c < 4; ++c) y[c] = i + c < run1 ? load_logit(q_row + base + i + c) : -INFINITY;
                }
#pragma unroll
                for (uint32_t c = 0; c < 4; ++c) y[c] = q.value(clean(y[c]));
            }
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c)
                if (x[c] > -INFINITY && !(x[c] < low)) sum += mass_of(base + i + c, x[c], y[c]);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        mine = sum;
        __syncthreads();
        if (lane == 0) sh.warps[warp] = sum;
        __syncthreads();
        uint64_t of_slice = 0;
        before = total = 0;
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += sh.warps[i];
            of_slice += sh.warps[i];
        }
        if (threadIdx.x < ranks) cluster.map_shared_rank(&sh, threadIdx.x)->total[turn][rank] = of_slice;
        cluster.sync();
        for (uint32_t i = 0; i < ranks; ++i) {
            if (i < rank) before += sh.total[turn][i];
            total += sh.total[turn][i];
        }
        if (total || weights == kOfTarget) break;
        weights = kOfTarget;  // nothing is left over
    }
    const uint64_t aim = aim_of(static_cast<double>(__ldg(a.draw_u + r)), total);
    if (!(before <= aim && aim < before + mine)) return;
    // the aim falls into this warp's run
    for (uint32_t i = run0; i < run1; i += 32) {
        const uint32_t at = i + lane;
        float x = -INFINITY;
        uint64_t m = 0;
        if (at < run1) {
            x = p.value(rq.target(t, base + at));
            if (x > -INFINITY && !(x < low)) m = mass_of(base + at, x, weights == kLeftOver ? q.value(rq.draft(t, base + at)) : 0.0f);
        }
        const uint64_t inc = warp_inclusive(m);
        if (before + inc - m <= aim && aim < before + inc) {
            a.out_tokens[t] = static_cast<int32_t>(base + at);
            if (a.logprobs) a.logprobs[t] = rq.log_share(p, x);
        }
        before += __shfl_sync(0xFFFFFFFFu, inc, 31);
        if (before > aim) break;
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
    const uint32_t type = a.draft.logits ? a.draft.type : a.target.type;
    if (type == AFX_TYPE_F32) return launch<P, float>(a, ranks, s);
    if (type == AFX_TYPE_BF16) return launch<P, __nv_bfloat16>(a, ranks, s);
    return launch<P, __half>(a, ranks, s);
}

uint64_t workspace_bytes_of(uint32_t n_tokens) { return (2 * sizeof(Kept) * static_cast<uint64_t>(n_tokens) + 255) / 256 * 256 + 256; }

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
    a.target = side_of(v.logits_dev, v.type, v.row_stride, v.sampling, kept);
    a.draft = side_of(v.draft_logits_dev, v.draft_type, v.draft_row_stride, v.draft_sampling, kept + v.n_tokens);
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
    a.run = ceil_div(a.slice, kWarps * 128) * 128;
    auto aligned = [&](const void* p, uint64_t stride, uint32_t bytes) {
        return !((reinterpret_cast<uintptr_t>(p) | (v.n_tokens > 1 ? stride * bytes : 0)) & (4 * bytes - 1));
    };
    a.wide = aligned(v.logits_dev, v.row_stride, size);
    a.draft_wide = v.draft_logits_dev && aligned(v.draft_logits_dev, v.draft_row_stride, draft_size);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (v.n_tokens) {
        const afx_status st = launch_records(a.target, a.draft, v.n_tokens, v.vocab, v.starts_dev, v.tokens_dev, v.n_requests, s);
        if (st != AFX_OK) return st;
    }
    if (v.type == AFX_TYPE_F32) return launch_draft<float>(a, ranks, s);
    if (v.type == AFX_TYPE_BF16) return launch_draft<__nv_bfloat16>(a, ranks, s);
    return launch_draft<__half>(a, ranks, s);
}
