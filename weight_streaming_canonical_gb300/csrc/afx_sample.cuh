// What sampling (afx_sample.cu) and verification of drafts (afx_verify.cu)
// share: the order of tokens, masses as integers, loads of logits, and the
// record of what a row keeps.
#pragma once

#include "afx_serving.cuh"

namespace afx {
namespace serve {

constexpr uint32_t kMaxCluster = 16;
constexpr float kMassOne = 17592186044416.0f;  // 2^44

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

// floor(u * total), below total.
__device__ __forceinline__ uint64_t aim_of(double u, uint64_t total) {
    const double scaled = u > 0.0 ? u * static_cast<double>(total) : 0.0;
    return scaled < static_cast<double>(total) ? min(static_cast<uint64_t>(scaled), total - 1) : total - 1;
}
// What temperature, top-k, top-p and min-p leave of a row: token i of logit z
// is kept where place(z, i) >= threshold and e^y >= least, y = (z - top) *
// inv_t; total is the kept weights' sum in 2^-44.  Of a row with infinite
// logits these count as 0 and all others as minus infinity.
struct Kept {
    float top, inv_t, least;  // top minus infinity: nothing to draw from
    uint32_t infinite;
    uint64_t threshold, total;
    __device__ __forceinline__ float value(float z) const { return infinite ? (z == INFINITY ? 0.0f : -INFINITY) : z; }
    __device__ __forceinline__ float scaled(float z) const { return (z - top) * inv_t; }  // z as value() gives it
    __device__ __forceinline__ float weight(float z, uint32_t i) const {
        if (!(z > -INFINITY) || place(z, i) < threshold) return 0.0f;
        const float w = expf(scaled(z));
        return w >= least ? w : 0.0f;
    }
};
static_assert(sizeof(Kept) == 32, "a record a sector");

// One side of a verification: logits by row, parameters by request.
struct Side {
    const void* logits;  // null: none
    uint64_t row_stride;
    const float *temperature, *top_p, *min_p;
    const int32_t* top_k;
    Kept* kept;  // [rows]
    uint32_t type;
};

// A row that keeps all its tokens, or (temperature 0) the first one alone, is
// not recorded: one pass over it says what there is to know.
__device__ __forceinline__ bool keeps_all(const Side& side, uint32_t request, uint32_t vocab) {
    // three loads at once
    const int32_t k = side.top_k ? __ldg(side.top_k + request) : 0;
    const float top_p = side.top_p ? __ldg(side.top_p + request) : 1.0f, min_p = side.min_p ? __ldg(side.min_p + request) : 0.0f;
    return !((k > 0) & (static_cast<uint32_t>(k) < vocab)) & !(top_p < 1.0f) & !(min_p > 0.0f);
}
__device__ __forceinline__ float temperature_of(const Side& side, uint32_t request) {
    return side.temperature ? __ldg(side.temperature + request) : 1.0f;
}
// 1 / T as afx_sample takes it
__device__ __forceinline__ float inverse_temperature(float t) {
    constexpr float kLeast = 3e-39f;  // 1 / T is finite from here on
    return t == INFINITY ? 1.17549435e-38f : 1.0f / fmaxf(t, kLeast);
}

// Records what the rows that a request's starts name keep, where they keep
// less than all: of the target's rows, and of the drafts' those that a draft comes from.
afx_status launch_records(const Side& target, const Side& draft, uint32_t rows, uint32_t vocab, const int32_t* starts, const int32_t* tokens,
                          uint32_t n_requests, cudaStream_t s);

// The draft that row t decides on, of a request whose rows end before `end`, or -1.
__device__ __forceinline__ int32_t draft_of(const int32_t* tokens, int32_t t, int32_t end, uint32_t vocab) {
    if (t + 1 >= end) return -1;
    const int32_t d = __ldg(tokens + t + 1);
    return d >= 0 && static_cast<uint32_t>(d) < vocab ? d : -1;
}

}  // namespace serve
}  // namespace afx
