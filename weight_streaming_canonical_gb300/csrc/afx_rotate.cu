// sm_103a rotary positions (afx_rotary_plan, afx_rotate, afx_rotate_write).
//
// Pair i of a head, (a, b), becomes (a cos - b sin, a sin + b cos) at the angle
// position * f_i.  An angle is held as a fraction of a turn: the plan has
// F_i = 2^64 f_i / 2 pi, whole turns left out, and position * F_i in 64-bit
// integers drops whole turns by itself, exactly, for negative positions too.
// Sine and cosine are those of its first 24 bits, by sincospif, turned on by
// the rest: right to float32's rounding, however far the position is and
// however near the angle is to where one of them is zero (a float32 product
// position * f_i is off by 2^-8 radians at position 131,072, an angle cut to
// float32 by up to 2^-25 of a half-turn).
//
// A CTA takes a few tokens: it works out their angles once (a pair a thread)
// into shared memory, and then all heads of these tokens use them, queries
// and keys alike.  A thread takes 8 pairs of a head, two runs of 8 elements
// that are 16-byte loads for 16-bit types; keys and values go to their slots
// in the cache in the same pass.
//
// Bound: HBM bandwidth; each element is read and written once.  32,701 tokens of
// 40 query and 8 key/value heads of 128, BF16: 139 us, 6.7 TB/s, as fast as a
// copy (185 us with one head's loads in flight a thread instead of four, 143 with eight
// tokens a CTA); 15,953 tokens of 28 and 4, FP16, three axes: 57 us,
// 5.2 TB/s; 64 tokens from float32: 2.8 us, less than a call takes the host.
#include <cmath>
#include <type_traits>

#include "afx_serving.cuh"

namespace afx {
namespace serve {

afx_status check_cache(const afx_kv_cache* c, uint32_t* shift);  // afx_kv.cu

namespace {

constexpr int kThreads = 256;
constexpr uint32_t kMostTokens = 4;  // of a CTA

struct Heads {  // one of queries, keys, values
    const uint8_t* src;
    uint8_t* dst;
    uint64_t src_token, src_head, dst_token, dst_head, dst_page;  // bytes
    uint32_t n;
};

struct RotateArgs {
    afx_rotary plan;
    Heads q, k, v;
    const int32_t* positions;
    uint64_t axis_stride;
    const int32_t* slots;  // null: no cache
    int32_t* status;
    uint32_t n_tokens, tokens;  // tokens: of a CTA
    uint32_t shift, n_slots;
};

template <typename T>
__device__ __forceinline__ float widen(T x);
template <>
__device__ __forceinline__ float widen<float>(float x) { return x; }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float widen<__half>(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }

// V elements as they lie in memory: loads of several go out before the first is widened.
template <typename T, int V>
struct Raw {
    uint4 w[V * sizeof(T) / 16];
    __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
        for (uint32_t i = 0; i < V * sizeof(T) / 16; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (uint32_t i = 0; i < V * sizeof(T) / 16; ++i) {
            const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    x[i * 4 + j] = __uint_as_float(u[j]);
                } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                    x[2 * j] = __uint_as_float(u[j] << 16), x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
                } else {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
                    x[2 * j] = f.x, x[2 * j + 1] = f.y;
                }
            }
        }
    }
};
template <typename T>
struct Raw<T, 1> {
    T v;
    __device__ __forceinline__ void load(const uint8_t* p) { v = *reinterpret_cast<const T*>(p); }
    __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = widen<T>(v); }
};
template <typename T, int V>
__device__ __forceinline__ void store_run(uint8_t* p, const float (&x)[V]) {
    if constexpr (V == 1) {
        *reinterpret_cast<T*>(p) = narrow<T>(x[0]);
    } else if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
                const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t*>(&h);
            }
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    }
}

// V pairs a thread: 8, or 1 where addresses, strides or sizes do not allow 16-byte accesses.
template <typename In, typename Out, int V>
__global__ void __launch_bounds__(kThreads, 4) rotate_kernel(const __grid_constant__ RotateArgs a) {
    __shared__ __align__(16) float turn[kMostTokens][2][AFX_ROTARY_MAX_PAIRS];  // cosines, sines
    __shared__ int32_t slot_of[kMostTokens];  // negative: padding
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_earlier();
    let_next_start();
    const uint32_t t0 = blockIdx.x * a.tokens, n = min(a.tokens, a.n_tokens - t0);
    const uint32_t half = a.plan.rotary_dim / 2;
    {
        if (threadIdx.x < n) {
            const int32_t slot = a.slots ? __ldg(a.slots + t0 + threadIdx.x) : 0;
            if (slot >= 0 && a.slots && static_cast<uint32_t>(slot) >= a.n_slots) raise(a.status, AFX_DEV_BAD_PAGE);
            slot_of[threadIdx.x] = slot;
        }
        // 8 pairs of 4 tokens a warp: the plan's values are read by all lanes alike (reads of the parameters at
        // addresses of each lane's own take turns) and each lane keeps its pair's
        for (uint32_t u = warp; u < ceil_div(half, 8) * ceil_div(n, 4); u += kThreads / 32) {
            const uint32_t c = u % ceil_div(half, 8) * 8, t = u / ceil_div(half, 8) * 4 + lane / 8;
            uint64_t step = 0;
            uint32_t axis = 0;
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
                const uint64_t s = a.plan.step[c + j];
                const uint32_t x = a.plan.axis[c + j];
                if (lane % 8 == j) step = s, axis = x;
            }
            const uint32_t i = c + lane % 8;
            if (t < n && i < half) {
                const int32_t pos = __ldg(a.positions + axis * a.axis_stride + t0 + t);
                // half-turns: the nearest multiple of 2^-23, which is a float32 (past 1 it goes on at -1, the same angle), and
                // what is left, at most 2^-24 (32-bit conversions alone: 64-bit ones made frames of a video 2 % slower)
                const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
                const uint32_t high = static_cast<uint32_t>(turns >> 32), near = (high + 128u) & ~255u;
                const float left = fmaf(__uint2float_rn(static_cast<uint32_t>(turns)), 0x1p-32f, __int2float_rn(static_cast<int32_t>(high - near))) *
                                   (0x1p-31f * 3.14159265f);
                float s, co;
                sincospif(__int2float_rn(static_cast<int32_t>(near)) * 0x1p-31f, &s, &co);
                turn[t][0][i] = fmaf(-left, s, co) * a.plan.amplitude;
                turn[t][1][i] = fmaf(left, co, s) * a.plan.amplitude;
            }
        }
    }
    __syncthreads();
    // a thread's place within a head stays, its heads go on by `rows`
    const uint32_t places = a.plan.head_dim / (2 * V), turned = half / V;
    const uint32_t place = threadIdx.x % places, rows = kThreads / places;
    if (threadIdx.x / places >= rows) return;
    const bool apart = a.plan.pairs == AFX_ROTARY_HALVES && place < turned;
    const uint32_t e0 = apart ? place * V : 2 * place * V, e1 = apart ? half + place * V : e0 + V;
    const uint32_t heads = a.q.n + a.k.n + a.v.n;
    constexpr int kAtOnce = V == 8 && sizeof(In) == 4 ? 2 : 4;
    uint32_t t = 0, h = threadIdx.x / places;
    while (t < n) {
        Raw<In, V> raw[kAtOnce][2];
        uint8_t* to[kAtOnce];
        uint32_t of[kAtOnce];  // its token; the highest bit: not turned
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            while (h >= heads && t < n) h -= heads, ++t;
            to[j] = nullptr;
            of[j] = t;
            if (t < n) {
                const bool is_q = h < a.q.n, is_v = h >= a.q.n + a.k.n;
                const Heads& s = is_q ? a.q : is_v ? a.v : a.k;
                const uint32_t in = is_q ? h : is_v ? h - a.q.n - a.k.n : h - a.q.n;
                const int32_t slot = slot_of[t];
                const uint64_t dst = is_q ? static_cast<uint64_t>(t0 + t) * s.dst_token
                                          : (static_cast<uint32_t>(slot) >> a.shift) * s.dst_page +
                                                (static_cast<uint32_t>(slot) & ((1u << a.shift) - 1)) * s.dst_token;
                if (slot >= 0 && (is_q || static_cast<uint32_t>(slot) < a.n_slots)) {
                    const uint8_t* from = s.src + static_cast<uint64_t>(t0 + t) * s.src_token + in * s.src_head;
                    raw[j][0].load(from + e0 * sizeof(In));
                    raw[j][1].load(from + e1 * sizeof(In));
                    to[j] = s.dst + dst + in * s.dst_head;
                    if (place >= turned || is_v) of[j] |= 0x80000000u;
                }
            }
            h += rows;
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (!to[j]) continue;
            float x[2][V];
            raw[j][0].get(x[0]);
            raw[j][1].get(x[1]);
            if (!(of[j] >> 31)) {
                const float* c = &turn[of[j]][0][place * V];
                const float* s = &turn[of[j]][1][place * V];
                float y[2][V];
                if (apart) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        y[0][i] = x[0][i] * c[i] - x[1][i] * s[i];
                        y[1][i] = x[0][i] * s[i] + x[1][i] * c[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {  // elements 2 i and 2 i + 1 of the 2 V
                        const float p = x[2 * i / V][2 * i % V], q = x[(2 * i + 1) / V][(2 * i + 1) % V];
                        y[2 * i / V][2 * i % V] = p * c[i] - q * s[i];
                        y[(2 * i + 1) / V][(2 * i + 1) % V] = p * s[i] + q * c[i];
                    }
                }
                store_run<Out, V>(to[j] + e0 * sizeof(Out), y[0]);
                store_run<Out, V>(to[j] + e1 * sizeof(Out), y[1]);
            } else {
                store_run<Out, V>(to[j] + e0 * sizeof(Out), x[0]);
                store_run<Out, V>(to[j] + e1 * sizeof(Out), x[1]);
            }
        }
    }
}

uint32_t type_size(uint32_t type) { return type == AFX_TYPE_F32 ? 4 : 2; }

template <typename In, typename Out>
afx_status launch(const RotateArgs& a, bool wide, uint32_t grid, cudaStream_t s) {
    AFX_SERVE_TRY(wide ? launch_early(rotate_kernel<In, Out, 8>, grid, kThreads, 0, s, a)
                       : launch_early(rotate_kernel<In, Out, 1>, grid, kThreads, 0, s, a),
                  "rotate_kernel launch");
    return AFX_OK;
}
template <typename In>
afx_status launch_out(const RotateArgs& a, uint32_t out, bool wide, uint32_t grid, cudaStream_t s) {
    if (out == AFX_TYPE_BF16) return launch<In, __nv_bfloat16>(a, wide, grid, s);
    if (out == AFX_TYPE_FP16) return launch<In, __half>(a, wide, grid, s);
    return launch<In, float>(a, wide, grid, s);
}

// Common to both calls: heads' sources and destinations are set.
afx_status run(RotateArgs& a, uint32_t in, uint32_t out, cudaStream_t stream) {
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    bool wide = a.plan.rotary_dim % 16 == 0 && a.plan.head_dim % 16 == 0;
    for (const Heads* h : {&a.q, &a.k, &a.v}) {
        if (h->n == 0) continue;
        const bool cached = h != &a.q;
        const uint64_t bits = reinterpret_cast<uintptr_t>(h->src) | reinterpret_cast<uintptr_t>(h->dst) | (a.n_tokens > 1 ? h->src_token : 0) |
                              (h->n > 1 ? h->src_head | h->dst_head : 0) | (a.n_tokens > 1 && !cached ? h->dst_token : 0);
        if (bits & 15u) wide = false;  // cache strides are multiples of 16 bytes
    }
    // as many tokens a CTA as share their angles' work, one where that would leave SMs idle
    a.tokens = a.n_tokens >= 16u * static_cast<uint32_t>(sms) ? kMostTokens : 1;
    const uint32_t grid = ceil_div(a.n_tokens, a.tokens);
    if (in == AFX_TYPE_BF16) return launch_out<__nv_bfloat16>(a, out, wide, grid, stream);
    if (in == AFX_TYPE_FP16) return launch_out<__half>(a, out, wide, grid, stream);
    return launch_out<float>(a, out, wide, grid, stream);
}

afx_status check_plan(const afx_rotary* r) {
    if (!r) return afx_fail(AFX_E_ARG, "null rotation plan", 0);
    if (r->head_dim == 0 || r->head_dim > 2 * AFX_ROTARY_MAX_PAIRS || r->head_dim % 2 || r->rotary_dim == 0 || r->rotary_dim % 2 ||
        r->rotary_dim > r->head_dim || r->pairs > AFX_ROTARY_NEIGHBOURS || r->n_axes == 0 || r->n_axes > AFX_ROTARY_MAX_AXES)
        return afx_fail(AFX_E_ARG, "not a plan of afx_rotary_plan", 0);
    for (uint32_t i = 0; i < r->rotary_dim / 2; ++i)
        if (r->axis[i] >= r->n_axes) return afx_fail(AFX_E_ARG, "not a plan of afx_rotary_plan", 0);
    return AFX_OK;
}

}  // namespace
}  // namespace serve
}  // namespace afx

using namespace afx::serve;

extern "C" afx_status afx_rotary_plan(uint32_t head_dim, uint32_t rotary_dim, uint32_t pairs, double base,
                                      const double* frequencies, uint32_t n_axes, const uint8_t* axis_of_pair, float amplitude,
                                      afx_rotary* out) {
    if (!out) return afx_fail(AFX_E_ARG, "null rotation plan", 0);
    if (head_dim == 0 || head_dim % 2 || head_dim > 2 * AFX_ROTARY_MAX_PAIRS)
        return afx_fail(AFX_E_ARG, "heads have 2 to 256 elements, an even number", 0);
    if (rotary_dim == 0 || rotary_dim % 2 || rotary_dim > head_dim)
        return afx_fail(AFX_E_ARG, "rotary_dim is even, from 2 to head_dim", 0);
    if (pairs != AFX_ROTARY_HALVES && pairs != AFX_ROTARY_NEIGHBOURS) return afx_fail(AFX_E_ARG, "unknown pairs", 0);
    if (n_axes == 0 || n_axes > AFX_ROTARY_MAX_AXES) return afx_fail(AFX_E_ARG, "1 to 8 axes", 0);
    if (!frequencies && !(base > 0.0 && std::isfinite(base))) return afx_fail(AFX_E_ARG, "the base must be above 0", 0);
    if (!std::isfinite(amplitude)) return afx_fail(AFX_E_ARG, "the amplitude must be finite", 0);
    afx_rotary r{};
    r.head_dim = head_dim;
    r.rotary_dim = rotary_dim;
    r.n_axes = n_axes;
    r.pairs = pairs;
    r.amplitude = amplitude;
    for (uint32_t i = 0; i < rotary_dim / 2; ++i) {
        const double f = frequencies ? frequencies[i] : std::pow(base, -2.0 * i / rotary_dim);
        if (!std::isfinite(f)) return afx_fail(AFX_E_ARG, "frequencies must be finite", 0);
        constexpr double kTwoPi = 6.283185307179586476925286766559;
        // Two roundings of a double, the quotient and kTwoPi: within 2^-52 of the frequency.  Below 1 turn by fmod,
        // which is exact; from 2^-1 on as 2^63 steps, so that the conversion stays in range
        const double turns = std::fmod(f / kTwoPi, 1.0), size = std::fabs(turns);
        const uint64_t step = static_cast<uint64_t>(size * 0x1p63) * 2;
        r.step[i] = turns < 0.0 ? 0 - step : step;
        r.axis[i] = axis_of_pair ? axis_of_pair[i] : 0;
        if (r.axis[i] >= n_axes) return afx_fail(AFX_E_ARG, "axis_of_pair names an axis that is not there", 0);
    }
    *out = r;
    return AFX_OK;
}

extern "C" afx_status afx_rotate(const afx_rotary* rotary, const int32_t* positions_dev, uint64_t axis_stride, uint32_t n_tokens,
                                 const void* x_dev, uint32_t x_type, uint64_t x_token_stride, uint64_t x_head_stride,
                                 uint32_t heads, void* y_dev, uint32_t y_type, uint64_t y_token_stride, uint64_t y_head_stride,
                                 afx_stream_t stream) {
    const afx_status st = check_plan(rotary);
    if (st != AFX_OK) return st;
    if (x_type > AFX_TYPE_F32 || y_type > AFX_TYPE_F32) return afx_fail(AFX_E_ARG, "unknown type", 0);
    if (heads > 65536) return afx_fail(AFX_E_ARG, "up to 65536 heads", 0);
    if (n_tokens > INT32_MAX) return afx_fail(AFX_E_ARG, "too many tokens", 0);
    if (n_tokens == 0 || heads == 0) return AFX_OK;
    if ((heads > 1 && y_head_stride < rotary->head_dim) || (n_tokens > 1 && y_token_stride < rotary->head_dim))
        return afx_fail(AFX_E_ARG, "rows of the result must not overlap", 0);
    if (x_dev == y_dev && (x_type != y_type || (n_tokens > 1 && x_token_stride != y_token_stride) || (heads > 1 && x_head_stride != y_head_stride)))
        return afx_fail(AFX_E_ARG, "in place, types and strides are the same", 0);
    if (!device_ptr_here(positions_dev, 4) || !device_ptr_here(x_dev, type_size(x_type)) || !device_ptr_here(y_dev, type_size(y_type)))
        return afx_fail(AFX_E_ARG, "the arrays must be memory of the current device", 0);
    RotateArgs a{};
    a.plan = *rotary;
    a.positions = positions_dev;
    a.axis_stride = axis_stride;
    a.n_tokens = n_tokens;
    a.q = Heads{static_cast<const uint8_t*>(x_dev), static_cast<uint8_t*>(y_dev), x_token_stride * type_size(x_type),
                x_head_stride * type_size(x_type), y_token_stride * type_size(y_type), y_head_stride * type_size(y_type), 0, heads};
    return run(a, x_type, y_type, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" afx_status afx_rotate_write(const afx_rotary* rotary, const int32_t* positions_dev, uint64_t axis_stride, const afx_qkv* in,
                                       void* q_out_dev, uint64_t q_out_token_stride, uint64_t q_out_head_stride,
                                       const afx_kv_cache* cache, const int32_t* slots_dev, afx_stream_t stream,
                                       int32_t* status_dev) {
    RotateArgs a{};
    afx_status st = check_plan(rotary);
    if (st == AFX_OK) st = check_cache(cache, &a.shift);
    if (st != AFX_OK) return st;
    if (!in || in->type > AFX_TYPE_F32) return afx_fail(AFX_E_ARG, "unknown type", 0);
    if (rotary->head_dim != cache->head_dim) return afx_fail(AFX_E_ARG, "the plan is for heads of another size than the cache's", 0);
    if (in->q_heads > 65536) return afx_fail(AFX_E_ARG, "up to 65536 heads", 0);
    if (in->n_tokens > INT32_MAX) return afx_fail(AFX_E_ARG, "too many tokens", 0);
    if (in->n_tokens == 0) return AFX_OK;
    const uint32_t dim = cache->head_dim, size = type_size(in->type), out = cache->format == AFX_FMT_BF16 ? AFX_TYPE_BF16 : AFX_TYPE_FP16;
    if (in->q_heads) {
        if ((in->q_heads > 1 && q_out_head_stride < dim) || (in->n_tokens > 1 && q_out_token_stride < dim))
            return afx_fail(AFX_E_ARG, "rows of the queries' result must not overlap", 0);
        if (in->q_dev == q_out_dev && (in->type != out || (in->n_tokens > 1 && in->q_token_stride != q_out_token_stride) ||
                                       (in->q_heads > 1 && in->q_head_stride != q_out_head_stride)))
            return afx_fail(AFX_E_ARG, "in place, types and strides are the same", 0);
        if (!device_ptr_here(in->q_dev, size) || !device_ptr_here(q_out_dev, 2)) return afx_fail(AFX_E_ARG, "the queries must be memory of the current device", 0);
    }
    if (!device_ptr_here(positions_dev, 4) || !device_ptr_here(in->k_dev, size) || !device_ptr_here(in->v_dev, size) || !device_ptr_here(slots_dev, 4) ||
        !device_ptr_here(cache->k_dev, 16) || !device_ptr_here(cache->v_dev, 16) || (status_dev && !device_ptr_here(status_dev, 4)))
        return afx_fail(AFX_E_ARG, "positions, keys, values, slots and the cache must be memory of the current device", 0);
    a.plan = *rotary;
    a.positions = positions_dev;
    a.axis_stride = axis_stride;
    a.slots = slots_dev;
    a.status = status_dev;
    a.n_tokens = in->n_tokens;
    a.n_slots = cache->n_pages * cache->page_tokens;
    a.q = Heads{static_cast<const uint8_t*>(in->q_dev), static_cast<uint8_t*>(q_out_dev), in->q_token_stride * size, in->q_head_stride * size,
                2 * q_out_token_stride, 2 * q_out_head_stride, 0, in->q_heads};
    a.k = Heads{static_cast<const uint8_t*>(in->k_dev), static_cast<uint8_t*>(cache->k_dev), in->k_token_stride * size, in->k_head_stride * size,
                2 * cache->token_stride, 2 * cache->head_stride, 2 * cache->page_stride, cache->kv_heads};
    a.v = Heads{static_cast<const uint8_t*>(in->v_dev), static_cast<uint8_t*>(cache->v_dev), in->v_token_stride * size, in->v_head_stride * size,
                2 * cache->token_stride, 2 * cache->head_stride, 2 * cache->page_stride, cache->kv_heads};
    return run(a, in->type, out, reinterpret_cast<cudaStream_t>(stream));
}
