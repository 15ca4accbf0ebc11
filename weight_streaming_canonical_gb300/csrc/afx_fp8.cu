// sm_103a products of E4M3 weights with a scale for each block of 128
// (afx_fp8_quantize, afx_fp8_product).
//
// fp8_quantize_kernel: for each token and block of 128 columns the largest
// magnitude a, scale = max(a / 448, 2^-126), values E4M3(x / scale).  Half a
// warp a block, eight elements a lane, four blocks in flight; the eight warps of a
// CTA take eight tokens, whose scales share a sector.
// Bound: HBM bandwidth for float32 (8191 tokens of 17,408: 104 us, 6.9 TB/s); for 16 bits it is below that
// (4096 of 17,408, BF16: 46.6 us, 4.6 TB/s; a warp a block took 65), with issue slots half busy and DRAM 28 % at 4096 of 5120.
//
// fp8_product_kernel: y = x W^T in steps of 128 columns, the block of the
// scales.  A step of a tile is
//     D  = X_b W_b^T                    (tcgen05, E4M3, float32 in tensor memory)
//     y += D * (x_scale[token] * w_scale[row block])
// where y stays in registers: lane = token, so that a thread has one token's
// factors.  The tensor cores cannot apply these themselves (their scaled form
// takes powers of two for every 32 elements), so a step's sums are read back.
// Four buffers of them in tensor memory keep the products going while the sums
// of others are read.
//
// Two shapes.  A CTA's tile is 128 tokens by N rows of W (64 or 128); a pair
// of CTAs (cta_group::2) has a tile of 256 tokens by 2 N rows (N 96 or 128): each
// loads its own 128 tokens and half of the rows, 32 KB a step of 256 rows where CTAs on
// their own would load 64 at the 60 bytes a cycle that an SM gets from L2.  A
// pair's step is two products of N rows each, with buffers of their own.  Which
// shape a product gets goes by what steps of each were measured to take (Launch).
//
// Roles of a CTA's 12 warps: 0-7 the sums (a quarter of the lanes and half of
// the columns each; they take registers from the others), 8 and 9 issue the products
// (of a pair, the first CTA's), 10 loads by TMA (128-byte rows with the 128-byte
// swizzle; columns past the matrix are zeros) into a ring of steps, 11 multiplies the
// tokens' scales with the row blocks' into shared memory.
// Where tiles are fewer than SMs, a cluster of CTAs shares a tile: each
// takes a run of steps, and their sums are added through distributed shared memory in
// the order of the CTAs.
//
// Bound: for few tokens reading W (1 token by 17,408 rows of 5120: 16 us,
// 5.4 TB/s; 64 by 5120 of 17,408: 20 us, 4.5 TB/s; the rest is the start and
// the last steps' way to the sums); for many the sums: 4096 tokens by 17,408 of
// 5120 in 316 to 339 us by the clock, 2.2 to 2.3 PFLOP/s, 215 us without reading the sums back, 165 with
// the products alone.  A step of 128 x 256 takes 970 cycles, of which the products
// take 520, while its sums are on their way: the wait for the products, 400 cycles of
// loads from tensor memory and multiply-adds (two warps a quarter), the way back.
// Sixteen warps with half as many columns took 361 us (what a step takes besides its columns doubles), one
// product of 256 rows with two buffers 349, a loop that waits for its barriers one
// by one 355.  Waits and arrivals stay within the CTA's scope: acquire and release for
// the whole cluster doubled the time of every step.
//
// Every wait is bounded: one that runs out raises AFX_DEV_TIMEOUT and a flag
// that all roles poll; copies and products in flight are waited for and the
// CTA frees its tensor memory and ends.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <cstdio>
#include <type_traits>

#include "afx_known.h"
#include "afx_ring.h"
#include "afx_tensor.cuh"

namespace cg = cooperative_groups;

namespace afx {
namespace serve {
namespace {

constexpr uint32_t kBlock = AFX_FP8_BLOCK;

// ---- rounding activations ----------------------------------------------------------

constexpr int kQuantThreads = 256;
constexpr uint32_t kQuantAtOnce = 2;  // pairs of blocks in flight a warp

struct QuantArgs {
    const void* x;
    uint8_t* q;
    float* scales;
    uint64_t x_stride, q_stride, scale_stride;
    uint32_t n_tokens, cols, blocks, per_cta;  // per_cta: blocks that a CTA does of its eight tokens
};

// x / scale, rounded to float32 as far as its rounding to E4M3 can tell.  With r the rounded reciprocal and q = x r, the quotient is
// q - r (q scale - x) (Markstein's correction) as long as q scale - x is exact, which tiny scales do not allow: those divide.
// q may be two last places off, one more than the theorem allows, so this rests on all cases that count: for each of the 2^23
// significands of a scale, each of the 16 of a border between two E4M3 values and the four float32 on either side
// of their product, the result was the divided one; so it was for all 2^23 significands over 448 (scale_of).
__device__ __forceinline__ void quotients(const float (&x)[8], float scale, float (&q)[8]) {
    if (scale < 0x1p-90f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x[i], scale);
        return;
    }
    const float r = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float near = x[i] * r;
        q[i] = fmaf(-r, fmaf(near, scale, -x[i]), near);  // this way round, what is left of -0 is +0, and -0 - r 0 is -0
    }
}

// max(a / 448, 2^-126) of a magnitude's bits, the quotient in the same way; NaN for NaN and infinity.
__device__ __forceinline__ float scale_of(uint32_t bits) {
    const float a = __uint_as_float(bits);
    if (bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    if (a < 0x1p-80f) return fmaxf(__fdiv_rn(a, 448.0f), 0x1p-126f);
    constexpr float r = 1.0f / 448.0f;
    const float near = a * r;
    return fmaf(r, fmaf(-near, 448.0f, a), near);
}

// Eight elements from i on, of a row's up to end (zeros past it), as they lie in memory.
template <typename T>
struct RawEight {
    uint32_t w[2 * sizeof(T)];
    __device__ __forceinline__ void load(const T* row, bool wide, uint32_t i, uint32_t end) {
        if (wide && i + 8 <= end) {
#pragma unroll
            for (uint32_t k = 0; k < sizeof(T) / 2; ++k) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + i) + k);
                w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (uint32_t c = 0; c < 8; ++c) w[c] = i + c < end ? __ldg(reinterpret_cast<const uint32_t*>(row + i + c)) : 0;
        } else {
            const uint16_t* r = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
            for (uint32_t c = 0; c < 8; c += 2)
                w[c / 2] = (i + c < end ? __ldg(r + i + c) : 0u) | (i + c + 1 < end ? __ldg(r + i + c + 1) : 0u) << 16;
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c) {
            if constexpr (sizeof(T) == 4) {
                x[c] = __uint_as_float(w[c]);
            } else if constexpr (std::is_same<T, __half>::value) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[c / 2]));
                x[c] = c % 2 ? f.y : f.x;
            } else {
                x[c] = __uint_as_float(c % 2 ? w[c / 2] & 0xFFFF0000u : w[c / 2] << 16);
            }
        }
    }
};

// Half a warp a block, eight elements a lane.  wide: runs of eight elements are aligned for 16-byte loads, of eight bytes
// for one store.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads, 6) fp8_quantize_kernel(const QuantArgs a, const bool wide) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, in = lane % 16 * 8;
    wait_for_earlier();
    let_next_start();
    const uint32_t t = blockIdx.x * (kQuantThreads / 32) + warp;
    if (t >= a.n_tokens) return;
    const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
    uint8_t* q = a.q + t * a.q_stride;
    const uint32_t b0 = blockIdx.y * a.per_cta, b1 = min(a.blocks, b0 + a.per_cta);
    for (uint32_t first = b0; first < b1; first += 2 * kQuantAtOnce) {
        RawEight<T> raw[kQuantAtOnce];
#pragma unroll
        for (uint32_t j = 0; j < kQuantAtOnce; ++j) {
            if (first + 2 * j >= b1) break;
            const uint32_t b = min(first + 2 * j + lane / 16, b1 - 1);  // a half without a block reads the other's
            raw[j].load(x, wide, b * kBlock + in, a.cols);
        }
#pragma unroll
        for (uint32_t j = 0; j < kQuantAtOnce; ++j) {
            const uint32_t b = first + 2 * j + lane / 16, c = b * kBlock + in;
            if (first + 2 * j >= b1) break;
            float v[8], q8[8];
            raw[j].get(v);
            uint32_t most = 0;  // of the magnitudes' bits, which NaN and infinity lead
#pragma unroll
            for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
            for (int d = 8; d; d >>= 1) most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
            const float scale = scale_of(most);
            quotients(v, scale, q8);
            uint32_t bytes[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)  // saturating: a quotient may be 448 and a rounding
                bytes[i] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q8[4 * i], q8[4 * i + 1]), __NV_SATFINITE, __NV_E4M3)) |
                           static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q8[4 * i + 2], q8[4 * i + 3]), __NV_SATFINITE, __NV_E4M3)) << 16;
            if (b >= b1) continue;
            if (wide && c + 8 <= a.cols) {
                *reinterpret_cast<uint2*>(q + c) = make_uint2(bytes[0], bytes[1]);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i)
                    if (c + i < a.cols) q[c + i] = static_cast<uint8_t>(bytes[i / 4] >> (8 * (i % 4)));
            }
            if (in == 0) a.scales[b * a.scale_stride + t] = scale;
        }
    }
}

// ---- the product -------------------------------------------------------------------

constexpr uint32_t kTokens = 128;   // of a CTA's tile
constexpr uint32_t kSumWarps = 8, kMmaWarp = 8, kLoadWarp = 10, kFactorWarp = 11;  // products: two warps
constexpr int kProductThreads = 384;
// registers a thread: as launched, then of the warps with the sums and of the
// others (what the ones add is what the others gave up)
constexpr int kRegsLaunch = 168, kRegsSums = 208, kRegsOther = 88;
static_assert(256 * kRegsSums + 128 * kRegsOther <= kProductThreads * kRegsLaunch, "register shares");
constexpr uint32_t kMostStages = 16;
constexpr uint32_t kSmemMost = 232448;  // 227 KB, what a CTA can have
constexpr uint32_t kMostSplit = 8;      // CTAs that share a tile
constexpr uint32_t kBufs = 4;           // buffers of sums in tensor memory

struct Ctl {
    uint64_t full[kMostStages], empty[kMostStages];
    uint64_t sums_full[kBufs], sums_empty[kBufs], factors_empty[kBufs], drain;
    uint32_t tmem;
    int32_t abort_flag;
    alignas(16) float factors[kBufs][2][kTokens];  // of a buffer's one or two row blocks
};
constexpr uint32_t kCtlBytes = 5120;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");
constexpr uint32_t kStageFloats = 32 * 33;  // of a warp, where y's rows are not whole sectors

struct ProductArgs {
    CUtensorMap x, w;
    const float *x_scales, *w_scales;
    uint8_t* y;
    int32_t* status;
    uint64_t x_scale_stride, y_stride;  // y_stride: elements
    uint32_t n_tokens, rows, blocks, row_blocks;
    uint32_t tiles_m, tiles, box, stages, split;
    uint32_t y_type, sectors;  // sectors: y's rows are whole sectors
};

__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, Ctl& ctl, int32_t* status) {
#pragma unroll 1
    for (uint32_t i = 0; i < kWaitPolls; ++i) {
        if (bar_try(b, parity)) return true;
        if ((i & 31u) == 31u && *reinterpret_cast<volatile int32_t*>(&ctl.abort_flag)) return false;
    }
    *reinterpret_cast<volatile int32_t*>(&ctl.abort_flag) = 1;
    raise(status, AFX_DEV_TIMEOUT);
    return false;
}

// Two barriers at once, tested side by side: a test takes some 180 cycles, also of a barrier that has been through for
// long.  All of the warp; once: the second one is not meant.
__device__ __forceinline__ bool bar_wait_both(uint64_t* b, uint32_t parity, uint64_t* c, uint32_t c_parity, bool once, Ctl& ctl, int32_t* status) {
    const bool first = bar_try(b, parity), second = once || bar_try(c, c_parity);
    if (__all_sync(0xFFFFFFFFu, first && second)) return true;
    return __all_sync(0xFFFFFFFFu, bar_wait(b, parity, ctl, status) && (once || bar_wait(c, c_parity, ctl, status)));
}

// A box of rows of bytes; of a pair, the bytes count at the first CTA's barrier.
template <bool kPair>
__device__ __forceinline__ void load_box(uint32_t lane, uint32_t dst, const CUtensorMap* map, uint32_t x, uint32_t y, uint32_t bar) {
    if constexpr (kPair)
        asm volatile(
            "{\n .reg .pred q;\n setp.ne.u32 q, %5, 0;\n"
            " @q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(lane)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred q;\n setp.ne.u32 q, %5, 0;\n"
            " @q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar), "r"(lane)
            : "memory");
}
// The same box into L2, which later writes of it reach.
__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, uint32_t x, uint32_t y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y) : "memory");
}

template <bool kPair>
__device__ __forceinline__ void mma_e4m3(uint32_t lane, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    if constexpr (kPair)
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
            " @q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lane)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
            " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lane)
            : "memory");
}
// An arrival at this barrier (of a pair: of both CTAs) once the products so far are done.
template <bool kPair>
__device__ __forceinline__ void commit_products(uint32_t lane, uint64_t* bar) {
    if constexpr (kPair)
        asm volatile(
            "{\n .reg .pred q;\n setp.ne.u32 q, %1, 0;\n"
            " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n}\n" ::"r"(smem_addr(bar)),
            "r"(lane), "h"(static_cast<uint16_t>(3))
            : "memory");
    else
        commit(lane, bar);
}

// Columns loaded from tensor memory may be used behind wait_columns: they are
// its operands, so that no use of them is moved before it.
__device__ __forceinline__ void load_columns(uint32_t addr, uint32_t (&v)[32]) { tmem_load32(addr, v); }
__device__ __forceinline__ void wait_columns(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void load_columns(uint32_t addr, uint32_t (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
                 : AFX_R8(v, 0), AFX_R8(v, 8)
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void wait_columns(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}

__device__ __forceinline__ uint32_t two_16(uint32_t type, float lo, float hi) {
    if (type == AFX_TYPE_BF16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&p);
    }
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void store_one(const ProductArgs& a, uint64_t at, float v) {
    if (a.y_type == AFX_TYPE_F32)
        reinterpret_cast<float*>(a.y)[at] = v;
    else
        reinterpret_cast<uint16_t*>(a.y)[at] = static_cast<uint16_t>(two_16(a.y_type, v, 0.0f));
}

// N: rows of W of one product: of a CTA's tile, or of half a pair's.
template <uint32_t N, bool kPair>
struct Tile {
    static constexpr uint32_t kRows = kPair ? 2 * N : N;         // of W
    static constexpr uint32_t kProducts = kPair ? 2 : 1;         // a step
    static constexpr uint32_t kColumns = kPair ? N : N / 2;      // of a sum warp
    static constexpr uint32_t kRuns = kColumns / 32;             // of them, in runs of 32
    static constexpr uint32_t kWidth = kRuns < 4 ? 32 : 16;      // of them, loaded at once; and how many loads the
    static constexpr uint32_t kLoads = kRuns < 4 ? 2 : 1;        // registers hold beside the sums
    static constexpr uint32_t kWBytes = N * kBlock;              // a CTA's part of a step's W
    static constexpr uint32_t kTmem = N * kBufs <= 256 ? 256 : 512;  // columns of tensor memory, a power of two
    static constexpr uint32_t kRowBlocks = N % kBlock && kBlock % N ? 2 : 1;  // that a product's rows are among
    static constexpr uint32_t kPartRow = kRows + 4;              // floats between tokens' sums in shared memory
    static constexpr uint32_t kArrivals = kPair ? kSumWarps / 2 : kSumWarps;  // that read a buffer, in one CTA
};

template <uint32_t N, bool kPair>
__global__ void __launch_bounds__(kProductThreads, 1) fp8_product_kernel(const __grid_constant__ ProductArgs a) {
    using T = Tile<N, kPair>;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
    uint8_t* w_ring = smem + kCtlBytes;
    uint8_t* x_ring = w_ring + a.stages * T::kWBytes;
    float* staging = reinterpret_cast<float*>(x_ring + a.stages * a.box * kBlock + (kTokens - a.box) * kBlock);  // where !sectors
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // CTAs of a cluster: a pair, or the `split` ones of a tile
    const uint32_t group = kPair ? 2 : a.split, rank = blockIdx.x % group;
    const uint32_t side = kPair ? rank : 0, part = kPair ? 0 : rank;
    // a group's tiles: one where several share it, else every gridDim.x / group-th; its steps of a tile
    const uint32_t step0 = static_cast<uint32_t>(static_cast<uint64_t>(a.blocks) * part / a.split),
                   step1 = static_cast<uint32_t>(static_cast<uint64_t>(a.blocks) * (part + 1) / a.split);
    const uint32_t first = blockIdx.x / group, stride = gridDim.x / group;
    auto tokens_of = [&](uint32_t tile) { return tile % a.tiles_m * (kPair ? 2 * kTokens : kTokens) + side * kTokens; };
    auto rows_of = [&](uint32_t tile) { return tile / a.tiles_m * T::kRows; };
    // this CTA's rows of a tile's product h
    auto w_row = [&](uint32_t r0, uint32_t h) { return r0 + h * N + side * (N / 2); };
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < a.stages; ++i) {
            bar_init(&ctl.full[i], 1);
            bar_init(&ctl.empty[i], T::kProducts);
        }
        for (uint32_t i = 0; i < kBufs; ++i) {
            bar_init(&ctl.sums_full[i], 2);  // the products and the factors
            bar_init(&ctl.sums_empty[i], kPair ? 2 * T::kArrivals : T::kArrivals);
            bar_init(&ctl.factors_empty[i], T::kArrivals);
        }
        bar_init(&ctl.drain, 2);
        ctl.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == kMmaWarp) {
        if constexpr (kPair) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(&ctl.tmem)), "r"(T::kTmem) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(&ctl.tmem)), "r"(T::kTmem) : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
        }
    }
    if (warp == kLoadWarp && first < a.tiles) {
        // the first steps' weights are on their way to L2 while the kernel before this one ends: where it writes
        // them, the copies below find what it wrote
        for (uint32_t i = lane; i < a.stages * T::kProducts; i += 32) {
            const uint32_t s = step0 + i / T::kProducts;
            if (s < step1) prefetch_box(&a.w, s * kBlock, w_row(rows_of(first), i % T::kProducts));
        }
    }
    fence_before();
    __syncthreads();
    if constexpr (kPair) cluster_sync();  // the barriers that the other CTA arrives at are there
    fence_after();
    const uint32_t tmem = ctl.tmem;
    wait_for_earlier();
    let_next_start();

    if (warp >= kSumWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsOther));
      if (warp == kLoadWarp) {
        const bool leader = elect();
        uint32_t it = 0, slot = 0, phase = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < a.tiles; tile += stride) {
            const uint32_t t0 = tokens_of(tile), r0 = rows_of(tile);
            for (uint32_t s = step0; s < step1; ++s, ++it) {
                if (it >= a.stages) {
                    ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.empty[slot], phase ^ 1u, ctl, a.status));
                    if (!ok) break;
                }
                const uint32_t bar = kPair ? peer_addr(smem_addr(&ctl.full[slot]), 0) : smem_addr(&ctl.full[slot]);
                if (leader && side == 0) bar_expect(&ctl.full[slot], (kPair ? 2 : 1) * (T::kWBytes + a.box * kBlock));
                __syncwarp();
                const uint32_t w = smem_addr(w_ring + slot * T::kWBytes);
                if constexpr (kPair) {
                    load_box<true>(leader, w, &a.w, s * kBlock, w_row(r0, 0), bar);
                    load_box<true>(leader, w + T::kWBytes / 2, &a.w, s * kBlock, w_row(r0, 1), bar);
                } else {
                    load_box<false>(leader, w, &a.w, s * kBlock, r0, bar);
                }
                load_box<kPair>(leader, smem_addr(x_ring + slot * a.box * kBlock), &a.x, s * kBlock, t0, bar);
                if (++slot == a.stages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok && side == 0)  // copies in flight write shared memory
            for (uint32_t q = it > a.stages ? it - a.stages : 0; q < it; ++q)
                if (!bar_drain(&ctl.full[q % a.stages], q / a.stages & 1u)) raise(a.status, AFX_DEV_UNDRAINED);
      } else if (warp < kLoadWarp) {
        // of a pair's step a product each, else every second step, whose slots are this warp's own (ring_stages): waiting
        // and issuing take one warp longer than the products
        const uint32_t m = warp - kMmaWarp;
        if (side == 0) {
            // float32 sums of E4M3 by E4M3, both with their columns contiguous
            constexpr uint32_t kInstruction = 1u << 4 | (N >> 3) << 17 | ((kPair ? 2 : 1) * kTokens >> 4) << 24;
            constexpr uint32_t kStride = kPair ? 1 : 2;  // steps
            const bool leader = elect();
            const uint64_t x_desc = operand(smem_addr(x_ring), 16), w_desc = operand(smem_addr(w_ring) + (kPair ? m * (T::kWBytes / 2) : 0), 16);
            const uint32_t own = (step1 - step0) * ((a.tiles - first + stride - 1) / stride);  // steps of this CTA's tiles
            uint32_t slot = kPair ? 0 : m % a.stages, phase = kPair ? 0 : m / a.stages & 1u;
            for (uint32_t it = kPair ? 0 : m; it < own; it += kStride) {
                const uint32_t unit = kPair ? 2 * it + m : it, buf = unit % kBufs;
                if (!bar_wait_both(&ctl.full[slot], phase, &ctl.sums_empty[buf], (unit / kBufs - 1) & 1u, unit < kBufs, ctl, a.status)) break;
                fence_after();
                const uint64_t xd = x_desc + slot * (a.box * kBlock >> 4), wd = w_desc + slot * (T::kWBytes >> 4);
#pragma unroll
                for (uint32_t k = 0; k < kBlock / 32; ++k)
                    mma_e4m3<kPair>(leader, tmem + buf * N, xd + k * 2, wd + k * 2, kInstruction, k != 0);
                commit_products<kPair>(leader, &ctl.empty[slot]);
                commit_products<kPair>(leader, &ctl.sums_full[buf]);
                slot += kStride;
                if (slot >= a.stages) {
                    slot -= a.stages;
                    phase ^= 1u;
                }
            }
            commit_products<kPair>(leader, &ctl.drain);  // arrivals above land before a CTA ends
        }
        if (!bar_drain(&ctl.drain, 0)) raise(a.status, AFX_DEV_UNDRAINED);
      } else if (warp == kFactorWarp) {
        // four tokens a lane, their scales loaded four steps at a time while the four before are used (a register that
        // is handed on each step waits for its load each step); the row blocks' for 32 steps, a lane a step
        constexpr uint32_t kScales = T::kProducts * T::kRowBlocks, kAhead = 4;
        uint32_t it = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < a.tiles; tile += stride) {
            const uint32_t t0 = tokens_of(tile), r0 = rows_of(tile);
            float x[kAhead][4], x_next[kAhead][4], w[kScales], w_next[kScales];
            auto x_scales = [&](uint32_t s) {
#pragma unroll
                for (uint32_t j = 0; j < kAhead; ++j)
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        const uint32_t t = t0 + lane + 32 * i;
                        x_next[j][i] = t < a.n_tokens && s + j < step1 ? __ldg(a.x_scales + (s + j) * a.x_scale_stride + t) : 0.0f;
                    }
            };
            auto w_scales = [&](uint32_t s) {
#pragma unroll
                for (uint32_t i = 0; i < kScales; ++i) {
                    const uint32_t rb = min((r0 + i / T::kRowBlocks * N) / kBlock + i % T::kRowBlocks, a.row_blocks - 1);
                    w_next[i] = s + lane < step1 ? __ldg(a.w_scales + static_cast<uint64_t>(rb) * a.blocks + s + lane) : 0.0f;
                }
            };
            x_scales(step0);
            w_scales(step0);
            for (uint32_t s0 = step0; ok && s0 < step1; s0 += kAhead) {
                const uint32_t in32 = (s0 - step0) & 31u;
                if (in32 == 0) {
#pragma unroll
                    for (uint32_t i = 0; i < kScales; ++i) w[i] = w_next[i];
                    w_scales(s0 + 32);
                }
#pragma unroll
                for (uint32_t j = 0; j < kAhead; ++j)
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) x[j][i] = x_next[j][i];
                x_scales(s0 + kAhead);
#pragma unroll
                for (uint32_t j = 0; j < kAhead; ++j) {
                    if (s0 + j >= step1) break;
#pragma unroll
                    for (uint32_t h = 0; h < T::kProducts; ++h, ++it) {
                        const uint32_t buf = it % kBufs;
                        if (h == 0 && it >= kBufs) {
                            const uint32_t parity = (it / kBufs - 1) & 1u;
                            ok = bar_wait_both(&ctl.factors_empty[buf], parity, &ctl.factors_empty[(buf + 1) % kBufs], parity, !kPair, ctl, a.status);
                            if (!ok) break;
                        }
#pragma unroll
                        for (uint32_t i = 0; i < T::kRowBlocks; ++i) {
                            const float f = __shfl_sync(0xFFFFFFFFu, w[h * T::kRowBlocks + i], in32 + j);
#pragma unroll
                            for (uint32_t c = 0; c < 4; ++c) ctl.factors[buf][i][lane + 32 * c] = x[j][c] * f;
                        }
                        __syncwarp();
                        if (lane == 0) bar_arrive(&ctl.sums_full[buf]);
                    }
                    if (!ok) break;
                }
            }
        }
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsSums));
        // a CTA alone: half of the columns; a pair: one of a step's two products
        const uint32_t lanes = warp % 4 * 32, half = warp / 4;
        const uint32_t column0 = kPair ? 0 : half * T::kColumns;  // in a buffer
        const uint32_t row_in_tile = half * T::kColumns;          // the same of W, in a pair's tile too
        uint32_t it = 0;
        bool ok = true, ready = false;
        for (uint32_t tile = first; ok && tile < a.tiles; tile += stride) {
            const uint32_t t0 = tokens_of(tile), r0 = rows_of(tile) + row_in_tile;
            const uint32_t token = t0 + lanes + lane;
            const bool any = t0 + lanes < a.n_tokens, real = token < a.n_tokens;
            const uint32_t rb0 = kPair ? r0 / kBlock : 0;
            uint64_t sum[T::kRuns][16];
#pragma unroll
            for (uint32_t r = 0; r < T::kRuns; ++r)
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[r][i] = 0;
            for (uint32_t s = step0; s < step1; ++s, ++it) {
                const uint32_t unit = kPair ? 2 * it + half : it, buf = unit % kBufs;
                if (!__all_sync(0xFFFFFFFFu, ready)) ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.sums_full[buf], unit / kBufs & 1u, ctl, a.status));
                if (!ok) break;
                fence_after();
                // the next one's barrier, tested while this one is worked on
                const uint32_t next_unit = unit + (kPair ? 2 : 1);
                ready = bar_try_now(&ctl.sums_full[next_unit % kBufs], next_unit / kBufs & 1u);
                const uint32_t empty = kPair ? peer_addr(smem_addr(&ctl.sums_empty[buf]), 0) : smem_addr(&ctl.sums_empty[buf]);
                auto release = [&] {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive_cluster(empty);
                        bar_arrive(&ctl.factors_empty[buf]);
                    }
                };
                if (any) {
                    const uint32_t from = tmem + (lanes << 16) + buf * N + column0;
                    const float f0 = ctl.factors[buf][0][lanes + lane], f1 = T::kRowBlocks > 1 ? ctl.factors[buf][1][lanes + lane] : f0;
                    // loads are under way while the columns before are added, where the registers hold both
                    constexpr uint32_t kWidth = T::kWidth, kPieces = T::kColumns / kWidth;
                    uint32_t v[T::kLoads][kWidth];
                    if (T::kLoads > 1) {
                        load_columns(from, v[0]);
                        wait_columns(v[0]);
                    }
#pragma unroll
                    for (uint32_t q = 0; q < kPieces; ++q) {
                        const uint32_t next = q + T::kLoads - 1;
                        if (next < kPieces) {
                            load_columns(from + next * kWidth, v[next % T::kLoads]);
                            if (T::kLoads == 1) wait_columns(v[0]);
                        }
                        if (q + 1 == kPieces) release();  // all have been read
                        const float f = T::kRowBlocks == 1 || (r0 + q * kWidth) / kBlock == rb0 ? f0 : f1;
                        const uint64_t ff = pack2(f, f);
#pragma unroll
                        for (uint32_t i = 0; i < kWidth / 2; ++i) {
                            uint64_t& to = sum[q * kWidth / 32][q * kWidth % 32 / 2 + i];
                            to = fma2(pack2(__uint_as_float(v[q % T::kLoads][2 * i]), __uint_as_float(v[q % T::kLoads][2 * i + 1])), ff, to);
                        }
                        if (T::kLoads > 1 && next < kPieces) wait_columns(v[next % T::kLoads]);
                    }
                } else {
                    release();
                }
            }
            if (!ok) break;
            if (!kPair && a.split > 1) {  // into shared memory, whose copies and products are all done with
                if (real) {
                    float* to = reinterpret_cast<float*>(w_ring) + (lanes + lane) * T::kPartRow + row_in_tile;
#pragma unroll
                    for (uint32_t r = 0; r < T::kRuns; ++r)
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float4 f;
                            unpack2(sum[r][i], &f.x, &f.y);
                            unpack2(sum[r][i + 1], &f.z, &f.w);
                            *reinterpret_cast<float4*>(to + r * 32 + i * 2) = f;
                        }
                }
            } else if (any) {
                const uint64_t at = static_cast<uint64_t>(token) * a.y_stride + r0;
#pragma unroll
                for (uint32_t r = 0; r < T::kRuns; ++r) {
                    const uint32_t row = r0 + r * 32;
                    if (row >= a.rows) continue;
                    if (a.sectors && row + 32 <= a.rows) {
                        if (!real) continue;
                        if (a.y_type == AFX_TYPE_F32) {
                            float* to = reinterpret_cast<float*>(a.y) + at + r * 32;
#pragma unroll
                            for (int i = 0; i < 16; i += 4) store_sector(to + 2 * i, reinterpret_cast<const uint32_t*>(&sum[r][i]));
                        } else {
                            uint16_t* to = reinterpret_cast<uint16_t*>(a.y) + at + r * 32;
#pragma unroll
                            for (int i = 0; i < 16; i += 8) {
                                uint32_t p[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    float lo, hi;
                                    unpack2(sum[r][i + j], &lo, &hi);
                                    p[j] = two_16(a.y_type, lo, hi);
                                }
                                store_sector(to + 2 * i, p);
                            }
                        }
                        continue;
                    }
                    // a token's 32 rows by 32 lanes, through shared memory
                    float* stage = staging + warp * kStageFloats;
#pragma unroll
                    for (int i = 0; i < 16; ++i) unpack2(sum[r][i], &stage[lane * 33 + 2 * i], &stage[lane * 33 + 2 * i + 1]);
                    __syncwarp();
                    const uint32_t here = min(32u, a.n_tokens - (t0 + lanes));
                    if (row + lane < a.rows)
                        for (uint32_t t = 0; t < here; ++t)
                            store_one(a, static_cast<uint64_t>(t0 + lanes + t) * a.y_stride + row + lane, stage[t * 33 + lane]);
                    __syncwarp();
                }
            }
        }
    }

    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        if constexpr (kPair)
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(T::kTmem) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(T::kTmem) : "memory");
    }
    if (kPair || a.split > 1) cluster_sync();  // every CTA's sums are there, and no arrival is to come
    if (!kPair && a.split > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        const uint32_t t0 = tokens_of(first), r0 = rows_of(first);
        const uint32_t tokens = t0 < a.n_tokens ? min(kTokens, a.n_tokens - t0) : 0;
        const float* sums = reinterpret_cast<const float*>(w_ring);
        for (uint32_t e = (part * kProductThreads + threadIdx.x) * 4; e < tokens * T::kRows; e += a.split * kProductThreads * 4) {
            const uint32_t t = e / T::kRows, c = e % T::kRows;
            if (r0 + c >= a.rows) continue;
            float4 v[kMostSplit];
#pragma unroll
            for (uint32_t i = 0; i < kMostSplit; ++i)
                if (i < a.split) v[i] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sums + t * T::kPartRow + c, i));
            float4 sum = v[0];
#pragma unroll
            for (uint32_t i = 1; i < kMostSplit; ++i)
                if (i < a.split) sum.x += v[i].x, sum.y += v[i].y, sum.z += v[i].z, sum.w += v[i].w;
            const uint64_t at = static_cast<uint64_t>(t0 + t) * a.y_stride + r0 + c;
            const float of[4] = {sum.x, sum.y, sum.z, sum.w};
            if (a.sectors) {  // rows are a multiple of 32
                if (a.y_type == AFX_TYPE_F32)
                    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.y) + at) = sum;
                else
                    *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.y) + at) = make_uint2(two_16(a.y_type, of[0], of[1]), two_16(a.y_type, of[2], of[3]));
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    if (r0 + c + i < a.rows) store_one(a, at + i, of[i]);
            }
        }
        cluster_sync();  // no CTA ends while its sums are read
    }
}

// Rows of bytes: `rows` rows of `cols` bytes `stride` apart, boxes of 128 columns and `box` rows.
afx_status byte_map(CUtensorMap* map, const uint8_t* p, uint32_t rows, uint32_t cols, uint64_t stride, uint32_t box) {
    const EncodeFn enc = encode_fn();
    if (!enc) return afx_fail(AFX_E_CUDA, "cuTensorMapEncodeTiled is not available from the driver", 0);
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {rows > 1 ? stride : (cols + 15ull) / 16 * 16};  // one row may have any
    const cuuint32_t boxes[2] = {kBlock, box};
    const cuuint32_t steps[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char msg[96];
        snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
        return afx_fail(AFX_E_CUDA, msg, 0);
    }
    return AFX_OK;
}

constexpr uint32_t kStagingBytes = kSumWarps * kStageFloats * sizeof(float);

// How a product is cut: tiles for CTAs, `split` to each, or for pairs.
struct Cut {
    uint32_t n;  // rows of one product
    bool pair;
    uint32_t split;
};

template <uint32_t N, bool kPair>
struct Launch {
    using T = Tile<N, kPair>;

    // Clusters of this kernel that run at once on the current device; asked once a device.  0 where that cannot be told.
    static uint32_t at_once(uint32_t split, int sms) {
        constexpr int kDevices = 16;
        static Known known[kDevices][kMostSplit + 1];
        const uint32_t size = split * (kPair ? 2 : 1);
        if (size == 1) return sms;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return 0;
        auto ask = [&](uint64_t* clusters) {
            if (prepare() != AFX_OK) return false;
            cudaLaunchAttribute at[2];
            cudaLaunchConfig_t cfg = config(size, size, nullptr, at);
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, fp8_product_kernel<N, kPair>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                return false;
            }
            *clusters = static_cast<uint64_t>(n);
            return true;
        };
        uint64_t n = 0;
        const bool told = dev < kDevices ? known[dev][split].get(&n, ask) : ask(&n);
        return told ? static_cast<uint32_t>(n) : 0;
    }
    static cudaLaunchConfig_t config(uint32_t grid, uint32_t cluster, cudaStream_t s, cudaLaunchAttribute (&at)[2]) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(kProductThreads);
        cfg.dynamicSmemBytes = kSmemMost;
        cfg.stream = s;
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = cluster;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 2;
        return cfg;
    }
    static afx_status prepare() {
        // the warps with the sums wait for the registers that they ask for: they must be there
        static Known known;
        uint64_t regs = 0;
        cudaError_t err = cudaSuccess;
        const bool told = known.get(&regs, [&](uint64_t* v) {
            cudaFuncAttributes f{};
            if ((err = cudaFuncGetAttributes(&f, fp8_product_kernel<N, kPair>)) == cudaSuccess) *v = static_cast<uint64_t>(f.numRegs);
            return err == cudaSuccess;
        });
        if (!told) {
            cudaGetLastError();
            return afx_fail(AFX_E_CUDA, "cudaFuncGetAttributes", err);
        }
        if (regs < kRegsLaunch) return afx_fail(AFX_E_CUDA, "fp8_product_kernel was built with too few registers", 0);
        AFX_SERVE_TRY(cudaFuncSetAttribute(fp8_product_kernel<N, kPair>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemMost)),
                      "cudaFuncSetAttribute");
        return AFX_OK;
    }
    // In cycles: a step of a tile (measured with other tiles on all SMs: 400 whatever the rows for up to 64 tokens,
    // 430 and 500 for 64 and 128 rows by 128 tokens, 900 and 970 for pairs of 192 and 256), a wave's
    // start and end and the join of a tile's CTAs.  Pairs against CTAs, each held to by turns, back to back, after a fill of
    // 512 MB and with the rounding: 4096 tokens by 17,408 rows of 5120 331, 339 and 349 us, CTAs 335, 344 and 360; 300 by 17,408 of
    // 5120 50, 54 and 50, CTAs 37, 45 and 38; 501 by 7168 of 5120 25, 29 and 26, CTAs 27, 31 and 28; 1000 by 7168 of
    // 5120 44, 48 and 46, CTAs 38, 42 and 41.  It misses at times: 700 by 5120 of 17,408 gets pairs, 75, 78 and 84, CTAs
    // 73, 78 and 81; 4096 by 7168 of 5120 CTAs, 155, 164 and 158, pairs 136, 141 and 150.  1 by 5120 of 5120: three CTAs of 128
    // rows to a tile 9.1 us, two 9.9, one 11.7, tiles of 64 rows 11.0.
    static void consider(const ProductArgs& a, int sms, Cut* best, double* least) {
        const uint32_t tokens = (kPair ? 2 : 1) * kTokens, tiles_m = ceil_div(a.n_tokens, tokens);
        const uint64_t tiles = static_cast<uint64_t>(tiles_m) * ceil_div(a.rows, T::kRows);
        const double step = kPair ? (N == 96 ? 900.0 : 970.0) : a.n_tokens <= 64 ? 400.0 : N == 64 ? 430.0 : 500.0;
        for (uint32_t split = 1; split <= (kPair ? 1 : kMostSplit) && split <= a.blocks; ++split) {
            const uint32_t slots = at_once(split, sms);
            if (slots == 0 || (split > 1 && tiles > slots)) continue;
            const double waves = static_cast<double>((tiles + slots - 1) / slots);
            double cost = waves * (ceil_div(a.blocks, split) * step + 600.0) + (split > 1 ? 2000.0 + 100.0 * split : 0.0);
            // W from memory, at what all SMs get of it; the smaller of the two is hidden in part
            const double memory = static_cast<double>(a.rows) * a.blocks * kBlock / 3400.0 + 3000.0;
            cost = cost > memory ? cost + 0.3 * memory : memory + 0.3 * cost;
            if (cost < *least) *least = cost, *best = Cut{N, kPair, split};
        }
    }
    static afx_status go(ProductArgs& a, uint32_t split, const uint8_t* w, uint32_t cols, uint64_t w_stride, const uint8_t* x, uint64_t x_stride, int sms,
                         cudaStream_t s) {
        a.split = split;
        const uint32_t group = split * (kPair ? 2 : 1);
        a.tiles_m = ceil_div(a.n_tokens, (kPair ? 2 : 1) * kTokens);
        const uint64_t tiles = static_cast<uint64_t>(a.tiles_m) * ceil_div(a.rows, T::kRows);
        // a CTA counts its steps in 32 bits
        if (tiles > INT32_MAX / 16 || (tiles / sms + 1) * 2 * a.blocks > INT32_MAX) return afx_fail(AFX_E_ARG, "the product has too many tiles", 0);
        a.tiles = static_cast<uint32_t>(tiles);
        a.box = kPair || a.n_tokens >= kTokens ? kTokens : ceil_div(a.n_tokens, 8) * 8;
        const uint32_t fixed = 1024 + kCtlBytes + (kTokens - a.box) * kBlock + (a.sectors || split > 1 ? 0 : kStagingBytes);
        // a pair's warps each take every step, a CTA's every second one
        a.stages = ring_stages(kSmemMost - fixed, T::kWBytes + a.box * kBlock, kMostStages, kPair ? 1 : 2);
        // the sums of a CTA of several lie over the ring, which holds as many steps with fewer tokens
        static_assert(kTokens * T::kPartRow * sizeof(float) <= (kSmemMost - 1024 - kCtlBytes) / (T::kWBytes + kTokens * kBlock) * (T::kWBytes + kTokens * kBlock),
                      "sums fit the ring");
        afx_status st = prepare();
        if (st == AFX_OK) st = byte_map(&a.x, x, a.n_tokens, cols, x_stride, a.box);
        if (st == AFX_OK) st = byte_map(&a.w, w, a.rows, cols, w_stride, kPair ? N / 2 : N);
        if (st != AFX_OK) return st;
        const uint32_t slots = split > 1 ? a.tiles : at_once(1, sms);
        if (slots == 0) return afx_fail(AFX_E_CUDA, "no cluster of fp8_product_kernel fits this device", 0);
        cudaLaunchAttribute at[2] = {};
        const cudaLaunchConfig_t cfg = config((a.tiles < slots ? a.tiles : slots) * group, group, s, at);
        AFX_SERVE_TRY(cudaLaunchKernelEx(&cfg, fp8_product_kernel<N, kPair>, a), "fp8_product_kernel launch");
        return AFX_OK;
    }
};

}  // namespace
}  // namespace serve
}  // namespace afx

using namespace afx::serve;

extern "C" afx_status afx_fp8_quantize(const void* x_dev, uint32_t type, uint64_t x_stride, uint32_t n_tokens, uint32_t cols,
                                       uint8_t* q_dev, uint64_t q_stride, float* scales_dev, uint64_t scale_stride,
                                       afx_stream_t stream) {
    if (type > AFX_TYPE_F32) return afx_fail(AFX_E_ARG, "unknown type", 0);
    if (n_tokens >= 1u << 24 || cols >= 1u << 24) return afx_fail(AFX_E_ARG, "tokens and columns must be below 2^24", 0);
    if (n_tokens == 0 || cols == 0) return AFX_OK;
    if (n_tokens > 1 && (x_stride < cols || q_stride < cols)) return afx_fail(AFX_E_ARG, "rows lie at least cols apart", 0);
    if (cols > kBlock && scale_stride < n_tokens) return afx_fail(AFX_E_ARG, "blocks' scales lie at least n_tokens apart", 0);
    const uint32_t size = type == AFX_TYPE_F32 ? 4 : 2;
    if (!device_ptr_here(x_dev, size) || !device_ptr_here(q_dev, 1) || !device_ptr_here(scales_dev, 4))
        return afx_fail(AFX_E_ARG, "the arrays must be memory of the current device", 0);
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    QuantArgs a{};
    a.x = x_dev;
    a.q = q_dev;
    a.scales = scales_dev;
    a.x_stride = x_stride;
    a.q_stride = q_stride;
    a.scale_stride = scale_stride;
    a.n_tokens = n_tokens;
    a.cols = cols;
    a.blocks = ceil_div(cols, kBlock);
    const bool wide = !((reinterpret_cast<uintptr_t>(x_dev) | (n_tokens > 1 ? x_stride * size : 0)) & 15u) &&
                      !((reinterpret_cast<uintptr_t>(q_dev) | (n_tokens > 1 ? q_stride : 0)) & 7u);
    // Eight tokens a CTA; their blocks over as many CTAs as fill the SMs ten times over (8191 tokens of 17,408 with a warp a block:
    // 110 us, 132 with CTAs for one filling, 124 with 40), in fours where there are many
    const uint32_t groups = ceil_div(n_tokens, kQuantThreads / 32);
    uint32_t parts = ceil_div(static_cast<uint32_t>(sms) * 64, groups);
    a.per_cta = ceil_div(a.blocks, parts);
    a.per_cta = a.per_cta <= 2 ? 2 : ceil_div(a.per_cta, 2 * kQuantAtOnce) * 2 * kQuantAtOnce;
    parts = ceil_div(a.blocks, a.per_cta);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(groups, parts);
    cfg.blockDim = dim3(kQuantThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    AFX_SERVE_TRY(type == AFX_TYPE_F32    ? cudaLaunchKernelEx(&cfg, fp8_quantize_kernel<float>, a, wide)
                  : type == AFX_TYPE_BF16 ? cudaLaunchKernelEx(&cfg, fp8_quantize_kernel<__nv_bfloat16>, a, wide)
                                          : cudaLaunchKernelEx(&cfg, fp8_quantize_kernel<__half>, a, wide),
                  "fp8_quantize_kernel launch");
    return AFX_OK;
}

extern "C" afx_status afx_fp8_product(const uint8_t* w_dev, uint64_t w_stride, const float* w_scales_dev, uint32_t rows, uint32_t cols,
                                      const uint8_t* x_dev, uint64_t x_stride, const float* x_scales_dev, uint64_t x_scale_stride,
                                      uint32_t n_tokens, void* y_dev, uint32_t y_type, uint64_t y_stride, afx_stream_t stream,
                                      int32_t* status_dev) {
    if (y_type > AFX_TYPE_F32) return afx_fail(AFX_E_ARG, "unknown type", 0);
    if (n_tokens >= 1u << 24 || rows >= 1u << 24 || cols == 0 || cols >= 1u << 24)
        return afx_fail(AFX_E_ARG, "tokens, rows and columns must be below 2^24, columns above 0", 0);
    if (n_tokens == 0 || rows == 0) return AFX_OK;
    if ((rows > 1 && (w_stride < cols || w_stride % 16 || w_stride >> 32)) || (n_tokens > 1 && (x_stride < cols || x_stride % 16 || x_stride >> 32)))
        return afx_fail(AFX_E_ARG, "rows of weights and activations lie a multiple of 16 bytes apart, at least cols, below 2^32", 0);
    if (cols > kBlock && x_scale_stride < n_tokens) return afx_fail(AFX_E_ARG, "blocks' scales lie at least n_tokens apart", 0);
    if (n_tokens > 1 && y_stride < rows) return afx_fail(AFX_E_ARG, "rows of the result lie at least `rows` apart", 0);
    const uint32_t size = y_type == AFX_TYPE_F32 ? 4 : 2;
    if (!device_ptr_here(w_dev, 16) || !device_ptr_here(x_dev, 16)) return afx_fail(AFX_E_ARG, "weights and activations must be 16-byte aligned memory of the current device", 0);
    if (!device_ptr_here(w_scales_dev, 4) || !device_ptr_here(x_scales_dev, 4) || !device_ptr_here(y_dev, size) || (status_dev && !device_ptr_here(status_dev, 4)))
        return afx_fail(AFX_E_ARG, "the arrays must be memory of the current device", 0);
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    ProductArgs a;
    a.x_scales = x_scales_dev;
    a.w_scales = w_scales_dev;
    a.y = static_cast<uint8_t*>(y_dev);
    a.status = status_dev;
    a.x_scale_stride = x_scale_stride;
    a.y_stride = y_stride;
    a.n_tokens = n_tokens;
    a.rows = rows;
    a.blocks = ceil_div(cols, kBlock);
    a.row_blocks = ceil_div(rows, kBlock);
    a.y_type = y_type;
    a.sectors = rows % 32 == 0 && !((reinterpret_cast<uintptr_t>(y_dev) | (n_tokens > 1 ? y_stride * size : 0)) & 31u);
    Cut cut{128, false, 1};
    double least = 1e300;
    Launch<64, false>::consider(a, sms, &cut, &least);
    Launch<128, false>::consider(a, sms, &cut, &least);
    if (n_tokens > kTokens) {
        Launch<96, true>::consider(a, sms, &cut, &least);
        Launch<128, true>::consider(a, sms, &cut, &least);
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cut.pair) {
        if (cut.n == 96) return Launch<96, true>::go(a, cut.split, w_dev, cols, w_stride, x_dev, x_stride, sms, s);
        return Launch<128, true>::go(a, cut.split, w_dev, cols, w_stride, x_dev, x_stride, sms, s);
    }
    if (cut.n == 64) return Launch<64, false>::go(a, cut.split, w_dev, cols, w_stride, x_dev, x_stride, sms, s);
    return Launch<128, false>::go(a, cut.split, w_dev, cols, w_stride, x_dev, x_stride, sms, s);
}
