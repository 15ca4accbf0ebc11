// sm_103a products of E4M3 weights with a scale for each block of 128
// (afx_fp8_quantize, afx_fp8_product).
//
// fp8_quantize_kernel: for each token and block of 128 columns the largest
// magnitude a, scale = max(a / 448, 2^-126), values E4M3(x / scale).  A warp a
// block, four elements a lane, several blocks in flight; the eight warps of a
// CTA take eight tokens, whose scales share a sector.
// Bound: HBM bandwidth; x is read once.
//
// fp8_product_kernel: y = x W^T, a tile of 128 tokens by BN rows of W a CTA, in
// steps of 128 columns, the block of the scales.  A step is
//     D  = X_b W_b^T                    (tcgen05, E4M3, float32 in tensor memory)
//     y += D * (x_scale[token] * w_scale[row block])
// where y stays in registers: lane = token, so that a thread has one token's
// scale and, with all its columns within one or two row blocks, a factor a
// run of 32 columns.  The tensor cores cannot apply these factors themselves
// (their scaled form takes powers of two for every 32 elements), so a step's
// sums are read back; two buffers of them in tensor memory let the products of
// one step run while the other's sums are read.
//
// Roles of a CTA's 12 warps: 0-7 the sums (a quarter of the lanes and half of
// the columns each; they take registers from the others), 8 issues the products, 9 loads by TMA (128-byte rows with the
// 128-byte swizzle; columns past the matrix are zeros) into a ring of steps.
// Where tiles are fewer than SMs, a cluster of CTAs shares a tile: each takes a run
// of steps, and their sums are added through distributed shared memory in the
// order of the CTAs.
//
// Every wait is bounded: one that runs out raises AFX_DEV_TIMEOUT and a flag
// that all roles poll; copies and products in flight are waited for and the
// CTA frees its tensor memory and ends.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include <cstdio>

#include "afx_tensor.cuh"

namespace cg = cooperative_groups;

namespace afx {
namespace serve {
namespace {

constexpr uint32_t kBlock = AFX_FP8_BLOCK;

// ---- rounding activations ----------------------------------------------------------

constexpr int kQuantThreads = 256;
constexpr uint32_t kQuantAtOnce = 4;  // blocks in flight a warp

struct QuantArgs {
    const void* x;
    uint8_t* q;
    float* scales;
    uint64_t x_stride, q_stride, scale_stride;
    uint32_t n_tokens, cols, blocks, per_cta;  // per_cta: blocks that a CTA does of its eight tokens
};

template <typename T>
struct alignas(4 * sizeof(T)) Four {
    T v[4];
};
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }

// wide: runs of four elements and bytes are aligned.
template <typename T>
__global__ void __launch_bounds__(kQuantThreads) fp8_quantize_kernel(const QuantArgs a, const bool wide) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_earlier();
    let_next_start();
    const uint32_t t = blockIdx.x * (kQuantThreads / 32) + warp;
    if (t >= a.n_tokens) return;
    const T* x = static_cast<const T*>(a.x) + t * a.x_stride;
    uint8_t* q = a.q + t * a.q_stride;
    const uint32_t b0 = blockIdx.y * a.per_cta, b1 = min(a.blocks, b0 + a.per_cta);
    for (uint32_t b = b0; b < b1; b += kQuantAtOnce) {
        float v[kQuantAtOnce][4];
#pragma unroll
        for (uint32_t j = 0; j < kQuantAtOnce; ++j) {
            const uint32_t c = (b + j) * kBlock + lane * 4;
            if (wide && b + j < b1 && c + 4 <= a.cols) {
                const Four<T> f = *reinterpret_cast<const Four<T>*>(x + c);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j][i] = widen(f.v[i]);
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i) v[j][i] = b + j < b1 && c + i < a.cols ? widen(x[c + i]) : 0.0f;
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < kQuantAtOnce; ++j) {
            if (b + j >= b1) break;
            uint32_t most = 0;  // of the magnitudes' bits, which NaN and infinity lead
#pragma unroll
            for (int i = 0; i < 4; ++i) most = max(most, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
            most = __reduce_max_sync(0xFFFFFFFFu, most);
            const float scale = most >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : fmaxf(__fdiv_rn(__uint_as_float(most), 448.0f), 0x1p-126f);
            const uint32_t c = (b + j) * kBlock + lane * 4;
            // saturating: a quotient may be 448 and a rounding
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[j][0], scale), __fdiv_rn(v[j][1], scale)), __NV_SATFINITE, __NV_E4M3),
                           hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[j][2], scale), __fdiv_rn(v[j][3], scale)), __NV_SATFINITE, __NV_E4M3);
            const uint32_t bytes = lo | hi << 16;
            if (wide && c + 4 <= a.cols) {
                *reinterpret_cast<uint32_t*>(q + c) = bytes;
            } else {
#pragma unroll
                for (uint32_t i = 0; i < 4; ++i)
                    if (c + i < a.cols) q[c + i] = static_cast<uint8_t>(bytes >> (8 * i));
            }
            if (lane == 0) a.scales[(b + j) * a.scale_stride + t] = scale;
        }
    }
}

// ---- the product -------------------------------------------------------------------

constexpr uint32_t kTokens = 128;   // of a tile
constexpr int kSumWarps = 8, kMmaWarp = 8, kLoadWarp = 9;
constexpr int kProductThreads = 384;
// registers a thread: as launched, then of the warps with the sums and of the
// others (what the ones add is what the others gave up)
constexpr int kRegsLaunch = 168, kRegsSums = 208, kRegsOther = 88;
static_assert(256 * kRegsSums + 128 * kRegsOther <= kProductThreads * kRegsLaunch, "register shares");
constexpr uint32_t kMostStages = 16;
constexpr uint32_t kSmemMost = 232448;  // 227 KB, what a CTA can have
constexpr uint32_t kMostSplit = 8;

struct Ctl {
    uint64_t full[kMostStages], empty[kMostStages];
    uint64_t sums_full[2], sums_empty[2], drain;
    uint32_t tmem;
    int32_t abort_flag;
};
constexpr uint32_t kCtlBytes = 512;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

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

__device__ __forceinline__ void load_box(uint32_t lane, uint32_t dst, const CUtensorMap* map, uint32_t x, uint32_t y, uint64_t* bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.u32 q, %5, 0;\n"
        " @q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_addr(bar)), "r"(lane)
        : "memory");
}

__device__ __forceinline__ void mma_e4m3(uint32_t lane, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lane)
        : "memory");
}

// The columns loaded by tmem_load32 may be used behind this: they are its
// operands, so that no use of them is moved before it.
__device__ __forceinline__ void wait_columns(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;\n"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]),
                   "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]),
                   "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]),
                   "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
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

template <int BN>
struct Tile {
    static constexpr uint32_t kRuns = BN / 64;       // runs of 32 columns a warp
    static constexpr uint32_t kWBytes = BN * kBlock;
    static constexpr uint32_t kColumns = BN == 64 ? 128 : BN == 128 ? 256 : 512;  // of tensor memory, a power of two
    static constexpr uint32_t kPartRow = BN + 4;     // floats between tokens' sums in shared memory
};

template <int BN>
__global__ void __launch_bounds__(kProductThreads, 1) fp8_product_kernel(const __grid_constant__ ProductArgs a) {
    using T = Tile<BN>;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem);
    uint8_t* w_ring = smem + 1024;
    uint8_t* x_ring = w_ring + a.stages * T::kWBytes;
    float* staging = reinterpret_cast<float*>(x_ring + a.stages * a.box * kBlock + (kTokens - a.box) * kBlock);  // where !sectors
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < a.stages; ++i) {
            bar_init(&ctl.full[i], 1);
            bar_init(&ctl.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(&ctl.sums_full[i], 1);
            bar_init(&ctl.sums_empty[i], kSumWarps);
        }
        bar_init(&ctl.drain, 1);
        ctl.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(&ctl.tmem)), "r"(T::kColumns) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctl.tmem;
    wait_for_earlier();
    let_next_start();

    // a CTA's tiles: one a cluster, or every gridDim.x-th; its steps of a tile
    const uint32_t rank = blockIdx.x % a.split;
    const uint32_t step0 = static_cast<uint32_t>(static_cast<uint64_t>(a.blocks) * rank / a.split),
                   step1 = static_cast<uint32_t>(static_cast<uint64_t>(a.blocks) * (rank + 1) / a.split);
    const uint32_t first = blockIdx.x / a.split, stride = gridDim.x / a.split;

    if (warp >= kSumWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsOther));
      if (warp == kLoadWarp) {
        const bool leader = elect();
        uint32_t it = 0, slot = 0, phase = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < a.tiles; tile += stride) {
            const uint32_t t0 = tile % a.tiles_m * kTokens, r0 = tile / a.tiles_m * BN;
            for (uint32_t s = step0; s < step1; ++s, ++it) {
                if (it >= a.stages) {
                    ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.empty[slot], phase ^ 1u, ctl, a.status));
                    if (!ok) break;
                }
                if (leader) bar_expect(&ctl.full[slot], T::kWBytes + a.box * kBlock);
                __syncwarp();
                load_box(leader, smem_addr(w_ring + slot * T::kWBytes), &a.w, s * kBlock, r0, &ctl.full[slot]);
                load_box(leader, smem_addr(x_ring + slot * a.box * kBlock), &a.x, s * kBlock, t0, &ctl.full[slot]);
                if (++slot == a.stages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        if (!ok)  // copies in flight write this CTA's shared memory
            for (uint32_t q = it > a.stages ? it - a.stages : 0; q < it; ++q)
                if (!bar_drain(&ctl.full[q % a.stages], q / a.stages & 1u)) raise(a.status, AFX_DEV_UNDRAINED);
      } else if (warp == kMmaWarp) {
        // float32 sums of E4M3 by E4M3, both with their columns contiguous
        constexpr uint32_t kInstruction = 1u << 4 | (BN >> 3) << 17 | (kTokens >> 4) << 24;
        const bool leader = elect();
        const uint64_t x_desc = operand(smem_addr(x_ring), 16), w_desc = operand(smem_addr(w_ring), 16);
        uint32_t it = 0, slot = 0, phase = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < a.tiles; tile += stride) {
            for (uint32_t s = step0; s < step1; ++s, ++it) {
                const uint32_t buf = it & 1u;
                ok = __all_sync(0xFFFFFFFFu, (it < 2 || bar_wait(&ctl.sums_empty[buf], ((it >> 1) - 1) & 1u, ctl, a.status)) &&
                                                 bar_wait(&ctl.full[slot], phase, ctl, a.status));
                if (!ok) break;
                fence_after();
                const uint64_t xd = x_desc + slot * (a.box * kBlock >> 4), wd = w_desc + slot * (T::kWBytes >> 4);
#pragma unroll
                for (uint32_t k = 0; k < kBlock / 32; ++k) mma_e4m3(leader, tmem + buf * BN, xd + k * 2, wd + k * 2, kInstruction, k != 0);
                commit(leader, &ctl.empty[slot]);
                commit(leader, &ctl.sums_full[buf]);
                if (++slot == a.stages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        commit(leader, &ctl.drain);  // arrivals above land before this CTA ends
        if (!bar_drain(&ctl.drain, 0)) raise(a.status, AFX_DEV_UNDRAINED);
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsSums));
        const uint32_t quarter = warp % 4, half = warp / 4;
        const uint32_t column0 = half * (BN / 2), lanes = quarter * 32;
        uint32_t it = 0;
        bool ok = true;
        for (uint32_t tile = first; ok && tile < a.tiles; tile += stride) {
            const uint32_t t0 = tile % a.tiles_m * kTokens, r0 = tile / a.tiles_m * BN + column0;
            const uint32_t token = t0 + lanes + lane;
            const bool any = t0 + lanes < a.n_tokens, real = token < a.n_tokens;
            uint64_t sum[T::kRuns][16];
#pragma unroll
            for (uint32_t r = 0; r < T::kRuns; ++r)
#pragma unroll
                for (int i = 0; i < 16; ++i) sum[r][i] = 0;
            // a token's scales two steps ahead; the row blocks' for 32 steps, a lane a step
            const float* xs = a.x_scales + (real ? token : 0);
            auto x_scale = [&](uint32_t s) { return real && s < step1 ? __ldg(xs + s * a.x_scale_stride) : 0.0f; };
            float now = x_scale(step0), next = x_scale(step0 + 1);
            const uint32_t rb0 = min(r0 / kBlock, a.row_blocks - 1), rb1 = min((r0 + BN / 2 - 1) / kBlock, a.row_blocks - 1);
            auto w_scale = [&](uint32_t rb, uint32_t s) { return s + lane < step1 ? __ldg(a.w_scales + static_cast<uint64_t>(rb) * a.blocks + s + lane) : 0.0f; };
            float w0 = w_scale(rb0, step0), w1 = w_scale(rb1, step0), w0_next = w_scale(rb0, step0 + 32), w1_next = w_scale(rb1, step0 + 32);
            for (uint32_t s = step0; s < step1; ++s, ++it) {
                const uint32_t buf = it & 1u, in32 = (s - step0) & 31u;
                if (in32 == 0 && s != step0) {
                    w0 = w0_next, w1 = w1_next;
                    w0_next = w_scale(rb0, s + 32), w1_next = w_scale(rb1, s + 32);
                }
                const float later = x_scale(s + 2);
                const float f0 = now * __shfl_sync(0xFFFFFFFFu, w0, in32), f1 = now * __shfl_sync(0xFFFFFFFFu, w1, in32);
                ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.sums_full[buf], it >> 1 & 1u, ctl, a.status));
                if (!ok) break;
                fence_after();
                if (any) {
                    const uint32_t from = tmem + (lanes << 16) + buf * BN + column0;
                    uint32_t v[2][32];
                    tmem_load32(from, v[0]);
#pragma unroll
                    for (uint32_t r = 0; r < T::kRuns; ++r) {
                        wait_columns(v[r & 1]);
                        if (r + 1 < T::kRuns) tmem_load32(from + (r + 1) * 32, v[(r + 1) & 1]);
                        const float f = (r0 + r * 32) / kBlock == rb0 ? f0 : f1;
                        const uint64_t ff = pack2(f, f);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            sum[r][i] = fma2(pack2(__uint_as_float(v[r & 1][2 * i]), __uint_as_float(v[r & 1][2 * i + 1])), ff, sum[r][i]);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) bar_arrive(&ctl.sums_empty[buf]);
                now = next, next = later;
            }
            if (!ok) break;
            if (a.split > 1) {  // into shared memory, whose copies and products are all done with
                if (real) {
                    float* part = reinterpret_cast<float*>(w_ring) + (lanes + lane) * T::kPartRow + column0;
#pragma unroll
                    for (uint32_t r = 0; r < T::kRuns; ++r)
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float4 f;
                            unpack2(sum[r][i], &f.x, &f.y);
                            unpack2(sum[r][i + 1], &f.z, &f.w);
                            *reinterpret_cast<float4*>(part + r * 32 + i * 2) = f;
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
                    float* stage = staging + warp * (32 * 33);
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
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(T::kColumns) : "memory");
    }
    if (a.split > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();  // every CTA's sums are there
        const uint32_t t0 = first % a.tiles_m * kTokens, r0 = first / a.tiles_m * BN;
        const uint32_t tokens = min(kTokens, a.n_tokens - t0);
        const float* part = reinterpret_cast<const float*>(w_ring);
        for (uint32_t e = rank * kProductThreads + threadIdx.x; e < tokens * BN; e += a.split * kProductThreads) {
            const uint32_t t = e / BN, c = e % BN;
            if (r0 + c >= a.rows) continue;
            float sum = 0.0f;
            for (uint32_t i = 0; i < a.split; ++i) sum += *cluster.map_shared_rank(part + t * T::kPartRow + c, i);
            store_one(a, static_cast<uint64_t>(t0 + t) * a.y_stride + r0 + c, sum);
        }
        cluster.sync();  // no CTA ends while its sums are read
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

constexpr uint32_t kStagingBytes = kSumWarps * 32 * 33 * sizeof(float);

template <int BN>
afx_status launch_product(ProductArgs& a, uint32_t grid, cudaStream_t s) {
    using T = Tile<BN>;
    const uint32_t fixed = 1024 + 1024 + (kTokens - a.box) * kBlock + (a.sectors || a.split > 1 ? 0 : kStagingBytes);
    const uint32_t step = T::kWBytes + a.box * kBlock;
    a.stages = (kSmemMost - fixed) / step;
    if (a.stages > kMostStages) a.stages = kMostStages;
    // the sums of a CTA of several lie over the ring
    static_assert(kTokens * T::kPartRow * sizeof(float) <= 3 * (T::kWBytes + kTokens * kBlock), "sums fit the ring");
    // the warps with the sums wait for the registers that they ask for: they must be there
    static std::once_flag once;
    static int regs = 0;
    std::call_once(once, [] {
        cudaFuncAttributes f{};
        if (cudaFuncGetAttributes(&f, fp8_product_kernel<BN>) == cudaSuccess)
            regs = f.numRegs;
        else
            cudaGetLastError();
    });
    if (regs < kRegsLaunch) return afx_fail(AFX_E_CUDA, "fp8_product_kernel was built with too few registers", 0);
    AFX_SERVE_TRY(cudaFuncSetAttribute(fp8_product_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemMost)),
                  "cudaFuncSetAttribute");
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kProductThreads);
    cfg.dynamicSmemBytes = kSmemMost;
    cfg.stream = s;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = a.split;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    AFX_SERVE_TRY(cudaLaunchKernelEx(&cfg, fp8_product_kernel<BN>, a), "fp8_product_kernel launch");
    return AFX_OK;
}

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
    if (!device_ptr(x_dev, size) || !device_ptr(q_dev, 1) || !device_ptr(scales_dev, 4))
        return afx_fail(AFX_E_ARG, "the arrays must be device memory", 0);
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
    const bool wide = !((reinterpret_cast<uintptr_t>(x_dev) | (n_tokens > 1 ? x_stride * size : 0)) & (4 * size - 1)) &&
                      !((reinterpret_cast<uintptr_t>(q_dev) | (n_tokens > 1 ? q_stride : 0)) & 3u);
    // eight tokens a CTA; their blocks over more CTAs while the SMs have room, four blocks a warp or more otherwise
    const uint32_t groups = ceil_div(n_tokens, kQuantThreads / 32);
    uint32_t parts = ceil_div(static_cast<uint32_t>(sms) * 8, groups);
    a.per_cta = ceil_div(a.blocks, parts);
    if (a.per_cta > 1) a.per_cta = ceil_div(a.per_cta, kQuantAtOnce) * kQuantAtOnce;
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
    if (!device_ptr(w_dev, 16) || !device_ptr(x_dev, 16)) return afx_fail(AFX_E_ARG, "weights and activations must be 16-byte aligned device memory", 0);
    if (!device_ptr(w_scales_dev, 4) || !device_ptr(x_scales_dev, 4) || !device_ptr(y_dev, size) || (status_dev && !device_ptr(status_dev, 4)))
        return afx_fail(AFX_E_ARG, "the arrays must be device memory", 0);
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
    a.tiles_m = ceil_div(n_tokens, kTokens);
    a.box = n_tokens >= kTokens ? kTokens : ceil_div(n_tokens, 8) * 8;
    a.y_type = y_type;
    a.sectors = rows % 32 == 0 && !((reinterpret_cast<uintptr_t>(y_dev) | (n_tokens > 1 ? y_stride * size : 0)) & 31u);
    // The tile's rows and the CTAs a tile, by what a wave of CTAs takes in cycles: a step's products take 2 BN, its
    // loads arrive at 64 bytes a cycle; and what a CTA takes besides
    uint32_t best_bn = 128, best_split = 1;
    double best = 1e300;
    for (uint32_t bn = 64; bn <= 256; bn += 64)
        for (uint32_t split = 1; split <= kMostSplit && split <= a.blocks; ++split) {
            const uint64_t ctas = static_cast<uint64_t>(a.tiles_m) * ceil_div(rows, bn) * split;
            if (split > 1 && ctas > static_cast<uint64_t>(sms)) continue;
            const double waves = static_cast<double>((ctas + sms - 1) / sms);
            const double step = 2.0 * bn > (bn + a.box) * 2.0 ? 2.0 * bn : (bn + a.box) * 2.0;
            const double cost = waves * (ceil_div(a.blocks, split) * step + 500.0 + 2.0 * bn) + (split > 1 ? 1500.0 + 200.0 * split : 0.0);
            if (cost < best) best = cost, best_bn = bn, best_split = split;
        }
    a.split = best_split;
    const uint64_t tiles = static_cast<uint64_t>(a.tiles_m) * ceil_div(rows, best_bn);
    if (tiles > INT32_MAX) return afx_fail(AFX_E_ARG, "the result has too many tiles", 0);
    a.tiles = static_cast<uint32_t>(tiles);
    const uint32_t grid = a.split > 1 || tiles < static_cast<uint64_t>(sms) ? a.tiles * a.split : static_cast<uint32_t>(sms);
    afx_status st = byte_map(&a.x, x_dev, n_tokens, cols, x_stride, a.box);
    if (st == AFX_OK) st = byte_map(&a.w, w_dev, rows, cols, w_stride, best_bn);
    if (st != AFX_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (best_bn == 64) return launch_product<64>(a, grid, s);
    if (best_bn == 128) return launch_product<128>(a, grid, s);
    if (best_bn == 192) return launch_product<192>(a, grid, s);
    return launch_product<256>(a, grid, s);
}
