// What the attention kernels share: the plan's records, the arguments and
// the two 16-bit types' arithmetic.
#pragma once

#include <cuda.h>

#include "afx_serving.cuh"

namespace afx {
namespace serve {

constexpr uint32_t kRows = 16;            // packed rows of a row-16 item
constexpr uint32_t kTileRows = 128;       // rows of a tensor-memory tile: one lane each
constexpr uint32_t kTileKeys = 128;       // keys of one step
constexpr uint32_t kGroupRows = 2 * kTileRows;

// The key names what the plan was made for: a workspace that holds no plan,
// or that of another description, is refused instead of read.
struct PlanHead {
    uint64_t key;
    uint64_t cost;          // of all tile groups x heads
    uint64_t share;         // cost of one CTA of the tile kernel
    uint32_t n_tokens;      // live rows of the queries
    uint32_t n_items;       // row-16 items
    uint32_t n_tiles;       // tile groups
    uint32_t prefix_kind;   // Source of the packed rows' prefix part
    uint32_t n_rest;        // tile groups whose output the join writes whatever CTAs had them
    uint32_t n_by_row;      // tokens that are not in tiles of their request's own
};

enum Source : uint32_t { kNone = 0, kRow16 = 1, kTile = 2 };

// A request's own keys (its tiles may have the prefix before them): its rows'
// first group, of kRows or kGroupRows rows each.
struct alignas(16) RequestInfo {
    uint32_t kind, first, pad[2];
};

// A token of the queries: its request, its first packed row among the
// request's, its place among the tokens that share the prefix's groups (or
// kInTiles, kAlone), and its request's own groups.
struct alignas(16) TokenInfo {
    uint32_t request, row, packed, pad;
    RequestInfo own;
};

// TokenInfo::packed of tokens that do not share the prefix's groups: in
// tiles of their request's own, or (no prefix) in 16-row items.
constexpr uint32_t kInTiles = 0xFFFFFFFEu, kAlone = 0xFFFFFFFFu;

// 16 packed rows of one source: its pieces' results start at part_row, piece
// s at part_row + s * rows.
struct alignas(16) Row16Group {
    uint32_t part_row, n_pieces, rows, pad;
};

struct alignas(16) Row16Item {
    int32_t request;        // -1: the prefix
    uint32_t row0, rows;    // packed rows of the source
    uint32_t key0, key1;    // keys of the source
    uint32_t part_row;      // where the results of its rows go
    uint32_t token0;        // first token of the source (prefix: tokens come from the packed list)
    int32_t seen;           // token i of the source sees keys below seen + i + 1 (prefix: all)
};

// Up to 256 packed rows and the keys they see: `prefix_keys` of the prefix,
// then `own_keys` of the request.  cost: kGroupCost and step_cost a step of 128
// keys; 0 without keys.
struct alignas(16) TileGroup {
    uint64_t cost_begin;    // of head 0; head h begins h * cost later
    uint64_t part_row;      // where the results of the first piece of head 0 go
    uint32_t cost;
    int32_t request;        // -1: packed rows of the batch on the prefix
    uint32_t row0, rows;
    uint32_t prefix_keys, own_keys;
    uint32_t token0;
    int32_t seen;
    uint32_t single;        // nothing else contributes to these rows
    uint32_t pad[3];
};

struct AttnLayout {
    uint64_t counter;       // 16-row units taken so far, by this layer
    uint64_t tokens, packed_token, groups16, items16, tiles, tile_first, rest, part_ml, part_o, total;
    uint64_t extra_row;     // rows of the tile kernel's further pieces: 256 a CTA
    uint64_t max_rows;      // rows of the 16-row kernel's pieces
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
    AttnLayout L;
    uint64_t plan_key;
    uint32_t table_cols, n_requests, n_tokens, prefix_len, group, kv_heads, shift, n_pages;
    uint32_t q_align;  // bytes every query row's address is a multiple of, at most 16
    uint32_t tile_ctas;  // 0: no tile groups, all rows go to the 16-row kernel
    float scale_log2;

    template <typename P>
    __device__ __forceinline__ P* at(uint64_t off) const { return reinterpret_cast<P*>(ws + off); }
};

// Keys that token row / group of a source sees.
__device__ __forceinline__ uint32_t visible(int32_t seen, uint32_t row, uint32_t group) {
    const int64_t v = static_cast<int64_t>(seen) + row / group + 1;
    return v > 0 ? static_cast<uint32_t>(v) : 0u;
}

// More than 128 rows: both tiles work on every step's keys.  Fewer: the tiles
// take the steps in turn, and half the products need as many keys (measured:
// some 3200 cycles a step for both, 2000 for one).
constexpr uint32_t kStepBoth = 8, kStepOne = 5;
// What a group costs besides: filling and emptying the pipe, masked steps, the
// output (24 requests of 5 to 11 tokens on 5722 keys in common: 77 us a call,
// caches flushed, 121 without; 78 of 5 to 12 tokens on 16,025: 311 and 516).
constexpr uint32_t kGroupCost = 20;
__host__ __device__ __forceinline__ uint32_t step_cost(uint32_t rows) { return rows > kTileRows ? kStepBoth : kStepOne; }

// Costs mostly fit 32 bits, where a division takes a fraction of the time.
__device__ __forceinline__ uint32_t divide(uint64_t a, uint64_t b) {
    return (a | b) >> 32 ? static_cast<uint32_t>(a / b) : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// The CTAs [first, last] of the tile kernel that hold pieces of a group's
// head; for a group with keys.
__device__ __forceinline__ void tile_ctas(const TileGroup& g, uint32_t h, uint64_t share, uint32_t* first, uint32_t* last) {
    const uint64_t begin = g.cost_begin + static_cast<uint64_t>(h) * g.cost;
    *first = divide(begin + kGroupCost + step_cost(g.rows) - 1, share);
    *last = divide(begin + g.cost - 1, share);
}

// The result row of a tile-kernel piece: the first piece of a group's head
// has rows of its own, a CTA's continued piece the CTA's.
__device__ __forceinline__ uint64_t tile_part_row(const TileGroup& g, uint32_t h, uint32_t first_cta, uint32_t cta, uint64_t extra_row) {
    const uint32_t rows = g.rows > kTileRows ? g.rows : 2 * g.rows;
    return cta == first_cta ? g.part_row + static_cast<uint64_t>(h) * rows : extra_row + static_cast<uint64_t>(cta) * kGroupRows;
}

// 16 bytes to shared memory; zeros where not real, and src is not read.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool real) {
    const uint32_t n = real ? 16u : 0u;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static constexpr uint32_t kMmaType = 1;  // in the tcgen05 instruction descriptor
    static constexpr float kUp = 0.0f;
    static constexpr float kHigh = 14.0f;
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
struct Elem<__half> {
    static constexpr uint32_t kMmaType = 0;
    static constexpr float kUp = 7.0f;
    static constexpr float kHigh = 15.0f;
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

// Weights are 2^(score - reference), the reference kUp below a maximum of the
// row's scores that lags behind by up to kLag powers of two (in the tile
// kernel, until the next step, by more: to where weights reach 2^kHigh): exact
// all the same (numerator and denominator use the same reference), and it
// saves scaling the sums on every small rise.  FP16 holds weights from 2^-25
// to 2^16 (the ones below 2^-14 to 2^-25 each): 7 powers of two up, 131,000
// keys that are each below 2^-26 of the largest one are still in the product
// with V as they are in the float32 sum; without, they were in the sum alone,
// up to 0.4 % of it.
constexpr float kLag = 8.0f;

constexpr float kLn2 = 0.693147180559945309f;

// afx_attention_tile.cu: whether the tile kernel can read this cache (its
// layout fits a tensor map), and that kernel over the plan's tile groups.
bool tiles_fit(const afx_kv_cache& cache);
afx_status launch_tiles(const AttnArgs& a, const afx_kv_cache& cache, cudaStream_t s);

}  // namespace serve
}  // namespace afx
