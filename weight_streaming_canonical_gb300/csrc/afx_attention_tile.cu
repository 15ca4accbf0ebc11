// sm_103a attention for many rows on the same keys: the tensor-core kernel
// of afx_attention (tcgen05, tensor memory, TMA).
//
// A tile group is up to 256 packed query rows of one key/value head, as two
// tiles of 128 rows, and the keys they see, in steps of 128.  A step of a
// tile is
//     S = Q K^T            (tcgen05, 128 x 128, float32 in tensor memory)
//     P = 2^(S * c - ref)  (one thread a row: lane = row)
//     O += P V             (P in tensor memory, V from shared memory)
// with the running reference and sum of the softmax in the row's thread.
// While one tile's threads work on their scores, the tensor cores work for
// the other tile.  With more than 128 rows both tiles use every step's keys;
// with fewer the two tiles hold the same rows and take the steps in turn
// (their results are two pieces of the same rows).
//
// Work split: the cost of all groups x heads, laid end to end, is cut into
// equal shares, one CTA each, whatever groups that cuts through; the join
// puts a group's pieces together.  So every SM gets the same number of
// steps whether there are two groups or thousands.  A piece that is a whole
// group of a request's own tiles is written to the output here.
//
// Roles of a CTA's 12 warps: 0-3 and 4-7 the rows of tile 0 and 1 (a row's
// 128 scores stay in its thread's registers: these warps take registers from
// the others), 8 issues the products, 9 loads keys and 10 values, each page of
// a step by TMA (64 elements x the page's tokens a box, 128-byte swizzle), into
// a ring of slots that runs ahead over groups, 11 loads queries (rows of any
// stride, so by 16-byte copies) as soon as a tile's last scores are done, while
// its rows still work: with the row warps loading their own queries, a group
// cost 20,000 cycles besides its steps, so 13,000.  Tensor memory: S0 S1 O0 O1;
// P replaces S in place for heads of 128, and has columns of its own for heads
// of 64.
//
// Bound: the products' chain (scores, weights, values, scores ...) of two
// tiles; 3200 cycles a step of both tiles, of which the products take 2048.
// 16 prompts of 200 to 500 tokens on 4100 keys in common, 40 heads of 128 on
// 8, BF16: 394 us, 1.16 PFLOP/s of what the masks leave, 61 % of a large library
// product's rate on this GPU.
//
// Every wait is bounded: one that runs out raises AFX_DEV_TIMEOUT and a
// flag that all roles poll, copies and products in flight are waited for,
// and the CTA frees its tensor memory and ends.
#include <cstdio>

#include "afx_attention.cuh"
#include "afx_tensor.cuh"

namespace afx {
namespace serve {
namespace {

constexpr int kSoftWarps = 8;
constexpr int kMmaWarp = 8, kLoadWarp = 9;  // keys; values: the warp after it
constexpr int kQueryWarp = 11;
constexpr int kTileThreads = 384;
// registers a thread: as launched, then of the row warps and of the others
// (what the row warps add is what the others gave up)
constexpr int kRegsLaunch = 168, kRegsRows = 208, kRegsOther = 88;
static_assert(256 * kRegsRows + 128 * kRegsOther <= kTileThreads * kRegsLaunch, "register shares");

template <int D>
struct Shape {
    static constexpr uint32_t kHalves = D / 64;                    // 128-byte wide column blocks of a tile
    static constexpr uint32_t kBlock = kTileKeys * 128;            // bytes of one
    static constexpr uint32_t kSlot = kHalves * kBlock;            // keys or values of a step
    static constexpr uint32_t kSlots = D == 128 ? 5 : 8;
    static constexpr uint32_t kQ = 2 * kSlot;                      // both tiles' queries
    static constexpr uint32_t kCtl = kQ + kSlots * kSlot;
    static constexpr uint32_t kSmem = kCtl + 1024 + 1024;          // control block, alignment
    // tensor memory columns
    static constexpr uint32_t kS = 0, kO = 256, kP = D == 128 ? 0 : 384;
    static constexpr uint32_t kPStep = D == 128 ? 128 : 64;
};

struct Ctl {
    uint64_t full[8], empty[8];
    uint64_t tail;                     // a last step's values, before their missing rows are zeroed
    uint64_t q_full[2], q_empty[2];    // a tile's queries
    uint64_t s_full[2], p_full[2][2], pv_done[2];
    uint64_t drain;
    // a tile's last 8 steps: a bit for 16 keys whose page lies outside the pool; read, and written at every step, from
    // the first such page on.  A step's word is written when the slot of its keys is free: the rows have weighed the
    // step 3 (heads of 128) or 6 (of 64) before it by then
    uint32_t any_absent, absent[2][8];
    uint32_t tmem;
    int32_t abort_flag;
};
static_assert(sizeof(Ctl) <= 1024, "control block");

struct TileArgs {
    CUtensorMap k, v;
    AttnArgs a;
    // where token and head stand among the map's outer dimensions (by stride, smallest first); page has the place that is left
    uint32_t token_at, head_at;
};

// ---- barriers, TMA, tensor memory ------------------------------------------------

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

__device__ __forceinline__ void load_box(uint32_t lane, uint32_t dst, const CUtensorMap* map, uint32_t x, uint32_t c1, uint32_t c2,
                                         uint32_t c3, uint32_t bar) {
    asm volatile(
        "{\n .reg .pred q;\n setp.ne.u32 q, %7, 0;\n"
        " @q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n}\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(c1), "r"(c2), "r"(c3), "r"(bar), "r"(lane)
        : "memory");
}

// The instructions below are issued by one lane of a converged warp: the
// predicate is in the instruction, not in a branch around it, so that
// descriptors and addresses stay in uniform registers.

// D = A B^T (+ D), A and B in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t lane, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lane)
        : "memory");
}
// The same with A in tensor memory.
__device__ __forceinline__ void mma_ts(uint32_t lane, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %4, 0;\n setp.ne.u32 q, %5, 0;\n"
        " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u), "r"(lane)
        : "memory");
}
// Multiplies 8 n columns of this thread's lane by f.  Rare: kept out of the
// row warps' loop, whose code is long enough.
__device__ __noinline__ void scale_columns(uint32_t addr, int n, float f) {
    for (int c = 0; c < n; ++c) {
        uint32_t v[8];
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n" : AFX_R8(v, 0) : "r"(addr + c * 8) : "memory");
        tmem_wait_load();
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(addr + c * 8), AFX_W8(v, 0) : "memory");
    }
}

// ---- a CTA's share -----------------------------------------------------------------

// The pieces of a CTA's share of the cost, in order; every role walks the
// same ones.
struct Walk {
    const TileGroup* groups;
    uint64_t at, end;
    uint32_t n, heads, cta, g;

    __device__ Walk(const AttnArgs& a, const PlanHead& head)
        : groups(a.at<TileGroup>(a.L.tiles)), n(head.n_tiles), heads(a.kv_heads), cta(blockIdx.x), g(0) {
        at = static_cast<uint64_t>(cta) * head.share;
        end = at + head.share < head.cost ? at + head.share : head.cost;
        if (at >= end) return;
        uint32_t lo = 0, hi = n;  // the group that holds `at`
#pragma unroll 1
        while (hi - lo > 1) {
            const uint32_t mid = (lo + hi) >> 1;
            if (groups[mid].cost_begin <= at)
                lo = mid;
            else
                hi = mid;
        }
        g = lo;
    }
    struct Piece {
        TileGroup g;
        uint32_t h, step0, step1;  // steps of 128 keys, prefix first
        uint32_t prefix_steps;
        bool both;                 // both tiles on every step
    };
    __device__ bool next(Piece* p) {
#pragma unroll 1
        while (at < end) {
#pragma unroll 1
            while (at >= groups[g].cost_begin + static_cast<uint64_t>(groups[g].cost) * heads) ++g;
            p->g = groups[g];
            const uint64_t in = at - p->g.cost_begin;
            p->h = divide(in, p->g.cost);
            const uint32_t off = static_cast<uint32_t>(in - static_cast<uint64_t>(p->h) * p->g.cost);
            const uint64_t stop = min(end, p->g.cost_begin + (static_cast<uint64_t>(p->h) + 1) * p->g.cost);
            const uint32_t off1 = off + static_cast<uint32_t>(stop - at), each = step_cost(p->g.rows);
            p->both = p->g.rows > kTileRows;
            p->prefix_steps = ceil_div(p->g.prefix_keys, kTileKeys);
            const uint32_t steps = p->prefix_steps + ceil_div(p->g.own_keys, kTileKeys);
            p->step0 = off > kGroupCost ? (off - kGroupCost) / each : 0;
            p->step1 = off1 > kGroupCost ? min(steps, (off1 - kGroupCost) / each) : 0;
            at = stop;
            if (p->step0 < p->step1) return true;  // else the share ends before the group's first step
        }
        return false;
    }
};

// The keys of step s of a group: `first` in its source, `n` of them.
__device__ __forceinline__ void step_keys(const Walk::Piece& p, uint32_t s, bool* prefix, uint32_t* first, uint32_t* n) {
    *prefix = s < p.prefix_steps;
    *first = (*prefix ? s : s - p.prefix_steps) * kTileKeys;
    const uint32_t all = *prefix ? p.g.prefix_keys : p.g.own_keys;
    *n = min(kTileKeys, all - *first);
}

// ---- the kernel ----------------------------------------------------------------------

template <typename T, int D>
__global__ void __launch_bounds__(kTileThreads, 1) attention_tile_kernel(const __grid_constant__ TileArgs args) {
    using Sh = Shape<D>;
    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Ctl& ctl = *reinterpret_cast<Ctl*>(smem + Sh::kCtl);
    const AttnArgs& a = args.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < Sh::kSlots; ++i) {
            bar_init(&ctl.full[i], 1);
            bar_init(&ctl.empty[i], 1);
        }
        bar_init(&ctl.tail, 1);
        for (int t = 0; t < 2; ++t) {
            bar_init(&ctl.q_full[t], 1);
            bar_init(&ctl.q_empty[t], 1);
            bar_init(&ctl.s_full[t], 1);
            bar_init(&ctl.p_full[t][0], kSoftWarps / 2);
            bar_init(&ctl.p_full[t][1], kSoftWarps / 2);
            bar_init(&ctl.pv_done[t], 1);
        }
        bar_init(&ctl.drain, 1);
        ctl.abort_flag = 0;
        ctl.any_absent = 0;
        for (int i = 0; i < 16; ++i) ctl.absent[i / 8][i % 8] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_addr(&ctl.tmem)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctl.tmem;
    wait_for_earlier();
    let_next_start();  // the plan is done, which is all that the 16-row kernel needs
    PlanHead head = *a.at<PlanHead>(0);
    if (head.key != a.plan_key) {
        if (threadIdx.x == 0) raise(a.status, AFX_DEV_BAD_PLAN);
        head.cost = 0;
    }
    Walk walk(a, head);
    Walk::Piece p;
    if (threadIdx.x == 0 && walk.at < walk.end) a.at<uint32_t>(a.L.tile_first)[blockIdx.x] = walk.g;  // for the join
    if (warp >= kSoftWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsOther));
      if (warp == kLoadWarp || warp == kLoadWarp + 1) {
        // ---- keys and values: slot 2 i of the sequence is step i's keys, 2 i + 1 its values.  A lane a page looks
        // the page up; one lane issues all copies, from values that are the same in the whole warp (a copy from each
        // lane on its own took 180 cycles a copy, one after the other)
        const uint32_t kv = warp - kLoadWarp;
        const CUtensorMap* map = kv ? &args.v : &args.k;
        const uint32_t box = min(1u << a.shift, kTileKeys), page_mask = (1u << a.shift) - 1;
        const bool leader = elect();
        uint32_t slot = kv, phase = 0, seq = kv, tails = 0;
        uint32_t any_gone = 0, of_tile[2] = {0, 0};  // boxes outside the pool; a tile's steps so far
        bool ok = true;
        while (ok && walk.next(&p)) {
            for (uint32_t s = p.step0; s < p.step1 && ok; ++s) {
                bool prefix;
                uint32_t first, n;
                step_keys(p, s, &prefix, &first, &n);
                const uint32_t used = ceil_div(n, box);  // boxes that hold keys of this step
                uint32_t page = 0;
                bool missing = false;
                if (static_cast<uint32_t>(lane) < used) {
                    const uint32_t col = (first + lane * box) >> a.shift;
                    const int32_t id = prefix ? __ldg(a.prefix_table + col) : __ldg(a.table + static_cast<uint64_t>(p.g.request) * a.table_cols + col);
                    missing = id < 0 || static_cast<uint32_t>(id) >= a.n_pages;
                    if (missing) raise(a.status, AFX_DEV_BAD_PAGE);
                    page = missing ? a.n_pages : id;  // past the map's end a box is zeros
                }
                const uint32_t gone = __ballot_sync(0xFFFFFFFFu, missing);
                if (seq >= Sh::kSlots) {
                    ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.empty[slot], phase ^ 1u, ctl, a.status));
                    if (!ok) break;
                }
                // a last step's values: rows past the keys must be zeros, whatever the page holds there (0 * NaN)
                const bool patch = kv == 1 && n < kTileKeys;
                uint64_t* bar = patch ? &ctl.tail : &ctl.full[slot];
                const uint32_t dst = smem_addr(smem + Sh::kQ) + slot * Sh::kSlot;
                if (kv == 0) {
                    any_gone |= gone;
                    if (any_gone) {  // the rows leave these keys out
                        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, lane < 8 && (gone >> (lane * 16 / box) & 1));
                        for (uint32_t t = 0; t < 2; ++t)
                            if (leader && (p.both || ((s - p.step0) & 1) == t)) ctl.absent[t][of_tile[t] % 8] = bits;
                        if (leader) ctl.any_absent = 1;
                    }
                    of_tile[0] += p.both || !((s - p.step0) & 1);
                    of_tile[1] += p.both || ((s - p.step0) & 1);
                }
                if (leader) bar_expect(bar, used * box * 128 * Sh::kHalves);
#pragma unroll 1
                for (uint32_t b = 0; b < used; ++b) {
                    const uint32_t id = __shfl_sync(0xFFFFFFFFu, page, b), token = first & page_mask;  // 0 but for pages of 256
                    const uint32_t c1 = args.token_at == 0 ? token : args.head_at == 0 ? p.h : id, c2 = args.token_at == 1 ? token : args.head_at == 1 ? p.h : id,
                                   c3 = args.token_at == 2 ? token : args.head_at == 2 ? p.h : id;
#pragma unroll
                    for (uint32_t hf = 0; hf < Sh::kHalves; ++hf)
                        load_box(leader, dst + hf * Sh::kBlock + b * box * 128, map, hf * 64, c1, c2, c3, smem_addr(bar));
                }
                __syncwarp();
                if (patch) {
                    ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.tail, tails & 1u, ctl, a.status));
                    if (!ok) {
                        if (!bar_drain(&ctl.tail, tails & 1u)) raise(a.status, AFX_DEV_UNDRAINED);
                        break;
                    }
                    ++tails;
                    uint8_t* v = smem + Sh::kQ + slot * Sh::kSlot;
                    for (uint32_t hf = 0; hf < Sh::kHalves; ++hf)
#pragma unroll 1
                        for (uint32_t i = n * 8 + lane; i < kTileKeys * 8; i += 32)
                            *reinterpret_cast<uint4*>(v + hf * Sh::kBlock + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_shared();
                    __syncwarp();
                    if (leader) bar_arrive(&ctl.full[slot]);
                }
                seq += 2;
                slot += 2;
                if (slot >= Sh::kSlots) {
                    slot -= Sh::kSlots;
                    phase ^= 1u;
                }
            }
        }
        if (!ok) {  // this warp's copies in flight land before the CTA ends
            uint32_t q = seq > Sh::kSlots ? seq - Sh::kSlots : 0;
            for (q += (q & 1u) != kv; q < seq; q += 2)
                if (!bar_drain(&ctl.full[q % Sh::kSlots], (q / Sh::kSlots) & 1u)) raise(a.status, AFX_DEV_UNDRAINED);
        }
      } else if (warp == kQueryWarp) {
        // ---- the queries, in the operand's swizzled order: a lane works out where a row lies, then 16 bytes a lane of
        // two (or four) rows at a time.  A tile's next ones are fetched while its rows finish with the last scores
        constexpr uint32_t kChunks = D / 8, kRowsAtOnce = 32 / kChunks;
        const T* q = static_cast<const T*>(a.q);
        const int32_t* packed = a.at<int32_t>(a.L.packed_token);
        const uint32_t c = lane % kChunks;
        uint32_t phases = 0, used = 0;  // a bit a tile
        bool ok = true;
        while (ok && walk.next(&p)) {
            const TileGroup& g = p.g;
            // lane l's rows: l, l + 32, ...; all into L2 while the products still use the rows before
            uint64_t at[kGroupRows / 32];
#pragma unroll
            for (uint32_t j = 0; j < kGroupRows / 32; ++j) {
                const uint32_t pr = g.row0 + min(j * 32 + lane, g.rows - 1), tok = pr / a.group;
                const uint32_t token = g.request < 0 ? __ldg(packed + tok) : g.token0 + tok;
                at[j] = reinterpret_cast<uint64_t>(q + token * a.q_token + (p.h * a.group + (pr - tok * a.group)) * a.q_head);
            }
#pragma unroll
            for (uint32_t j = 0; j < kGroupRows / 32; ++j)
                if (j * 32 + lane < g.rows)
#pragma unroll
                    for (uint32_t b = 0; b < D * 2; b += 128) asm volatile("prefetch.global.L2 [%0];\n" ::"l"(at[j] + b));
#pragma unroll 1
            for (uint32_t t = 0; t < (p.both ? 2u : 1u); ++t) {
                if (used >> t & 1) {
                    ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.q_empty[t], phases >> t & 1, ctl, a.status));
                    if (!ok) break;
                    phases ^= 1u << t;
                }
                used |= 1u << t;
                const uint32_t dst = smem_addr(smem) + t * Sh::kSlot + (c / 8) * Sh::kBlock;
#pragma unroll 1
                for (uint32_t r0 = 0; r0 < kTileRows; r0 += 32) {
                    const uint64_t src = at[0];
#pragma unroll
                    for (uint32_t j = 0; j + 1 < kGroupRows / 32; ++j) at[j] = at[j + 1];
                    auto each = [&](auto&& copy) {
#pragma unroll
                        for (uint32_t i = 0; i < 32 / kRowsAtOnce; ++i) {
                            const uint32_t in32 = i * kRowsAtOnce + lane / kChunks, in_tile = r0 + in32;
                            copy(dst + in_tile * 128 + (((c % 8) ^ (in_tile & 7)) * 16), __shfl_sync(0xFFFFFFFFu, src, in32) + c * 16,
                                 t * kTileRows + in_tile < g.rows);
                        }
                    };
                    if (a.q_align == 16) {
                        each([](uint32_t to, uint64_t from, bool real) { copy16(to, reinterpret_cast<const void*>(from), real); });
                    } else {
                        each([](uint32_t to, uint64_t from, bool real) {
                            const uint16_t* e = reinterpret_cast<const uint16_t*>(from);
                            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (real) w[k] = __ldg(e + 2 * k) | static_cast<uint32_t>(__ldg(e + 2 * k + 1)) << 16;
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
                        });
                    }
                }
                asm volatile("cp.async.wait_all;\n" ::: "memory");
                fence_async_shared();
                __syncwarp();
                if (lane == 0) bar_arrive(&ctl.q_full[t]);
            }
        }
      } else if (warp == kMmaWarp) {
        // ---- the products.  The whole warp walks the steps and waits; one
        // lane, the same throughout, issues (descriptors stay warp-uniform)
        // float32 accumulator, A and B of the cache's type, M = 128; values have their head elements contiguous (bit 16)
        constexpr uint32_t kBase = (1u << 4) | (Elem<T>::kMmaType << 7) | (Elem<T>::kMmaType << 10) | ((kTileRows >> 4) << 24);
        constexpr uint32_t kQk = kBase | ((kTileKeys >> 3) << 17), kPv = kBase | (1u << 16) | ((D >> 3) << 17);
        const bool leader = elect();
        const uint64_t q_desc = operand(smem_addr(smem), 16), k_desc = operand(smem_addr(smem + Sh::kQ), 16),
                       v_desc = operand(smem_addr(smem + Sh::kQ), Sh::kBlock);
        const uint32_t qk = kQk | (a.scale_log2 < 0.0f ? 1u << 13 : 0u);  // a negative scale: -q instead
        uint32_t q_phase = 0, p_count[2] = {0, 0};
        uint32_t k_slot = 0, k_phase = 0;  // ring position of the next keys or values to use
        bool ok = true;
        auto uniform = [&](bool r) { return __all_sync(0xFFFFFFFFu, r); };
        auto slot_full = [&](uint32_t slot, uint32_t phase) {
            const bool r = uniform(bar_wait(&ctl.full[slot], phase, ctl, a.status));
            fence_after();
            return r;
        };
        auto step_on = [&](uint32_t& slot, uint32_t& phase) {
            if (++slot == Sh::kSlots) {
                slot = 0;
                phase ^= 1u;
            }
        };
        auto scores = [&](uint32_t t, uint32_t slot, bool own_q, bool release, bool last_q) {
            const uint64_t qd = q_desc + (own_q ? t * (Sh::kSlot >> 4) : 0), kd = k_desc + slot * (Sh::kSlot >> 4);
#pragma unroll
            for (uint32_t ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks / 4) * (Sh::kBlock >> 4) + (ks % 4) * 2;
                mma_ss(leader, tmem + Sh::kS + t * kTileKeys, qd + off, kd + off, qk, ks != 0);
            }
            if (release) commit(leader, &ctl.empty[slot]);
            commit(leader, &ctl.s_full[t]);
            if (last_q) commit(leader, &ctl.q_empty[own_q ? t : 0]);
        };
        // the weights come in two halves of 64 keys; false: a wait gave up
        auto values = [&](uint32_t t, uint32_t slot, bool first, bool release) {
            const uint64_t vd = v_desc + slot * (Sh::kSlot >> 4);
            const uint32_t phase = p_count[t]++ & 1u;
#pragma unroll
            for (uint32_t half = 0; half < 2; ++half) {
                if (!uniform(bar_wait(&ctl.p_full[t][half], phase, ctl, a.status))) return false;
                fence_after();
#pragma unroll
                for (uint32_t ks = half * 4; ks < half * 4 + 4; ++ks)
                    mma_ts(leader, tmem + Sh::kO + t * D, tmem + Sh::kP + t * Sh::kPStep + ks * 8, vd + ks * (2048 >> 4), kPv, !first || ks != 0);
            }
            if (release) commit(leader, &ctl.empty[slot]);
            commit(leader, &ctl.pv_done[t]);  // last: the row threads wait for it before the CTA ends
            return true;
        };
        while (ok && walk.next(&p)) {
            const uint32_t n = p.step1 - p.step0;
            const bool both = p.both;
            ok = slot_full(k_slot, k_phase);
            // scores of step 0; then, with both tiles on every step, a tile at a time the values of step i and the
            // scores of step i + 1 (whose place in tensor memory the weights of step i held); with the tiles taking
            // turns the scores of step i + 1, of the other tile, first
#pragma unroll 1
            for (uint32_t t = 0; t < (both ? 2u : 1u) && ok; ++t) {
                ok = uniform(bar_wait(&ctl.q_full[t], q_phase >> t & 1, ctl, a.status));
                q_phase ^= 1u << t;
                fence_after();
                if (ok) scores(t, k_slot, both, !both || t == 1, n == 1);
            }
            uint32_t v_slot = 0;
#pragma unroll 1
            for (uint32_t u = 0; u < (both ? 2 * n : n) && ok; ++u) {
                const uint32_t t = u & 1, i = both ? u >> 1 : u;
                const bool more = i + 1 < n, last = !both || t == 1;
                if (!both || t == 0) {  // on to step i's values and step i + 1's keys
                    step_on(k_slot, k_phase);
                    v_slot = k_slot;
                    const uint32_t v_phase = k_phase;
                    step_on(k_slot, k_phase);
                    ok = !more || slot_full(k_slot, k_phase);
                    if (ok && more && !both) scores(t ^ 1, k_slot, false, true, i + 2 == n);
                    ok = ok && slot_full(v_slot, v_phase);
                }
                ok = ok && values(t, v_slot, both ? i == 0 : i < 2, last);
                if (ok && more && both) scores(t, k_slot, true, last, i + 2 == n);
            }
        }
        if (!ok && leader) {  // products in flight finish before the tensor memory is freed
            commit(1, &ctl.drain);
            if (!bar_drain(&ctl.drain, 0)) raise(a.status, AFX_DEV_UNDRAINED);
        }
        __syncwarp();
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsRows));
        // ---- one row a thread
        const uint32_t t = warp >> 2, in_tile = threadIdx.x & 127;
        const uint32_t lanes = (static_cast<uint32_t>(warp & 3) * 32u) << 16;
        const uint32_t s_col = tmem + lanes + Sh::kS + t * kTileKeys, p_col = tmem + lanes + Sh::kP + t * Sh::kPStep,
                       o_col = tmem + lanes + Sh::kO + t * D;
        float* part_o = a.at<float>(a.L.part_o);
        float2* part_ml = a.at<float2>(a.L.part_ml);
        const float scale = fmaxf(fabsf(a.scale_log2), 1e-30f);  // not 0: masked scores stay minus infinity
        constexpr float kRise = kLag + Elem<T>::kUp;
        uint32_t s_count = 0, pv_count = 0;
        bool ok = true;
        while (ok && walk.next(&p)) {
            const TileGroup& g = p.g;
            const uint32_t row = (p.both ? t * kTileRows : 0) + in_tile;
            const bool live = row < g.rows;
            const bool warp_live = (p.both ? t * kTileRows : 0) + (warp & 3) * 32 < g.rows;
            const uint32_t limit = g.request < 0 || !live ? g.own_keys : min(g.own_keys, visible(g.seen, g.row0 + row, a.group));
            const uint32_t all_see = g.request < 0 ? g.own_keys : visible(g.seen, g.row0, a.group);  // own keys every row sees
            float ref = -INFINITY, sum = 0.0f, seen_most = -INFINITY;
            const uint32_t first = p.step0 + (p.both ? 0 : t), stride = p.both ? 1 : 2;
            uint32_t done = 0;  // steps of this tile
            // a new reference: the sums so far are scaled to it (the scores' barrier of this step says that the
            // product with the last step's weights is done too)
            auto rebase = [&](float most) {
                const float next = most > ref + kRise ? most - Elem<T>::kUp : ref;
                const float f = next == -INFINITY ? 1.0f : exp2_approx(ref - next);
                ref = next;
                sum *= f;
                if (done > 0) scale_columns(o_col, D / 8, f);
            };
            for (uint32_t s = first; s < p.step1 && ok; s += stride, ++done) {
                ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.s_full[t], s_count++ & 1u, ctl, a.status));
                if (!ok) break;
                fence_after();
                if (warp_live) {
                    bool prefix;
                    uint32_t key, n;
                    step_keys(p, s, &prefix, &key, &n);
                    const uint32_t sees = prefix ? n : (limit > key ? min(n, limit - key) : 0u);
                    uint32_t absent = 0;
                    if (__builtin_expect(*reinterpret_cast<volatile uint32_t*>(&ctl.any_absent), 0))
                        absent = *reinterpret_cast<volatile uint32_t*>(&ctl.absent[t][(s_count - 1) % 8]);
                    const bool whole = n == kTileKeys && (prefix || key + kTileKeys <= all_see) && absent == 0;
                    uint32_t x[kTileKeys];
                    auto mask = [&](uint32_t half) {
                        if (__builtin_expect(whole, 1)) return;
#pragma unroll
                        for (uint32_t w = half * 2; w < half * 2 + 2; ++w) {
                            const uint32_t in = sees > w * 32 ? min(32u, sees - w * 32) : 0;  // keys of these 32 that are seen
                            const uint32_t real = (in ? 0xFFFFFFFFu >> (32 - in) : 0) &
                                                  ~((absent >> (2 * w) & 1 ? 0xFFFFu : 0u) | (absent >> (2 * w + 1) & 1 ? 0xFFFF0000u : 0u));
#pragma unroll
                            for (uint32_t j = 0; j < 32; ++j)
                                if (!(real >> j & 1)) x[w * 32 + j] = 0xFF800000u;  // -inf
                        }
                    };
                    auto half_most = [&](uint32_t half) {
                        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (uint32_t j = 0; j < 64; j += 2)
                            top[(j / 2) & 3] = fmaxf(top[(j / 2) & 3], fmaxf(__uint_as_float(x[half * 64 + j]), __uint_as_float(x[half * 64 + j + 1])));
                        return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
                    };
                    uint64_t add[2];
                    uint32_t w[32];
                    auto weigh = [&](const uint32_t* from) {
                        const uint64_t factor = pack2(scale, scale), base = ref == -INFINITY ? 0 : pack2(-ref, -ref);
                        add[0] = add[1] = 0;
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            float e0, e1;
                            unpack2(fma2(pack2(__uint_as_float(from[2 * j]), __uint_as_float(from[2 * j + 1])), factor, base), &e0, &e1);
                            e0 = exp2_approx(e0);
                            e1 = exp2_approx(e1);
                            add[j & 1] = add2(add[j & 1], pack2(e0, e1));
                            w[j] = Elem<T>::pack(e0, e1);  // rounded to the cache's type for the product with V; the sum keeps all bits
                        }
                    };
                    auto publish = [&](uint32_t half) {
                        tmem_store32(p_col + half * 32, w);
                        tmem_wait_store();
                        fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive(&ctl.p_full[t][half]);
                    };
                    auto added = [&]() {
                        float s0, s1;
                        unpack2(add2(add[0], add[1]), &s0, &s1);
                        return s0 + s1;
                    };
                    // The weights of the first half with the reference as it stands, while the second half is on its
                    // way; the maximum of the step is the next step's reference.  Only where it would lift a weight
                    // past 2^kHigh is the reference moved first and the half done again.
                    tmem_load32(s_col, x);
                    tmem_load32(s_col + 32, x + 32);
                    tmem_wait_load();
                    if (__builtin_expect(done > 0 && __any_sync(0xFFFFFFFFu, seen_most > ref + kRise), 0)) rebase(seen_most);
                    tmem_load32(s_col + 64, x + 64);
                    tmem_load32(s_col + 96, x + 96);
                    mask(0);
                    float most = half_most(0);
                    if (done == 0) ref = most - Elem<T>::kUp;
#pragma unroll 1
                    for (bool again = false;; again = true) {
                        weigh(x);
                        if (again) break;
                        tmem_wait_load();
                        mask(1);
                        most = fmaxf(most, half_most(1));
                        if (__builtin_expect(!__any_sync(0xFFFFFFFFu, most > ref + Elem<T>::kHigh), 1)) break;
                        rebase(most);
                    }
                    seen_most = most;
                    publish(0);
                    sum += added();
                    weigh(x + 64);
                    publish(1);
                    sum += added();
                } else {
                    fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        bar_arrive(&ctl.p_full[t][0]);
                        bar_arrive(&ctl.p_full[t][1]);
                    }
                }
            }
            if (!ok) break;
            if (done > 0) {
                ok = __all_sync(0xFFFFFFFFu, bar_wait(&ctl.pv_done[t], (pv_count + done - 1) & 1u, ctl, a.status));
                if (!ok) break;
                fence_after();
            }
            pv_count += done;
            if (warp_live) {
                uint32_t cta0, cta1;
                tile_ctas(g, p.h, head.share, &cta0, &cta1);
                const bool final = g.single && cta0 == cta1 && p.both;
                const uint32_t in_piece = p.both ? row : t * (walk.cta == cta0 ? g.rows : kTileRows) + row;
                const uint64_t pr = tile_part_row(g, p.h, cta0, walk.cta, a.L.extra_row) + in_piece;
                const bool empty = done == 0 || sum == 0.0f;  // nothing seen: zeros (with NaN among the scores the sum is NaN)
                const float inv = empty ? 0.0f : 1.0f / sum;
                // to the output only from a request's own tiles, whose tokens follow one another
                const uint32_t packed_row = g.row0 + row, tok = packed_row / a.group;
                const uint64_t token = g.token0 + tok, qh = p.h * a.group + (packed_row - tok * a.group);
                T* out = static_cast<T*>(a.out) + token * a.out_token + qh * a.out_head;
#pragma unroll 1
                for (uint32_t c = 0; done > 0 && c < D; c += 32) {
                    uint32_t o[32];
                    __syncwarp();
                    tmem_load32(o_col + c, o);
                    tmem_wait_load();
                    if (!live) continue;
                    if (!final) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) store_sector(part_o + pr * D + c + j, o + j);
                        continue;
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        w[j] = empty ? 0u : Elem<T>::pack(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                    if (reinterpret_cast<uintptr_t>(out) & 31u) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            reinterpret_cast<uint16_t*>(out)[c + j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
                    } else {
                        store_sector(out + c, w);
                        store_sector(out + c + 16, w + 8);
                    }
                }
                if (live) {
                    if (!final)
                        part_ml[pr] = make_float2(ref, sum);
                    else if (a.lse)
                        a.lse[token * (static_cast<uint64_t>(a.kv_heads) * a.group) + qh] =
                            empty ? -INFINITY : (ref + log2f(sum)) * kLn2;
                }
            }
            fence_before();  // O has been read before the next piece's products, which wait for this tile's weights
            __syncwarp();
        }
    }

    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// ---- host side -----------------------------------------------------------------------

struct PoolDim {
    uint64_t size, stride;  // elements
    uint32_t box, which;    // 0 token, 1 head, 2 page
};

// The pool's outer dimensions, smallest stride first; a dimension of one
// element may have any stride and goes last.
void pool_dims(const afx_kv_cache& c, PoolDim (&d)[3]) {
    d[0] = PoolDim{c.page_tokens, c.token_stride, c.page_tokens < kTileKeys ? c.page_tokens : kTileKeys, 0};
    d[1] = PoolDim{c.kv_heads, c.kv_heads > 1 ? c.head_stride : 0, 1, 1};
    d[2] = PoolDim{c.n_pages, c.n_pages > 1 ? c.page_stride : 0, 1, 2};
    auto after = [](const PoolDim& x, const PoolDim& y) { return x.size == 1 ? y.size != 1 : y.size != 1 && x.stride > y.stride; };
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2; ++j)
            if (after(d[j], d[j + 1])) {
                const PoolDim x = d[j];
                d[j] = d[j + 1];
                d[j + 1] = x;
            }
    for (int i = 0; i < 3; ++i)
        if (d[i].size == 1) d[i].stride = i ? d[i - 1].stride * d[i - 1].size : c.head_dim;
}

// A box is 64 elements of up to 128 tokens of a page's head.
afx_status pool_map(CUtensorMap* map, void* pool, const afx_kv_cache& c, const PoolDim (&d)[3]) {
    const EncodeFn enc = encode_fn();
    if (!enc) return afx_fail(AFX_E_CUDA, "cuTensorMapEncodeTiled is not available from the driver", 0);
    const cuuint64_t dims[4] = {c.head_dim, d[0].size, d[1].size, d[2].size};
    const cuuint64_t strides[3] = {2 * d[0].stride, 2 * d[1].stride, 2 * d[2].stride};
    const cuuint32_t box[4] = {64, d[0].box, d[1].box, d[2].box};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, c.format == AFX_FMT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, pool, dims,
                           strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        char msg[96];
        snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (CUresult %d)", static_cast<int>(r));
        return afx_fail(AFX_E_CUDA, msg, 0);
    }
    return AFX_OK;
}

template <typename T, int D>
afx_status launch(const TileArgs& args, cudaStream_t s) {
    // the row warps wait for the registers that they ask for: they must be there
    static Known known;
    uint64_t regs = 0;
    cudaError_t err = cudaSuccess;
    const bool told = known.get(&regs, [&](uint64_t* v) {
        cudaFuncAttributes at{};
        if ((err = cudaFuncGetAttributes(&at, attention_tile_kernel<T, D>)) == cudaSuccess) *v = static_cast<uint64_t>(at.numRegs);
        return err == cudaSuccess;
    });
    if (!told) {
        cudaGetLastError();
        return afx_fail(AFX_E_CUDA, "cudaFuncGetAttributes", err);
    }
    if (regs < kRegsLaunch) return afx_fail(AFX_E_CUDA, "attention_tile_kernel was built with too few registers", 0);
    AFX_SERVE_TRY(cudaFuncSetAttribute(attention_tile_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(Shape<D>::kSmem)),
                  "cudaFuncSetAttribute");
    AFX_SERVE_TRY(launch_early(attention_tile_kernel<T, D>, args.a.tile_ctas, kTileThreads, Shape<D>::kSmem, s, args), "attention_tile_kernel launch");
    return AFX_OK;
}

}  // namespace

bool tiles_fit(const afx_kv_cache& cache) {
    PoolDim d[3];
    pool_dims(cache, d);
    // a tensor map wants each stride to be a multiple of the one before it, and below 2^40 bytes
    return d[0].stride >= cache.head_dim && d[1].stride % d[0].stride == 0 && d[2].stride % d[1].stride == 0 &&
           2 * d[2].stride < (uint64_t{1} << 40);
}

afx_status launch_tiles(const AttnArgs& a, const afx_kv_cache& cache, cudaStream_t s) {
    TileArgs args;
    args.a = a;
    PoolDim d[3];
    pool_dims(cache, d);
    for (uint32_t i = 0; i < 3; ++i) {
        if (d[i].which == 0) args.token_at = i;
        if (d[i].which == 1) args.head_at = i;
    }
    afx_status st = pool_map(&args.k, cache.k_dev, cache, d);
    if (st == AFX_OK) st = pool_map(&args.v, cache.v_dev, cache, d);
    if (st != AFX_OK) return st;
    if (cache.format == AFX_FMT_BF16)
        return cache.head_dim == 128 ? launch<__nv_bfloat16, 128>(args, s) : launch<__nv_bfloat16, 64>(args, s);
    return cache.head_dim == 128 ? launch<__half, 128>(args, s) : launch<__half, 64>(args, s);
}

}  // namespace serve
}  // namespace afx
