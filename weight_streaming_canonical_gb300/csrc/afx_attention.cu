// sm_103a attention over paged keys and values for a batch that shares a
// long prefix (afx_attention_workspace, afx_attention_plan, afx_attention).
//
// Row (t, h) of the queries sees the prefix, common to the batch, and its
// own request's cached tokens up to its position.  With s = scale * q.k,
//     out = sum_j softmax(s)_j v_j,   lse = log sum_j e^(s_j).
// Two key sets A, B with running maxima m, sums l = sum e^(s - m) and
// weighted values o join as m = max(m_A, m_B), l = l_A e^(m_A - m) + l_B
// e^(m_B - m), and o likewise.  So the prefix is one problem for the whole
// batch: all tokens' rows of a key/value head (the "packed" rows, token by
// token, the G = q_heads / kv_heads heads of a token next to one another)
// against one copy of its keys, read once a row tile instead of once a
// request; each request's own tokens are a second, small problem; and long
// key ranges are cut into pieces that run side by side.  All of it is a
// list of items (a tile of packed rows x a range of keys) that one plan
// kernel writes a step (the lengths are on the GPU, and every layer of the
// step uses the same list), one attention kernel works off and one join
// kernel puts together in a fixed order.
//
// Two kernels work items off, side by side: the 16-row kernel here (mma.sync,
// every warp on its own: one or a few new tokens a request, where reading the
// keys is all) and the tile kernel (afx_attention_tile.cu: tcgen05, 256
// rows).  A request with 128 packed rows or more, a prompt, has tiles of its
// own that run over the prefix and its own keys in one go and mostly write
// the output themselves; the others share tiles on the prefix.
//
// Bound: few rows, the read of the cache (two requests on 131,000 common keys,
// 537 MB: 88 us, 6.1 TB/s, in the 16-row kernel); many rows, the products
// (see the tile kernel); small batches, the chain of plan, attention and join
// (4 requests on 1003 keys: each alone 6, 10 and 8 us).
//
// Times beside the constants below: one call of plan and attention between
// two events, caches flushed; both sides in one run.
#include <initializer_list>

#include "afx_attention.cuh"

namespace afx {
namespace serve {

afx_status check_cache(const afx_kv_cache* c, uint32_t* shift);  // afx_kv.cu

namespace {

constexpr uint32_t kPlanThreads = 1024;
constexpr uint32_t kMaxRequests = AFX_KV_MAX_REQUESTS;
constexpr uint32_t kKeyAlign = 64;     // 16-row items' key ranges start at multiples of this
constexpr uint32_t kMinKeys = 64;     // keys of a 16-row item, at least, where a range is cut
// 16-row items x heads that the cuts aim at: a unit a warp of the GPU (152 SMs
// of 8 warps), or two where there are many groups, of uneven lengths (64
// requests of 200 to 1000 tokens on 8192 in common: 78 us with two, 80 with
// one; two requests on 131,000 keys, whose join has more pieces with two: 117
// with one, 122 with two; 5 on 8000: 32 and 40).
constexpr uint32_t kTargetUnits = 2432, kFewUnits = 1216;
// Up to this many rows of a source go to the 16-row kernel, two groups reading
// the same keys, and a batch of no more rows goes without the tile kernel.  25
// rows on 500, 8000 and 64,000 keys: 24, 32 and 77 us, with the limit at 16
// rows 31-34, 43 and 88; two requests of 24 and 16 rows on 1284 keys each: 26
// and 47.  A limit of 48 costs 45 rows on 8000 and 64,000 keys 36 and 85 us
// where they take 43 and 88 now.
constexpr uint32_t kTileFrom = 32;
constexpr uint32_t kFuseRows = 128;    // packed rows from which a request's tiles take the prefix along
// Cost of a tile CTA, at least: one step where the other SMs would be idle (two
// prompts of 43 tokens, 24 heads on 2, on 600 keys 42 us, on 500 of their own
// 40; with twelve steps 57 and 59, with four 46 and 41).  Where the 16-row
// kernel has as much to do (a key of a head there takes an SM as long as a
// 16th of a unit of cost here), twelve, for a CTA's start costs as much as
// four steps: 64 requests with 8192 keys in common, 78 us, with one step 91.
constexpr uint32_t kMinShare = kStepBoth, kMinShareBeside = 12 * kStepBoth, kKeysOfCost = 16;
constexpr uint32_t kFewTokens = 8, kManyMax = 512;
constexpr uint32_t kManyPieces = 128;  // of a row, from which its join takes 16 warps

__host__ __device__ inline uint64_t up(uint64_t v, uint64_t a) { return (v + a - 1) / a * a; }

// ---- the plan ----------------------------------------------------------------------

template <int N>
struct Counts {
    uint64_t v[N];
};

// Exclusive sums over the CTA's threads; *total gets the sums.
template <int N>
__device__ Counts<N> block_exclusive(const Counts<N>& mine, Counts<N>* total) {
    __shared__ uint64_t warps[N][32], sums[N];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    Counts<N> inc = mine;
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t o = __shfl_up_sync(0xFFFFFFFFu, inc.v[i], d);
            if (lane >= d) inc.v[i] += o;
        }
        if (lane == 31) warps[i][warp] = inc.v[i];
    }
    __syncthreads();
    for (int i = warp; i < N; i += n_warps) {  // a warp a sum: the warps' totals
        const uint64_t x = lane < n_warps ? warps[i][lane] : 0;
        uint64_t y = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint64_t o = __shfl_up_sync(0xFFFFFFFFu, y, d);
            if (lane >= d) y += o;
        }
        warps[i][lane] = y - x;
        if (lane == 31) sums[i] = y;
    }
    __syncthreads();
    Counts<N> out;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        out.v[i] = warps[i][warp] + inc.v[i] - mine.v[i];
        total->v[i] = sums[i];
    }
    return out;
}

struct Many {
    uint32_t request, mark;
    RequestInfo own;
};

// How a request's rows are worked off.
struct Kind {
    uint32_t own;    // Source
    bool fused;      // its tiles take the prefix along (or there is none)
};

__device__ __forceinline__ Kind kind_of(const AttnArgs& a, uint32_t rows) {
    const bool tile = a.tile_ctas && rows > kTileFrom;
    return Kind{rows == 0 ? kNone : tile ? kTile : kRow16, a.prefix_len == 0 || (tile && rows >= kFuseRows)};
}

__device__ __forceinline__ uint32_t tile_cost(uint32_t rows, uint32_t prefix_keys, uint32_t own_keys) {
    const uint32_t steps = ceil_div(prefix_keys, kTileKeys) + ceil_div(own_keys, kTileKeys);
    return steps ? kGroupCost + step_cost(rows) * steps : 0;
}

// One CTA.  Requests' rows are cut into groups of 16 (or 256 for the tile
// kernel).  A 16-row group's keys are cut into pieces of `piece` keys, chosen
// so that all pieces x heads come to about kTargetUnits (enough to fill the
// GPU, and a bound on the workspace), but not below kMinKeys; the tile
// groups' cost is cut into one share a CTA.
__global__ void __launch_bounds__(kPlanThreads) attention_plan_kernel(const AttnArgs a) {
    PlanHead* head = a.at<PlanHead>(0);
    TokenInfo* tokens = a.at<TokenInfo>(a.L.tokens);
    int32_t* packed_token = a.at<int32_t>(a.L.packed_token);
    Row16Group* groups = a.at<Row16Group>(a.L.groups16);
    Row16Item* items = a.at<Row16Item>(a.L.items16);
    TileGroup* tiles = a.at<TileGroup>(a.L.tiles);
    const uint32_t R = a.n_requests, G = a.group;
    const uint32_t threads = blockDim.x, per = ceil_div(R, threads);
    const uint32_t r0 = min(R, threadIdx.x * per), r1 = min(R, r0 + per);
    const uint64_t max_len = static_cast<uint64_t>(a.table_cols) << a.shift;

    wait_for_earlier();
    let_next_start();
    __shared__ uint32_t n_many;
    __shared__ Many many[kManyMax];  // requests of more than a few tokens
    if (threadIdx.x == 0) {
        n_many = 0;
        *a.at<uint32_t>(a.L.counter) = 0;
    }
    // the lengths have to make sense before anything is addressed by them
    bool bad = false;
    Counts<3> first{};  // keys of the 16-row groups, tokens that share the prefix's groups, 16-row groups
    if (threadIdx.x == 0 && a.starts[0] != 0) bad = true;
    for (uint32_t r = r0; r < r1; ++r) {
        const int32_t s = a.starts[r], e = a.starts[r + 1], len = a.lens[r];
        if (s < 0 || e < s || static_cast<uint32_t>(e) > a.n_tokens || len < 0 || static_cast<uint64_t>(len) > max_len) {
            bad = true;
            continue;
        }
        const uint32_t rows = static_cast<uint32_t>(e - s) * G;
        const Kind k = kind_of(a, rows);
        if (k.own == kRow16)
            for (uint32_t row = 0; row < rows; row += kRows) {
                first.v[0] += visible(len - (e - s), min(rows, row + kRows) - 1, G);
                first.v[2] += 1;
            }
        if (!k.fused) first.v[1] += e - s;
    }
    const bool refused = __syncthreads_or(bad) != 0;
    if (refused) {
        if (threadIdx.x == 0) {
            raise(a.status, AFX_DEV_BAD_LENGTH);
            *head = PlanHead{a.plan_key, 0, 0, 0, 0, 0, kNone, 0, 0};
        }
        return;
    }
    Counts<3> all;
    uint32_t packed = static_cast<uint32_t>(block_exclusive(first, &all).v[1]);
    const uint32_t prefix_rows = static_cast<uint32_t>(all.v[1]) * G;
    const uint32_t prefix_kind = prefix_rows == 0 ? kNone : a.tile_ctas && prefix_rows > kTileFrom ? kTile : kRow16;
    const uint32_t groups_p = prefix_kind == kRow16 ? ceil_div(prefix_rows, kRows) : 0;
    const uint32_t tiles_p = prefix_kind == kTile ? ceil_div(prefix_rows, kGroupRows) : 0;
    const uint64_t keys = all.v[0] + static_cast<uint64_t>(groups_p) * a.prefix_len;
    const uint32_t target = (all.v[2] + groups_p) * a.kv_heads * 4 >= kFewUnits ? kTargetUnits : kFewUnits;
    const uint64_t units = target / a.kv_heads ? target / a.kv_heads : 1;
    const uint64_t want = up((keys + units - 1) / units, kKeyAlign);
    const uint32_t piece = static_cast<uint32_t>(want < kMinKeys ? kMinKeys : want < (1u << 31) ? want : 1u << 31);

    // the prefix of the tokens that share it
    const uint32_t pieces_p = groups_p ? ceil_div(a.prefix_len, piece) : 0;
    for (uint32_t g = threadIdx.x; g < groups_p; g += threads) {
        const uint32_t row0 = g * kRows;
        groups[g] = Row16Group{row0 * pieces_p, pieces_p, min(kRows, prefix_rows - row0), 0};
    }
    for (uint32_t i = threadIdx.x; i < groups_p * pieces_p; i += threads) {
        // piece by piece, so that the groups that read the same keys run together
        const uint32_t s = i / groups_p, row0 = (i % groups_p) * kRows, rows = min(kRows, prefix_rows - row0);
        items[i] = Row16Item{-1, row0, rows, s * piece, min(a.prefix_len, (s + 1) * piece), row0 * pieces_p + s * rows, 0, 0};
    }
    auto write_token = [&](uint32_t r, uint32_t t, uint32_t mark, uint32_t i, const RequestInfo& own) {
        tokens[t] = TokenInfo{r, i * G, mark >= kInTiles ? mark : mark + i, 0, own};
        if (mark < kInTiles) packed_token[mark + i] = static_cast<int32_t>(t);
    };
    // not written by the tile kernel: two tiles' sums, or none
    auto rests = [](uint32_t m, uint32_t keys, bool single) { return single && (m <= kTileRows || keys == 0); };
    // the requests' own keys
    auto walk = [&](uint32_t r, auto&& row16, auto&& tile) {
        const uint32_t s = a.starts[r], n = a.starts[r + 1] - s, rows = n * G;
        const int32_t seen = a.lens[r] - static_cast<int32_t>(n);
        const Kind k = kind_of(a, rows);
        if (k.own == kRow16)
            for (uint32_t row = 0; row < rows; row += kRows) {
                const uint32_t m = min(kRows, rows - row);
                row16(row, m, visible(seen, row + m - 1, G), s, seen);
            }
        if (k.own == kTile)
            for (uint32_t row = 0; row < rows; row += kGroupRows) {
                const uint32_t m = min(kGroupRows, rows - row);
                tile(row, m, k.fused ? a.prefix_len : 0u, visible(seen, row + m - 1, G), s, seen, k.fused);
            }
    };
    // groups | tile groups << 32, pieces, their rows, cost, rows of tile pieces, rest | tokens by row << 32
    constexpr uint64_t kHigh = 1ull << 32;
    Counts<6> mine{};
    for (uint32_t r = r0; r < r1; ++r) {
        const uint32_t n = a.starts[r + 1] - a.starts[r];
        const Kind k = kind_of(a, n * G);
        if (!(k.fused && k.own == kTile)) mine.v[5] += kHigh * n;
        walk(
            r,
            [&](uint32_t, uint32_t m, uint32_t end, uint32_t, int32_t) {
                const uint32_t pieces = ceil_div(end, piece);
                mine.v[0] += 1;
                mine.v[1] += pieces;
                mine.v[2] += static_cast<uint64_t>(pieces) * m;
            },
            [&](uint32_t, uint32_t m, uint32_t prefix, uint32_t own, uint32_t, int32_t, bool single) {
                mine.v[0] += kHigh;
                mine.v[3] += static_cast<uint64_t>(tile_cost(m, prefix, own)) * a.kv_heads;
                mine.v[4] += static_cast<uint64_t>(m > kTileRows ? m : 2 * m) * a.kv_heads;
                mine.v[5] += rests(m, prefix + own, single);
            });
    }
    Counts<6> total;
    const Counts<6> at = block_exclusive(mine, &total);
    const uint32_t n_tiles = tiles_p + static_cast<uint32_t>(total.v[0] >> 32);
    const uint32_t cost_full = tile_cost(kGroupRows, a.prefix_len, 0);
    const uint64_t tile_row0 = a.L.max_rows;  // rows of the tile kernel's first pieces start here
    uint64_t cost_p = 0, rows_p = 0;
    if (tiles_p) {
        for (uint32_t g = threadIdx.x; g < tiles_p; g += threads) {
            const uint32_t row0 = g * kGroupRows, rows = min(kGroupRows, prefix_rows - row0);
            tiles[g] = TileGroup{static_cast<uint64_t>(g) * cost_full * a.kv_heads, tile_row0 + static_cast<uint64_t>(row0) * a.kv_heads,
                                 tile_cost(rows, a.prefix_len, 0), -1, row0, rows, a.prefix_len, 0, 0, 0, 0, {}};
        }
        const uint32_t last = prefix_rows - (tiles_p - 1) * kGroupRows;
        cost_p = (static_cast<uint64_t>(tiles_p - 1) * cost_full + tile_cost(last, a.prefix_len, 0)) * a.kv_heads;
        rows_p = (static_cast<uint64_t>(tiles_p - 1) * kGroupRows + (last > kTileRows ? last : 2 * last)) * a.kv_heads;
    }
    uint32_t g = static_cast<uint32_t>(at.v[0]) + groups_p, it = static_cast<uint32_t>(at.v[1]) + groups_p * pieces_p,
             pr = static_cast<uint32_t>(at.v[2]) + (groups_p ? prefix_rows * pieces_p : 0), tg = static_cast<uint32_t>(at.v[0] >> 32) + tiles_p;
    uint32_t* rest = a.at<uint32_t>(a.L.rest) + static_cast<uint32_t>(at.v[5]);
    uint64_t cost = at.v[3] + cost_p, trow = tile_row0 + at.v[4] + rows_p;
    for (uint32_t r = r0; r < r1; ++r) {
        const uint32_t s = a.starts[r], e = a.starts[r + 1];
        const Kind k = kind_of(a, (e - s) * G);
        const RequestInfo own{k.own, k.own == kTile ? tg : g, {}};
        walk(
            r,
            [&](uint32_t row, uint32_t m, uint32_t end, uint32_t token0, int32_t seen) {
                const uint32_t pieces = ceil_div(end, piece);
                groups[g++] = Row16Group{pr, pieces, m, 0};
                for (uint32_t p = 0; p < pieces; ++p, pr += m)
                    items[it++] = Row16Item{static_cast<int32_t>(r), row, m, p * piece, min(end, (p + 1) * piece), pr, token0, seen};
            },
            [&](uint32_t row, uint32_t m, uint32_t prefix, uint32_t own, uint32_t token0, int32_t seen, bool single) {
                const uint32_t c = tile_cost(m, prefix, own);
                if (rests(m, prefix + own, single)) *rest++ = tg;
                tiles[tg++] = TileGroup{cost, trow, c, static_cast<int32_t>(r), row, m, prefix, own, token0, seen, single, {}};
                cost += static_cast<uint64_t>(c) * a.kv_heads;
                trow += static_cast<uint64_t>(m > kTileRows ? m : 2 * m) * a.kv_heads;
            });
        // its tokens: a few here, more by a warp below
        const uint32_t mark = k.fused ? (k.own == kTile ? kInTiles : kAlone) : packed;
        if (e - s <= kFewTokens) {
            for (uint32_t t = s; t < e; ++t) write_token(r, t, mark, t - s, own);
        } else {
            const uint32_t i = atomicAdd(&n_many, 1u);
            if (i < kManyMax)
                many[i] = Many{r, mark, own};
            else
                for (uint32_t t = s; t < e; ++t) write_token(r, t, mark, t - s, own);
        }
        if (!k.fused) packed += e - s;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x / 32; i < min(n_many, kManyMax); i += threads / 32) {
        const Many m = many[i];
        const uint32_t s = a.starts[m.request], e = a.starts[m.request + 1];
        for (uint32_t t = s + threadIdx.x % 32; t < e; t += 32) write_token(m.request, t, m.mark, t - s, m.own);
    }
    if (threadIdx.x == 0) {
        const uint64_t c = total.v[3] + cost_p, ctas = a.tile_ctas ? a.tile_ctas : 1;
        const uint64_t share = (c + ctas - 1) / ctas;
        const uint32_t n_items = groups_p * pieces_p + static_cast<uint32_t>(total.v[1]);
        const uint64_t least = keys * a.kv_heads >= kKeysOfCost * c ? kMinShareBeside : kMinShare;
        *head = PlanHead{a.plan_key, c, share < least ? least : share, static_cast<uint32_t>(a.starts[R]), n_items, n_tiles, prefix_kind, static_cast<uint32_t>(total.v[5]), static_cast<uint32_t>(total.v[5] >> 32)};
    }
}

// ---- 16 packed rows x a range of keys ------------------------------------------------

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

constexpr int kWarps = 4;
constexpr int kBlockKeys = 16;  // keys of one step of a warp; divides every page size
constexpr int kStages = 3;

template <int D>
constexpr size_t rows16_smem() {
    return static_cast<size_t>(kWarps) * kStages * 2 * kBlockKeys * D * 2;
}

// A unit is an item's rows and keys of one key/value head; every warp takes
// units on its own, steps of 16 keys, with no barrier anywhere: the next one
// from a counter, for many CTAs start only when one of the tile kernel's ends
// (64 requests of 200 to 1000 tokens: 23 us after its last one's end with
// every warp's units fixed).  Its copies
// run kStages - 1 steps ahead, over the ends of units, so that memory stays
// busy while a unit's results are written and the next one's queries loaded.
// Two CTAs an SM: 8 warps with 16 KB each in flight.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32, 2) attention_rows16_kernel(const AttnArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kChunks = D / 8;                     // 16-byte chunks of a key
    constexpr uint32_t kTile = kBlockKeys * D * 2;     // bytes of a step's keys
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // The plan was done before the tile kernel, which let this one start, and
    // the two kernels' results do not meet: they run side by side, and only
    // the end of this one waits for the end of that one.
    if (!a.tile_ctas) wait_for_earlier();
    let_next_start();
    const PlanHead head = *a.at<PlanHead>(0);
    if (head.key != a.plan_key && threadIdx.x == 0) raise(a.status, AFX_DEV_BAD_PLAN);
    const uint32_t n_units = head.key == a.plan_key ? head.n_items * a.kv_heads : 0;
    uint32_t* counter = a.at<uint32_t>(a.L.counter);
    __shared__ uint32_t rings[kWarps][4];  // units whose copies have begun: the copies are at most four units ahead
    uint32_t* ring = rings[warp];
    uint32_t opened = 0;
    const Row16Item* items = a.at<Row16Item>(a.L.items16);
    const int32_t* packed = a.at<int32_t>(a.L.packed_token);
    float* part_o = a.at<float>(a.L.part_o);
    float2* part_ml = a.at<float2>(a.L.part_ml);
    const T* q = static_cast<const T*>(a.q);
    const T* kp = static_cast<const T*>(a.k);
    const T* vp = static_cast<const T*>(a.v);
    const uint32_t mine = smem_addr(smem) + warp * (kStages * 2 * kTile);
    const uint32_t page_mask = (1u << a.shift) - 1;

    // the copies: unit c_unit's step c_block goes into stage c_stage
    uint32_t c_unit = 0, c_block = 0, c_blocks = 0, c_key0 = 0, c_key1 = 0, c_stage = 0;
    uint64_t c_head = 0;
    const int32_t* c_pages = nullptr;
    uint32_t c_page = 0;  // lane l: the page of step c_block / 32 * 32 + l
    uint32_t c_gone = 0;  // a bit each of these 32 steps: the page lies outside the pool, the keys are left out
    uint32_t absent = 0;  // the same, a bit a stage
    auto open = [&]() {
        if (lane == 0) {
            c_unit = atomicAdd(counter, 1u);
            ring[opened & 3] = c_unit;
        }
        c_unit = __shfl_sync(0xFFFFFFFFu, c_unit, 0);
        ++opened;
        if (c_unit >= n_units) return;
        const Row16Item& it = items[c_unit / a.kv_heads];
        c_key0 = it.key0;
        c_key1 = it.key1;
        c_blocks = ceil_div(c_key1 - c_key0, kBlockKeys);
        c_block = 0;
        c_head = (c_unit % a.kv_heads) * a.head_stride;
        c_pages = it.request < 0 ? a.prefix_table : a.table + static_cast<uint64_t>(it.request) * a.table_cols;
    };
    auto copy_next = [&]() {
        if (c_unit < n_units) {
            if (c_block % 32 == 0) {  // 32 steps' pages at a time
                const uint32_t i = c_block + lane;
                const int32_t id = i < c_blocks ? __ldg(c_pages + ((c_key0 + i * kBlockKeys) >> a.shift)) : 0;
                const bool gone = id < 0 || static_cast<uint32_t>(id) >= a.n_pages;
                if (gone) raise(a.status, AFX_DEV_BAD_PAGE);
                c_page = gone ? 0 : id;
                c_gone = __ballot_sync(0xFFFFFFFFu, gone);
            }
            const uint32_t key = c_key0 + c_block * kBlockKeys;
            uint32_t end = c_key1;
            if (c_gone | absent) {
                const uint32_t gone = c_gone >> (c_block % 32) & 1;
                absent = (absent & ~(1u << c_stage)) | gone << c_stage;
                if (gone) end = 0;
            }
            const uint64_t page = __shfl_sync(0xFFFFFFFFu, c_page, c_block % 32);
            // a lane copies every (32 / kChunks)-th key from its own on, the same 16 bytes of each
            const uint32_t row0 = lane / kChunks, chunk = lane % kChunks;
            const uint64_t from = page * a.page_stride + c_head + ((key & page_mask) + row0) * a.token_stride + chunk * 8;
            const T* k_from = kp + from;
            const T* v_from = vp + from;
            const uint64_t hop = (32 / kChunks) * a.token_stride;
            const uint32_t buf = mine + c_stage * 2 * kTile;
#pragma unroll
            for (int c = 0; c < kBlockKeys * kChunks / 32; ++c) {
                const uint32_t row = c * (32 / kChunks) + row0;
                const bool real = key + row < end;  // past the range: zeros, whatever the page holds there
                const uint32_t dst = buf + row * (D * 2) + ((chunk ^ (row & 7)) * 16);
                copy16(dst, k_from, real);
                copy16(dst + kTile, v_from, real);
                k_from += hop;
                v_from += hop;
            }
            if (++c_block == c_blocks) open();
            c_stage = c_stage + 1 == kStages ? 0 : c_stage + 1;
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    if (n_units) open();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) copy_next();

    uint32_t stage = 0;
    for (uint32_t done = 0; done < opened; ++done) {
        __syncwarp();
        const uint32_t unit = ring[done & 3];
        if (unit >= n_units) break;
        const Row16Item it = items[unit / a.kv_heads];
        const uint32_t h = unit % a.kv_heads;
        // the queries as A fragments: rows lane / 4 and lane / 4 + 8
        uint32_t qf[D / 16][4];
        uint32_t limit[2];  // keys the row sees
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint32_t i = lane / 4 + half * 8, row = it.row0 + i;
            const bool live = i < it.rows;
            limit[half] = it.request < 0 || !live ? UINT32_MAX : visible(it.seen, row, a.group);
            const uint64_t token = !live ? 0 : it.request < 0 ? packed[row / a.group] : it.token0 + row / a.group;
            const T* src = q + token * a.q_token + (h * a.group + row % a.group) * a.q_head + (lane % 4) * 2;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t v = 0;
                    if (live) {
                        const T* s = src + ks * 16 + kk * 8;
                        if (a.q_align >= 4)
                            v = *reinterpret_cast<const uint32_t*>(s);
                        else
                            v = *reinterpret_cast<const uint16_t*>(s) |
                                static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(s + 1)) << 16;
                    }
                    qf[ks][kk * 2 + half] = v;
                }
        }
        const uint32_t min_limit = it.request < 0 ? UINT32_MAX : visible(it.seen, it.row0, a.group);

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][j] = 0.0f;
        constexpr float kRise = kLag + Elem<T>::kUp;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};  // references and sums

        for (uint32_t key = it.key0; key < it.key1; key += kBlockKeys) {
            copy_next();
            asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 1) : "memory");
            __syncwarp();
            const uint32_t buf = mine + stage * 2 * kTile;
            const uint32_t at_stage = 1u << stage;
            stage = stage + 1 == kStages ? 0 : stage + 1;
            float s[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b[4];
                const uint32_t row = (lane / 16) * 8 + lane % 8, chunk = ks * 2 + ((lane / 8) & 1);
                ldmatrix4(b, buf + row * (D * 2) + ((chunk ^ (row & 7)) * 16));
                Elem<T>::mma(s[0], qf[ks], b[0], b[1]);
                Elem<T>::mma(s[1], qf[ks], b[2], b[3]);
            }
            const bool whole = key + kBlockKeys <= it.key1 && key + kBlockKeys <= min_limit && absent == 0;
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float x = s[n][j] * a.scale_log2;
                    const uint32_t kk = key + n * 8 + (lane % 4) * 2 + (j & 1);
                    if (!whole && (absent & at_stage || kk >= it.key1 || kk >= limit[j >> 1])) x = -INFINITY;
                    s[n][j] = x;
                    top[j >> 1] = fmaxf(top[j >> 1], x);
                }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                top[half] = fmaxf(top[half], __shfl_xor_sync(0xFFFFFFFFu, top[half], 1));
                top[half] = fmaxf(top[half], __shfl_xor_sync(0xFFFFFFFFu, top[half], 2));
            }
            if (__any_sync(0xFFFFFFFFu, top[0] > m[0] + kRise || top[1] > m[1] + kRise)) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float next = fmaxf(m[half], top[half] - Elem<T>::kUp);
                    const float f = next == -INFINITY ? 1.0f : exp2_approx(m[half] - next);
                    m[half] = next;
                    l[half] *= f;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][half * 2] *= f;
                        o[n][half * 2 + 1] *= f;
                    }
                }
            }
            const float ref[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[n][j] = exp2_approx(s[n][j] - ref[j >> 1]);
                    l[j >> 1] += s[n][j];
                }
            // the weights as A fragments, rounded to the cache's type for
            // the product with V (the sums above keep all their bits)
            const uint32_t p[4] = {Elem<T>::pack(s[0][0], s[0][1]), Elem<T>::pack(s[0][2], s[0][3]),
                                   Elem<T>::pack(s[1][0], s[1][1]), Elem<T>::pack(s[1][2], s[1][3])};
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                const uint32_t row = ((lane / 8) & 1) * 8 + lane % 8, chunk = n * 2 + lane / 16;
                ldmatrix4_t(b, buf + kTile + row * (D * 2) + ((chunk ^ (row & 7)) * 16));
                Elem<T>::mma(o[n * 2], p, b[0], b[1]);
                Elem<T>::mma(o[n * 2 + 1], p, b[2], b[3]);
            }
            __syncwarp();  // the stage is read before it is filled again
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 1);
            l[half] += __shfl_xor_sync(0xFFFFFFFFu, l[half], 2);
            const uint32_t row = lane / 4 + half * 8;
            if (row < it.rows) {
                const uint64_t at = static_cast<uint64_t>(it.part_row + row) * a.kv_heads + h;
                if (lane % 4 == 0) part_ml[at] = make_float2(m[half], l[half]);
                float2* to = reinterpret_cast<float2*>(part_o + at * D + (lane % 4) * 2);
#pragma unroll
                for (int n = 0; n < D / 8; ++n) to[n * 4] = make_float2(o[n][half * 2], o[n][half * 2 + 1]);
            }
        }
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    if (a.tile_ctas) wait_for_earlier();
}

// ---- the join ------------------------------------------------------------------------

// The pieces of one row's results: the prefix's (where the row shares it),
// then those of its request's own keys.
struct Pieces {
    uint32_t n16, n_tile, ctas, rows16, group_rows;
    uint64_t at16, step16;               // 16-row pieces: first row, distance
    uint64_t first, further;             // tile pieces: of the first CTA, of the CTAs after it
    uint32_t in, two;

    __device__ uint32_t count() const { return n16 + n_tile; }
    __device__ uint64_t row(uint32_t p) const {
        if (p < n16) return at16 + p * step16;
        p -= n16;
        const uint32_t cta = two ? p / 2 : p, lane = two ? p % 2 : 0;
        return cta == 0 ? first + lane * group_rows + in : further + static_cast<uint64_t>(cta - 1) * kGroupRows + lane * kTileRows + in;
    }
};

__device__ __forceinline__ Pieces pieces_of(const AttnArgs& a, const PlanHead& head, uint32_t kind, uint32_t first_group, uint32_t row,
                                            uint32_t h) {
    Pieces p{};
    if (kind == kRow16) {
        const Row16Group g = a.at<Row16Group>(a.L.groups16)[first_group + row / kRows];
        p.n16 = g.n_pieces;
        p.at16 = static_cast<uint64_t>(g.part_row + row % kRows) * a.kv_heads + h;
        p.step16 = static_cast<uint64_t>(g.rows) * a.kv_heads;
    } else if (kind == kTile) {
        const TileGroup g = a.at<TileGroup>(a.L.tiles)[first_group + row / kGroupRows];
        if (g.cost) {
            uint32_t c0, c1;
            tile_ctas(g, h, head.share, &c0, &c1);
            p.two = g.rows <= kTileRows;
            p.n_tile = (c1 - c0 + 1) * (p.two ? 2 : 1);
            p.group_rows = g.rows;
            p.in = row % kGroupRows;
            p.first = tile_part_row(g, h, c0, c0, a.L.extra_row);
            p.further = tile_part_row(g, h, c0, c0 + 1, a.L.extra_row);
        }
    }
    return p;
}

constexpr int kJoinThreads = 128, kJoinWarps = kJoinThreads / 32, kSplitThreads = 512;
constexpr uint32_t kJoinRows = 8;  // rows of a tile group that a warp puts together at a time

// A lane's elements of an output row, in one store where its address allows.
template <typename T, int N>
__device__ __forceinline__ void store_row(T* out, const float (&v)[N]) {
    if (reinterpret_cast<uintptr_t>(out) & (N * 2 - 1)) {
#pragma unroll
        for (int j = 0; j < N; ++j) out[j] = Elem<T>::from(v[j]);
    } else if constexpr (N == 4) {
        *reinterpret_cast<uint2*>(out) = make_uint2(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]));
    } else {
        *reinterpret_cast<uint32_t*>(out) = Elem<T>::pack(v[0], v[1]);
    }
}

// A lane's elements of a piece's row.
template <int N>
__device__ __forceinline__ void load_part(const float* from, float (&v)[N]) {
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const float2 x = *reinterpret_cast<const float2*>(from);
        v[0] = x.x, v[1] = x.y;
    }
}

// Whether a piece has a key that the row sees: its maximum is minus infinity
// also where all scores are NaN (a maximum passes over them), but not its sum 0.
__device__ __forceinline__ bool has_keys(float2 ml) { return ml.x != -INFINITY || ml.y != 0.0f; }

// Eight rows of a tile group's head, put together from its pieces by a warp.
template <typename T, int D>
__device__ void join_group_rows(const AttnArgs& a, const TileGroup& g, uint32_t h, uint32_t row0, uint32_t c0, uint32_t c1) {
    constexpr int kPer = D / 32;
    const int lane = threadIdx.x & 31;
    const uint32_t q_heads = a.kv_heads * a.group, rows = g.rows;
    const float* part_o = a.at<float>(a.L.part_o);
    const float2* part_ml = a.at<float2>(a.L.part_ml);
    constexpr uint32_t kAtOnce = 2;  // pieces taken at a time (mostly there are two): lane = 8 piece + row, twice
    const uint32_t lanes = rows <= kTileRows ? 2 : 1, n = g.cost ? (c1 - c0 + 1) * lanes : 0;
    const uint32_t slot = lane / kJoinRows % kAtOnce, mine = min(row0 + lane % kJoinRows, rows - 1);
    float top = -INFINITY, sum = 0.0f, acc[kJoinRows][kPer] = {};
#pragma unroll 1
    for (uint32_t base = 0; base < n; base += kAtOnce) {
        const uint32_t p = min(base + slot, n - 1), c = c0 + p / lanes;
        const uint64_t row = tile_part_row(g, h, c0, c, a.L.extra_row) + (p % lanes) * (c == c0 ? rows : kTileRows) + mine;
        float v[kJoinRows][kAtOnce][kPer];  // all loads, then all sums
#pragma unroll
        for (uint32_t r = 0; r < kJoinRows; ++r)
#pragma unroll
            for (uint32_t q = 0; q < kAtOnce; ++q) load_part(part_o + __shfl_sync(0xFFFFFFFFu, row, q * kJoinRows + r) * D + lane * kPer, v[r][q]);
        const float2 ml = base + slot < n ? part_ml[row] : make_float2(-INFINITY, 0.0f);
        const float most = fmaxf(top, fmaxf(ml.x, __shfl_xor_sync(0xFFFFFFFFu, ml.x, 8)));
        const float ref = most == -INFINITY ? 0.0f : most, keep = exp2_approx(top - ref), f = exp2_approx(ml.x - ref);
        top = most;
        const float part = f * ml.y;
        sum = sum * keep + (part + __shfl_xor_sync(0xFFFFFFFFu, part, 8));
        const uint32_t real = __ballot_sync(0xFFFFFFFFu, has_keys(ml));  // of the others the sums may never have been written
#pragma unroll
        for (uint32_t r = 0; r < kJoinRows; ++r) {
            const float k = __shfl_sync(0xFFFFFFFFu, keep, r);
#pragma unroll
            for (int j = 0; j < kPer; ++j) acc[r][j] *= k;
#pragma unroll
            for (uint32_t q = 0; q < kAtOnce; ++q) {
                const float fr = __shfl_sync(0xFFFFFFFFu, f, q * kJoinRows + r);
#pragma unroll
                for (int j = 0; j < kPer; ++j) acc[r][j] += real >> (q * kJoinRows + r) & 1 ? fr * v[r][q][j] : 0.0f;
            }
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const uint32_t pr = g.row0 + mine, tok = pr / a.group, token = g.token0 + tok, qh = h * a.group + (pr - tok * a.group);
    if (a.lse && lane < static_cast<int>(kJoinRows) && row0 + lane < rows)
        a.lse[static_cast<uint64_t>(token) * q_heads + qh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    const uint64_t dst = token * a.out_token + qh * a.out_head;
#pragma unroll
    for (uint32_t r = 0; r < kJoinRows; ++r) {
        const float scale = __shfl_sync(0xFFFFFFFFu, inv, r);
        const uint64_t to = __shfl_sync(0xFFFFFFFFu, dst, r);
        if (row0 + r < rows) {
            float o[kPer];
#pragma unroll
            for (int j = 0; j < kPer; ++j) o[j] = acc[r][j] * scale;
            store_row<T, kPer>(static_cast<T*>(a.out) + to + lane * kPer, o);
        }
    }
}

// Rows in tiles of their request's own: mostly the tile kernel has written
// the output.  What is left are group heads that the border between two CTAs'
// shares cuts, found from the borders, those without keys, and those of 128
// rows or fewer, whose two tiles took steps in turn.
template <typename T, int D>
__device__ void join_tiles(const AttnArgs& a, const PlanHead& head, uint32_t block, uint32_t blocks) {
    const TileGroup* tiles = a.at<TileGroup>(a.L.tiles);
    const uint32_t per = blockDim.x / 32, warps = blocks * per, me = block * per + (threadIdx.x >> 5);
    const uint32_t borders = head.cost ? static_cast<uint32_t>((head.cost - 1) / head.share) : 0;
    constexpr uint32_t kUnits = kGroupRows / kJoinRows;
    for (uint32_t u = me; u < borders * kUnits; u += warps) {
        const uint32_t b = u / kUnits + 1, row0 = u % kUnits * kJoinRows;
        const TileGroup& g = tiles[a.at<uint32_t>(a.L.tile_first)[b]];
        if (!g.single || g.rows <= kTileRows || row0 >= g.rows || !g.cost) continue;
        const uint32_t h = divide(b * head.share - g.cost_begin, g.cost);
        uint32_t c0, c1;
        tile_ctas(g, h, head.share, &c0, &c1);
        if (c0 + 1 == b && c1 >= b) join_group_rows<T, D>(a, g, h, row0, c0, c1);
    }
    for (uint32_t u = me; u < head.n_rest * a.kv_heads * kUnits; u += warps) {
        const uint32_t row0 = u % kUnits * kJoinRows, gh = u / kUnits, h = gh % a.kv_heads;
        const TileGroup& g = tiles[a.at<uint32_t>(a.L.rest)[gh / a.kv_heads]];
        if (row0 >= g.rows) continue;
        uint32_t c0 = 0, c1 = 0;
        if (g.cost) tile_ctas(g, h, head.share, &c0, &c1);
        join_group_rows<T, D>(a, g, h, row0, c0, c1);
    }
}

// Rows outside tiles of their request's own, span at a time a warp (kSplit: one
// row a CTA, whose warps, 4 or 16, share its pieces: few rows, each of many), then
// join_tiles.  Pieces are added in a fixed order.
template <typename T, int D, bool kSplit>
__global__ void __launch_bounds__(kSplit ? kSplitThreads : kJoinThreads) attention_join_kernel(const AttnArgs a, uint32_t span) {
    constexpr int kPer = D / 32;
    constexpr int kMostWarps = kSplit ? kSplitThreads / 32 : 1;
    __shared__ float sh_acc[kMostWarps][D];
    __shared__ float2 sh_ml[kMostWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t q_heads = a.kv_heads * a.group;
    wait_for_earlier();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.at<uint32_t>(a.L.counter) = 0;  // for the next layer
    const PlanHead head = *a.at<PlanHead>(0);
    if (head.key != a.plan_key) return;
    const uint32_t n_rows = head.n_tokens * q_heads;  // below 2^31

    struct Sources {
        Pieces pre, own;
        uint32_t t, qh;
    };
    auto sources = [&](uint32_t w) {
        Sources s;
        s.t = w / q_heads;
        s.qh = w - s.t * q_heads;
        const TokenInfo info = a.at<TokenInfo>(a.L.tokens)[s.t];
        const uint32_t h = s.qh / a.group, gh = s.qh - h * a.group;
        s.own = pieces_of(a, head, info.own.kind, info.own.first, info.row + gh, h);
        s.pre = pieces_of(a, head, info.packed >= kInTiles ? static_cast<uint32_t>(kNone) : head.prefix_kind, 0, info.packed * a.group + gh, h);
        return s;
    };
    auto join = [&](const Sources& s) {
        const float* part_o = a.at<float>(a.L.part_o);
        const float2* part_ml = a.at<float2>(a.L.part_ml);
        float top = -INFINITY, sum = 0.0f, acc[kPer] = {};
        const uint32_t n = s.pre.count() + s.own.count();
        const uint32_t step = kSplit ? blockDim.x / 32 : 1;
        const uint32_t off = kSplit ? warp : 0;  // this warp's pieces: off, off + step, ...
        for (uint32_t b = off; b < n; b += 32 * step) {
            const uint32_t p = b + lane * step;
            const uint64_t row = p >= n ? 0 : p < s.pre.count() ? s.pre.row(p) : s.own.row(p - s.pre.count());
            const float2 ml = p < n ? part_ml[row] : make_float2(-INFINITY, 0.0f);
            float most = fmaxf(top, ml.x);
#pragma unroll
            for (int d = 16; d; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, d));
            const bool real = has_keys(ml);  // else its sums may never have been written
            const uint32_t live = __ballot_sync(0xFFFFFFFFu, real);
            if (!live) continue;  // none of these pieces has a key that the row sees
            const float ref = most == -INFINITY ? 0.0f : most, keep = exp2_approx(top - ref);
            top = most;
            sum *= keep;
#pragma unroll
            for (int j = 0; j < kPer; ++j) acc[j] *= keep;
            const float f = real ? exp2_approx(ml.x - ref) : 0.0f;
            float part = f * ml.y;
            const uint32_t m = min(32u, ceil_div(n - b, step));
#pragma unroll
            for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(0xFFFFFFFFu, part, d);
            sum += part;
            constexpr uint32_t kAtOnce = kSplit ? 8 : 4;  // loads in flight; past the last piece: row 0
            for (uint32_t j = 0; j < m; j += kAtOnce) {
                float v[kAtOnce][kPer];
#pragma unroll
                for (uint32_t i = 0; i < kAtOnce; ++i) load_part(part_o + __shfl_sync(0xFFFFFFFFu, row, j + i) * D + lane * kPer, v[i]);
#pragma unroll
                for (uint32_t i = 0; i < kAtOnce; ++i) {
                    const float fj = __shfl_sync(0xFFFFFFFFu, f, j + i);
#pragma unroll
                    for (int k = 0; k < kPer; ++k) acc[k] += live >> (j + i) & 1 ? fj * v[i][k] : 0.0f;
                }
            }
        }
        if constexpr (kSplit) {
            if (lane == 0) sh_ml[warp] = make_float2(top, sum);
#pragma unroll
            for (int j = 0; j < kPer; ++j) sh_acc[warp][lane * kPer + j] = acc[j];
            __syncthreads();
            if (warp) return;  // the first warp goes on
            top = -INFINITY;
            sum = 0.0f;
            for (uint32_t w = 0; w < step; ++w) top = fmaxf(top, sh_ml[w].x);
#pragma unroll
            for (int j = 0; j < kPer; ++j) acc[j] = 0.0f;
            const float ref = top == -INFINITY ? 0.0f : top;
            for (uint32_t w = 0; w < step; ++w) {
                const float f = exp2_approx(sh_ml[w].x - ref);
                sum += f * sh_ml[w].y;
#pragma unroll
                for (int j = 0; j < kPer; ++j) acc[j] += f * sh_acc[w][lane * kPer + j];
            }
        }
        // a row that sees no key: zeros, and the logarithm of an empty sum
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        T* out = static_cast<T*>(a.out) + s.t * a.out_token + s.qh * a.out_head + lane * kPer;
#pragma unroll
        for (int j = 0; j < kPer; ++j) acc[j] *= inv;
        store_row<T, kPer>(out, acc);
        if (a.lse && lane == 0)
            a.lse[static_cast<uint64_t>(s.t) * q_heads + s.qh] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    };
    const TokenInfo* tokens = a.at<TokenInfo>(a.L.tokens);
    if constexpr (kSplit) {
        if (blockIdx.x < n_rows && tokens[blockIdx.x / q_heads].packed != kInTiles) join(sources(blockIdx.x));
    } else if (head.n_by_row) {
        for (uint64_t at = static_cast<uint64_t>(blockIdx.x * kJoinWarps + warp) * span; at < n_rows; at += static_cast<uint64_t>(gridDim.x) * kJoinWarps * span) {
            const uint32_t base = static_cast<uint32_t>(at);
            bool todo = false;
            if (static_cast<uint32_t>(lane) < span && base + lane < n_rows) todo = tokens[(base + lane) / q_heads].packed != kInTiles;
            for (uint32_t rest = __ballot_sync(0xFFFFFFFFu, todo); rest; rest &= rest - 1) join(sources(base + __ffs(rest) - 1));
        }
    }
    if (head.n_by_row < head.n_tokens) join_tiles<T, D>(a, head, blockIdx.x, gridDim.x);
}

// ---- host side -----------------------------------------------------------------------

// Checks the description and lays the workspace out from it.
afx_status prepare(const afx_attention_args* d, AttnArgs* a) {
    if (!d) return afx_fail(AFX_E_ARG, "null attention description", 0);
    uint32_t shift = 0;
    const afx_status st = check_cache(&d->cache, &shift);
    if (st != AFX_OK) return st;
    const afx_kv_cache& c = d->cache;
    if (d->q_heads == 0 || d->q_heads % c.kv_heads || d->q_heads / c.kv_heads > 1024)
        return afx_fail(AFX_E_ARG, "q_heads must be a multiple of the cache's heads, at most 1024 times", 0);
    if (d->n_requests == 0 || d->n_requests > kMaxRequests) return afx_fail(AFX_E_ARG, "1 to 16384 requests", 0);
    if (d->n_tokens == 0 || static_cast<uint64_t>(d->n_tokens) * d->q_heads > INT32_MAX)
        return afx_fail(AFX_E_ARG, "n_tokens * q_heads must be from 1 to 2^31 - 1", 0);
    if (d->table_cols == 0 || static_cast<uint64_t>(d->table_cols) * c.page_tokens > INT32_MAX)
        return afx_fail(AFX_E_ARG, "a table row holds 1 page or more and fewer than 2^31 tokens", 0);
    if (d->prefix_len > INT32_MAX) return afx_fail(AFX_E_ARG, "prefix_len must be below 2^31", 0);
    if (!(d->scale > -INFINITY && d->scale < INFINITY)) return afx_fail(AFX_E_ARG, "scale must be finite", 0);
    if (!device_ptr(d->starts_dev, 4) || !device_ptr(d->lens_dev, 4) || !device_ptr(d->table_dev, 4) ||
        (d->prefix_len && !device_ptr(d->prefix_table_dev, 4)))
        return afx_fail(AFX_E_ARG, "starts, lens and tables must be device memory", 0);
    a->k = c.k_dev;
    a->v = c.v_dev;
    a->page_stride = c.page_stride;
    a->token_stride = c.token_stride;
    a->head_stride = c.head_stride;
    a->table = d->table_dev;
    a->prefix_table = d->prefix_table_dev;
    a->starts = d->starts_dev;
    a->lens = d->lens_dev;
    a->table_cols = d->table_cols;
    a->n_requests = d->n_requests;
    a->n_tokens = d->n_tokens;
    a->prefix_len = d->prefix_len;
    a->kv_heads = c.kv_heads;
    a->group = d->q_heads / c.kv_heads;
    a->shift = shift;
    a->n_pages = c.n_pages;
    a->scale_log2 = static_cast<float>(static_cast<double>(d->scale) * 1.4426950408889634074);
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    const bool few = static_cast<uint64_t>(d->n_tokens) * a->group <= kTileFrom;
    a->tile_ctas = !few && tiles_fit(c) ? static_cast<uint32_t>(sms) : 0u;
    // bounds on what the plan writes.  16-row groups: where tiles serve the
    // larger ones, kTileFrom rows a request and on the prefix; every group has one
    // piece, and the cuts add at most kTargetUnits / kv_heads.  Tile groups:
    // full ones, and a last one a request; a group of 128 rows or fewer has
    // its first piece's results twice.  Rows that share the prefix are in
    // requests of fewer than kFuseRows rows
    const uint64_t rows = static_cast<uint64_t>(d->n_tokens) * a->group, R = d->n_requests;
    const uint64_t extra = kTargetUnits / c.kv_heads + 1;
    const bool tiles = a->tile_ctas != 0;
    const uint64_t small = tiles ? (rows < kTileFrom * R ? rows : kTileFrom * R) + kTileFrom : 2 * rows;
    const uint64_t groups = tiles ? (R + 1) * (kTileFrom / kRows) : 2 * (rows / kRows + 1) + R;
    const uint64_t shared = rows < kFuseRows * R ? rows : kFuseRows * R;
    const uint64_t tile_rows = tiles ? rows + 2 * shared + 2 * kTileRows : 0;
    AttnLayout& L = a->L;
    L.max_rows = (small + extra * kRows) * c.kv_heads;
    L.extra_row = L.max_rows + tile_rows * c.kv_heads;
    const uint64_t part_rows = L.extra_row + static_cast<uint64_t>(a->tile_ctas) * kGroupRows;
    uint64_t off = up(sizeof(PlanHead), 256);
    auto take = [&](uint64_t bytes) {
        const uint64_t at = off;
        off = up(off + bytes, 256);
        return at;
    };
    L.counter = take(4);
    L.tokens = take(sizeof(TokenInfo) * static_cast<uint64_t>(d->n_tokens));
    L.packed_token = take(4ull * d->n_tokens);
    L.groups16 = take(sizeof(Row16Group) * groups);
    L.items16 = take(sizeof(Row16Item) * (groups + extra));
    L.tiles = take(sizeof(TileGroup) * (tiles ? 2 * (rows / kGroupRows + 1) + R : 0));
    L.tile_first = take(4ull * a->tile_ctas);
    L.rest = take(4ull * (tiles ? 2 * (rows / kGroupRows + 1) + R : 0));
    L.part_ml = take(8ull * part_rows);
    L.part_o = take(4ull * part_rows * c.head_dim);
    L.total = off;
    uint64_t key = 0x61667850u;
    for (uint64_t v : {L.total, static_cast<uint64_t>(d->n_tokens), static_cast<uint64_t>(d->n_requests),
                       static_cast<uint64_t>(d->prefix_len), static_cast<uint64_t>(d->table_cols),
                       static_cast<uint64_t>(a->group), static_cast<uint64_t>(c.kv_heads), static_cast<uint64_t>(shift),
                       static_cast<uint64_t>(a->tile_ctas)})
        key = (key ^ v) * 0x9E3779B97F4A7C15ull + 1;
    a->plan_key = key;
    return AFX_OK;
}

// A thread a request, up to the most a CTA has; with fewer the sums over the
// CTA cost less.
uint32_t plan_threads(uint32_t requests) {
    const uint32_t n = (requests + 31) / 32 * 32;
    return n < 128 ? 128 : n > kPlanThreads ? kPlanThreads : n;
}

afx_status bind_workspace(AttnArgs* a, void* ws, uint64_t bytes, int32_t* status) {
    if (bytes < a->L.total) return afx_fail(AFX_E_NOSPACE, "the attention workspace is smaller than afx_attention_workspace", 0);
    if (!device_ptr(ws, 256)) return afx_fail(AFX_E_ARG, "the workspace must be 256-byte aligned device memory", 0);
    if (status && !device_ptr(status, 4)) return afx_fail(AFX_E_ARG, "the status word must be device memory", 0);
    a->ws = static_cast<uint8_t*>(ws);
    a->status = status;
    return AFX_OK;
}

template <typename T, int D>
afx_status launch(const AttnArgs& a, const afx_kv_cache& cache, cudaStream_t s) {
    const int sms = current_sms();
    if (sms <= 0) return afx_fail(AFX_E_CUDA, "cannot query the SM count", 0);
    if (a.tile_ctas) {
        const afx_status st = launch_tiles(a, cache, s);
        if (st != AFX_OK) return st;
    }
    const size_t smem = rows16_smem<D>();
    AFX_SERVE_TRY(cudaFuncSetAttribute(attention_rows16_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem)),
                  "cudaFuncSetAttribute");
    AFX_SERVE_TRY(launch_early(attention_rows16_kernel<T, D>, sms * 2, kWarps * 32, smem, s, a), "attention_rows16_kernel launch");
    const uint64_t rows = static_cast<uint64_t>(a.n_tokens) * a.kv_heads * a.group;
    // a request can have tiles of its own from kFuseRows rows on, without a prefix from kTileFrom + 1
    const bool own_tiles = a.tile_ctas && static_cast<uint64_t>(a.n_tokens) * a.group > (a.prefix_len ? kFuseRows - 1 : kTileFrom);
    const uint32_t most = sms * 8, least = own_tiles ? most : 0;
    if (rows <= most) {  // a CTA a row
        const uint32_t n = static_cast<uint32_t>(rows);
        // more warps where rows are few and cut into many pieces (12 rows a head of two on 35,737 keys: 39 us, 67 with
        // 4 warps; two requests on 131,000: 117 and 126).  By the prefix alone, whose length the host has: requests
        // whose own tokens are as many take the 4 warps (one of 100,000 tokens: 108 us)
        const bool many = kFewUnits / a.kv_heads >= kManyPieces && a.prefix_len / kMinKeys >= kManyPieces;
        const uint32_t threads = many && !least && rows <= static_cast<uint64_t>(sms) ? kSplitThreads : kJoinThreads;
        AFX_SERVE_TRY(launch_early(attention_join_kernel<T, D, true>, n < least ? least : n, threads, 0, s, a, 1u), "attention_join_kernel launch");
    } else {
        const uint64_t span = rows <= static_cast<uint64_t>(sms) * 256 ? 1 : 32, per = span * kJoinWarps, need = (rows + per - 1) / per;
        const uint32_t n = need > most ? most : static_cast<uint32_t>(need);
        AFX_SERVE_TRY(launch_early(attention_join_kernel<T, D, false>, n < least ? least : n, kJoinThreads, 0, s, a, static_cast<uint32_t>(span)),
                      "attention_join_kernel launch");
    }
    return AFX_OK;
}

}  // namespace
}  // namespace serve
}  // namespace afx

using namespace afx::serve;

extern "C" afx_status afx_attention_workspace(const afx_attention_args* args, uint64_t* bytes) {
    AttnArgs a{};
    if (!bytes) return afx_fail(AFX_E_ARG, "null pointer", 0);
    const afx_status st = prepare(args, &a);
    if (st != AFX_OK) return st;
    *bytes = a.L.total;
    return AFX_OK;
}

extern "C" afx_status afx_attention_plan(const afx_attention_args* args, void* workspace_dev, uint64_t workspace_bytes,
                                         afx_stream_t stream, int32_t* status_dev) {
    AttnArgs a{};
    afx_status st = prepare(args, &a);
    if (st == AFX_OK) st = bind_workspace(&a, workspace_dev, workspace_bytes, status_dev);
    if (st != AFX_OK) return st;
    AFX_SERVE_TRY(launch_early(attention_plan_kernel, 1, plan_threads(args->n_requests), 0, reinterpret_cast<cudaStream_t>(stream), a),
                  "attention_plan_kernel launch");
    return AFX_OK;
}

extern "C" afx_status afx_attention(const afx_attention_args* args, const void* q_dev, uint64_t q_token_stride,
                                    uint64_t q_head_stride, void* out_dev, uint64_t out_token_stride,
                                    uint64_t out_head_stride, float* lse_dev, void* workspace_dev,
                                    uint64_t workspace_bytes, afx_stream_t stream, int32_t* status_dev) {
    AttnArgs a{};
    afx_status st = prepare(args, &a);
    if (st == AFX_OK) st = bind_workspace(&a, workspace_dev, workspace_bytes, status_dev);
    if (st != AFX_OK) return st;
    if (!device_ptr(q_dev, 2) || !device_ptr(out_dev, 2) || (lse_dev && !device_ptr(lse_dev, 4)))
        return afx_fail(AFX_E_ARG, "queries, outputs and lse must be device memory", 0);
    a.q = q_dev;
    a.out = out_dev;
    a.lse = lse_dev;
    a.q_token = q_token_stride;
    a.q_head = q_head_stride;
    a.out_token = out_token_stride;
    a.out_head = out_head_stride;
    const uintptr_t q_bits = reinterpret_cast<uintptr_t>(q_dev) | 2 * q_token_stride | 2 * q_head_stride;
    a.q_align = q_bits & 3u ? 2 : q_bits & 15u ? 4 : 16;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool bf = args->cache.format == AFX_FMT_BF16, wide = args->cache.head_dim == 128;
    if (bf) return wide ? launch<__nv_bfloat16, 128>(a, args->cache, s) : launch<__nv_bfloat16, 64>(a, args->cache, s);
    return wide ? launch<__half, 128>(a, args->cache, s) : launch<__half, 64>(a, args->cache, s);
}
