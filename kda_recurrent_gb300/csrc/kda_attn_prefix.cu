// Attention of one new token for rows that share the first tokens of their caches (sm_103a).
//
//     x_j = scale q . k_j,  p = softmax(x),  o = sum_j p_j v_j
//
// The rows of a group hold the same first tokens in the same pages. Their query heads of one key head, laid end to
// end, are the rows of a matrix, so that the prefix is a product of tiles of 128 query rows and 128 tokens: S = Q
// K^T and O += P V with tcgen05, accumulators in tensor memory. Each key and value is read once for up to 256 query
// rows instead of once a row. This kernel takes whole tiles of tokens; what is left of the prefix and each row's own
// tokens are the token stream of kda_attn_decode.cu, which joins both sides' (m, l, o).
//
// Schedule. An item is (group, key head, pair of tiles of query rows). A step of it takes one tile of tokens for two
// tiles of query rows, or, when it has at most 128 query rows, two tiles of tokens for the one: either way two
// groups of four warps each have a tile of scores to work on while the tensor core forms the other's. All items'
// steps, laid end to end, are cut into equal shares for the CTAs, one on an SM; a share's part of an item is left
// in the workspace as (m, l, o). The sums run in a fixed order.
//
// Roles: eight warps in two groups for the softmax (a thread a query row, the 128 scores in its registers), one that
// loads keys and values by TMA into a ring of five tiles, a box for each page (or 128 tokens of it) and half of the
// channels, and one that issues the products. The probabilities replace their scores in tensor memory as BF16 (2^-8
// of each, which averages out over a prefix; their sum is formed from the unrounded ones) and are the A operand
// of P V from there. O is scaled down only when a row's maximum has grown by more than 2^8 since it was last fixed.
//
// Tokens of missing pages: their scores are masked, and their rows of the tiles cleared, since a probability of zero
// does not mask a NaN. All waits are bounded; on expiry the CTA records KDA_ERR_DEVICE_TIMEOUT, waits for its own
// copies and products in flight, frees its tensor memory and returns.
#include <algorithm>

#include "kda_dependent.cuh"
#include "kda_internal.cuh"
#include "kda_mma.cuh"
#include "kda_prefix.cuh"
#include "kda_tc.cuh"
#include "kda_tc_bf16.cuh"

namespace kda {
namespace {

constexpr int kT = kPrefixTile;
constexpr int kTile = kT * kHeadDim * 2, kHalf = kTile / 2;  // two halves of 64 channels: 128 rows of 128 bytes
constexpr int kRing = 5;
constexpr int kWarpLoad = 8, kWarpMma = 9;  // the eight before them: softmax
constexpr int kThreads = 10 * 32;
constexpr int kLive = 16;  // masks kept (more tiles than the loads can be ahead of the softmax)
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;  // log2: how far a maximum may grow before O is scaled
constexpr int32_t kLeastRows = 2;  // of a group, for its prefix to be shared

constexpr uint32_t kTmemCols = 512;  // all: the base is column 0
constexpr uint32_t kColS = 0, kColO = 256;  // of the first group of warps; the second's are 128 columns further
constexpr uint32_t kIdescS = instr_desc(1, 128, 128), kIdescO = instr_desc(1, 128, 128) | kTransB;
constexpr uint64_t kDescV = desc_mn(kHalf);

struct Bars {
    uint64_t full[kRing], empty[kRing];
    // of each group of warps: queries written (4 warps), scores done, probabilities written (4 warps), P V done
    uint64_t q[2], s[2], p[2], o[2];
    uint64_t drain;
    uint32_t live[kLive];  // of a tile of keys: a bit for eight tokens
    int64_t sums[kThreads / 32], offset;  // where the CTA's share begins: the place in its first group
    int32_t group;
    uint32_t tmem;
    int32_t abort;
};
constexpr int kQ = kRing * kTile;
constexpr int kBars = kQ + 2 * kTile;
constexpr int kSmem = kBars + (int)sizeof(Bars);
static_assert(kSmem <= 227 * 1024, "one CTA on an SM");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// Wait of a warp, bounded, with one decision for all its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Bars *B) {
    const uint32_t addr = smem_addr(bar);
    volatile int32_t *const abort = &B->abort;
    uint64_t since = 0;
    bool ok = true;
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity), "r"(kSuspendHintNs)
            : "memory");
        if (__all_sync(0xffffffffu, done)) break;
        const uint64_t now = global_ns();
        if (since == 0) since = now;
        if (now - since > kWaitLimitNs) *abort = 1;
        if (__any_sync(0xffffffffu, *abort)) { ok = false; break; }
    }
    return ok;
}

// A group's query rows and tiles of shared tokens (0: nothing is shared), and the steps of one key head.
struct Group {
    int32_t row0, rows, tiles;  // rows of the batch
    int32_t tokens;             // a row of fewer is no part of what is shared
};

__device__ __forceinline__ int query_rows(const AttnPrefixArgs &a, const Group &g) { return g.rows * a.d.group; }
__device__ __forceinline__ int pair_steps(int q_rows, int pair, int tiles) {
    return q_rows - pair * kPrefixSlots > kT ? tiles : (tiles + 1) / 2;
}
__device__ __forceinline__ int64_t head_steps(const AttnPrefixArgs &a, const Group &g) {
    const int rows = query_rows(a, g), pairs = (rows + kPrefixSlots - 1) / kPrefixSlots;
    return pairs == 0 ? 0 : (int64_t)(pairs - 1) * g.tiles + pair_steps(rows, pairs - 1, g.tiles);
}

// (of ordered cu_groups)
__device__ __forceinline__ Group group_at(const AttnPrefixArgs &a, int g) {
    Group x;
    x.row0 = a.cu_groups[g];
    x.rows = a.cu_groups[g + 1] - x.row0;
    x.tokens = min(max(a.prefix_lens[g], 0), a.d.c.capacity);
    x.tiles = x.rows >= kLeastRows ? x.tokens / kT : 0;
    return x;
}

// A CTA's walk over its share: the segments of items in it.
struct Walk {
    Group g;
    int32_t index, head, pair;  // the item
    int32_t step, steps;        // the segment's first step; the item's steps
    int32_t n;                  // the segment's steps
    int32_t rows;               // the item's query rows (1 .. 256), from row pair * 256 of the group's
    int64_t first, left;        // place of the item's first step; steps of the share from the segment on
};

__device__ __forceinline__ void set_item(const AttnPrefixArgs &a, Walk &w) {
    const int rows = query_rows(a, w.g);
    w.rows = min(rows - w.pair * kPrefixSlots, kPrefixSlots);
    w.steps = pair_steps(rows, w.pair, w.g.tiles);
    w.n = (int)min((int64_t)(w.steps - w.step), w.left);
}

__device__ __forceinline__ void next_segment(const AttnPrefixArgs &a, Walk &w) {
    w.left -= w.n;
    if (w.left <= 0) return;
    w.first += w.steps;
    w.step = 0;
    if (++w.pair * kPrefixSlots >= query_rows(a, w.g)) {
        w.pair = 0;
        if (++w.head == a.d.c.num_kv_heads) {
            w.head = 0;
            do w.g = group_at(a, ++w.index);  // (there is one with steps: the share holds another)
            while (w.g.tiles == 0 && w.index + 1 < a.groups);
        }
    }
    set_item(a, w);
}

__global__ void __launch_bounds__(kThreads, 1)
    kda_attn_prefix_kernel(const AttnPrefixArgs a, const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars *const B = reinterpret_cast<Bars *>(smem + kBars);
    const AttnDecodeArgs &p = a.d;
    const PagedCache &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x, ctas = gridDim.x;

    if ((smem_addr(smem) & 1023) != 0) {  // (never: there is no other shared memory)
        if (threadIdx.x == 0) report_error(p.status, KDA_ERR_DEVICE_TIMEOUT, cta);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&B->full[i], 1), mbar_init(&B->empty[i], 1);
        for (int w = 0; w < 2; ++w) mbar_init(&B->q[w], 4), mbar_init(&B->s[w], 1), mbar_init(&B->p[w], 4), mbar_init(&B->o[w], 1);
        mbar_init(&B->drain, 1);
        B->abort = 0;
        fence_mbar_init();
        prefetch_map(&map_k);
        prefetch_map(&map_v);
    }
    wait_for_prior();
    allow_next();

    // ---- the steps of all groups, and where this CTA's share begins
    auto steps_of = [&](int g) { return g < a.groups ? (int64_t)c.num_kv_heads * head_steps(a, group_at(a, g)) : 0; };
    bool bad = false;
    for (int g = threadIdx.x; g < a.groups; g += kThreads) {
        const int lo = a.cu_groups[g], hi = a.cu_groups[g + 1], n = a.prefix_lens[g];
        bad |= lo < 0 || hi < lo || hi > c.batch;
        if (cta == 0 && (lo < 0 || hi < lo || hi > c.batch || n < 0 || n > c.capacity)) report_error(p.status, KDA_ERR_DEVICE_INPUT, g);
    }
    bad = __syncthreads_or(bad);  // then nothing is taken as shared: the rows' own tables hold all of their tokens
    auto block_sum = [&](int64_t x, int64_t &before) {
        int64_t sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        __syncthreads();
        if (lane == 31) B->sums[warp] = sum;
        __syncthreads();
        int64_t total = 0;
        before = sum - x;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += B->sums[w];
            total += B->sums[w];
        }
        return total;
    };
    int64_t mine = 0, before0 = 0;
    if (!bad)
        for (int g = threadIdx.x; g < a.groups; g += kThreads) mine += steps_of(g);
    const int64_t total = block_sum(mine, before0), per = max((total + ctas - 1) / ctas, (int64_t)1);
    const int64_t lo = min(cta * per, total), hi = min(lo + per, total);
    if (lo < hi) {
        int64_t first = 0;
        for (int g0 = 0; g0 < a.groups; g0 += kThreads) {
            int64_t x = mine, before = before0, sum = total;
            if (a.groups > kThreads) x = steps_of(g0 + threadIdx.x), sum = block_sum(x, before);
            const int64_t off = lo - first - before;
            if (off >= 0 && off < x) B->group = g0 + threadIdx.x, B->offset = off;
            first += sum;
        }
    }
    // ---- each row's start: this CTA's of every group's rows
    if (!bad) {
        for (int g = threadIdx.x; g < a.groups; g += kThreads) {
            const Group x = group_at(a, g);
            for (int b = x.row0 + cta; b < x.row0 + x.rows; b += ctas)
                a.x.start[b] = row_length(c, b, p.status, true) >= x.tokens ? x.tiles * kT : 0;
        }
    }
    // rows of no group
    {
        const int from = bad ? c.batch : a.cu_groups[0], to = bad ? c.batch : a.cu_groups[a.groups];
        for (int b = cta * kThreads + threadIdx.x; b < c.batch; b += ctas * kThreads)
            if (b < from || b >= to) a.x.start[b] = 0;
    }
    __syncthreads();
    if (lo >= hi) return;

    if (warp == kWarpMma) {
        tmem_alloc(&B->tmem, kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B->tmem, base = smem_addr(smem);
    Walk w;
    w.index = B->group;
    w.g = group_at(a, w.index);
    w.left = hi - lo;
    {
        const int64_t per_head = head_steps(a, w.g), off = B->offset;
        w.head = (int)(off / per_head);
        const int64_t in_head = off - w.head * per_head;
        const int pairs = (query_rows(a, w.g) + kPrefixSlots - 1) / kPrefixSlots;
        w.pair = (int)min(in_head / w.g.tiles, (int64_t)(pairs - 1));
        w.step = (int)(in_head - (int64_t)w.pair * w.g.tiles);
        w.first = lo - w.step;
        set_item(a, w);
    }
    // Tiles of tokens: a step's are tile s for both groups of warps, or 2 s + i for group i (if there is one).
    // In the ring a step has its keys, then its values.

    if (warp == kWarpLoad) {
        const int rows_a_box = min(c.page_size, kT), boxes = kT / rows_a_box;
        const int sub = lane >> 1, half = lane & 1;  // this lane's box
        const bool on = sub < boxes;
        int leader = -1, leader_of = -1;
        uint32_t count = 0;  // tiles so far
        bool ok = true;
        for (; ok && w.left > 0; next_segment(a, w)) {
            if (leader_of != w.index) {  // the first row that holds the whole prefix: the others' pages are the same
                leader = w.g.row0;
                for (int b0 = 0; b0 < w.g.rows; b0 += 32) {
                    const int b = w.g.row0 + b0 + lane;
                    const bool has = b0 + lane < w.g.rows && row_length(c, b, p.status, false) >= w.g.tokens;
                    const uint32_t who = __ballot_sync(0xffffffffu, has);
                    if (who) { leader = w.g.row0 + b0 + __ffs(who) - 1; break; }
                }
                leader_of = w.index;
            }
            const int32_t *const table = c.block_table + (size_t)leader * c.max_pages;
            const bool shared = w.rows > kT;
            auto page_of = [&](int tile) {
                int page = -1;
                if (on) page = table[(tile * kT + sub * rows_a_box) >> c.page_shift];
                if (page >= c.num_pages) {
                    report_error(p.status, KDA_ERR_DEVICE_INPUT, leader);
                    page = -1;
                }
                return page;
            };
            auto load = [&](const CUtensorMap *map, int tile, int page, bool keys) {
                const int slot = count % kRing;
                if (count >= kRing && !wait_warp(&B->empty[slot], (count / kRing - 1) & 1, B)) return false;
                const uint32_t dst = base + slot * kTile + half * kHalf + sub * rows_a_box * 128;
                const uint32_t missing = __ballot_sync(0xffffffffu, on && page < 0);
                uint32_t live = 0xffffu;
                if (missing) {
                    for (int i = 0; i < boxes; ++i)
                        if ((missing >> (2 * i)) & 1) live &= ~(((1u << (rows_a_box / 8)) - 1) << (i * rows_a_box / 8));
                    if (on && page < 0)
                        for (int i = 0; i < rows_a_box * 8; ++i)
                            *reinterpret_cast<uint4 *>(smem + (dst - base) + i * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    __syncwarp();
                }
                if (lane == 0) {
                    if (keys) B->live[count % kLive] = live;
                    expect_tx(&B->full[slot], (2 * boxes - __popc(missing)) * rows_a_box * 128);
                }
                __syncwarp();
                if (on && page >= 0) tma_load(dst, map, 64 * half, (tile * kT) & (c.page_size - 1), w.head, page, &B->full[slot]);
                ++count;
                return true;
            };
            int t = shared ? w.step : 2 * w.step;
            int page0 = page_of(t), page1 = shared || t + 1 >= w.g.tiles ? -1 : page_of(t + 1);
            for (int i = 0; ok && i < w.n; ++i) {
                const int now0 = page0, now1 = page1, now = t;
                const bool two = !shared && now + 1 < w.g.tiles;
                t += shared ? 1 : 2;
                if (i + 1 < w.n) {
                    page0 = page_of(t);
                    if (!shared && t + 1 < w.g.tiles) page1 = page_of(t + 1);
                }
                ok = load(&map_k, now, now0, true) && (!two || load(&map_k, now + 1, now1, true)) && load(&map_v, now, now0, false) &&
                     (!two || load(&map_v, now + 1, now1, false));
            }
        }
        if (!ok)  // what was asked for has to arrive before the CTA leaves
            for (uint32_t i = count > kRing ? count - kRing : 0; i < count; ++i) mbar_wait(&B->full[i % kRing], (i / kRing) & 1);
    } else if (warp == kWarpMma) {
        uint32_t count = 0, used[2] = {0, 0}, queries[2] = {0, 0};
        bool ok = true;
        for (; ok && w.left > 0; next_segment(a, w)) {
            const bool shared = w.rows > kT;
            // step i of the segment: its tiles in the ring, and whether group g has one
            auto has = [&](int i, int g) { return shared || g == 0 || 2 * (w.step + i) + 1 < w.g.tiles; };
            auto keys_at = [&](int i, int g) { return count + (shared ? 2 * i : 4 * i + g); };
            auto values_at = [&](int i, int g) { return count + (shared ? 2 * i + 1 : 4 * i + (has(i, 1) ? 2 : 1) + g); };
            auto scores = [&](int i, int g) {
                if (!has(i, g)) return true;
                const uint32_t k = keys_at(i, g), slot = k % kRing;
                if (!wait_warp(&B->full[slot], (k / kRing) & 1, B)) return false;
                const uint64_t dq = at(kDescK, base + kQ + g * kTile), dk = at(kDescK, base + slot * kTile);
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t off = ((s >> 2) * kHalf + (s & 3) * 32) >> 4;
                    mma_ss(tmem + kColS + 128 * g, dq + off, dk + off, kIdescS, s > 0);
                }
                commit(&B->s[g]);
                if (!shared || g == 1) commit(&B->empty[slot]);
                return true;
            };
            auto products = [&](int i, int g) {
                if (!has(i, g)) return true;
                const uint32_t v = values_at(i, g), slot = v % kRing;
                if (!wait_warp(&B->full[slot], (v / kRing) & 1, B) || !wait_warp(&B->p[g], used[g] & 1, B)) return false;
                ++used[g];
                tc_fence_after();
                const uint64_t dv = at(kDescV, base + slot * kTile);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_ts(tmem + kColO + 128 * g, tmem + kColS + 128 * g + 8 * s, dv + s * 128, kIdescO, i > 0 || s > 0);
                commit(&B->o[g]);
                if (!shared || g == 1) commit(&B->empty[slot]);
                return true;
            };
            for (int g = 0; ok && g < 2; ++g) {
                if (!has(0, g)) continue;
                ok = wait_warp(&B->q[g], queries[g] & 1, B);
                ++queries[g];
            }
            if (!ok) break;
            tc_fence_after();
            ok = scores(0, 0) && scores(0, 1);
            for (int i = 0; ok && i < w.n; ++i) {
                ok = products(i, 0) && (i + 1 >= w.n || scores(i + 1, 0));
                ok = ok && products(i, 1) && (i + 1 >= w.n || scores(i + 1, 1));
            }
            const int last = w.step + w.n - 1;
            count += shared ? 2 * w.n : 4 * w.n - (2 * last + 1 < w.g.tiles ? 0 : 2);
        }
        commit(&B->drain);  // every earlier product is done when this arrives
        mbar_wait(&B->drain, 0);
    } else {
        const int g = warp >> 2, quad = warp & 3, r = 32 * quad + lane;  // the group of warps; the row of its tile
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16), col_s = lanes + kColS + 128 * g, col_o = lanes + kColO + 128 * g;
        const float scale2 = fabsf(p.scale) * kLog2e;
        const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;  // (the scale's sign goes to the queries)
        uint32_t count = 0, used = 0;  // tiles in the ring; tiles of this group
        bool ok = true;
        for (; ok && w.left > 0; next_segment(a, w)) {
            const bool shared = w.rows > kT;
            const int mine = shared ? g * kT + r : r;  // the query row of the item
            const bool valid = mine < w.rows;
            const int in_group = w.pair * kPrefixSlots + mine, row = in_group / p.group;
            const int64_t head = (int64_t)(w.g.row0 + row) * p.num_q_heads + w.head * p.group + (in_group - row * p.group);
            // (a group of warps without a tile writes no queries: it could come by here again before the other)
            if (shared || g == 0 || 2 * w.step + 1 < w.g.tiles) {
                const uint4 *const src = reinterpret_cast<const uint4 *>(p.q + head * kHeadDim);
                uint8_t *const dst = smem + kQ + g * kTile + r * 128;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (valid) x = __ldg(src + i);
                    x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
                    *reinterpret_cast<uint4 *>(dst + (i >> 3) * kHalf + (((i & 7) ^ (r & 7)) << 4)) = x;
                }
                fence_async_smem();
                arrive_warp(&B->q[g]);
            }
            if (valid && w.step == 0 && (shared || g == 0)) {
                // this segment begins the item: where its other parts will be
                const int64_t last = (w.first + w.steps - 1) / per;
                PrefixCut cut;
                cut.per = shared ? 1 : 2;
                cut.slot = shared ? g * kT + r : r;
                cut.cta = cta + 1;
                cut.ctas = (int)(last - cta);
                a.x.cuts[head] = cut;
            }
            float m = kNegInf, l = 0.0f;
            bool any = false;
            for (int i = 0; ok && i < w.n; ++i) {
                if (!(shared || g == 0 || 2 * (w.step + i) + 1 < w.g.tiles)) break;  // (the item's last step)
                ok = wait_warp(&B->s[g], used & 1, B);
                if (!ok) break;
                tc_fence_after();
                const uint32_t live = *reinterpret_cast<volatile uint32_t *>(&B->live[(count + (shared ? 2 * i : 4 * i + g)) % kLive]);
                float s[4][32];
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_ld32(col_s + 32 * b, s[b]);
                tmem_wait_ld();
                if (live != 0xffffu) {
#pragma unroll
                    for (int b = 0; b < 4; ++b)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!((live >> (4 * b + (j >> 3))) & 1)) s[b][j] = kNegInf;
                }
                float top[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    top[b] = s[b][0];
#pragma unroll
                    for (int j = 1; j < 32; ++j) top[b] = fmaxf(top[b], s[b][j]);
                }
                // (NaN scores are passed over, and make their row's sum NaN)
                const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale2;
                const bool grow = !any ? true : now > m + kSlack;
                if (!any) {
                    m = now == now ? now : kNegInf;  // (-inf * 0)
                    any = true;
                } else if (__any_sync(0xffffffffu, grow)) {
                    const float to = fmaxf(m, now), f = to == kNegInf ? 1.0f : ex2(m - to);
                    ok = wait_warp(&B->o[g], (used - 1) & 1, B);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int b = 0; b < 8; ++b) {
                        float o[16];
                        tmem_ld16(col_o + 16 * b, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= f;
                        tmem_st16(col_o + 16 * b, o);
                    }
                    l *= f;
                    m = to;
                }
                const float ref = m == kNegInf ? 0.0f : m;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float pk[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float x0 = ex2(fmaf(s[b][2 * j], scale2, -ref)), x1 = ex2(fmaf(s[b][2 * j + 1], scale2, -ref));
                        if (live != 0xffffu && !((live >> (4 * b + (j >> 2))) & 1)) x0 = x1 = 0.0f;
                        sum[j & 1] += x0;
                        sum[2 + (j & 1)] += x1;
                        pk[j] = __uint_as_float(pack_bf16(x0, x1));
                    }
                    tmem_st16(col_s + 16 * b, pk);
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                tmem_wait_st();
                tc_fence_before();
                arrive_warp(&B->p[g]);
                ++used;
            }
            if (!ok) break;
            const int last = w.step + w.n - 1;
            count += shared ? 2 * w.n : 4 * w.n - (2 * last + 1 < w.g.tiles ? 0 : 2);
            // ---- the segment's part
            if (any) {
                ok = wait_warp(&B->o[g], (used - 1) & 1, B);
                if (!ok) break;
                tc_fence_after();
            }
            const int64_t part = w.step == 0 ? (shared ? 0 : (int64_t)g * a.x.heads) + head
                                             : 3 * (int64_t)a.x.heads + (int64_t)cta * kPrefixSlots + g * kT + r;
            if (valid) a.x.ml[part] = make_float2(m, l);
            float4 *const dst = reinterpret_cast<float4 *>(a.x.o + part * kHeadDim);
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                float o[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = 0.0f;
                if (any) {
                    tmem_ld16(col_o + 16 * b, o);
                    tmem_wait_ld();
                }
                if (valid)
#pragma unroll
                    for (int j = 0; j < 4; ++j) dst[4 * b + j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && B->abort) report_error(p.status, KDA_ERR_DEVICE_TIMEOUT, cta);
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// A cache's tokens as [pages][heads][page size][128], in boxes of a page's (or 128) tokens of one head x 64 channels.
cudaError_t page_map(CUtensorMap *map, const __nv_bfloat16 *base, const PagedCache &c, int64_t page_stride) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {kHeadDim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_kv_heads, (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {kHeadDim * 2, (cuuint64_t)c.page_size * kHeadDim * 2, (cuuint64_t)page_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)std::min(c.page_size, kT), 1, 1}, step[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<__nv_bfloat16 *>(base), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t configure_once() {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kda_attn_prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return cudaSuccess;
}

}  // namespace

int64_t attn_prefix_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads, int64_t capacity, int32_t sms) {
    return attn_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, capacity, false, sms) +
           prefix_layout(nullptr, nullptr, batch, num_q_heads, sms);
}

cudaError_t launch_attn_prefix(const AttnPrefixArgs &args, cudaStream_t stream) {
    if (args.groups == 0) return launch_attn_decode(args.d, stream);
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    AttnPrefixArgs a = args;
    const PagedCache &c = a.d.c;
    prefix_layout(&a.x,
                  static_cast<char *>(a.d.ws) + attn_decode_workspace_bytes(c.batch, a.d.num_q_heads, c.num_kv_heads, c.capacity, false, sms),
                  c.batch, a.d.num_q_heads, sms);
    CUtensorMap map_k, map_v;
    cudaError_t e = page_map(&map_k, c.k, c, c.k_page_stride);
    if (e == cudaSuccess) e = page_map(&map_v, c.v, c, c.v_page_stride);
    if (e == cudaSuccess) e = configure_once();
    if (e == cudaSuccess) e = launch_dependent(kda_attn_prefix_kernel, dim3((unsigned)sms), kThreads, kSmem, stream, a, map_k, map_v);
    if (e == cudaSuccess) e = launch_attn_tails(a.d, a.x, stream);
    return e;
}

}  // namespace kda
