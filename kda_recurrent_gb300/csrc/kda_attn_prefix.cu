// Attention of one new token for rows that share the first tokens of their caches (sm_103a).
//
//     x_j = scale q . k_j,  p = softmax(x),  o = sum_j p_j v_j
//
// The rows of a group hold the same first tokens in the same pages. Their query heads of one key head, laid end to
// end, are the rows of a matrix, so that the prefix is a product of tiles of 128 query rows and 128 tokens: S = Q
// K^T and O += P V with tcgen05, accumulators in tensor memory. Each key and value is read once for up to 256 query
// rows instead of once a row. Whole tiles of tokens are taken so; what is left of the prefix and each row's own tokens
// are the token stream of kda_attn_stream.cuh. A second kernel joins both sides' (m, l, o).
//
// Schedule. An item is (group, key head, pair of tiles of query rows). A step of it takes one tile of tokens for two
// tiles of query rows, or, when it has at most 128 query rows, two tiles of tokens for the one: either way two
// groups of four warps each have a tile of scores to work on while the tensor core forms the other's. All items'
// steps, laid end to end, are cut into equal shares for the CTAs, one on an SM; a share's part of an item is left
// in the workspace as (m, l, o). The sums run in a fixed order.
//
// One launch does both kinds of work: each CTA counts the steps and the rest's tiles, and the CTAs are dealt to the two so
// that both end together. As two launches, one after the other, 25 shapes of 2 to 512 rows took 1.22 times as long (32
// rows in 4 groups of 2048 to 8192 shared tokens 53.0 and now 43.6 us, 512 rows in 16 groups 290 and 284, 128 rows behind
// 32768 169.5 and 158).
//
// Roles: eight warps in two groups for the softmax (a thread a query row, 64 scores at a time in its registers), one that
// loads keys by TMA into a ring of three tiles and one that loads values into a ring of two, a box for each page (or 128
// tokens of it) and half of the channels, and one for each group that issues its products. Half a tile's scores are
// formed while the other half's softmax runs. The probabilities replace their scores in tensor memory as BF16 and are the
// A operand of P V from there. O is scaled down only when a row's maximum has grown by more than 2^8 since it was last fixed.
//
// Rounding. One BF16 term a probability: each is off by at most 2^-8 of itself, an output so by at most 2^-8 sum_j p_j |v_j|
// (the sum of the probabilities is formed from the unrounded ones, in 32 bits). For independent values that is the same share
// of an output at any length, since the output shrinks like the error: 0.0016 of its rms beside 0.0017 of the output's own
// rounding, together 0.0023 measured, where the token stream with its two terms has the 0.0017. Two terms here (the upper 16
// bits and the rest) measured 0.0017, too, but are half as many products more: 32 rows in 4 groups 46.3 instead of 43.2 us,
// 512 rows 304 and 284, 128 rows behind 32768 tokens 192 and 157. One term, because its error stays within a step of the
// output's type; so the last bits of an output can change where a call passes from the one form to the other (kFewBytes).
//
// What bounds it. 128 rows of 64 heads behind 32768 tokens: 1.4e11 operations and 408 MB in 158 us, 885 TFLOP/s. A step has
// 16.8 MFLOP (1.33 us of an SM's products at the library's rate) and 32768 exponentials (0.54 us), and takes 1.8 to 2.0 us,
// from L2 or HBM: the warps that issue products wait for the tensor core most of the time, which reads 320 KB of shared
// memory a step (1.3 us at 128 bytes a clock), since scores in half tiles read the queries twice. Scores by whole tiles
// read 256 KB, but then a group's softmax waits for them: 128 rows 168 and so 179 us, 512 rows 301 and 294, 32 rows in 4 groups
// 44.8 and 44.2, the geometric mean of 25 shapes the same. With two tiles of tokens for at most 128 query rows a step takes 1.7 us
// from L2 and 2.9 from HBM, 6.7 TB/s.
// 512 rows in 16 groups, 1.22 GB: 284 us, 4.3 TB/s; the rest's stream is about 200 ns of an SM for a tile of 16 tokens with the
// beginnings of its short rows, and the prefixes' steps 2.9 us. Both kinds of CTAs end unevenly: the stream's at 228 to 262 us
// (their mean 241), the prefixes' at 167 to 279 (215).
// 32 rows in 4 groups, by stamps in a copy that takes 45 us: lengths and dealing 1.8 us, first scores at 10 (queries and keys from memory,
// the code's first pass), eight steps 16, last products and the part 3.4; the CTAs whose share crosses an item begin and
// end twice, and are the last at 40 (mean 33); the join 41 to 45.
//
// Tokens of missing pages: their scores are masked, and their rows of the tiles cleared, since a probability of zero
// does not mask a NaN. All waits are bounded; on expiry the CTA records KDA_ERR_DEVICE_TIMEOUT, waits for its own
// copies and products in flight, frees its tensor memory and returns.
#include <algorithm>

#include "kda_attn_stream.cuh"
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
constexpr int kKeyRing = 3, kValueRing = 2, kRing = kKeyRing + kValueRing;
constexpr int kWarpKeys = 8, kWarpMma = 10;  // (9: values; 11: the second group's products); the eight before them: softmax
constexpr int kThreads = 12 * 32;
constexpr int kLive = 8;  // masks kept (more tiles than the loads can be ahead of the softmax)
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;  // log2: how far a maximum may grow before O is scaled
// What the work takes of an SM, in ns, by which the CTAs are dealt to its two kinds: a step of a prefix whose tokens several
// pairs of tiles of query rows read at the same time, or one alone (that of one pair, or any when there are more items than
// CTAs for them), the beginning and end of an item, a tile of 16 tokens of the rest. Only their ratios count, and they are
// fitted, not measured each by itself (a tile takes 190 to 200 ns, a step 1.8 to 2.9 us). Over 25 shapes (2 to 512 rows of 8 to
// 64 query heads on 1 or 8 key heads, in 1 to 16 groups, 128 to 32768 shared tokens, 64 to 1024 of the rest), geometric mean of the
// time over that of two launches: 0.821; with 2000 or 2600 for the dearer step 0.822 (512 rows in 16 groups 298 and 290 instead of
// 284 us), with 4000 an item 0.821. With the dearer one decided by the pairs alone 0.831 (296), and then with 130, 145 or 180 a tile 0.824, 0.828
// and 0.846 (128 rows behind 32768 tokens 175, 165 and 158 instead of 157).
constexpr float kStepNs = 1600.0f, kColdStepNs = 2300.0f, kItemNs = 3000.0f, kTileNs = 160.0f;
constexpr int32_t kLeastRows = 2;  // of a group, for its prefix to be shared

constexpr uint32_t kTmemCols = 512;  // all: the base is column 0
constexpr uint32_t kColS = 0, kColO = 256;  // of the first group of warps; the second's are 128 columns further
constexpr uint32_t kIdescS = instr_desc(1, 128, 64), kIdescO = instr_desc(1, 128, 128) | kTransB;
constexpr uint64_t kDescV = desc_mn(kHalf);

struct Bars {
    uint64_t full[kRing], empty[kRing];  // of the keys' places, then the values'
    // of each group of warps: queries written (4 warps); for half a tile's tokens: scores done, probabilities written
    // (4 warps); P V done
    // (for the last tile of a segment)
    uint64_t q[2], s[2][2], p[2][2], o[2][2];
    uint64_t drain[2];
    uint32_t live[kLive];  // of a tile of keys: a bit for eight tokens
    int64_t sums[kThreads / 32];
    uint32_t tiles[kThreads / 32];
    float2 cost[kThreads / 32];
    int32_t group, offset;  // where the CTA's share begins: its first group, and the place in that
    uint32_t tmem;
    int32_t abort;
};
constexpr int kQ = kRing * kTile;
constexpr int kBars = kQ + 2 * kTile;
constexpr int kSmem = kBars + (int)sizeof(Bars);
static_assert(kSmem <= 227 * 1024 && kBars >= stream::kSmem<uint32_t>, "one CTA on an SM, of either kind");

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Two numbers at a time.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 y;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return y;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 y;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(y.x), "=f"(y.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return y;
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ uint32_t try_wait(const uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(kSuspendHintNs)
        : "memory");
    return done;
}

// Wait of a warp for up to three phases, bounded, with one decision for all its lanes. (One after the other, waits for
// phases that are long complete take some 150 cycles each.) What follows a first try is not inlined: the kernel's
// many waits would be a sixth of its instructions, which every launch has to fetch anew.
__device__ __noinline__ bool wait_on(const uint64_t *b0, uint32_t p0, const uint64_t *b1, uint32_t p1, const uint64_t *b2, uint32_t p2, Bars *B) {
    volatile int32_t *const abort = &B->abort;
    const uint64_t since = global_ns();
    for (;;) {
        const uint32_t done = try_wait(b0, p0) & try_wait(b1, p1) & try_wait(b2, p2);
        if (__all_sync(0xffffffffu, done)) return true;
        if (global_ns() - since > kWaitLimitNs) *abort = 1;
        if (__any_sync(0xffffffffu, *abort)) return false;
    }
}

template <int kCount>
__device__ __forceinline__ bool wait_all(uint64_t *const (&bar)[kCount], const uint32_t (&parity)[kCount], Bars *B) {
    uint32_t done = 1;
#pragma unroll
    for (int i = 0; i < kCount; ++i) done &= try_wait(bar[i], parity[i]);
    if (__all_sync(0xffffffffu, done)) return true;
    return wait_on(bar[0], parity[0], bar[1 % kCount], parity[1 % kCount], bar[2 % kCount], parity[2 % kCount], B);
}

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Bars *B) {
    uint64_t *const bars[1] = {bar};
    const uint32_t parities[1] = {parity};
    return wait_all(bars, parities, B);
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
__device__ __forceinline__ Group group_of(const AttnPrefixArgs &a, int lo, int hi, int tokens) {
    Group x;
    x.row0 = lo;
    x.rows = hi - lo;
    x.tokens = min(max(tokens, 0), a.d.c.capacity);
    x.tiles = x.rows >= kLeastRows ? x.tokens / kT : 0;
    return x;
}
__device__ __forceinline__ Group group_at(const AttnPrefixArgs &a, int g) {
    return group_of(a, a.cu_groups[g], a.cu_groups[g + 1], a.prefix_lens[g]);
}

// How many of a row's n tokens are taken with its group's: whole tiles of the group's prefix, if the row holds that.
struct GroupStarts {
    static constexpr bool kTail = true;
    const AttnPrefixArgs &a;
    bool none;  // nothing is shared
    __device__ __forceinline__ int operator()(int b, int n) const {
        if (none || b < a.cu_groups[0] || b >= a.cu_groups[a.groups]) return 0;
        int lo = 0, hi = a.groups - 1;  // the last group that begins at the row or before it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.cu_groups[mid] <= b) lo = mid;
            else hi = mid - 1;
        }
        const Group g = group_at(a, lo);
        return n >= g.tokens ? g.tiles * kT : 0;
    }
};

// A CTA's walk over its share: the segments of items in it.
struct Walk {
    Group g;
    int32_t index, head, pair;  // the item
    int32_t step, steps;        // the segment's first step; the item's steps
    int32_t n;                  // the segment's steps
    int32_t rows;               // the item's query rows (1 .. 256), from row pair * 256 of the group's
    int32_t first, left;        // place of the item's first step; steps of the share from the segment on
};

__device__ __forceinline__ void set_item(const AttnPrefixArgs &a, Walk &w) {
    const int rows = query_rows(a, w.g);
    w.rows = min(rows - w.pair * kPrefixSlots, kPrefixSlots);
    w.steps = pair_steps(rows, w.pair, w.g.tiles);
    w.n = min(w.steps - w.step, w.left);
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

// The segment's tiles of keys (and of values), and the steps of it that group g of warps has a tile in: all, but for
// the second group's at the end of an item with an odd number of tiles.
__device__ __forceinline__ int tiles_in(const Walk &w) {
    return w.rows > kT ? w.n : 2 * w.n - (2 * (w.step + w.n) - 1 < w.g.tiles ? 0 : 1);
}
__device__ __forceinline__ int steps_in(const Walk &w, int g) { return w.rows > kT || g == 0 ? w.n : tiles_in(w) - w.n; }

// The loads of the keys' or the values' tiles, by one warp: tile s for step s, or 2 s and 2 s + 1. A lane asks for a box
// of a page (or 128 tokens of it) and half of the channels. (Asked for by one elected lane after another the 16 boxes
// of a tile of small pages take 55.9 instead of 55.0 us with 32 rows in 4 groups; by 16-byte copies of all lanes 58.6.)
__device__ __forceinline__ void load_tiles(const AttnPrefixArgs &a, Walk w, int per, const CUtensorMap *map, bool keys, uint8_t *smem, Bars *B) {
    const PagedCache &c = a.d.c;
    const int lane = threadIdx.x & 31, rows_a_box = min(c.page_size, kT), boxes = kT / rows_a_box;
    const uint32_t ring = keys ? kKeyRing : kValueRing, place0 = keys ? 0 : kKeyRing;
    uint64_t *const full = B->full + place0, *const empty = B->empty + place0;
    const int sub = lane >> 1, half = lane & 1;  // this lane's box
    int leader = -1, leader_of = -1, done = 0;
    uint32_t count = 0, slot = 0, turn = 0;  // tiles so far; the next one's place, and the times that was used
    bool ok = true;
    for (; ok && w.left > 0; next_segment(a, w)) {
        const bool changed = leader_of != w.index;
        if (changed) leader = w.g.row0, leader_of = w.index;
        auto page_at = [&](int tile) {
            return sub < boxes && leader >= 0 ? c.block_table[(size_t)leader * c.max_pages + ((tile * kT + sub * rows_a_box) >> c.page_shift)] : -1;
        };
        auto page_of = [&](int page) {
            if (page >= c.num_pages) {
                report_error(a.d.status, KDA_ERR_DEVICE_INPUT, leader);
                page = -1;
            }
            return page;
        };
        // The order of the tiles is free. CTAs that work on other query rows of the same tokens read them at the same
        // time, once from HBM, when each begins where its tile's number modulo the length of a share is the number of
        // steps that it has done.
        const int begin = w.rows > kT ? w.step : 2 * w.step, tiles = tiles_in(w);
        int tile = begin;
        if (w.rows > kT) {
            int ahead = (done - w.step) % per;
            if (ahead < 0) ahead += per;
            if (ahead < tiles) tile += ahead;
        }
        done += w.n;
        int next = page_at(tile);
        // The pages are those of the first row that holds the whole prefix: most often the first one, whose table is
        // read beside the rows' lengths. (If none does, nobody takes what is formed here, and no table is looked at.)
        bool found = !changed;
        for (int b0 = 0; !found && b0 < w.g.rows; b0 += 32) {
            const int b = w.g.row0 + b0 + lane;
            const bool has = b0 + lane < w.g.rows && row_length(c, b, a.d.status, false) >= w.g.tokens;
            const uint32_t who = __ballot_sync(0xffffffffu, has);
            if (!who) continue;
            leader = w.g.row0 + b0 + __ffs(who) - 1;
            if (leader != w.g.row0) next = page_at(tile);
            found = true;
        }
        if (!found) leader = next = -1;
        next = page_of(next);
        for (int i = 0; i < tiles; ++i) {
            const int page = next, now = tile;
            if (++tile == begin + tiles) tile = begin;
            if (i + 1 < tiles) next = page_of(page_at(tile));
            ok = turn == 0 || wait_warp(&empty[slot], (turn - 1) & 1, B);
            if (!ok) break;
            const bool on = sub < boxes, gone = on && page < 0;
            const uint32_t missing = __ballot_sync(0xffffffffu, gone);
            uint32_t live = 0xffffu;
            uint8_t *const box = smem + (place0 + slot) * kTile + half * kHalf + sub * rows_a_box * 128;
            if (missing) {  // clear their rows
                for (int i = 0; i < boxes; ++i)
                    if ((missing >> (2 * i)) & 1) live &= ~(((1u << (rows_a_box / 8)) - 1) << (i * rows_a_box / 8));
                for (int e = 0; gone && e < rows_a_box * 8; ++e) reinterpret_cast<uint4 *>(box)[e] = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
            }
            if (lane == 0) {
                if (keys) B->live[count % kLive] = live;
                expect_tx(&full[slot], (2 * boxes - __popc(missing)) * rows_a_box * 128);
            }
            __syncwarp();
            if (on && !gone) tma_load(smem_addr(box), map, 64 * half, (now * kT) & (c.page_size - 1), w.head, page, &full[slot]);
            ++count;
            if (++slot == ring) slot = 0, ++turn;
        }
    }
    // What was asked for has to arrive before the CTA leaves, also where this warp has done all of its work and another
    // one gives up. (Without that the products' warps wait for the same tiles anyway.)
    for (uint32_t i = count > ring ? count - ring : 0; i < count; ++i) mbar_wait(&full[i % ring], (i / ring) & 1);
}

// The products of group g of warps, issued by one warp: S = Q K^T of a step behind O += P V of the one before. Both
// groups' warps pass every place of the rings, in order, and free it, so that neither is ever two turns of a ring
// ahead of the other (the barriers' parity could not tell).
__device__ __forceinline__ void issue_products(const AttnPrefixArgs &a, Walk w, int g, uint8_t *smem, Bars *B) {
    const uint32_t lead = elect_lead();
    const uint32_t base = smem_addr(smem), tmem = B->tmem, col_s = tmem + kColS + 128 * g, col_o = tmem + kColO + 128 * g;
    const uint64_t dq = at(kDescK, base + kQ + g * kTile);
    uint32_t k_slot = 0, k_turn = 0, v_slot = 0, v_turn = 0;  // the next places
    uint32_t used = 0, queries = 0;                           // tiles, and segments, of this group
    bool ok = true;
    for (; ok && w.left > 0; next_segment(a, w)) {
        const bool shared = w.rows > kT;
        const int tiles = tiles_in(w), steps = steps_in(w, g);
        // the tiles of step i that are the other group's alone: before (or after) this one's
        auto skip = [&](int i, int other, uint32_t ring, uint32_t place0, uint32_t &slot, uint32_t &turn) {
            if (shared || other == g || 2 * i + other >= tiles) return true;
            if (!wait_warp(&B->full[place0 + slot], turn & 1, B)) return false;
            arrive_warp(&B->empty[place0 + slot]);
            if (++slot == ring) slot = 0, ++turn;
            return true;
        };
        auto scores = [&](int half) {  // of half the tokens of the next place's tile
            const uint64_t dk = at(kDescK, base + k_slot * kTile + half * (kHalf / 2));
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const uint32_t off = ((s >> 2) * kHalf + (s & 3) * 32) >> 4;
                mma_ss(lead, col_s + 64 * half, dq + off, dk + off, kIdescS, s > 0);
            }
            commit(lead, &B->s[g][half]);
            if (half == 1) commit(lead, &B->empty[k_slot]);
        };
        auto next_keys = [&] {
            if (++k_slot == kKeyRing) k_slot = 0, ++k_turn;
        };
        ok = skip(0, 0, kKeyRing, 0, k_slot, k_turn);
        if (ok && steps > 0) {
            uint64_t *const bars[2] = {&B->q[g], &B->full[k_slot]};
            const uint32_t parities[2] = {queries & 1, k_turn & 1};
            ok = wait_all(bars, parities, B);
            if (!ok) break;
            ++queries;
            tc_fence_after();
            scores(0);
            scores(1);
            next_keys();
        }
        ok = ok && skip(0, 1, kKeyRing, 0, k_slot, k_turn);
        for (int i = 0; ok && i < w.n; ++i) {
            ok = skip(i, 0, kValueRing, kKeyRing, v_slot, v_turn) && (i + 1 == w.n || skip(i + 1, 0, kKeyRing, 0, k_slot, k_turn));
            if (!ok) break;
            if (i < steps) {
                const bool more = i + 1 < steps;
                // (without a next tile its wait is the values' again)
                uint64_t *const values = &B->full[kKeyRing + v_slot];
                uint64_t *const bars[3] = {values, more ? &B->full[k_slot] : values, &B->p[g][0]};
                const uint32_t parities[3] = {v_turn & 1, more ? k_turn & 1 : v_turn & 1, used & 1};
                ok = wait_all(bars, parities, B);
                const uint64_t dv = at(kDescV, base + (kKeyRing + v_slot) * kTile);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (half == 1) ok = wait_warp(&B->p[g][1], used & 1, B);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma_ts(lead, col_o, col_s + 64 * half + 8 * s, dv + (4 * half + s) * 128, kIdescO, i > 0 || half > 0 || s > 0);
                    if (!more) commit(lead, &B->o[g][half]);
                    if (half == 1) commit(lead, &B->empty[kKeyRing + v_slot]);
                    if (more) scores(half);
                    if (more && half == 1) next_keys();
                }
                if (!ok) break;
                ++used;
                if (++v_slot == kValueRing) v_slot = 0, ++v_turn;
            }
            ok = skip(i, 1, kValueRing, kKeyRing, v_slot, v_turn) && (i + 1 == w.n || skip(i + 1, 1, kKeyRing, 0, k_slot, k_turn));
        }
    }
    commit(lead, &B->drain[g]);  // every earlier product is done when this arrives
    mbar_wait(&B->drain[g], 0);
}

__global__ void __launch_bounds__(kThreads, 1)
    kda_attn_prefix_kernel(const AttnPrefixArgs a, const stream::Args rest, const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars *const B = reinterpret_cast<Bars *>(smem + kBars);
    const AttnDecodeArgs &p = a.d;
    const PagedCache &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

    if ((smem_addr(smem) & 1023) != 0) {  // (never: there is no other shared memory)
        if (threadIdx.x == 0) report_error(p.status, KDA_ERR_DEVICE_TIMEOUT, cta);
        return;
    }
    if (threadIdx.x == 0) {
        // (a place is freed by both groups' warps)
        for (int i = 0; i < kRing; ++i) mbar_init(&B->full[i], 1), mbar_init(&B->empty[i], 2);
        for (int w = 0; w < 2; ++w) {
            mbar_init(&B->q[w], 4);
            for (int h = 0; h < 2; ++h) mbar_init(&B->s[w][h], 1), mbar_init(&B->p[w][h], 4), mbar_init(&B->o[w][h], 1);
        }
        mbar_init(&B->drain[0], 1), mbar_init(&B->drain[1], 1);
        B->abort = 0;
        fence_mbar_init();
        prefetch_map(&map_k);
        prefetch_map(&map_v);
    }
    if (warp == kWarpMma) {
        tmem_alloc(&B->tmem, kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    wait_for_prior();
    allow_next();

    // ---- the steps of all groups, and where this CTA's share begins
    bool bad = false;
    Walk w;
    w.g.row0 = w.g.rows = w.g.tiles = w.g.tokens = 0;
    auto group_steps = [&](int g, Group &x, float2 &cost) {
        x.row0 = x.rows = x.tiles = x.tokens = 0;
        if (g >= a.groups) return (int64_t)0;
        const int lo = a.cu_groups[g], hi = a.cu_groups[g + 1], n = a.prefix_lens[g];
        const bool wrong = lo < 0 || hi < lo || hi > c.batch;
        if (cta == 0 && (wrong || n < 0 || n > c.capacity)) report_error(p.status, KDA_ERR_DEVICE_INPUT, g);
        bad |= wrong;
        if (!wrong) x = group_of(a, lo, hi, n);
        const int64_t steps = (int64_t)c.num_kv_heads * head_steps(a, x);
        if (x.tiles > 0) {
            const int pairs = (query_rows(a, x) + kPrefixSlots - 1) / kPrefixSlots;
            const float items = (float)(c.num_kv_heads * pairs);
            cost.x += (float)steps * (pairs > 1 ? kStepNs : kColdStepNs) + items * kItemNs, cost.y += items;
        }
        return steps;
    };
    auto scan = [&](int64_t x) {  // inclusive, over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    auto warp_sum = [](float2 x) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x.x += __shfl_xor_sync(0xffffffffu, x.x, o), x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
        return x;
    };
    int64_t all;
    int per = 1, offset = 0;  // the length of a share; this one's place in its first group
    int ctas = 0;             // of the prefixes; the others stream what is left of the rows
    auto share = [&](float2 cost) {
        bad |= all > 0x3fffffff;  // (tables that repeat their pages very often: places are 32-bit numbers below)
        const int total = bad ? 0 : (int)all;
        const GroupStarts starts = {a, bad};
        uint32_t tiles = 0;
        for (int b = threadIdx.x; b < c.batch; b += kThreads) {
            const int n = row_length(c, b, p.status, cta == 0);
            tiles += (uint32_t)(n - starts(b, n) + stream::kTokens - 1) / stream::kTokens;
        }
        tiles = __reduce_add_sync(0xffffffffu, tiles);
        if (lane == 0) B->tiles[warp] = tiles;
        __syncthreads();
        tiles = __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? B->tiles[lane] : 0);
        // both kinds of work end together, by what a step and a tile take of an SM
        const float rest_ns = (float)tiles * (float)(c.num_kv_heads * rest.q_tiles) * kTileNs;
        auto deal = [&](float ns) {
            return total == 0 ? 0 : min(max((int)((float)gridDim.x * (ns / (ns + rest_ns)) + 0.5f), 1), (int)gridDim.x - 1);
        };
        ctas = deal(cost.x);
        if (cost.y > (float)ctas) ctas = deal((float)total * kColdStepNs + cost.y * kItemNs);
        per = max((total + ctas - 1) / max(ctas, 1), 1);
        ctas = (total + per - 1) / per;  // (the last ones' shares would be empty)
        w.first = min(cta * per, total);
        w.left = cta < ctas ? min(per, total - w.first) : 0;
    };
    if (a.groups <= 32) {  // each warp by itself
        Group x;
        float2 cost = make_float2(0.0f, 0.0f);
        const int64_t mine = group_steps(lane, x, cost), sum = scan(mine);
        all = __shfl_sync(0xffffffffu, sum, 31);
        bad = __any_sync(0xffffffffu, bad);
        share(warp_sum(cost));
        const int64_t off = w.first - (sum - mine);
        const uint32_t here = __ballot_sync(0xffffffffu, w.left > 0 && off >= 0 && off < mine);
        w.index = here ? __ffs(here) - 1 : 0;
        offset = __shfl_sync(0xffffffffu, (int)off, w.index);
        w.g.row0 = __shfl_sync(0xffffffffu, x.row0, w.index), w.g.rows = __shfl_sync(0xffffffffu, x.rows, w.index);
        w.g.tiles = __shfl_sync(0xffffffffu, x.tiles, w.index), w.g.tokens = __shfl_sync(0xffffffffu, x.tokens, w.index);
    } else {
        Group x;
        auto block_scan = [&](int64_t v, int64_t &total) {
            const int64_t sum = scan(v);
            __syncthreads();  // (the sums before have been read)
            if (lane == 31) B->sums[warp] = sum;
            __syncthreads();
            int64_t before = 0;
            total = 0;
            for (int i = 0; i < kThreads / 32; ++i) before += i < warp ? B->sums[i] : 0, total += B->sums[i];
            return sum + before;
        };
        int64_t mine = 0;
        float2 cost = make_float2(0.0f, 0.0f), unused = cost;
        for (int g = threadIdx.x; g < a.groups; g += kThreads) mine += group_steps(g, x, cost);
        cost = warp_sum(cost);
        if (lane == 0) B->cost[warp] = cost;
        bad = __syncthreads_or(bad);  // then nothing is taken as shared: the rows' own tables hold all of their tokens
        block_scan(mine, all);
        share(warp_sum(lane < kThreads / 32 ? B->cost[lane] : make_float2(0.0f, 0.0f)));
        int64_t before = 0;
        for (int g0 = 0; w.left > 0 && g0 < a.groups; g0 += kThreads) {
            int64_t total;
            mine = group_steps(g0 + threadIdx.x, x, unused);
            const int64_t sum = block_scan(mine, total), off = w.first - before - (sum - mine);
            if (off >= 0 && off < mine) B->group = g0 + threadIdx.x, B->offset = (int)off;
            before += total;
        }
        __syncthreads();
        if (w.left > 0) {
            w.index = B->group, offset = B->offset;
            w.g = group_at(a, w.index);
        }
    }
    tc_fence_after();
    const uint32_t tmem = B->tmem;
    if (cta >= ctas) {
        if (warp == kWarpMma) tmem_dealloc(tmem, kTmemCols);
        // 12 warps of 168 registers (64512): eight of 232 and four of 40
        if (warp >= stream::kWarps) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
            return;
        }
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        stream::walk_share<uint32_t>(rest, cta - ctas, gridDim.x - ctas, smem, GroupStarts{a, bad},
                                     [] { asm volatile("bar.sync 1, %0;" ::"n"(stream::kThreads) : "memory"); });
        return;
    }
    if (w.left > 0) {
        const int per_head = (int)head_steps(a, w.g), pairs = (query_rows(a, w.g) + kPrefixSlots - 1) / kPrefixSlots;
        w.head = offset / per_head;
        const int in_head = offset - w.head * per_head;
        w.pair = min(in_head / w.g.tiles, pairs - 1);
        w.step = in_head - w.pair * w.g.tiles;
        w.first -= w.step;
        set_item(a, w);
    }
    if (warp >= kWarpKeys) {
        if (warp < kWarpMma) {
            load_tiles(a, w, per, warp == kWarpKeys ? &map_k : &map_v, warp == kWarpKeys, smem, B);
        } else {
            issue_products(a, w, warp - kWarpMma, smem, B);
        }
    } else {
        const int g = warp >> 2, quad = warp & 3, r = 32 * quad + lane;  // the group of warps; the row of its tile
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + 128 * g, col_s = lanes + kColS, col_o = lanes + kColO;
        const float scale2 = fabsf(p.scale) * kLog2e;
        uint32_t count = 0, used = 0, segments = 0;  // tiles before the segment; tiles, and segments, of this group
        bool ok = true;
        for (; ok && w.left > 0; next_segment(a, w)) {
            const bool shared = w.rows > kT;
            const int mine = shared ? g * kT + r : r;  // the query row of the item
            const bool valid = mine < w.rows;
            const int in_group = w.pair * kPrefixSlots + mine, row = in_group / p.group;
            const int head = (w.g.row0 + row) * p.num_q_heads + w.head * p.group + (in_group - row * p.group);
            const int steps = steps_in(w, g);
            if (steps > 0) {  // (a group without a tile writes no queries: it could come by here again before the other)
                // a half-warp reads a row, into the rows of the two swizzled halves
                const uint32_t flip = p.scale < 0.0f ? 0x80008000u : 0u;  // (the scale's sign goes to the queries)
                const int sub = lane >> 4, chunk = lane & 15;
                uint8_t *const dst = smem + kQ + g * kTile + (chunk >> 3) * kHalf + 32 * quad * 128;
                uint4 x[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int from = __shfl_sync(0xffffffffu, valid ? head : -1, 2 * i + sub);
                    x[i] = make_uint4(0, 0, 0, 0);
                    if (from >= 0) x[i] = reinterpret_cast<const uint4 *>(p.q + (int64_t)from * kHeadDim)[chunk];
                }
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    *reinterpret_cast<uint4 *>(dst + (2 * i + sub) * 128 + (((chunk & 7) ^ ((2 * i + sub) & 7)) << 4)) =
                        make_uint4(x[i].x ^ flip, x[i].y ^ flip, x[i].z ^ flip, x[i].w ^ flip);
                fence_async_smem();
                arrive_warp(&B->q[g]);
            }
            if (valid && w.step == 0 && (shared || g == 0)) {
                // this segment begins the item: where its other parts will be
                PrefixCut cut;
                cut.per = shared ? 1 : 2;
                cut.slot = mine;
                cut.cta = cta + 1;
                cut.ctas = (w.first + w.steps - 1) / per - cta;
                a.x.cuts[head] = cut;
            }
            float m = kNegInf, l = 0.0f;
            for (int i = 0; ok && i < steps; ++i, ++used) {
                const uint32_t mask = count + (shared ? i : 2 * i + g);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t col = col_s + 64 * half;
                    ok = wait_warp(&B->s[g][half], used & 1, B);
                    if (!ok) break;
                    tc_fence_after();
                    float s[2][32], sc = scale2;
                    tmem_ld32(col, s[0]);
                    tmem_ld32(col + 32, s[1]);
                    const uint32_t live = (*reinterpret_cast<volatile uint32_t *>(&B->live[mask % kLive]) >> (8 * half)) & 0xffu;
                    tmem_wait_ld();
                    if (live != 0xffu) {
                        const bool zero = scale2 == 0.0f;  // (then -inf would not stay what it is)
                        if (zero) sc = 1.0f;
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                s[b][j] = (live >> (4 * b + (j >> 3))) & 1 ? (zero ? s[b][j] * 0.0f : s[b][j]) : kNegInf;
                    }
                    float top[4];
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const float *const x = &s[b >> 1][16 * (b & 1)];
                        top[b] = fmaxf(x[0], x[15]);
#pragma unroll
                        for (int j = 1; j < 15; j += 2) top[b] = max3(top[b], x[j], x[j + 1]);
                    }
                    // (NaN scores are passed over, and make their row's sum NaN)
                    const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sc;
                    if (i == 0 && half == 0) {
                        m = fmaxf(m, now);
                    } else if (__any_sync(0xffffffffu, now > m + kSlack)) {
                        const float to = fmaxf(m, now), f = to == kNegInf ? 1.0f : ex2(m - to);
                        // P V of the half tile before this one: what was issued behind it are this tile's second scores,
                        // or the next one's first; in the segment's last tile nothing was
                        if (half == 0) ok = wait_warp(&B->s[g][1], used & 1, B);
                        else if (i + 1 < steps) ok = wait_warp(&B->s[g][0], (used + 1) & 1, B);
                        else ok = wait_warp(&B->o[g][0], segments & 1, B);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
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
                    const float ref = m == kNegInf ? 0.0f : -m;
                    const float2 by = make_float2(sc, sc), less = make_float2(ref, ref);
                    float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float pk[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 x = fma2(make_float2(s[b][2 * j], s[b][2 * j + 1]), by, less);
                            x = make_float2(ex2(x.x), ex2(x.y));
                            sum[j & 1] = add2(sum[j & 1], x);
                            pk[j] = __uint_as_float(pack_bf16(x.x, x.y));
                        }
                        tmem_st16(col + 16 * b, pk);
                    }
                    sum[0] = add2(sum[0], sum[1]);
                    l += sum[0].x + sum[0].y;
                    tmem_wait_st();
                    tc_fence_before();
#ifdef KDA_TEST_WITHHOLD_HANDOFF  // failure-detection test: one hand-off never comes
                    if (used != KDA_TEST_WITHHOLD_HANDOFF || half == 0)
#endif
                    arrive_warp(&B->p[g][half]);
                }
            }
            if (!ok) break;
            count += tiles_in(w);
            // ---- the segment's part
            const int part = w.step == 0 ? (shared ? 0 : g * a.x.heads) + head : 3 * a.x.heads + cta * kPrefixSlots + g * kT + r;
            if (steps > 0) {
                ok = wait_warp(&B->o[g][1], segments & 1, B);
                ++segments;
                if (!ok) break;
                tc_fence_after();
            }
            if (valid) a.x.ml[part] = make_float2(m, l);
            // 64 channels at a time through the warp's own rows of the query tile, which have been read, so that a half-warp
            // writes a row
            const int rows_here = min(max(w.rows - (mine - lane), 0), 32), sub = lane >> 4, chunk = lane & 15;
            uint8_t *const rows = smem + kQ + g * kTile + 32 * quad * 128;
#pragma unroll 1
            for (int half = 0; half < 2 && rows_here > 0; ++half) {
                float o[2][32];
#pragma unroll
                for (int j = 0; j < 32; ++j) o[0][j] = o[1][j] = 0.0f;
                if (steps > 0) {
                    tmem_ld32(col_o + 64 * half, o[0]);
                    tmem_ld32(col_o + 64 * half + 32, o[1]);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<float4 *>(rows + b * kHalf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                            make_float4(o[b][4 * j], o[b][4 * j + 1], o[b][4 * j + 2], o[b][4 * j + 3]);
                __syncwarp();
#pragma unroll 4
                for (int r0 = 0; r0 < rows_here; r0 += 2) {
                    const int from = r0 + sub, to = __shfl_sync(0xffffffffu, valid ? part : -1, from);
                    const float4 x = *reinterpret_cast<const float4 *>(rows + (chunk >> 3) * kHalf + from * 128 + (((chunk & 7) ^ (from & 7)) << 4));
                    if (to >= 0) reinterpret_cast<float4 *>(a.x.o + (int64_t)to * kHeadDim + 64 * half)[chunk] = x;
                }
                __syncwarp();
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

// Joins all parts of a query row: those of its prefix and those of the rest, in this order, by `per_row` half-warps of
// a CTA, which take every per_row-th part. A lane has eight channels, and four parts' loads in flight. (With a warp a
// row, 32768 rows of two or three parts: 21.7 instead of 18.2 us from a cold cache.)
constexpr int kJoinThreads = 256, kHalves = kJoinThreads / 16;

__global__ void __launch_bounds__(kJoinThreads, 3) kda_attn_prefix_join_kernel(const stream::Args a, int per_row) {
    __shared__ float s_m[kHalves], s_l[kHalves];
    __shared__ float4 s_o[kHalves][32];
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int64_t head = (int64_t)blockIdx.x * (kHalves / per_row) + half / per_row;
    const int first = half % per_row;
    allow_next();
    wait_for_prior();
    float m = kNegInf, l = 0.0f, o[8] = {};
    auto add = [&](float pm, float pl, float ref, const float4 (&x)[2]) {
        const float f = ex2(pm - ref);
        l = fmaf(pl, f, l);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            o[4 * i] = fmaf(x[i].x, f, o[4 * i]), o[4 * i + 1] = fmaf(x[i].y, f, o[4 * i + 1]);
            o[4 * i + 2] = fmaf(x[i].z, f, o[4 * i + 2]), o[4 * i + 3] = fmaf(x[i].w, f, o[4 * i + 3]);
        }
    };
    if (head < a.x.heads) {
        const int tail = a.x.tails[head];
        const PrefixCut pre = a.x.cuts[head];
        const int before = a.x.start[head / a.p.num_q_heads] == 0 ? 0 : a.x.parts_of(pre);
        stream::Cut cut;
        cut.count = tail == kTailHome ? 1 : 0;
        if (tail >= 0) cut = a.ws.cuts[tail];
        const int row = tail >= 0 ? (int)(head - cut.head) : 0, n = before + cut.count;
        constexpr int kAhead = 4;
        for (int i = first; i < n; i += kAhead * per_row) {
            float pm[kAhead], pl[kAhead];
            float4 po[kAhead][2];
            float top = m;
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const int x = i + e * per_row;
                pm[e] = kNegInf, pl[e] = 0.0f, po[e][0] = po[e][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (x >= n) continue;
                const float *src;
                if (x < before || tail < 0) {
                    const int64_t part = x < before ? a.x.part_at(pre, head, x) : 2 * (int64_t)a.x.heads + head;
                    const float2 ml = a.x.ml[part];
                    pm[e] = ml.x, pl[e] = ml.y;
                    src = a.x.o + part * kHeadDim;
                } else {
                    const stream::Part *const part = a.ws.parts + cut.part_at(x - before);
                    pm[e] = part->m[row], pl[e] = part->l[row];
                    src = part->o[row];
                }
                po[e][0] = reinterpret_cast<const float4 *>(src)[2 * lane], po[e][1] = reinterpret_cast<const float4 *>(src)[2 * lane + 1];
            }
#pragma unroll
            for (int e = 0; e < kAhead; ++e) top = fmaxf(top, pm[e]);
            const float ref = top == kNegInf ? 0.0f : top, keep = ex2(m - ref);
            l *= keep;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= keep;
#pragma unroll
            for (int e = 0; e < kAhead; ++e) add(pm[e], pl[e], ref, po[e]);
            m = top;
        }
    }
    if (per_row > 1) {
        if (lane == 0) s_m[half] = m, s_l[half] = l;
        s_o[half][2 * lane] = make_float4(o[0], o[1], o[2], o[3]), s_o[half][2 * lane + 1] = make_float4(o[4], o[5], o[6], o[7]);
        __syncthreads();
        if (first > 0) return;
        m = kNegInf, l = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = 0.0f;
        for (int w = 0; w < per_row; ++w) m = fmaxf(m, s_m[half + w]);
        const float ref = m == kNegInf ? 0.0f : m;
        for (int w = 0; w < per_row; ++w) {
            const float4 x[2] = {s_o[half + w][2 * lane], s_o[half + w][2 * lane + 1]};
            add(s_m[half + w], s_l[half + w], ref, x);
        }
    }
    if (head >= a.x.heads) return;
    const float inv = 1.0f / l;  // (l = 0: zeros, whatever the values)
    uint4 y = make_uint4(0, 0, 0, 0);
    if (l != 0.0f) y = make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv), pack_bf16(o[4] * inv, o[5] * inv),
                                  pack_bf16(o[6] * inv, o[7] * inv));
    reinterpret_cast<uint4 *>(a.p.out + head * kHeadDim)[lane] = y;
    if (lane == 0 && a.p.lse) a.p.lse[head] = l == 0.0f ? kNegInf : ((m == kNegInf ? 0.0f : m) + log2f(l)) * stream::kLn2;
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

// Where each row reads its own tokens alone anyway: no groups, or so few tokens in all rows' tables that reading them
// row by row takes less than a second launch with its parts. Row by row and shared, in us: 4 rows of 2048 tokens on 8/8
// heads (35 MB) 12.4 and 13.5; 16 of 512 on 64/8 (38 MB) 14.7 and 14.8; 5 of 2048 on 8/8 (43 MB) 13.7 and 13.7; 6 (52 MB) 14.5
// and 13.5; 16 of 768 on 64/8 (55 MB) 16.8 and 15.5; 8 of 2048 on 8/8 (69 MB) 16.3 and 13.8; 8 of 4096 on 32/8 (136 MB)
// 24.6 and 15.8; 64 of 2048 on 64/8 in two groups (554 MB) 74 and 25.5. (With one key head, two rows and 32768 tokens it is
// 19.3 and 22.3.) The host knows the tables' width and not the rows' lengths: short rows in wide tables are shared, too, which
// costs few of them something (512 shared tokens, tables of 576 and of 32768: 4 rows on 8/8 heads 8.5 and 11.8, 8 rows on 32/8
// 9.8 and 12.8, 16 rows 12.2 and 12.9).
constexpr int64_t kFewBytes = 48LL << 20;

cudaError_t launch_attn_prefix(const AttnPrefixArgs &args, cudaStream_t stream) {
    const int64_t reads = (int64_t)args.d.c.batch * args.d.c.num_kv_heads * ((args.d.group + 15) / 16) * args.d.c.capacity;
    if (args.groups == 0 || reads <= kFewBytes / (2 * kHeadDim * 2)) return launch_attn_decode(args.d, stream);
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    AttnPrefixArgs a = args;
    const PagedCache &c = a.d.c;
    prefix_layout(&a.x,
                  static_cast<char *>(a.d.ws) + attn_decode_workspace_bytes(c.batch, a.d.num_q_heads, c.num_kv_heads, c.capacity, false, sms),
                  c.batch, a.d.num_q_heads, sms);
    stream::Args rest;
    if (!stream::stream_args(&rest, a.d, sms)) return launch_attn_decode(args.d, stream);  // (more than 2^35 tokens of all tables)
    rest.x = a.x;
    CUtensorMap map_k, map_v;
    cudaError_t e = page_map(&map_k, c.k, c, c.k_page_stride);
    if (e == cudaSuccess) e = page_map(&map_v, c.v, c, c.v_page_stride);
    if (e == cudaSuccess) e = configure_once();
    if (e == cudaSuccess) e = launch_dependent(kda_attn_prefix_kernel, dim3((unsigned)sms), kThreads, kSmem, stream, a, rest, map_k, map_v);
    if (e != cudaSuccess) return e;
    // half-warps of a query row: all of a CTA's for few rows, which can have long rests in many parts
    int per_row = kHalves;
    while (per_row > 1 && (int64_t)a.x.heads * per_row > (int64_t)sms * 3 * kHalves) per_row /= 2;
    const int rows = kHalves / per_row;
    return launch_dependent(kda_attn_prefix_join_kernel, dim3((unsigned)((a.x.heads + rows - 1) / rows)), kJoinThreads, 0, stream, rest,
                            per_row);
}

}  // namespace kda
