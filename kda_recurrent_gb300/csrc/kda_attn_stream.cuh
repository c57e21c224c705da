// The token stream of attention over a paged key-value cache (sm_103a): what a CTA does of it. kda_attn_decode.cu launches
// it for whole rows, kda_attn_prefix.cu for what is left of rows behind a shared prefix, on some of its CTAs.
//
// Every cached token is read once (512 bytes a key head) and used by the query heads that share
// its key head, so the kernel is an HBM stream. An item is a (row, key head, 16 of its query
// heads); a key head with more of them is read once for every 16. Its tokens come in tiles of 16. All items'
// tiles, laid end to end, are cut into equal shares, one for each CTA (one on an SM) and in it one for each of
// its eight warps, so that any mixture of lengths keeps every warp busy to the end. A warp walks its share
// alone: its own ring of cp.async stages (three tiles, so about 128 KiB are in flight on an SM), no barrier
// with other warps. It keeps the running maximum m, sum l = sum 2^(x - m) and o of its 16 query rows in
// registers; the products are m16n8k16 BF16 tensor-core instructions whose 16 rows are the query heads.
// (Tensor memory and tcgen05 would need 64 or 128 rows; the rows here are 1 to 16, and the tensor work is a
// few percent of the time.) The probabilities are split into two BF16 terms for P V, which costs
// nothing here and leaves the output's own rounding as the only one. A value that is not finite meets only
// the first term (the second may be zero or negative, and would make an infinite channel NaN).
//
// An item inside one share is finished by its warp. An item cut between shares leaves (m, l, o) of each
// part in the workspace; a CTA whose whole share lies in one item joins its warps' parts first, so that
// a long cache leaves one part an SM. A second kernel joins an item's parts in their order, which makes
// the result independent of timing. With `weight`, the first kernel stores the scores (4 bytes a query
// head beside the token's 512) and a third adds 2^(x - lse) to the weights.
//
// 64 rows of 4096 to 32768 tokens, 8 key heads: 727-746 us, 6.8-7.0 TB/s (1.00-1.03 of a copy's rate). 16 rows of
// 1600 tokens, 8 key heads: about 24 us, with weights 30, of which the stream is 16 and the rest start (3: lengths,
// places, first tiles), join, weights and the gaps between the launches. One row of 1000 tokens on 8 heads: 7.7
// us, all latency.
//
// The order of the 128 channels inside a product is free, so the fragments are laid out for 16-byte
// shared-memory reads: a lane's 16 bytes of a key row serve two k-steps, and of a value row eight column
// tiles, which leaves a lane with 16 consecutive output channels. Two swizzles (keys: bit 2 of the
// chunk with the row's parity; values: bits 1-2 with the row pair) keep the reads free of bank
// conflicts.
#pragma once

#include <algorithm>

#include "kda_internal.cuh"
#include "kda_mma.cuh"
#include "kda_prefix.cuh"

namespace kda {
namespace stream {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kTokens = 16;  // of a tile
constexpr int kRows = 16;    // query heads of an item
constexpr int kStages = 3;
constexpr int kStageBytes = 2 * kTokens * kHeadDim * 2;
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr int kMinTiles = 4;  // the least share of a CTA (1000 tokens on 8 heads: 7.5 us; two tiles 7.4, eight 9.1)
constexpr float kNegInf = -INFINITY;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A part of an item: (m, l) of its rows, then o.
struct Part {
    float m[kRows], l[kRows];
    float o[kRows][kHeadDim];
};

// The parts of a cut item, in their order; part i is part_at(i) of the workspace. Kept for the first share that
// begins inside the item (count = 0: the share's beginning cuts no item, or not for the first time).
struct Cut {
    int32_t cta_a, warp_a, n_a;  // its first CTA: parts of n_a warps from warp_a on (or the CTA's one)
    int32_t mid;                 // CTAs that lie inside it
    int32_t cta_b, count;        // its last CTA; all parts
    int32_t head, rows;          // its first row's place among all (row, query head) pairs; its rows
    __device__ __forceinline__ int64_t part_at(int i) const {
        const int64_t share = i < n_a         ? (int64_t)cta_a * kWarps + warp_a + i
                              : i < n_a + mid ? (int64_t)(cta_a + 1 + i - n_a) * kWarps
                                              : (int64_t)cta_b * kWarps + (i - n_a - mid);
        return 2 * share + (i == 0 ? 1 : 0);
    }
};

struct Workspace {
    Cut *cuts;      // [shares]
    float *lse2;    // [batch][query heads]: log2(sum 2^x)
    Part *parts;    // [shares][2]: of an item begun in an earlier share, and of one begun in this share
    float *scores;  // [batch][query heads][capacity] (with weights): x in log2 units
};

__host__ __device__ __forceinline__ int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }

__host__ __device__ __forceinline__ int64_t workspace_layout(Workspace *w, char *base, int64_t batch, int64_t q_heads,
                                                             int64_t capacity, bool with_weight, int64_t shares) {
    int64_t at = 0;
    if (w) w->cuts = reinterpret_cast<Cut *>(base + at);
    at += align16(shares * (int64_t)sizeof(Cut));
    if (w) w->lse2 = reinterpret_cast<float *>(base + at);
    at += align16(batch * q_heads * 4);
    if (w) w->parts = reinterpret_cast<Part *>(base + at);
    at += shares * 2 * (int64_t)sizeof(Part);
    if (w) w->scores = reinterpret_cast<float *>(base + at);
    if (with_weight) at += align16(batch * q_heads * capacity * 4);
    return at;
}

struct Args {
    AttnDecodeArgs p;
    Workspace ws;
    int32_t q_tiles;  // items of a key head
    PrefixParts x;    // (tails only)
};

// What the CTAs of a stream share: what they know of their beginning, then (kTail or not) the warps' last parts.
template <typename U>
struct Shared {
    U sum[kWarps], off[kWarps + 1];
    int32_t row[kWarps + 1], len[kWarps + 1];
    float m[kWarps][kRows], l[kWarps][kRows];
};
template <typename U>
constexpr int kSmem = kRingBytes + kWarps * kStages * 4 + (int)sizeof(Shared<U>);  // (from a 128-byte boundary on)

// Where a row of n tokens begins for the stream: all of it is in tiles (NoStarts), or only its tokens from a start on, a
// multiple of 128 tokens, so that tiles lie in pages as without it. What comes before is then in parts that the row is
// joined with later, like the parts of the rest (kTail).
struct NoStarts {
    static constexpr bool kTail = false;
    __device__ __forceinline__ int operator()(int, int) const { return 0; }
};

// All items' tiles, laid end to end, are cut into CTAs' shares of `per` tiles and those into warps' shares of
// warp_share tiles (the last of each may be shorter): equal numbers rather than equal fractions, because then
// one division places a tile. U is uint32_t when every place fits (the host knows a bound of the total).
template <typename U>
__device__ __forceinline__ U cta_share(U total, int ctas) {
    const U per = (total + ctas - 1) / (U)ctas;
    return per < (U)kMinTiles ? (U)kMinTiles : per;
}

template <typename U>
__device__ __forceinline__ U warp_share(U tiles) {
    return tiles == 0 ? 1 : (tiles + kWarps - 1) / kWarps;
}

__device__ __forceinline__ int page_at(const PagedCache &c, int b, int j, DeviceStatus *st) {
    const int page = c.block_table[(size_t)b * c.max_pages + (j >> c.page_shift)];
    if (page >= c.num_pages) {
        report_error(st, KDA_ERR_DEVICE_INPUT, b);
        return -1;
    }
    return page;
}

// A place in the sequence of tiles: tile `tile` of the `tiles` of item `item` of row b, which has n
// tokens (from token `start` on).
struct Place {
    int b, item, tile, tiles, n, start;
};

template <typename Starts>
__device__ __forceinline__ void set_row(Place &at, const Args &a, int b, const Starts &starts) {
    at.b = b;
    const int n = row_length(a.p.c, b, a.p.status, false);
    at.start = starts(b, n);
    at.n = n - at.start;
    at.tiles = (at.n + kTokens - 1) / kTokens;
}

template <typename Starts>
__device__ __forceinline__ void next_tile(Place &at, const Args &a, int items, const Starts &starts) {
    if (++at.tile < at.tiles) return;
    at.tile = 0;
    if (++at.item < items) return;
    at.item = 0;
    do set_row(at, a, at.b + 1, starts);  // the next row with a token (there is one: the share holds another tile)
    while (at.n == 0 && at.b + 1 < a.p.c.batch);
}

// The cut of the item whose tiles are [x0, x1).
template <typename U>
__device__ __forceinline__ Cut cut_of(U x0, U x1, U total, U per) {
    const U ca = x0 / per, cb = (x1 - 1) / per, a0 = ca * per, b0 = cb * per;
    const U a1 = min(a0 + per, total), b1 = min(b0 + per, total);
    const U wa = warp_share<U>(a1 - a0), wb = warp_share<U>(b1 - b0);
    const U first = (x0 - a0) / wa, last_a = (min(x1, a1) - 1 - a0) / wa, last_b = (x1 - 1 - b0) / wb;
    const bool inside = a0 == x0 && a1 <= x1;  // the first CTA lies inside the item
    Cut c;
    c.cta_a = (int)ca;
    c.cta_b = (int)cb;
    c.mid = cb > ca ? (int)(cb - ca - 1) : 0;
    c.warp_a = inside ? 0 : (int)first;
    c.n_a = inside ? 1 : (int)(last_a - first + 1);
    c.count = c.n_a + c.mid + (cb > ca ? (b1 == x1 ? 1 : (int)last_b + 1) : 0);
    return c;
}

// Two BF16 numbers: those that are not finite as zeros; the larger magnitude of each (NaN if either is one).
__device__ __forceinline__ uint32_t only_finite(uint32_t x) { return x & ~((not_finite(x) >> 15) * 0xffffu); }
__device__ __forceinline__ uint32_t max_abs(uint32_t x, uint32_t y) {
    uint32_t z;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
    return z;
}

// A finished row by one warp: lane's four channels of o over the sum l, at maximum m.
template <bool kTail>
__device__ __forceinline__ void write_row(const Args &a, size_t head, int lane, float m, float l, float4 o) {
    if constexpr (kTail) {  // to be joined with what comes before
        const int64_t part = 2 * (int64_t)a.x.heads + (int64_t)head;
        if (lane == 0) a.x.ml[part] = make_float2(m, l), a.x.tails[head] = kTailHome;
        *reinterpret_cast<float4 *>(a.x.o + part * kHeadDim + 4 * lane) = o;
        return;
    }
    const float inv = 1.0f / l;  // (l = 0: zeros, whatever the values)
    reinterpret_cast<uint2 *>(a.p.out + head * kHeadDim)[lane] =
        l == 0.0f ? make_uint2(0, 0) : make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (lane == 0) {
        const float v = l == 0.0f ? kNegInf : (m == kNegInf ? 0.0f : m) + log2f(l);
        if (a.p.lse) a.p.lse[head] = v * kLn2;
        a.ws.lse2[head] = v;
    }
}

// The work of CTA `cta` of `ctas`, by its first kWarps warps, whose barrier `sync` is.
template <typename U, typename Starts, typename Sync>
__device__ __forceinline__ void walk_share(const Args &a, int cta, int ctas, uint8_t *smem, const Starts &starts, const Sync &sync) {
    constexpr bool kTail = Starts::kTail;
    Shared<U> &S = *reinterpret_cast<Shared<U> *>(smem + kRingBytes + kWarps * kStages * 4);
    const AttnDecodeArgs &p = a.p;
    const PagedCache &c = p.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int items = c.num_kv_heads * a.q_tiles;
    const int share = cta * kWarps + warp;

    // ---- the total, then the row and tile where each warp's share begins, and where the CTA's last tile is
    auto length_of = [&](int b) {
        if (b >= c.batch) return 0;
        const int n = row_length(c, b, p.status, cta == 0), start = starts(b, n);
        if (kTail && b % ctas == cta) a.x.start[b] = start;  // (for the join)
        return n - start;
    };
    auto tiles_of = [&](int n) { return (U)((n + kTokens - 1) / kTokens) * (U)items; };
    auto block_sum = [&](U x, U &before) {  // inclusive prefix sum's total, and the sum before this thread
        U sum = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const U y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        sync();
        if (lane == 31) S.sum[warp] = sum;
        sync();
        U total = 0;
        before = sum - x;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += S.sum[w];
            total += S.sum[w];
        }
        return total;
    };
    const int n0 = length_of(threadIdx.x);
    U mine = tiles_of(n0), before0;
    for (int b = threadIdx.x + kThreads; b < c.batch; b += kThreads) mine += tiles_of(length_of(b));
    const U total = block_sum(mine, before0);
    const U per = cta_share(total, ctas);
    const U cta_lo = min((U)cta * per, total), cta_hi = min(cta_lo + per, total);
    const U per_warp = warp_share<U>(cta_hi - cta_lo);
    U first = 0;
    for (int b0 = 0; b0 < c.batch && cta_lo < cta_hi; b0 += kThreads) {
        // (a batch that fits the block has its sums from above)
        int n = n0;
        U before = before0, sum = total;
        if (c.batch > kThreads) n = length_of(b0 + threadIdx.x), sum = block_sum(tiles_of(n), before);
        const U x = tiles_of(n);
#pragma unroll
        for (int w = 0; w <= kWarps; ++w) {  // (w = kWarps: the CTA's last tile)
            const U place = w == kWarps ? cta_hi - 1 : cta_lo + w * per_warp;
            const U off = place - first - before;  // (wraps when the place lies before)
            if (off < x) S.row[w] = b0 + threadIdx.x, S.off[w] = off, S.len[w] = n;
        }
        first += sum;
    }
    sync();
    const U begin = min(cta_lo + warp * per_warp, cta_hi), end = min(begin + per_warp, cta_hi);
    Place at = {-1, 0, 0, 0, 0, 0};
    if (begin < end) {
        if (kTail) {
            set_row(at, a, S.row[warp], starts);
        } else {
            at.b = S.row[warp], at.n = S.len[warp], at.start = 0;
            at.tiles = (at.n + kTokens - 1) / kTokens;
        }
        at.item = (int)(S.off[warp] / (U)at.tiles);
        at.tile = (int)(S.off[warp] - (U)at.item * at.tiles);
    }
    // Whether the CTA's tiles are all of one item and of several warps, which then join before they leave: its
    // first tile's item, and the end of that.
    bool one_item = false;
    int cta_item = 0, cta_tile = 0, cta_tiles = 0;
    if (cta_hi - cta_lo > per_warp && S.row[0] == S.row[kWarps]) {
        cta_tiles = (S.len[0] + kTokens - 1) / kTokens;
        cta_item = (int)(S.off[0] / (U)cta_tiles);
        cta_tile = (int)(S.off[0] - (U)cta_item * cta_tiles);
        one_item = cta_hi - cta_lo <= (U)(cta_tiles - cta_tile);
    }
    auto empty_rows = [&] {
        for (int b = cta; b < c.batch; b += ctas) {
            const int n = row_length(c, b, p.status, false);
            if (n > starts(b, n)) continue;
            const size_t h0 = (size_t)b * p.num_q_heads;
            if constexpr (kTail) {
                for (int i = threadIdx.x; i < p.num_q_heads; i += kThreads) a.x.tails[h0 + i] = kTailNone;
            } else {
                for (int i = threadIdx.x; i < p.num_q_heads * (kHeadDim / 8); i += kThreads)
                    reinterpret_cast<uint4 *>(p.out + h0 * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
                for (int i = threadIdx.x; i < p.num_q_heads; i += kThreads) {
                    if (p.lse) p.lse[h0 + i] = kNegInf;
                    a.ws.lse2[h0 + i] = kNegInf;
                }
            }
        }
    };
    if (begin >= end) {
        if (lane == 0) a.ws.cuts[share].count = 0;
        if (!one_item) {
            empty_rows();
            return;
        }
    }

    // ---- the ring
    uint8_t *const ring = smem + warp * (kStages * kStageBytes);
    uint32_t *const live = reinterpret_cast<uint32_t *>(smem + kRingBytes) + warp * kStages;  // a bit a token
    const uint32_t ring_addr = smem_addr(ring);
    const int half_row = lane >> 4, chunk = lane & 15;
    Place load = at;
    U to_load = end - begin;  // (0: a warp that is only there for the join)
    auto pages_of = [&](const Place &x) {  // of the tile's two groups of eight tokens
        const int j = x.start + x.tile * kTokens;
        int2 pg;
        pg.x = page_at(c, x.b, j, p.status);
        pg.y = c.page_shift > 3 ? pg.x : j + 8 < x.start + x.n ? page_at(c, x.b, j + 8, p.status) : -1;
        return pg;
    };
    int2 pages = make_int2(-1, -1);
    if (to_load > 0) pages = pages_of(load);
    auto fetch = [&](int stage) {
        if (to_load > 0) {
            const int j0 = load.tile * kTokens, h = load.item / a.q_tiles, mask = c.page_size - 1;
            const int left = load.n - j0, first = load.start + j0;  // tokens
            uint32_t bits = left >= kTokens ? 0xffffu : (1u << left) - 1;
            if (pages.x < 0) bits &= 0xff00u;
            if (pages.y < 0) bits &= 0x00ffu;
            const uint32_t dst = ring_addr + stage * kStageBytes + half_row * 256;
            // two pages' places of the tile's tokens (of this lane's first row and piece), eight tokens from each
            size_t at_k[2], at_v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int page = e == 0 ? pages.x : pages.y;
                const size_t row = ((size_t)h * c.page_size + ((first + 8 * e) & mask) + half_row) * kHeadDim + chunk * 8;
                at_k[e] = page < 0 ? 0 : (size_t)page * c.k_page_stride + row, at_v[e] = page < 0 ? 0 : (size_t)page * c.v_page_stride + row;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {  // (a row that is off lies in the cache, too, but is not read)
                const uint32_t bytes = (bits >> (2 * i + half_row)) & 1 ? 16u : 0u;
                const size_t off = 2 * (i & 3) * kHeadDim;
                cp_async_16(dst + i * 512 + ((chunk ^ (half_row << 2)) << 4), c.k + at_k[i >> 2] + off, bytes);
                cp_async_16(dst + kStageBytes / 2 + i * 512 + ((chunk ^ ((i & 3) << 1)) << 4), c.v + at_v[i >> 2] + off, bytes);
            }
            if (lane == 0) live[stage] = bits;
            if (--to_load > 0) {
                next_tile(load, a, items, starts);
                pages = pages_of(load);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(s);
    // While the first tiles come: if the share's beginning is the first to cut its item, the second kernel joins
    // the item for it. (Found here, because there it would delay everything.)
    if (begin < end) {
        Cut cut;
        cut.count = 0;
        if (at.tile > 0) {
            const U x0 = begin - at.tile;
            // where the share before this one begins (the CTA before is a full one)
            const U before = warp > 0 ? begin - per_warp : begin - ((per - 1) % warp_share(per) + 1);
            if (before <= x0) {
                cut = cut_of<U>(x0, x0 + at.tiles, total, per);
                if (cut.count == 1) cut.count = 0;  // one CTA's, joined there
                const int h = at.item / a.q_tiles, q0 = (at.item - h * a.q_tiles) * kRows;
                cut.head = at.b * p.num_q_heads + h * p.group + q0;
                cut.rows = min(kRows, p.group - q0);
                if (kTail && cut.count > 1 && lane < cut.rows) a.x.tails[cut.head + lane] = share;
            }
        }
        if (lane == 0) a.ws.cuts[share] = cut;
    }
    empty_rows();

    // ---- the share
    const int g = lane >> 2, t = lane & 3;
    const float scale2 = p.scale * kLog2e;
    int stage = 0;
    U left = end - begin;
    while (left > 0) {
        // a segment: this share's tiles of one item
        const int h = at.item / a.q_tiles, q0 = (at.item - h * a.q_tiles) * kRows;
        const int rows = min(kRows, p.group - q0);  // query heads
        const size_t head0 = (size_t)at.b * p.num_q_heads + (size_t)h * p.group + q0;
        const bool from_start = at.tile == 0;
        uint32_t qa[8][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (g < rows) x = reinterpret_cast<const uint4 *>(p.q + (head0 + g) * kHeadDim)[t + 4 * j];
            if (g + 8 < rows) y = reinterpret_cast<const uint4 *>(p.q + (head0 + g + 8) * kHeadDim)[t + 4 * j];
            qa[2 * j][0] = x.x, qa[2 * j][1] = y.x, qa[2 * j][2] = x.y, qa[2 * j][3] = y.y;
            qa[2 * j + 1][0] = x.z, qa[2 * j + 1][1] = y.z, qa[2 * j + 1][2] = x.w, qa[2 * j + 1][3] = y.w;
        }
        float o[16][4];
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.0f, 0.0f};
        const int tiles = (int)min((U)(at.tiles - at.tile), left);
        for (int i = 0; i < tiles; ++i, ++at.tile) {
            cp_async_wait<kStages - 2>();
            __syncwarp();
            const uint8_t *const ks = ring + stage * kStageBytes, *const vs = ks + kStageBytes / 2;
            const uint32_t bits = live[stage];
            float s[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
                const int r = 8 * nt + g;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 k = *reinterpret_cast<const uint4 *>(ks + r * 256 + (((t + 4 * j) ^ ((r & 1) << 2)) << 4));
                    mma_bf16_16816(s[nt], qa[2 * j], k.x, k.y);
                    mma_bf16_16816(s[nt], qa[2 * j + 1], k.z, k.w);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool on = (bits >> (8 * nt + 2 * t + (e & 1))) & 1;
                    s[nt][e] = on ? s[nt][e] * scale2 : kNegInf;
                }
            }
            if (p.weight) {
                float *const dst = a.ws.scores + (head0 + g) * c.capacity + at.tile * kTokens + 2 * t;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
                    if (at.tile * kTokens + 8 * nt < c.capacity) {  // (the capacity is a multiple of eight)
                        if (g < rows) *reinterpret_cast<float2 *>(dst + 8 * nt) = make_float2(s[nt][0], s[nt][1]);
                        if (g + 8 < rows)
                            *reinterpret_cast<float2 *>(dst + 8 * (size_t)c.capacity + 8 * nt) = make_float2(s[nt][2], s[nt][3]);
                    }
            }
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {  // rows g and g + 8
                float top = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float now = fmaxf(m[r], top);
                const float ref = now == kNegInf ? 0.0f : now;
                if (__any_sync(0xffffffffu, now != m[r])) {
                    const float keep = ex2(m[r] - ref);
                    l[r] *= keep;
#pragma unroll
                    for (int i2 = 0; i2 < 16; ++i2) o[i2][2 * r] *= keep, o[i2][2 * r + 1] *= keep;
                    m[r] = now;
                }
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const float p0 = ex2(s[nt][2 * r] - ref), p1 = ex2(s[nt][2 * r + 1] - ref);
                    l[r] += p0 + p1;
                    const uint32_t w = pack_bf16(p0, p1);
                    hi[2 * nt + r] = w;
                    lo[2 * nt + r] = pack_bf16(p0 - __uint_as_float(w << 16), p1 - __uint_as_float(w & 0xffff0000u));
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                // the next tile is asked for here, between the products: with every other place, and with copies whose
                // addresses are formed one by one, the rest of 128 rows takes longer (512 rows of 4096 tokens on 152 SMs 1227
                // us, at the loop's beginning 1302, addresses one by one 1310; without a prefix 1217, 1294 and 1217)
                if (half == 1) fetch(stage == 0 ? kStages - 1 : stage - 1);
                uint4 v[4];  // rows 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                for (int i2 = 0; i2 < 4; ++i2) {
                    const int r = 2 * t + (i2 & 1) + 8 * (i2 >> 1);
                    v[i2] = *reinterpret_cast<const uint4 *>(vs + r * 256 + (((g + 8 * half) ^ (((r >> 1) & 3) << 1)) << 4));
                }
                uint32_t *const v0 = &v[0].x, *const v1 = &v[1].x, *const v2 = &v[2].x, *const v3 = &v[3].x;
                auto add = [&](const uint32_t (&p)[4], int w) {
                    mma_bf16_16816(o[8 * half + 2 * w], p, __byte_perm(v0[w], v1[w], 0x5410), __byte_perm(v2[w], v3[w], 0x5410));
                    mma_bf16_16816(o[8 * half + 2 * w + 1], p, __byte_perm(v0[w], v1[w], 0x7632), __byte_perm(v2[w], v3[w], 0x7632));
                };
                uint32_t top = 0;
#pragma unroll
                for (int w = 0; w < 4; ++w) top = max_abs(max_abs(max_abs(v0[w], v1[w]), max_abs(v2[w], v3[w])), top);
                if (!__any_sync(0xffffffffu, not_finite(top) != 0)) {
#pragma unroll
                    for (int w = 0; w < 4; ++w) add(hi, w), add(lo, w);
                } else {
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        add(hi, w);
                        v0[w] = only_finite(v0[w]), v1[w] = only_finite(v1[w]), v2[w] = only_finite(v2[w]), v3[w] = only_finite(v3[w]);
                        add(lo, w);
                    }
                }
            }
            __syncwarp();  // the stage is read before a later fetch overwrites it
            stage = stage == kStages - 1 ? 0 : stage + 1;
        }
        left -= tiles;
        const bool whole = from_start && at.tile == at.tiles;
        if (one_item) {  // (the share's only segment) to shared memory, over the warp's ring
            cp_async_wait<0>();
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                const int row = g + 8 * r;
                if (t == 0) S.m[warp][row] = m[r], S.l[warp][row] = l[r];
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float4 *const dst = reinterpret_cast<float4 *>(ring + row * 512 + (64 * half + 16 * t + 8 * e) * 4);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            dst[i] = make_float4(o[8 * half + 4 * i][2 * r + e], o[8 * half + 4 * i + 1][2 * r + e],
                                                 o[8 * half + 4 * i + 2][2 * r + e], o[8 * half + 4 * i + 3][2 * r + e]);
                    }
            }
            break;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            const int row = g + 8 * r;
            if (row >= rows) continue;
            if (!kTail && whole) {
                const float inv = 1.0f / l[r];
                const float v = l[r] == 0.0f ? kNegInf : m[r] + log2f(l[r]);
                if (t == 0) {
                    if (p.lse) p.lse[head0 + row] = v * kLn2;
                    a.ws.lse2[head0 + row] = v;
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint4 *const dst = reinterpret_cast<uint4 *>(p.out + (head0 + row) * kHeadDim + 64 * half + 16 * t);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {  // eight channels: one accumulator column of eight tiles
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            w[i] = l[r] == 0.0f ? 0 : pack_bf16(o[8 * half + 2 * i][2 * r + e] * inv, o[8 * half + 2 * i + 1][2 * r + e] * inv);
                        dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            } else {
                Part *const part = a.ws.parts + 2 * (size_t)share + (from_start ? 1 : 0);
                float *o_row = part->o[row];
                if (kTail && whole) {
                    const int64_t home = 2 * (int64_t)a.x.heads + (int64_t)(head0 + row);
                    o_row = a.x.o + home * kHeadDim;
                    if (t == 0) a.x.ml[home] = make_float2(m[r], l[r]), a.x.tails[head0 + row] = kTailHome;
                } else if (t == 0) {
                    part->m[row] = m[r], part->l[row] = l[r];
                }
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float4 *const dst = reinterpret_cast<float4 *>(o_row + 64 * half + 16 * t + 8 * e);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            dst[i] = make_float4(o[8 * half + 4 * i][2 * r + e], o[8 * half + 4 * i + 1][2 * r + e],
                                                 o[8 * half + 4 * i + 2][2 * r + e], o[8 * half + 4 * i + 3][2 * r + e]);
                    }
            }
        }
        if (left > 0) {  // the next item
            --at.tile;
            next_tile(at, a, items, starts);
        }
    }
    cp_async_wait<0>();
    if (!one_item) return;
    // ---- the warps' parts of the CTA's one item: a warp joins every eighth row
    sync();
    const int b = S.row[0], warps = (int)((cta_hi - cta_lo + per_warp - 1) / per_warp);
    const int h = cta_item / a.q_tiles, q0 = (cta_item - h * a.q_tiles) * kRows, rows = min(kRows, p.group - q0);
    const bool whole = cta_tile == 0 && cta_hi - cta_lo == (U)cta_tiles;
    for (int row = warp; row < rows; row += kWarps) {
        float top = kNegInf, l = 0.0f;
        for (int w = 0; w < warps; ++w) top = fmaxf(top, S.m[w][row]);
        const float ref = top == kNegInf ? 0.0f : top;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int w = 0; w < warps; ++w) {
            const float f = ex2(S.m[w][row] - ref);
            const float4 x = *reinterpret_cast<const float4 *>(smem + w * (kStages * kStageBytes) + row * 512 + lane * 16);
            l = fmaf(S.l[w][row], f, l);
            o = make_float4(fmaf(x.x, f, o.x), fmaf(x.y, f, o.y), fmaf(x.z, f, o.z), fmaf(x.w, f, o.w));
        }
        if (whole) {
            write_row<kTail>(a, (size_t)b * p.num_q_heads + (size_t)h * p.group + q0 + row, lane, top, l, o);
        } else {
            Part *const part = a.ws.parts + 2 * (size_t)(cta * kWarps) + (cta_tile == 0 ? 1 : 0);
            if (lane == 0) part->m[row] = top, part->l[row] = l;
            *reinterpret_cast<float4 *>(&part->o[row][4 * lane]) = o;
        }
    }
}

// Fills `a` (but for the parts of a prefix) for a call; whether the places of its tiles fit 32 bits.
inline bool stream_args(Args *a, const AttnDecodeArgs &p, int32_t sms) {
    a->p = p;
    a->q_tiles = (p.group + kRows - 1) / kRows;
    workspace_layout(&a->ws, static_cast<char *>(p.ws), p.c.batch, p.num_q_heads, p.c.capacity, p.weight != nullptr, (int64_t)sms * kWarps);
    // do the tiles there can be, and the end of the last CTA's share, fit 32 bits?
    const int64_t most = (int64_t)p.c.batch * p.c.num_kv_heads * a->q_tiles * ((p.c.capacity + kTokens - 1) / kTokens);
    return most < 0x7fffffffLL;
}

}  // namespace stream
}  // namespace kda
