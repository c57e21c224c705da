// Eviction from a paged key-value cache by accumulated attention weight (sm_103a).
//
// For each (row, key head) longer than the budget, keep the first `sink` and last `recent`
// tokens and the heaviest others (ties: the earlier), packed in order. Two kernels:
//
//  1. Selection, one CTA (or, for few long rows, a cluster) per (row, key head). Weights map to 32-bit keys whose unsigned order
//     is the weights' order; a radix select finds the key T of the last candidate kept (digits of
//     11, 11 and 10 bits from the top: a histogram of the candidates that share the prefix, then
//     the digit where the count from above reaches what is needed; a digit whose tokens all stay
//     ends it). One ordered pass then writes the kept positions: a token's new position is the
//     number kept before it, #(key > T) + min(#(key == T), ties kept) over the tokens before it,
//     which one prefix sum of the two packed counts gives.
//  2. The copy of the kept tokens' keys and values. In place a token moves to an equal or
//     earlier position, so a CTA that owns a slice of columns and walks the tokens in order,
//     reading a tile before it writes it, never overwrites a token still to be read: later
//     tiles' sources lie beyond every position written so far. Slices of columns do not
//     touch each other, which is what the CTAs of one head split by when few heads leave the
//     GPU idle; between disjoint pages the tokens split too.
//
// Bound: the copy's HBM traffic for long rows (32 rows of 8192 to 16384 tokens, 8 heads, cut to 4096: 184 us,
// 25 of them the selection; 5.96 TB/s over the whole, 0.88 of a copy's rate), latency for short ones (2 rows of
// 1500 tokens, 8 heads, cut to 512: 7.4 us; the selection's chain is a row's length beside its weights, two or
// three digits of four barriers each, and the ordered pass).
#include <algorithm>

#include "kda_dependent.cuh"
#include "kda_internal.cuh"
#include "kda_mma.cuh"

namespace kda {
namespace {

constexpr int kElems = 4;  // tokens per thread of a tile
constexpr int kHeld = 4;   // tiles of a block, held in registers together
constexpr int kBins = 2048;

// Unsigned key with the weights' order; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Four tokens' weights from position j (a multiple of four) of a row of n; 0 past its end.
__device__ __forceinline__ float4 four_weights(const float *w, int j, int n) {
    if (j + 4 <= n) return *reinterpret_cast<const float4 *>(w + j);
    return make_float4(j < n ? w[j] : 0.0f, j + 1 < n ? w[j + 1] : 0.0f, j + 2 < n ? w[j + 2] : 0.0f, 0.0f);
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The two words at `p` of this CTA's shared memory, in that of CTA `rank` of the cluster.
__device__ __forceinline__ uint2 load_cluster(const uint32_t *p, int rank) {
    uint32_t at;
    uint2 x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(at));
    return x;
}

// A row by a cluster of kParts CTAs, each with at most a block of its tokens, or by one.
template <int kThreads, int kParts>
__global__ void __launch_bounds__(kThreads) kda_evict_select_kernel(const CacheEvictArgs a) {
    constexpr bool kSplit = kParts > 1;
    constexpr int kWarps = kThreads / 32, kTile = kThreads * kElems, kBlock = kHeld * kTile;
    constexpr int kOwn = kBins / kThreads;  // digits of a thread
    __shared__ __align__(16) uint32_t s_hist[kBins];
    __shared__ uint32_t s_pick[3], s_sum[kWarps], s_warp[2][kWarps];
    __shared__ __align__(8) uint32_t s_total[2];
    wait_for_prior();
    allow_next();
    const int bh = blockIdx.x / kParts, part = blockIdx.x % kParts;
    const int b = bh / a.c.num_kv_heads, h = bh - b * a.c.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float *const w = a.weight + (size_t)bh * a.c.capacity;  // dst may alias: plain loads
    float *const dst = a.dst_weight + (size_t)bh * a.c.capacity;
    int32_t *const kept = a.kept + (size_t)bh * a.budget;
    // A row of one block stays in registers for all passes; a longer one is read again by each, a block's loads
    // together. Where every row is of one block, it is loaded beside its length, up to the capacity.
    const bool short_rows = !kSplit && a.c.capacity <= kBlock;
    float4 held[kHeld];
    auto load_block = [&](int j0, int n) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) held[i] = four_weights(w, j0 + i * kTile + 4 * tid, n);
    };
    if (short_rows) load_block(0, a.c.capacity);
    const int n = row_length(a.c, b, a.status, tid == 0 && h == 0);
    const int m = min(n, a.budget);
    const int every = kParts * kThreads, mine0 = part * kThreads + tid;
    for (int64_t i = (int64_t)m + mine0; i < a.budget; i += every) kept[i] = -1;
    if (n <= a.budget) {
        for (int i = mine0; i < n; i += every) {
            kept[i] = i;
            dst[i] = w[i];
        }
        return;
    }
    const int per = kSplit ? ((n + kParts - 1) / kParts + 3) / 4 * 4 : n;
    const int begin = kSplit ? min(part * per, n) : 0, end = kSplit ? min(begin + per, n) : n;  // this CTA's tokens
    if (!short_rows) load_block(begin, end);
    const int lo = a.sink, hi = n - a.recent;  // candidates: [lo, hi), more than are needed
    uint32_t need = a.budget - a.sink - a.recent, prefix = 0;
    if (need > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass < 2 ? 2048 : 1024;
            const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xffffffffu << 21 : 0xffffffffu << 10;
            for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4 *>(s_hist)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            auto count = [&](const float4 &x4, int j) {
                const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t key = weight_key(x[e]);
                    // (adding up equal digits of a warp first, by a match, took longer than their conflicts)
                    if (j + e >= lo && j + e < min(hi, end) && (key & above) == prefix) atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1u);
                }
            };
            for (int j0 = begin; j0 < end; j0 += kBlock) {
                if (!kSplit && n > kBlock) load_block(j0, n);
#pragma unroll
                for (int i = 0; i < kHeld; ++i)
                    if (j0 + i * kTile + 128 * warp < end) count(held[i], j0 + i * kTile + 4 * tid);
            }
            if (kSplit) cluster_sync(); else __syncthreads();
            // a thread owns kOwn digits; the one where the count from above reaches `need`
            uint32_t c[kOwn], own = 0;
#pragma unroll
            for (int i = 0; i < kOwn; i += 2) {
                uint2 x[kParts];
#pragma unroll
                for (int r = 0; r < kParts; ++r)
                    x[r] = kSplit ? load_cluster(&s_hist[kOwn * tid + i], r) : *reinterpret_cast<const uint2 *>(&s_hist[kOwn * tid + i]);
                c[i] = c[i + 1] = 0;
#pragma unroll
                for (int r = 0; r < kParts; ++r) c[i] += x[r].x, c[i + 1] += x[r].y;
                own += c[i] + c[i + 1];
            }
            uint32_t from = own;  // over this thread's digits and the higher ones of its warp
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_down_sync(0xffffffffu, from, o);
                if (lane + o < 32) from += x;
            }
            if (lane == 0) s_sum[warp] = from;
            __syncthreads();
            uint32_t higher = from - own + __reduce_add_sync(0xffffffffu, lane > warp && lane < kWarps ? s_sum[lane] : 0u);
            if (higher < need && need <= higher + own) {
#pragma unroll
                for (int i = kOwn - 1; i >= 0; --i) {
                    if (higher < need && need <= higher + c[i]) s_pick[0] = kOwn * tid + i, s_pick[1] = need - higher, s_pick[2] = c[i];
                    higher += c[i];
                }
            }
            if (kSplit) cluster_sync(); else __syncthreads();  // (the counts have been read)
            prefix |= s_pick[0] << shift;
            need = s_pick[1];
            if (need == s_pick[2]) {  // all with this prefix stay: no further digit decides
                --prefix;             // (not 0, which would be all candidates, and those are more)
                need = 0;
                break;
            }
        }
    } else {
        prefix = 0xffffffffu;  // no weight has this key: none of the candidates stays
    }
    // prefix: the key T of the last candidate kept; need: how many tokens with that key stay
    uint32_t sure0 = 0, ties0 = 0;  // before this tile: tokens kept for certain, tokens with key T
    int odd = 0;
    auto flags = [&](const float4 &x4, int j, uint32_t (&flag)[kElems]) {
        // ties << 16 | kept for certain (the sums stay below 2^16: a block has at most 2^14 tokens)
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
        uint32_t sum = 0;
#pragma unroll
        for (int e = 0; e < kElems; ++e) {
            const uint32_t key = weight_key(x[e]);
            const bool safe = j + e < lo || j + e >= hi;
            flag[e] = j + e >= end ? 0u : (safe || key > prefix) ? 1u : key == prefix ? 1u << 16 : 0u;
            sum += flag[e];
        }
        return sum;
    };
    if (kSplit) {  // those of the CTAs before (whose weights have been read by now, too)
        uint32_t flag[kElems], sum = 0;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) sum += flags(held[i], begin + i * kTile + 4 * tid, flag);
        sum = __reduce_add_sync(0xffffffffu, sum);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            sum = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_sum[lane] : 0u);
            if (lane == 0) s_total[0] = sum;
        }
        cluster_sync();
#pragma unroll
        for (int r = 0; r < kParts; ++r) {
            const uint32_t x = load_cluster(s_total, r).x;
            sure0 += r < part ? x & 0xffffu : 0u;
            ties0 += r < part ? x >> 16 : 0u;
        }
    }
    auto emit = [&](const float4 &x4, int j) {
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
        uint32_t flag[kElems];
        const uint32_t mine = flags(x4, j, flag);
        uint32_t sum = mine;  // inclusive over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) s_warp[odd][warp] = sum;
        // one barrier a tile (the sums alternate between two arrays): after it the tile's weights have been
        // read, so that they may be overwritten
        __syncthreads();
        const uint32_t all = lane < kWarps ? s_warp[odd][lane] : 0u;
        const uint32_t total = __reduce_add_sync(0xffffffffu, all);
        const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? all : 0u) + sum - mine;
        uint32_t sure = sure0 + (before & 0xffffu), ties = ties0 + (before >> 16);
#pragma unroll
        for (int e = 0; e < kElems; ++e) {
            if (flag[e] == 1u || (flag[e] != 0u && ties < need)) {
                const uint32_t at = sure + min(ties, need);
                kept[at] = j + e;
                dst[at] = x[e];
            }
            sure += flag[e] & 0xffffu;
            ties += flag[e] >> 16;
        }
        sure0 += total & 0xffffu;
        ties0 += total >> 16;
        odd ^= 1;
    };
    for (int j0 = begin; j0 < end; j0 += kBlock) {
        if (!kSplit && n > kBlock) load_block(j0, n);  // (in place: no token of this block has been overwritten yet)
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (j0 + i * kTile < end) emit(held[i], j0 + i * kTile + 4 * tid);
    }
    // (in place: every tile is done before its tail is cleared; a cluster's CTAs leave when the others have read
    // their shared memory)
    if (kSplit) cluster_sync(); else __syncthreads();
    for (int i = m + mine0; i < n; i += every) dst[i] = 0.0f;
}

// Threads of a row's CTA: short rows take 256, whose barriers cost less and of which several CTAs share an SM.
// Whole call with 256 and 1024, in us: 8 row-heads of up to 600 tokens 6.0 and 6.9, of 1500 6.7 and 7.2, of
// 4096 8.2 and 7.5; 296 of 600 15.0 and 17.5, of 4096 61.3 and 60.5.
constexpr int kShortThreads = 256, kLongThreads = 1024, kShortRow = 2048;
// Few long rows are each split over a cluster, as long as its CTAs can hold the row. Whole call, cut to an eighth,
// by one CTA and by eight, in us: 8 row-heads of 16384 tokens 15.6 and 20.3, of 32768 27.7 and 23.2, 2 of 131072
// 88 and 30 (the eight exchange 64 KiB a digit and wait for one another eight times).
constexpr int kSplitParts = 8, kSplitRow = 32768;

constexpr int kCopyWarps = 8;
constexpr int kCopyThreads = kCopyWarps * 32;
constexpr int kCopyUnroll = 8;                     // 16-byte vectors a lane moves of a tile
constexpr int kTileBytes = 32 * kCopyUnroll * 16;  // of a warp

struct Move {
    const __nv_bfloat16 *src;
    __nv_bfloat16 *dst;  // NULL: nothing to do
};

// Position j of a row moves to position i; `head`: the key head's place in a page, ps and pd the two pages.
__device__ __forceinline__ Move move_of(const CacheEvictArgs &a, __nv_bfloat16 *head, int64_t stride, int b, int i, int j, int ps, int pd) {
    const PagedCache &c = a.c;
    const int mask = c.page_size - 1;
    if (j < 0) return {nullptr, nullptr};
    if (ps < 0 || ps >= c.num_pages || pd < 0 || pd >= c.num_pages) {
        report_error(a.status, KDA_ERR_DEVICE_INPUT, b);
        return {nullptr, nullptr};
    }
    if (ps == pd && ((i ^ j) & mask) == 0) return {nullptr, nullptr};  // it stays where it is
    return {head + (int64_t)ps * stride + (int64_t)(j & mask) * kHeadDim, head + (int64_t)pd * stride + (int64_t)(i & mask) * kHeadDim};
}

// A warp's tile of a stage (its vectors, then its moves, kVecs vectors each): loads begun, and stored.
template <int kVecs>
__device__ __forceinline__ void fetch_tile(uint8_t *stage, int lane) {
    const Move *const moves = reinterpret_cast<const Move *>(stage + kTileBytes);
    const uint32_t to = smem_addr(stage) + lane * 16;
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        const Move mv = moves[u * (32 / kVecs) + lane / kVecs];
        if (mv.dst) cp_async_16(to + u * 512, mv.src + lane % kVecs * 8, 16u);
    }
}

template <int kVecs>
__device__ __forceinline__ void store_tile(const uint8_t *stage, int lane) {
    const Move *const moves = reinterpret_cast<const Move *>(stage + kTileBytes);
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) {
        __nv_bfloat16 *const dst = moves[u * (32 / kVecs) + lane / kVecs].dst;
        if (dst) *reinterpret_cast<uint4 *>(dst + lane % kVecs * 8) = *reinterpret_cast<const uint4 *>(stage + lane * 16 + u * 512);
    }
}

// Between disjoint pages: a warp moves 16 kept tokens' keys or values, all loads (position -> pages -> rows, by
// cp.async) before the stores; 48 warps an SM hide each other's latency, about 190 KiB in flight. 256 row-heads
// cut to 4096 tokens of 8192 to 16384: 182 us with the selection; warps that walk up to 16 such tiles through a
// ring of three: 187; the same by one wave of CTAs: 200.
constexpr int kCopyTokens = 2 * kCopyUnroll;  // of a warp
constexpr int kCopyStage = kTileBytes + kCopyTokens * (int)sizeof(Move);

__global__ void __launch_bounds__(kCopyThreads) kda_evict_copy_kernel(const CacheEvictArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    const PagedCache &c = a.c;
    const int bh = blockIdx.x, b = bh / c.num_kv_heads, h = bh - b * c.num_kv_heads;
    const bool values = blockIdx.y == 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *const stage = smem + warp * kCopyStage;
    allow_next();
    wait_for_prior();  // the selection is complete
    const int m = min(row_length(c, b, a.status, false), a.budget);  // (the same from the new lengths)
    if (blockIdx.y == 0 && blockIdx.z == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = m;
    const int64_t stride = values ? c.v_page_stride : c.k_page_stride;
    __nv_bfloat16 *const head = (values ? c.v : c.k) + (size_t)h * c.page_size * kHeadDim;
    const int32_t *const from = c.block_table + (size_t)b * c.max_pages, *const to = a.dst_table + (size_t)b * c.max_pages;
    for (int64_t i0 = ((int64_t)blockIdx.z * kCopyWarps + warp) * kCopyTokens; i0 < m; i0 += (int64_t)gridDim.z * kCopyWarps * kCopyTokens) {
        if (lane < kCopyTokens) {
            const int i = (int)i0 + lane, j = i < m ? a.kept[(size_t)bh * a.budget + i] : -1;
            int ps = 0, pd = 0;
            if (j >= 0) ps = from[j >> c.page_shift], pd = to[i >> c.page_shift];
            reinterpret_cast<Move *>(stage + kTileBytes)[lane] = move_of(a, head, stride, b, i, j, ps, pd);
        }
        __syncwarp();
        fetch_tile<16>(stage, lane);
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
        store_tile<16>(stage, lane);
        __syncwarp();
    }
}

// In place. A CTA has a slice of kVecs 16-byte vectors of a (row, key head)'s keys or values, and walks its
// tokens in order; a tile of the whole CTA is read before any of it is written. So few CTAs run at once: a warp
// moves its part of a tile through its own ring, rows arriving two tiles ahead, their moves looked up one step
// further ahead, so that only the rows' own latency is left and about 128 KiB are in flight on an SM.
constexpr int kCopyStages = 3;

template <int kVecs>
constexpr int kPackSmem = kCopyWarps * kCopyStages * (kTileBytes + 32 * kCopyUnroll / kVecs * (int)sizeof(Move));
template <int kVecs>  // CTAs on an SM: of its 228 KiB each takes 1 KiB more
constexpr int kPackCtas = 228 * 1024 / (kPackSmem<kVecs> + 1024);
static_assert(kPackCtas<4> == 1 && kPackCtas<8> == 2 && kPackCtas<16> == 2, "the moves of narrow slices take a third of their memory");

template <int kVecs>
__global__ void __launch_bounds__(kCopyThreads) kda_evict_pack_kernel(const CacheEvictArgs a) {
    constexpr int kSlices = 16 / kVecs;
    constexpr int kTokens = 32 * kCopyUnroll / kVecs;  // 16, 32 or 64
    constexpr int kEach = (kTokens + 31) / 32;         // tokens a lane looks up
    constexpr int kStep = kTokens * kCopyWarps;        // tokens of a tile of the CTA
    constexpr int kStageBytes = kTileBytes + kTokens * (int)sizeof(Move);
    extern __shared__ __align__(16) uint8_t smem[];
    const PagedCache &c = a.c;
    const int bh = blockIdx.x, b = bh / c.num_kv_heads, h = bh - b * c.num_kv_heads;
    const int slice = blockIdx.y % kSlices;
    const bool values = blockIdx.y >= kSlices;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    allow_next();
    wait_for_prior();  // the selection is complete
    const int m = min(row_length(c, b, a.status, false), a.budget);  // (the same from the new lengths)
    if (blockIdx.y == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = m;
    const int64_t stride = values ? c.v_page_stride : c.k_page_stride;
    __nv_bfloat16 *const head = (values ? c.v : c.k) + (size_t)h * c.page_size * kHeadDim + slice * kVecs * 8;
    const int32_t *const kept = a.kept + (size_t)bh * a.budget;
    const int32_t *const table = c.block_table + (size_t)b * c.max_pages;
    uint8_t *const ring = smem + warp * (kCopyStages * kStageBytes);
    const int tiles = (m + kStep - 1) / kStep;

    int j[kEach], jp[kEach], ps[kEach], pd[kEach];  // positions of one tile; of the tile before it, with pages
    auto token = [&](int tile, int e) { return warp * kTokens + tile * kStep + lane + 32 * e; };
    auto positions = [&](int tile) {
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            j[e] = tile < tiles && lane + 32 * e < kTokens && token(tile, e) < m ? kept[token(tile, e)] : -1;
    };
    auto pages = [&](int tile) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            jp[e] = j[e];
            if (j[e] >= 0) ps[e] = table[j[e] >> c.page_shift], pd[e] = table[token(tile, e) >> c.page_shift];
        }
    };
    auto fetch = [&](int tile) {
        uint8_t *const stage = ring + (tile % kCopyStages) * kStageBytes;
        if (tile < tiles) {
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                if (lane + 32 * e < kTokens)
                    reinterpret_cast<Move *>(stage + kTileBytes)[lane + 32 * e] =
                        move_of(a, head, stride, b, token(tile, e), jp[e], ps[e], pd[e]);
            __syncwarp();
            fetch_tile<kVecs>(stage, lane);
        }
        cp_async_commit();
    };
    positions(0);
    pages(0);
    positions(1);
    fetch(0);
    pages(1);
    positions(2);
    fetch(1);
    pages(2);
    positions(3);
    for (int tile = 0; tile < tiles; ++tile) {
        fetch(tile + 2);
        pages(tile + 3);
        positions(tile + 4);
        cp_async_wait<2>();
        __syncthreads();
        store_tile<kVecs>(ring + (tile % kCopyStages) * kStageBytes, lane);
        __syncwarp();
    }
    cp_async_wait<0>();
}

template <int kVecs>
cudaError_t launch_pack(const CacheEvictArgs &a, cudaStream_t stream) {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kda_evict_pack_kernel<kVecs>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPackSmem<kVecs>);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    const dim3 grid((unsigned)(a.c.batch * a.c.num_kv_heads), 2 * (16 / kVecs));
    return launch_dependent(kda_evict_pack_kernel<kVecs>, grid, kCopyThreads, kPackSmem<kVecs>, stream, a);
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream) {
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    const dim3 rows_heads((unsigned)(a.c.batch * a.c.num_kv_heads));
    const bool split = a.c.capacity >= kSplitRow && a.c.capacity <= kSplitParts * kLongThreads * kElems * kHeld &&
                       (int64_t)rows_heads.x * kSplitParts <= sms;
    const cudaError_t e =
        split ? launch_clusters(kSplitParts, kda_evict_select_kernel<kLongThreads, kSplitParts>, dim3(rows_heads.x * kSplitParts),
                                kLongThreads, 0, stream, a)
        : a.c.capacity <= kShortRow ? launch_dependent(kda_evict_select_kernel<kShortThreads, 1>, rows_heads, kShortThreads, 0, stream, a)
                                    : launch_dependent(kda_evict_select_kernel<kLongThreads, 1>, rows_heads, kLongThreads, 0, stream, a);
    if (e != cudaSuccess) return e;
    const int rows = a.c.batch * a.c.num_kv_heads;
    if (a.dst_table != a.c.block_table) {
        const int parts = (std::min(a.budget, a.c.capacity) + kCopyWarps * kCopyTokens - 1) / (kCopyWarps * kCopyTokens);
        constexpr int kSmem = kCopyWarps * kCopyStage;
        static_assert(kSmem <= 48 * 1024, "no opt-in");
        return launch_dependent(kda_evict_copy_kernel, dim3((unsigned)rows, 2, (unsigned)std::min(parts, 65535)), kCopyThreads, kSmem,
                                stream, a);
    }
    // The narrowest slices whose CTAs still run at once. Whole call for 2000 of 4096 tokens of 8, 19, 20, 30, 64, 76,
    // 144 and 312 row-heads with slices of 64 / 128 / 256 bytes, in us: 12 / 15 / 23, 13 / 16 / 24, 18 / 16 / 24,
    // 19 / 16 / 24, 35 / 25 / 34, 40 / 29 / 36, 73 / 55 / 53, 191 / 124 / 127.
    if (4 * 2 * (int64_t)rows <= kPackCtas<4> * sms) return launch_pack<4>(a, stream);
    if (2 * 2 * (int64_t)rows <= kPackCtas<8> * sms) return launch_pack<8>(a, stream);
    return launch_pack<16>(a, stream);
}

}  // namespace kda
