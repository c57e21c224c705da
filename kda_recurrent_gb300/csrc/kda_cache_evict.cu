// Eviction from a paged key-value cache by accumulated attention weight (sm_103a).
//
// For each (row, key head) longer than the budget, keep the first `sink` and last `recent`
// tokens and the heaviest others (ties: the earlier), packed in order. Two kernels:
//
//  1. Selection, one CTA per (row, key head). Weights map to 32-bit keys whose unsigned order
//     is the weights' order; a radix select finds the key T of the last candidate kept (digits of
//     11, 11 and 10 bits from the top: a histogram of the candidates that share the prefix, then
//     the digit where the count from above reaches what is needed). One ordered pass then
//     writes the kept positions: a token's new position is the number kept before it,
//     #(key > T) + min(#(key == T), ties kept) over the tokens before it, which one prefix
//     sum of the two packed counts gives.
//  2. The copy of the kept tokens' keys and values. In place a token moves to an equal or
//     earlier position, so a CTA that owns a slice of columns and walks the tokens in order,
//     reading a tile before it writes it, never overwrites a token still to be read: later
//     tiles' sources lie beyond every position written so far. Slices of columns do not
//     touch each other, which is what the CTAs of one head split by when few heads leave the
//     GPU idle; between disjoint pages the tokens split too.
#include <algorithm>

#include "kda_dependent.cuh"
#include "kda_internal.cuh"
#include "kda_mma.cuh"

namespace kda {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelElems = 4;                        // tokens per thread of a tile
constexpr int kSelTile = kSelThreads * kSelElems;
constexpr int kHeld = 4;                            // tiles of a block, held in registers together
constexpr int kBlock = kHeld * kSelTile;
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

__global__ void __launch_bounds__(kSelThreads, 1) kda_evict_select_kernel(const CacheEvictArgs a) {
    __shared__ uint32_t s_hist[kBins], s_pick[2], s_sum[kSelWarps];
    __shared__ uint64_t s_warp[2][kSelWarps];
    wait_for_prior();
    allow_next();
    const int bh = blockIdx.x, b = bh / a.c.num_kv_heads, h = bh - b * a.c.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = row_length(a.c, b, a.status, tid == 0 && h == 0);
    const int m = min(n, a.budget);
    const float *const w = a.weight + (size_t)bh * a.c.capacity;  // dst may alias: plain loads
    float *const dst = a.dst_weight + (size_t)bh * a.c.capacity;
    int32_t *const kept = a.kept + (size_t)bh * a.budget;
    for (int64_t i = (int64_t)m + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
    if (n <= a.budget) {
        for (int i = tid; i < n; i += kSelThreads) {
            kept[i] = i;
            dst[i] = w[i];
        }
        return;
    }
    // a row of one block stays in registers for all passes; a longer one is read again by each, a block's
    // loads together
    float4 held[kHeld];
    auto load_block = [&](int j0) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) held[i] = four_weights(w, j0 + i * kSelTile + 4 * tid, n);
    };
    load_block(0);
    const int lo = a.sink, hi = n - a.recent;  // candidates: [lo, hi), more than are needed
    uint32_t need = a.budget - a.sink - a.recent, prefix = 0;
    if (need > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass < 2 ? 2048 : 1024;
            const uint32_t above = pass == 0 ? 0u : pass == 1 ? 0xffffffffu << 21 : 0xffffffffu << 10;
            for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
            __syncthreads();
            auto count = [&](const float4 &x4, int j) {
                const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t key = weight_key(x[e]);
                    // (adding up equal digits of a warp first, by a match, took longer than their conflicts)
                    if (j + e >= lo && j + e < hi && (key & above) == prefix) atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1u);
                }
            };
            for (int j0 = 0; j0 < n; j0 += kBlock) {
                if (n > kBlock) load_block(j0);
#pragma unroll
                for (int i = 0; i < kHeld; ++i) count(held[i], j0 + i * kSelTile + 4 * tid);
            }
            __syncthreads();
            // thread i owns digits 2 i and 2 i + 1; the digit where the count from above reaches `need`
            const uint32_t c0 = s_hist[2 * tid], c1 = s_hist[2 * tid + 1];
            uint32_t from = c0 + c1;  // over this thread's digits and the higher ones of its warp
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_down_sync(0xffffffffu, from, o);
                if (lane + o < 32) from += x;
            }
            if (lane == 0) s_sum[warp] = from;
            __syncthreads();
            uint32_t rest = lane > warp ? s_sum[lane] : 0;  // (32 warps: a lane for each)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
            const uint32_t higher = from + rest - c0 - c1;  // above digit 2 i + 1
            if (higher < need && need <= higher + c1) s_pick[0] = 2 * tid + 1, s_pick[1] = need - higher;
            if (higher + c1 < need && need <= higher + c1 + c0) s_pick[0] = 2 * tid, s_pick[1] = need - higher - c1;
            __syncthreads();
            prefix |= s_pick[0] << shift;
            need = s_pick[1];
        }
    } else {
        prefix = 0xffffffffu;  // no weight has this key: none of the candidates stays
    }
    // prefix: the key T of the last candidate kept; need: how many tokens with that key stay
    uint64_t run = 0;  // tokens before this tile: (key == T) << 32 | kept for certain
    int odd = 0;
    auto emit = [&](const float4 &x4, int j) {
        const float x[4] = {x4.x, x4.y, x4.z, x4.w};
        uint64_t mine = 0, flag[kSelElems];
#pragma unroll
        for (int e = 0; e < kSelElems; ++e) {
            const uint32_t key = weight_key(x[e]);
            const bool safe = j + e < lo || j + e >= hi;
            flag[e] = j + e >= n ? 0ull : (safe || key > prefix) ? 1ull : key == prefix ? 1ull << 32 : 0ull;
            mine += flag[e];
        }
        uint64_t sum = mine;  // inclusive over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) s_warp[odd][warp] = sum;
        // one barrier a tile (the sums alternate between two arrays): after it the tile's weights have been
        // read, so that they may be overwritten
        __syncthreads();
        const uint64_t all = s_warp[odd][lane];
        uint64_t before = lane < warp ? all : 0, total = all;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, o);
            total += __shfl_xor_sync(0xffffffffu, total, o);
        }
        before += run + sum - mine;
#pragma unroll
        for (int e = 0; e < kSelElems; ++e) {
            const uint32_t sure = (uint32_t)before, ties = (uint32_t)(before >> 32);
            const bool stays = flag[e] == 1ull || (flag[e] != 0 && ties < need);
            if (stays) {
                const uint32_t at = sure + min(ties, need);
                kept[at] = j + e;
                dst[at] = x[e];
            }
            before += flag[e];
        }
        run += total;
        odd ^= 1;
    };
    for (int j0 = 0; j0 < n; j0 += kBlock) {
        if (n > kBlock) load_block(j0);  // (in place: no token of this block has been overwritten yet)
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (j0 + i * kSelTile < n) emit(held[i], j0 + i * kSelTile + 4 * tid);
    }
    __syncthreads();  // (in place: every tile is done before its tail is cleared)
    for (int i = m + tid; i < n; i += kSelThreads) dst[i] = 0.0f;
}

constexpr int kCopyWarps = 8;
constexpr int kCopyThreads = kCopyWarps * 32;
constexpr int kCopyStages = 3;
constexpr int kCopyUnroll = 8;                             // 16-byte vectors a lane moves of a tile
constexpr int kTileBytes = 32 * kCopyUnroll * 16;          // of a warp

struct Move {
    int64_t src, dst;  // elements from the cache's base; dst < 0: nothing to do
};

// kVecs: 16-byte vectors of a token's row that this CTA's slice holds (16, 8 or 4). A warp moves tiles of
// kTokens tokens through its own ring: rows arrive by cp.async two tiles ahead, their moves (position ->
// pages -> offsets, two dependent loads) are looked up one step further ahead, so that only the rows'
// own latency is left and about 128 KiB are in flight on an SM. (Rows held in registers instead, eight
// a thread: 4.1 TB/s read and written.) kOrdered: in place, a tile of the whole CTA is read before any
// of it is written.
template <int kVecs, bool kOrdered>
__global__ void __launch_bounds__(kCopyThreads) kda_evict_copy_kernel(const CacheEvictArgs a, int rows_per_cta) {
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
    const int m = min(row_length(c, b, a.status, false), a.budget);  // (the same from the new lengths)
    const int64_t begin = (int64_t)blockIdx.z * rows_per_cta;
    const int end = (int)min((int64_t)m, begin + rows_per_cta);
    wait_for_prior();  // the selection is complete
    if (blockIdx.y == 0 && blockIdx.z == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = m;
    if (begin >= end) return;
    const int64_t stride = values ? c.v_page_stride : c.k_page_stride;
    const int mask = c.page_size - 1;
    __nv_bfloat16 *const cache = (values ? c.v : c.k) + (size_t)h * c.page_size * kHeadDim + (slice * kVecs + lane % kVecs) * 8;
    const int32_t *const kept = a.kept + (size_t)bh * a.budget;
    const int32_t *const from = c.block_table + (size_t)b * c.max_pages, *const to = a.dst_table + (size_t)b * c.max_pages;
    uint8_t *const ring = smem + warp * (kCopyStages * kStageBytes);
    const int tiles = (end - (int)begin + kStep - 1) / kStep;
    const int mine = (int)begin + warp * kTokens;  // this warp's first token; + kStep a tile

    int j[kEach], jp[kEach], ps[kEach], pd[kEach];  // positions of one tile; of the tile before it, with pages
    auto positions = [&](int tile) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = mine + tile * kStep + lane + 32 * e;
            j[e] = tile < tiles && lane + 32 * e < kTokens && i < end ? kept[i] : -1;
        }
    };
    auto pages = [&](int tile) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = mine + tile * kStep + lane + 32 * e;
            jp[e] = j[e];
            if (j[e] >= 0) ps[e] = from[j[e] >> c.page_shift], pd[e] = to[i >> c.page_shift];
        }
    };
    auto fetch = [&](int tile) {
        uint8_t *const stage = ring + (tile % kCopyStages) * kStageBytes;
        Move *const moves = reinterpret_cast<Move *>(stage + kTileBytes);
        if (tile < tiles) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                if (lane + 32 * e >= kTokens) continue;
                const int i = mine + tile * kStep + lane + 32 * e;
                Move mv = {0, -1};
                if (jp[e] >= 0) {
                    if (ps[e] < 0 || ps[e] >= c.num_pages || pd[e] < 0 || pd[e] >= c.num_pages)
                        report_error(a.status, KDA_ERR_DEVICE_INPUT, b);
                    else if (ps[e] != pd[e] || ((i ^ jp[e]) & mask) != 0)  // else it stays where it is
                        mv = {(int64_t)ps[e] * stride + (int64_t)(jp[e] & mask) * kHeadDim,
                              (int64_t)pd[e] * stride + (int64_t)(i & mask) * kHeadDim};
                }
                moves[lane + 32 * e] = mv;
            }
            __syncwarp();
            const uint32_t dst = smem_addr(stage) + lane * 16;
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u) {
                const Move mv = moves[u * (32 / kVecs) + lane / kVecs];
                if (mv.dst >= 0) cp_async_16(dst + u * 512, cache + mv.src, 16u);
            }
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
        if (kOrdered) __syncthreads(); else __syncwarp();
        const uint8_t *const stage = ring + (tile % kCopyStages) * kStageBytes;
        const Move *const moves = reinterpret_cast<const Move *>(stage + kTileBytes);
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            const int64_t dst = moves[u * (32 / kVecs) + lane / kVecs].dst;
            if (dst >= 0) *reinterpret_cast<uint4 *>(cache + dst) = *reinterpret_cast<const uint4 *>(stage + lane * 16 + u * 512);
        }
        __syncwarp();  // the stage is read before it is filled again
    }
    cp_async_wait<0>();
}

template <int kVecs, bool kOrdered>
cudaError_t launch_copy(const CacheEvictArgs &a, int rows_per_cta, unsigned parts, cudaStream_t stream) {
    constexpr int kSmem = kCopyWarps * kCopyStages * (kTileBytes + 32 * kCopyUnroll / kVecs * (int)sizeof(Move));
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kda_evict_copy_kernel<kVecs, kOrdered>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return launch_dependent(kda_evict_copy_kernel<kVecs, kOrdered>,
                            dim3((unsigned)(a.c.batch * a.c.num_kv_heads), 2 * (16 / kVecs), parts), kCopyThreads, kSmem, stream, a,
                            rows_per_cta);
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream) {
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    const cudaError_t e =
        launch_dependent(kda_evict_select_kernel, dim3((unsigned)(a.c.batch * a.c.num_kv_heads)), kSelThreads, 0, stream, a);
    if (e != cudaSuccess) return e;
    const int most = std::min(a.budget, a.c.capacity);  // tokens a row can keep
    const int64_t ctas = (int64_t)a.c.batch * a.c.num_kv_heads * 2;
    if (a.dst_table != a.c.block_table) {
        // one tile a CTA, or up to sixteen where that still leaves several CTAs for every SM
        const int tile = 2 * kCopyUnroll * kCopyWarps;
        const int64_t tiles = (most + tile - 1) / tile;
        const int64_t per = std::max<int64_t>((tiles + 65534) / 65535, std::min<int64_t>(16, ctas * tiles / (8 * sms)));
        const int rows = (int)(std::max<int64_t>(per, 1) * tile);
        return launch_copy<16, false>(a, rows, (unsigned)(((int64_t)most + rows - 1) / rows), stream);
    }
    if (ctas >= 4 * sms) return launch_copy<16, true>(a, most, 1, stream);
    if (ctas >= 2 * sms) return launch_copy<8, true>(a, most, 1, stream);
    return launch_copy<4, true>(a, most, 1, stream);
}

}  // namespace kda
