// Eviction from a paged key-value cache by accumulated attention weight (sm_103a).
//
// For each (row, key head) longer than the budget, keep the first `sink` and last `recent`
// tokens and the heaviest others (ties: the earlier), packed in order. Two kernels:
//
//  1. Selection, one CTA per (row, key head). Weights map to 32-bit keys whose unsigned order
//     is the weights' order; a radix select finds the key T of the last candidate kept (eight
//     bits at a time from the top: a histogram of the candidates that share the prefix, then
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

#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelElems = 4;                        // tokens per thread of a tile
constexpr int kSelTile = kSelThreads * kSelElems;
constexpr int kBins = 256;

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Unsigned key with the weights' order; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) kda_evict_select_kernel(const CacheEvictArgs a) {
    __shared__ uint32_t s_hist[kBins], s_pick[2];
    __shared__ uint64_t s_warp[kSelWarps];
    pdl_launch_dependents();
    const int bh = blockIdx.x, b = bh / a.c.num_kv_heads, h = bh - b * a.c.num_kv_heads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = row_length(a.c, b, a.status, tid == 0 && h == 0);
    const int m = min(n, a.budget);
    const float *const w = a.weight + (size_t)bh * a.c.capacity;  // dst may alias: plain loads
    float *const dst = a.dst_weight + (size_t)bh * a.c.capacity;
    int32_t *const kept = a.kept + (size_t)bh * a.budget;
    for (int i = m + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
    if (n <= a.budget) {
        for (int i = tid; i < n; i += kSelThreads) {
            kept[i] = i;
            dst[i] = w[i];
        }
        return;
    }
    const int lo = a.sink, hi = n - a.recent;  // candidates: [lo, hi), more than are needed
    uint32_t need = a.budget - a.sink - a.recent, prefix = 0;
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
            __syncthreads();
            const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int j = lo + tid; j < hi; j += kSelThreads) {
                const uint32_t key = weight_key(w[j]);
                if ((key & above) == prefix) atomicAdd(&s_hist[(key >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (warp == 0) {  // lane i owns digits [8 i, 8 i + 8)
                uint32_t c[8], sum = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e] = s_hist[8 * lane + e], sum += c[e];
                uint32_t from = sum;  // count of the digits of this lane and above
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t x = __shfl_down_sync(0xffffffffu, from, o);
                    if (lane + o < 32) from += x;
                }
                uint32_t higher = from - sum;
                if (higher < need && need <= from) {
#pragma unroll
                    for (int e = 7; e >= 0; --e) {
                        if (higher < need && need <= higher + c[e]) s_pick[0] = 8 * lane + e, s_pick[1] = need - higher;
                        higher += c[e];
                    }
                }
            }
            __syncthreads();
            prefix |= s_pick[0] << shift;
            need = s_pick[1];
            __syncthreads();
        }
    } else {
        prefix = 0xffffffffu;  // no weight has this key: none of the candidates stays
    }
    // prefix: the key T of the last candidate kept; need: how many tokens with that key stay
    uint64_t run = 0;  // tokens before this tile: (key == T) << 32 | kept for certain
    for (int j0 = 0; j0 < n; j0 += kSelTile) {
        const int j = j0 + tid * kSelElems;
        float x[kSelElems];
        uint64_t mine = 0, flag[kSelElems];
#pragma unroll
        for (int e = 0; e < kSelElems; ++e) {
            x[e] = j + e < n ? w[j + e] : 0.0f;
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
        if (lane == 31) s_warp[warp] = sum;
        __syncthreads();  // also: the tile's weights are read before any of them is overwritten
        uint64_t before = run + sum - mine, total = 0;
        for (int i = 0; i < kSelWarps; ++i) {
            if (i < warp) before += s_warp[i];
            total += s_warp[i];
        }
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
        __syncthreads();
    }
    for (int i = m + tid; i < n; i += kSelThreads) dst[i] = 0.0f;
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 8;

// kVecs: 16-byte vectors of a token's row that this CTA's slice holds (16, 8 or 4). kOrdered: in place, a
// tile is read by all before any of it is written.
template <int kVecs, bool kOrdered>
__global__ void __launch_bounds__(kCopyThreads) kda_evict_copy_kernel(const CacheEvictArgs a, int rows_per_cta) {
    constexpr int kSlices = 16 / kVecs;
    constexpr int kStep = kCopyThreads / kVecs;  // tokens of one pass over the threads
    constexpr int kTile = kStep * kCopyUnroll;
    const PagedCache &c = a.c;
    const int bh = blockIdx.x, b = bh / c.num_kv_heads, h = bh - b * c.num_kv_heads;
    const int slice = blockIdx.y % kSlices;
    const bool values = blockIdx.y >= kSlices;
    const int m = min(row_length(c, b, a.status, false), a.budget);  // (the same from the new lengths)
    const int64_t begin = (int64_t)blockIdx.z * rows_per_cta;
    const int end = (int)min((int64_t)m, begin + rows_per_cta);
    pdl_wait();  // the selection is complete
    if (blockIdx.y == 0 && blockIdx.z == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = m;
    __nv_bfloat16 *const cache = values ? c.v : c.k;
    const int64_t stride = values ? c.v_page_stride : c.k_page_stride;
    const int32_t *const kept = a.kept + (size_t)bh * a.budget;
    const int32_t *const from = c.block_table + (size_t)b * c.max_pages, *const to = a.dst_table + (size_t)b * c.max_pages;
    const int first = threadIdx.x / kVecs, mask = c.page_size - 1;
    const size_t base = (size_t)h * c.page_size * kHeadDim + (slice * kVecs + threadIdx.x % kVecs) * 8;
    // A token's move: its source and destination in the cache (equal: nothing to do). The moves of the next
    // tile are looked up while this one's rows are on their way.
    auto look_up = [&](int i, int64_t &src, int64_t &dst) {
        src = dst = 0;
        if (i >= end) return;
        const int j = kept[i], ps = from[j >> c.page_shift], pd = to[i >> c.page_shift];
        if (ps < 0 || ps >= c.num_pages || pd < 0 || pd >= c.num_pages) {
            report_error(a.status, KDA_ERR_DEVICE_INPUT, b);
            return;
        }
        src = (int64_t)ps * stride + (int64_t)(j & mask) * kHeadDim;
        dst = (int64_t)pd * stride + (int64_t)(i & mask) * kHeadDim;
    };
    int64_t src[kCopyUnroll], dst[kCopyUnroll];
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u) look_up((int)begin + u * kStep + first, src[u], dst[u]);
    for (int i0 = (int)begin; i0 < end; i0 += kTile) {
        uint4 x[kCopyUnroll];
        int64_t at[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            at[u] = src[u] == dst[u] ? -1 : dst[u];
            if (at[u] >= 0) x[u] = *reinterpret_cast<const uint4 *>(cache + base + src[u]);
        }
        if (i0 + kTile < end)
#pragma unroll
            for (int u = 0; u < kCopyUnroll; ++u) look_up(i0 + kTile + u * kStep + first, src[u], dst[u]);
        if (kOrdered) __syncthreads();  // the tile is read before any of it is overwritten
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (at[u] >= 0) *reinterpret_cast<uint4 *>(cache + base + at[u]) = x[u];
    }
}

template <int kVecs, bool kOrdered>
cudaError_t launch_copy(const CacheEvictArgs &a, int rows_per_cta, unsigned parts, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.c.batch * a.c.num_kv_heads), 2 * (16 / kVecs), parts);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_evict_copy_kernel<kVecs, kOrdered>, a, rows_per_cta);
}

}  // namespace

cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream) {
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    kda_evict_select_kernel<<<(unsigned)(a.c.batch * a.c.num_kv_heads), kSelThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int most = std::min(a.budget, a.c.capacity);  // tokens a row can keep
    const int64_t ctas = (int64_t)a.c.batch * a.c.num_kv_heads * 2;
    if (a.dst_table != a.c.block_table) {
        // one tile a CTA, or up to four where that still leaves several CTAs for every SM
        const int tile = 16 * kCopyUnroll;
        const int64_t tiles = (most + tile - 1) / tile;
        const int64_t per = std::max<int64_t>((tiles + 65534) / 65535, std::min<int64_t>(4, ctas * tiles / (8 * sms)));
        const int rows = (int)(std::max<int64_t>(per, 1) * tile);
        return launch_copy<16, false>(a, rows, (unsigned)(((int64_t)most + rows - 1) / rows), stream);
    }
    if (ctas >= 4 * sms) return launch_copy<16, true>(a, most, 1, stream);
    if (ctas >= 2 * sms) return launch_copy<8, true>(a, most, 1, stream);
    return launch_copy<4, true>(a, most, 1, stream);
}

}  // namespace kda
