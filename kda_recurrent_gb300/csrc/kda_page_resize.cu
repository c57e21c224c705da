// Pages of a key-value cache handed out on the GPU as rows grow and shrink, and the slots of the new tokens
// (sm_103a).
//
// A row of n tokens holds ceil(n / page_size) pages. Free pages lie in a ring [first, first + count); rows that
// grow take from its front, in row order, rows that shrink give back to its end, so that what a call takes and
// what it gives never meet. The pages that a row shares with others, the first ones of its table, it does not
// give back. Where each row's pages and tokens begin follows from prefix sums over the rows, which every CTA
// forms by itself, 1024 rows at a time (8 bytes a row); tokens and pages find their row in the sums by
// bisection. Nothing here is wide: it is a chain of dependent reads (lengths, sums, table or ring, map), and the
// launch is most of a small call.
//
// Few new tokens and small tables are one CTA's. Otherwise one launch of CTAs all over the GPU does everything: a cluster
// gives pages back and sets the lengths and the state, the others map tokens, four a thread, and take the pages. Where the
// lengths or the state are written over those before the call, which all CTAs read, that is not possible: then one
// cluster does everything, or, with many tokens, a second launch of one cluster what the first kind does here. In us, calls back to back:
//     outputs apart, one CTA and the whole GPU: 64 tokens 2.5 and 3.3, 1024 3.5 and 2.9, 2048 4.1 and 3.0, 4096 5.1 and 3.1;
//     with 65536 entries of tables, 64 rows, 8.2 and 4.8; 1000 rows of 64000 entries 6.9 and 7.5
//     in place, one CTA and a cluster: 1024 tokens 3.5 and 4.4, 2048 4.1 and 4.7, 4096 5.1 and 4.4; 16384 entries 4.0
//     and 6.8, 64000 (1000 rows) 7.0 and 9.3, 65536 (64 rows) 8.2 and 7.7, 131072 14.2 and 7.8
//     in place, a cluster and two launches: 8192 tokens 5.1 and 7.0, 16384 5.8 and 7.1, 32768 7.2 and 7.0
// 64 rows that grow by a token from a cold cache: 3.5 us; 1000 rows of a serving step's changes 9.0 (in place 16.3); 8
// prompts of 16384 tokens, 2.1 MB, 4.0 (in place 7.7).
//
// Pages given back are compacted (a missing page of the table is not given back) in table order: each thread
// counts four entries, and the CTAs of the cluster exchange their counts through distributed shared memory.
#include <algorithm>

#include "kda_dependent.cuh"
#include "kda_internal.cuh"
#include "kda_mma.cuh"

namespace kda {
namespace {

constexpr int kMaxThreads = 1024;  // rows at a time, too
constexpr int kMaxCluster = 8;
constexpr int kGive = 4;  // entries of a thread at a time
constexpr uint32_t kMost = 0x7fffffffu;
// (tokens, entries of all tables) of one CTA, where the outputs are apart from the inputs and where not; of one cluster
constexpr int kOneTokens = 512, kOnePages = 32768, kOneTokensInPlace = 2048, kOnePagesInPlace = 65536, kFewTokens = 16384;

// Sums of counts that stop at 2^31 - 1 (adding so is associative, too).
__device__ __forceinline__ uint32_t add(uint32_t x, uint32_t y) { return min(x + y, kMost); }

// All threads of the cluster; what they wrote before is visible to all of them behind it.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(const void *local, uint32_t rank, uint32_t x) {
    uint32_t addr;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(x) : "memory");
}

// The first of n inclusive sums above x (there is one).
__device__ __forceinline__ int row_of(const uint32_t *sums, int n, uint32_t x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// kMaps: pages taken, slots, positions and rows of the new tokens. kState: pages given back, lengths and state.
// kQuad: tokens of a thread at a time (1, or 4 that are written together). With both and kWide the first cluster has the
// state and the CTAs behind it the maps; otherwise all CTAs do all.
template <bool kMaps, bool kState, int kQuad, bool kWide>
__global__ void __launch_bounds__(kMaxThreads, 1) kda_page_resize_kernel(const PageResizeArgs p) {
    __shared__ uint32_t s_tok[kMaxThreads], s_take[kMaxThreads], s_give[kMaxThreads];  // inclusive sums of a chunk's rows
    __shared__ int32_t s_old[kMaxThreads], s_new[kMaxThreads];
    __shared__ uint32_t s_keep[kMaxThreads];  // pages from the table's beginning on that the row does not give back
    __shared__ uint32_t s_warp[3][32];
    __shared__ uint32_t s_given[2][kMaxCluster];
    __shared__ uint32_t s_used;  // pages really taken
    const int threads = blockDim.x, warps = threads >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)blockIdx.x;
    const bool state = kState && (!kWide || rank < kMaxCluster), maps = kMaps && (!kWide || rank >= kMaxCluster);
    const int ctas = !kWide ? (int)gridDim.x : state ? kMaxCluster : (int)gridDim.x - kMaxCluster;  // (the state's are one cluster)
    const int me = (kWide && maps ? rank - kMaxCluster : rank) * threads + threadIdx.x, all = ctas * threads;
    const int F = p.num_pages, ps = p.page_size;
    if (threadIdx.x == 0) s_used = 0;  // (first read behind the chunk's barriers)
    wait_for_prior();
    allow_next();
    int first = p.free_state[0], count = p.free_state[1];
    if (first < 0 || first >= F || count < 0 || count > F) {
        if (maps && me == 0) report_error(p.status, KDA_ERR_DEVICE_INPUT, -1);
        first = 0, count = 0;
    }
    auto pages = [&](int n) { return (uint32_t)((n + ps - 1) >> p.page_shift); };
    auto valid = [&](int page, int row) {  // a page of the table or the ring; -1 for one that does not exist
        if (page >= F) report_error(p.status, KDA_ERR_DEVICE_INPUT, row);
        return page >= 0 && page < F ? page : -1;
    };
    auto free_page = [&](uint32_t i, int row) {
        uint32_t at = (uint32_t)first + i;  // (both below F)
        if (at >= (uint32_t)F) at -= F;
        const int page = p.free_pages[at];
        if (page < 0) report_error(p.status, KDA_ERR_DEVICE_INPUT, row);
        return valid(page, row);
    };
    if (maps && me == 0 && p.cu_tokens) p.cu_tokens[0] = 0;
    if (state && ctas > 1) cluster_barrier();  // every CTA has begun: its shared memory may be written

    uint32_t tokens = 0, taken = 0, given = 0;  // of the rows before the chunk
    int round = 0;
    uint32_t quad = me;  // this thread's next tokens
    for (int r0 = 0; r0 < p.batch; r0 += threads) {
        const int rows = min(threads, p.batch - r0), r = r0 + threadIdx.x;
        int n = 0, m = 0;
        if ((int)threadIdx.x < rows) {
            n = p.seq_lens[r], m = p.new_lens[r];
            if (n < 0 || n > p.capacity || m < 0 || m > p.capacity) {
                if (kMaps && rank == 0) report_error(p.status, KDA_ERR_DEVICE_INPUT, r);
                n = min(max(n, 0), p.capacity), m = min(max(m, 0), p.capacity);
            }
        }
        const uint32_t held = pages(n), want = pages(m);
        uint32_t keep = want;
        if (p.shared_pages && (int)threadIdx.x < rows) {
            int shared = p.shared_pages[r];
            if (shared < 0 || shared > p.max_pages) {
                if (kMaps && rank == 0) report_error(p.status, KDA_ERR_DEVICE_INPUT, r);
                shared = min(max(shared, 0), p.max_pages);
            }
            keep = max(want, (uint32_t)shared);
        }
        uint32_t x[3] = {m > n ? (uint32_t)(m - n) : 0u, want > held ? want - held : 0u, held > keep ? held - keep : 0u};
        const uint32_t my_tokens = x[0], my_take = x[1];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x[i], o);
                if (lane >= o) x[i] = add(x[i], y);
            }
            if (lane == 31) s_warp[i][warp] = x[i];
        }
        __syncthreads();
        uint32_t total[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {  // (the warps' sums, by every warp)
            uint32_t y = lane < warps ? s_warp[i][lane] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t z = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) y = add(y, z);
            }
            total[i] = __shfl_sync(0xffffffffu, y, 31);
            const uint32_t before = __shfl_sync(0xffffffffu, y, max(warp - 1, 0));
            if (warp > 0) x[i] = add(x[i], before);
        }
        s_tok[threadIdx.x] = x[0], s_take[threadIdx.x] = x[1], s_give[threadIdx.x] = x[2];
        s_old[threadIdx.x] = n, s_new[threadIdx.x] = m, s_keep[threadIdx.x] = keep;
        // in order: the first row whose pages are not there, and all later ones that need pages, get none
        const bool served = my_take == 0 || add(taken, x[1]) <= (uint32_t)count;
        const uint32_t left = (uint32_t)count - min(taken, (uint32_t)count);
        if (kMaps && !served && rank == 0) report_error(p.status, KDA_ERR_DEVICE_INPUT, r);
        if (kMaps && rank == 0 && (int)threadIdx.x < rows && p.cu_tokens) p.cu_tokens[r + 1] = (int)add(tokens, x[0]);
        if (kMaps && rank == 0 && my_tokens > 0 && p.has_maps && add(tokens, x[0]) > (uint32_t)p.max_tokens)
            report_error(p.status, KDA_ERR_DEVICE_INPUT, r);
        __syncthreads();

        // ---- pages taken
        const uint32_t takes = min(total[1], left);
        for (uint32_t i = me; maps && i < takes; i += all) {
            const int row = row_of(s_take, rows, i);
            if (s_take[row] > left) continue;  // the row that does not fit
            const uint32_t have = pages(s_old[row]), before = row > 0 ? s_take[row - 1] : 0;
            p.block_table[(size_t)(r0 + row) * p.max_pages + have + (i - before)] = free_page(taken + i, r0 + row);
        }
        // ---- slots of the new tokens
        if (maps && p.has_maps) {
            const uint32_t end = min(add(tokens, total[0]), (uint32_t)p.max_tokens);  // (of this chunk's rows)
            for (; quad * kQuad < end; quad += all) {
                const uint32_t t0 = max(quad * kQuad, tokens), t1 = min((quad + 1) * kQuad, end);
                int64_t slot[kQuad];
                int position[kQuad], of_row[kQuad];
                int row = t0 < t1 ? row_of(s_tok, rows, t0 - tokens) : 0, page = -1;
                uint32_t page_at = ~0u;
#pragma unroll
                for (int e = 0; e < kQuad; ++e) {
                    const uint32_t t = quad * kQuad + e;
                    if (t < t0 || t >= t1) continue;
                    while (s_tok[row] <= t - tokens) ++row, page_at = ~0u;
                    const int j = s_old[row] + (int)(t - tokens - (row > 0 ? s_tok[row - 1] : 0));
                    const uint32_t pg = (uint32_t)j >> p.page_shift;
                    if (p.slots && pg != page_at) {
                        const uint32_t have = pages(s_old[row]), take0 = row > 0 ? s_take[row - 1] : 0;
                        page = -1;
                        if (pages(s_new[row]) <= have || s_take[row] <= left)
                            page = pg < have ? valid(p.block_table[(size_t)(r0 + row) * p.max_pages + pg], r0 + row)
                                             : free_page(taken + take0 + (pg - have), r0 + row);
                        page_at = pg;
                    }
                    slot[e] = page < 0 ? -1 : ((int64_t)page << p.page_shift) + (j & (ps - 1));
                    position[e] = j;
                    of_row[e] = r0 + row;
                }
                const uint32_t t = quad * kQuad;
                if (kQuad == 4 && p.wide_maps && t1 - t0 == kQuad) {
                    if (p.slots) {
                        *reinterpret_cast<longlong2 *>(p.slots + t) = make_longlong2(slot[0], slot[1 % kQuad]);
                        *reinterpret_cast<longlong2 *>(p.slots + t + 2) = make_longlong2(slot[2 % kQuad], slot[3 % kQuad]);
                    }
                    if (p.positions) *reinterpret_cast<int4 *>(p.positions + t) = make_int4(position[0], position[1 % kQuad], position[2 % kQuad], position[3 % kQuad]);
                    if (p.rows) *reinterpret_cast<int4 *>(p.rows + t) = make_int4(of_row[0], of_row[1 % kQuad], of_row[2 % kQuad], of_row[3 % kQuad]);
                } else {
#pragma unroll
                    for (int e = 0; e < kQuad; ++e) {
                        if (t + e < t0 || t + e >= t1) continue;
                        if (p.slots) p.slots[t + e] = slot[e];
                        if (p.positions) p.positions[t + e] = position[e];
                        if (p.rows) p.rows[t + e] = of_row[e];
                    }
                }
                if ((quad + 1) * kQuad > end) break;  // (the rest is of later rows)
            }
        }
        // ---- pages given back, behind the ring's end
        for (uint32_t base = 0; state && base < total[2]; base += (uint32_t)all * kGive, ++round) {
            int page[kGive], mine = 0, row[kGive];
            const uint32_t i0 = base + (uint32_t)me * kGive;
            int at_row = i0 < total[2] ? row_of(s_give, rows, i0) : 0;
#pragma unroll
            for (int e = 0; e < kGive; ++e) {  // (all loads before any check, whose report would keep them in order)
                const uint32_t i = i0 + e;
                page[e] = -1, row[e] = 0;
                if (i < total[2]) {
                    while (s_give[at_row] <= i) ++at_row;
                    row[e] = at_row;
                    const uint32_t before = at_row > 0 ? s_give[at_row - 1] : 0;
                    page[e] = p.block_table[(size_t)(r0 + at_row) * p.max_pages + s_keep[at_row] + (i - before)];
                }
            }
#pragma unroll
            for (int e = 0; e < kGive; ++e) page[e] = valid(page[e], r0 + row[e]), mine += page[e] >= 0;
            uint32_t sum = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            __syncthreads();  // (s_warp has been read)
            if (lane == 31) s_warp[0][warp] = sum;
            __syncthreads();
            uint32_t block = lane < warps ? s_warp[0][lane] : 0, at = given + sum - mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, block, o);
                if (lane >= o) block += y;
            }
            const uint32_t below = __shfl_sync(0xffffffffu, block, max(warp - 1, 0));
            if (warp > 0) at += below;
            block = __shfl_sync(0xffffffffu, block, 31);
            if (ctas > 1) {
                if ((int)threadIdx.x < ctas) store_remote(&s_given[round & 1][rank], threadIdx.x, block);
                cluster_barrier();
                block = 0;
                for (int c = 0; c < ctas; ++c) {
                    if (c < rank) at += s_given[round & 1][c];
                    block += s_given[round & 1][c];
                }
            }
#pragma unroll
            for (int e = 0; e < kGive; ++e) {
                if (page[e] < 0) continue;
                if (at < (uint32_t)(F - count)) {
                    uint32_t to = (uint32_t)first + count + at;
                    while (to >= (uint32_t)F) to -= F;  // (at most twice)
                    p.free_pages[to] = page[e];
                } else {  // more pages than there are: one was given back twice
                    report_error(p.status, KDA_ERR_DEVICE_INPUT, r0 + row[e]);
                }
                ++at;
            }
            given = min(given + block, (uint32_t)(F - count));
        }
        // ---- the rows' new lengths, when no CTA reads the old ones any more
        const uint32_t end = add(taken, x[1]);
        const int best = served && my_take > 0 ? (int)end : 0;
        if (state && ctas > 1) cluster_barrier();
        if (state && rank == 0 && (int)threadIdx.x < rows) p.out_lens[r] = served ? m : n;
        // pages really taken: the sum at the last row that was served
        if (state) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, (uint32_t)best);
            if (lane == 0 && top > 0) atomicMax(&s_used, top);
        }
        tokens = add(tokens, total[0]);
        taken = add(taken, total[1]);
        __syncthreads();
    }
    if (maps && p.has_maps) {
        for (uint32_t i = tokens + me; i < (uint32_t)p.max_tokens; i += all) {
            if (p.slots) p.slots[i] = -1;
            if (p.positions) p.positions[i] = 0;
            if (p.rows) p.rows[i] = -1;
        }
    }
    if (!state) return;
    if (ctas > 1) cluster_barrier();  // the state has been read
    else __syncthreads();
    if (me == 0) {
        const uint32_t used = s_used;
        uint32_t at = (uint32_t)first + used;
        if (at >= (uint32_t)F) at -= F;
        p.out_state[0] = (int)at;
        p.out_state[1] = (int)((uint32_t)count - used + given);
    }
}

// Whether `out` and `in`, both of n numbers, have none in common.
bool apart(const int32_t *out, const int32_t *in, int64_t n) {
    const intptr_t x = reinterpret_cast<intptr_t>(out), y = reinterpret_cast<intptr_t>(in);
    return (x < y ? y - x : x - y) >= n * 4;
}

}  // namespace

cudaError_t launch_page_resize(const PageResizeArgs &p, cudaStream_t stream) {
    const bool others = apart(p.out_lens, p.seq_lens, p.batch) && apart(p.out_lens, p.new_lens, p.batch) &&
                        (!p.shared_pages || apart(p.out_lens, p.shared_pages, p.batch)) && apart(p.out_state, p.free_state, 2);
    if ((int64_t)p.batch * p.max_pages <= (others ? kOnePages : kOnePagesInPlace) && p.max_tokens <= (others ? kOneTokens : kOneTokensInPlace)) {
        const unsigned threads = p.batch <= 256 && p.max_tokens <= 1024 ? 256 : kMaxThreads;
        return launch_dependent(kda_page_resize_kernel<true, true, 1, false>, dim3(1), threads, 0, stream, p);
    }
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    const int threads = p.batch <= 256 ? 256 : kMaxThreads, quads = (p.max_tokens + 3) / 4;
    const int ctas = std::max(std::min((quads + threads - 1) / threads, sms * (kMaxThreads / threads)), 1);
    if (others) {
        const int grid = (kMaxCluster + ctas + kMaxCluster - 1) / kMaxCluster * kMaxCluster;
        return launch_clusters(kMaxCluster, kda_page_resize_kernel<true, true, 4, true>, dim3((unsigned)grid), (unsigned)threads, 0, stream, p);
    }
    if (p.max_tokens <= kFewTokens)
        return launch_clusters(kMaxCluster, kda_page_resize_kernel<true, true, 1, false>, dim3(kMaxCluster), kMaxThreads, 0, stream, p);
    const cudaError_t e = launch_dependent(kda_page_resize_kernel<true, false, 4, false>, dim3((unsigned)ctas), (unsigned)threads, 0, stream, p);
    if (e != cudaSuccess) return e;
    return launch_clusters(kMaxCluster, kda_page_resize_kernel<false, true, 1, false>, dim3(kMaxCluster), kMaxThreads, 0, stream, p);
}

}  // namespace kda
