// Linear attention with a decay for each head, prompt form (sm_103a, tcgen05 / TMEM / TMA).
//
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// Chunks of C = 128 tokens. With G the inclusive prefix sum of g over the chunk and S the state
// before it, the chunk is four products of 128 x 128 tiles:
//     A   = Q K^T                                  scores
//     P   = A . exp(G_i - G_j) for j <= i, else 0
//     O   = scale (Diag(exp G) (Q S) + P V)
//     S' = exp(G_last) S + D,   D = K^T (Diag(exp(G_last - G_j)) V)
// All inputs of the products are BF16 tiles in shared memory (P in tensor memory), accumulators
// FP32 in tensor memory. What is rounded to BF16 on the way to an output: P, and the copy of S that
// the queries read; each adds about the error of the output's own rounding. The state must carry
// more (it is an FP32 output, summed over thousands of tokens): its decayed values are split into two
// BF16 terms, hi + lo, 17 bits of mantissa, at the price of a second product (K is exact), and S itself
// stays FP32 in the registers of the state warps. D does not depend on S, so the only serial work
// from chunk to chunk is S' = exp(G_last) S + D and its rounding into the next chunk's operand.
//
// One CTA per chain (or window of a chain), 20 warps in five roles:
//   warp 0        a chunk's prefix and suffix sums of g, and its TMA loads: Q, K, V tiles (128-byte
//                 swizzle) into a ring of five 32 KiB tiles
//   warp 1        issues every MMA: A, Q S, D by quarters of 32 tokens (hi then lo), P V
//   warp 3        TMA stores of O
//   warps 4-11    A -> P in place in tensor memory, then O: both accumulators -> BF16 -> the tile that
//                 held V
//   warps 12-19   S in registers (row dk, 64 columns a thread): the update and the operand of Q S; V ->
//                 hi, lo by quarters into a ring of two
// The values are decayed, not the keys, because V is only read by the last product of the chunk, so that
// the split needs no scores. (Half of it on warps 4-11 put it on the chain from the scores to P V: 8%
// slower; two extra warps took 1.5k cycles a quarter; four extra warps left too few registers for the
// state. Half of D before Q S: 9% slower, since Q's tile, which the next V replaces, is then freed late.) O leaves through shared memory because a
// thread's row-wise 32-byte stores (32 rows an instruction) kept the load/store unit busy for 2k
// cycles a chunk, during which the MMAs' operand reads took four times their time (2.56 ms at
// 8 x 16384 x 96 heads).
// The suffix sums G_last - G_j are scanned from the end, not formed as differences, so that a
// strong decay early in a chunk costs the later tokens' weights no precision. A log decay below
// -128 counts as -128 (both decay to zero in FP32), which keeps the sums finite.
//
// Bound: 1 KiB of HBM traffic a token and head against 164 KFLOP of BF16 products.
//
// Few chains leave most SMs idle. A chain is then cut into windows: a first pass computes each
// window's end state from zero (the update half of the kernel) and its total decay, an
// elementwise pass chains the windows' start states, S_{w+1} = exp(g_w) S_w + D_w, and the chunk
// kernel runs every window from its start state. The same is done for the chains of a short last
// wave, whose windows are launched behind the whole chains.
//
// All waits are bounded; on expiry the CTA records KDA_ERR_DEVICE_TIMEOUT, waits for its own
// copies and MMAs in flight, frees its tensor memory and returns.
#include <cuda.h>

#include <algorithm>

#include "kda_internal.cuh"
#include "kda_mma.cuh"
#include "kda_tc.cuh"

namespace kda {
namespace {

constexpr int kC = 128;  // tokens of a chunk
constexpr int kTile = kC * kHeadDim * 2;
constexpr int kHalf = kTile / 2;  // a tile is two halves of 64 columns: 128 rows of 128 bytes
constexpr int kRing = 5;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinLogDecay = -128.0f;

constexpr int kWarpMma = 1, kWarpAlloc = 2, kWarpStore = 3, kWarpO = 4, kWarpS = 12;
constexpr int kOutWarps = 8, kStateWarps = 8;
constexpr int kStateThreads = kStateWarps * 32;
constexpr int kThreads = (kWarpS + kStateWarps) * 32;

struct Gates {
    float prefix[kC];  // log2 units: inclusive prefix sums, and sums over the later tokens
    float suffix[kC];  // (as factors, 2^suffix)
    float decay;       // of the whole chunk
    float pad[3];
};

struct Bars {
    uint64_t full[kRing], empty[kRing];  // TMA -> users, users (tcgen05.commit) -> TMA
    uint64_t scores;   // A done
    uint64_t p;        // P written (8 warps)
    uint64_t split[2], split_free[2];  // hi and lo of a quarter written (8 warps), and read
    uint64_t tail;     // rows past the window's last token cleared (8 warps)
    uint64_t d;        // D done
    uint64_t d_free;   // D read (8 warps)
    uint64_t s;        // S operand written (8 warps)
    uint64_t qs;       // Q S done: the S operand is free
    uint64_t o;        // P V done (and everything before it)
    uint64_t o_free;   // both output accumulators read (8 warps)
    uint64_t o_tile[2];  // O written to the chunk's V tile (8 warps)
    uint64_t stored[2];  // and read by the stores
    uint64_t gate[2], gate_free[2];
    uint64_t drain;
    uint32_t tmem;
    int32_t abort;
};

// ---- shared memory (bytes); the swizzled tiles need 1024-byte alignment
constexpr int kQuarter = 32;                          // tokens
constexpr int kSplitHalf = kQuarter * 128;            // 64 columns of a quarter
constexpr int kSplitLo = 2 * kSplitHalf, kSplitStage = 2 * kSplitLo;
constexpr int kSplit = kRing * kTile;
constexpr int kS = kSplit + 2 * kSplitStage;
constexpr int kGates = kS + kTile;
constexpr int kBars = kGates + 2 * (int)sizeof(Gates);
constexpr int kSmem = kBars + (int)sizeof(Bars);
static_assert(kSmem <= 227 * 1024, "one CTA per SM");

// ---- tensor memory (columns)
constexpr uint32_t kTmemCols = 512;
// (all 512 are allocated, so the base is column 0)
constexpr uint32_t kColA = 0;  // A (128); each 32 columns then hold their part of P in the first 16
constexpr uint32_t kColO = 128, kColQS = 256, kColD = 384;

constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;  // MN-major operands
constexpr uint32_t kIdescQK = instr_desc(1, 128, 128);
constexpr uint32_t kIdescQS = instr_desc(1, 128, 128) | kTransB;
constexpr uint32_t kIdescD = instr_desc(1, 128, 128) | kTransA | kTransB;
constexpr uint32_t kIdescPV = instr_desc(1, 128, 128) | kTransB;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Operand descriptors: the constant part plus the address in 16-byte units (under 2^14 for any
// address in shared memory, so an offset adds without carry).
//   K-major, 128-byte swizzle: smem_desc_sw128.
//   MN-major, 128-byte swizzle: 128-byte rows hold 64 elements along M or N, eight rows (along K)
//   make a 1024-byte group; `lbo` = distance between blocks of 64 along M or N.
__device__ __forceinline__ constexpr uint64_t desc_mn(uint32_t lbo) {
    return (uint64_t)(lbo >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint64_t kDescK = (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
constexpr uint64_t kDescMn = desc_mn(kHalf), kDescSplit = desc_mn(kSplitHalf);

__device__ __forceinline__ uint64_t at(uint64_t desc, uint32_t saddr) { return desc | (saddr >> 4); }

// Every lane of the warp calls these with the same operands (which keeps them in uniform
// registers); one elected lane issues, always the same one, so that its commits follow its MMAs.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

// Bounded wait of one thread that also gives up as soon as any thread of the CTA has.
__device__ __forceinline__ bool wait_one(uint64_t *bar, uint32_t parity, Bars *B, DeviceStatus *st) {
    const uint32_t addr = smem_addr(bar);
    uint64_t start = 0;
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(parity), "r"(kSuspendHintNs)
            : "memory");
        if (done) return true;
        if (*reinterpret_cast<volatile int32_t *>(&B->abort)) return false;
        const uint64_t now = global_ns();
        if (start == 0) {
            start = now;
        } else if (now - start > kWaitLimitNs) {
            *reinterpret_cast<volatile int32_t *>(&B->abort) = 1;
            report_error(st, KDA_ERR_DEVICE_TIMEOUT, (int)blockIdx.x);
            return false;
        }
    }
}

// The same for a whole warp, with one decision for all its lanes.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Bars *B, DeviceStatus *st) {
    return __all_sync(0xffffffffu, wait_one(bar, parity, B, st));
}

// One arrival for a warp, after what its lanes did.
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct Plan {
    int32_t wins;        // windows of each windowed chain (1: none)
    int32_t seq_chains;  // chains before the windowed ones
};

struct ChunkArgs {
    LinearPrefillArgs p;
    Plan plan;
    float *slots;  // windowed chain lc, window w: the window's own end state, then the start of window w + 1
    float *decay;  // windowed chain lc, window w: its total decay (log2)
};

__device__ __forceinline__ float *slot_of(const ChunkArgs &a, int lc, int w) {
    return a.slots + ((size_t)lc * (a.plan.wins - 1) + w) * (kHeadDim * kHeadDim);
}

// Chains in order of their sequences' lengths, longest first (ties by index; more than kRanked
// sequences keep index order): CTAs start in index order, so the longest start first.
constexpr int kRanked = 256;

__device__ __forceinline__ int seq_of_rank(const LinearPrefillArgs &a, int j, int *scratch) {
    const int N = a.num_seqs;
    if (N <= 1 || N > kRanked) return j;
    int *len = scratch, *pick = scratch + kRanked;
    for (int i = threadIdx.x; i < N; i += blockDim.x)
        len[i] = (int)((unsigned)__ldg(a.cu_seqlens + i + 1) - (unsigned)__ldg(a.cu_seqlens + i));
    __syncthreads();
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
        const int li = len[i];
        int r = 0;
        for (int m = 0; m < N; ++m) r += (len[m] > li) | ((len[m] == li) & (m < i));
        if (r == j) *pick = i;
    }
    __syncthreads();
    const int n = *pick;
    __syncthreads();
    return n;
}

struct Span {
    int bos, eos;  // tokens of the window
    bool first, last, live;
};

// Window w (of at most W) of sequence n.
__device__ __forceinline__ Span span_of(const LinearPrefillArgs &a, int n, int w, int W, bool report) {
    int sb = a.cu_seqlens[n], se = a.cu_seqlens[n + 1];
    if (sb < 0 || se < sb || se > a.total_tokens) {
        if (report && threadIdx.x == 0) report_error(a.status, KDA_ERR_DEVICE_INPUT, n);
        sb = min(max(sb, 0), a.total_tokens);
        se = min(max(se, sb), a.total_tokens);
    }
    const int chunks = (se - sb + kC - 1) / kC;
    const int per = max(1, (chunks + W - 1) / W);
    const int wins = max(1, (chunks + per - 1) / per);
    Span s;
    s.live = w < wins;
    s.first = w == 0;
    s.last = w >= wins - 1;
    s.bos = s.live ? sb + kC * per * w : se;
    s.eos = s.last ? se : s.bos + kC * per;
    return s;
}

// hi and lo of 32 tokens of V by the state warps: a row of the quarter at `tile` (eight threads a row, a
// thread the same 16 bytes of both halves) times its factor f, rows past the last token as zeros, into
// the split stage at `to`.
__device__ __forceinline__ void split_quarter(const uint8_t *tile, uint8_t *to, float f, bool live) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint4 in = *reinterpret_cast<const uint4 *>(tile + i * kHalf);
        if (!live) in = make_uint4(0, 0, 0, 0);
        const uint32_t u[4] = {in.x, in.y, in.z, in.w};
        uint32_t hi[4], rest[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float y0 = __uint_as_float(u[e] << 16) * f, y1 = __uint_as_float(u[e] & 0xffff0000u) * f;
            hi[e] = pack_bf16(y0, y1);
            rest[e] = pack_bf16(y0 - __uint_as_float(hi[e] << 16), y1 - __uint_as_float(hi[e] & 0xffff0000u));
        }
        *reinterpret_cast<uint4 *>(to + i * kSplitHalf) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(to + kSplitLo + i * kSplitHalf) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
    }
}

// Parity of the release of tile i on its slot: V tiles of the full kernel are released through `stored`,
// so the slot's `empty` barrier has one phase for each of its other tiles up to i.
__device__ __forceinline__ uint32_t empty_parity(int i, bool with_v) {
    const int uses = i / kRing;  // earlier tiles on the slot: i % kRing + kRing u for u < uses
    if (with_v) return uses & 1;
    // tile j is a V tile when j % 3 == 2; over three uses of a slot (15 tiles) exactly one is
    const int first = i % kRing;
    int vs = uses / 3;
    for (int u = uses / 3 * 3; u < uses; ++u) vs += (first + kRing * u) % 3 == 2;
    return (uses - vs) & 1;
}

// kStates: only the state update, from zero, over the windows of the windowed chains but the last.
template <bool kStates>
__global__ void __launch_bounds__(kThreads, 1)
    kda_linear_chunk_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                            const __grid_constant__ CUtensorMap map_o) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const LinearPrefillArgs &p = a.p;
    Bars *B = reinterpret_cast<Bars *>(smem + kBars);
    // the shuffle tells the compiler that the role is one for the warp
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, H = p.num_heads;
    const int W = a.plan.wins;
    // the item: a whole chain, or window w of windowed chain lc
    int pos = blockIdx.x, w = 0, lc = -1;
    if (kStates || pos >= a.plan.seq_chains) {
        const int per = kStates ? W - 1 : W;
        const int i = kStates ? pos : pos - a.plan.seq_chains;
        lc = i / per;
        w = i - lc * per;
        pos = a.plan.seq_chains + lc;
    }
    const int h = pos % H;
    const int n = seq_of_rank(p, pos / H, reinterpret_cast<int *>(smem));
    const Span sp = span_of(p, n, w, lc >= 0 ? W : 1, h == 0 && w == 0 && !kStates);
    if (kStates) pdl_launch_dependents();
    if (!sp.live || (kStates && sp.last)) {
        if (!kStates) pdl_wait();  // every CTA ends after the launches before: see the last lines
        return;
    }
    const int nchunks = (sp.eos - sp.bos + kC - 1) / kC;
    const size_t chain = ((size_t)n * H + h) * (kHeadDim * kHeadDim);
    const float *const start = kStates ? nullptr : lc >= 0 && !sp.first ? slot_of(a, lc, w - 1)
                                               : p.init_state ? p.init_state + chain : nullptr;
    float *const end = kStates ? slot_of(a, lc, w) : sp.last && p.final_state ? p.final_state + chain : nullptr;
    // the last chunk's update is needed only where somebody reads the end state
    const int updates = end ? nchunks : nchunks - 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&B->full[i], 1), mbar_init(&B->empty[i], 1);
        mbar_init(&B->scores, 1);
        mbar_init(&B->p, kOutWarps);
        for (int i = 0; i < 2; ++i) mbar_init(&B->split[i], kStateWarps), mbar_init(&B->split_free[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&B->o_tile[i], kOutWarps), mbar_init(&B->stored[i], 1);
        mbar_init(&B->tail, kStateWarps);
        mbar_init(&B->d, 1);
        mbar_init(&B->d_free, kStateWarps);
        mbar_init(&B->s, kStateWarps);
        mbar_init(&B->qs, 1);
        mbar_init(&B->o, 1);
        mbar_init(&B->o_free, kOutWarps);
        for (int i = 0; i < 2; ++i) mbar_init(&B->gate[i], 1), mbar_init(&B->gate_free[i], kStateWarps + (kStates ? 0 : kOutWarps));
        mbar_init(&B->drain, 1);
        // the swizzled tiles are laid out for a 1024-byte-aligned base
        B->abort = (smem_addr(smem) & 1023u) != 0;
        if (B->abort) report_error(p.status, KDA_ERR_CUDA, 0);
        fence_mbar_init();
    }
    if (warp == kWarpAlloc) {
        tmem_alloc(&B->tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    fence_async_smem();  // the ranking's scratch lies where the first tiles go
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;
    if (threadIdx.x == 0 && B->tmem != 0) {
        report_error(p.status, KDA_ERR_CUDA, 1);
        B->abort = 1;
    }
    __syncthreads();
    const uint32_t base = smem_addr(smem);
    constexpr int kPer = kStates ? 2 : 3;  // tiles of a chunk: (Q,) K, V
    const int last_rows = sp.eos - sp.bos - (nchunks - 1) * kC;  // of the last chunk
    int issued = 0;                        // loads issued (warp 0)

    if (B->abort) {
        // nothing has started
    } else if (warp == 0) {
        float run = 0.0f;  // total decay of the window so far
        for (int c = 0; c < nchunks; ++c) {
            const int t0 = sp.bos + c * kC, L = min(kC, sp.eos - t0), b = c & 1;
            float g[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = 4 * lane + e;
                g[e] = t < L ? p.log_decay[(size_t)(t0 + t) * p.decay_token_stride + h] : 0.0f;
            }
            bool ok = true;
            for (int which = 0; which < kPer; ++which, ++issued) {
                const int slot = issued % kRing;
                if (issued >= kRing) {  // the tile five loads ago has been read
                    const int before = issued - kRing, cb = before / kPer;
                    const bool is_v = !kStates && before - cb * kPer == kPer - 1;  // then also as O
                    ok = is_v ? wait_warp(&B->stored[cb & 1], (cb >> 1) & 1, B, p.status)
                              : wait_warp(&B->empty[slot], empty_parity(before, kStates), B, p.status);
                    if (!ok) break;
                }
                const CUtensorMap *map = which == kPer - 1 ? &map_v : which == kPer - 2 ? &map_k : &map_q;
                if (lane == 0) {
                    expect_tx(&B->full[slot], kTile);
                    tma_load(base + slot * kTile, map, 0, h, t0, &B->full[slot]);
                    tma_load(base + slot * kTile + kHalf, map, 64, h, t0, &B->full[slot]);
                }
                __syncwarp();
            }
            if (!ok) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) g[e] = (g[e] < kMinLogDecay ? kMinLogDecay : g[e]) * kLog2e;
            const float mine = (g[0] + g[1]) + (g[2] + g[3]);
            float up = mine, down = mine;  // inclusive over the lanes before, and after
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, up, o), y = __shfl_down_sync(0xffffffffu, down, o);
                if (lane >= o) up += x;
                if (lane + o < 32) down += y;
            }
            float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 0) before = 0.0f;
            if (lane == 31) after = 0.0f;
            const float total = __shfl_sync(0xffffffffu, down, 0);
            if (c >= 2 && !wait_warp(&B->gate_free[b], ((c >> 1) - 1) & 1, B, p.status)) break;
            Gates *G = reinterpret_cast<Gates *>(smem + kGates) + b;
            const float p0 = before + g[0], p1 = p0 + g[1], p2 = p1 + g[2], p3 = p2 + g[3];
            *reinterpret_cast<float4 *>(&G->prefix[4 * lane]) = make_float4(p0, p1, p2, p3);
            const float s2 = after + g[3], s1 = s2 + g[2], s0 = s1 + g[1];
            *reinterpret_cast<float4 *>(&G->suffix[4 * lane]) = make_float4(ex2(s0), ex2(s1), ex2(s2), ex2(after));
            // exp2f, not the 2^-22 of the hardware's: this error repeats every chunk and adds up over
            // the chunks that a slowly decaying state remembers
            if (lane == 0) G->decay = exp2f(total);
            arrive_warp(&B->gate[b]);
            run += total;
        }
        if (kStates && lane == 0) a.decay[(size_t)lc * W + w] = run;
    } else if (warp == kWarpMma) {
        for (int c = 0; c < nchunks; ++c) {
            const int iq = c * kPer, ik = iq + kPer - 2, iv = ik + 1;
            const uint32_t k = base + (ik % kRing) * kTile, q = base + (iq % kRing) * kTile, v = base + (iv % kRing) * kTile;
            const int L = c + 1 < nchunks ? kC : last_rows;
            if (!wait_warp(&B->full[ik % kRing], (ik / kRing) & 1, B, p.status)) break;
            if (!kStates) {
                if (!wait_warp(&B->full[iq % kRing], (iq / kRing) & 1, B, p.status)) break;
                if (c > 0 && !wait_warp(&B->o, (c - 1) & 1, B, p.status)) break;  // P of the last chunk has been read
                const uint64_t dq = at(kDescK, q), dk = at(kDescK, k);
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint32_t off = ((s >> 2) * kHalf + (s & 3) * 32) >> 4;
                    mma_ss(tmem + kColA, dq + off, dk + off, kIdescQK, s > 0);
                }
                commit(&B->scores);
                if (!wait_warp(&B->s, c & 1, B, p.status)) break;
                if (c > 0 && !wait_warp(&B->o_free, (c - 1) & 1, B, p.status)) break;
                tc_fence_after();
                const uint64_t ds = at(kDescMn, base + kS);
#pragma unroll
                for (int s = 0; s < 8; ++s)
                    mma_ss(tmem + kColQS, dq + (((s >> 2) * kHalf + (s & 3) * 32) >> 4), ds + s * 128, kIdescQS, s > 0);
                commit(&B->qs);
                commit(&B->empty[iq % kRing]);
            }
            if (L < kC && !wait_warp(&B->tail, 0, B, p.status)) break;
            if (c < updates) {
                if (c > 0 && !wait_warp(&B->d_free, (c - 1) & 1, B, p.status)) break;
                bool lost = false;
#pragma unroll 1
                for (int q = 0; q * kQuarter < L; ++q) {
                    const int use = 4 * c + q, st = use & 1;
                    lost = !wait_warp(&B->split[st], (use >> 1) & 1, B, p.status);
                    if (lost) break;
                    tc_fence_after();
                    const uint64_t da = at(kDescMn, k + q * kQuarter * 128), db = at(kDescSplit, base + kSplit + st * kSplitStage);
#pragma unroll
                    for (int s = 0; s < 4; ++s)  // hi, hi, lo, lo
                        mma_ss(tmem + kColD, da + (s & 1) * 128, db + (((s >> 1) * kSplitLo + (s & 1) * 2048) >> 4), kIdescD,
                               q > 0 || s > 0);
                    commit(&B->split_free[st]);
                }
                if (lost) break;
                commit(&B->d);
            }
            commit(&B->empty[ik % kRing]);
            if (!wait_warp(&B->full[iv % kRing], (iv / kRing) & 1, B, p.status)) break;
            if (!kStates) {
                if (!wait_warp(&B->p, c & 1, B, p.status)) break;
                tc_fence_after();
                const uint64_t dv = at(kDescMn, v);
                if (L == kC) {
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_ts(tmem + kColO, tmem + kColA + 32 * (s >> 1) + 8 * (s & 1), dv + s * 128, kIdescPV, s > 0);
                } else {
                    for (int s = 0; s * 16 < L; ++s)
                        mma_ts(tmem + kColO, tmem + kColA + 32 * (s >> 1) + 8 * (s & 1), dv + s * 128, kIdescPV, s > 0);
                }
                commit(&B->o);
            }
            if (kStates) commit(&B->empty[iv % kRing]);
        }
        commit(&B->drain);  // every earlier commit has reached its barrier when this one has
        mbar_wait(&B->drain, 0);
    } else if (warp == kWarpStore && !kStates) {
        // lane 4 h + q stores rows [32 q, 32 q + 32) of half h, unless they are not all tokens of the window
        // (then their warp has stored what is left)
        const int quad = lane & 3, half = lane >> 2;
        for (int c = 0; c < nchunks; ++c) {
            if (!wait_warp(&B->o_tile[c & 1], (c >> 1) & 1, B, p.status)) break;
            const int iv = c * kPer + kPer - 1;
            if (lane < 8 && (c + 1 < nchunks || 32 * quad + 32 <= last_rows)) {
                tma_store(&map_o, base + (iv % kRing) * kTile + half * kHalf + quad * 4096, 64 * half, h, sp.bos + c * kC + 32 * quad);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            arrive_warp(&B->stored[c & 1]);
        }
        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    } else if (warp < kWarpO || (kStates && warp < kWarpS)) {
        // idle
    } else if (warp < kWarpS) {
        const int quad = warp & 3, half = (warp - kWarpO) >> 2, row = 32 * quad + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        for (int c = 0; c < nchunks; ++c) {
            const Gates *G = reinterpret_cast<const Gates *>(smem + kGates) + (c & 1);
            if (!wait_warp(&B->gate[c & 1], (c >> 1) & 1, B, p.status)) break;
            const float gi = G->prefix[row], lam = p.scale * ex2(gi);
            if (!wait_warp(&B->scores, c & 1, B, p.status)) break;
            tc_fence_after();
            // this warp's blocks of 32 columns: every other one
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int b = 2 * i + half;
                float f[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = 0.0f;
                if (b <= quad) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float s[16], e[16];
                        tmem_ld16(lanes + kColA + 32 * b + 16 * u, s);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 gj = *reinterpret_cast<const float4 *>(&G->prefix[32 * b + 16 * u + j]);
                            e[j] = ex2(gi - gj.x), e[j + 1] = ex2(gi - gj.y), e[j + 2] = ex2(gi - gj.z), e[j + 3] = ex2(gi - gj.w);
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) s[j] = (b < quad || 16 * u + j <= lane) ? s[j] * e[j] : 0.0f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[8 * u + j] = __uint_as_float(pack_bf16(s[2 * j], s[2 * j + 1]));
                    }
                }
                tmem_st16(lanes + kColA + 32 * b, f);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive_warp(&B->p);
            if (lane == 0) mbar_arrive(&B->gate_free[c & 1]);
            if (!wait_warp(&B->o, c & 1, B, p.status)) break;
            tc_fence_after();
            // rows of 128 bytes into the V tile, which nobody reads any more, for warp 3 to store; a warp whose
            // rows are not all tokens of the window stores them itself
            const int iv = c * kPer + kPer - 1, t = sp.bos + c * kC + row;
            const bool whole = c + 1 < nchunks || 32 * quad + 32 <= last_rows;
            uint8_t *const rows = smem + (iv % kRing) * kTile + half * kHalf + quad * 4096;
            uint4 *const dst = reinterpret_cast<uint4 *>(p.out + ((size_t)t * H + h) * kHeadDim + 64 * half);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float o[16], x[16];
                tmem_ld16(lanes + kColO + 64 * half + 16 * b, o);
                tmem_ld16(lanes + kColQS + 64 * half + 16 * b, x);
                tmem_wait_ld();
                uint32_t pk[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    pk[j] = pack_bf16(fmaf(lam, x[2 * j], p.scale * o[2 * j]), fmaf(lam, x[2 * j + 1], p.scale * o[2 * j + 1]));
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 y = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                    if (whole)
                        *reinterpret_cast<uint4 *>(rows + lane * 128 + (((2 * b + i) ^ (lane & 7)) << 4)) = y;
                    else if (t < sp.eos)
                        dst[2 * b + i] = y;
                }
            }
            tc_fence_before();
            fence_async_smem();
            arrive_warp(&B->o_free);
            if (lane == 0) mbar_arrive(&B->o_tile[c & 1]);
        }
    } else {
        const int quad = warp & 3, half = (warp - kWarpS) >> 2, row = 32 * quad + lane;  // row: dk
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + kColD + 64 * half;
        uint8_t *const s_row = smem + kS + half * kHalf + row * 128;
        float S[64];
        if (!kStates && lc >= 0 && !sp.first) pdl_wait();  // the slots are written by the launch before
        if (start) {
            const float4 *src = reinterpret_cast<const float4 *>(start + (size_t)row * kHeadDim + 64 * half);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float4 x = src[i];
                S[4 * i] = x.x, S[4 * i + 1] = x.y, S[4 * i + 2] = x.z, S[4 * i + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) S[i] = 0.0f;
        }
        auto publish = [&] {  // S as the BF16 operand of Q S
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4 *>(s_row + ((i ^ (row & 7)) << 4)) =
                    make_uint4(pack_bf16(S[8 * i], S[8 * i + 1]), pack_bf16(S[8 * i + 2], S[8 * i + 3]),
                               pack_bf16(S[8 * i + 4], S[8 * i + 5]), pack_bf16(S[8 * i + 6], S[8 * i + 7]));
            fence_async_smem();
            arrive_warp(&B->s);
        };
        const int tid = threadIdx.x - kWarpS * 32;
        // Splits chunk c's V, once its gate sums and V are there. In a chunk that is not full, first clears the
        // rows past the last token: they hold another sequence's keys and values, which a zero in the
        // other operand does not silence if they are not finite. The quarters of all chunks count through
        // the ring of two stages (only the last chunk may have fewer than four).
        auto split = [&](int c) {
            const int ik = c * kPer + kPer - 2, iv = ik + 1;
            if (!wait_warp(&B->gate[c & 1], (c >> 1) & 1, B, p.status)) return false;
            if (!wait_warp(&B->full[iv % kRing], (iv / kRing) & 1, B, p.status)) return false;
            if (c + 1 == nchunks && last_rows < kC) {
                if (!wait_warp(&B->full[ik % kRing], (ik / kRing) & 1, B, p.status)) return false;
                uint8_t *const keys = smem + (ik % kRing) * kTile, *const values = smem + (iv % kRing) * kTile;
                for (int x = tid; x < 2048; x += kStateThreads)
                    if (((x & 1023) >> 3) >= last_rows)
                        *reinterpret_cast<uint4 *>(values + x * 16) = *reinterpret_cast<uint4 *>(keys + x * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                arrive_warp(&B->tail);
            }
            if (c >= updates) return true;
            const int L = c + 1 < nchunks ? kC : last_rows;
            const Gates *G = reinterpret_cast<const Gates *>(smem + kGates) + (c & 1);
            const uint8_t *const tile = smem + (iv % kRing) * kTile + tid * 16;
#pragma unroll 1
            for (int q = 0; q * kQuarter < L; ++q) {
                const int use = 4 * c + q, st = use & 1, t = q * kQuarter + (tid >> 3);
                if (use >= 2 && !wait_warp(&B->split_free[st], ((use >> 1) - 1) & 1, B, p.status)) return false;
                split_quarter(tile + q * kQuarter * 128, smem + kSplit + st * kSplitStage + tid * 16, G->suffix[t], t < L);
                fence_async_smem();
                arrive_warp(&B->split[st]);
            }
            return true;
        };
        bool ok = true;
        for (int c = 0; c < nchunks; ++c) {
            if (!kStates) {  // S for the queries
                ok = c == 0 || wait_warp(&B->qs, (c - 1) & 1, B, p.status);
                if (!ok) break;
                publish();
            }
            ok = split(c);
            if (!ok) break;
            const float decay = (reinterpret_cast<const Gates *>(smem + kGates) + (c & 1))->decay;
            arrive_warp(&B->gate_free[c & 1]);
            if (c < updates) {
                ok = wait_warp(&B->d, c & 1, B, p.status);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float d[16];
                    tmem_ld16(lanes + 16 * b, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) S[16 * b + j] = fmaf(S[16 * b + j], decay, d[j]);
                }
                tc_fence_before();
                arrive_warp(&B->d_free);  // (only with an update: an arrival for a chunk without one could complete
                                          // a second phase before the MMA warp has seen the first)
            }
        }
        pdl_wait();  // an initial state in the same place has been read by the launches before
        if (ok && end) {
            float4 *dst = reinterpret_cast<float4 *>(end + (size_t)row * kHeadDim + 64 * half);
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[i] = make_float4(S[4 * i], S[4 * i + 1], S[4 * i + 2], S[4 * i + 3]);
        }
    }
    __syncwarp();
    __syncthreads();
    if (B->abort) {  // wait (bounded) for what is still in flight before the memory is given back
        if (threadIdx.x == 0)
            for (int i = max(0, issued - kRing); i < issued; ++i) mbar_wait(&B->full[i % kRing], (i / kRing) & 1);
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kWarpAlloc) tmem_dealloc(B->tmem, kTmemCols);
    // whatever follows this grid on the stream also follows the launches that it may overlap
    pdl_wait();
}

// S_{w+1} = exp2(g_w) S_w + D_w over the windows of a windowed chain, in place in its slots; one
// float4 of the state a thread, the windows' own states loaded ahead.
constexpr int kScanThreads = 128;
constexpr int kScanCtas = kHeadDim * kHeadDim / (4 * kScanThreads);

__global__ void __launch_bounds__(kScanThreads) kda_linear_scan_kernel(const ChunkArgs a) {
    __shared__ int scratch[kRanked + 1];
    const int lc = blockIdx.x / kScanCtas, part = blockIdx.x - lc * kScanCtas;
    const int pos = a.plan.seq_chains + lc, h = pos % a.p.num_heads, W = a.plan.wins;
    const int n = seq_of_rank(a.p, pos / a.p.num_heads, scratch);
    pdl_launch_dependents();
    const size_t off = ((size_t)part * kScanThreads + threadIdx.x) * 4;
    float4 S = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.p.init_state)
        S = *reinterpret_cast<const float4 *>(a.p.init_state + ((size_t)n * a.p.num_heads + h) * (kHeadDim * kHeadDim) + off);
    pdl_wait();
    constexpr int kAhead = 16;  // one round of loads for most plans (4: 7.4 us for 16 windows)
    for (int w0 = 0; w0 < W - 1; w0 += kAhead) {
        float4 d[kAhead];
        float g[kAhead];
        bool on[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int w = w0 + i;
            const Span sp = span_of(a.p, n, w, W, false);
            on[i] = w < W - 1 && sp.live && !sp.last;
            if (on[i]) {
                d[i] = *reinterpret_cast<const float4 *>(slot_of(a, lc, w) + off);
                g[i] = exp2f(a.decay[(size_t)lc * W + w]);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (!on[i]) continue;
            S = make_float4(fmaf(S.x, g[i], d[i].x), fmaf(S.y, g[i], d[i].y), fmaf(S.z, g[i], d[i].z), fmaf(S.w, g[i], d[i].w));
            *reinterpret_cast<float4 *>(slot_of(a, lc, w0 + i) + off) = S;
        }
    }
}

using EncodeTiled = decltype(&cuTensorMapEncodeTiled);

EncodeTiled encode_tiled() {
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return fn;
}

// [T][H][128] BF16, in boxes of `rows` tokens x one head x 64 columns; tokens past T read as zeros.
cudaError_t token_map(CUtensorMap *map, const __nv_bfloat16 *base, int32_t T, int32_t H, cuuint32_t rows) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {kHeadDim, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {kHeadDim * 2, (cuuint64_t)H * kHeadDim * 2};
    const cuuint32_t box[3] = {64, 1, rows}, step[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(base), dims, strides, box,
                              step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool kStates>
cudaError_t configure_once() {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kda_linear_chunk_kernel<kStates>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return cudaSuccess;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t stream, bool dependent,
                   const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = dependent ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Chains that fill at most a third of the GPU, alone or as a last wave, are cut into windows.
Plan plan_linear(int32_t num_seqs, int32_t total_tokens, int32_t num_heads, int32_t sms) {
    const int64_t chains = (int64_t)num_seqs * num_heads;
    Plan p = {1, (int32_t)chains};
    if (chains <= 0 || sms <= 0) return p;
    const int64_t tail = chains % sms;
    const int64_t most = ((int64_t)total_tokens + kC - 1) / kC;  // chunks of any one sequence
    if (tail == 0 || tail * 3 > sms) return p;
    const int64_t wins = std::min<int64_t>(sms / tail, most);
    if (wins < 3) return p;
    p.wins = (int32_t)wins;
    p.seq_chains = (int32_t)(chains - tail);
    return p;
}

int64_t slot_bytes(int64_t tail, int64_t wins) { return tail * (wins - 1) * (kHeadDim * kHeadDim * 4LL); }

}  // namespace

int64_t linear_prefill_workspace_bytes(int32_t num_seqs, int32_t total_tokens, int32_t num_heads, int32_t sms) {
    const Plan p = plan_linear(num_seqs, total_tokens, num_heads, sms);
    if (p.wins == 1) return 0;
    const int64_t tail = (int64_t)num_seqs * num_heads - p.seq_chains;
    return slot_bytes(tail, p.wins) + (tail * p.wins * 4 + 255) / 256 * 256;
}

cudaError_t launch_linear_prefill(const LinearPrefillArgs &args, cudaStream_t stream) {
    const int64_t chains = (int64_t)args.num_seqs * args.num_heads;
    if (args.total_tokens == 0) {  // every sequence is empty: final = initial
        const size_t bytes = (size_t)chains * kHeadDim * kHeadDim * 4;
        if (!args.init_state) return cudaMemsetAsync(args.final_state, 0, bytes, stream);
        if (args.init_state == args.final_state) return cudaSuccess;
        return cudaMemcpyAsync(args.final_state, args.init_state, bytes, cudaMemcpyDeviceToDevice, stream);
    }
    ChunkArgs a;
    a.p = args;
    a.plan = {1, (int32_t)chains};
    a.slots = nullptr;
    a.decay = nullptr;
    if (args.ws) {
        int32_t sms = 0;
        if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
        a.plan = plan_linear(args.num_seqs, args.total_tokens, args.num_heads, sms);
    }
    const int64_t tail = chains - a.plan.seq_chains;
    CUtensorMap mq, mk, mv, mo;
    cudaError_t e = token_map(&mq, args.q, args.total_tokens, args.num_heads, kC);
    if (e == cudaSuccess) e = token_map(&mk, args.k, args.total_tokens, args.num_heads, kC);
    if (e == cudaSuccess) e = token_map(&mv, args.v, args.total_tokens, args.num_heads, kC);
    if (e == cudaSuccess) e = token_map(&mo, args.out, args.total_tokens, args.num_heads, 32);
    if (e == cudaSuccess) e = configure_once<false>();
    if (e != cudaSuccess) return e;
    if (tail > 0) {
        a.slots = static_cast<float *>(args.ws);
        a.decay = a.slots + slot_bytes(tail, a.plan.wins) / 4;
        e = configure_once<true>();
        if (e != cudaSuccess) return e;
        e = launch(kda_linear_chunk_kernel<true>, (unsigned)(tail * (a.plan.wins - 1)), kThreads, kSmem, stream, false, a, mq, mk, mv, mo);
        if (e != cudaSuccess) return e;
        e = launch(kda_linear_scan_kernel, (unsigned)(tail * kScanCtas), kScanThreads, 0, stream, true, a);
        if (e != cudaSuccess) return e;
    }
    return launch(kda_linear_chunk_kernel<false>, (unsigned)(a.plan.seq_chains + tail * a.plan.wins), kThreads, kSmem, stream,
                  tail > 0, a, mq, mk, mv, mo);
}

}  // namespace kda
