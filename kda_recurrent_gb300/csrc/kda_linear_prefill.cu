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
//   warp 2        allocates tensor memory, then the watchdog
//   warp 3        TMA stores of O
//   warps 4-11    A -> P in place in tensor memory, then O: both accumulators -> BF16 -> the tile that
//                 held V
//   warps 12-19   S in registers (row dk, 64 columns a thread): the operand of Q S; V -> hi, lo by quarters
//                 into a ring of two; the update
// The values are decayed, not the keys, because V is only read by the last product of the chunk, so that
// the split needs no scores. It is the longest part of a chunk's chain (0.85k cycles a quarter, most of
// them latency). Measured and dropped: half of it on warps 4-11 behind P (8% slower, it delays D) or
// between P and O (10%, it waits for the next V); on two extra warps (1.5k cycles a quarter); on four (too
// few registers for the state); half of D before Q S (9%, Q's tile, which the next V replaces, is then
// freed late); the next chunk's first quarter split before this chunk's update, or its first two (6 and 13%,
// the same V comes too late for that). In the state pass, which has no P and O, warps 4-11 do every other
// quarter.
//
// O leaves through shared memory because a thread's row-wise 32-byte stores (32 rows an instruction) kept
// the load/store unit busy for 2k cycles a chunk, during which the MMAs' operand reads took four times
// their time (2.56 ms at 8 x 16384 x 96 heads); the end state likewise (5k cycles by direct stores).
// These measurements are in cycles of about 1.85 GHz, all SMs busy.
//
// The suffix sums G_last - G_j are scanned from the end, not formed as differences, so that a
// strong decay early in a chunk costs the later tokens' weights in the state no precision. The scores' exponents
// G_i - G_j are differences of prefix sums: behind many decays near the least one they lose up to 5e-4 of a
// score, a quarter of what its rounding to BF16 may take. A log decay below -128 counts as -128 (both decay to
// zero in FP32), which keeps the sums finite.
//
// Bound: 1 KiB of HBM traffic a token and head against 164 KFLOP of BF16 products, so bandwidth where there
// are chains for every SM: 8 x 16384 tokens x 96 heads take 2.18 to 2.26 ms by machine, 5.7 to 5.9 TB/s (0.85-0.88 of
// a copy's rate), 16 sequences of 256 to 4096 tokens x 32 heads 166-170 us, 5.2 TB/s. A chain alone takes 3.0 us a chunk (its own
// latency: split, D, the update, the operand of the next Q S), about what its share of the bandwidth allows
// when all SMs run one.
//
// Few chains leave most SMs idle. A chain is then cut into windows: a first pass computes each
// window's end state from zero (the update half of the kernel) and its total decay, an
// elementwise pass chains the windows' start states, S_{w+1} = exp(g_w) S_w + D_w, and the chunk
// kernel runs every window from its start state. The same is done for the chains of a short last
// wave, whose windows are launched behind the whole chains. Every window starts from a slot of the
// workspace, the first one too (from a copy of the initial state): the chain's last window, on another CTA,
// may store the end state over the initial one before the first window has begun.
//
// A value that is not finite belongs to its channel's outputs from its token on, but P V carries it to the chunk's
// earlier tokens too (0 inf = NaN). The output warps add 0 times each element of P V to a sum, which is NaN then;
// in that rare case they form the outputs of those tokens again, by single products. At 8 x 16384 x 96 heads this
// takes 1.2%, the saturating conversion in the split 0.6% (looking through the values instead: 6% from the split,
// which is the chunk's critical path, 7% from the output warps, as the chunks are short of shared-memory
// bandwidth).
//
// All waits are bounded; on expiry the CTA records KDA_ERR_DEVICE_TIMEOUT, waits for its own
// copies and MMAs in flight, frees its tensor memory and returns.
#include <cuda.h>

#include <algorithm>

#include "kda_dependent.cuh"
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
constexpr int32_t kTimedOut = 1, kMisplaced = 2;  // why a CTA gave up

struct Gates {
    float prefix[kC];  // log2 units: inclusive prefix sums, and sums over the later tokens
    float suffix[kC];  // (as factors, 2^suffix)
    float decay;       // of the whole chunk
    float pad[3];
};

// Sequences in order of length, longest first (ties by index): items are handed out in index order, so that the
// longest chains are the first ones. More than kRanked sequences keep index order.
constexpr int kRanked = 256;

// A chain, or a window of one. nchunks < 0: there are no more items.
struct Item {
    const float *start;  // state before it, or NULL for zeros
    float *total;        // where its total decay goes (state pass)
    int32_t h, bos, eos, nchunks, updates, last_rows;
    int32_t end_row;     // where its end state goes: row of the end states' tensor, or -1
};

struct Bars {
    uint64_t full[kRing], empty[kRing];  // TMA -> users, users (tcgen05.commit) -> TMA
    uint64_t scores;   // A done
    uint64_t p;        // P written (8 warps)
    uint64_t split[2], split_free[2];  // hi and lo of a quarter written (8 warps), and read
    uint64_t tail[2];  // rows past the window's last token cleared (8 warps)
    uint64_t d;        // D done
    uint64_t d_free;   // D read (8 warps)
    uint64_t s;        // S operand written (8 warps)
    uint64_t qs;       // Q S done: the S operand is free
    uint64_t o;        // P V done (and everything before it)
    uint64_t o_free;   // both output accumulators read (8 warps)
    uint64_t o_tile[2];  // O written to the chunk's V tile (8 warps)
    uint64_t stored[2];  // and read by the stores
    uint64_t gate[2], gate_free[2];
    uint64_t item[2], item_free[2];  // work items handed to the roles
    uint64_t state_read;             // an end state has left shared memory (8 warps)
    uint64_t next;                   // the answer to the request for another item
    uint64_t drain;
    uint64_t finished;  // all roles' warps are done
    uint4 answer;
    Item items[2];
    uint32_t tmem;
    int32_t abort, progress;  // progress: chunks issued
    uint8_t order[kRanked];  // sequences by length, longest first
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

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap *map, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(src)
                 : "memory");
}

__device__ __forceinline__ void tma_store(const CUtensorMap *map, uint32_t src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(src)
                 : "memory");
}

__device__ __forceinline__ void expect_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

// Asks for the index of a CTA of this grid that has not been launched (16 bytes to `answer`, completed
// on `bar`); taken() is the index, or -1 when there was none left.
__device__ __forceinline__ void try_cancel(uint4 *answer, uint64_t *bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_addr(answer)),
                 "r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ int taken(const uint4 *answer) {
    uint32_t x, ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        ".reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %1, 1, 0, p;\n\t"
        "mov.u32 %0, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
        : "=r"(x), "=r"(ok)
        : "r"(smem_addr(answer))
        : "memory");
    return ok ? (int)x : -1;
}

// Wait of a warp, with one decision for all its lanes. It is bounded by the watchdog warp, which raises the
// abort flag when the CTA has made no progress for kWaitLimitNs: with a timer in each of the kernel's
// thirty waits, whose roles share an instruction cache, the kernel was 8 KiB longer. The lanes vote inside
// the loop, so that the compiler sees one exit for the warp: with the vote behind the loop it took
// what follows for divergent, and eight MMAs needed 900 cycles to issue instead of 300 (8 x 16384 x 96
// heads: 2.56 ms).
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Bars *B) {
    const uint32_t addr = smem_addr(bar);
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
        if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int32_t *>(&B->abort))) { ok = false; break; }
    }
    return ok;
}

// The watchdog: returns when all roles' warps have finished, after raising the abort flag if the CTA made no
// progress for kWaitLimitNs. (It sleeps on the barrier, not on a timer, because its return ends the CTA.)
__device__ __forceinline__ void watch(Bars *B) {
    volatile int32_t *const abort = &B->abort, *const progress = &B->progress;
    const uint32_t addr = smem_addr(&B->finished);
    uint64_t since = global_ns();
    int32_t seen = 0;
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], 0, %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(addr), "r"(kSuspendHintNs)
            : "memory");
        if (done) return;
        const int32_t now = *progress;
        if (now != seen) {
            seen = now;
            since = global_ns();
        } else if (global_ns() - since > kWaitLimitNs && !*abort) {
            *abort = kTimedOut;
        }
    }
}

// One arrival for a warp, after what its lanes did.
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

struct Plan {
    int32_t wins;        // windows of each windowed chain (1: none)
    int32_t seq_chains;  // chains before the windowed ones
};

struct ChunkArgs {
    LinearPrefillArgs p;
    Plan plan;
    float *slots;  // windowed chain lc, window w: the end state of window w - 1 alone, then the start of window w
    float *decay;  // windowed chain lc, window w: its total decay (log2)
    int32_t take_over;  // whether a CTA takes over items of CTAs not launched yet: in a grid of one wave, it
                        // would only take those that are about to start on an idle SM
};

__device__ __forceinline__ float *slot_of(const ChunkArgs &a, int lc, int w) {
    return a.slots + ((size_t)lc * a.plan.wins + w) * (kHeadDim * kHeadDim);
}

// order[r] = the sequence of rank r; holds CTA barriers. `scratch`: kRanked ints.
__device__ __forceinline__ void rank_sequences(const LinearPrefillArgs &a, int *scratch, uint8_t *order) {
    const int N = a.num_seqs;
    if (N > kRanked) return;
    if (N == 1) {
        if (threadIdx.x == 0) order[0] = 0;
        __syncthreads();
        return;
    }
#pragma unroll 1
    for (int i = threadIdx.x; i < N; i += blockDim.x)  // wrapping difference: any input orders
        scratch[i] = (int)((unsigned)__ldg(a.cu_seqlens + i + 1) - (unsigned)__ldg(a.cu_seqlens + i));
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
        const int li = scratch[i];
        int r = 0;
#pragma unroll 1
        for (int m = 0; m < N; ++m) r += (scratch[m] > li) | ((scratch[m] == li) & (m < i));
        order[r] = (uint8_t)i;
    }
    __syncthreads();
}

struct Span {
    int bos, eos;  // tokens of the window
    bool first, last, live;
};

// Window w (of at most W) of sequence n.
__device__ __forceinline__ Span span_of(const LinearPrefillArgs &a, int n, int w, int W, bool report) {
    int sb = a.cu_seqlens[n], se = a.cu_seqlens[n + 1];
    if (sb < 0 || se < sb || se > a.total_tokens) {
        if (report && (threadIdx.x & 31) == 0) report_error(a.status, KDA_ERR_DEVICE_INPUT, n);
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
// the split stage at `to`. hi saturates: an infinity becomes the largest number and an infinity, whose products
// with a key have one sign.
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
            hi[e] = pack_bf16_finite(y0, y1);
            rest[e] = pack_bf16(y0 - __uint_as_float(hi[e] << 16), y1 - __uint_as_float(hi[e] & 0xffff0000u));
        }
        *reinterpret_cast<uint4 *>(to + i * kSplitHalf) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(to + kSplitLo + i * kSplitHalf) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
    }
}

__device__ __forceinline__ float dot2(uint32_t x, uint32_t y, float sum) {  // of two BF16 pairs
    sum = fmaf(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u), sum);
    return fmaf(__uint_as_float(x << 16), __uint_as_float(y << 16), sum);
}

// lam * (Q S) + scale * sum_{j <= row} P_ij v_j again, token by token in FP32, for the channels of a row's 64 that a
// value which is not finite reached from a later token of its chunk only (0.06 to 3.3 ms a chunk). `out` holds the row's outputs, its 16-byte
// groups swizzled by `swizzle`; Q S is at `qs` in tensor memory. Called by whole warps; `live`: the row is a token.
__device__ __noinline__ void repair_row(const LinearPrefillArgs &p, int h, int t0, int row, int rows, int half, bool live, float lam,
                                        uint32_t qs, uint4 *out, int swizzle) {
    const size_t stride = (size_t)p.num_heads * kHeadDim, first = (size_t)t0 * stride + (size_t)h * kHeadDim;
    const __nv_bfloat16 *const v = p.v + first + 64 * half, *const k = p.k + first, *const q = p.q + first + row * stride;
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
        __syncwarp();
        float x[16];
        tmem_ld16(qs + 16 * (i >> 1), x);
        tmem_wait_ld();
        uint32_t own[4] = {}, later[4] = {};  // two channels each
#pragma unroll 8
        for (int j = 0; j < rows; ++j) {
            const uint4 w = *reinterpret_cast<const uint4 *>(v + j * stride + 8 * i);
            const uint32_t u[4] = {not_finite(w.x), not_finite(w.y), not_finite(w.z), not_finite(w.w)};
#pragma unroll
            for (int e = 0; e < 4; ++e) (j <= row ? own[e] : later[e]) |= u[e];
        }
        uint32_t any = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) any |= later[e] &= ~own[e];
        if (!live || any == 0) continue;
        float sum[8] = {}, decay = 0.0f;
#pragma unroll 1
        for (int j = row; j >= 0; --j) {
            float s = 0.0f;
#pragma unroll 4
            for (int d = 0; d < kHeadDim; d += 8) {
                const uint4 a = *reinterpret_cast<const uint4 *>(q + d), b = *reinterpret_cast<const uint4 *>(k + j * stride + d);
                s = dot2(a.x, b.x, dot2(a.y, b.y, dot2(a.z, b.z, dot2(a.w, b.w, s))));
            }
            s *= ex2(decay);
#pragma unroll
            for (int c = 0; c < 8; ++c) sum[c] = fmaf(s, __bfloat162float(v[j * stride + 8 * i + c]), sum[c]);
            const float g = p.log_decay[(size_t)(t0 + j) * p.decay_token_stride + h];
            decay += (g < kMinLogDecay ? kMinLogDecay : g) * kLog2e;
        }
        uint4 *const at = out + (i ^ swizzle);
        const uint4 w = *at;
        uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x0 = i & 1 ? x[8 + 2 * e] : x[2 * e], x1 = i & 1 ? x[9 + 2 * e] : x[2 * e + 1];
            const uint32_t mask = (later[e] >> 15) * 0xffffu;
            y[e] = (y[e] & ~mask) | (pack_bf16(fmaf(lam, x0, p.scale * sum[2 * e]), fmaf(lam, x1, p.scale * sum[2 * e + 1])) & mask);
        }
        *at = make_uint4(y[0], y[1], y[2], y[3]);
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
#pragma unroll 1
    for (int u = uses / 3 * 3; u < uses; ++u) vs += (first + kRing * u) % 3 == 2;
    return (uses - vs) & 1;
}

// The work item of index i: a whole chain, or a window of a windowed chain.
template <bool kStates>
__device__ __forceinline__ Item item_of(const ChunkArgs &a, int i, const uint8_t *order) {
    const LinearPrefillArgs &p = a.p;
    const int W = a.plan.wins, H = p.num_heads;
    int pos = i, w = 0, lc = -1;
    if (kStates || i >= a.plan.seq_chains) {
        const int per = kStates ? W - 1 : W;
        if (!kStates) i -= a.plan.seq_chains;
        lc = i / per;
        w = i - lc * per;
        pos = a.plan.seq_chains + lc;
    }
    const int h = pos % H, rank = pos / H;
    const int n = p.num_seqs <= kRanked ? order[rank] : rank;
    const Span sp = span_of(p, n, w, lc >= 0 ? W : 1, !kStates && h == 0 && w == 0);
    const size_t chain = ((size_t)n * H + h) * (kHeadDim * kHeadDim);
    Item it;
    it.h = h;
    it.bos = sp.bos;
    it.eos = sp.eos;
    it.nchunks = (sp.eos - sp.bos + kC - 1) / kC;
    it.start = nullptr;
    it.end_row = -1;
    it.total = nullptr;
    if (kStates) {
        if (!sp.live || sp.last) {
            it.nchunks = 0;
        } else {
            it.end_row = (lc * W + w + 1) * kHeadDim;
            it.total = a.decay + (size_t)lc * W + w;
        }
    } else if (sp.live) {
        if (lc >= 0 && (!sp.first || p.init_state)) it.start = slot_of(a, lc, w);
        else if (p.init_state) it.start = p.init_state + chain;
        it.end_row = sp.last && p.final_state ? (n * H + h) * kHeadDim : -1;
    }
    // the last chunk's update is needed only where somebody reads the end state
    it.updates = it.end_row >= 0 ? it.nchunks : it.nchunks - 1;
    it.last_rows = it.eos - it.bos - (it.nchunks - 1) * kC;
    return it;
}

// kStates: only the state update, from zero, over the windows of the windowed chains but the last.
//
// A CTA runs item after item (its own index first, then those of CTAs of the grid that have not been
// launched, which it takes over by clusterlaunchcontrol), and the roles go from one item's last chunk to
// the next one's first without emptying the pipeline. It asks for the next item when it begins one, which
// hides the answer's latency, also in items of one chunk, but holds that item back from SMs that run out of
// work earlier: items are handed out in index order, one ahead of when they are begun. All counters that give a
// barrier's phase run on over the items.
template <bool kStates>
__global__ void __launch_bounds__(kThreads, 1)
    kda_linear_chunk_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap map_q,
                            const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                            const __grid_constant__ CUtensorMap map_o, const __grid_constant__ CUtensorMap map_s) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const LinearPrefillArgs &p = a.p;
    Bars *B = reinterpret_cast<Bars *>(smem + kBars);
    // the shuffle tells the compiler that the role is one for the warp
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, H = p.num_heads;
    if (threadIdx.x == 32) {
        prefetch_map(&map_k);
        prefetch_map(&map_v);
        prefetch_map(&map_s);
        if (!kStates) prefetch_map(&map_q), prefetch_map(&map_o);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) mbar_init(&B->full[i], 1), mbar_init(&B->empty[i], 1);
        mbar_init(&B->scores, 1);
        mbar_init(&B->p, kOutWarps);
        mbar_init(&B->d, 1);
        mbar_init(&B->d_free, kStateWarps);
        mbar_init(&B->s, kStateWarps);
        mbar_init(&B->qs, 1);
        mbar_init(&B->o, 1);
        mbar_init(&B->o_free, kOutWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B->split[i], kStateWarps);
            mbar_init(&B->split_free[i], 1);
            mbar_init(&B->tail[i], kStateWarps);
            mbar_init(&B->o_tile[i], kOutWarps);
            mbar_init(&B->stored[i], 1);
            mbar_init(&B->gate[i], 1);
            mbar_init(&B->gate_free[i], kStateWarps + kOutWarps);
            mbar_init(&B->item[i], 1);
            mbar_init(&B->item_free[i], 1 + kStateWarps + kOutWarps + (kStates ? 0 : 1));
        }
        mbar_init(&B->state_read, kStateWarps);
        mbar_init(&B->next, 1);
        mbar_init(&B->drain, 1);
        mbar_init(&B->finished, (kStates ? 2 : 3) + kOutWarps + kStateWarps);
        // the swizzled tiles are laid out for a 1024-byte-aligned base
        B->abort = (smem_addr(smem) & 1023u) != 0 ? kMisplaced : 0;
        B->progress = 0;
        if (B->abort) report_error(p.status, KDA_ERR_CUDA, 0);
        fence_mbar_init();
    }
    wait_for_prior();
    if (kStates) allow_next();
    rank_sequences(p, reinterpret_cast<int *>(smem), B->order);
    fence_async_smem();  // the ranking's scratch lies where the first tiles go
    __syncthreads();
    // Tensor memory is allocated while warp 0 begins to load.
    constexpr uint32_t tmem = 0;
    if (warp == kWarpAlloc) {
        tmem_alloc(&B->tmem, kTmemCols);
        tmem_relinquish();
        if (lane == 0 && *reinterpret_cast<volatile uint32_t *>(&B->tmem) != tmem) {
            report_error(p.status, KDA_ERR_CUDA, 1);
            *reinterpret_cast<volatile int32_t *>(&B->abort) = kMisplaced;
        }
    }
    if (warp != 0) {
        tc_fence_before();
        asm volatile("bar.sync 1, %0;" ::"n"(kThreads - 32) : "memory");
        tc_fence_after();
    }
    const uint32_t base = smem_addr(smem);
    constexpr int kPer = kStates ? 2 : 3;  // tiles of a chunk: (Q,) K, V
    int issued = 0;                        // loads issued (warp 0)
    int asked = 0, told = 0;               // next items asked for, and answers seen (warp 0)

    // The k-th item, for every role but warp 0; nchunks < 0 after the last (and if the CTA gave up). The
    // shuffles tell the compiler that the values are one for the warp.
    auto next_item = [&](int k) {
        const bool ok = wait_warp(&B->item[k & 1], (k >> 1) & 1, B);
        const Item &from = B->items[k & 1];
        Item it;
        it.start = from.start;
        it.h = __shfl_sync(0xffffffffu, from.h, 0);
        it.bos = __shfl_sync(0xffffffffu, from.bos, 0);
        it.eos = __shfl_sync(0xffffffffu, from.eos, 0);
        it.nchunks = __shfl_sync(0xffffffffu, ok ? from.nchunks : -1, 0);
        it.updates = __shfl_sync(0xffffffffu, from.updates, 0);
        it.last_rows = __shfl_sync(0xffffffffu, from.last_rows, 0);
        it.end_row = __shfl_sync(0xffffffffu, from.end_row, 0);
        arrive_warp(&B->item_free[k & 1]);
        return it;
    };

    // hi and lo of the quarters of chunk g (L tokens, values at `tile`) by the 256 threads of a group; `use`
    // counts the quarters of all chunks through the ring of two stages. odd < 0: all quarters, else those of
    // that parity.
    auto split = [&](const uint8_t *tile, int g, int L, int &use, int odd, int tid) {
        const Gates *G = reinterpret_cast<const Gates *>(smem + kGates) + (g & 1);
#pragma unroll 1
        for (int r = 0; r < L; r += kQuarter, ++use) {
            const int st = use & 1, t = r + (tid >> 3);
            if (odd >= 0 && st != odd) continue;
            if (use >= 2 && !wait_warp(&B->split_free[st], ((use >> 1) - 1) & 1, B)) return false;
            split_quarter(tile + tid * 16 + r * 128, smem + kSplit + st * kSplitStage + tid * 16, G->suffix[t], t < L);
            fence_async_smem();
            arrive_warp(&B->split[st]);
        }
        return true;
    };

    if (B->abort) {
        // nothing has started
    } else if (warp == 0) {
        int g = 0, index = blockIdx.x;  // g: chunks of the items before
        for (int k = 0;; ++k) {
            Item it;
            it.nchunks = -1;
            if (index >= 0) it = item_of<kStates>(a, index, B->order);
            if (k >= 2 && !wait_warp(&B->item_free[k & 1], ((k >> 1) - 1) & 1, B)) break;
            if (lane == 0) B->items[k & 1] = it;
            arrive_warp(&B->item[k & 1]);
            if (index < 0) break;
            if (a.take_over) {
                if (lane == 0) {
                    fence_async_smem();
                    expect_tx(&B->next, 16);
                    try_cancel(&B->answer, &B->next);
                }
                ++asked;
            }
            bool ok = true;
            float run = 0.0f;  // total decay of the window so far
            for (int c = 0; c < it.nchunks; ++c, ++g) {
                const int t0 = it.bos + c * kC, L = min(kC, it.eos - t0), b = g & 1;
                float x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 4 * lane + e;
                    x[e] = t < L ? p.log_decay[(size_t)(t0 + t) * p.decay_token_stride + it.h] : 0.0f;
                }
#pragma unroll 1
                for (int which = 0; which < kPer; ++which, ++issued) {
                    const int slot = issued % kRing;
                    if (issued >= kRing) {  // the tile five loads ago has been read
                        const int before = issued - kRing, cb = before / kPer;
                        const bool is_v = !kStates && before - cb * kPer == kPer - 1;  // then also as O
                        ok = is_v ? wait_warp(&B->stored[cb & 1], (cb >> 1) & 1, B)
                                  : wait_warp(&B->empty[slot], empty_parity(before, kStates), B);
                        if (!ok) break;
                    }
                    const CUtensorMap *map = which == kPer - 1 ? &map_v : which == kPer - 2 ? &map_k : &map_q;
                    if (lane == 0) {
                        expect_tx(&B->full[slot], kTile);
                        tma_load(base + slot * kTile, map, 0, it.h, t0, &B->full[slot]);
                        tma_load(base + slot * kTile + kHalf, map, 64, it.h, t0, &B->full[slot]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = (x[e] < kMinLogDecay ? kMinLogDecay : x[e]) * kLog2e;
                const float mine = (x[0] + x[1]) + (x[2] + x[3]);
                float up = mine, down = mine;  // inclusive over the lanes before, and after
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, up, o), z = __shfl_down_sync(0xffffffffu, down, o);
                    if (lane >= o) up += y;
                    if (lane + o < 32) down += z;
                }
                float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, down, 1);
                if (lane == 0) before = 0.0f;
                if (lane == 31) after = 0.0f;
                const float total = __shfl_sync(0xffffffffu, down, 0);
                ok = g < 2 || wait_warp(&B->gate_free[b], ((g >> 1) - 1) & 1, B);
                if (!ok) break;
                Gates *G = reinterpret_cast<Gates *>(smem + kGates) + b;
                const float p0 = before + x[0], p1 = p0 + x[1], p2 = p1 + x[2], p3 = p2 + x[3];
                *reinterpret_cast<float4 *>(&G->prefix[4 * lane]) = make_float4(p0, p1, p2, p3);
                const float s2 = after + x[3], s1 = s2 + x[2], s0 = s1 + x[1];
                *reinterpret_cast<float4 *>(&G->suffix[4 * lane]) = make_float4(ex2(s0), ex2(s1), ex2(s2), ex2(after));
                // exp2f, not the 2^-22 of the hardware's: this error repeats every chunk and adds up over
                // the chunks that a slowly decaying state remembers
                if (lane == 0) G->decay = exp2f(total);
                arrive_warp(&B->gate[b]);
                run += total;
            }
            if (!ok) break;
            if (kStates && lane == 0 && it.total) *it.total = run;
            index = -1;
            if (!a.take_over) continue;
            if (!wait_warp(&B->next, k & 1, B)) break;
            ++told;
            index = taken(&B->answer);
            __syncwarp();
        }
    } else if (warp == kWarpMma) {
        int g = 0, u = 0, use = 0, tl = 0;  // chunks, updates, quarters and partial chunks so far
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Item it = next_item(k);
            if (it.nchunks < 0) break;
            for (int c = 0; c < it.nchunks; ++c, ++g) {
                ok = false;
                if (lane == 0) *reinterpret_cast<volatile int32_t *>(&B->progress) = g + 1;
                const int iq = g * kPer, ik = iq + kPer - 2, iv = ik + 1;
                const uint32_t k = base + (ik % kRing) * kTile, q = base + (iq % kRing) * kTile, v = base + (iv % kRing) * kTile;
                const int L = c + 1 < it.nchunks ? kC : it.last_rows;
                if (!wait_warp(&B->full[ik % kRing], (ik / kRing) & 1, B)) break;
                if (!kStates) {
                    if (!wait_warp(&B->full[iq % kRing], (iq / kRing) & 1, B)) break;
                    if (g > 0 && !wait_warp(&B->o, (g - 1) & 1, B)) break;  // P of the last chunk has been read
                    const uint64_t dq = at(kDescK, q), dk = at(kDescK, k);
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t off = ((s >> 2) * kHalf + (s & 3) * 32) >> 4;
                        mma_ss(tmem + kColA, dq + off, dk + off, kIdescQK, s > 0);
                    }
                    commit(&B->scores);
                    if (!wait_warp(&B->s, g & 1, B)) break;
                    if (g > 0 && !wait_warp(&B->o_free, (g - 1) & 1, B)) break;
                    tc_fence_after();
                    const uint64_t ds = at(kDescMn, base + kS);
#pragma unroll
                    for (int s = 0; s < 8; ++s)
                        mma_ss(tmem + kColQS, dq + (((s >> 2) * kHalf + (s & 3) * 32) >> 4), ds + s * 128, kIdescQS, s > 0);
                    commit(&B->qs);
                    commit(&B->empty[iq % kRing]);
                }
                if (L < kC) {
                    if (!wait_warp(&B->tail[tl & 1], (tl >> 1) & 1, B)) break;
                    ++tl;
                }
                if (c < it.updates) {
                    if (u > 0 && !wait_warp(&B->d_free, (u - 1) & 1, B)) break;
                    bool lost = false;
#pragma unroll 1
                    for (int r = 0; r < L; r += kQuarter, ++use) {
                        const int st = use & 1;
                        lost = !wait_warp(&B->split[st], (use >> 1) & 1, B);
                        if (lost) break;
                        tc_fence_after();
                        const uint64_t da = at(kDescMn, k + r * 128), db = at(kDescSplit, base + kSplit + st * kSplitStage);
#pragma unroll
                        for (int s = 0; s < 4; ++s)  // hi, hi, lo, lo
                            mma_ss(tmem + kColD, da + (s & 1) * 128, db + (((s >> 1) * kSplitLo + (s & 1) * 2048) >> 4), kIdescD,
                                   r > 0 || s > 0);
                        commit(&B->split_free[st]);
                    }
                    if (lost) break;
                    commit(&B->d);
                    ++u;
                }
                commit(&B->empty[ik % kRing]);
                if (!wait_warp(&B->full[iv % kRing], (iv / kRing) & 1, B)) break;
                if (!kStates) {
                    if (!wait_warp(&B->p, g & 1, B)) break;
                    tc_fence_after();
                    const uint64_t dv = at(kDescMn, v);
#pragma unroll
                    for (int s = 0; s < 8; ++s)  // (16 tokens past the last one would be zeros)
                        if (s * 16 < L) mma_ts(tmem + kColO, tmem + kColA + 32 * (s >> 1) + 8 * (s & 1), dv + s * 128, kIdescPV, s > 0);
                    commit(&B->o);
                }
                if (kStates) commit(&B->empty[iv % kRing]);
                ok = true;
            }
            if (it.nchunks == 0) ok = true;
        }
        commit(&B->drain);  // every earlier commit has reached its barrier when this one has
        mbar_wait(&B->drain, 0);
    } else if (warp == kWarpStore && !kStates) {
        // lane 4 h + q stores rows [32 q, 32 q + 32) of half h, unless they are not all tokens of the window
        // (then their warp has stored what is left)
        const int quad = lane & 3, half = lane >> 2;
        int g = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Item it = next_item(k);
            if (it.nchunks < 0) break;
            for (int c = 0; c < it.nchunks; ++c, ++g) {
                ok = wait_warp(&B->o_tile[g & 1], (g >> 1) & 1, B);
                if (!ok) break;
                const int iv = g * kPer + kPer - 1;
                if (lane < 8 && (c + 1 < it.nchunks || 32 * quad + 32 <= it.last_rows)) {
                    tma_store(&map_o, base + (iv % kRing) * kTile + half * kHalf + quad * 4096, 64 * half, it.h, it.bos + c * kC + 32 * quad);
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                }
                arrive_warp(&B->stored[g & 1]);
            }
        }
    } else if (warp == kWarpAlloc) {
        watch(B);
    } else if (kStates && warp >= kWarpO && warp < kWarpS) {
        // the state pass has no outputs: these warps split the odd quarters
        const int tid = threadIdx.x - kWarpO * 32;
        int g = 0, use = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Item it = next_item(k);
            if (it.nchunks < 0) break;
            for (int c = 0; c < it.nchunks; ++c, ++g) {
                const int iv = g * kPer + kPer - 1, L = c + 1 < it.nchunks ? kC : it.last_rows;
                ok = wait_warp(&B->gate[g & 1], (g >> 1) & 1, B) && wait_warp(&B->full[iv % kRing], (iv / kRing) & 1, B) &&
                     split(smem + (iv % kRing) * kTile, g, L, use, 1, tid);
                if (!ok) break;
                arrive_warp(&B->gate_free[g & 1]);
            }
        }
    } else if (warp < kWarpO) {
        // idle
    } else if (warp < kWarpS) {
        const int quad = warp & 3, half = (warp - kWarpO) >> 2, row = 32 * quad + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        int g = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Item it = next_item(k);
            if (it.nchunks < 0) break;
            for (int c = 0; c < it.nchunks; ++c, ++g) {
                ok = false;
                const Gates *G = reinterpret_cast<const Gates *>(smem + kGates) + (g & 1);
                if (!wait_warp(&B->gate[g & 1], (g >> 1) & 1, B)) break;
                const float gi = G->prefix[row], lam = p.scale * ex2(gi);
                if (!wait_warp(&B->scores, g & 1, B)) break;
                tc_fence_after();
                // this warp's blocks of 32 columns: every other one
#pragma unroll 1
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
                if (lane == 0) mbar_arrive(&B->gate_free[g & 1]);
                if (!wait_warp(&B->o, g & 1, B)) break;
                tc_fence_after();
                // rows of 128 bytes into the V tile, which nobody reads any more, for warp 3 to store; a warp whose
                // rows are not all tokens of the window stores them itself
                const int iv = g * kPer + kPer - 1, t = it.bos + c * kC + row;
                const bool whole = c + 1 < it.nchunks || 32 * quad + 32 <= it.last_rows;
                uint8_t *const rows = smem + (iv % kRing) * kTile + half * kHalf + quad * 4096;
                uint4 *const dst = reinterpret_cast<uint4 *>(p.out + ((size_t)t * H + it.h) * kHeadDim + 64 * half);
                float finite[4] = {};
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float o[16], x[16];
                    tmem_ld16(lanes + kColO + 64 * half + 16 * b, o);
                    tmem_ld16(lanes + kColQS + 64 * half + 16 * b, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) finite[j & 3] = fmaf(o[j], 0.0f, finite[j & 3]);
                    uint32_t pk[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        pk[j] = pack_bf16(fmaf(lam, x[2 * j], p.scale * o[2 * j]), fmaf(lam, x[2 * j + 1], p.scale * o[2 * j + 1]));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint4 y = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                        if (whole)
                            *reinterpret_cast<uint4 *>(rows + lane * 128 + (((2 * b + i) ^ (lane & 7)) << 4)) = y;
                        else if (t < it.eos)
                            dst[2 * b + i] = y;
                    }
                }
                if (__any_sync(0xffffffffu, (finite[0] + finite[1]) + (finite[2] + finite[3]) != 0.0f && t < it.eos))
                    repair_row(p, it.h, it.bos + c * kC, row, c + 1 < it.nchunks ? kC : it.last_rows, half, t < it.eos, lam,
                               lanes + kColQS + 64 * half, whole ? reinterpret_cast<uint4 *>(rows + lane * 128) : dst, whole ? lane & 7 : 0);
                tc_fence_before();
                fence_async_smem();
                arrive_warp(&B->o_free);
                if (lane == 0) mbar_arrive(&B->o_tile[g & 1]);
                ok = true;
            }
            if (it.nchunks == 0) ok = true;
        }
    } else {
        const int quad = warp & 3, half = (warp - kWarpS) >> 2, row = 32 * quad + lane;  // row: dk
        const int tid = threadIdx.x - kWarpS * 32;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + kColD + 64 * half;
        uint8_t *const s_row = smem + kS + half * kHalf + row * 128;
        int g = 0, u = 0, use = 0, tl = 0;  // chunks, updates, quarters and partial chunks so far
        float S[64];
        int stored = 0;  // end states that have left shared memory
        bool ok = true, storing = false;
        for (int k = 0; ok; ++k) {
            const Item it = next_item(k);
            if (it.nchunks < 0) break;
            const size_t mine = (size_t)row * kHeadDim + 64 * half;
            if (it.start) {
                const float4 *src = reinterpret_cast<const float4 *>(it.start + mine);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float4 x = src[i];
                    S[4 * i] = x.x, S[4 * i + 1] = x.y, S[4 * i + 2] = x.z, S[4 * i + 3] = x.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 64; ++i) S[i] = 0.0f;
            }
            if (storing) {  // the last item's end state, by all state warps
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                arrive_warp(&B->state_read);
                ok = wait_warp(&B->state_read, stored & 1, B);
                if (!ok) break;
                ++stored;
                storing = false;
            }
            for (int c = 0; c < it.nchunks; ++c, ++g) {
                ok = false;
                if (!kStates) {  // S as the BF16 operand of Q S
                    if (g > 0 && !wait_warp(&B->qs, (g - 1) & 1, B)) break;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4 *>(s_row + ((i ^ (row & 7)) << 4)) =
                            make_uint4(pack_bf16(S[8 * i], S[8 * i + 1]), pack_bf16(S[8 * i + 2], S[8 * i + 3]),
                                       pack_bf16(S[8 * i + 4], S[8 * i + 5]), pack_bf16(S[8 * i + 6], S[8 * i + 7]));
                    fence_async_smem();
#ifdef KDA_TEST_WITHHOLD_HANDOFF  // failure-detection test: one hand-off never comes
                    if (g != KDA_TEST_WITHHOLD_HANDOFF)
#endif
                        arrive_warp(&B->s);
                }
                const int ik = g * kPer + kPer - 2, iv = ik + 1;
                const int L = c + 1 < it.nchunks ? kC : it.last_rows;
                const Gates *G = reinterpret_cast<const Gates *>(smem + kGates) + (g & 1);
                if (!wait_warp(&B->gate[g & 1], (g >> 1) & 1, B)) break;
                if (!wait_warp(&B->full[iv % kRing], (iv / kRing) & 1, B)) break;
                uint8_t *const values = smem + (iv % kRing) * kTile;
                if (L < kC) {
                    // The rows past the last token hold another sequence's keys and values, which a zero in the
                    // other operand does not silence if they are not finite: clear them.
                    if (!wait_warp(&B->full[ik % kRing], (ik / kRing) & 1, B)) break;
                    uint8_t *const keys = smem + (ik % kRing) * kTile;
#pragma unroll 1
                    for (int x = tid; x < 2048; x += kStateThreads)
                        if (((x & 1023) >> 3) >= L)
                            *reinterpret_cast<uint4 *>(values + x * 16) = *reinterpret_cast<uint4 *>(keys + x * 16) = make_uint4(0, 0, 0, 0);
                    fence_async_smem();
                    arrive_warp(&B->tail[tl & 1]);
                    ++tl;
                }
                if (c < it.updates && !split(values, g, L, use, kStates ? 0 : -1, tid)) break;
                const float decay = G->decay;
                arrive_warp(&B->gate_free[g & 1]);
                if (c < it.updates) {
                    if (!wait_warp(&B->d, u & 1, B)) break;
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
                    arrive_warp(&B->d_free);  // (only with an update: an arrival for a chunk without one could
                                              // complete a second phase before the MMA warp has seen the first)
                    ++u;
                }
                ok = true;
            }
            if (it.nchunks == 0) ok = true;
            if (ok && it.end_row >= 0) {
                // 32 columns at a time (128-byte rows, swizzled), each by one TMA store, through the warp's own 4 KiB
                // of the S operand, once the last chunk's queries have read it, then of the split stages, which the
                // last D has read; they are waited for when the next item writes there (1.6% at 16 ragged sequences
                // of 32 heads). The state pass, which shares the split stages with warps 4-11, has one item.
                if (!kStates && g > 0 && !wait_warp(&B->qs, (g - 1) & 1, B)) {
                    ok = false;
                    break;
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint8_t *const stage = smem + (kStates || r == 0 ? kS : kSplit) + (half * 4 + quad) * 4096;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4 *>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                            make_float4(S[32 * r + 4 * i], S[32 * r + 4 * i + 1], S[32 * r + 4 * i + 2], S[32 * r + 4 * i + 3]);
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store(&map_s, smem_addr(stage), 64 * half + 32 * r, it.end_row + 32 * quad);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        if (kStates) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    }
                    __syncwarp();
                }
                storing = !kStates;
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    __syncwarp();
    if (lane == 0 && warp != kWarpAlloc && !(kStates && warp == kWarpStore)) mbar_arrive(&B->finished);
    __syncthreads();
    if (B->abort) {  // wait (bounded) for what is still in flight before the memory is given back
        if (threadIdx.x == 0) {
            if (B->abort == kTimedOut) report_error(p.status, KDA_ERR_DEVICE_TIMEOUT, (int)blockIdx.x);
#pragma unroll 1
            for (int i = max(0, issued - kRing); i < issued; ++i) mbar_wait(&B->full[i % kRing], (i / kRing) & 1);
            if (asked > told) mbar_wait(&B->next, told & 1);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == kWarpAlloc) tmem_dealloc(B->tmem, kTmemCols);
}

// S_{w+1} = exp2(g_w) S_w + D_w over the windows of a windowed chain, in place in its slots, from a copy of the
// initial state in the first; one float4 of the state a thread, the windows' own states loaded ahead.
constexpr int kScanThreads = 128;
constexpr int kScanCtas = kHeadDim * kHeadDim / (4 * kScanThreads);

__global__ void __launch_bounds__(kScanThreads) kda_linear_scan_kernel(const ChunkArgs a) {
    __shared__ int scratch[kRanked];
    __shared__ uint8_t order[kRanked];
    const int lc = blockIdx.x / kScanCtas, part = blockIdx.x - lc * kScanCtas;
    const int pos = a.plan.seq_chains + lc, h = pos % a.p.num_heads, W = a.plan.wins;
    allow_next();
    wait_for_prior();
    rank_sequences(a.p, scratch, order);
    const int n = a.p.num_seqs <= kRanked ? order[pos / a.p.num_heads] : pos / a.p.num_heads;
    const size_t off = ((size_t)part * kScanThreads + threadIdx.x) * 4;
    float4 S = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.p.init_state)
        S = *reinterpret_cast<const float4 *>(a.p.init_state + ((size_t)n * a.p.num_heads + h) * (kHeadDim * kHeadDim) + off);
    if (a.p.init_state) *reinterpret_cast<float4 *>(slot_of(a, lc, 0) + off) = S;
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
                d[i] = *reinterpret_cast<const float4 *>(slot_of(a, lc, w + 1) + off);
                g[i] = exp2f(a.decay[(size_t)lc * W + w]);
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (!on[i]) continue;
            S = make_float4(fmaf(S.x, g[i], d[i].x), fmaf(S.y, g[i], d[i].y), fmaf(S.z, g[i], d[i].z), fmaf(S.w, g[i], d[i].w));
            *reinterpret_cast<float4 *>(slot_of(a, lc, w0 + i + 1) + off) = S;
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

// States [states][128][128] FP32 as rows of 128, in boxes of 32 rows x 32 columns.
cudaError_t state_map(CUtensorMap *map, const void *base, int64_t states) {
    const EncodeTiled encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {kHeadDim, (cuuint64_t)states * kHeadDim};
    const cuuint64_t strides[1] = {kHeadDim * 4};
    const cuuint32_t box[2] = {32, 32}, step[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
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

// Chains that fill at most a third of the GPU, alone or as a last wave, are cut into windows, if the longest
// of them can be expected to gain: the lengths are on the device, so it is taken to be what it is on average
// for lengths uniform over [0, L], 2 / (num_seqs + 1) of all chunks. A chunk takes 3.0 us of a chain's time,
// windows cost about 12 us and run through a window's chunks twice (the first time faster). Whole chains
// against windows, in us: 8 chains (19 windows) of 4 chunks 17 and 21, of 8 29 and 22, of 64 194 and 41; 24
// chains (6 windows) of 6 chunks 23 and 25, of 12 41 and 30; 48 chains (3 windows) of 16 chunks 54 and 55, of
// 24 77 and 67.
constexpr int64_t kLeastGain = 5;  // chunks

Plan plan_linear(int32_t num_seqs, int32_t total_tokens, int32_t num_heads, int32_t sms) {
    const int64_t chains = (int64_t)num_seqs * num_heads;
    Plan p = {1, (int32_t)chains};
    if (chains <= 0 || sms <= 0) return p;
    const int64_t tail = chains % sms;
    const int64_t most = ((int64_t)total_tokens + kC - 1) / kC;  // chunks of any one sequence
    if (tail == 0 || tail * 3 > sms || most == 0) return p;
    const int64_t wins = std::min<int64_t>(sms / tail, most), longest = 2 * most / (num_seqs + 1);
    if (longest - 2 * ((longest + wins - 1) / wins) < kLeastGain) return p;
    p.wins = (int32_t)wins;
    p.seq_chains = (int32_t)(chains - tail);
    return p;
}

int64_t slot_bytes(int64_t tail, int64_t wins) { return tail * wins * (kHeadDim * kHeadDim * 4LL); }

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
    a.take_over = 0;
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    if (args.ws) {
        a.plan = plan_linear(args.num_seqs, args.total_tokens, args.num_heads, sms);
    }
    const int64_t tail = chains - a.plan.seq_chains;
    CUtensorMap mq, mk, mv, mo, ms;
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
        e = state_map(&ms, a.slots, tail * a.plan.wins);
        if (e != cudaSuccess) return e;
        e = launch_dependent(kda_linear_chunk_kernel<true>, (unsigned)(tail * (a.plan.wins - 1)), kThreads, kSmem, stream, a, mq, mk, mv, mo,
                   ms);
        if (e != cudaSuccess) return e;
        e = launch_dependent(kda_linear_scan_kernel, (unsigned)(tail * kScanCtas), kScanThreads, 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    const int64_t items = a.plan.seq_chains + tail * a.plan.wins;
    a.take_over = items > sms;
    // (without a final state the map is not used)
    e = args.final_state ? state_map(&ms, args.final_state, chains) : state_map(&ms, args.q, 1);
    if (e != cudaSuccess) return e;
    return launch_dependent(kda_linear_chunk_kernel<false>, (unsigned)items, kThreads, kSmem, stream, a, mq, mk, mv, mo, ms);
}

}  // namespace kda
