// Queries and keys on their way into attention (sm_103a): the norm of each head, the rotation by position, and
// the write of keys and values into the pages of the key-value cache, in one pass.
//
//     y = x (mean x^2 + eps)^-1/2 w                      (where a weight is given)
//     (a, b) -> m (a cos - b sin, b cos + a sin)         for the pairs of the first `rot` channels, angle pos f_i
//
// Every number is read once and written once, so the kernel is a stream: eight lanes hold a head (two pieces of
// 16 bytes a lane), a warp eight heads at a time, and the next eight are on their way while these are computed. A
// lane's two pieces hold both members of its pairs, in either layout, so that only the norm's sum crosses lanes
// (three shuffles; with sixteen lanes a head, and the halves' pairs exchanged by shuffles, 131072 tokens of 64/8 heads
// took 1031 us instead of 813-818, 6.6 TB/s, 0.97 of a copy's rate). With many tokens a warp walks all heads of a token, so
// that its angles are computed once; with few, a token's heads are shared between warps (1 token of 32/8 heads 2.9 us,
// by one warp 6.4; 333 tokens 5.1 and 7.8; 2432 tokens, a warp each, 11.1).
//
// The angle: pos f_i in radians loses its fraction in 32 bits (at a million tokens the error is 0.03). Each
// f_i / 2 pi is kept as a 64-bit fraction of a turn, from a product in 64-bit floating point (error 2^-53 of
// it); pos times that, modulo 2^64, is exact, and its upper half is the angle as a signed 32-bit fraction of a
// turn. That fraction's error is 2^-32 of a turn and what 2^-53 of f_i becomes over pos steps (2^-31 together at a
// million, 2^-22 at the last position, 2^31), for one integer multiplication and no range reduction. As radians in 32-bit floating
// point, in [-pi, pi], it is off by up to 2^-24.3 of a turn (near half a turn, over all fractions; 2^-21.6 in radians), and
// sine and cosine are the hardware's (2^-20.9): together less than 2^-20, which a BF16 result does not show.
//
// What stays empty: a pass is eight heads of one token, and whole tokens are dealt to 2432 warps. With head counts that are no
// multiple of eight places are idle (60000 tokens of 24 heads, values included, 124 us for 109 at a copy's rate; of 10 heads
// 81 for 45, of 3, 4 and 8 heads 51 for 14, 18 and 36), and the last round of tokens is (2432 tokens of 48 heads 11.5 us, 2433
// 14.8, 5000 27, 12000 50 for 44).
#include <algorithm>

#include "kda_dependent.cuh"
#include "kda_internal.cuh"
#include "kda_mma.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtas = 2;   // on an SM
constexpr int kLoads = 2;  // heads of a lane at a time
constexpr int kHeads = 4 * kLoads;  // of a warp at a time
enum Layout { kNone, kHalves, kInterleaved };

struct Args {
    QkRopeArgs p;
    int32_t heads;   // of a token: queries, keys, and values where they go to the cache
    int32_t split;   // warps of a token
};

__device__ __forceinline__ void unpack(const uint4 &u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}
__device__ __forceinline__ uint4 pack(const float *x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

template <int kLayout>
__global__ void __launch_bounds__(kThreads, kCtas) kda_qk_rope_kernel(const Args a) {
    __shared__ uint64_t s_turn[kHeadDim / 2];                     // f_i as a fraction of a turn
    __shared__ __align__(16) float s_weight[2][kHeadDim];         // of queries, of keys
    const QkRopeArgs &p = a.p;
    const int lane = threadIdx.x & 31, sub = lane >> 3, l = lane & 7, pairs = p.rot >> 1;
    const bool norms = p.q_weight != nullptr || p.k_weight != nullptr;
    wait_for_prior();
    allow_next();
    if (norms) {
        const int which = threadIdx.x >> 7, c = threadIdx.x & 127;
        const void *const w = which == 0 ? p.q_weight : p.k_weight;
        if (w) s_weight[which][c] = p.weight_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[c]) : static_cast<const float *>(w)[c];
    }
    if (kLayout != kNone && threadIdx.x < pairs) {
        double turns = (double)p.inv_freq[threadIdx.x] * 0.15915494309189533577;  // 1 / (2 pi)
        turns -= floor(turns);
        s_turn[threadIdx.x] = turns < 1.0 ? (uint64_t)(turns * 18446744073709551616.0) : 0;
    }
    const int64_t worker = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t first = worker / a.split, workers = (int64_t)gridDim.x * kWarps / a.split;
    const int part = (int)(worker - first * a.split);
    // this lane's two pieces of eight channels, as numbers of 16 bytes; which of them turn
    const int n = p.rot >> 4;  // (halves) lanes with pairs
    const int pa = kLayout != kHalves || l < n ? l : n + l, pb = kLayout != kHalves ? 8 + l : l < n ? n + l : 8 + l;
    const bool turn_a = kLayout == kHalves ? l < n : 8 * pa < p.rot, turn_b = kLayout == kHalves ? l < n : 8 * pb < p.rot;

    auto load = [&](uint4 (&raw)[kLoads][2], int64_t t, int h0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int h = h0 + 4 * i + sub, hk = h - p.num_q_heads, hv = hk - p.num_kv_heads;
            const __nv_bfloat16 *src = p.q + t * p.q_stride + (int64_t)h * kHeadDim;
            if (hk >= 0) src = p.k + t * p.k_stride + (int64_t)hk * kHeadDim;
            if (hv >= 0) src = p.v + t * p.v_stride + (int64_t)hv * kHeadDim;
            raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
            if (h < a.heads) {
                raw[i][0] = reinterpret_cast<const uint4 *>(src)[pa];
                raw[i][1] = reinterpret_cast<const uint4 *>(src)[pb];
            }
        }
    };
    uint4 raw[kLoads][2], ahead[kLoads][2];
    int64_t t = first, slot_ahead = -1;
    int h0 = part * kHeads, pos_ahead = 0;
    auto place = [&](int64_t t) {
        if (p.slots) slot_ahead = p.slots[t];
        if (kLayout != kNone) pos_ahead = p.positions[t];
    };
    const bool idle = h0 >= a.heads || t >= p.tokens;
    if (!idle) {
        load(ahead, t, h0);
        place(t);
    }
    __syncthreads();
    if (idle) return;
    float cs[8], sn[8], w[16];
    int w_of = -1;  // what w holds
    int64_t slot = -1;
    while (t < p.tokens) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) raw[i][0] = ahead[i][0], raw[i][1] = ahead[i][1];
        if (h0 == part * kHeads) {  // a new token
            slot = slot_ahead;
            if (slot >= p.num_pages << p.page_shift) {
                if (p.slots && lane == 0) report_error(p.status, KDA_ERR_DEVICE_INPUT, (int32_t)t);
                slot = -1;
            }
            // halves: of pairs 8 l .. 8 l + 7; interleaved: of the four pairs in either piece
#pragma unroll
            for (int i = 0; kLayout != kNone && i < 8; ++i) {
                const int pair = kLayout == kHalves ? 8 * l + i : 4 * (i < 4 ? pa : pb) + (i & 3);
                const uint64_t turn = (uint64_t)(int64_t)pos_ahead * s_turn[pair & (kHeadDim / 2 - 1)];
                __sincosf((float)(int32_t)(turn >> 32) * 1.4629180792671596e-9f, &sn[i], &cs[i]);  // 2 pi / 2^32
                sn[i] *= p.magnitude;
                cs[i] *= p.magnitude;
            }
        }
        int next_h = h0 + a.split * kHeads;
        int64_t next_t = t;
        if (next_h >= a.heads) next_h = part * kHeads, next_t += workers;
        if (next_t < p.tokens) {
            load(ahead, next_t, next_h);
            if (next_t != t) place(next_t);
        }
        const int64_t page = slot >> p.page_shift, in_page = slot & ((1 << p.page_shift) - 1);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int h = h0 + 4 * i + sub, hk = h - p.num_q_heads, hv = hk - p.num_kv_heads;
            const bool is_q = hk < 0;
            float x[16];
            unpack(raw[i][0], x);
            unpack(raw[i][1], x + 8);
            if (norms) {
                float sum[2] = {0.0f, 0.0f};
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[e & 1] = fmaf(x[e], x[e], sum[e & 1]);
                sum[0] += sum[1];
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
                const float r = rsqrtf(fmaf(sum[0], 1.0f / kHeadDim, p.eps));
                if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
                    if (w_of != (is_q ? 0 : 1)) {
                        w_of = is_q ? 0 : 1;
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<float4 *>(w + e) = *reinterpret_cast<const float4 *>(&s_weight[w_of][8 * (e < 8 ? pa : pb) + (e & 7)]);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] *= r * w[e];
                }
            }
            if (kLayout == kHalves) {
                if (turn_a) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float u = x[e], v = x[8 + e];
                        x[e] = fmaf(u, cs[e], -v * sn[e]);
                        x[8 + e] = fmaf(v, cs[e], u * sn[e]);
                    }
                }
            } else if (kLayout == kInterleaved) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (!(e < 4 ? turn_a : turn_b)) continue;
                    const float u = x[2 * e], v = x[2 * e + 1];
                    x[2 * e] = fmaf(u, cs[e], -v * sn[e]);
                    x[2 * e + 1] = fmaf(v, cs[e], u * sn[e]);
                }
            }
            const uint4 ya = hv < 0 ? pack(x) : raw[i][0], yb = hv < 0 ? pack(x + 8) : raw[i][1];
            auto store = [&](__nv_bfloat16 *dst) {
                reinterpret_cast<uint4 *>(dst)[pa] = ya;
                reinterpret_cast<uint4 *>(dst)[pb] = yb;
            };
            if (is_q) {
                store(p.q_out + t * p.q_out_stride + (int64_t)h * kHeadDim);
            } else if (hv < 0) {
                if (p.k_out) store(p.k_out + t * p.k_out_stride + (int64_t)hk * kHeadDim);
                if (slot >= 0) store(p.k_cache + page * p.k_page_stride + (((int64_t)hk << p.page_shift) + in_page) * kHeadDim);
            } else if (h < a.heads && slot >= 0) {
                store(p.v_cache + page * p.v_page_stride + (((int64_t)hv << p.page_shift) + in_page) * kHeadDim);
            }
        }
        t = next_t;
        h0 = next_h;
    }
}

}  // namespace

cudaError_t launch_qk_rope(const QkRopeArgs &p, cudaStream_t stream) {
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    Args a;
    a.p = p;
    a.heads = p.num_q_heads + p.num_kv_heads * (p.slots ? 2 : 1);
    // Tokens that fill the GPU's warps (kCtas CTAs an SM) have a warp each; fewer are shared between warps.
    const int64_t warps = (int64_t)sms * kCtas * kWarps, most = (a.heads + kHeads - 1) / kHeads;
    a.split = (int32_t)std::max<int64_t>(1, std::min(most, warps / std::max(p.tokens, 1)));
    a.split = std::min(a.split, kWarps);
    while (kWarps % a.split != 0) ++a.split;  // (the warps of a token lie in one CTA)
    const int64_t ctas = ((int64_t)p.tokens * a.split + kWarps - 1) / kWarps;
    const dim3 grid((unsigned)std::min<int64_t>(ctas, (int64_t)sms * kCtas));
    if (p.rot == 0) return launch_dependent(kda_qk_rope_kernel<kNone>, grid, kThreads, 0, stream, a);
    if (p.interleaved) return launch_dependent(kda_qk_rope_kernel<kInterleaved>, grid, kThreads, 0, stream, a);
    return launch_dependent(kda_qk_rope_kernel<kHalves>, grid, kThreads, 0, stream, a);
}

}  // namespace kda
