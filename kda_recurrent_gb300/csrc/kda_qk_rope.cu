// Queries and keys on their way into attention (sm_103a): the norm of each head, the rotation by position, and
// the write of keys and values into the pages of the key-value cache, in one pass.
//
//     y = x (mean x^2 + eps)^-1/2 w                      (where a weight is given)
//     (a, b) -> m (a cos - b sin, b cos + a sin)         for the pairs of the first `rot` channels, angle pos f_i
//
// Every number is read once and written once, so the kernel is a stream: a half-warp holds a head (16 bytes a
// lane), a warp eight heads at a time with all loads before any arithmetic. With many tokens a warp walks all
// heads of a token, so that its angles are computed once; with few, a token's heads are shared between warps.
//
// The angle: pos f_i in radians loses its fraction in 32 bits (at a million tokens the error is 0.03). Each
// f_i / 2 pi is kept as a 64-bit fraction of a turn, from a product in 64-bit floating point (error 2^-53 of
// it); pos times that, modulo 2^64, is exact, and its upper half is the angle as a signed 32-bit fraction of a
// turn. So the angle's error is 2^-32 of a turn and what 2^-53 of f_i becomes over pos steps (2^-31 at a
// million), for one integer multiplication and no range reduction; sine and cosine of an angle in [-pi, pi] are
// the hardware's (2^-20.9), which a BF16 result does not show.
#include <algorithm>

#include "kda_dependent.cuh"
#include "kda_internal.cuh"
#include "kda_mma.cuh"

namespace kda {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtas = 2;            // on an SM
constexpr int kLoads = 4;           // of a lane at a time
constexpr int kHeads = 2 * kLoads;  // of a warp at a time
enum Layout { kNone, kHalves, kInterleaved };

struct Args {
    QkRopeArgs p;
    int32_t heads;   // of a token: queries, keys, and values where they go to the cache
    int32_t split;   // warps of a token
};

__device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

__device__ __forceinline__ void load_weight(const QkRopeArgs &p, const void *w, int chunk, float (&x)[8]) {
    if (!w) return;
    if (p.weight_bf16) {
        unpack(__ldg(static_cast<const uint4 *>(w) + chunk), x);
    } else {
        const float4 a = __ldg(static_cast<const float4 *>(w) + 2 * chunk), b = __ldg(static_cast<const float4 *>(w) + 2 * chunk + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

template <int kLayout>
__global__ void __launch_bounds__(kThreads, kCtas) kda_qk_rope_kernel(const Args a) {
    __shared__ uint64_t s_turn[kHeadDim / 2];  // f_i as a fraction of a turn
    const QkRopeArgs &p = a.p;
    const int lane = threadIdx.x & 31, sub = lane >> 4, chunk = lane & 15, pairs = p.rot >> 1;
    wait_for_prior();
    allow_next();
    if (kLayout != kNone) {
        if (threadIdx.x < pairs) {
            double turns = (double)__ldg(p.inv_freq + threadIdx.x) * 0.15915494309189533577;  // 1 / (2 pi)
            turns -= floor(turns);
            s_turn[threadIdx.x] = turns < 1.0 ? (uint64_t)(turns * 18446744073709551616.0) : 0;
        }
        __syncthreads();
    }
    const int64_t worker = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t first = worker / a.split, workers = (int64_t)gridDim.x * kWarps / a.split;
    const int part = (int)(worker - first * a.split);
    float wq[8], wk[8];
    load_weight(p, p.q_weight, chunk, wq);
    load_weight(p, p.k_weight, chunk, wk);
    // whether this lane's channels turn, and the lane with their partners
    const bool turned = kLayout != kNone && 8 * chunk < p.rot;
    const int reach = p.rot >> 4, partner = !turned ? lane : chunk < reach ? lane + reach : lane - reach;
    constexpr int kAngles = kLayout == kInterleaved ? 4 : 8;
    const int angle0 = kLayout == kInterleaved ? 4 * chunk : chunk < reach ? 8 * chunk : 8 * (chunk - reach);
    const float side = kLayout == kHalves && chunk < reach ? -p.magnitude : p.magnitude;

    auto load = [&](uint4 (&raw)[kLoads], int64_t t, int h0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int h = h0 + 2 * i + sub, hk = h - p.num_q_heads, hv = hk - p.num_kv_heads;
            const __nv_bfloat16 *src = p.q + t * p.q_stride + (int64_t)h * kHeadDim;
            if (hk >= 0) src = p.k + t * p.k_stride + (int64_t)hk * kHeadDim;
            if (hv >= 0) src = p.v + t * p.v_stride + (int64_t)hv * kHeadDim;
            raw[i] = make_uint4(0, 0, 0, 0);
            if (h < a.heads) raw[i] = *(reinterpret_cast<const uint4 *>(src) + chunk);
        }
    };
    // the next eight heads (and the next token's place) are on their way while these are computed
    uint4 raw[kLoads], ahead[kLoads];
    int64_t t = first, slot_ahead = -1;
    int h0 = part * kHeads, pos_ahead = 0;
    auto place = [&](int64_t t) {
        if (p.slots) slot_ahead = __ldg(p.slots + t);
        if (kLayout != kNone) pos_ahead = __ldg(p.positions + t);
    };
    if (h0 >= a.heads || t >= p.tokens) return;
    load(ahead, t, h0);
    place(t);
    float cs[kAngles], sn[kAngles];
    int64_t slot = -1;
    while (t < p.tokens) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) raw[i] = ahead[i];
        if (h0 == part * kHeads) {  // a new token
            slot = slot_ahead;
            if (slot >= p.num_pages << p.page_shift) {
                if (p.slots && lane == 0) report_error(p.status, KDA_ERR_DEVICE_INPUT, (int32_t)t);
                slot = -1;
            }
#pragma unroll
            for (int i = 0; kLayout != kNone && i < kAngles; ++i) {
                const uint64_t turn = (uint64_t)(int64_t)pos_ahead * s_turn[(angle0 + i) & (kHeadDim / 2 - 1)];
                __sincosf((float)(int32_t)(turn >> 32) * 1.4629180792671596e-9f, &sn[i], &cs[i]);  // 2 pi / 2^32
                sn[i] *= side;
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
            const int h = h0 + 2 * i + sub, hk = h - p.num_q_heads, hv = hk - p.num_kv_heads;
            uint4 y = raw[i];
            float x[8];
            unpack(y, x);
            const bool is_q = hk < 0;
            if (p.q_weight || p.k_weight) {
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float r = rsqrtf(fmaf(sum, 1.0f / kHeadDim, p.eps));
                if (is_q ? p.q_weight != nullptr : p.k_weight != nullptr) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= r * (is_q ? wq[e] : wk[e]);
                }
            }
            if (kLayout == kHalves) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float other = __shfl_sync(0xffffffffu, x[e], partner);
                    if (turned) x[e] = fmaf(x[e], cs[e], other * sn[e]);
                }
            } else if (kLayout == kInterleaved) {
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float b = x[2 * e + 1];
                        x[2 * e + 1] = fmaf(b, cs[e], x[2 * e] * sn[e]);
                        x[2 * e] = fmaf(x[2 * e], cs[e], -b * sn[e]);
                    }
                }
            }
            if (hv < 0) y = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
            if (is_q) {
                reinterpret_cast<uint4 *>(p.q_out + t * p.q_out_stride + (int64_t)h * kHeadDim)[chunk] = y;
            } else if (hv < 0) {
                if (p.k_out) reinterpret_cast<uint4 *>(p.k_out + t * p.k_out_stride + (int64_t)hk * kHeadDim)[chunk] = y;
                if (slot >= 0)
                    reinterpret_cast<uint4 *>(p.k_cache + page * p.k_page_stride + (((int64_t)hk << p.page_shift) + in_page) * kHeadDim)[chunk] = y;
            } else if (h < a.heads && slot >= 0) {
                reinterpret_cast<uint4 *>(p.v_cache + page * p.v_page_stride + (((int64_t)hv << p.page_shift) + in_page) * kHeadDim)[chunk] = y;
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
