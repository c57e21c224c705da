// Attention of one new token over a paged key-value cache (sm_103a): the launches of the token stream
// (kda_attn_stream.cuh) for whole rows, the join of items that were cut between shares, and the weights.
#include <algorithm>

#include "kda_attn_stream.cuh"
#include "kda_dependent.cuh"
#include "kda_internal.cuh"
#include "kda_mma.cuh"

namespace kda {

using namespace stream;

namespace {

template <typename U>
__global__ void __launch_bounds__(kThreads, 1) kda_attn_decode_kernel(const Args a) {
    extern __shared__ __align__(128) uint8_t smem[];
    wait_for_prior();
    allow_next();
    walk_share<U>(a, blockIdx.x, gridDim.x, smem, NoStarts(), [] { __syncthreads(); });
}

// Adds parts i, i + step, ... of row `row` to (m, l, o), four loads in flight (eight take registers that would
// leave an SM half the CTAs: 128 rows of 100 tokens 15.6 us instead of 14.6).
__device__ __forceinline__ void add_parts(const Part *parts, const Cut &cut, int row, int lane, int i, int step, float &m, float &l,
                                          float4 &o) {
    const int n = cut.count;
    constexpr int kAhead = 4;
    for (; i < n; i += kAhead * step) {
        float pm[kAhead], pl[kAhead];
        float4 po[kAhead];
        float top = m;
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const int x = i + e * step;
            pm[e] = kNegInf, pl[e] = 0.0f, po[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (x < n) {
                const Part *const part = parts + cut.part_at(x);
                pm[e] = part->m[row], pl[e] = part->l[row];
                po[e] = *reinterpret_cast<const float4 *>(&part->o[row][4 * lane]);
            }
        }
#pragma unroll
        for (int e = 0; e < kAhead; ++e) top = fmaxf(top, pm[e]);
        const float ref = top == kNegInf ? 0.0f : top, keep = ex2(m - ref);
        l *= keep;
        o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
        for (int e = 0; e < kAhead; ++e) {
            const float f = ex2(pm[e] - ref);
            l = fmaf(pl[e], f, l);
            o = make_float4(fmaf(po[e].x, f, o.x), fmaf(po[e].y, f, o.y), fmaf(po[e].z, f, o.z), fmaf(po[e].w, f, o.w));
        }
        m = top;
    }
}

// Joins the cut items: CTA (i, row) those of the eight shares of the first kernel's CTA i, a warp for each, or
// all warps for an item of more parts than a CTA has shares (it reaches beyond the CTA, so there is one at most).
// 8 x 8000 tokens: 12.0 us, with one warp for up to 64 parts 14.4; 1 x 100000 tokens: 18, with one warp 31.
constexpr int kManyParts = kWarps;

__global__ void __launch_bounds__(kThreads, 4) kda_attn_join_kernel(const Args a) {
    __shared__ float s_m[kWarps], s_l[kWarps];
    __shared__ float4 s_o[kWarps][32];
    __shared__ Cut s_cut;
    __shared__ int s_many;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y;
    if (threadIdx.x == 0) s_many = 0;
    allow_next();
    wait_for_prior();
    const Cut cut = a.ws.cuts[blockIdx.x * kWarps + warp];
    __syncthreads();
    if (cut.count > 0 && row < cut.rows) {
        if (cut.count > kManyParts) {
            if (lane == 0) s_cut = cut, s_many = 1;
        } else {
            float m = kNegInf, l = 0.0f;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            add_parts(a.ws.parts, cut, row, lane, 0, 1, m, l, o);
            write_row<false>(a, (size_t)cut.head + row, lane, m, l, o);
        }
    }
    __syncthreads();
    if (!s_many) return;
    float m = kNegInf, l = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    add_parts(a.ws.parts, s_cut, row, lane, warp, kWarps, m, l, o);
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
    s_o[warp][lane] = o;
    __syncthreads();
    if (warp > 0) return;
    m = kNegInf, l = 0.0f;
    o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, s_m[w]);
    const float ref = m == kNegInf ? 0.0f : m;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w] - ref);
        const float4 x = s_o[w][lane];
        l = fmaf(s_l[w], f, l);
        o = make_float4(fmaf(x.x, f, o.x), fmaf(x.y, f, o.y), fmaf(x.z, f, o.z), fmaf(x.w, f, o.w));
    }
    write_row<false>(a, (size_t)s_cut.head + row, lane, m, l, o);
}

// weight[b][h][j] += sum over the query heads of key head h of 2^(x_j - lse), four tokens a thread. A score of
// -inf has no weight whatever the lse (which a NaN key elsewhere in the row makes NaN). Tokens of a missing page
// are not written: a page holds whole groups of four, so those are the groups that have no other score. The grid
// covers the table's width, which is what the host knows; CTAs past their row's length leave at once.
constexpr int kWeightThreads = 256, kWeightTokens = 4 * kWeightThreads;

__global__ void __launch_bounds__(kWeightThreads) kda_attn_weight_kernel(const Args a) {
    const AttnDecodeArgs &p = a.p;
    const int bh = blockIdx.x, b = bh / p.c.num_kv_heads;
    allow_next();
    wait_for_prior();
    const int n = row_length(p.c, b, p.status, false);
    const size_t head0 = (size_t)bh * p.group;
    constexpr int kAhead = 8;
    float4 x[kAhead], old;
    auto load = [&](int64_t j) {
        const float *const scores = a.ws.scores + head0 * p.c.capacity + j;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < p.group) x[i] = *reinterpret_cast<const float4 *>(scores + (size_t)i * p.c.capacity);
        old = *reinterpret_cast<const float4 *>(p.weight + (size_t)bh * p.c.capacity + j);
    };
    for (int64_t j = (int64_t)blockIdx.y * kWeightTokens + 4 * threadIdx.x; j < n; j += (int64_t)gridDim.y * kWeightTokens) {
        load(j);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        bool any = false;
        auto add = [&](const float4 &x4, int i) {
            const float lse = a.ws.lse2[head0 + i];
            auto weight = [&](float x) { return x == kNegInf ? 0.0f : ex2(x - lse); };
            any |= x4.x != kNegInf || x4.y != kNegInf || x4.z != kNegInf || x4.w != kNegInf;
            sum = make_float4(sum.x + weight(x4.x), sum.y + weight(x4.y), sum.z + weight(x4.z), sum.w + weight(x4.w));
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < p.group) add(x[i], i);
#pragma unroll 4
        for (int i = kAhead; i < p.group; ++i)
            add(*reinterpret_cast<const float4 *>(a.ws.scores + (head0 + i) * p.c.capacity + j), i);
        if (!any) continue;
        float *const w = p.weight + (size_t)bh * p.c.capacity + j;
        if (j + 4 <= n) {
            *reinterpret_cast<float4 *>(w) = make_float4(old.x + sum.x, old.y + sum.y, old.z + sum.z, old.w + sum.w);
        } else {
            const float s[4] = {old.x + sum.x, old.y + sum.y, old.z + sum.z, old.w + sum.w};
            for (int e = 0; j + e < n; ++e) w[e] = s[e];
        }
    }
}

template <typename U>
cudaError_t configure_once() {
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !configured[dev]) {
        e = cudaFuncSetAttribute(kda_attn_decode_kernel<U>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<U>);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) configured[dev] = true;
    }
    return cudaSuccess;
}

}  // namespace

int64_t attn_decode_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t, int64_t capacity, bool with_weight,
                                    int32_t sms) {
    return workspace_layout(nullptr, nullptr, batch, num_q_heads, capacity, with_weight, (int64_t)sms * kWarps);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs &p, cudaStream_t stream) {
    int32_t sms = 0;
    if (sm_count_of_current_device(&sms) != KDA_OK) return cudaErrorInvalidDevice;
    Args a;
    a.x = PrefixParts();
    const bool small = stream_args(&a, p, sms);
    cudaError_t e = small ? configure_once<uint32_t>() : configure_once<uint64_t>();
    if (e != cudaSuccess) return e;
    e = small ? launch_dependent(kda_attn_decode_kernel<uint32_t>, dim3((unsigned)sms), kThreads, kSmem<uint32_t>, stream, a)
              : launch_dependent(kda_attn_decode_kernel<uint64_t>, dim3((unsigned)sms), kThreads, kSmem<uint64_t>, stream, a);
    if (e != cudaSuccess) return e;
    e = launch_dependent(kda_attn_join_kernel, dim3((unsigned)sms, (unsigned)std::min(p.group, kRows)), kThreads, 0, stream, a);
    if (e != cudaSuccess || !p.weight) return e;
    const dim3 grid((unsigned)(p.c.batch * p.c.num_kv_heads), (unsigned)std::min((p.c.capacity + kWeightTokens - 1) / kWeightTokens, 65535));
    return launch_dependent(kda_attn_weight_kernel, grid, kWeightThreads, 0, stream, a);
}

}  // namespace kda
