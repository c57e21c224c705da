// Attention of one new token over a paged key-value cache (sm_103a).
//
//     x_j = scale q . k_j,  p = softmax(x),  o = sum_j p_j v_j
//
// One CTA per (row, query head): its warps take every fourth cached token each, keeping a
// running maximum m, sum l = sum e^{x - m} and o; the warps' parts are joined at the end. The
// weights need the final sum, so a second kernel forms them once lse is known.
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4;
constexpr float kNegInf = -INFINITY;

// Page of token j of row b, or -1 (missing). A bad table entry is recorded.
__device__ __forceinline__ int page_of(const PagedCache &c, int b, int j, DeviceStatus *st) {
    const int page = c.block_table[(size_t)b * c.max_pages + (j >> c.page_shift)];
    if (page >= c.num_pages) {
        report_error(st, KDA_ERR_DEVICE_INPUT, b);
        return -1;
    }
    return page;
}

__device__ __forceinline__ size_t row_offset(const PagedCache &c, int64_t page_stride, int page, int h, int j) {
    return (size_t)page * page_stride + ((size_t)h * c.page_size + (j & (c.page_size - 1))) * kHeadDim;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void load4(const __nv_bfloat16 *p, float (&x)[4]) {
    const uint2 w = *reinterpret_cast<const uint2 *>(p);
    x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xffff0000u);
    x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xffff0000u);
}

__device__ __forceinline__ float score(const AttnDecodeArgs &a, const float (&q)[4], int page, int h, int j, int lane) {
    float k[4];
    load4(a.c.k + row_offset(a.c, a.c.k_page_stride, page, h, j) + 4 * lane, k);
    return a.scale * warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]);
}

__global__ void __launch_bounds__(kWarps * 32) kda_attn_decode_kernel(const AttnDecodeArgs a, float *lse) {
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kHeadDim];
    const int b = blockIdx.x / a.num_q_heads, hq = blockIdx.x - b * a.num_q_heads, h = hq / a.group;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = row_length(a.c, b, a.status, threadIdx.x == 0 && hq == 0);
    float q[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, m = kNegInf, l = 0.0f;
    load4(a.q + (size_t)blockIdx.x * kHeadDim + 4 * lane, q);
    for (int j = warp; j < n; j += kWarps) {
        const int page = page_of(a.c, b, j, a.status);
        if (page < 0) continue;
        const float x = score(a, q, page, h, j, lane);
        const float top = fmaxf(m, x);
        const float ref = top == kNegInf ? 0.0f : top;
        const float keep = expf(m - ref), p = expf(x - ref);
        float v[4];
        load4(a.c.v + row_offset(a.c, a.c.v_page_stride, page, h, j) + 4 * lane, v);
        l = fmaf(l, keep, p);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(o[e], keep, p * v[e]);
        m = top;
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int e = 0; e < 4; ++e) s_o[warp][4 * lane + e] = o[e];
    __syncthreads();
    float top = kNegInf, sum = 0.0f, out = 0.0f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    const float ref = top == kNegInf ? 0.0f : top;
    for (int w = 0; w < kWarps; ++w) {
        const float f = expf(s_m[w] - ref);
        sum = fmaf(s_l[w], f, sum);
        out = fmaf(s_o[w][threadIdx.x], f, out);
    }
    a.out[(size_t)blockIdx.x * kHeadDim + threadIdx.x] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : out / sum);
    if (threadIdx.x == 0) {
        const float v = sum == 0.0f ? kNegInf : ref + logf(sum);
        lse[blockIdx.x] = v;
        if (a.lse) a.lse[blockIdx.x] = v;
    }
}

// weight[b][h][j] += sum over the group's query heads of exp(x_j - lse): one warp per token.
__global__ void __launch_bounds__(kWarps * 32) kda_attn_weight_kernel(const AttnDecodeArgs a, const float *lse) {
    const int b = blockIdx.x / a.c.num_kv_heads, h = blockIdx.x - b * a.c.num_kv_heads;
    const int lane = threadIdx.x & 31;
    const int n = row_length(a.c, b, a.status, false);
    for (int j = blockIdx.y * kWarps + (threadIdx.x >> 5); j < n; j += gridDim.y * kWarps) {
        const int page = page_of(a.c, b, j, a.status);
        if (page < 0) continue;
        float sum = 0.0f;
        for (int g = 0; g < a.group; ++g) {
            const size_t row = (size_t)b * a.num_q_heads + h * a.group + g;
            float q[4];
            load4(a.q + row * kHeadDim + 4 * lane, q);
            const float x = score(a, q, page, h, j, lane);
            sum += lse[row] == kNegInf ? 0.0f : expf(x - lse[row]);
        }
        if (lane == 0) a.weight[(size_t)blockIdx.x * a.c.capacity + j] += sum;
    }
}

}  // namespace

int64_t attn_decode_workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t, int64_t, bool, int32_t) {
    return ((int64_t)batch * num_q_heads * 4 + 15) / 16 * 16;
}

cudaError_t launch_attn_decode(const AttnDecodeArgs &a, cudaStream_t stream) {
    float *lse = static_cast<float *>(a.ws);
    kda_attn_decode_kernel<<<(unsigned)a.c.batch * (unsigned)a.num_q_heads, kWarps * 32, 0, stream>>>(a, lse);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !a.weight) return e;
    const unsigned parts = (unsigned)((a.c.capacity + 255) / 256);
    const dim3 grid((unsigned)(a.c.batch * a.c.num_kv_heads), parts < 1024u ? parts : 1024u);
    kda_attn_weight_kernel<<<grid, kWarps * 32, 0, stream>>>(a, lse);
    return cudaGetLastError();
}

}  // namespace kda
