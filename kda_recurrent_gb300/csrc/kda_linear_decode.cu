// Linear attention with a decay for each head, single-token form on a slot pool (sm_103a).
//
//     S <- exp(g) S + k v^T,   o = scale S^T q      for every (row, head), in place
//
// The state is the whole cost: 64 KiB (FP32) or 32 KiB (BF16) read and written per item, so this
// is an HBM stream. A CTA owns a block of columns of one item's state (columns are independent), 128 or 256
// bytes of every row; a thread owns 16 bytes of every kRows-th row, issues all its loads before any
// arithmetic, and sums its rows' share of the outputs, which are joined by shuffles and through shared
// memory in a fixed order. 4096 rows of 8 heads, FP32: 621 us, 6.95 TB/s (a copy reaches 6.78); 333 rows of 32
// heads, BF16: 104 us, 6.80 TB/s; one row of 8 heads: 1.7 us, a launch's latency and two dependent loads.
#include "kda_dependent.cuh"
#include "kda_internal.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int kElems = 4;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int kElems = 8;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&x)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

template <typename T, int kSegment>
__global__ void __launch_bounds__(kThreads) kda_linear_decode_kernel(const LinearDecodeArgs a) {
    using V = Vec<T>;
    constexpr int E = V::kElems;
    constexpr int kCols = kSegment / 16;      // threads across a row
    constexpr int kWidth = kCols * E;         // columns
    constexpr int kRows = kThreads / kCols;   // rows in flight
    constexpr int kPasses = kHeadDim / kRows;
    constexpr int kBlocks = kHeadDim / kWidth;
    __shared__ float s_q[kHeadDim], s_k[kHeadDim], s_o[kThreads / 32][kWidth];
    const int item = blockIdx.x / kBlocks, j0 = (blockIdx.x - item * kBlocks) * kWidth;
    const int r = item / a.num_heads, h = item - r * a.num_heads;
    const int tid = threadIdx.x;
    const size_t tok = (size_t)item * kHeadDim;
    wait_for_prior();
    allow_next();
    const int32_t slot = a.slot_idx[r];
    if (slot < 0 || slot >= a.num_slots) {
        if (slot >= 0 && tid == 0 && h == 0 && j0 == 0) report_error(a.status, KDA_ERR_DEVICE_INPUT, r);
        if (tid < kWidth) a.out[tok + j0 + tid] = __float2bfloat16_rn(0.0f);
        return;
    }
    const int cg = tid % kCols, rg = tid / kCols;
    uint4 *const S = reinterpret_cast<uint4 *>(static_cast<T *>(a.state_pool) +
                                               ((size_t)slot * a.num_heads + h) * (kHeadDim * kHeadDim) + rg * kHeadDim + j0) + cg;
    constexpr int kStride = kRows * kHeadDim / E;  // from a thread's row to its next
    uint4 w[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) w[i] = __ldcs(S + i * kStride);
    if (tid < kHeadDim) {
        s_q[tid] = __bfloat162float(a.q[tok + tid]);
        s_k[tid] = __bfloat162float(a.k[tok + tid]);
    }
    float v[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __bfloat162float(a.v[tok + j0 + cg * E + e]), o[e] = 0.0f;
    const float decay = expf(a.log_decay[(size_t)r * a.decay_row_stride + h]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const float q = s_q[rg + i * kRows], k = s_k[rg + i * kRows];
        float x[E];
        V::unpack(w[i], x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = fmaf(x[e], decay, k * v[e]);
            o[e] = fmaf(q, x[e], o[e]);
        }
        __stcs(S + i * kStride, V::pack(x));
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
        for (int x = kCols; x < 32; x <<= 1) o[e] += __shfl_xor_sync(0xffffffffu, o[e], x);
        if ((tid & 31) < kCols) s_o[tid >> 5][cg * E + e] = o[e];
    }
    __syncthreads();
    if (tid < kWidth) {
        float sum = 0.0f;
#pragma unroll
        for (int g = 0; g < kThreads / 32; ++g) sum += s_o[g][tid];
        a.out[tok + j0 + tid] = __float2bfloat16_rn(a.scale * sum);
    }
}

// Segments of 256 bytes stream best; few items spread over more CTAs with 128. In us with 128 and 256 (and
// with 512) bytes a row: FP32 32 items 2.15, 2.26 (2.80), 255 items 6.69, 6.68 (6.57), 32768 items 637, 621
// (622); BF16 32 items 1.79, 2.09, 512 items 7.41, 7.46, 700 items 9.26, 8.86, 32768 items 361, 319.
constexpr int64_t kWideBytes = 20 << 20;  // of states

template <typename T, int kSegment>
cudaError_t launch_t(const LinearDecodeArgs &a, cudaStream_t stream) {
    const int64_t ctas = (int64_t)a.rows * a.num_heads * (kHeadDim * (int64_t)sizeof(T) / kSegment);
    return launch_dependent(kda_linear_decode_kernel<T, kSegment>, dim3((unsigned)ctas), kThreads, 0, stream, a);
}

template <typename T>
cudaError_t launch_t(const LinearDecodeArgs &a, cudaStream_t stream) {
    const int64_t bytes = (int64_t)a.rows * a.num_heads * (kHeadDim * kHeadDim * (int64_t)sizeof(T));
    return bytes < kWideBytes ? launch_t<T, 128>(a, stream) : launch_t<T, 256>(a, stream);
}

}  // namespace

cudaError_t launch_linear_decode(const LinearDecodeArgs &a, cudaStream_t stream) {
    return a.state_dtype == KDA_STATE_F32 ? launch_t<float>(a, stream) : launch_t<__nv_bfloat16>(a, stream);
}

}  // namespace kda
