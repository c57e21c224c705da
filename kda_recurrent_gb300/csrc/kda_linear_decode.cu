// Linear attention with a decay for each head, single-token form on a slot pool (sm_103a).
//
//     S <- exp(g) S + k v^T,   o = scale S^T q      for every (row, head), in place
//
// The state is the whole cost: 64 KiB (FP32) or 32 KiB (BF16) read and written per item. One
// CTA per item; thread (r, c) owns 16 bytes of columns (c) of every kRows-th row of the state
// and sums its rows' share of the outputs, which are joined through shared memory.
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

template <typename T>
__global__ void __launch_bounds__(kThreads) kda_linear_decode_kernel(const LinearDecodeArgs a) {
    using V = Vec<T>;
    constexpr int E = V::kElems;
    constexpr int kCols = kHeadDim / E;       // threads across a row
    constexpr int kRows = kThreads / kCols;   // rows in flight
    __shared__ float s_q[kHeadDim], s_k[kHeadDim], s_o[kRows][kHeadDim];
    const int item = blockIdx.x, r = item / a.num_heads, h = item - r * a.num_heads;
    const int tid = threadIdx.x;
    const size_t tok = (size_t)item * kHeadDim;
    const int32_t slot = a.slot_idx[r];
    if (slot < 0 || slot >= a.num_slots) {
        if (slot >= 0 && tid == 0) report_error(a.status, KDA_ERR_DEVICE_INPUT, r);
        if (tid < kHeadDim) a.out[tok + tid] = __float2bfloat16_rn(0.0f);
        return;
    }
    if (tid < kHeadDim) {
        s_q[tid] = __bfloat162float(a.q[tok + tid]);
        s_k[tid] = __bfloat162float(a.k[tok + tid]);
    }
    __syncthreads();
    const float decay = expf(a.log_decay[(size_t)r * a.decay_row_stride + h]);
    const int cg = tid % kCols, rg = tid / kCols;
    T *const S = static_cast<T *>(a.state_pool) + ((size_t)slot * a.num_heads + h) * (kHeadDim * kHeadDim);
    float v[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = __bfloat162float(a.v[tok + cg * E + e]), o[e] = 0.0f;
    for (int i = rg; i < kHeadDim; i += kRows) {
        uint4 *const at = reinterpret_cast<uint4 *>(S + i * kHeadDim + cg * E);
        float x[E];
        V::unpack(*at, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = fmaf(x[e], decay, s_k[i] * v[e]);
            o[e] = fmaf(s_q[i], x[e], o[e]);
        }
        *at = V::pack(x);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[rg][cg * E + e] = o[e];
    __syncthreads();
    if (tid < kHeadDim) {
        float sum = 0.0f;
        for (int g = 0; g < kRows; ++g) sum += s_o[g][tid];
        a.out[tok + tid] = __float2bfloat16_rn(a.scale * sum);
    }
}

}  // namespace

cudaError_t launch_linear_decode(const LinearDecodeArgs &a, cudaStream_t stream) {
    const unsigned items = (unsigned)a.rows * (unsigned)a.num_heads;
    if (a.state_dtype == KDA_STATE_F32)
        kda_linear_decode_kernel<float><<<items, kThreads, 0, stream>>>(a);
    else
        kda_linear_decode_kernel<__nv_bfloat16><<<items, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
