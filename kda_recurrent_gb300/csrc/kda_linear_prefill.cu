// Linear attention with a decay for each head, prompt form (sm_103a).
//
//     S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
//
// Token by token: one CTA per (sequence, head) chain, thread j holding column j of the
// 128 x 128 state in registers; k and q of a token are shared through shared memory.
#include "kda_internal.cuh"

namespace kda {
namespace {

__global__ void __launch_bounds__(kHeadDim) kda_linear_prefill_kernel(const LinearPrefillArgs a) {
    __shared__ float s_k[kHeadDim], s_q[kHeadDim];
    const int h = blockIdx.x % a.num_heads, n = blockIdx.x / a.num_heads, j = threadIdx.x;
    int bos = a.cu_seqlens[n], eos = a.cu_seqlens[n + 1];
    if (bos < 0 || eos < bos || eos > a.total_tokens) {
        if (j == 0 && h == 0) report_error(a.status, KDA_ERR_DEVICE_INPUT, n);
        bos = min(max(bos, 0), a.total_tokens);
        eos = min(max(eos, bos), a.total_tokens);
    }
    const size_t base = (size_t)blockIdx.x * kHeadDim * kHeadDim + j;
    float S[kHeadDim];
#pragma unroll
    for (int i = 0; i < kHeadDim; ++i) S[i] = a.init_state ? a.init_state[base + i * kHeadDim] : 0.0f;
    for (int t = bos; t < eos; ++t) {
        const size_t at = ((size_t)t * a.num_heads + h) * kHeadDim + j;
        __syncthreads();
        s_k[j] = __bfloat162float(a.k[at]);
        s_q[j] = __bfloat162float(a.q[at]);
        const float v = __bfloat162float(a.v[at]);
        const float decay = expf(a.log_decay[(size_t)t * a.decay_token_stride + h]);
        __syncthreads();
        float o = 0.0f;
#pragma unroll
        for (int i = 0; i < kHeadDim; ++i) {
            S[i] = fmaf(S[i], decay, s_k[i] * v);
            o = fmaf(s_q[i], S[i], o);
        }
        a.out[at] = __float2bfloat16_rn(a.scale * o);
    }
    if (a.final_state)
#pragma unroll
        for (int i = 0; i < kHeadDim; ++i) a.final_state[base + i * kHeadDim] = S[i];
}

}  // namespace

int64_t linear_prefill_workspace_bytes(int32_t, int32_t, int32_t, int32_t) { return 0; }

cudaError_t launch_linear_prefill(const LinearPrefillArgs &a, cudaStream_t stream) {
    kda_linear_prefill_kernel<<<(unsigned)a.num_seqs * (unsigned)a.num_heads, kHeadDim, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
