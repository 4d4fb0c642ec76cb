// kda_la_prefill.cu -- linear attention with one decay per head and token,
// whole prompts (sm_103a):
//     S_t = exp(g_t) S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t.
// One CTA per (sequence, head), one thread per value row, token by token.
#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kStage = 16;

__global__ void __launch_bounds__(kHeadDim) la_recurrent_kernel(LaArgs a) {
    __shared__ float q[kStage][kHeadDim], k[kStage][kHeadDim];
    const int64_t n = blockIdx.x / a.H, h = blockIdx.x - n * a.H;
    const int64_t hk = h / (a.H / a.Hk);
    const int r = threadIdx.x;
    int64_t tok0, len;
    if (a.cu_seqlens) {
        if (!*a.valid) return;
        tok0 = a.cu_seqlens[n];
        len = a.cu_seqlens[n + 1] - tok0;
    } else {
        tok0 = n * a.tokens_per_seq;
        len = a.tokens_per_seq;
    }
    const auto qp = static_cast<const __nv_bfloat16*>(a.q), kp = static_cast<const __nv_bfloat16*>(a.k);
    const auto vp = static_cast<const __nv_bfloat16*>(a.v);
    const auto out = static_cast<__nv_bfloat16*>(a.out);
    const int64_t srow = (blockIdx.x * static_cast<int64_t>(kHeadDim) + r) * kHeadDim;
    float s[kHeadDim];
#pragma unroll
    for (int c = 0; c < kHeadDim; ++c) {
        s[c] = 0.f;
        if (a.init_state)
            s[c] = a.state_f32 ? static_cast<const float*>(a.init_state)[srow + c]
                               : __bfloat162float(static_cast<const __nv_bfloat16*>(a.init_state)[srow + c]);
    }
    for (int64_t t0 = 0; t0 < len; t0 += kStage) {
        const int m = static_cast<int>(len - t0 < kStage ? len - t0 : kStage);
        __syncthreads();
        for (int i = 0; i < m; ++i) {
            const int64_t at = ((tok0 + t0 + i) * a.Hk + hk) * kHeadDim + r;
            q[i][r] = __bfloat162float(qp[at]);
            k[i][r] = __bfloat162float(kp[at]);
        }
        __syncthreads();
        for (int i = 0; i < m; ++i) {
            const int64_t tok = tok0 + t0 + i;
            const float d = expf(a.g[tok * a.g_stride + h]);
            const float v = __bfloat162float(vp[(tok * a.H + h) * kHeadDim + r]);
            float o = 0.f;
#pragma unroll
            for (int c = 0; c < kHeadDim; ++c) {
                s[c] = fmaf(s[c], d, v * k[i][c]);
                o = fmaf(s[c], q[i][c], o);
            }
            out[(tok * a.H + h) * kHeadDim + r] = __float2bfloat16_rn(a.scale * o);
        }
    }
    if (a.final_state)
#pragma unroll
        for (int c = 0; c < kHeadDim; ++c) {
            if (a.state_f32)
                static_cast<float*>(a.final_state)[srow + c] = s[c];
            else
                static_cast<__nv_bfloat16*>(a.final_state)[srow + c] = __float2bfloat16_rn(s[c]);
        }
}

}  // namespace

cudaError_t launch_la_prefill(const LaArgs& a, cudaStream_t stream) {
    const int64_t blocks = a.N * a.H;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    la_recurrent_kernel<<<static_cast<unsigned>(blocks), kHeadDim, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
