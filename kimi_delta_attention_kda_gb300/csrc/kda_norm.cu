// kda_norm.cu -- the norms around a block (sm_103a).
//
// kda_gated_norm, per row of 128 channels:
//     y = x / sqrt(mean(x^2) + eps) * w * act(gate), or the norm of x act(gate) times w;
// kda_residual_norm, per row of any width:
//     u = x or x / sqrt(mean(x^2) + eps) * w_post,  r' = r + scale gate u,
//     y = r' / sqrt(mean(r'^2) + eps) * w.
// Both are bound by HBM: every element is read once and written once, and a
// row stays in registers between its sums and its outputs.  Sums and all
// arithmetic are FP32; outputs are rounded once.
#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

__device__ __forceinline__ float sigmoid(float z) { return 1.f / (1.f + __expf(-z)); }

// Eight consecutive elements as FP32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x); x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
    x[4] = bf16_lo(r.z); x[5] = bf16_hi(r.z); x[6] = bf16_lo(r.w); x[7] = bf16_hi(r.w);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                              pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }

// ------------------------------------------------------------- gated norm
// 16 lanes share a row, 8 channels (16 bytes) each; a thread has kRows rows,
// whose loads are all issued before the first sum.
constexpr int kGnThreads = 256;
constexpr int kGnPass = kGnThreads / 16;   // rows of a CTA at a time

template <typename W, int kAct, bool kFirst, int kRows>
__global__ void __launch_bounds__(kGnThreads)
    gated_norm_kernel(const __nv_bfloat16* x, const W* weight, const __nv_bfloat16* gate,
                      __nv_bfloat16* out, int64_t rows, float eps) {
    const int sub = threadIdx.x & 15;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (kGnPass * kRows) + (threadIdx.x >> 4);
    float a[kRows][8], z[kRows][8], w[8];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = row0 + i * kGnPass;
        if (r < rows) {
            load8(x + r * kHeadDim + 8 * sub, a[i]);
            if (kAct != KDA_ACT_NONE) load8(gate + r * kHeadDim + 8 * sub, z[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) a[i][j] = z[i][j] = 0.f;
        }
    }
    load8(weight + 8 * sub, w);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float s = 1.f;
            if (kAct != KDA_ACT_NONE) s = sigmoid(z[i][j]);
            if (kAct == KDA_ACT_SILU) s *= z[i][j];
            z[i][j] = s;
            if (kFirst) a[i][j] *= s;
            ss = fmaf(a[i][j], a[i][j], ss);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rms = 1.f / sqrtf(ss * (1.f / kHeadDim) + eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[i][j] *= rms * w[j];
            if (!kFirst) a[i][j] *= z[i][j];
        }
        const int64_t r = row0 + i * kGnPass;
        if (r < rows) store8(out + r * kHeadDim + 8 * sub, a[i]);
    }
}

template <typename W, int kAct, bool kFirst>
cudaError_t run_gated(const void* x, const void* weight, const void* gate, void* out, int64_t rows,
                      float eps, cudaStream_t stream) {
    const auto xp = static_cast<const __nv_bfloat16*>(x);
    const auto gp = static_cast<const __nv_bfloat16*>(gate);
    const auto op = static_cast<__nv_bfloat16*>(out);
    const auto wp = static_cast<const W*>(weight);
    constexpr int kRows = 2;
    const int64_t blocks = (rows + kGnPass * kRows - 1) / (kGnPass * kRows);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    gated_norm_kernel<W, kAct, kFirst, kRows>
        <<<static_cast<unsigned>(blocks), kGnThreads, 0, stream>>>(xp, wp, gp, op, rows, eps);
    return cudaGetLastError();
}

// ---------------------------------------------------------- residual norm
// One row per CTA of kThreads threads; a thread holds kGroups groups of kVec
// consecutive elements (kVec 1: widths that are no multiple of 8).
template <int kThreads>
__device__ __forceinline__ float block_sum(float x, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (kThreads == 32) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[warp] = x;
    __syncthreads();
    float y = lane < kThreads / 32 ? buf[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    return y;
}

template <typename T, int kVec>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[kVec]) {
    if constexpr (kVec == 8)
        load8(p, x);
    else
        x[0] = to_f32(*p);
}
template <typename T, int kVec>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[kVec]) {
    if constexpr (kVec == 8)
        store8(p, x);
    else
        from_f32(p, x[0]);
}

template <typename R, typename W, int kVec, int kGroups, int kThreads>
__global__ void __launch_bounds__(kThreads) residual_norm_kernel(ResidualNormArgs p) {
    __shared__ float buf[2][32];
    const int64_t D = p.dim, base = static_cast<int64_t>(blockIdx.x) * D;
    const auto x = static_cast<const __nv_bfloat16*>(p.x) + base;
    const auto res = static_cast<const R*>(p.residual) + base;
    const auto post = static_cast<const W*>(p.post_weight);
    const auto gate = static_cast<const W*>(p.gate);
    const auto weight = static_cast<const W*>(p.weight);
    float u[kGroups][kVec], r[kGroups][kVec];
    const float inv_d = 1.f / static_cast<float>(D);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int64_t at = (static_cast<int64_t>(i) * kThreads + threadIdx.x) * kVec;
#pragma unroll
        for (int j = 0; j < kVec; ++j) u[i][j] = r[i][j] = 0.f;
        if (at < D) {
            load_vec<__nv_bfloat16, kVec>(x + at, u[i]);
            load_vec<R, kVec>(res + at, r[i]);
        }
    }
    if (post) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) ss = fmaf(u[i][j], u[i][j], ss);
        const float rms = 1.f / sqrtf(block_sum<kThreads>(ss, buf[0]) * inv_d + p.eps);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int64_t at = (static_cast<int64_t>(i) * kThreads + threadIdx.x) * kVec;
            if (at < D) {
                float w[kVec];
                load_vec<W, kVec>(post + at, w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) u[i][j] *= rms * w[j];
            }
        }
    }
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int64_t at = (static_cast<int64_t>(i) * kThreads + threadIdx.x) * kVec;
        if (at < D) {
            if (gate) {
                float w[kVec];
                load_vec<W, kVec>(gate + at, w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) u[i][j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                r[i][j] = fmaf(p.scale, u[i][j], r[i][j]);
                ss = fmaf(r[i][j], r[i][j], ss);
            }
            store_vec<R, kVec>(static_cast<R*>(p.residual_out) + base + at, r[i]);
        }
    }
    const float rms = 1.f / sqrtf(block_sum<kThreads>(ss, buf[1]) * inv_d + p.eps);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int64_t at = (static_cast<int64_t>(i) * kThreads + threadIdx.x) * kVec;
        if (at < D) {
            float w[kVec];
            load_vec<W, kVec>(weight + at, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) r[i][j] *= rms * w[j];
            store_vec<__nv_bfloat16, kVec>(static_cast<__nv_bfloat16*>(p.out) + base + at, r[i]);
        }
    }
}

template <typename R, typename W, int kVec, int kGroups, int kThreads>
cudaError_t run_residual(const ResidualNormArgs& p, cudaStream_t stream) {
    residual_norm_kernel<R, W, kVec, kGroups, kThreads>
        <<<static_cast<unsigned>(p.rows), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename R, typename W>
cudaError_t pick_residual(const ResidualNormArgs& p, cudaStream_t stream) {
    const int64_t D = p.dim;
    if (D % 8 == 0) {
        if (D <= 1024) return run_residual<R, W, 8, 1, 128>(p, stream);
        if (D <= 4096) return run_residual<R, W, 8, 2, 256>(p, stream);
        if (D <= 12288) return run_residual<R, W, 8, 3, 512>(p, stream);
        return run_residual<R, W, 8, 4, 1024>(p, stream);
    }
    if (D <= 512) return run_residual<R, W, 1, 4, 128>(p, stream);
    if (D <= 4096) return run_residual<R, W, 1, 8, 512>(p, stream);
    return run_residual<R, W, 1, 32, 1024>(p, stream);
}

}  // namespace

cudaError_t launch_gated_norm(const void* x, const void* weight, const void* gate, void* out,
                              int64_t rows, int activation, bool gate_first, bool weight_f32,
                              float eps, cudaStream_t stream) {
    if (rows <= 0) return cudaSuccess;
#define KDA_GN(ACT, FIRST)                                                                     \
    return weight_f32 ? run_gated<float, ACT, FIRST>(x, weight, gate, out, rows, eps, stream)  \
                      : run_gated<__nv_bfloat16, ACT, FIRST>(x, weight, gate, out, rows, eps, stream)
    if (activation == KDA_ACT_SIGMOID) {
        if (gate_first) KDA_GN(KDA_ACT_SIGMOID, true);
        KDA_GN(KDA_ACT_SIGMOID, false);
    }
    if (activation == KDA_ACT_SILU) {
        if (gate_first) KDA_GN(KDA_ACT_SILU, true);
        KDA_GN(KDA_ACT_SILU, false);
    }
    KDA_GN(KDA_ACT_NONE, false);
#undef KDA_GN
}

cudaError_t launch_residual_norm(const ResidualNormArgs& p, int sms, cudaStream_t stream) {
    (void)sms;
    if (p.rows <= 0) return cudaSuccess;
    if (p.rows > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.residual_f32)
        return p.weight_f32 ? pick_residual<float, float>(p, stream)
                            : pick_residual<float, __nv_bfloat16>(p, stream);
    return p.weight_f32 ? pick_residual<__nv_bfloat16, float>(p, stream)
                        : pick_residual<__nv_bfloat16, __nv_bfloat16>(p, stream);
}

}  // namespace kda
