// kda_step.cu -- single-token steps on a pool of states (sm_103a).
//
// kda_decode, per (sequence, head), with khat and qhat the L2-normalised key
// and query:
//     S <- S Diag(exp g);  u = beta (v - S khat);  S <- S + u khat^T;  o = s S qhat
// kda_la_decode:
//     S <- exp(g) S + v k^T;  o = s S q
// Rows of S (value channels) are independent given k, q and the decay, and
// the output needs no second look at the state:
//     s S_new q = s (S_old' q + u (k . q)),   S_old' the decayed state,
// so S k and S q are formed in one pass over registers, reduced together, and
// the state is read and written once.
//
// Bound by HBM: 2 x 64 KB (FP32) or 2 x 32 KB (BF16) per (sequence, head)
// against 0.25 MFLOP.  Eight lanes share a row, 16 key channels each, in
// 16-byte loads that cover 128 contiguous bytes, so a row's sums take three
// shuffles; a warp has four rows at a time.  All arithmetic is FP32; a BF16
// state is rounded once per step, when it is stored.
//
// Four CTAs share a (sequence, head), 32 rows each.  Where there are enough to
// fill the SMs, two warps take four rows a lane group: the state's loads are all
// under way before the first sum, and a lane group's exponentials and norms
// serve four rows.  Else eight warps take one each, which is sooner done.
// Measured on GB300, L2 flushed, 64 sequences x 96 heads (floors at the 6.80 TB/s
// of a plain copy): FP32 state la_decode 121 us, kda_decode 123 (floor 118.5,
// 119), BF16 65 and 75 (59.3, 60); one CTA of eight warps for all 128 rows took
// 83 for the last, because fewer, larger CTAs start and end together.  6 states:
// 6.1 us with one row a lane group, 8.2 with four.
#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int kPer = 16;        // key channels of a lane

struct StepParams {
    StepArgs a;
    int group;                  // H / Hk
};

// The lane's 16 key channels: FP32 states 4 sub + 32 i + {0..3}, BF16 states
// 8 sub + 64 i + {0..7}, so that each 16-byte access of eight lanes is contiguous.
template <bool kF32>
__device__ __forceinline__ int channel(int sub, int i) {
    return kF32 ? 4 * sub + 32 * (i >> 2) + (i & 3) : 8 * sub + 64 * (i >> 3) + (i & 7);
}

template <bool kF32>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, int sub, float (&x)[kPer]) {
    if (kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint2 r = *reinterpret_cast<const uint2*>(p + channel<true>(sub, 4 * i));
            x[4 * i] = bf16_lo(r.x); x[4 * i + 1] = bf16_hi(r.x);
            x[4 * i + 2] = bf16_lo(r.y); x[4 * i + 3] = bf16_hi(r.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 r = *reinterpret_cast<const uint4*>(p + channel<false>(sub, 8 * i));
            x[8 * i] = bf16_lo(r.x); x[8 * i + 1] = bf16_hi(r.x);
            x[8 * i + 2] = bf16_lo(r.y); x[8 * i + 3] = bf16_hi(r.y);
            x[8 * i + 4] = bf16_lo(r.z); x[8 * i + 5] = bf16_hi(r.z);
            x[8 * i + 6] = bf16_lo(r.w); x[8 * i + 7] = bf16_hi(r.w);
        }
    }
}

template <bool kF32>
__device__ __forceinline__ void load_f32(const float* p, int sub, float (&x)[kPer]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 r = *reinterpret_cast<const float4*>(p + channel<kF32>(sub, 4 * i));
        x[4 * i] = r.x; x[4 * i + 1] = r.y; x[4 * i + 2] = r.z; x[4 * i + 3] = r.w;
    }
}

// A lane's part of a row as loaded: 64 bytes of FP32 or 32 of BF16.
template <bool kF32>
struct RowPart {
    uint4 w[kF32 ? 4 : 2];
};
template <bool kF32>
__device__ __forceinline__ RowPart<kF32> load_row(const void* row, int sub) {
    RowPart<kF32> r;
    const uint4* p = reinterpret_cast<const uint4*>(row) + sub;
#pragma unroll
    for (int i = 0; i < (kF32 ? 4 : 2); ++i) r.w[i] = p[8 * i];
    return r;
}
template <bool kF32>
__device__ __forceinline__ void unpack(const RowPart<kF32>& r, float (&x)[kPer]) {
#pragma unroll
    for (int i = 0; i < (kF32 ? 4 : 2); ++i) {
        const uint32_t w[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (kF32) {
                x[4 * i + j] = __uint_as_float(w[j]);
            } else {
                x[8 * i + 2 * j] = bf16_lo(w[j]);
                x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
            }
        }
    }
}
template <bool kF32>
__device__ __forceinline__ void store_row(void* row, int sub, const float (&x)[kPer]) {
    uint4* p = reinterpret_cast<uint4*>(row) + sub;
    if (kF32) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[8 * i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                  __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            p[8 * i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                                  pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
    }
}

// Sum over the eight lanes that share a row.
__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    return x;
}
__device__ __forceinline__ float dot(const float (&x)[kPer], const float (&y)[kPer]) {
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) {
        s0 = fmaf(x[i], y[i], s0);
        s1 = fmaf(x[i + 1], y[i + 1], s1);
    }
    return s0 + s1;
}

// One CTA: kPasses times kThreads / 8 value rows of one (sequence, head).
template <bool kDelta, bool kF32, int kPasses, int kThreads>
__global__ void __launch_bounds__(kThreads) step_kernel(StepParams p) {
    const StepArgs& a = p.a;
    constexpr int kPassRows = kThreads / 8;
    constexpr int kParts = kHeadDim / (kPassRows * kPasses);
    const int64_t unit = blockIdx.x / kParts;
    const int part = static_cast<int>(blockIdx.x % kParts);
    const int64_t n = unit / a.H, h = unit - n * a.H;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane & 7;
    const int row0 = part * kPassRows * kPasses + 4 * warp + (lane >> 3);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + unit * kHeadDim;

    int64_t slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.pool) {
        if (slot >= a.pool && threadIdx.x == 0) atomicOr(a.status, kDevBadSlots);
        if (sub == 0)
#pragma unroll
            for (int i = 0; i < kPasses; ++i) out[row0 + kPassRows * i] = __float2bfloat16_rn(0.f);
        return;
    }
    constexpr int kRowBytes = kHeadDim * (kF32 ? 4 : 2);
    uint8_t* state = static_cast<uint8_t*>(a.state) +
                     ((slot * a.H + h) * kHeadDim + row0) * static_cast<int64_t>(kRowBytes);
    RowPart<kF32> raw[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) raw[i] = load_row<kF32>(state + i * kPassRows * kRowBytes, sub);

    const int64_t qk = (n * a.Hk + h / p.group) * kHeadDim;
    float q[kPer], k[kPer], e[kDelta ? kPer : 1];
    load_bf16<kF32>(static_cast<const __nv_bfloat16*>(a.q) + qk, sub, q);
    load_bf16<kF32>(static_cast<const __nv_bfloat16*>(a.k) + qk, sub, k);
    float v[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
        v[i] = __bfloat162float(
            static_cast<const __nv_bfloat16*>(a.v)[unit * kHeadDim + row0 + kPassRows * i]);
    float decay = 1.f, beta = 1.f;
    if (kDelta) {
        float g[kPer];
        load_f32<kF32>(a.g + unit * kHeadDim, sub, g);
        beta = __bfloat162float(static_cast<const __nv_bfloat16*>(a.beta)[unit]);
        if (a.beta_logit) beta = 1.f / (1.f + expf(-beta));
        const float rq = 1.f / sqrtf(sum8(dot(q, q)) + 1e-6f);
        const float rk = 1.f / sqrtf(sum8(dot(k, k)) + 1e-6f);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            e[i] = expf(g[i]);
            q[i] *= rq;
            k[i] *= rk;
        }
    } else {
        decay = expf(a.g[a.g_stride ? n * a.g_stride + h : h]);
    }
    const float kq = sum8(dot(k, q));
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        float s[kPer];
        unpack<kF32>(raw[i], s);
        float u = v[i], o;
        if (kDelta) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) s[j] *= e[j];
            u = beta * (v[i] - sum8(dot(s, k)));
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) s[j] *= decay;
        }
        o = a.scale * fmaf(u, kq, sum8(dot(s, q)));
#pragma unroll
        for (int j = 0; j < kPer; ++j) s[j] = fmaf(u, k[j], s[j]);
        store_row<kF32>(state + i * kPassRows * kRowBytes, sub, s);
        if (sub == 0) out[row0 + kPassRows * i] = __float2bfloat16_rn(o);
    }
}

template <bool kDelta, bool kF32>
cudaError_t launch(const StepParams& p, int sms, cudaStream_t stream) {
    const int64_t units = p.a.N * p.a.H;
    if (units * 4 > 0x7fffffffLL) return cudaErrorInvalidValue;
    const unsigned ctas = static_cast<unsigned>(units * 4);
    if (units >= sms)
        step_kernel<kDelta, kF32, 4, 64><<<ctas, 64, 0, stream>>>(p);
    else
        step_kernel<kDelta, kF32, 1, 256><<<ctas, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_step(const StepArgs& a, bool delta, int sms, cudaStream_t stream) {
    if (a.N <= 0) return cudaSuccess;
    StepParams p;
    p.a = a;
    p.group = static_cast<int>(a.H / a.Hk);
    if (delta) return a.state_f32 ? launch<true, true>(p, sms, stream) : launch<true, false>(p, sms, stream);
    return a.state_f32 ? launch<false, true>(p, sms, stream) : launch<false, false>(p, sms, stream);
}

}  // namespace kda
