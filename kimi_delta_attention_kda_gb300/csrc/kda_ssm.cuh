// kda_ssm.cuh -- what prompts and single tokens of the selective state space scan
// have in common: the step, a lane's states and their decay (sm_103a).
#pragma once

#include <cfloat>

#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_seq.cuh"
#include "kda_vec.cuh"

namespace kda {

constexpr int kChannels = kSsmChannels;  // channels of a CTA
constexpr float kLog2e = 1.4426950408889634f;

// softplus(u) = max(u, 0) + log(1 + exp(-|u|)).  log(1 + t) / t on [0, 1] is a
// polynomial of degree 8 fitted to the least relative error (3e-8; 1.8e-7 as evaluated
// in FP32).  (Packed pairs would cost more: their operands take three registers'
// reads each, where a constant is part of the scalar instruction.)  NaN stays,
// through the exponential.
__device__ __forceinline__ float softplus(float u) {
    const float t = exp2_fast(fabsf(u) * -kLog2e);
    float p = 0.00523268804f;
    p = fmaf(p, t, -0.0295052137f);
    p = fmaf(p, t, 0.0782259107f);
    p = fmaf(p, t, -0.136632428f);
    p = fmaf(p, t, 0.191060051f);
    p = fmaf(p, t, -0.24842982f);
    p = fmaf(p, t, 0.333190978f);
    p = fmaf(p, t, -0.499994934f);
    p = fmaf(p, t, 0.99999994f);
    return fmaf(t, p, fmaxf(u, 0.f));
}

// Up to 8 (4) values as loaded where they cannot be read as a vector.
__device__ __forceinline__ uint4 gather8(const __nv_bfloat16* p, int n) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? reinterpret_cast<const uint16_t*>(p)[i] : 0u;
    return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}
__device__ __forceinline__ uint4 gather4(const float* p, int n) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's states, of one channel, kBlocks times four of them in pairs.
template <int kBlocks>
struct State {
    uint64_t h[kBlocks][2];
};

// Rates in units of log 2, finite: 2^(-FLT_MAX s) is 0 for every step s above 1e-36, and 1 for
// a step of 0, where minus infinity would give NaN.  (NaN stays.)
template <int kBlocks>
__device__ __forceinline__ void to_log2(State<kBlocks>& rate) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 v = halves(mul_pair(rate.h[k][i], pair(kLog2e, kLog2e)));
            rate.h[k][i] = pair(v.x < -FLT_MAX ? -FLT_MAX : v.x, v.y < -FLT_MAX ? -FLT_MAX : v.y);
        }
}

// The rates of states behind S, which the lanes of a short row have: any below 0, as an infinite step
// times 0 would make NaN of them, and so of y.  Two from state n on.
__device__ __forceinline__ void no_rates(uint64_t& rate, int n, int S) {
    const float2 v = halves(rate);
    rate = pair(n < S ? v.x : -1.f, n + 1 < S ? v.y : -1.f);
}

// What the exponential of x takes from a state, on average: it comes out 6e-9 too small for
// arguments above -2^-8, and 2.2e-8 below (measured on GB300 in steps of a half octave:
// 5e-9 .. 1e-8 and 1.4e-8 .. 3e-8), and is 1 above -2^-23.
__device__ __forceinline__ float lost(float x) {
    const float part = x > -0x1p-8f ? 6e-9f : 2.2e-8f;
    return x > -0x1p-23f ? 1e-30f : part;   // (not 0, for states that are infinite)
}

// h <- exp2(A s) h + b for a lane's states (A in units of log 2).
template <int kBlocks>
__device__ __forceinline__ void decay(State<kBlocks>& s, const State<kBlocks>& rate, uint64_t dt, const uint64_t (&b)[kBlocks][2]) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 e = halves(mul_pair(rate.h[k][i], dt));
            s.h[k][i] = fma_pair(pair(exp2_fast(e.x), exp2_fast(e.y)), s.h[k][i], b[k][i]);
        }
}

}  // namespace kda
