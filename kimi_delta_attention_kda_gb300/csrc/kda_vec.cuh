// kda_vec.cuh -- elements by the vector: loads and stores of several
// consecutive elements as FP32, packed FP32 pairs, and the sigmoid (sm_103a).
#pragma once

#include "kda_common.cuh"

namespace kda {

// The sigmoid from t = exp(-|z|): 1 / (1 + t), or t / (1 + t) for z < 0, so that
// the divisor is at most 2 and small values keep their bits (1 / (1 + exp(-z))
// with the fast division is 0 for z below -87.3, where its divisor passes 2^126).
// 0 and 1 at the infinities, NaN stays.  t as a square keeps the exponential in
// the hardware instruction's range of normal numbers.  It is off by 2^-21 + 2^-24
// |z| of its value, 6e-6 at |z| = 95 against 2^-9 of the BF16 output; an IEEE
// division here made the gated norm bound by its arithmetic.
__device__ __forceinline__ float sigmoid(float z) {
    float h, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(fabsf(z) * -0.72134752044448170f));   // log2(e) / 2
    const float t = h * h;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));
    return z < 0.f ? t * r : r;
}

__device__ __forceinline__ void unpack8(const uint4& r, float (&x)[8]) {
    x[0] = bf16_lo(r.x); x[1] = bf16_hi(r.x); x[2] = bf16_lo(r.y); x[3] = bf16_hi(r.y);
    x[4] = bf16_lo(r.z); x[5] = bf16_hi(r.z); x[6] = bf16_lo(r.w); x[7] = bf16_hi(r.w);
}
// Eight consecutive elements as FP32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), x);
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
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
// kVec consecutive elements: 8 or 4, or 2 or 1 where rows start at any element.
template <int kVec, typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[kVec]) {
    if constexpr (kVec == 8) {
        load8(p, x);
    } else if constexpr (kVec == 4 && sizeof(T) == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else if constexpr (kVec == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    } else if constexpr (kVec == 1) {
        x[0] = static_cast<float>(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        x[0] = v.x;
        x[1] = v.y;
    } else {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
        x[0] = bf16_lo(v);
        x[1] = bf16_hi(v);
    }
}
template <int kVec, typename T>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[kVec]) {
    if constexpr (kVec == 8)
        store8(p, x);
    else if constexpr (kVec == 1)
        from_f32(p, x[0]);
    else if constexpr (kVec == 4 && sizeof(T) == 4)
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else if constexpr (kVec == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    else if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
    else
        *reinterpret_cast<uint32_t*>(p) = pack_bf16(x[0], x[1]);
}

// Two FP32 values in a register pair, for the packed instructions: one issue
// slot for both, each rounded as by the scalar instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 halves(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// x sigmoid(x) of two values, as sigmoid() has it.
__device__ __forceinline__ uint64_t silu_pair(uint64_t x) {
    const float2 v = halves(x);
    float h0, h1, r0, r1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h0) : "f"(fabsf(v.x) * -0.72134752044448170f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h1) : "f"(fabsf(v.y) * -0.72134752044448170f));
    const uint64_t h = pair(h0, h1), t = mul_pair(h, h);
    const float2 e = halves(t), d = halves(add_pair(t, pair(1.f, 1.f)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(d.y));
    return mul_pair(mul_pair(x, pair(v.x < 0.f ? e.x : 1.f, v.y < 0.f ? e.y : 1.f)), pair(r0, r1));
}
// 2^x, off by 1.4e-7 of its value at most (2e-8 on average; 8e-8 and 6e-9 on
// [-0.001, 0]): measured on GB300.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace kda
