// kda_la_prefill.cu -- linear attention with one decay per head and token,
// whole prompts, on the tcgen05 tensor cores (sm_103a):
//     S_t = exp(g_t) S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t.
//
// A sequence is taken in chunks of 128 tokens.  With G_i the sum of the
// decays of the chunk's tokens up to i, G the chunk's whole sum and S the
// state before the chunk, the chunk's outputs and the state after it are
//     o_i = scale ( exp(G_i) S q_i + sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j )
//     S   <- exp(G) S + sum_j exp(G - G_j) v_j k_j^T.
// Every exponent is at most 0, so nothing overflows whatever the decays are;
// exp(G - G_j) is formed from a sum that starts behind j, so that it is exact
// to FP32 even where G and G_j are large.
//
// As products of 128 x 128 tiles (i, j tokens; c value, d key channels):
//     D1[i][j] = Q K^T              Q, K from shared memory
//     P[i][j]  = scale exp(G_i - G_j) D1, causal, BF16, in tensor memory
//     O[i][c]  = Q' S^T + P V       Q' = scale exp(G_i) Q (BF16), S^T BF16 in shared memory
//     S^T[d][c] <- exp(G) S^T + K'^T V   K'^T[d][j] = exp(G - G_j) k_jd, in tensor memory
// S^T is FP32 in tensor memory: the state warps read it, write its BF16 copy
// to shared memory and exp(G) S^T back, and K'^T V accumulates on that.
// K' is split by truncation into three BF16 parts whose sum is the FP32
// value, so the state is accurate to FP32: with two parts (16 bits) the final
// state was off by 2e-6 of its norm, against 1e-7 for FP32 arithmetic.
// P, Q' and the S operand are rounded to BF16 once each: their error stays in
// the BF16 output they go to, and S itself is not touched by it.
//
// One CTA per SM walks (sequence or segment, head) units.  Warps: 8 state
// (K' parts, S), 4 score (P), 4 output (Q', O), one each for the loads, the
// MMA issue and the decay sums.  Tensor memory columns: D1 and P [0, 128),
// O [128, 256), S^T [256, 384), K' [384, 480) (two buffers of 32 tokens x 3
// parts).
//
// A value that is not finite must not reach earlier tokens of its chunk: a
// zero of P times an infinite V is NaN.  S^T shows it (its whole column is
// then not finite).  The state warps clear such values in shared memory once
// S^T has them, and the output warps add their products for j <= i alone,
// with V from global memory.
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_tcgen05.cuh"

namespace kda {
namespace {

constexpr int kC = kLaChunk;
constexpr uint32_t kSmemBase = 1024;
constexpr uint32_t kSlab = 16384;   // 128 rows x 64 BF16, 128-byte swizzle
constexpr uint32_t kTile = 2 * kSlab;
constexpr int kStateWarps = 8, kScoreWarp = 8, kOutWarp = 12, kLoadWarp = 16, kMmaWarp = 17, kDecayWarp = 18;
constexpr int kThreads = 19 * 32;
constexpr uint32_t kColD1 = 0, kColO = 128, kColS = 256, kColK = 384, kTmemCols = 512;
constexpr uint32_t kKBuf = 48, kKPart = 16;   // K' buffer and part, in columns
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMinDecay = -150.f;           // in base 2: exp2 of it is 0 in FP32

// Shared memory.  The state pass (kStates) has no Q and no S operand, and a
// third stage of K and V in their place.
template <bool kStates>
struct Smem {
    static constexpr int kStages = kStates ? 3 : 2;
    static constexpr uint32_t kK = 0, kV = kK + kStages * kTile, kQ = kV + kStages * kTile,
                              kS = kQ + (kStates ? 0 : kStages * kTile), kMisc = kS + (kStates ? 0 : kTile);
    // G (prefix sums), W (exp of the sums behind a token), C (exp of the sum
    // from a token to the end of its block of 32): two buffers each.
    static constexpr uint32_t kG = kMisc, kW = kG + 2 * kC * 4, kCf = kW + 2 * kC * 4, kBars = kCf + 2 * 96 * 4;
    static constexpr int kNumBars = 4 * kStages + 4 + 18;
    static constexpr uint32_t kFlag = kBars + 8 * kNumBars, kTmemPtr = kFlag + 8, kBytes = kTmemPtr + 8;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};

struct Bars {
    uint64_t *full_k, *full_v, *full_q, *empty_k, *empty_v, *empty_q;   // [stages]
    uint64_t *qk, *p, *kp_full, *kp_empty, *z_done, *checked, *s_ready, *qs_done, *q_scaled, *o_done, *o_free;
    uint64_t *dec_full, *dec_empty, *done;
};
template <bool kStates>
__device__ __forceinline__ Bars make_bars(uint8_t* smem) {
    constexpr int n = Smem<kStates>::kStages;
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + Smem<kStates>::kBars);
    Bars r;
    r.full_k = b; b += n;
    r.full_v = b; b += n;
    r.empty_k = b; b += n;
    r.empty_v = b; b += n;
    r.full_q = b; b += 2;
    r.empty_q = b; b += 2;
    r.qk = b++;
    r.p = b++;
    r.kp_full = b; b += 2;
    r.kp_empty = b; b += 2;
    r.z_done = b++;
    r.checked = b++;
    r.s_ready = b++;
    r.qs_done = b++;
    r.q_scaled = b++;
    r.o_done = b++;
    r.o_free = b++;
    r.dec_full = b; b += 2;
    r.dec_empty = b; b += 2;
    r.done = b++;
    return r;
}

struct Kernel {
    LaArgs a;
    LaSegments sg;      // sg.starts null: no segments
    int64_t units;
};

// One (sequence or segment, head).
struct Unit {
    int64_t n, h, tok0, len;
    int64_t slot;       // (segment, head) row of the segments' buffers
    bool last;          // writes the final state
    int nch;
};
template <bool kStates>
__device__ __forceinline__ Unit unit_at(const Kernel& p, int64_t u) {
    Unit w;
    const int64_t s = u / p.a.H;
    w.h = u - s * p.a.H;
    w.slot = u;
    w.last = true;
    if (!p.sg.starts) {
        w.n = s;
        if (p.a.cu_seqlens) {
            w.tok0 = p.a.cu_seqlens[s];
            w.len = p.a.cu_seqlens[s + 1] - w.tok0;
        } else {
            w.tok0 = s * p.a.tokens_per_seq;
            w.len = p.a.tokens_per_seq;
        }
    } else if (p.sg.seg_begin) {
        w.n = p.sg.seg_seq[s];
        w.tok0 = p.sg.seg_tokens[s];
        w.len = s < p.sg.seg_begin[p.a.N] ? p.sg.seg_tokens[s + 1] - w.tok0 : 0;
        w.last = s + 1 == p.sg.seg_begin[w.n + 1];
        if (w.len == 0) w.last = false;   // padding of the segment table
    } else {
        w.n = s / p.sg.segs;
        const int64_t j = s - w.n * p.sg.segs;
        w.tok0 = w.n * p.a.tokens_per_seq + j * p.sg.seg_tokens_each;
        w.last = j + 1 == p.sg.segs;
        w.len = w.last ? p.a.tokens_per_seq - j * p.sg.seg_tokens_each : p.sg.seg_tokens_each;
    }
    if (kStates && w.last) w.len = 0;     // nothing follows a sequence's last segment
    w.nch = static_cast<int>((w.len + kC - 1) / kC);
    return w;
}
__device__ __forceinline__ int valid_of(const Unit& w, int c) {
    const int64_t left = w.len - static_cast<int64_t>(c) * kC;
    return left < kC ? static_cast<int>(left) : kC;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t prmt_hi(uint32_t lo, uint32_t hi) {   // the upper halves of two words
    return __byte_perm(lo, hi, 0x7632);
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, int32_t x, int32_t y, const void* src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(tmap), "r"(x), "r"(y), "r"(smem_u32(src)) : "memory");
}
// Shared-memory descriptors as (low word, constant high word): the low word
// is the start address over 16 and the leading offset, so a step inside a
// tile is an addition, and an MMA's operands cost the issuing warp one each.
// K-major operands (128-byte swizzle): 8-row groups 1024 B apart.  Operands
// whose M or N index is contiguous: rows of 64 elements of it, 8-row groups of
// K 1024 B apart, the next 64 elements one slab (the leading offset) further.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (tc::kSwizzle128B << 29);
constexpr uint32_t kLeadK = 1u << 16, kLeadMn = (kSlab >> 4) << 16;
__host__ __device__ constexpr uint32_t k_step(int k) { return ((k >> 2) * kSlab + 32 * (k & 3)) >> 4; }   // K-major, 16 elements
__host__ __device__ constexpr uint32_t mn_step(int k) { return (k * 2048) >> 4; }                        // 16 rows
template <uint32_t kId>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %3, 0;\n mov.b64 a, {%1, %4};\n mov.b64 b, {%2, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n}\n" ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(acc),
        "n"(kDescHi), "n"(kId) : "memory");
}
template <uint32_t kId>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %3, 0;\n mov.b64 b, {%2, %4};\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %5, p;\n}\n" ::"r"(d), "r"(a), "r"(b_lo), "r"(acc),
        "n"(kDescHi), "n"(kId) : "memory");
}
constexpr uint32_t kIdesc = tc::idesc_bf16(128, 128);
constexpr uint32_t kIdescMn = kIdesc | (1u << 16);   // B is MN-major

__device__ __forceinline__ void st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// Wait, with the whole warp, for a phase of an mbarrier.  A wait that polls
// takes issue slots from the other warps of its scheduler, so the loop is two
// instructions a try, with a bound on tries in place of a clock (kTries x 8
// tries of 20 cycles and more: over a second).
constexpr uint32_t kTries = 1u << 24;
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, int* status) {
    uint32_t ok = 0;
    const uint32_t at = smem_u32(bar);
#pragma unroll 1
    for (uint32_t n = 0; n < kTries; ++n) {
        asm volatile(
            "{\n .reg .pred p;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra.uni D%=;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra.uni D%=;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra.uni D%=;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra.uni D%=;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra.uni D%=;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra.uni D%=;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra.uni D%=;\n"
            " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
            "D%=:\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok) : "r"(at), "r"(parity) : "memory");
        if (ok) break;
    }
    if (__all_sync(0xffffffffu, ok)) return true;
    if ((threadIdx.x & 31) == 0) atomicOr(status, kDevPipeTimeout);
    return false;
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar, int lane) {
    __syncwarp();
    mbar_arrive_if(bar, lane == 0);
}

// --------------------------------------------------------------- load warp
template <bool kStates>
__device__ __forceinline__ void load_role(const Kernel& p, const CUtensorMap* qmap, const CUtensorMap* kmap,
                                          const CUtensorMap* vmap, uint8_t* smem, const Bars& b, int lane) {
    using M = Smem<kStates>;
    constexpr int n = M::kStages;
    const int64_t group = p.a.H / p.a.Hk;
    int64_t it = 0;
    int issued[3] = {0, 0, 0};   // tiles of K, V, Q under way or done
    bool ok = true;
    for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
        const Unit w = unit_at<kStates>(p, u);
        const int xk = static_cast<int>(w.h / group * kHeadDim), xv = static_cast<int>(w.h * kHeadDim);
        for (int c = 0; c < w.nch && ok; ++c, ++it) {
            const int s = static_cast<int>(it % n);
            const uint32_t ph = static_cast<uint32_t>((it / n) - 1) & 1u;
            const int y = static_cast<int>(w.tok0 + static_cast<int64_t>(c) * kC);
            for (int t = 0; t < (kStates ? 2 : 3) && ok; ++t) {
                uint64_t* empty = t == 0 ? b.empty_k : t == 1 ? b.empty_v : b.empty_q;
                uint64_t* full = t == 0 ? b.full_k : t == 1 ? b.full_v : b.full_q;
                if (it >= n) ok = wait_phase(&empty[s], ph, p.a.status);
                if (!ok) break;
                if (lane == 0) {
                    uint8_t* dst = smem + (t == 0 ? M::kK : t == 1 ? M::kV : M::kQ) + s * kTile;
                    const CUtensorMap* map = t == 0 ? kmap : t == 1 ? vmap : qmap;
                    const int x = t == 1 ? xv : xk;
                    mbar_arrive_expect_tx(&full[s], kTile);
                    tma_load_2d(dst, map, x, y, &full[s]);
                    tma_load_2d(dst + kSlab, map, x + 64, y, &full[s]);
                }
                ++issued[t];
                __syncwarp();
            }
        }
    }
    // No copy may be under way when the CTA ends.
    for (int t = 0; t < 3; ++t)
        for (int s = 0; s < n; ++s)
            if (issued[t] > s)
                mbar_wait_bounded(&(t == 0 ? b.full_k : t == 1 ? b.full_v : b.full_q)[s],
                                  static_cast<uint32_t>((issued[t] - 1 - s) / n) & 1u, p.a.status);
}

// -------------------------------------------------------------- decay warp
template <bool kStates>
__device__ __forceinline__ void decay_role(const Kernel& p, uint8_t* smem, const Bars& b, int lane) {
    using M = Smem<kStates>;
    int64_t it = 0;
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
        const Unit w = unit_at<kStates>(p, u);
        for (int c = 0; c < w.nch; ++c, ++it) {
            const int buf = static_cast<int>(it & 1);
            const int valid = valid_of(w, c);
            const int64_t tok = w.tok0 + static_cast<int64_t>(c) * kC + 4 * lane;
            float x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                x[r] = 0.f;
                if (4 * lane + r < valid) {
                    x[r] = p.a.g[(tok + r) * p.a.g_stride + w.h] * kLog2e;
                    if (x[r] < kMinDecay) x[r] = kMinDecay;   // -inf too; NaN stays
                }
            }
            // Prefix and suffix sums, each from its own end.
            float pre[4], suf[4];
            pre[0] = x[0];
            suf[3] = 0.f;
#pragma unroll
            for (int r = 1; r < 4; ++r) {
                pre[r] = pre[r - 1] + x[r];
                suf[3 - r] = suf[4 - r] + x[4 - r];
            }
            float up = pre[3], down = suf[0] + x[0];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, up, o), z = __shfl_down_sync(0xffffffffu, down, o);
                if (lane >= o) up += y;
                if (lane + o < 32) down += z;
            }
            float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 0) before = 0.f;
            if (lane == 31) behind = 0.f;
            float g[4], wt[4], cf[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) g[r] = before + pre[r];
            const float ref = __shfl_sync(0xffffffffu, g[3], lane | 7);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                wt[r] = 4 * lane + r < valid ? exp2f(behind + suf[r]) : 0.f;
                cf[r] = ex2(ref - g[r]);
            }
            if (it >= 2 && !wait_phase(&b.dec_empty[buf], static_cast<uint32_t>((it >> 1) - 1) & 1u, p.a.status))
                return;
            *reinterpret_cast<float4*>(smem + M::kG + buf * kC * 4 + 16 * lane) = make_float4(g[0], g[1], g[2], g[3]);
            *reinterpret_cast<float4*>(smem + M::kW + buf * kC * 4 + 16 * lane) = make_float4(wt[0], wt[1], wt[2], wt[3]);
            if (lane < 24)
                *reinterpret_cast<float4*>(smem + M::kCf + buf * 96 * 4 + 16 * lane) = make_float4(cf[0], cf[1], cf[2], cf[3]);
            arrive_warp(&b.dec_full[buf], lane);
        }
    }
}

// ---------------------------------------------------------------- MMA warp
// Per chunk: K'^T V of the first 64 tokens, D1, K'^T V of the other 64, Q' S^T,
// P V.  D1 overwrites the P of the chunk before, whose product is complete by
// then (the first half runs meanwhile); the CTA's first chunk starts with D1.
template <bool kStates>
struct Issue {
    using M = Smem<kStates>;
    static constexpr uint32_t kBase = kSmemBase >> 4;
    template <int s>
    static __device__ __forceinline__ void scores() {
        constexpr uint32_t dk = (kBase + ((M::kK + s * kTile) >> 4)) | kLeadK, dq = (kBase + ((M::kQ + s * kTile) >> 4)) | kLeadK;
#pragma unroll
        for (int k = 0; k < 8; ++k) mma_ss<kIdesc>(kColD1, dq + k_step(k), dk + k_step(k), k > 0);
    }
    template <int s, int q>
    static __device__ __forceinline__ void state(bool fresh) {
        constexpr uint32_t dv = (kBase + ((M::kV + s * kTile) >> 4)) | kLeadMn;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int part = 0; part < 3; ++part) {
                const uint32_t a = kColK + kKBuf * (q & 1) + kKPart * part + 8 * t;
                if (q == 0 && t == 0 && part == 0)
                    mma_ts<kIdescMn>(kColS, a, dv + mn_step(2 * q + t), fresh ? 0u : 1u);
                else
                    mma_ts<kIdescMn>(kColS, a, dv + mn_step(2 * q + t), 1u);
            }
    }
    template <int s>
    static __device__ __forceinline__ void incoming() {
        constexpr uint32_t dq = (kBase + ((M::kQ + s * kTile) >> 4)) | kLeadK, ds = (kBase + (M::kS >> 4)) | kLeadMn;
#pragma unroll
        for (int k = 0; k < 8; ++k) mma_ss<kIdescMn>(kColO, dq + k_step(k), ds + mn_step(k), k > 0);
    }
    template <int s>
    static __device__ __forceinline__ void inside() {
        constexpr uint32_t dv = (kBase + ((M::kV + s * kTile) >> 4)) | kLeadMn;
#pragma unroll
        for (int k = 0; k < 8; ++k) mma_ts<kIdescMn>(kColO, kColD1 + 8 * k, dv + mn_step(k), 1u);
    }
};

template <bool kStates, int s>
__device__ __forceinline__ bool mma_chunk(const Kernel& p, uint8_t* smem, const Bars& b, bool leader, int64_t it, bool fresh) {
    using M = Smem<kStates>;
    using I = Issue<kStates>;
    constexpr int n = M::kStages;
    int* status = p.a.status;
    const volatile int* flag = reinterpret_cast<const volatile int*>(smem + M::kFlag);
    const uint32_t st = static_cast<uint32_t>(it / n) & 1u, ph = static_cast<uint32_t>(it & 1), pv = ph ^ 1u;
    auto scores = [&]() {
        if (!wait_phase(&b.full_k[s], st, status) || !wait_phase(&b.full_q[s], st, status)) return false;
        if (it > 0) {
            if (!wait_phase(b.o_done, pv, status)) return false;
            if (flag[(it - 1) & 1] == static_cast<int>(it) && !wait_phase(b.o_free, pv, status)) return false;   // P still read
        }
        tc::fence_after_sync();
        if (leader) {
            I::template scores<s>();
            tc::commit(b.qk);
            tc::commit(&b.empty_k[s]);
        }
        __syncwarp();
        return true;
    };
    auto state = [&](auto qc) {
        constexpr int q = decltype(qc)::value;
        if (!wait_phase(&b.kp_full[q & 1], q >> 1, status)) return false;   // two uses a chunk
        tc::fence_after_sync();
        if (leader) {
            I::template state<s, q>(kStates && fresh);
            tc::commit(&b.kp_empty[q & 1]);
            if (q == 3) tc::commit(b.z_done);
            if (kStates && q == 3) tc::commit(&b.empty_v[s]);
        }
        __syncwarp();
        return true;
    };
    if (!kStates && it == 0 && !scores()) return false;
    if (!wait_phase(&b.full_v[s], st, status) || !wait_phase(b.s_ready, ph, status)) return false;
    if (!state(std::integral_constant<int, 0>()) || !state(std::integral_constant<int, 1>())) return false;
    if (!kStates && it > 0 && !scores()) return false;
    if (!state(std::integral_constant<int, 2>()) || !state(std::integral_constant<int, 3>())) return false;
    if (kStates) return true;
    if (!wait_phase(b.q_scaled, ph, status) || (it > 0 && !wait_phase(b.o_free, pv, status))) return false;
    tc::fence_after_sync();
    if (leader) {
        I::template incoming<s>();
        tc::commit(b.qs_done);
    }
    __syncwarp();
    if (!wait_phase(b.checked, ph, status) || !wait_phase(b.p, ph, status)) return false;
    tc::fence_after_sync();
    if (leader) {
        I::template inside<s>();
        tc::commit(b.o_done);
    }
    __syncwarp();
    return true;
}

template <bool kStates>
__device__ __forceinline__ void mma_role(const Kernel& p, uint8_t* smem, const Bars& b, uint32_t tmem, int lane) {
    constexpr int n = Smem<kStates>::kStages;
    const bool leader = elect_one();
    int64_t it = 0;
    int s = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
        const Unit w = unit_at<kStates>(p, u);
        for (int c = 0; c < w.nch && ok; ++c, ++it) {
            if (s == 0)
                ok = mma_chunk<kStates, 0>(p, smem, b, leader, it, c == 0);
            else if (s == 1)
                ok = mma_chunk<kStates, 1>(p, smem, b, leader, it, c == 0);
            else if (n == 3)
                ok = mma_chunk<kStates, n == 3 ? 2 : 0>(p, smem, b, leader, it, c == 0);
            s = s + 1 == n ? 0 : s + 1;
        }
    }
    // Every MMA must be complete before tensor memory is released.
    if (leader) tc::commit(b.done);
    __syncwarp();
    wait_phase(b.done, 0, p.a.status);
}

// Clears the values that are not finite in two 16-byte columns of a slab of
// V, with one warp; true if there were any.
__device__ __forceinline__ bool clear_not_finite(uint8_t* slab, int chunk, int lane) {
    bool any = false;
#pragma unroll 1
    for (int r = lane; r < kC; r += 32)
#pragma unroll 1
        for (int x = chunk; x < chunk + 2; ++x) {
            uint32_t* at = reinterpret_cast<uint32_t*>(slab + r * 128 + ((x ^ (r & 7)) << 4));
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v = at[j];
                if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
                if ((v & 0x7f800000u) == 0x7f800000u) v &= 0xffffu;
                any |= v != at[j];
                at[j] = v;
            }
        }
    return __any_sync(0xffffffffu, any);
}

// ------------------------------------------------------------- state warps
// Warp ws: key channels 32 (ws % 4) .. + 31, one per lane (the tensor-memory
// lanes it may access); value channels 64 (ws / 4) .. + 63 of S; of K', the
// 16 tokens 16 (ws / 4) .. of each 32.
// 32 of a lane's value channels of a state in global memory ([value][key],
// stride 128), or zeros.
__device__ __forceinline__ void load_state(const void* base, bool f32, int64_t at, uint32_t (&x)[32]) {
    if (!base) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0u;
    } else if (f32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = static_cast<const uint32_t*>(base)[at + i * kHeadDim];
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            x[i] = static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at + i * kHeadDim]) << 16;
    }
}
__device__ __forceinline__ void store_state(void* base, bool f32, int64_t at, const uint32_t (&x)[32]) {
    if (f32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) static_cast<uint32_t*>(base)[at + i * kHeadDim] = x[i];
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
            static_cast<__nv_bfloat16*>(base)[at + i * kHeadDim] = __float2bfloat16_rn(__uint_as_float(x[i]));
    }
}

template <bool kStates>
__device__ __forceinline__ void state_role(const Kernel& p, uint8_t* smem, const Bars& b, uint32_t tmem, int ws, int lane) {
    using M = Smem<kStates>;
    constexpr int n = M::kStages;
    int* status = p.a.status;
    volatile int* flag = reinterpret_cast<volatile int*>(smem + M::kFlag);
    const int half = ws >> 2, key = 32 * (ws & 3) + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * (ws & 3)) << 16);
    const uint32_t scol = trow + kColS + 64 * half;
    const uint32_t kbase = (key >> 6) * kSlab + 16 * half * 128 + 2 * (key & 7);
    const uint32_t kchunk = ((key & 63) >> 3) << 4;
    int64_t it = 0;
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
        const Unit w = unit_at<kStates>(p, u);
        const int64_t at = ((w.n * p.a.H + w.h) * kHeadDim + 64 * half) * kHeadDim + key;
        const int64_t seg_at = (w.slot * kHeadDim + 64 * half) * kHeadDim + key;
        const void* init = p.sg.starts ? static_cast<const void*>(p.sg.starts) : p.a.init_state;
        const bool init_f32 = p.sg.starts || p.a.state_f32;
        const int64_t init_at = p.sg.starts ? seg_at : at;
        const bool final = !kStates && w.last && p.a.final_state;
        if (w.nch == 0) {
            if (final)
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    uint32_t x[32];
                    load_state(init, init_f32, init_at + 32 * i * kHeadDim, x);
                    store_state(p.a.final_state, p.a.state_f32, at + 32 * i * kHeadDim, x);
                }
            continue;
        }
        float total = 0.f;
        for (int c = 0; c < w.nch; ++c, ++it) {
            const int s = static_cast<int>(it % n), buf = static_cast<int>(it & 1);
            const uint32_t st = static_cast<uint32_t>(it / n) & 1u, ph = static_cast<uint32_t>(it & 1);
            uint8_t* K = smem + M::kK + s * kTile;
            uint8_t* V = smem + M::kV + s * kTile;
            const int valid = valid_of(w, c);
            if (!wait_phase(&b.full_k[s], st, status) ||
                !wait_phase(&b.dec_full[buf], static_cast<uint32_t>(it >> 1) & 1u, status))
                return;
            if (valid < kC) {
                // Rows behind the sequence's end: another sequence's tokens,
                // or anything.  V's are cleared here, K's below.
                if (!wait_phase(&b.full_v[s], st, status)) return;
                for (int r = valid + ws; r < kC; r += kStateWarps)
                    if (lane < 16)
                        *reinterpret_cast<uint4*>(V + (lane >> 3) * kSlab + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
            }
            // K' of tokens 32 q + 16 half .. + 15: three truncated parts.
            auto form = [&](int q) -> bool {
                const uint8_t* src = K + kbase + 32 * q * 128;
                const float4* wp = reinterpret_cast<const float4*>(smem + M::kW + buf * kC * 4) + 8 * q + 4 * half;
                uint32_t kb[16];
                float4 w4[4];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    kb[i] = *reinterpret_cast<const uint16_t*>(src + i * 128 + (kchunk ^ ((i & 7) << 4)));
#pragma unroll
                for (int i = 0; i < 4; ++i) w4[i] = wp[i];
                if (valid < kC) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (32 * q + 16 * half + i >= valid) kb[i] = 0;
                }
                uint32_t hi[8], mid[8], lo[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float w0 = i & 1 ? w4[i >> 1].z : w4[i >> 1].x, w1 = i & 1 ? w4[i >> 1].w : w4[i >> 1].y;
                    float x0 = __uint_as_float(kb[2 * i] << 16), x1 = __uint_as_float(kb[2 * i + 1] << 16);
                    mul2v(x0, x1, w0, w1);
                    const uint32_t a0 = __float_as_uint(x0), a1 = __float_as_uint(x1);
                    sub2(x0, x1, __uint_as_float(a0 & 0xffff0000u), __uint_as_float(a1 & 0xffff0000u));
                    const uint32_t b0 = __float_as_uint(x0), b1 = __float_as_uint(x1);
                    sub2(x0, x1, __uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u));
                    hi[i] = prmt_hi(a0, a1);
                    mid[i] = prmt_hi(b0, b1);
                    lo[i] = prmt_hi(__float_as_uint(x0), __float_as_uint(x1));
                }
                if (q == 3) stage_release(&b.empty_k[s], lane);
                const int64_t use = 2 * it + (q >> 1);
                if (use > 0 && !wait_phase(&b.kp_empty[q & 1], static_cast<uint32_t>(use - 1) & 1u, status)) return false;
                tc::fence_after_sync();
                const uint32_t col = trow + kColK + kKBuf * (q & 1) + 8 * half;
                st_x8(col, hi);
                st_x8(col + kKPart, mid);
                st_x8(col + 2 * kKPart, lo);
                tc::wait_st();
                tc::fence_before_sync();
                arrive_warp(&b.kp_full[q & 1], lane);
                return true;
            };
            if (!form(0)) return;
            const float sum = reinterpret_cast<const float*>(smem + M::kG)[buf * kC + kC - 1];
            const float d = exp2f(sum);
            total += sum;
            // The state before this chunk: its BF16 copy as the B operand of
            // Q' S^T (row d: 128 value channels), once the last chunk's
            // product has read its own, and the decayed state.
            if (!kStates && it > 0 && !wait_phase(b.qs_done, ph ^ 1u, status)) return;
            if (!kStates || c > 0) {
                tc::fence_after_sync();
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    uint32_t x[32];
                    if (c == 0) {
                        load_state(init, init_f32, init_at + 32 * i * kHeadDim, x);
                    } else {
                        tc::ld_x32(scol + 32 * i, x);
                        tc::wait_ld();
                    }
                    if (!kStates) {
                        uint8_t* row = smem + M::kS + half * kSlab + key * 128;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t y[4];
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                y[r] = pack_bf16(__uint_as_float(x[8 * j + 2 * r]), __uint_as_float(x[8 * j + 2 * r + 1]));
                            *reinterpret_cast<uint4*>(row + (((4 * i + j) ^ (key & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * d);
                    tc::st_x32(scol + 32 * i, x);
                }
                if (!kStates) fence_proxy_async_smem();
                tc::wait_st();
                tc::fence_before_sync();
            }
            arrive_warp(b.s_ready, lane);
#pragma unroll 1
            for (int q = 1; q < 4; ++q)
                if (!form(q)) return;
            arrive_warp(&b.dec_empty[buf], lane);
            if (!wait_phase(b.z_done, ph, status)) return;
            tc::fence_after_sync();
            if (!kStates) {
                // Each warp watches 16 value channels: a V that is not finite
                // spoils its channel in every lane.
                uint32_t z[16];
                ld_x16(scol + 16 * (ws & 3), z);
                tc::wait_ld();
                float chk = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) chk = fmaf(__uint_as_float(z[i]), 0.f, chk);
                if (__any_sync(0xffffffffu, !(chk == 0.f))) {
                    // The flag of a chunk is its number, so none has to be cleared.
                    if (clear_not_finite(V + half * kSlab, 2 * (ws & 3), lane) && lane == 0)
                        flag[buf] = static_cast<int>(it + 1);
                    fence_proxy_async_smem();
                    __threadfence_block();
                }
                arrive_warp(b.checked, lane);
            }
        }
        if (kStates || final) {
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {
                uint32_t x[32];
                tc::ld_x32(scol + 32 * i, x);
                tc::wait_ld();
                if (kStates)
                    store_state(p.sg.starts, true, seg_at + 32 * i * kHeadDim, x);
                else
                    store_state(p.a.final_state, p.a.state_f32, at + 32 * i * kHeadDim, x);
            }
            if (kStates && ws == 0 && lane == 0) p.sg.decay[w.slot] = total;
            tc::fence_before_sync();
        }
    }
}

// ------------------------------------------------------------- score warps
// Warp wp: rows (tokens) 32 wp .. + 31, one per lane.  Blocks of 32 columns
// before the row's own take exp(G_i - G_j) as a row factor to the end of the
// block times a column factor from there, both at most 1: one exponential
// per row and block instead of one per score.
__device__ __forceinline__ void score_role(const Kernel& p, uint8_t* smem, const Bars& b, uint32_t tmem, int wp, int lane) {
    using M = Smem<false>;
    int* status = p.a.status;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * wp) << 16) + kColD1;
    const float scale = p.a.scale;
    int64_t it = 0;
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
        const Unit w = unit_at<false>(p, u);
        for (int c = 0; c < w.nch; ++c, ++it) {
            const int buf = static_cast<int>(it & 1);
            const float* G = reinterpret_cast<const float*>(smem + M::kG) + buf * kC;
            const float4* Cf = reinterpret_cast<const float4*>(smem + M::kCf + buf * 96 * 4);
            if (!wait_phase(&b.dec_full[buf], static_cast<uint32_t>(it >> 1) & 1u, status)) return;
            const float gi = G[32 * wp + lane];
            if (!wait_phase(b.qk, static_cast<uint32_t>(it & 1), status)) return;
            tc::fence_after_sync();
            // A block's columns of P, 16 blk .. + 15, held scores of blocks
            // already read.
            auto full = [&](int blk, const uint32_t (&x)[32]) {
                const float f = scale * ex2(gi - G[32 * blk + 31]);
                uint32_t pk[16];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 cf = Cf[8 * blk + j];
                    float y0 = __uint_as_float(x[4 * j]), y1 = __uint_as_float(x[4 * j + 1]);
                    float y2 = __uint_as_float(x[4 * j + 2]), y3 = __uint_as_float(x[4 * j + 3]);
                    mul2(y0, y1, f);
                    mul2(y2, y3, f);
                    mul2v(y0, y1, cf.x, cf.y);
                    mul2v(y2, y3, cf.z, cf.w);
                    pk[2 * j] = pack_bf16(y0, y1);
                    pk[2 * j + 1] = pack_bf16(y2, y3);
                }
                tc::st_x16(trow + 16 * blk, pk);
            };
            uint32_t x[32];
#pragma unroll 1
            for (int blk = 0; blk < wp; ++blk) {
                tc::ld_x32(trow + 32 * blk, x);
                tc::wait_ld();
                full(blk, x);
            }
            tc::ld_x32(trow + 32 * wp, x);
            uint32_t pk[16];
            float ex[32];
            const float4* Gb = reinterpret_cast<const float4*>(G + 32 * wp);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 g4 = Gb[j];
                ex[4 * j] = scale * ex2(gi - g4.x);
                ex[4 * j + 1] = scale * ex2(gi - g4.y);
                ex[4 * j + 2] = scale * ex2(gi - g4.z);
                ex[4 * j + 3] = scale * ex2(gi - g4.w);
            }
            tc::wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
                const float y0 = j > lane ? 0.f : __uint_as_float(x[j]) * ex[j];
                const float y1 = j + 1 > lane ? 0.f : __uint_as_float(x[j + 1]) * ex[j + 1];
                pk[j / 2] = pack_bf16(y0, y1);
            }
            tc::st_x16(trow + 16 * wp, pk);
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = 0u;
#pragma unroll 1
            for (int blk = wp + 1; blk < 4; ++blk) tc::st_x16(trow + 16 * blk, pk);
            tc::wait_st();
            tc::fence_before_sync();
            arrive_warp(b.p, lane);
            arrive_warp(&b.dec_empty[buf], lane);
        }
    }
}

// x[c] += pj v[c] where v[c] is not finite, for 32 channels.
__device__ __forceinline__ void add_not_finite(uint32_t (&x)[32], const __nv_bfloat16* v, float pj, bool on) {
    if (!on) return;
#pragma unroll
    for (int ch = 0; ch < 4; ++ch) {
        const uint4 v4 = reinterpret_cast<const uint4*>(v)[ch];
        const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            uint32_t& o0 = x[8 * ch + 2 * r];
            uint32_t& o1 = x[8 * ch + 2 * r + 1];
            if ((vw[r] & 0x7f80u) == 0x7f80u)
                o0 = __float_as_uint(fmaf(pj, bf16_lo(vw[r]), __uint_as_float(o0)));
            if ((vw[r] & 0x7f800000u) == 0x7f800000u)
                o1 = __float_as_uint(fmaf(pj, bf16_hi(vw[r]), __uint_as_float(o1)));
        }
    }
}

// ------------------------------------------------------------ output warps
// Warp we: rows (tokens) 32 we .. + 31, one per lane.
__device__ __forceinline__ void output_role(const Kernel& p, const CUtensorMap* omap, uint8_t* smem, const Bars& b,
                                            uint32_t tmem, int we, int lane) {
    using M = Smem<false>;
    int* status = p.a.status;
    const volatile int* flag = reinterpret_cast<const volatile int*>(smem + M::kFlag);
    const int row = 32 * we + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * we) << 16);
    int64_t it = 0;
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
        const Unit w = unit_at<false>(p, u);
        for (int c = 0; c < w.nch; ++c, ++it) {
            const int s = static_cast<int>(it & 1);   // two stages, two decay buffers
            const uint32_t st = static_cast<uint32_t>(it >> 1) & 1u, ph = static_cast<uint32_t>(it & 1);
            uint8_t* Qrow = smem + M::kQ + s * kTile + row * 128;
            const int64_t vstride = p.a.H * kHeadDim;
            const __nv_bfloat16* v0 = static_cast<const __nv_bfloat16*>(p.a.v) +
                                      (w.tok0 + static_cast<int64_t>(c) * kC) * vstride + w.h * kHeadDim;
            const int valid = valid_of(w, c);
            // Q' in place, once D1 has been formed from Q.  The factor goes in
            // as two BF16 parts of one fused multiply-add: one rounding.
            if (!wait_phase(&b.dec_full[s], st, status)) return;
            const float e = p.a.scale * ex2(reinterpret_cast<const float*>(smem + M::kG)[s * kC + row]);
            arrive_warp(&b.dec_empty[s], lane);
            if (!wait_phase(&b.full_q[s], st, status) || !wait_phase(b.qk, ph, status)) return;
            const __nv_bfloat16 eh = __float2bfloat16_rn(e);
            const __nv_bfloat162 e1 = __bfloat162bfloat162(eh);
            const __nv_bfloat162 e2 = __bfloat162bfloat162(__float2bfloat16_rn(e - __bfloat162float(eh)));
#pragma unroll
            for (int sl = 0; sl < 2; ++sl) {
                uint4 v[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    v[x] = *reinterpret_cast<const uint4*>(Qrow + sl * kSlab + ((x ^ (row & 7)) << 4));
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v[x]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = __hfma2(h[j], e1, __hmul2(h[j], e2));
                    *reinterpret_cast<uint4*>(Qrow + sl * kSlab + ((x ^ (row & 7)) << 4)) = v[x];
                }
            }
            fence_proxy_async_smem();
            arrive_warp(b.q_scaled, lane);

            if (!wait_phase(b.o_done, ph, status)) return;
            tc::fence_after_sync();
            const bool bad = flag[s] == static_cast<int>(it + 1);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) +
                                 ((w.tok0 + static_cast<int64_t>(c) * kC + row) * p.a.H + w.h) * kHeadDim;
#pragma unroll 1
            for (int blk = 0; blk < 4; ++blk) {
                uint32_t x[32];
                tc::ld_x32(trow + kColO + 32 * blk, x);
                tc::wait_ld();
                if (bad) {
#pragma unroll 1
                    for (int j = 0; j < 32 * (we + 1); j += 2) {
                        uint32_t pp;
                        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];"
                                     : "=r"(pp) : "r"(trow + kColD1 + (j >> 1)));
                        tc::wait_ld();
                        add_not_finite(x, v0 + j * vstride + 32 * blk, bf16_lo(pp), j <= row && j < valid);
                        add_not_finite(x, v0 + (j + 1) * vstride + 32 * blk, bf16_hi(pp), j < row && j + 1 < valid);
                    }
                }
                if (blk == 3) {
                    // O and P are read, and V by every product.
                    tc::fence_before_sync();
                    arrive_warp(b.o_free, lane);
                    stage_release(&b.empty_v[s], lane);
                }
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) {
                    uint32_t y[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        y[r] = pack_bf16(__uint_as_float(x[8 * ch + 2 * r]), __uint_as_float(x[8 * ch + 2 * r + 1]));
                    const uint4 v = make_uint4(y[0], y[1], y[2], y[3]);
                    if (valid == kC)   // through Q's stage, which every product has read
                        *reinterpret_cast<uint4*>(Qrow + (blk >> 1) * kSlab + (((4 * (blk & 1) + ch) ^ (row & 7)) << 4)) = v;
                    else if (row < valid)
                        reinterpret_cast<uint4*>(out)[4 * blk + ch] = v;
                }
            }
            if (valid == kC) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    const uint8_t* src = smem + M::kQ + s * kTile + 32 * we * 128;
                    const int y = static_cast<int>(w.tok0 + static_cast<int64_t>(c) * kC + 32 * we);
                    const int x = static_cast<int>(w.h * kHeadDim);
                    tma_store_2d(omap, x, y, src);
                    tma_store_2d(omap, x + 64, y, src + kSlab);
                    bulk_commit();
                    bulk_wait_read_all();
                }
            }
            stage_release(&b.empty_q[s], lane);
        }
    }
    if (lane == 0) bulk_wait_all();
}

template <bool kStates>
__global__ void __launch_bounds__(kThreads, 1)
    la_kernel(const Kernel p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap) {
    using M = Smem<kStates>;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (p.a.valid && !*p.a.valid) return;
    if (smem_u32(smem) != kSmemBase) {   // the tiles' swizzle needs it; shared memory starts so
        if (threadIdx.x == 0) atomicOr(p.a.status, kDevPipeTimeout);
        return;
    }
    const Bars b = make_bars<kStates>(smem);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + M::kTmemPtr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < M::kStages; ++s) {
            mbar_init(&b.full_k[s], 1);
            mbar_init(&b.full_v[s], 1);
            mbar_init(&b.empty_k[s], kStates ? kStateWarps : kStateWarps + 1);
            mbar_init(&b.empty_v[s], kStates ? 1 : 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&b.full_q[s], 1);
            mbar_init(&b.empty_q[s], 4);
            mbar_init(&b.kp_full[s], kStateWarps);
            mbar_init(&b.kp_empty[s], 1);
            mbar_init(&b.dec_full[s], 1);
            mbar_init(&b.dec_empty[s], kStates ? kStateWarps : kStateWarps + 8);
        }
        mbar_init(b.qk, 1);
        mbar_init(b.p, 4);
        mbar_init(b.z_done, 1);
        mbar_init(b.checked, kStateWarps);
        mbar_init(b.s_ready, kStateWarps);
        mbar_init(b.qs_done, 1);
        mbar_init(b.q_scaled, 4);
        mbar_init(b.o_done, 1);
        mbar_init(b.o_free, 4);
        mbar_init(b.done, 1);
        reinterpret_cast<int*>(smem + M::kFlag)[0] = 0;
        reinterpret_cast<int*>(smem + M::kFlag)[1] = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tc::tmem_alloc(tmem_ptr, kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_ptr;

    if (warp < kStateWarps)
        state_role<kStates>(p, smem, b, tmem, warp, lane);
    else if (warp == kLoadWarp)
        load_role<kStates>(p, &qmap, &kmap, &vmap, smem, b, lane);
    else if (warp == kMmaWarp)
        mma_role<kStates>(p, smem, b, tmem, lane);
    else if (warp == kDecayWarp)
        decay_role<kStates>(p, smem, b, lane);
    else if (!kStates && warp < kOutWarp)
        score_role(p, smem, b, tmem, warp - kScoreWarp, lane);
    else if (!kStates)
        output_role(p, &omap, smem, b, tmem, warp - kOutWarp, lane);

    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// The segments' incoming states: per (sequence, head), S_0 = init and
// S_{j+1} = exp(D_j) S_j + Z_j, in place over Z.  A CTA has 1024 of the 16384
// elements; eight segments are loaded at a time.
constexpr int kScanThreads = 256, kScanParts = kHeadDim * kHeadDim / (4 * kScanThreads);
__global__ void __launch_bounds__(kScanThreads) la_scan_kernel(const Kernel p) {
    if (p.a.valid && !*p.a.valid) return;
    const int64_t unit = blockIdx.x / kScanParts;
    const int64_t n = unit / p.a.H, h = unit - n * p.a.H;
    const int64_t e = (blockIdx.x % kScanParts) * (4 * kScanThreads) + 4 * threadIdx.x;
    const int64_t s0 = p.sg.seg_begin ? p.sg.seg_begin[n] : n * p.sg.segs;
    const int64_t s1 = p.sg.seg_begin ? p.sg.seg_begin[n + 1] : s0 + p.sg.segs;
    constexpr int64_t kState = kHeadDim * kHeadDim;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.a.init_state) {
        if (p.a.state_f32) {
            s = *reinterpret_cast<const float4*>(static_cast<const float*>(p.a.init_state) + unit * kState + e);
        } else {
            const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.a.init_state) + unit * kState + e);
            s = make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
        }
    }
    if (s0 == s1 && p.a.final_state) {   // an empty sequence
        if (p.a.state_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.a.final_state) + unit * kState + e) = s;
        else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.final_state) + unit * kState + e) =
                make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
    }
    for (int64_t j0 = s0; j0 < s1; j0 += 8) {
        float4 z[8];
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j0 + i + 1 < s1) {
                z[i] = *reinterpret_cast<const float4*>(p.sg.starts + ((j0 + i) * p.a.H + h) * kState + e);
                d[i] = p.sg.decay[(j0 + i) * p.a.H + h];
            }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j0 + i < s1) {
                *reinterpret_cast<float4*>(p.sg.starts + ((j0 + i) * p.a.H + h) * kState + e) = s;
                if (j0 + i + 1 < s1) {
                    const float f = exp2f(d[i]);
                    s = make_float4(fmaf(f, s.x, z[i].x), fmaf(f, s.y, z[i].y), fmaf(f, s.z, z[i].z), fmaf(f, s.w, z[i].w));
                }
            }
    }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        else
            cudaGetLastError();
    });
    return fn;
}

// BF16 [tokens][heads * 128] in boxes of `rows` tokens x 64 channels.
cudaError_t encode_tokens(CUtensorMap* map, const void* base, int64_t tokens, int64_t heads, int rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    alignas(64) static const char kNone[16] = {};
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(heads * kHeadDim), static_cast<cuuint64_t>(tokens > 0 ? tokens : 1)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(heads * kHeadDim * 2)};
    const cuuint32_t box[2] = {64u, static_cast<cuuint32_t>(rows)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base ? base : kNone), dims, strides,
                           box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <bool kStates>
cudaError_t configure() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static bool configured[64] = {};
    if (configured[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(la_kernel<kStates>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(Smem<kStates>::kBytes));
    if (e == cudaSuccess) configured[dev] = true;
    return e;
}

}  // namespace

cudaError_t launch_la_prefill(const LaArgs& a, const LaSegments& sg, int sms, cudaStream_t stream, int* launches) {
    Kernel p;
    p.a = a;
    p.sg = sg;
    p.units = (sg.starts ? sg.total : a.N) * a.H;
    if (p.units <= 0) return cudaSuccess;
    CUtensorMap qm, km, vm, om;
    cudaError_t e;
    if ((e = configure<false>()) != cudaSuccess || (e = configure<true>()) != cudaSuccess) return e;
    if ((e = encode_tokens(&qm, a.q, a.tokens, a.Hk, kC)) != cudaSuccess ||
        (e = encode_tokens(&km, a.k, a.tokens, a.Hk, kC)) != cudaSuccess ||
        (e = encode_tokens(&vm, a.v, a.tokens, a.H, kC)) != cudaSuccess ||
        (e = encode_tokens(&om, a.out, a.tokens, a.H, 32)) != cudaSuccess)
        return e;
    const unsigned grid = static_cast<unsigned>(p.units < sms ? p.units : sms);
    if (sg.starts) {
        la_kernel<true><<<grid, kThreads, Smem<true>::kBytes, stream>>>(p, qm, km, vm, om);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        la_scan_kernel<<<static_cast<unsigned>(a.N * a.H * kScanParts), kScanThreads, 0, stream>>>(p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        *launches += 2;
    }
    la_kernel<false><<<grid, kThreads, Smem<false>::kBytes, stream>>>(p, qm, km, vm, om);
    *launches += 1;
    return cudaGetLastError();
}

}  // namespace kda
