// kda_la_prefill.cu -- linear attention with one decay per head and token,
// whole prompts, on the tcgen05 tensor cores (sm_103a):
//     S_t = exp(g_t) S_{t-1} + v_t k_t^T,  o_t = scale S_t q_t.
//
// A sequence is taken in chunks of 128 tokens.  With G_i the sum of the
// decays of the chunk's tokens up to i, G the chunk's whole sum and S the
// state before the chunk, the chunk's outputs and the state after it are
//     o_i = scale ( exp(G_i) S q_i + sum_{j <= i} exp(G_i - G_j) (q_i . k_j) v_j )
//     S   <- exp(G) S + sum_j exp(G - G_j) v_j k_j^T.
// Every exponent here is at most 0, whatever the decays are;
// exp(G - G_j) is formed from a sum that starts behind j, so that it is exact
// to FP32 even where G and G_j are large.
//
// As products of 128 x 128 tiles (i, j tokens; c value, d key channels):
//     D1[i][j]  = Q K^T
//     P[i][j]   = 2^e_i exp(-G_j) D1, causal, BF16, in tensor memory
//     O[i][c]   = scale r_i (Q' S^T + P V)   Q' = 2^e_i Q, S^T BF16 in shared memory
//     S^T[d][c] <- exp(G) S^T + K'^T V       K'^T[d][j] = exp(G - G_j) k_jd, in tensor memory
// with exp(G_i) = 2^e_i r_i: e_i is 0, and Q' is Q, down to a decay of 2^-48, and
// what of a row's exponent is below that: no factor of P is above 2^48, which
// leaves 2^79 for q, k and v, and Q' has the bits of Q.  Most chunks' queries
// need no pass over them: a chain of chunks 3% faster than with r_i in [1, 2).
// S^T is FP32 in tensor memory: the state warps read it, write its BF16 copy
// to shared memory and exp(G) S^T back, and K'^T V accumulates on that.
// K' is split by truncation into three BF16 parts whose sum is the FP32
// value, so the state is accurate to FP32: final states are off by 2e-7 to 4e-7 of
// their norm; with two parts (16 bits) a key is short of 2^-17 to 2^-16 of itself,
// always to one side, and states of random keys would be off by 1e-5.
// P and the S operand are rounded to BF16 once each: their error stays in the
// BF16 output they go to, which is off by 2.4e-3 of its norm where its own
// rounding alone is 1.7e-3, and S itself is not touched by it.
//
// One CTA per SM walks its units, a sequence's tokens or a part of them for one
// head.  Warps: 8 key (K'), 8 state (S), 4 score (P), 4 query (Q'), 4 output
// (O), one each for the loads, the MMA issue and the decay sums.  Tensor memory
// columns: D1 and P [0, 128), O [128, 256), S^T [256, 384), K' [384, 480) (two
// buffers of 32 tokens x 3 parts).
//
// Measured on GB300 (T = 8192; a call among others, and from a flushed L2): an
// uncut chain takes 2.35 us a chunk with one head (151 us), 2.6 with 96 (168, 175;
// floor 119 at a plain copy's 6.80 TB/s), of which the six products' MMA time is
// 1.6, and in which shared memory moves 480 KB, four fifths of its rate.  With 152
// heads, every SM loading, HBM's 2.9 us a chunk bind (199, 204 to 216; floor 188).
// 6 heads, cut into spans: 28, 37; floor 7.6.  The output kernels spill a little
// at their 64 registers: 28 bytes stored and 84 loaded in the fixed layout, 60 and
// 172 in the packed one.
//
// A value that is not finite must not reach earlier tokens of its chunk: a
// zero of P times an infinite V is NaN.  S^T shows it (its whole column is
// then not finite).  The state warps clear such values in shared memory once
// S^T has them, and the output warps add their products for j <= i alone,
// with V from global memory.
#include <cudaTypedefs.h>

#include <mutex>

#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_tcgen05.cuh"
#include "kda_wait.cuh"

namespace kda {
namespace {

constexpr int kC = kLaChunk;
constexpr uint32_t kSlab = 16384;   // 128 rows x 64 BF16, 128-byte swizzle
constexpr uint32_t kTile = 2 * kSlab;
// First warp of each role; 8 key, 8 state, 4 score, 4 query and 4 output warps.
constexpr int kStateWarp = 8, kScoreWarp = 16, kQueryWarp = 20, kOutWarp = 24, kLoadWarp = 28, kMmaWarp = 29, kDecayWarp = 30;
constexpr int kKeyWarps = 8, kStateWarps = 8;
constexpr int kThreads = 31 * 32;
constexpr uint32_t kColD1 = 0, kColO = 128, kColS = 256, kColK = 384, kTmemCols = 512;
constexpr uint32_t kKBuf = 48, kKPart = 16;   // K' buffer and part, in columns
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRowRange = 48.f;             // in base 2: a row's decay that P's factors make good
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
    static constexpr int kNumBars = 6 * kStages + 16;
    static constexpr uint32_t kFlag = kBars + 8 * kNumBars, kTmemPtr = kFlag + 8, kBytes = kTmemPtr + 8;
    static_assert(kBytes <= 232448, "shared memory of one CTA");
};

struct Bars {
    uint64_t *full_k, *full_v, *full_q, *empty_k, *empty_v, *empty_q;   // [stages], one after the other
    uint64_t *qk, *kp_full, *kp_empty, *z_done, *s_ready, *qs_ready, *qs_done, *pv_ready, *o_done;
    uint64_t *dec_full, *dec_empty, *done;
};
template <bool kStates>
__device__ __forceinline__ Bars make_bars(uint8_t* smem) {
    constexpr int n = Smem<kStates>::kStages;
    uint64_t* b = reinterpret_cast<uint64_t*>(smem + Smem<kStates>::kBars);
    Bars r;
    r.full_k = b;
    r.full_v = b + n;
    r.full_q = b + 2 * n;
    r.empty_k = b + 3 * n;
    r.empty_v = b + 4 * n;
    r.empty_q = b + 5 * n;
    b += 6 * n;
    r.qk = b;
    r.kp_full = b + 1;
    r.kp_empty = b + 3;
    r.z_done = b + 5;
    r.s_ready = b + 6;
    r.qs_ready = b + 7;
    r.qs_done = b + 8;
    r.pv_ready = b + 9;
    r.o_done = b + 10;
    r.dec_full = b + 11;
    r.dec_empty = b + 13;
    r.done = b + 15;
    return r;
}

struct Kernel {
    LaArgs a;
    LaSegments sg;      // sg.starts null: no cut
    uint32_t units, heads;
};
// What a CTA does: units of (sequence, head), one every grid's width; of
// (segment, head) for a fixed layout's cut; and for a packed batch's, decided on
// the device, the parts of its span, for one head.  The layout is a constant:
// with both in one kernel every role's code is longer, and a chunk slower by 1%.
template <bool kStates_, bool kPacked_>
struct Work {
    static constexpr bool kStates = kStates_, kPacked = kPacked_;
    const LaArgs& a;
    const LaSegments& sg;
    const uint32_t& heads;
    uint32_t base, step, end;
    bool cut;
    __device__ __forceinline__ explicit Work(const Kernel& p)
        : a(p.a), sg(p.sg), heads(p.heads), base(0), step(gridDim.x), end(p.units), cut(p.sg.starts) {
        if (kPacked) {
            cut = sg.cut && *sg.cut != 0;
            if (cut) {
                const uint32_t s = blockIdx.x / heads;
                step = 1;
                base = end = 0;
                if (s < sg.spans) {
                    base = sg.first[s];
                    end = sg.first[s + 1];
                    // Only a span's last part can go on in the next.
                    if (kStates && base < end) base = end - 1;
                }
            }
        }
    }
    // Of an uncut packed batch: its sequences, longest first (or null).
    __device__ __forceinline__ const int32_t* order() const { return !kPacked || cut ? nullptr : sg.order; }
    // The CTA's i-th unit: in rows of the grid's width, where the units come
    // longest first every other row backwards.
    __device__ __forceinline__ uint32_t unit(uint32_t i) const {
        const uint32_t at = !kPacked || step > 1 ? blockIdx.x : 0;
        return base + i * step + ((i & 1) && order() ? step - 1 - at : at);
    }
    __device__ __forceinline__ uint32_t rows() const { return (end - base + step - 1) / step; }
};

// One (sequence or part of one, head).
struct Unit {
    int n, h, tok0, len;
    uint32_t slot;      // (span, head) row of the spans' buffers
    bool mid;           // goes on from the span before
    bool last;          // writes the final state
    int nch;
};
template <class Work>
__device__ __forceinline__ Unit unit_at(const Work& p, uint32_t u) {
    Unit w;
    if (Work::kPacked && p.cut) {
        const int4 part = p.sg.part[u];
        w.n = part.x;
        w.h = blockIdx.x % p.heads;
        w.tok0 = part.y;
        w.len = part.z;
        w.slot = blockIdx.x;
        w.mid = part.w & kLaMid;
        w.last = part.w & kLaLast;
    } else {
        const uint32_t s = u / p.heads;
        w.h = u - s * p.heads;
        w.slot = u;
        w.mid = false;
        w.last = true;
        if (Work::kPacked) {
            w.n = p.order() ? p.order()[s] : s;
            w.tok0 = static_cast<int>(p.a.cu_seqlens[w.n]);
            w.len = static_cast<int>(p.a.cu_seqlens[w.n + 1]) - w.tok0;
        } else if (p.cut) {
            const uint32_t segs = static_cast<uint32_t>(p.sg.segs);
            const int each = static_cast<int>(p.sg.seg_tokens_each), per = static_cast<int>(p.a.tokens_per_seq);
            w.n = s / segs;
            const int j = s - w.n * segs;
            w.tok0 = w.n * per + j * each;
            w.mid = j > 0;
            w.last = j + 1 == static_cast<int>(segs);
            w.len = w.last ? per - j * each : each;
        } else {
            w.n = s;
            w.len = static_cast<int>(p.a.tokens_per_seq);
            w.tok0 = s * w.len;
        }
    }
    if (Work::kStates && w.last) w.len = 0;     // nothing of the sequence follows
    w.nch = (w.len + kC - 1) / kC;
    return w;
}

// A chunk's place in the rings: the chunk's number on this CTA, its stage and
// the parity of the stage's use.
// (With two stages both are bits of the number: fewer registers to keep.)
template <int kStages>
struct Pos {
    uint32_t it = 0, st_ = 0;
    int s_ = 0;
    __device__ __forceinline__ void next() {
        ++it;
        if (kStages != 2 && ++s_ == kStages) {
            s_ = 0;
            st_ ^= 1u;
        }
    }
    __device__ __forceinline__ int s() const { return kStages == 2 ? static_cast<int>(it & 1u) : s_; }
    __device__ __forceinline__ uint32_t st() const { return kStages == 2 ? (it >> 1) & 1u : st_; }
    __device__ __forceinline__ uint32_t ph() const { return it & 1u; }            // once a chunk
    __device__ __forceinline__ uint32_t dec_ph() const { return (it >> 1) & 1u; }   // two buffers
};

// f(unit, chunk, valid tokens, place) for every chunk of this CTA, until it fails.
template <class Work, class F>
__device__ __forceinline__ void walk(const Work& p, F f) {
    Pos<Smem<Work::kStates>::kStages> x;
#pragma unroll 1
    for (uint32_t i = 0; i < p.rows(); ++i) {
        if (p.unit(i) >= p.end) continue;
        const Unit w = unit_at(p, p.unit(i));
#pragma unroll 1
        for (int c = 0; c < w.nch; ++c) {
            if (!f(w, c, min(kC, w.len - c * kC), x)) return;
            x.next();
        }
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// e_i of a row.
__device__ __forceinline__ float row_shift(float g) { return fminf(floorf(g) + kRowRange, 0.f); }
__device__ __forceinline__ uint32_t prmt_hi(uint32_t lo, uint32_t hi) {   // the upper halves of two words
    return __byte_perm(lo, hi, 0x7632);
}
__device__ __forceinline__ void tma_store_2d(const void* tmap, int32_t x, int32_t y, const void* src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(tmap), "r"(x), "r"(y), "r"(smem_u32(src)) : "memory");
}
// Shared-memory descriptors as (low word, constant high word): the low word
// is the start address over 16 and the leading offset, so a step inside a
// tile is an addition.  K-major operands (128-byte swizzle): 8-row groups
// 1024 B apart.  Operands whose N index is contiguous: rows of 64 elements of
// it, 8-row groups of K 1024 B apart, the next 64 elements one slab (the
// leading offset) further.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (tc::kSwizzle128B << 29);
constexpr uint32_t kLeadK = 1u << 16, kLeadMn = (kSlab >> 4) << 16;
__host__ __device__ constexpr uint32_t k_step(int k) { return ((k >> 2) * kSlab + 32 * (k & 3)) >> 4; }   // K-major, 16 elements
__host__ __device__ constexpr uint32_t mn_step(int k) { return (k * 2048) >> 4; }                        // 16 rows
constexpr uint32_t kIdesc = tc::idesc_bf16(128, 128);
constexpr uint32_t kIdescMn = kIdesc | (1u << 16);   // B is MN-major
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
__device__ __forceinline__ void ld_x8(uint32_t taddr, uint32_t (&r)[8]) { tc::ld_x8(taddr, r); }
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
template <class Work>
__device__ __forceinline__ void load_role(const Work& p, const CUtensorMap* qmap, const CUtensorMap* kmap,
                                          const CUtensorMap* vmap, uint8_t* smem, const Bars& b, int lane) {
    constexpr bool kStates = Work::kStates;
    using M = Smem<kStates>;
    constexpr int n = M::kStages, tiles = kStates ? 2 : 3;
    const uint32_t group = static_cast<uint32_t>(p.a.H / p.a.Hk);
    uint32_t issued = 0;   // tiles under way or done, K, V, Q, K, ..
    walk(p, [&](const Unit& w, int c, int, const Pos<n>& x) {
        const int y = w.tok0 + c * kC;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            // (The barriers and tiles of K, V and Q follow one another.)
            if (x.it >= n && !wait_phase(&b.empty_k[t * n + x.s()], x.st() ^ 1u, p.a.status)) return false;
            if (lane == 0) {
                uint64_t* full = &b.full_k[t * n + x.s()];
                uint8_t* dst = smem + (t * n + x.s()) * kTile;
                const CUtensorMap* map = t == 0 ? kmap : t == 1 ? vmap : qmap;
                const int col = static_cast<int>(t == 1 ? w.h : w.h / group) * kHeadDim;
                mbar_arrive_expect_tx(full, kTile);
                tma_load_2d(dst, map, col, y, full);
                tma_load_2d(dst + kSlab, map, col + 64, y, full);
            }
            ++issued;
            __syncwarp();
        }
        return true;
    });
    // No copy may be under way when the CTA ends: the last uses of each stage.
#pragma unroll 1
    for (uint32_t i = issued > tiles * n ? issued - tiles * n : 0; i < issued; ++i) {
        const uint32_t it = i / tiles, t = i % tiles;
        if (!wait_phase(&b.full_k[t * n + it % n], (it / n) & 1u, p.a.status)) break;
    }
}

// -------------------------------------------------------------- decay warp
// The decays are single words, a row of heads apart: on a loaded memory
// system a load takes 3 us and more, so the lines are brought to L2 four
// chunks ahead and the words one chunk ahead.
template <class Work>
__device__ __forceinline__ void decay_role(const Work& p, uint8_t* smem, const Bars& b, int lane) {
    constexpr bool kStates = Work::kStates;
    using M = Smem<kStates>;
    constexpr int kAhead = 4;
    float next[4] = {0.f, 0.f, 0.f, 0.f};
    walk(p, [&](const Unit& w, int c, int valid, const Pos<M::kStages>& at) {
        const uint32_t buf = at.it & 1u;
        const int64_t stride = p.a.g_stride;
        // This lane's four tokens of chunk i: up to `left` of them are there.
        auto source = [&](int i) { return p.a.g + static_cast<int64_t>(w.tok0 + i * kC + 4 * lane) * stride + w.h; };
        auto fetch = [&](int i) {
            const int left = w.len - i * kC - 4 * lane;
            const float* src = source(i);
#pragma unroll
            for (int r = 0; r < 4; ++r) next[r] = r < left ? src[r * stride] : 0.f;
        };
        auto prefetch = [&](int i) {
            const int left = w.len - i * kC - 4 * lane;
            const float* src = source(i);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + r * stride));
        };
        if (c == 0) {
            fetch(0);
#pragma unroll 1
            for (int i = 1; i < kAhead; ++i) prefetch(i);
        }
        prefetch(c + kAhead);
        float x[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            x[r] = next[r] * kLog2e;
            if (x[r] < kMinDecay) x[r] = kMinDecay;   // -inf too; NaN stays
        }
        fetch(c + 1);
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
#pragma unroll 1
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
            wt[r] = 4 * lane + r < valid ? ex2(behind + suf[r]) : 0.f;
            cf[r] = ex2(ref - g[r]);
        }
        if (at.it >= 2 && !wait_phase(&b.dec_empty[buf], at.dec_ph() ^ 1u, p.a.status)) return false;
        *reinterpret_cast<float4*>(smem + M::kG + buf * kC * 4 + 16 * lane) = make_float4(g[0], g[1], g[2], g[3]);
        *reinterpret_cast<float4*>(smem + M::kW + buf * kC * 4 + 16 * lane) = make_float4(wt[0], wt[1], wt[2], wt[3]);
        if (lane < 24)
            *reinterpret_cast<float4*>(smem + M::kCf + buf * 96 * 4 + 16 * lane) = make_float4(cf[0], cf[1], cf[2], cf[3]);
        arrive_warp(&b.dec_full[buf], lane);
        return true;
    });
}

// ---------------------------------------------------------------- MMA warp
// Per chunk: D1, K'^T V in quarters of 32 tokens, Q' S^T, P V.  D1 overwrites
// the P of the chunk before, whose product it waits for; P and Q' are formed
// while K'^T V runs, and the next chunk's state between Q' S^T and its K'^T V.
template <class Work>
__device__ __forceinline__ void mma_role(const Work& p, uint8_t* smem, const Bars& b, uint32_t tmem, int lane) {
    constexpr bool kStates = Work::kStates;
    using M = Smem<kStates>;
    constexpr int n = M::kStages;
    int* status = p.a.status;
    const volatile uint32_t* flag = reinterpret_cast<const volatile uint32_t*>(smem + M::kFlag);
    const bool leader = elect_one();
    const uint32_t base = (smem_u32(smem) >> 4) & 0x3FFFu, ds = base + (M::kS >> 4) + kLeadMn;
    walk(p, [&](const Unit&, int c, int, const Pos<n>& x) {
        const uint32_t ph = x.ph(), pv = ph ^ 1u, it = x.it;
        const uint32_t tile = base + x.s() * (kTile >> 4);
        const uint32_t dk = tile + (M::kK >> 4) + kLeadK, dv = tile + (M::kV >> 4) + kLeadMn, dq = tile + (M::kQ >> 4) + kLeadK;
        if (!wait_phase(&b.full_k[x.s()], x.st(), status)) return false;
        if (!kStates) {
            if (!wait_phase(&b.full_q[x.s()], x.st(), status)) return false;
            if (it > 0) {
                if (!wait_phase(b.o_done, pv, status)) return false;
                // P is read once more where V is not finite: until V's stage is released.
                if (flag[pv] == it && !wait_phase(&b.empty_v[x.s() ^ 1], x.s() ? x.st() : x.st() ^ 1u, status)) return false;
            }
            tc::fence_after_sync();
            if (leader) {
#pragma unroll
                for (int k = 0; k < 8; ++k) mma_ss<kIdesc>(tmem + kColD1, dq + k_step(k), dk + k_step(k), k > 0);
                tc::commit(b.qk);
                tc::commit(&b.empty_k[x.s()]);
            }
            __syncwarp();
        }
        if (!wait_phase(&b.full_v[x.s()], x.st(), status) || !wait_phase(b.s_ready, ph, status)) return false;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            if (!wait_phase(&b.kp_full[q & 1], q >> 1, status)) return false;   // two uses a chunk
            tc::fence_after_sync();
            if (leader) {
                const uint32_t kp = tmem + kColK + kKBuf * (q & 1), v = dv + q * mn_step(2);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int part = 0; part < 3; ++part)
                        mma_ts<kIdescMn>(tmem + kColS, kp + kKPart * part + 8 * t, v + mn_step(t),
                                         t + part > 0 ? 1u : static_cast<uint32_t>(!kStates || c + q > 0));
                tc::commit(&b.kp_empty[q & 1]);
                if (q == 3) {
                    tc::commit(b.z_done);
                    if (kStates) tc::commit(&b.empty_v[x.s()]);
                }
            }
            __syncwarp();
        }
        if (kStates) return true;
        if (!wait_phase(b.qs_ready, ph, status)) return false;
        tc::fence_after_sync();
        if (leader) {
#pragma unroll
            for (int k = 0; k < 8; ++k) mma_ss<kIdescMn>(tmem + kColO, dq + k_step(k), ds + mn_step(k), k > 0);
            tc::commit(b.qs_done);
        }
        __syncwarp();
        if (!wait_phase(b.pv_ready, ph, status)) return false;
        tc::fence_after_sync();
        if (leader) {
#pragma unroll
            for (int k = 0; k < 8; ++k) mma_ts<kIdescMn>(tmem + kColO, tmem + kColD1 + 8 * k, dv + mn_step(k), 1u);
            tc::commit(b.o_done);
        }
        __syncwarp();
        return true;
    });
    // Every MMA must be complete before tensor memory is released.
    if (leader) tc::commit(b.done);
    __syncwarp();
    wait_phase(b.done, 0, status);
}

// --------------------------------------------------------------- key warps
// Warp wk: key channels 32 (wk % 4) .. + 31 (the tensor-memory lanes it may
// access) of the 16 tokens 16 (wk / 4) .. of each 32.  Transposing matrix loads
// give a thread the same key channel of two neighbouring tokens in a word,
// which is how the A operand wants them.
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// 16 lanes x 8 columns: words (lane / 4, lane % 4) of the 8 x 4 blocks (rows
// 0-7, 8-15) of columns 0-3, then of columns 4-7.
__device__ __forceinline__ void st_16x8(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

template <class Work>
__device__ __forceinline__ void key_role(const Work& p, uint8_t* smem, const Bars& b, uint32_t tmem, int wk, int lane) {
    constexpr bool kStates = Work::kStates;
    using M = Smem<kStates>;
    constexpr int n = M::kStages;
    int* status = p.a.status;
    const int half = wk >> 2, kg = 4 * (wk & 3) + (lane >> 3);
    const uint32_t src0 = smem_u32(smem) + M::kK + (kg >> 3) * kSlab + (16 * half + (lane & 7)) * 128 +
                          (((kg & 7) ^ (lane & 7)) << 4);
    const uint32_t dst = tmem + (static_cast<uint32_t>(32 * (wk & 3)) << 16) + kColK + 8 * half;
    const int tok = 16 * half + 2 * (lane & 3);
    walk(p, [&](const Unit&, int, int valid, const Pos<n>& x) {
        const uint32_t buf = x.it & 1u;
        if (!wait_phase(&b.full_k[x.s()], x.st(), status) || !wait_phase(&b.dec_full[buf], x.dec_ph(), status)) return false;
        if (valid < kC) {
            // Rows behind the sequence's end: another sequence's tokens, or
            // anything.  V's are cleared here, K's below.
            uint8_t* V = smem + M::kV + x.s() * kTile;
            if (!wait_phase(&b.full_v[x.s()], x.st(), status)) return false;
#pragma unroll 1
            for (int r = valid + wk; r < kC; r += kKeyWarps)
                if (lane < 16)
                    *reinterpret_cast<uint4*>(V + (lane >> 3) * kSlab + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
        }
        const uint32_t src = src0 + x.s() * kTile;
        const float* W = reinterpret_cast<const float*>(smem + M::kW) + buf * kC + tok;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
            // Three truncated parts of k w: the upper halves of k w, of what
            // is left, and of what is left then.
            uint32_t part[3][2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t r[4];
                ldsm_x4_t(r, src + (32 * q + 8 * t) * 128);
                const float2 w2 = *reinterpret_cast<const float2*>(W + 32 * q + 8 * t);
                // (Tokens behind the end: k is cleared, w is 0.)
                const int left = valid - (32 * q + 8 * t + tok);
                const uint32_t keep = left > 1 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    r[m] &= keep;
                    float x0 = bf16_lo(r[m]), x1 = bf16_hi(r[m]);
                    mul2v(x0, x1, w2.x, w2.y);
                    const uint32_t a0 = __float_as_uint(x0), a1 = __float_as_uint(x1);
                    sub2(x0, x1, __uint_as_float(a0 & 0xffff0000u), __uint_as_float(a1 & 0xffff0000u));
                    const uint32_t b0 = __float_as_uint(x0), b1 = __float_as_uint(x1);
                    sub2(x0, x1, __uint_as_float(b0 & 0xffff0000u), __uint_as_float(b1 & 0xffff0000u));
                    part[0][t][m] = prmt_hi(a0, a1);
                    part[1][t][m] = prmt_hi(b0, b1);
                    part[2][t][m] = prmt_hi(__float_as_uint(x0), __float_as_uint(x1));
                }
            }
            const uint32_t use = 2 * x.it + (q >> 1);
            if (use > 0 && !wait_phase(&b.kp_empty[q & 1], (use - 1) & 1u, status)) return false;
            tc::fence_after_sync();
            const uint32_t col = dst + kKBuf * (q & 1);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                st_16x8(col + kKPart * i, part[i][0][0], part[i][0][1], part[i][1][0], part[i][1][1]);
                st_16x8(col + kKPart * i + (16u << 16), part[i][0][2], part[i][0][3], part[i][1][2], part[i][1][3]);
            }
            tc::wait_st();
            tc::fence_before_sync();
            arrive_warp(&b.kp_full[q & 1], lane);
        }
        stage_release(&b.empty_k[x.s()], lane);
        arrive_warp(&b.dec_empty[buf], lane);
        return true;
    });
}

// ------------------------------------------------------------- state warps
// Warp ws: key channels 32 (ws % 4) .. + 31, one per lane (the tensor-memory
// lanes it may access); value channels 64 (ws / 4) .. + 63.
//
// The paths that run once per unit, or never on finite values, are calls with
// short loops: they stay out of the instruction cache's way.

// Clears the values that are not finite in two 16-byte columns of a slab of
// V, with one warp; true if there were any.
__device__ __noinline__ bool clear_not_finite(uint8_t* slab, int chunk, int lane) {
    bool any = false;
#pragma unroll 1
    for (int r = lane; r < kC; r += 32)
#pragma unroll 1
        for (int x = 0; x < 8; ++x) {
            uint32_t* at = reinterpret_cast<uint32_t*>(slab + r * 128 + (((chunk + (x >> 2)) ^ (r & 7)) << 4)) + (x & 3);
            uint32_t v = *at;
            if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
            if ((v & 0x7f800000u) == 0x7f800000u) v &= 0xffffu;
            any |= v != *at;
            *at = v;
        }
    return __any_sync(0xffffffffu, any);
}
__device__ __forceinline__ float load_elem(const void* base, bool f32, int64_t at) {
    if (!base) return 0.f;
    return f32 ? static_cast<const float*>(base)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
}
__device__ __forceinline__ void store_elem(void* base, bool f32, int64_t at, float x) {
    if (f32)
        static_cast<float*>(base)[at] = x;
    else
        static_cast<__nv_bfloat16*>(base)[at] = __float2bfloat16_rn(x);
}
// This thread's 64 value channels of a state in global memory ([value][key];
// zeros for none): into tensor memory, and back.  The loads of 32 channels are
// under way at once: one after the other they took 6 us.
__device__ __noinline__ void state_in(const void* base, bool f32, int64_t at, uint32_t scol) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i, at += 32 * kHeadDim) {
        uint32_t x[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = 0u;
        if (base && f32) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = static_cast<const uint32_t*>(base)[at + j * kHeadDim];
        } else if (base) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = static_cast<const uint16_t*>(base)[at + j * kHeadDim];
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] <<= 16;
        }
        tc::st_x32(scol + 32 * i, x);
    }
    tc::wait_st();
}
__device__ __noinline__ void state_out(void* base, bool f32, int64_t at, uint32_t scol) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i, at += 32 * kHeadDim) {
        uint32_t x[32];
        tc::ld_x32(scol + 32 * i, x);
        tc::wait_ld();
        if (f32) {
#pragma unroll
            for (int j = 0; j < 32; ++j) static_cast<uint32_t*>(base)[at + j * kHeadDim] = x[j];
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                static_cast<__nv_bfloat16*>(base)[at + j * kHeadDim] = __float2bfloat16_rn(__uint_as_float(x[j]));
        }
    }
}

template <class Work>
__device__ __forceinline__ void state_role(const Work& p, uint8_t* smem, const Bars& b, uint32_t tmem, int ws, int lane) {
    constexpr bool kStates = Work::kStates;
    using M = Smem<kStates>;
    constexpr int n = M::kStages;
    int* status = p.a.status;
    volatile uint32_t* flag = reinterpret_cast<volatile uint32_t*>(smem + M::kFlag);
    const int half = ws >> 2, key = 32 * (ws & 3) + lane;
    const uint32_t scol = tmem + (static_cast<uint32_t>(32 * (ws & 3)) << 16) + kColS + 64 * half;
    uint8_t* row = smem + M::kS + half * kSlab + key * 128;
    const int64_t lane_at = 64 * half * kHeadDim + key;
    Pos<n> x;
#pragma unroll 1
    for (uint32_t row_i = 0; row_i < p.rows(); ++row_i) {
        if (p.unit(row_i) >= p.end) continue;
        const Unit w = unit_at(p, p.unit(row_i));
        // (Offsets are formed where they are used: held over the chunks they cost
        // spilled registers.)
        auto own_at = [&] { return (static_cast<int64_t>(w.n) * p.a.H + w.h) * (kHeadDim * kHeadDim) + lane_at; };
        auto slot_at = [&](uint32_t slot) { return static_cast<int64_t>(slot) * (kHeadDim * kHeadDim) + lane_at; };
        if (w.nch == 0) {
            if (!kStates && w.last && p.a.final_state)
#pragma unroll 1
                for (int i = 0; i < 64; ++i)
                    store_elem(p.a.final_state, p.a.state_f32, own_at() + i * kHeadDim,
                               load_elem(p.a.init_state, p.a.state_f32, own_at() + i * kHeadDim));
            continue;
        }
        if (!kStates) {
            // (Where final states overwrite the initial ones, a sequence's last
            // part may be done before its first has begun.)
            const bool copied = p.sg.inits && !w.last;
            if (w.mid)
                state_in(p.sg.starts, true, slot_at(w.slot), scol);
            else
                state_in(copied ? p.sg.inits : p.a.init_state, copied || p.a.state_f32, own_at(), scol);
        }
        float total = 0.f;
#pragma unroll 1
        for (int c = 0; c < w.nch; ++c, x.next()) {
            const uint32_t buf = x.it & 1u, ph = x.ph();
            if (!wait_phase(&b.dec_full[buf], x.dec_ph(), status)) return;
            const float sum = reinterpret_cast<const float*>(smem + M::kG)[buf * kC + kC - 1];
            arrive_warp(&b.dec_empty[buf], lane);
            const float d = ex2(sum);
            total += sum;
            // The state before this chunk: its BF16 copy as the B operand of
            // Q' S^T (row d: 128 value channels), once the last chunk's
            // product has read its own, and the decayed state.
            if (!kStates && x.it > 0 && !wait_phase(b.qs_done, ph ^ 1u, status)) return;
            tc::fence_after_sync();
            if (!kStates || c > 0) {
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    uint32_t r[32];
                    tc::ld_x32(scol + 32 * i, r);
                    tc::wait_ld();
                    if (!kStates)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                y[e] = pack_bf16(__uint_as_float(r[8 * j + 2 * e]), __uint_as_float(r[8 * j + 2 * e + 1]));
                            *reinterpret_cast<uint4*>(row + (((4 * i + j) ^ (key & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float y0 = __uint_as_float(r[j]), y1 = __uint_as_float(r[j + 1]);
                        mul2(y0, y1, d);
                        r[j] = __float_as_uint(y0);
                        r[j + 1] = __float_as_uint(y1);
                    }
                    tc::st_x32(scol + 32 * i, r);
                }
            }
            if (!kStates) fence_proxy_async_smem();
            tc::wait_st();
            tc::fence_before_sync();
            arrive_warp(b.s_ready, lane);
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
                    // The flag of a chunk is its number + 1, so none has to be cleared.
                    if (clear_not_finite(smem + M::kV + x.s() * kTile + half * kSlab, 2 * (ws & 3), lane) && lane == 0)
                        flag[buf] = x.it + 1;
                    fence_proxy_async_smem();
                    __threadfence_block();
                }
                arrive_warp(b.pv_ready, lane);
            }
        }
        if (kStates) {
            // (For the next span of this head.)
            state_out(p.sg.starts, true, slot_at(w.slot + p.heads), scol);
            if (ws == 0 && lane == 0) p.sg.decay[w.slot + p.heads] = total;
        } else if (w.last && p.a.final_state) {
            state_out(p.a.final_state, p.a.state_f32, own_at(), scol);
        }
        tc::fence_before_sync();
    }
}

// ------------------------------------------------------------- score warps
// Warp wp: rows (tokens) 32 wp .. + 31, one per lane.  Blocks of 32 columns
// before the row's own take 2^e_i exp(-G_j) as a row factor to the end of the
// block times a column factor from there, at most 2^48 and 1: one exponential
// per row and block instead of one per score.
template <class Work>
__device__ __forceinline__ void score_role(const Work& p, uint8_t* smem, const Bars& b, uint32_t tmem, int wp, int lane) {
    using M = Smem<false>;
    int* status = p.a.status;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * wp) << 16) + kColD1;
    walk(p, [&](const Unit&, int, int, const Pos<2>& at) {
        const uint32_t buf = at.it & 1u;
        const float* G = reinterpret_cast<const float*>(smem + M::kG) + buf * kC;
        const float4* Cf = reinterpret_cast<const float4*>(smem + M::kCf + buf * 96 * 4);
        if (!wait_phase(&b.dec_full[buf], at.dec_ph(), status)) return false;
        const float gi = row_shift(G[32 * wp + lane]);
        if (!wait_phase(b.qk, at.ph(), status)) return false;
        tc::fence_after_sync();
        // A block's columns of P, 16 blk .. + 15, held scores of blocks read
        // before it.
        uint32_t x[32];
#pragma unroll 1
        for (int blk = 0; blk < wp; ++blk) {
            tc::ld_x32(trow + 32 * blk, x);
            const float f = ex2(gi - G[32 * blk + 31]);
            tc::wait_ld();
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
        }
        const float4* Gb = reinterpret_cast<const float4*>(G + 32 * wp);
        tc::ld_x32(trow + 32 * wp, x);
        tc::wait_ld();
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float4 g4 = Gb[j];
            const float gj[4] = {g4.x, g4.y, g4.z, g4.w};
            float y[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                y[r] = 4 * j + r > lane ? 0.f : __uint_as_float(x[4 * j + r]) * ex2(gi - gj[r]);
            pk[2 * j] = pack_bf16(y[0], y[1]);
            pk[2 * j + 1] = pack_bf16(y[2], y[3]);
        }
        tc::st_x16(trow + 16 * wp, pk);
#pragma unroll
        for (int j = 0; j < 16; ++j) pk[j] = 0u;
#pragma unroll 1
        for (int blk = wp + 1; blk < 4; ++blk) tc::st_x16(trow + 16 * blk, pk);
        tc::wait_st();
        tc::fence_before_sync();
        arrive_warp(b.pv_ready, lane);
        arrive_warp(&b.dec_empty[buf], lane);
        return true;
    });
}

// ------------------------------------------------------------- query warps
// Warp wq: rows (tokens) 32 wq .. + 31, one per lane.  Q' in place, once D1
// has been formed from Q.
template <class Work>
__device__ __forceinline__ void query_role(const Work& p, uint8_t* smem, const Bars& b, int wq, int lane) {
    using M = Smem<false>;
    int* status = p.a.status;
    const int row = 32 * wq + lane;
    walk(p, [&](const Unit&, int, int, const Pos<2>& at) {
        const uint32_t buf = at.it & 1u;
        uint8_t* Qrow = smem + M::kQ + at.s() * kTile + row * 128;
        if (!wait_phase(&b.dec_full[buf], at.dec_ph(), status)) return false;
        const float shift = row_shift(reinterpret_cast<const float*>(smem + M::kG)[buf * kC + row]);
        arrive_warp(&b.dec_empty[buf], lane);
        const __nv_bfloat162 e2 = __bfloat162bfloat162(__float2bfloat16_rn(ex2(shift)));
        if (!wait_phase(&b.full_q[at.s()], at.st(), status) || !wait_phase(b.qk, at.ph(), status)) return false;
        const int slabs = __any_sync(0xffffffffu, shift < 0.f) ? 2 : 0;
#pragma unroll 1
        for (int sl = 0; sl < slabs; ++sl, Qrow += kSlab) {
            uint4 v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) v[x] = *reinterpret_cast<const uint4*>(Qrow + ((x ^ (row & 7)) << 4));
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&v[x]);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = __hmul2(h[j], e2);
                *reinterpret_cast<uint4*>(Qrow + ((x ^ (row & 7)) << 4)) = v[x];
            }
        }
        if (slabs) fence_proxy_async_smem();
        arrive_warp(b.qs_ready, lane);
        return true;
    });
}

// ------------------------------------------------------------ output warps
// Warp we: rows (tokens) 32 we .. + 31, one per lane.

// Adds P_ij v_j to this row's O where v_j is not finite, for j <= i.
// v: the chunk's first token of this head in global memory.
__device__ __noinline__ void add_not_finite(uint32_t trow, const __nv_bfloat16* v, int64_t vstride, int row, int valid) {
    const int first = row & ~31;
#pragma unroll 1
    for (int col = 0; col < kHeadDim; col += 8) {
        uint32_t x[8];
        ld_x8(trow + kColO + col, x);
        tc::wait_ld();
#pragma unroll 1
        for (int j = 0; j < first + 32; ++j) {
            uint32_t pp;
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(pp) : "r"(trow + kColD1 + (j >> 1)));
            tc::wait_ld();
            if (j <= row && j < valid) {
                const float pj = j & 1 ? bf16_hi(pp) : bf16_lo(pp);
                const uint4 v4 = *reinterpret_cast<const uint4*>(v + j * vstride + col);
                const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if ((vw[r] & 0x7f80u) == 0x7f80u)
                        x[2 * r] = __float_as_uint(fmaf(pj, bf16_lo(vw[r]), __uint_as_float(x[2 * r])));
                    if ((vw[r] & 0x7f800000u) == 0x7f800000u)
                        x[2 * r + 1] = __float_as_uint(fmaf(pj, bf16_hi(vw[r]), __uint_as_float(x[2 * r + 1])));
                }
            }
            __syncwarp();
        }
        st_x8(trow + kColO + col, x);
    }
    tc::wait_st();
}

template <class Work>
__device__ __forceinline__ void output_role(const Work& p, const CUtensorMap* omap, uint8_t* smem, const Bars& b,
                                            uint32_t tmem, int we, int lane) {
    using M = Smem<false>;
    int* status = p.a.status;
    const volatile uint32_t* flag = reinterpret_cast<const volatile uint32_t*>(smem + M::kFlag);
    const int row = 32 * we + lane;
    const uint32_t trow = tmem + (static_cast<uint32_t>(32 * we) << 16);
    arrive_warp(b.qs_ready, lane);   // O is free for the first chunk
    walk(p, [&](const Unit& w, int c, int valid, const Pos<2>& at) {
        uint8_t* Qrow = smem + M::kQ + at.s() * kTile + row * 128;
        // The chunk's first token of this head, in V and the output.
        auto first = [&]() { return (w.tok0 + c * kC) * p.a.H * kHeadDim + w.h * kHeadDim; };
        const uint32_t buf = at.it & 1u;
        if (!wait_phase(&b.dec_full[buf], at.dec_ph(), status)) return false;
        const float gi = reinterpret_cast<const float*>(smem + M::kG)[buf * kC + row];
        arrive_warp(&b.dec_empty[buf], lane);
        const float f = p.a.scale * ex2(gi - row_shift(gi));
        if (!wait_phase(b.o_done, at.ph(), status)) return false;
        tc::fence_after_sync();
        if (flag[at.it & 1u] == at.it + 1)
            add_not_finite(trow, static_cast<const __nv_bfloat16*>(p.a.v) + first(), p.a.H * kHeadDim, row, valid);
        stage_release(&b.empty_v[at.s()], lane);
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
            uint32_t x[32];
            tc::ld_x32(trow + kColO + 32 * blk, x);
            tc::wait_ld();
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float y0 = __uint_as_float(x[2 * r]), y1 = __uint_as_float(x[2 * r + 1]);
                mul2(y0, y1, f);
                x[r] = pack_bf16(y0, y1);
            }
            if (valid == kC) {   // through Q's stage, which every product has read
                uint8_t* slab = Qrow + (blk >> 1) * kSlab;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch)
                    *reinterpret_cast<uint4*>(slab + (((4 * (blk & 1) + ch) ^ (row & 7)) << 4)) =
                        make_uint4(x[4 * ch], x[4 * ch + 1], x[4 * ch + 2], x[4 * ch + 3]);
            } else if (row < valid) {
                uint4* out = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.a.out) + first() + row * p.a.H * kHeadDim) + 4 * blk;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) out[ch] = make_uint4(x[4 * ch], x[4 * ch + 1], x[4 * ch + 2], x[4 * ch + 3]);
            }
        }
        tc::fence_before_sync();
        arrive_warp(b.qs_ready, lane);   // O and P are read
        if (valid == kC) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                const uint8_t* src = smem + M::kQ + at.s() * kTile + 32 * we * 128;
                const int y = w.tok0 + c * kC + 32 * we, x = w.h * kHeadDim;
                tma_store_2d(omap, x, y, src);
                tma_store_2d(omap, x + 64, y, src + kSlab);
                bulk_commit();
                bulk_wait_read_all();
            }
        }
        stage_release(&b.empty_q[at.s()], lane);
        return true;
    });
    if (lane == 0) bulk_wait_all();
}

template <bool kStates, bool kPacked>
__global__ void __launch_bounds__(kThreads, 1)
    la_kernel(const __grid_constant__ Kernel kernel, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap) {
    using M = Smem<kStates>;
    extern __shared__ __align__(1024) uint8_t smem[];
    // The next kernel may be placed where this one leaves room.  Every kernel of
    // a call waits for the end of the one before it ahead of its first read or
    // write of global memory: only that wait makes the writes of the kernels
    // before visible to it, a launch let come early does not.
    if (!kStates) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (kPacked) {
        asm volatile("griddepcontrol.wait;" ::: "memory");   // the offsets; the cut is decided before
        if (kStates) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    bool valid = !kPacked || !kernel.a.valid || *kernel.a.valid;
    if (kPacked && !kernel.a.valid) {
        // A small packed batch checks its offsets here: no kernel before this one.
        const int64_t* cu = kernel.a.cu_seqlens;
        bool ok = threadIdx.x > 0 || (cu[0] == 0 && cu[kernel.a.N] == kernel.a.tokens);
        for (int64_t n = threadIdx.x; n < kernel.a.N; n += kThreads) ok = ok && cu[n] <= cu[n + 1];
        valid = __syncthreads_and(ok);
        if (!valid && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(kernel.a.status, kDevBadSeqlens);
    }
    const Work<kStates, kPacked> p(kernel);
    if (!valid || (kStates && !p.cut)) return;
    if (smem_u32(smem) & 1023u) {   // the tiles' swizzle needs it; shared memory starts so
        if (threadIdx.x == 0) atomicOr(p.a.status, kDevPipeTimeout);
        return;
    }
    const Bars b = make_bars<kStates>(smem);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + M::kTmemPtr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // What the first chunk reads, on its way to L2 while the barriers and the
    // tensor memory are made ready.
    if (warp >= kLoadWarp && p.rows() > 0 && p.unit(0) < p.end) {
        const Unit w = unit_at(p, p.unit(0));
        if (w.nch > 0 && warp == kLoadWarp && lane == 0) {
            const int kcol = static_cast<int>(w.h / static_cast<uint32_t>(p.a.H / p.a.Hk)) * kHeadDim, vcol = w.h * kHeadDim;
#pragma unroll 1
            for (int x = 0; x < kHeadDim; x += 64) {
                tma_prefetch_l2_2d(&kmap, kcol + x, w.tok0);
                tma_prefetch_l2_2d(&vmap, vcol + x, w.tok0);
                if (!kStates) tma_prefetch_l2_2d(&qmap, kcol + x, w.tok0);
            }
        } else if (warp == kDecayWarp) {
#pragma unroll 1
            for (int r = lane; r < kC && r < w.len; r += 32)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p.a.g + (w.tok0 + r) * p.a.g_stride + w.h));
        }
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < M::kStages; ++s) {
            mbar_init(&b.full_k[s], 1);
            mbar_init(&b.full_v[s], 1);
            mbar_init(&b.full_q[s], 1);
            mbar_init(&b.empty_k[s], kStates ? kKeyWarps : kKeyWarps + 1);
            mbar_init(&b.empty_v[s], kStates ? 1 : 4);
            mbar_init(&b.empty_q[s], 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&b.kp_full[s], kKeyWarps);
            mbar_init(&b.kp_empty[s], 1);
            mbar_init(&b.dec_full[s], 1);
            mbar_init(&b.dec_empty[s], kKeyWarps + kStateWarps + (kStates ? 0 : 12));
        }
        mbar_init(b.qk, 1);
        mbar_init(b.z_done, 1);
        mbar_init(b.s_ready, kStateWarps);
        mbar_init(b.qs_ready, 8);             // query: Q' written; output: the last O read
        mbar_init(b.qs_done, 1);
        mbar_init(b.pv_ready, kStateWarps + 4);   // state: V is finite; score: P written
        mbar_init(b.o_done, 1);
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
    if (!kPacked) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (kStates) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }

    if (warp < kStateWarp)
        key_role(p, smem, b, tmem, warp, lane);
    else if (warp < kScoreWarp)
        state_role(p, smem, b, tmem, warp - kStateWarp, lane);
    else if (warp == kLoadWarp)
        load_role(p, &qmap, &kmap, &vmap, smem, b, lane);
    else if (warp == kMmaWarp)
        mma_role(p, smem, b, tmem, lane);
    else if (warp == kDecayWarp)
        decay_role(p, smem, b, lane);
    else if constexpr (!kStates) {
        if (warp < kQueryWarp)
            score_role(p, smem, b, tmem, warp - kScoreWarp, lane);
        else if (warp < kOutWarp)
            query_role(p, smem, b, warp - kQueryWarp, lane);
        else
            output_role(p, &omap, smem, b, tmem, warp - kOutWarp, lane);
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// The spans' incoming states: per (sequence, head), from S = init over the spans
// that it goes on in, S <- exp(D) S + Z, in place over Z.  kSplit warps share
// 128 kVec of the 16384 elements and take the spans kSplit kEach at a time: each
// warp loads up to kEach of them at once, composes them, and starts from what
// the warps before it compose to.  Few (sequence, head) units: eight warps a
// part, or a part's spans come one latency after the other (21 us for 128 spans
// of one head; 6 so).  Many: a warp a part, or the parts do (80 us for 96 units
// of 5).  kEach 4 for few spans: with the registers of 16 the CTAs of 6 heads
// would need three waves, and the output kernel, which starts when the last scan
// CTA has, would start with the third.
constexpr int kScanWarps = 8;
template <int kSplit, int kEach, int kVec>
__global__ void __launch_bounds__(32 * kScanWarps) la_scan_kernel(const __grid_constant__ Kernel p) {
    __shared__ float4 zsum[kScanWarps][kVec][32];
    __shared__ float dsum[kScanWarps];
    constexpr int64_t kState = kHeadDim * kHeadDim;
    constexpr uint32_t kParts = kHeadDim * kHeadDim / (128 * kVec), kGroups = kScanWarps / kSplit;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (p.a.valid && !*p.a.valid) return;
    if (p.sg.cut && !*p.sg.cut) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, place = warp % kSplit;
    const uint32_t parts = static_cast<uint32_t>(p.a.N) * p.heads * kParts;
    auto step = [](float d, const float4& a, const float4& z) {
        return make_float4(fmaf(d, a.x, z.x), fmaf(d, a.y, z.y), fmaf(d, a.z, z.z), fmaf(d, a.w, z.w));
    };
    // (kSplit 8: the whole CTA has the same part, so its barriers match.)
    for (uint32_t part = blockIdx.x * kGroups + warp / kSplit; part < parts; part += gridDim.x * kGroups) {
        const uint32_t unit = part / kParts, n = unit / p.heads, h = unit - n * p.heads;
        const int64_t e = (part % kParts) * (128 * kVec) + 4 * lane;
        int64_t s0 = n * p.sg.segs + 1, s1 = s0 + p.sg.segs - 1;
        if (p.sg.inner) {
            const int2 in = p.sg.inner[n];
            s0 = in.x;
            s1 = in.y;
        }
        if (s0 >= 0 && s0 >= s1) continue;   // the sequence is within one span
        float4 s[kVec];
#pragma unroll
        for (int v = 0; v < kVec; ++v) {
            const int64_t at = unit * kState + e + 128 * v;
            s[v] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (p.a.init_state) {
                if (p.a.state_f32) {
                    s[v] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.a.init_state) + at);
                } else {
                    const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.a.init_state) + at);
                    s[v] = make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
                }
            }
            if (p.sg.inits && place == 0) *reinterpret_cast<float4*>(p.sg.inits + at) = s[v];
            if (s0 < 0 && p.a.final_state && place == 0) {   // an empty sequence
                if (p.a.state_f32)
                    *reinterpret_cast<float4*>(static_cast<float*>(p.a.final_state) + at) = s[v];
                else
                    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.final_state) + at) =
                        make_uint2(pack_bf16(s[v].x, s[v].y), pack_bf16(s[v].z, s[v].w));
            }
        }
        for (int64_t base = s0; base < s1; base += kSplit * kEach) {
            const int64_t left = s1 - base;
            const int count = left < kSplit * kEach ? static_cast<int>(left) : kSplit * kEach;
            const int each = (count + kSplit - 1) / kSplit;
            const int mine = min(each, max(0, count - place * each));   // spans of this warp
            const int64_t first = base + place * each;
            float4 z[kEach][kVec];
            float d[kEach];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const bool there = i < mine;
                d[i] = there ? p.sg.decay[(first + i) * p.a.H + h] : 0.f;
#pragma unroll
                for (int v = 0; v < kVec; ++v)
                    z[i][v] = there ? *reinterpret_cast<const float4*>(p.sg.starts + ((first + i) * p.a.H + h) * kState + e + 128 * v)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float4 at[kVec];
            if (kSplit == 1) {
#pragma unroll
                for (int i = 0; i < kEach; ++i) d[i] = ex2(d[i]);
#pragma unroll
                for (int v = 0; v < kVec; ++v) at[v] = s[v];
            } else {
                float4 sum[kVec];
                float total = 0.f;
#pragma unroll
                for (int v = 0; v < kVec; ++v) sum[v] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (i < mine) {
                        total += d[i];
                        d[i] = ex2(d[i]);
#pragma unroll
                        for (int v = 0; v < kVec; ++v) sum[v] = step(d[i], sum[v], z[i][v]);
                    }
                __syncthreads();
#pragma unroll
                for (int v = 0; v < kVec; ++v) zsum[warp][v][lane] = sum[v];
                if (lane == 0) dsum[warp] = ex2(total);
                __syncthreads();
#pragma unroll 1
                for (int g = 0; g < kSplit; ++g)
#pragma unroll
                    for (int v = 0; v < kVec; ++v) {
                        if (g == place) at[v] = s[v];
                        s[v] = step(dsum[g], s[v], zsum[g][v][lane]);
                    }
            }
#pragma unroll
            for (int i = 0; i < kEach; ++i)
                if (i < mine)
#pragma unroll
                    for (int v = 0; v < kVec; ++v) {
                        at[v] = step(d[i], at[v], z[i][v]);
                        *reinterpret_cast<float4*>(p.sg.starts + ((first + i) * p.a.H + h) * kState + e + 128 * v) = at[v];
                    }
            if (kSplit == 1)
#pragma unroll
                for (int v = 0; v < kVec; ++v) s[v] = at[v];
        }
    }
}

// A packed batch: checks the offsets' contract (kda_meta.cu) and decides, from
// the lengths, whether to cut.  Without a cut the longest sequence is the least
// it takes; with one, every SM has a span of W chunks, and takes kLaCutChunkUs
// for each (kda_launch.h has the costs).  8 sequences of 33,333 tokens, 12 heads:
// the longest 65 chunks, 178 us uncut and 134 cut; all 33, 100 and 130.  20,000
// tokens, 16 heads, the longest 154 chunks: 405 and 119.
constexpr int kCutThreads = 1024, kCutThreadsFew = 128;   // few: up to 128 sequences

template <int kThreads>
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    x = (threadIdx.x & 31) < kThreads / 32 ? buf[threadIdx.x & 31] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads)
    la_cut_kernel(const int64_t* cu, int64_t N, int64_t T, int64_t H, int sms, LaSegments sg, int forced, int32_t* valid,
                  int* status) {
    __shared__ int64_t buf[32];
    __shared__ int longest_of[32];
    __shared__ int length;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int64_t bad = tid == 0 && (cu[0] != 0 || cu[N] != T), chunks = 0;
    int longest = 0;
    for (int64_t n = tid; n < N; n += kThreads) {
        const int64_t len = cu[n + 1] - cu[n];
        if (len < 0 || cu[n] < 0 || cu[n + 1] > T) {
            bad = 1;
            continue;
        }
        const int c = static_cast<int>((len + kC - 1) / kC);
        chunks += c;
        longest = max(longest, c);
    }
    bad = block_sum<kThreads>(bad, buf);
    chunks = block_sum<kThreads>(chunks, buf);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) longest_of[warp] = longest;
    __syncthreads();
    if (tid == 0) {
        *valid = bad ? 0 : 1;
        if (bad) atomicOr(status, kDevBadSeqlens);
        for (int i = 0; i < kThreads / 32; ++i) longest = max(longest, longest_of[i]);
        const float all = static_cast<float>(chunks);
        const float uncut = kLaChunkUs * fmaxf(static_cast<float>(longest), all * H / sms + 0.5f * longest);
        const int64_t width = sg.starts ? (chunks + sg.spans - 1) / sg.spans : 0;
        const bool pays = kLaCutUs + static_cast<float>(width) * kLaCutChunkUs < uncut;
        length = !sg.starts || bad || chunks == 0 ? 0 : forced > 0 ? forced : pays ? static_cast<int>(width) : 0;
        if (sg.starts) *sg.cut = length > 0;
    }
    __syncthreads();
    const int W = length;
    if (W == 0) {
        // The sequences by length, longest first (ties by index).
        if (sg.order && bad == 0)
            for (int64_t n = tid; n < N; n += kThreads) {
                const int64_t len = cu[n + 1] - cu[n];
                int rank = 0;
                for (int64_t m = 0; m < N; ++m) {
                    const int64_t other = cu[m + 1] - cu[m];
                    rank += other > len || (other == len && m < n);
                }
                sg.order[rank] = static_cast<int32_t>(n);
            }
        return;
    }
    // The sequences' chunks lie one after the other, cut every W chunks.  Every
    // cut and every sequence that is not empty begins a part, in this order: a
    // cut first where both are at one place (its part is empty then).
    int64_t carry = 0;   // chunks, and in the upper half sequences, before
    for (int64_t base = 0; base < N; base += kThreads) {
        const int64_t n = base + tid;
        const int64_t len = n < N ? cu[n + 1] - cu[n] : 0, count = (len + kC - 1) / kC, own = count | (len > 0 ? int64_t(1) << 32 : 0);
        int64_t x = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) buf[warp] = x;
        __syncthreads();
        int64_t before = carry, all = 0;
        for (int i = 0; i < kThreads / 32; ++i) {
            if (i < warp) before += buf[i];
            all += buf[i];
        }
        before += x - own;
        if (n < N) {
            const int rank = static_cast<int>(before >> 32), x0 = static_cast<int>(before), x1 = x0 + static_cast<int>(count);
            const int s0 = x0 / W, first = static_cast<int>(cu[n]);
            sg.inner[n] = make_int2(-1, -1);
            if (count > 0) {
                auto part = [&](int from, int s) {      // of span s, from chunk `from`
                    const int to = min(x1, (s + 1) * W), skip = (from - x0) * kC;
                    const int tokens = min(static_cast<int>(len) - skip, (to - from) * kC);
                    return make_int4(static_cast<int>(n), first + skip, tokens, (from > x0 ? kLaMid : 0) | (to == x1 ? kLaLast : 0));
                };
                if (s0 * W == x0) {
                    sg.first[s0] = s0 + rank;
                    sg.part[s0 + rank] = make_int4(static_cast<int>(n), first, 0, kLaMid);
                }
                sg.part[s0 + rank + 1] = part(x0, s0);
                int s = s0 + 1;
                for (; s * W < x1; ++s) {
                    sg.first[s] = s + rank + 1;
                    sg.part[s + rank + 1] = part(s * W, s);
                }
                sg.inner[n] = make_int2(s0 + 1, s);
            }
        }
        carry += all;
    }
    const int parted = static_cast<int>((static_cast<int>(carry) + W - 1) / W);
    for (int s = parted + tid; s <= sg.spans; s += kThreads) sg.first[s] = parted + static_cast<int>(carry >> 32);
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

// Programmatic dependence: a kernel is launched while the one before it ends,
// and waits for it where it reads what that one wrote.  3 sequences of 77 tokens,
// one call after the other: 10.2 us a call without, 7.5 so.
cudaLaunchConfig_t after_config(dim3 grid, dim3 block, size_t smem, cudaStream_t stream, cudaLaunchAttribute* after) {
    after->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    after->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = after;
    cfg.numAttrs = 1;
    return cfg;
}

template <bool kStates, bool kPacked>
cudaError_t configure() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    static bool configured[64] = {};
    if (configured[dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(la_kernel<kStates, kPacked>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(Smem<kStates>::kBytes));
    if (e == cudaSuccess) configured[dev] = true;
    return e;
}

}  // namespace

cudaError_t launch_la_cut(const int64_t* cu_seqlens, int64_t n_seqs, int64_t tokens, int64_t H, int sms, const LaSegments& sg,
                          int forced, int32_t* valid, int* status, cudaStream_t stream) {
    cudaLaunchAttribute after;
    const bool few = n_seqs <= kCutThreadsFew;
    const cudaLaunchConfig_t cfg = after_config(dim3(1), dim3(few ? kCutThreadsFew : kCutThreads), 0, stream, &after);
    return cudaLaunchKernelEx(&cfg, few ? la_cut_kernel<kCutThreadsFew> : la_cut_kernel<kCutThreads>, cu_seqlens, n_seqs, tokens,
                              H, sms, sg, forced, valid, status);
}

template <bool kPacked>
static cudaError_t launch(const LaArgs& a, const LaSegments& sg, int sms, cudaStream_t stream, int* launches) {
    Kernel p;
    p.a = a;
    p.sg = sg;
    const int64_t spans = sg.starts ? sg.spans * a.H : 0;
    // A packed batch's units or, cut, spans: one of the two comes to nothing.
    const int64_t units = sg.starts && !sg.cut ? spans : a.N * a.H;
    if (units <= 0) return cudaSuccess;
    if (units > 0x7fffffffLL || spans > 0x7fffffffLL) return cudaErrorInvalidValue;
    p.units = static_cast<uint32_t>(units);
    p.heads = static_cast<uint32_t>(a.H);
    CUtensorMap qm, km, vm, om;
    cudaError_t e;
    if ((e = configure<false, kPacked>()) != cudaSuccess || (e = configure<true, kPacked>()) != cudaSuccess) return e;
    if ((e = encode_tokens(&qm, a.q, a.tokens, a.Hk, kC)) != cudaSuccess ||
        (e = encode_tokens(&km, a.k, a.tokens, a.Hk, kC)) != cudaSuccess ||
        (e = encode_tokens(&vm, a.v, a.tokens, a.H, kC)) != cudaSuccess ||
        (e = encode_tokens(&om, a.out, a.tokens, a.H, 32)) != cudaSuccess)
        return e;
    int64_t grid = units < sms ? units : sms;
    if (sg.cut && grid < spans) grid = spans;
    cudaLaunchAttribute after;
    cudaLaunchConfig_t cfg = after_config(dim3(1), dim3(kThreads), 0, stream, &after);
    if (sg.starts) {
        cfg.gridDim = dim3(static_cast<unsigned>(sg.cut ? spans : grid));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Smem<true>::kBytes;
        if ((e = cudaLaunchKernelEx(&cfg, la_kernel<true, kPacked>, p, qm, km, vm, om)) != cudaSuccess) return e;
        const bool many = a.N * a.H >= 24, few = (sg.cut ? sg.spans : sg.segs) <= 4 * kScanWarps;
        const int64_t parts = a.N * a.H * (many || !few ? 128 : 64), ctas = many ? (parts + kScanWarps - 1) / kScanWarps : parts;
        const int64_t most = static_cast<int64_t>(sms) * (many ? 4 : few ? 3 : 2);
        cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most));
        cfg.blockDim = dim3(32 * kScanWarps);
        cfg.dynamicSmemBytes = 0;
        if ((e = cudaLaunchKernelEx(&cfg, many ? la_scan_kernel<1, 8, 1> : few ? la_scan_kernel<8, 4, 2> : la_scan_kernel<8, 16, 1>,
                                    p)) != cudaSuccess)
            return e;
        *launches += 2;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Smem<false>::kBytes;
    if ((e = cudaLaunchKernelEx(&cfg, la_kernel<false, kPacked>, p, qm, km, vm, om)) != cudaSuccess) return e;
    *launches += 1;
    return cudaSuccess;
}

cudaError_t launch_la_prefill(const LaArgs& a, const LaSegments& sg, int sms, cudaStream_t stream, int* launches) {
    return a.cu_seqlens ? launch<true>(a, sg, sms, stream, launches) : launch<false>(a, sg, sms, stream, launches);
}

}  // namespace kda
