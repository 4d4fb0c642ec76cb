// kda_ssm.cu -- the selective state space scan (sm_103a).
//
// For each channel d of a sequence, with states n = 0 .. S - 1:
//     dt = softplus(dt_raw + bias_d),  h[n] <- exp(dt A[d][n]) h[n] + dt x B[n],
//     y = sum_n C[n] h[n] + D_d x,  out = y silu(z);
// B and C are shared by a group of channels.
//
// Prompts (ssm_kernel).  The decays differ in every channel and state, so there is
// no product of matrices in it: 8 S + 20 operations for 8 bytes, of which S
// exponentials, bound by the SMs.  A CTA has 32 channels and a span of tokens, 32 at
// a time: half of its threads form dt, dt x and the rows of B and C as FP32 in
// shared memory; the warps of the other half walk 16 channels and half of the states
// through the tokens, two channels and two states (of every 16) in a lane's
// registers, so that what a lane reads serves four.  The states lie as the A operand of an
// m16n8k8 product (TF32), four registers that it takes as they are: rows are
// channels, and column j of the B operand is token j's C, so that one instruction
// gives sum_n C[n] h[n] of 16 channels, without shuffles.  That takes h to TF32 on its
// way to out (cut to 10 bits: at most 2^-10 of |C[n] h[n]|, where out's own rounding to
// BF16 is 2^-9 of out); the states themselves stay FP32.
//
// Few (sequence, channel) chains are cut into spans of tokens: a first launch
// forms the state each span ends with (and the sum of its dt: the decay over a
// span is exp(A sum dt)), a second one each span's incoming state from those
// before it, and its outputs.
#include <type_traits>

#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_seq.cuh"
#include "kda_vec.cuh"

namespace kda {
namespace {

constexpr int kRole = 128;               // threads that walk, and threads that stage and finish
constexpr int kThreads = 2 * kRole;
constexpr int kTile = kSsmTile;          // tokens at a time
constexpr int kChannels = kSsmChannels;  // channels of a CTA, 8 a warp
static_assert(kRole == 4 * kTile && kChannels == 32, "a thread stages 8 channels of one token");
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

// y <- y silu(z), eight times.  Above -80, z / (1 + exp(-z)) as it stands, six
// instructions where sigmoid(), whose small values keep their bits, takes ten.
__device__ __forceinline__ void gate8(const float (&z)[8], float (&y)[8]) {
    float least = z[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) least = fminf(least, z[j]);
    if (least > -80.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + exp2_fast(z[j] * -kLog2e)));
            y[j] *= z[j] * r;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= z[j] * sigmoid(z[j]);
    }
}

// Shared memory of one of two buffers, which the walk is bound by (256 bytes a cycle
// where neighbouring lanes read the same 16 bytes, 128 else): for each token and two
// channels 8 apart (dt, dt, dt x, dt x), the rows of B and of C, and y, a sum over each
// half of the states.  Strides that keep the lanes' accesses on different banks.
constexpr int kStepStride = 4 * (kTile + 1), kStepHalf = 8 * kStepStride + 8;
constexpr int kStepWords = 2 * kStepHalf;
constexpr int kYStride = kChannels + 4;
template <int kBlocks, bool kStates>
struct Buffer {
    static constexpr int kRow = 16 * kBlocks, kRowC = kRow + 8;
    static constexpr int kB = kStepWords, kC = kB + kTile * kRow, kY = kC + (kStates ? 0 : kTile * kRowC);
    static constexpr int kHalf = kTile * kYStride;   // of y
    static constexpr int kXZ = kY + (kStates ? 0 : 2 * kHalf);   // x and z of each staging thread, for its outputs
    static constexpr int kWords = kXZ + (kStates ? 0 : 8 * kRole);
};
// The pair of channels that channel ch is of, at a token: (dt, dt, dt x, dt x).
__device__ __forceinline__ int step_at(int ch, int token) { return (ch >> 4) * kStepHalf + (ch & 7) * kStepStride + 4 * token; }

// What a staging thread fetches of a tile: of one token eight channels' x, z and dt, and
// four values of every 16 of B and C.
template <int kBlocks>
struct Fetched {
    uint4 x, z, dt[2], b[kBlocks], c[kBlocks];
};
__device__ __forceinline__ uint4 two_pieces(const uint8_t* p) {
    const uint2 lo = *reinterpret_cast<const uint2*>(p), hi = *reinterpret_cast<const uint2*>(p + 16);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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

// A lane's states.  Prompts: pairs of two channels, 16 k + 8 half + 2 c + i of
// channels g and g + 8 of the warp's 16 (g the lane's place among eight, c among
// four).  Single tokens: states 16 k + 4 c + 2 i and the next of one channel.
template <int kBlocks>
struct State {
    uint64_t h[kBlocks][2];
};

// Two values from state n0 on of a row of S.
template <typename T>
__device__ __forceinline__ float2 load_two(const T* row, int n0, int S) {
    if (S % 2 == 0) {
        float v[2] = {0.f, 0.f};
        if (n0 < S) load_vec<2>(row + n0, v);
        return make_float2(v[0], v[1]);
    }
    return make_float2(n0 < S ? static_cast<float>(row[n0]) : 0.f, n0 + 1 < S ? static_cast<float>(row[n0 + 1]) : 0.f);
}
template <typename T>
__device__ __forceinline__ void store_two(T* row, int n0, int S, float2 v) {
    if (S % 2 == 0) {
        const float w[2] = {v.x, v.y};
        if (n0 < S) store_vec<2>(row + n0, w);
    } else {
        if (n0 < S) from_f32(row + n0, v.x);
        if (n0 + 1 < S) from_f32(row + n0 + 1, v.y);
    }
}
// The lane's states of two rows of S (of channels 8 apart).
template <int kBlocks>
__device__ __forceinline__ void load_rows(const void* p, bool f32, int64_t row, int64_t row8, int n0, int S, State<kBlocks>& s) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        float2 a, b;
        if (f32) {
            a = load_two(static_cast<const float*>(p) + row * S, 16 * k + n0, S);
            b = load_two(static_cast<const float*>(p) + row8 * S, 16 * k + n0, S);
        } else {
            a = load_two(static_cast<const __nv_bfloat16*>(p) + row * S, 16 * k + n0, S);
            b = load_two(static_cast<const __nv_bfloat16*>(p) + row8 * S, 16 * k + n0, S);
        }
        s.h[k][0] = pair(a.x, b.x);
        s.h[k][1] = pair(a.y, b.y);
    }
}
template <int kBlocks>
__device__ __forceinline__ void store_rows(void* p, bool f32, int64_t row, bool live, int64_t row8, bool live8, int n0, int S,
                                           const State<kBlocks>& s) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const float2 x = halves(s.h[k][0]), y = halves(s.h[k][1]);
        const float2 a = make_float2(x.x, y.x), b = make_float2(x.y, y.y);
        if (f32) {
            if (live) store_two(static_cast<float*>(p) + row * S, 16 * k + n0, S, a);
            if (live8) store_two(static_cast<float*>(p) + row8 * S, 16 * k + n0, S, b);
        } else {
            if (live) store_two(static_cast<__nv_bfloat16*>(p) + row * S, 16 * k + n0, S, a);
            if (live8) store_two(static_cast<__nv_bfloat16*>(p) + row8 * S, 16 * k + n0, S, b);
        }
    }
}
// Four values of a single token's state, which nobody reads before the next token:
// a streaming store (128 sequences of 12,288 channels 35 us, with a plain one 40).
template <typename T>
__device__ __forceinline__ void store_four(T* row, const float (&v)[4]) {
    if constexpr (sizeof(T) == 4)
        __stcs(reinterpret_cast<float4*>(row), make_float4(v[0], v[1], v[2], v[3]));
    else
        __stcs(reinterpret_cast<uint2*>(row), make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])));
}
// A lane's values of a row of S as loaded, four at a time.  With kFull S is 16
// kBlocks and they can be read so.
template <int kBlocks, typename T>
struct Row {
    using Four = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
    Four r[kBlocks];

    template <bool kFull>
    __device__ __forceinline__ void load(const T* row, int c, int S) {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int n0 = 16 * k + 4 * c;
            if constexpr (kFull) {
                r[k] = *reinterpret_cast<const Four*>(row + n0);
            } else if constexpr (sizeof(T) == 4) {
                r[k] = gather4(row + n0, S - n0);
            } else {
                const uint4 v = gather8(row + n0, S - n0 < 4 ? S - n0 : 4);
                r[k] = make_uint2(v.x, v.y);
            }
        }
    }
    __device__ __forceinline__ void unpack(State<kBlocks>& s) const {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            if constexpr (sizeof(T) == 4) {
                s.h[k][0] = pair(__uint_as_float(r[k].x), __uint_as_float(r[k].y));
                s.h[k][1] = pair(__uint_as_float(r[k].z), __uint_as_float(r[k].w));
            } else {
                s.h[k][0] = pair(bf16_lo(r[k].x), bf16_hi(r[k].x));
                s.h[k][1] = pair(bf16_lo(r[k].y), bf16_hi(r[k].y));
            }
        }
    }
    template <bool kFull>
    __device__ static __forceinline__ void store(T* row, int c, int S, const State<kBlocks>& s) {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int n0 = 16 * k + 4 * c;
            const float2 a = halves(s.h[k][0]), b = halves(s.h[k][1]);
            const float v[4] = {a.x, a.y, b.x, b.y};
            if constexpr (kFull) {
                store_four(row + n0, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + i < S) from_f32(row + n0 + i, v[i]);
            }
        }
    }
};
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

// D = A B, or A B + D, for one m16n8k8 tile of TF32 operands, the sum in FP32.
__device__ __forceinline__ void mma_tf32_first(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)), "f"(0.f));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

// A CTA's part of the work: a group's channels from ch0 on, and tokens [begin, end).
struct Part {
    int64_t begin, end;
    int64_t seq, seq_end;    // the sequence of token `begin` and its end
    int64_t first_span;      // outputs: the spans before whose states meet here, up to `span`
    int64_t span;
    bool fresh;              // the sequence's first token is here: its initial state
    bool run;
};

template <bool kStates, bool kPacked>
__device__ __forceinline__ Part part_of(const SsmArgs& a, int64_t span) {
    Part w = {};
    w.run = true;
    w.span = w.first_span = span;
    if (kPacked) {
        w.begin = span * a.span_tokens;
        w.end = w.begin + a.span_tokens < a.tokens ? w.begin + a.span_tokens : a.tokens;
        if (kStates) {
            // The sequence that goes on behind the span, if there is one.
            w.seq = ended_by(a.cu_seqlens, a.N, w.end);
            if (w.seq >= a.N || a.cu_seqlens[w.seq] >= w.end) {
                w.run = false;
                return w;
            }
            const int64_t first = a.cu_seqlens[w.seq];
            w.fresh = first >= w.begin;
            if (w.fresh) w.begin = first;
            w.seq_end = w.end;
        } else {
            // The first span also has the empty sequences before the first token.
            w.seq = span == 0 ? 0 : ended_by(a.cu_seqlens, a.N, w.begin);
            const int64_t first = a.cu_seqlens[w.seq];
            w.fresh = first >= w.begin;
            w.first_span = w.fresh ? span : quotient(first, a.span_tokens);
            w.seq_end = a.cu_seqlens[w.seq + 1];
        }
    } else {
        w.seq = quotient(span, a.spans_per_seq);
        const int64_t s = span - w.seq * a.spans_per_seq, first = w.seq * a.tokens_per_seq;
        w.begin = first + s * a.span_tokens;
        w.seq_end = first + a.tokens_per_seq;
        w.end = w.begin + a.span_tokens < w.seq_end ? w.begin + a.span_tokens : w.seq_end;
        w.fresh = s == 0;
        w.first_span = span - s;
        w.run = !kStates || s + 1 < a.spans_per_seq;
    }
    return w;
}

// Half of the warps walk; the other half stage the tile ahead and finish the one
// behind, so that there are warps enough to hide each other's latencies.
// kFast: BF16 dt, B and C, 16 kBlocks states, groups of whole 32 channels, a
// softplus, and rows that can be read four values at a time, which leaves out two
// fifths of the staging's instructions.
template <int kBlocks, bool kStates, bool kPacked, bool kFast>
__global__ void __launch_bounds__(kThreads, kBlocks > 1 ? 2 : 3) ssm_kernel(SsmArgs a) {
    using Buf = Buffer<kBlocks, kStates>;
    extern __shared__ __align__(16) float smem[];
    wait_for_kernel_before();
    if (kStates) let_next_kernel_come();
    if (kPacked && !offsets_hold(a.cu_seqlens, a.N, a.tokens, a.valid, a.status)) return;
    const int64_t span = quotient(blockIdx.x, a.tiles), tile = blockIdx.x - span * a.tiles;
    const Part w = part_of<kStates, kPacked>(a, span);
    if (!w.run) return;
    const int64_t group = quotient(tile, a.tiles_per_group), per = quotient(a.dim, a.groups);
    const int64_t ch0 = group * per + (tile - group * a.tiles_per_group) * kChannels;
    const int channels = kFast || (group + 1) * per - ch0 > kChannels ? kChannels : static_cast<int>((group + 1) * per - ch0);
    const int S = kFast ? 16 * kBlocks : static_cast<int>(a.nstate);
    const int tid = threadIdx.x & (kRole - 1);
    const int total = static_cast<int>(w.end - w.begin);   // tokens; tiles i = 0 .. tiles - 1 of them
    const int tiles = total / kTile + (total % kTile > 0);

    if (threadIdx.x >= kRole) {
        // ---- staging: of one token four channels and the four 8 further on, and a
        // quarter of its rows of B and C
        const int tok = tid >> 2, mine = 16 * (tid >> 1 & 1) + 4 * (tid & 1);
        auto clip = [](int n) { return n < 0 ? 0 : n < 4 ? n : 4; };
        const int count = clip(channels - mine), count8 = clip(channels - mine - 8);
        const bool wide = kFast || (a.vec && count8 == 4), wide_keys = kFast || a.vec_bc, gated = !kStates && a.z;
        const bool dt_f32 = !kFast && a.dt_f32, bc_f32 = !kFast && a.bc_f32;
        float bias[8], skip[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = mine + (i & 3) + 2 * (i & 4);
            bias[i] = a.dt_bias && at < channels ? a.dt_bias[ch0 + at] : 0.f;
            skip[i] = !kStates && a.D && at < channels ? a.D[ch0 + at] : 0.f;
        }
        // This thread's rows of the tile to fetch next, and to finish.
        const int es = bc_f32 ? 4 : 2, dts = dt_f32 ? 4 : 2;
        const int64_t t0 = w.begin + tok;
        auto xp = static_cast<const uint8_t*>(a.x) + (t0 * a.ldx + ch0 + mine) * 2;
        auto zp = static_cast<const uint8_t*>(a.z) + (t0 * a.ldz + ch0 + mine) * 2;
        auto dp = static_cast<const uint8_t*>(a.dt) + (t0 * a.lddt + ch0 + mine) * dts;
        auto bp = static_cast<const uint8_t*>(a.B) + (t0 * a.ldb + group * S + 4 * (tid & 3)) * es;
        auto cp = static_cast<const uint8_t*>(a.C) + (t0 * a.ldc + group * S + 4 * (tid & 3)) * es;
        auto op = static_cast<__nv_bfloat16*>(a.out) + t0 * a.dim + ch0 + mine;
        int ahead = total - tok;   // tokens from this thread's next one to fetch to the end
        Fetched<kBlocks> f;
        auto fetch = [&]() {
            const uint4 none = make_uint4(0, 0, 0, 0);
            if (ahead > 0) {
                if (wide) {
                    f.x = two_pieces(xp);
                    if (gated) f.z = two_pieces(zp);
                    if (dt_f32) {
                        f.dt[0] = *reinterpret_cast<const uint4*>(dp);
                        f.dt[1] = *reinterpret_cast<const uint4*>(dp + 32);
                    } else {
                        f.dt[0] = two_pieces(dp);
                    }
                } else {
                    auto eight = [&](const uint8_t* p) {
                        const uint4 lo = gather8(reinterpret_cast<const __nv_bfloat16*>(p), count),
                                    hi = gather8(reinterpret_cast<const __nv_bfloat16*>(p + 16), count8);
                        return make_uint4(lo.x, lo.y, hi.x, hi.y);
                    };
                    f.x = eight(xp);
                    if (gated) f.z = eight(zp);
                    if (dt_f32) {
                        f.dt[0] = gather4(reinterpret_cast<const float*>(dp), count);
                        f.dt[1] = gather4(reinterpret_cast<const float*>(dp + 32), count8);
                    } else {
                        f.dt[0] = eight(dp);
                    }
                }
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    const int have = S - 16 * k - 4 * (tid & 3);
                    const uint8_t *b = bp + 16 * k * es, *cc = cp + 16 * k * es;
                    if (!kFast && have <= 0) {
                        f.b[k] = f.c[k] = none;
                    } else if (wide_keys && bc_f32) {
                        f.b[k] = *reinterpret_cast<const uint4*>(b);
                        if (!kStates) f.c[k] = *reinterpret_cast<const uint4*>(cc);
                    } else if (wide_keys) {
                        const uint2 rb = *reinterpret_cast<const uint2*>(b);
                        f.b[k].x = rb.x;
                        f.b[k].y = rb.y;
                        if (!kStates) {
                            const uint2 rc = *reinterpret_cast<const uint2*>(cc);
                            f.c[k].x = rc.x;
                            f.c[k].y = rc.y;
                        }
                    } else if (bc_f32) {
                        f.b[k] = gather4(reinterpret_cast<const float*>(b), have);
                        if (!kStates) f.c[k] = gather4(reinterpret_cast<const float*>(cc), have);
                    } else {
                        f.b[k] = gather8(reinterpret_cast<const __nv_bfloat16*>(b), have < 4 ? have : 4);
                        if (!kStates) f.c[k] = gather8(reinterpret_cast<const __nv_bfloat16*>(cc), have < 4 ? have : 4);
                    }
                }
            } else {   // behind the end nothing is added
                f.x = f.z = f.dt[0] = f.dt[1] = none;
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) f.b[k] = f.c[k] = none;
            }
            xp += a.tile_x;
            if (gated) zp += a.tile_z;
            dp += a.tile_dt;
            bp += a.tile_b;
            if (!kStates) cp += a.tile_c;
            ahead -= kTile;
        };
        // To the nearest TF32 value, which a BF16 one is.
        auto tf32 = [](float v) {
            uint32_t r;
            asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
            return __uint_as_float(r);
        };
        auto four = [&](const uint4& r) {
            return bc_f32 ? make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w))
                          : make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
        };
        // (dt and what it stands for are of the tile before the next to fetch.)
        auto stage = [&](float* buf) {
            float dt[8], x[8];
            unpack8(f.x, x);
            if (dt_f32) {
                dt[0] = __uint_as_float(f.dt[0].x); dt[1] = __uint_as_float(f.dt[0].y);
                dt[2] = __uint_as_float(f.dt[0].z); dt[3] = __uint_as_float(f.dt[0].w);
                dt[4] = __uint_as_float(f.dt[1].x); dt[5] = __uint_as_float(f.dt[1].y);
                dt[6] = __uint_as_float(f.dt[1].z); dt[7] = __uint_as_float(f.dt[1].w);
            } else {
                unpack8(f.dt[0], dt);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dt[j] += bias[j];
                if (kFast || a.softplus) dt[j] = softplus(dt[j]);
            }
            if (ahead <= -kTile)   // behind the end nothing decays either
#pragma unroll
                for (int j = 0; j < 8; ++j) dt[j] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<float4*>(buf + step_at(mine + j, tok)) = make_float4(dt[j], dt[j + 4], dt[j] * x[j], dt[j + 4] * x[j + 4]);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                const int n0 = 16 * k + 4 * (tid & 3);
                *reinterpret_cast<float4*>(buf + Buf::kB + tok * Buf::kRow + n0) = four(f.b[k]);
                if (!kStates) {
                    const float4 v = four(f.c[k]);
                    *reinterpret_cast<float4*>(buf + Buf::kC + tok * Buf::kRowC + n0) =
                        bc_f32 ? make_float4(tf32(v.x), tf32(v.y), tf32(v.z), tf32(v.w)) : v;
                }
            }
            if (!kStates) {
                uint4* xz = reinterpret_cast<uint4*>(buf + Buf::kXZ) + tid;
                xz[0] = f.x;
                if (gated) xz[kRole] = f.z;
            }
        };
        // A token's outputs from its y: the skip, the gate and one rounding.
        int left = total - tok;   // tokens from this thread's next one to finish to the end
        auto finish = [&](const float* buf) {
            if (left > 0) {
                const float* p = buf + Buf::kY + tok * kYStride + mine;
                const uint4* xz = reinterpret_cast<const uint4*>(buf + Buf::kXZ) + tid;
                float y[8], x[8], z[8];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float4 v = *reinterpret_cast<const float4*>(p + 8 * j), u = *reinterpret_cast<const float4*>(p + Buf::kHalf + 8 * j);
                    y[4 * j] = v.x + u.x; y[4 * j + 1] = v.y + u.y; y[4 * j + 2] = v.z + u.z; y[4 * j + 3] = v.w + u.w;
                }
                if (a.D) {
                    unpack8(xz[0], x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = fmaf(skip[j], x[j], y[j]);
                }
                if (gated) {
                    unpack8(xz[kRole], z);
                    gate8(z, y);
                }
                if (wide) {
                    *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                    *reinterpret_cast<uint2*>(op + 8) = make_uint2(pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (j < count) op[j] = __float2bfloat16_rn(y[j]);
                        if (j < count8) op[j + 8] = __float2bfloat16_rn(y[j + 4]);
                    }
                }
            }
            op += a.tile_out;
            left -= kTile;
        };
        // While tile i is walked, i - 1 is finished, i + 1 staged and i + 2 fetched.
        float *buf = smem, *other = smem + Buf::kWords;
        if (tiles > 0) {
            fetch();
            stage(buf);
            if (tiles > 1) fetch();
        }
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            if (!kStates && i > 0) finish(other);
            if (i + 1 < tiles) {
                stage(other);
                if (i + 2 < tiles) fetch();
            }
            __syncthreads();
            float* const was = buf;
            buf = other;
            other = was;
        }
        if (!kStates && tiles > 0) finish(other);
        return;
    }

    // ---- the walk: 16 channels and a half of every 16 states for each warp
    const int warp = tid >> 5, lane = tid & 31, c = lane & 3, half = warp & 1;
    const int local = 16 * (warp >> 1) + (lane >> 2), n0 = 8 * half + 2 * c;
    const bool live = local < channels, live8 = local + 8 < channels;
    const int64_t ch = ch0 + (live ? local : 0), ch8 = ch0 + (live8 ? local + 8 : 0);
    State<kBlocks> rate, s;
    load_rows<kBlocks>(a.A, true, ch, ch8, n0, S, rate);
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) rate.h[k][i] = mul_pair(rate.h[k][i], pair(kLog2e, kLog2e));
    auto initial = [&](int64_t seq) {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) s.h[k][0] = s.h[k][1] = 0ull;
        if (a.init_state) load_rows<kBlocks>(a.init_state, a.state_f32, seq * a.dim + ch, seq * a.dim + ch8, n0, S, s);
    };
    auto ending = [&](int64_t seq) {
        if (a.final_state)
            store_rows<kBlocks>(a.final_state, a.state_f32, seq * a.dim + ch, live, seq * a.dim + ch8, live8, n0, S, s);
    };
    if (w.fresh) {
        initial(w.seq);
    } else {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) s.h[k][0] = s.h[k][1] = 0ull;
        if (!kStates) {
            // The states of the sequence's spans before this one, each decayed over
            // those behind it; the first one's has the initial state in it.
#pragma unroll 4
            for (int64_t i = w.first_span; i < span; ++i) {
                State<kBlocks> add;
                load_rows<kBlocks>(a.span_states, true, i * a.dim + ch, i * a.dim + ch8, n0, 16 * kBlocks, add);
                decay<kBlocks>(s, rate, pair(a.span_steps[i * a.dim + ch], a.span_steps[i * a.dim + ch8]), add.h);
            }
        }
    }
    // The states of the sequences that end at token t of the span, and the next one's.
    int64_t seq = w.seq, seq_end = w.seq_end - w.begin;
    auto close = [&](int64_t t) {
        while (t == seq_end) {
            ending(seq);
            if (!kPacked || ++seq >= a.N) break;
            seq_end = a.cu_seqlens[seq + 1] - w.begin;
            initial(seq);
        }
    };
    if (!kStates) close(0);
    uint64_t steps = 0ull;   // the sums of dt
    const int step0 = step_at(local, 0), rows0 = Buf::kB + n0;
    const int keys0 = Buf::kC + (lane >> 2) * Buf::kRowC + n0, y0 = Buf::kY + half * Buf::kHalf + 2 * c * kYStride + local;
    // Eight tokens from t on of the tile at `base`; with `ends`, sequences may end
    // among them.  (Tokens behind the span's end change nothing: only the last span
    // has them, and no sequence behind it.)  y: of tokens 2 c and 2 c + 1, and of
    // the second channel, as the product's accumulators have them.
    auto walk = [&](auto ends, const float* buf, int64_t base, int t, float (&y)[4]) {
        float ck[kBlocks][2];
        if (!kStates)
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                const float2 v = *reinterpret_cast<const float2*>(buf + keys0 + t * Buf::kRowC + 16 * k);
                ck[k][0] = v.x;
                ck[k][1] = v.y;
            }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint64_t b[kBlocks][2];
            const ulonglong2 dd = *reinterpret_cast<const ulonglong2*>(buf + step0 + 4 * (t + j));   // both dt, both dt x
            const float2 du = halves(dd.y);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                const float2 v = *reinterpret_cast<const float2*>(buf + rows0 + (t + j) * Buf::kRow + 16 * k);
                b[k][0] = pair(du.x * v.x, du.y * v.x);
                b[k][1] = pair(du.x * v.y, du.y * v.y);
            }
            decay<kBlocks>(s, rate, dd.x, b);
            if (kStates) {
                steps = add_pair(steps, dd.x);
            } else {
                float acc[4];
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    const float2 lo = halves(s.h[k][0]), hi = halves(s.h[k][1]);
                    if (k == 0)
                        mma_tf32_first(acc, lo.x, lo.y, hi.x, hi.y, ck[k][0], ck[k][1]);
                    else
                        mma_tf32(acc, lo.x, lo.y, hi.x, hi.y, ck[k][0], ck[k][1]);
                }
                // (The columns of the other tokens hold nothing of use.)
                if (c == j >> 1) {
                    y[j & 1] = acc[j & 1];
                    y[2 + (j & 1)] = acc[2 + (j & 1)];
                }
                if (decltype(ends)::value) close(base + t + j + 1);
            }
        }
    };
    auto store_y = [&](float* buf, int t, const float (&y)[4]) {
        float* at = buf + y0 + t * kYStride;
        at[0] = y[0];
        at[kYStride] = y[1];
        at[8] = y[2];
        at[kYStride + 8] = y[3];
    };
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        float* buf = smem + (i & 1) * Buf::kWords;
        const int64_t base = static_cast<int64_t>(i) * kTile;
        if (base + kTile <= total && (!kPacked || kStates || seq_end >= base + kTile)) {
            // (y is stored behind all loads: the compiler keeps their order.)
            float y[kTile / 8][4];
#pragma unroll
            for (int t = 0; t < kTile; t += 8) walk(std::false_type{}, buf, base, t, y[t / 8]);
            if (!kStates)
#pragma unroll
                for (int t = 0; t < kTile; t += 8) store_y(buf, t, y[t / 8]);
            if (kPacked && !kStates) close(base + kTile);
        } else {
#pragma unroll 1
            for (int t = 0; t < kTile && base + t < total; t += 8) {
                float y[4];
                walk(std::integral_constant<bool, kPacked && !kStates>{}, buf, base, t, y);
                if (!kStates) store_y(buf, t, y);
            }
        }
        __syncthreads();
    }
    if (!kPacked && !kStates && total == seq_end && total > 0) close(total);
    if (kStates) {
        store_rows<kBlocks>(a.span_states, true, span * a.dim + ch, live, span * a.dim + ch8, live8, n0, 16 * kBlocks, s);
        if (c == 0 && half == 0) {
            if (live) a.span_steps[span * a.dim + ch] = halves(steps).x;
            if (live8) a.span_steps[span * a.dim + ch8] = halves(steps).y;
        }
    }
}

// ---- single tokens: four lanes a channel, four sequences a thread
// Bound by HBM: each state is read and written once, 2 x 4 S bytes (FP32) a
// channel.  Lane i of a channel's four loads x, dt and z of sequence i, forms its
// step and its gate and hands the step to the other three; the sums over the
// states come back to it, so that nothing is computed four times, and the rates are
// read once for four sequences.  All loads are issued before the first value is
// used.  kFull: 16 kBlocks states, and rows of B and C that can be read four
// values at a time.
constexpr int kStepThreads = 4 * kChannels;
template <int kBlocks, bool kFull, bool kStateF32, bool kKeysF32>
__global__ void __launch_bounds__(kStepThreads, kBlocks == 1 ? 8 : kBlocks == 2 ? 4 : 3) ssm_decode_kernel(SsmArgs a, int blocks) {
    wait_for_kernel_before();
    constexpr int kTogether = kBlocks == 1 ? 4 : 1;   // sequences whose states and rows are under way together
    using StateT = std::conditional_t<kStateF32, float, __nv_bfloat16>;
    using KeyT = std::conditional_t<kKeysF32, float, __nv_bfloat16>;
    const int c = threadIdx.x & 3, S = kFull ? 16 * kBlocks : static_cast<int>(a.nstate);
    const int part = static_cast<int>(blockIdx.x / static_cast<uint32_t>(blocks)), n0 = 4 * part;
    const int ch_raw = (static_cast<int>(blockIdx.x) - part * blocks) * kChannels + static_cast<int>(threadIdx.x >> 2);
    const int dim = static_cast<int>(a.dim), N = static_cast<int>(a.N);
    const bool live = ch_raw < dim;
    const int ch = live ? ch_raw : dim - 1;
    const int group = a.groups > 1 ? static_cast<uint32_t>(ch) / static_cast<uint32_t>(dim / static_cast<int>(a.groups)) : 0;

    // The sequences' slots (-1: none) are the same for the whole CTA.
    int slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) slot[i] = n0 + i < N ? (a.slots ? a.slots[n0 + i] : n0 + i) : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (slot[i] >= a.pool) {
            if (ch_raw == 0 && c == 0) atomicOr(a.status, kDevBadSlots);
            slot[i] = -1;
        }
    // (A state's row is below 2^32 bytes, see kSsmMaxDim.)
    const uint32_t state_bytes = static_cast<uint32_t>(dim) * S * sizeof(StateT);
    uint8_t* base = static_cast<uint8_t*>(a.state) + static_cast<uint64_t>(static_cast<uint32_t>(ch)) * (S * sizeof(StateT));
    auto row_at = [&](int i) { return reinterpret_cast<StateT*>(base + static_cast<uint64_t>(static_cast<uint32_t>(slot[i])) * state_bytes); };
    Row<kBlocks, StateT> states[kTogether];
    Row<kBlocks, KeyT> bs[kTogether], cs[kTogether];
    const KeyT *b_row = static_cast<const KeyT*>(a.B) + n0 * a.ldb + group * S, *c_row = static_cast<const KeyT*>(a.C) + n0 * a.ldc + group * S;
    auto load = [&](int i, int to) {
        if (slot[i] >= 0) {
            states[to].template load<kFull>(row_at(i), c, S);
            bs[to].template load<kFull>(b_row, c, S);
            cs[to].template load<kFull>(c_row, c, S);
        }
        b_row += a.ldb;
        c_row += a.ldc;
    };
    if (kTogether == 4)
#pragma unroll
        for (int i = 0; i < kTogether; ++i) load(i, i);
    const int own = n0 + c;
    __nv_bfloat16 x_raw = __float2bfloat16_rn(0.f), z_raw = x_raw;
    uint32_t dt_raw = 0;
    if (own < N) {   // (read for a padding row too, and not used)
        x_raw = static_cast<const __nv_bfloat16*>(a.x)[own * a.ldx + ch];
        if (a.z) z_raw = static_cast<const __nv_bfloat16*>(a.z)[own * a.ldz + ch];
        dt_raw = a.dt_f32 ? static_cast<const uint32_t*>(a.dt)[own * a.lddt + ch] : static_cast<const uint16_t*>(a.dt)[own * a.lddt + ch];
    }
    Row<kBlocks, float> rates;
    rates.template load<kFull>(a.A + static_cast<uint64_t>(static_cast<uint32_t>(ch)) * S, c, S);
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f, skip = a.D ? a.D[ch] : 0.f;

    float dt = __uint_as_float(a.dt_f32 ? dt_raw : dt_raw << 16) + bias;
    if (a.softplus) dt = softplus(dt);
    const float x = __bfloat162float(x_raw), z = __bfloat162float(z_raw), du = dt * x;
    State<kBlocks> rate;
    rates.unpack(rate);
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) rate.h[k][i] = mul_pair(rate.h[k][i], pair(kLog2e, kLog2e));
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = kTogether == 4 ? i : 0;
        if (kTogether == 1) load(i, 0);
        const float step = __shfl_sync(0xffffffffu, dt, i, 4), add = __shfl_sync(0xffffffffu, du, i, 4);
        y[i] = 0.f;
        if (slot[i] >= 0) {
            State<kBlocks> s, b, key;
            states[at].unpack(s);
            bs[at].unpack(b);
            cs[at].unpack(key);
            uint64_t sum = 0ull;
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) b.h[k][j] = mul_pair(b.h[k][j], pair(add, add));
            decay<kBlocks>(s, rate, pair(step, step), b.h);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) sum = fma_pair(key.h[k][j], s.h[k][j], sum);
            y[i] = halves(sum).x + halves(sum).y;
            if (live) Row<kBlocks, StateT>::template store<kFull>(row_at(i), c, S, s);
        }
    }
    // Lane i gets the sum of sequence i over the four lanes.
    const bool up = c & 2, right = c & 1;
    float keep0 = up ? y[2] : y[0], keep1 = up ? y[3] : y[1];
    keep0 += __shfl_xor_sync(0xffffffffu, up ? y[0] : y[2], 2);
    keep1 += __shfl_xor_sync(0xffffffffu, up ? y[1] : y[3], 2);
    float sum = right ? keep1 : keep0;
    sum += __shfl_xor_sync(0xffffffffu, right ? keep0 : keep1, 1);
    if (a.D) sum = fmaf(skip, x, sum);
    if (a.z) sum *= z * sigmoid(z);
    const int mine = right ? (up ? slot[3] : slot[1]) : up ? slot[2] : slot[0];
    if (live && own < N) static_cast<__nv_bfloat16*>(a.out)[own * a.dim + ch] = __float2bfloat16_rn(mine >= 0 ? sum : 0.f);
}

template <int kBlocks, bool kStates, bool kPacked, bool kFast>
cudaError_t run(const SsmArgs& a, cudaStream_t stream) {
    constexpr int bytes = 8 * Buffer<kBlocks, kStates>::kWords;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(ssm_kernel<kBlocks, kStates, kPacked, kFast>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    if (a.spans > 0x7fffffffLL / a.tiles) return cudaErrorInvalidValue;
    return launch_after(ssm_kernel<kBlocks, kStates, kPacked, kFast>, dim3(static_cast<unsigned>(a.spans * a.tiles)), dim3(kThreads),
                        bytes, stream, a);
}

template <int kBlocks, bool kFast>
cudaError_t prefill(const SsmArgs& a, cudaStream_t stream, int* launches) {
    cudaError_t e;
    if (a.span_states) {
        e = a.cu_seqlens ? run<kBlocks, true, true, kFast>(a, stream) : run<kBlocks, true, false, kFast>(a, stream);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    e = a.cu_seqlens ? run<kBlocks, false, true, kFast>(a, stream) : run<kBlocks, false, false, kFast>(a, stream);
    if (e == cudaSuccess) ++*launches;
    return e;
}
template <int kBlocks>
cudaError_t prefill(const SsmArgs& a, cudaStream_t stream, int* launches) {
    const bool fast = a.vec && a.vec_bc && !a.dt_f32 && !a.bc_f32 && a.softplus && a.nstate == 16 * kBlocks &&
                      a.dim / a.groups % kChannels == 0;
    return fast ? prefill<kBlocks, true>(a, stream, launches) : prefill<kBlocks, false>(a, stream, launches);
}

template <int kBlocks, bool kFull, bool kStateF32, bool kKeysF32>
cudaError_t decode(const SsmArgs& a, cudaStream_t stream) {
    const int64_t blocks = (a.dim + kChannels - 1) / kChannels, parts = (a.N + 3) / 4;
    if (parts > 0x7fffffffLL / blocks) return cudaErrorInvalidValue;
    return launch_after(ssm_decode_kernel<kBlocks, kFull, kStateF32, kKeysF32>, dim3(static_cast<unsigned>(blocks * parts)),
                        dim3(kStepThreads), 0, stream, a, static_cast<int>(blocks));
}
template <int kBlocks, bool kFull>
cudaError_t pick_decode(const SsmArgs& a, cudaStream_t stream) {
    if (a.state_f32)
        return a.bc_f32 ? decode<kBlocks, kFull, true, true>(a, stream) : decode<kBlocks, kFull, true, false>(a, stream);
    return a.bc_f32 ? decode<kBlocks, kFull, false, true>(a, stream) : decode<kBlocks, kFull, false, false>(a, stream);
}
template <int kBlocks>
cudaError_t pick_decode(const SsmArgs& a, cudaStream_t stream) {
    return a.nstate == 16 * kBlocks && a.vec_bc ? pick_decode<kBlocks, true>(a, stream)
                                                : pick_decode<kBlocks, false>(a, stream);
}

bool multiple(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// Rows of a tensor that can be read n elements of `size` bytes at a time.
bool rows_of(const void* p, int64_t ld, int64_t tokens, int size, int n) {
    return !p || (multiple(p, static_cast<uintptr_t>(size * n)) && (tokens < 2 || ld % n == 0));
}
void set_vectors(SsmArgs* a) {
    a->vec = a->dim / a->groups % 4 == 0 && rows_of(a->x, a->ldx, a->tokens, 2, 4) && rows_of(a->z, a->ldz, a->tokens, 2, 4) &&
             rows_of(a->dt, a->lddt, a->tokens, a->dt_f32 ? 4 : 2, 4);
    const int size = a->bc_f32 ? 4 : 2;
    a->vec_bc = a->nstate % 4 == 0 && rows_of(a->B, a->ldb, a->tokens, size, 4) && rows_of(a->C, a->ldc, a->tokens, size, 4);
}

}  // namespace

cudaError_t launch_ssm_prefill(SsmArgs a, cudaStream_t stream, int* launches) {
    if (a.N <= 0 || a.dim <= 0) return cudaSuccess;
    set_vectors(&a);
    const int64_t bc = a.bc_f32 ? 4 : 2;
    a.tile_x = kTile * a.ldx * 2;
    a.tile_z = kTile * a.ldz * 2;
    a.tile_dt = kTile * a.lddt * (a.dt_f32 ? 4 : 2);
    a.tile_b = kTile * a.ldb * bc;
    a.tile_c = kTile * a.ldc * bc;
    a.tile_out = kTile * a.dim;
    if (a.nstate <= 16) return prefill<1>(a, stream, launches);
    if (a.nstate <= 32) return prefill<2>(a, stream, launches);
    return prefill<4>(a, stream, launches);
}

cudaError_t launch_ssm_decode(SsmArgs a, cudaStream_t stream) {
    if (a.N <= 0 || a.dim <= 0) return cudaSuccess;
    set_vectors(&a);
    if (a.nstate <= 16) return pick_decode<1>(a, stream);
    return a.nstate <= 32 ? pick_decode<2>(a, stream) : pick_decode<4>(a, stream);
}

}  // namespace kda
