// kda_ssm.cu -- the selective state space scan (sm_103a).
//
// For each channel d of a sequence, with states n = 0 .. S - 1:
//     dt = softplus(dt_raw + bias_d),  h[n] <- exp(dt A[d][n]) h[n] + dt x B[n],
//     y = sum_n C[n] h[n] + D_d x,  out = y silu(z);
// B and C are shared by a group of channels.
//
// Prompts (ssm_kernel).  The decays differ in every channel and state, so there is
// no product of matrices in it: 8 S + 20 operations for 8 bytes, of which S
// exponentials, bound by the SMs' arithmetic.  A CTA has 32 channels and a span of
// tokens, 32 at a time: its threads form dt, dt x and the rows of B and C as FP32
// in shared memory, then a warp walks 8 channels through the tokens with the
// states in registers, four lanes a channel and S / 4 states a lane.  The states
// lie as the A operand of an m16n8k8 product (TF32): for one token, its rows are
// the 8 channels' states twice over, half of the 16 states in each, and
// column 2 t + i of the B operand has half i of token t's C, so that one
// instruction gives sum_n C[n] h[n] of 8 channels, without shuffles.  That takes
// h to TF32 on its way to out (cut to 10 bits: at most 2^-10 of |C[n] h[n]|, where out's own
// rounding to BF16 is 2^-9 of out); the states themselves stay FP32.
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

// softplus(u) = max(u, 0) + log(1 + exp(-|u|)) of n pairs.  log(1 + t) / t on [0, 1]
// is a polynomial of degree 8 fitted to the least relative error (3e-8; 1.8e-7 as
// evaluated in FP32), all pairs a coefficient at a time.  NaN stays (through exp).
template <int n>
__device__ __forceinline__ void softplus(float2 (&u)[n]) {
    constexpr float c[] = {0.99999994f,   -0.499994934f, 0.333190978f,  -0.24842982f, 0.191060051f,
                           -0.136632428f, 0.0782259107f, -0.0295052137f, 0.00523268804f};
    uint64_t t[n], p[n];
#pragma unroll
    for (int i = 0; i < n; ++i) {
        t[i] = pair(exp2_fast(fabsf(u[i].x) * -kLog2e), exp2_fast(fabsf(u[i].y) * -kLog2e));
        p[i] = pair(c[8], c[8]);
    }
#pragma unroll
    for (int k = 7; k >= 0; --k) {
        const uint64_t ck = pair(c[k], c[k]);
#pragma unroll
        for (int i = 0; i < n; ++i) p[i] = fma_pair(p[i], t[i], ck);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) u[i] = halves(fma_pair(t[i], p[i], pair(fmaxf(u[i].x, 0.f), fmaxf(u[i].y, 0.f))));
}

// Shared memory of one of two buffers: (dt, dt, dt x, dt x) for each channel and
// token, as the packed instructions take them (made from one value each, the pairs
// cost two more instructions a token), the rows of B and C, and y.  Strides that keep the lanes'
// accesses on different banks: a warp reads one token of 8 channels (16 bytes each),
// a thread writes 8 channels of one token (8 words more for each 8 channels).
constexpr int kStepStride = 4 * (kTile + 1);
constexpr int kStepWords = kChannels * kStepStride + 8 * (kChannels / 8);
constexpr int kYStride = kChannels + 4;
template <int kBlocks, bool kStates>
struct Buffer {
    static constexpr int kRow = 16 * kBlocks;
    static constexpr int kB = kStepWords, kC = kB + kTile * kRow, kY = kC + (kStates ? 0 : kTile * kRow);
    static constexpr int kXZ = kY + (kStates ? 0 : kTile * kYStride);   // x and z of each staging thread, for its outputs
    static constexpr int kWords = kXZ + (kStates ? 0 : 8 * kRole);
};
__device__ __forceinline__ int step_at(int ch, int token) { return ch * kStepStride + 8 * (ch >> 3) + 4 * token; }

// What a thread stages of a tile, as loaded: 8 channels of one token, and for
// each block of 16 states 4 values of B and of C.
template <int kBlocks>
struct Fetched {
    uint4 x, z, dt[2], b[kBlocks], c[kBlocks];
};

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

template <int kBlocks>
struct State {   // a lane's 4 kBlocks states of its channel: 16 k + 4 c + {0 .. 3}, c the lane's place among four
    uint64_t h[kBlocks][2];
};

// Four values from state n0 on of a row of S.
template <typename T>
__device__ __forceinline__ void load_states(const T* row, int n0, int S, float (&v)[4]) {
    if (S % 4 == 0) {
        if (n0 < S) {
            if constexpr (sizeof(T) == 4) {
                const float4 r = *reinterpret_cast<const float4*>(row + n0);
                v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
            } else {
                const uint2 r = *reinterpret_cast<const uint2*>(row + n0);
                v[0] = bf16_lo(r.x); v[1] = bf16_hi(r.x); v[2] = bf16_lo(r.y); v[3] = bf16_hi(r.y);
            }
        } else {
            v[0] = v[1] = v[2] = v[3] = 0.f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = n0 + i < S ? static_cast<float>(row[n0 + i]) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store_states(T* row, int n0, int S, const float (&v)[4]) {
    if (S % 4 == 0) {
        if (n0 < S) {
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<float4*>(row + n0) = make_float4(v[0], v[1], v[2], v[3]);
            else
                *reinterpret_cast<uint2*>(row + n0) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n0 + i < S) from_f32(row + n0 + i, v[i]);
    }
}

template <int kBlocks>
__device__ __forceinline__ void load_row(const void* p, bool f32, int64_t row, int c, int S, State<kBlocks>& s) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        float v[4];
        if (f32)
            load_states(static_cast<const float*>(p) + row * S, 16 * k + 4 * c, S, v);
        else
            load_states(static_cast<const __nv_bfloat16*>(p) + row * S, 16 * k + 4 * c, S, v);
        s.h[k][0] = pair(v[0], v[1]);
        s.h[k][1] = pair(v[2], v[3]);
    }
}
template <int kBlocks>
__device__ __forceinline__ void store_row(void* p, bool f32, int64_t row, int c, int S, const State<kBlocks>& s) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
        const float2 a = halves(s.h[k][0]), b = halves(s.h[k][1]);
        const float v[4] = {a.x, a.y, b.x, b.y};
        if (f32)
            store_states(static_cast<float*>(p) + row * S, 16 * k + 4 * c, S, v);
        else
            store_states(static_cast<__nv_bfloat16*>(p) + row * S, 16 * k + 4 * c, S, v);
    }
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
                store_states(row, n0, 16 * kBlocks, v);
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
template <int kBlocks, bool kStates, bool kPacked>
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
    const int channels = static_cast<int>((group + 1) * per - ch0 < kChannels ? (group + 1) * per - ch0 : kChannels);
    const int S = static_cast<int>(a.nstate);
    const int tid = threadIdx.x & (kRole - 1);
    const int64_t total = w.end - w.begin;   // tokens; tiles i = 0 .. tiles - 1 of them
    const int tiles = static_cast<int>((total + kTile - 1) / kTile);

    if (threadIdx.x >= kRole) {
        // ---- staging: 8 channels of a token, a quarter of its rows of B and C
        const int mine = 8 * (tid & 3), tok = tid >> 2;   // first channel within the CTA, token within the tile
        const int count = channels - mine < 8 ? (channels - mine > 0 ? channels - mine : 0) : 8;
        const bool wide = a.vec && count == 8, gated = !kStates && a.z;
        float bias[8], skip[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            bias[i] = a.dt_bias && i < count ? a.dt_bias[ch0 + mine + i] : 0.f;
            skip[i] = !kStates && a.D && i < count ? a.D[ch0 + mine + i] : 0.f;
        }
        // This thread's rows of the tile to fetch next, and to finish.
        const int es = a.bc_f32 ? 4 : 2, dts = a.dt_f32 ? 4 : 2;
        const int64_t t0 = w.begin + tok;
        auto xp = static_cast<const __nv_bfloat16*>(a.x) + t0 * a.ldx + ch0 + mine;
        auto zp = static_cast<const __nv_bfloat16*>(a.z) + t0 * a.ldz + ch0 + mine;
        auto dp = static_cast<const uint8_t*>(a.dt) + (t0 * a.lddt + ch0 + mine) * dts;
        auto bp = static_cast<const uint8_t*>(a.B) + (t0 * a.ldb + group * S + 4 * (tid & 3)) * es;
        auto cp = static_cast<const uint8_t*>(a.C) + (t0 * a.ldc + group * S + 4 * (tid & 3)) * es;
        auto op = static_cast<__nv_bfloat16*>(a.out) + t0 * a.dim + ch0 + mine;
        const int64_t xs = kTile * a.ldx, zs = kTile * a.ldz, ds = kTile * a.lddt * dts, bs = kTile * a.ldb * es,
                      cs = kTile * a.ldc * es, os = kTile * a.dim;
        auto fetch = [&](int i, Fetched<kBlocks>& f) {
            if (i * kTile + tok < total) {
                if (wide) {
                    f.x = *reinterpret_cast<const uint4*>(xp);
                    if (gated) f.z = *reinterpret_cast<const uint4*>(zp);
                    f.dt[0] = *reinterpret_cast<const uint4*>(dp);
                    if (a.dt_f32) f.dt[1] = *reinterpret_cast<const uint4*>(dp + 16);
                } else {
                    f.x = gather8(xp, count);
                    if (gated) f.z = gather8(zp, count);
                    if (a.dt_f32) {
                        f.dt[0] = gather4(reinterpret_cast<const float*>(dp), count);
                        f.dt[1] = gather4(reinterpret_cast<const float*>(dp) + 4, count - 4);
                    } else {
                        f.dt[0] = gather8(reinterpret_cast<const __nv_bfloat16*>(dp), count);
                    }
                }
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    const int have = S - 16 * k - 4 * (tid & 3);
                    const uint8_t *b = bp + 16 * k * es, *cc = cp + 16 * k * es;
                    if (have <= 0) {
                        f.b[k] = f.c[k] = make_uint4(0, 0, 0, 0);
                    } else if (a.vec_bc && a.bc_f32) {
                        f.b[k] = *reinterpret_cast<const uint4*>(b);
                        if (!kStates) f.c[k] = *reinterpret_cast<const uint4*>(cc);
                    } else if (a.vec_bc) {
                        const uint2 rb = *reinterpret_cast<const uint2*>(b);
                        f.b[k].x = rb.x;
                        f.b[k].y = rb.y;
                        if (!kStates) {
                            const uint2 rc = *reinterpret_cast<const uint2*>(cc);
                            f.c[k].x = rc.x;
                            f.c[k].y = rc.y;
                        }
                    } else if (a.bc_f32) {
                        f.b[k] = gather4(reinterpret_cast<const float*>(b), have);
                        if (!kStates) f.c[k] = gather4(reinterpret_cast<const float*>(cc), have);
                    } else {
                        f.b[k] = gather8(reinterpret_cast<const __nv_bfloat16*>(b), have < 4 ? have : 4);
                        if (!kStates) f.c[k] = gather8(reinterpret_cast<const __nv_bfloat16*>(cc), have < 4 ? have : 4);
                    }
                }
            } else {
                f.x = f.z = f.dt[0] = f.dt[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) f.b[k] = f.c[k] = make_uint4(0, 0, 0, 0);
            }
            xp += xs;
            if (gated) zp += zs;
            dp += ds;
            bp += bs;
            if (!kStates) cp += cs;
        };
        // To the nearest TF32 value, which a BF16 one is.
        auto tf32 = [](float v) {
            uint32_t r;
            asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
            return __uint_as_float(r);
        };
        auto four = [&](const uint4& r) {
            return a.bc_f32 ? make_float4(__uint_as_float(r.x), __uint_as_float(r.y), __uint_as_float(r.z), __uint_as_float(r.w))
                            : make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
        };
        auto stage = [&](int i, const Fetched<kBlocks>& f) {
            float* buf = smem + (i & 1) * Buf::kWords;
            float u[8], x[8];
            unpack8(f.x, x);
            if (a.dt_f32) {
                u[0] = __uint_as_float(f.dt[0].x); u[1] = __uint_as_float(f.dt[0].y);
                u[2] = __uint_as_float(f.dt[0].z); u[3] = __uint_as_float(f.dt[0].w);
                u[4] = __uint_as_float(f.dt[1].x); u[5] = __uint_as_float(f.dt[1].y);
                u[6] = __uint_as_float(f.dt[1].z); u[7] = __uint_as_float(f.dt[1].w);
            } else {
                unpack8(f.dt[0], u);
            }
            float2 dt[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) dt[j] = make_float2(u[2 * j] + bias[2 * j], u[2 * j + 1] + bias[2 * j + 1]);
            if (a.softplus) softplus(dt);
            if (i * kTile + tok >= total)   // behind the end nothing decays and nothing is added
#pragma unroll
                for (int j = 0; j < 4; ++j) dt[j] = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float v = dt[j].x * x[2 * j], v1 = dt[j].y * x[2 * j + 1];
                *reinterpret_cast<float4*>(buf + step_at(mine + 2 * j, tok)) = make_float4(dt[j].x, dt[j].x, v, v);
                *reinterpret_cast<float4*>(buf + step_at(mine + 2 * j + 1, tok)) = make_float4(dt[j].y, dt[j].y, v1, v1);
            }
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                const int at = tok * Buf::kRow + 16 * k + 4 * (tid & 3);
                *reinterpret_cast<float4*>(buf + Buf::kB + at) = four(f.b[k]);
                if (!kStates) {
                    // (In the order in which the product's B operand takes them.)
                    const float4 v = four(f.c[k]);
                    *reinterpret_cast<float4*>(buf + Buf::kC + at) =
                        a.bc_f32 ? make_float4(tf32(v.x), tf32(v.z), tf32(v.y), tf32(v.w)) : make_float4(v.x, v.z, v.y, v.w);
                }
            }
            if (!kStates) {
                uint4* xz = reinterpret_cast<uint4*>(buf + Buf::kXZ) + tid;
                xz[0] = f.x;
                if (gated) xz[kRole] = f.z;
            }
        };
        // A token's outputs from its y: the skip, the gate and one rounding.
        auto finish = [&](int i) {
            const float* buf = smem + (i & 1) * Buf::kWords;
            if (i * kTile + tok < total) {
                float y[8], x[8], z[8];
                const float4* p = reinterpret_cast<const float4*>(buf + Buf::kY + tok * kYStride + mine);
                const float4 lo = p[0], hi = p[1];
                y[0] = lo.x; y[1] = lo.y; y[2] = lo.z; y[3] = lo.w; y[4] = hi.x; y[5] = hi.y; y[6] = hi.z; y[7] = hi.w;
                const uint4* xz = reinterpret_cast<const uint4*>(buf + Buf::kXZ) + tid;
                if (a.D) {
                    unpack8(xz[0], x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = fmaf(skip[j], x[j], y[j]);
                }
                if (gated) {
                    unpack8(xz[kRole], z);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= z[j] * sigmoid(z[j]);
                }
                if (wide) {
                    store8(op, y);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < count) op[j] = __float2bfloat16_rn(y[j]);
                }
            }
            op += os;
        };
        Fetched<kBlocks> f;
        if (tiles > 0) {
            fetch(0, f);
            stage(0, f);
            fetch(1, f);
        }
        __syncthreads();
        for (int i = 0; i < tiles; ++i) {
            if (!kStates && i > 0) finish(i - 1);
            if (i + 1 < tiles) {
                stage(i + 1, f);
                fetch(i + 2, f);
            }
            __syncthreads();
        }
        if (!kStates && tiles > 0) finish(tiles - 1);
        return;
    }

    // ---- the walk: a warp's 8 channels, four lanes each
    const int warp = tid >> 5, lane = tid & 31, c = lane & 3;
    const int local = 8 * warp + (lane >> 2);
    const bool live = local < channels;
    const int64_t ch = ch0 + (live ? local : 0);
    State<kBlocks> rate, s;
    load_row<kBlocks>(a.A, true, ch, c, S, rate);
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) rate.h[k][i] = mul_pair(rate.h[k][i], pair(kLog2e, kLog2e));
    auto initial = [&](int64_t seq) {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) s.h[k][0] = s.h[k][1] = 0ull;
        if (a.init_state) load_row<kBlocks>(a.init_state, a.state_f32, seq * a.dim + ch, c, S, s);
    };
    auto ending = [&](int64_t seq) {
        if (a.final_state && live) store_row<kBlocks>(a.final_state, a.state_f32, seq * a.dim + ch, c, S, s);
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
                load_row<kBlocks>(a.span_states, true, i * a.dim + ch, c, 16 * kBlocks, add);
                const float dt = a.span_steps[i * a.dim + ch];
                decay<kBlocks>(s, rate, pair(dt, dt), add.h);
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
    float steps = 0.f;   // the sum of dt
    const int step0 = step_at(local, 0), rows0 = Buf::kB + 4 * c, y0 = Buf::kY + c * kYStride + local;
    const int keys0 = Buf::kC + (lane >> 3) * Buf::kRow + 4 * c + 2 * ((lane >> 2) & 1);
    // Four tokens from t on of the tile at `base`; with `ends`, sequences may end
    // among them.  (Tokens behind the span's end change nothing: only the last span
    // has them, and no sequence behind it.)
    auto walk = [&](auto ends, const float* buf, int64_t base, int t) {
        float ck[kBlocks][2], y = 0.f;
        if (!kStates)
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                const float2 v = *reinterpret_cast<const float2*>(buf + keys0 + t * Buf::kRow + 16 * k);
                ck[k][0] = v.x;
                ck[k][1] = v.y;
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint64_t b[kBlocks][2];
            const ulonglong2 dd = *reinterpret_cast<const ulonglong2*>(buf + step0 + 4 * (t + j));   // dt twice, dt x twice
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(buf + rows0 + (t + j) * Buf::kRow + 16 * k);
                b[k][0] = mul_pair(dd.y, v.x);
                b[k][1] = mul_pair(dd.y, v.y);
            }
            decay<kBlocks>(s, rate, dd.x, b);
            if (kStates) {
                steps += halves(dd.x).x;
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
                // (The columns of the group's other tokens hold nothing of use.)
                if (c == j) y = acc[0] + acc[3];
                if (decltype(ends)::value) close(base + t + j + 1);
            }
        }
        return y;   // of token t + c
    };
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        float* buf = smem + (i & 1) * Buf::kWords;
        const int64_t base = static_cast<int64_t>(i) * kTile;
        if (base + kTile <= total && (!kPacked || kStates || seq_end >= base + kTile)) {
            // (y is stored behind all loads: the compiler keeps their order.)
            float y[kTile / 4];
#pragma unroll
            for (int t = 0; t < kTile; t += 4) y[t / 4] = walk(std::false_type{}, buf, base, t);
            if (!kStates)
#pragma unroll
                for (int t = 0; t < kTile; t += 4) buf[y0 + t * kYStride] = y[t / 4];
            if (kPacked && !kStates) close(base + kTile);
        } else {
#pragma unroll 1
            for (int t = 0; t < kTile && base + t < total; t += 4) {
                const float y = walk(std::integral_constant<bool, kPacked && !kStates>{}, buf, base, t);
                if (!kStates) buf[y0 + t * kYStride] = y;
            }
        }
        __syncthreads();
    }
    if (!kPacked && !kStates && total == seq_end && total > 0) close(total);
    if (kStates && live) {
        store_row<kBlocks>(a.span_states, true, span * a.dim + ch, c, 16 * kBlocks, s);
        if (c == 0) a.span_steps[span * a.dim + ch] = steps;
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

    float2 dt[1] = {make_float2(__uint_as_float(a.dt_f32 ? dt_raw : dt_raw << 16) + bias, 0.f)};
    if (a.softplus) softplus(dt);
    const float x = __bfloat162float(x_raw), z = __bfloat162float(z_raw), du = dt[0].x * x;
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
        const float step = __shfl_sync(0xffffffffu, dt[0].x, i, 4), add = __shfl_sync(0xffffffffu, du, i, 4);
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

template <int kBlocks, bool kStates, bool kPacked>
cudaError_t run(const SsmArgs& a, int64_t spans, cudaStream_t stream) {
    constexpr int bytes = 2 * Buffer<kBlocks, kStates>::kWords * 4;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(ssm_kernel<kBlocks, kStates, kPacked>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    if (spans > 0x7fffffffLL / a.tiles) return cudaErrorInvalidValue;
    return launch_after(ssm_kernel<kBlocks, kStates, kPacked>, dim3(static_cast<unsigned>(spans * a.tiles)), dim3(kThreads),
                        bytes, stream, a);
}

template <int kBlocks>
cudaError_t prefill(const SsmArgs& a, cudaStream_t stream, int* launches) {
    cudaError_t e;
    if (a.span_states) {
        e = a.cu_seqlens ? run<kBlocks, true, true>(a, a.spans, stream) : run<kBlocks, true, false>(a, a.spans, stream);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    e = a.cu_seqlens ? run<kBlocks, false, true>(a, a.spans, stream) : run<kBlocks, false, false>(a, a.spans, stream);
    if (e == cudaSuccess) ++*launches;
    return e;
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
    a->vec = a->dim / a->groups % 8 == 0 && rows_of(a->x, a->ldx, a->tokens, 2, 8) && rows_of(a->z, a->ldz, a->tokens, 2, 8) &&
             (a->dt_f32 ? rows_of(a->dt, a->lddt, a->tokens, 4, 4) : rows_of(a->dt, a->lddt, a->tokens, 2, 8));
    const int size = a->bc_f32 ? 4 : 2;
    a->vec_bc = a->nstate % 4 == 0 && rows_of(a->B, a->ldb, a->tokens, size, 4) && rows_of(a->C, a->ldc, a->tokens, size, 4);
}

}  // namespace

cudaError_t launch_ssm_prefill(SsmArgs a, cudaStream_t stream, int* launches) {
    if (a.N <= 0 || a.dim <= 0) return cudaSuccess;
    set_vectors(&a);
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
