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
#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_seq.cuh"
#include "kda_vec.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = kSsmTile;          // tokens at a time
constexpr int kChannels = kSsmChannels;  // channels of a CTA, 8 a warp
static_assert(kThreads == 4 * kTile && kChannels == 32, "a thread stages 8 channels of one token");
constexpr float kLog2e = 1.4426950408889634f;

// log(1 + t) / t on [0, 1]: a polynomial of degree 8 fitted to the least relative
// error (3e-8; 1.8e-7 as evaluated in FP32).
__device__ __forceinline__ uint64_t log1p_over(uint64_t t) {
    constexpr float c[] = {0.99999994f,   -0.499994934f, 0.333190978f,  -0.24842982f, 0.191060051f,
                           -0.136632428f, 0.0782259107f, -0.0295052137f, 0.00523268804f};
    uint64_t p = pair(c[8], c[8]);
#pragma unroll
    for (int i = 7; i >= 0; --i) p = fma_pair(p, t, pair(c[i], c[i]));
    return p;
}
// softplus(u) = max(u, 0) + log(1 + exp(-|u|)) of two values.  NaN stays.
__device__ __forceinline__ float2 softplus(float2 u) {
    const float2 m = make_float2(-fabsf(u.x) * kLog2e, -fabsf(u.y) * kLog2e);
    const uint64_t t = pair(exp2_fast(m.x), exp2_fast(m.y));
    const uint64_t top = pair(u.x < 0.f ? 0.f : u.x, u.y < 0.f ? 0.f : u.y);
    return halves(fma_pair(t, log1p_over(t), top));
}

// Shared memory of one of two buffers: (dt, dt x) as [channel][token] pairs, the
// rows of B and C, and y.  Strides that keep the lanes' accesses on different banks:
// a warp reads two tokens of 8 channels (16 bytes, 68 words apart), a thread
// writes one token of 8 channels (8 words more for each 8 channels).
constexpr int kStepStride = 2 * (kTile + 2);
constexpr int kStepWords = kChannels * kStepStride + 8 * (kChannels / 8);
constexpr int kYStride = kChannels + 4;
template <int kBlocks, bool kStates>
struct Buffer {
    static constexpr int kRow = 16 * kBlocks;
    static constexpr int kB = kStepWords, kC = kB + kTile * kRow, kY = kC + (kStates ? 0 : kTile * kRow);
    static constexpr int kWords = kY + (kStates ? 0 : kTile * kYStride);
};
__device__ __forceinline__ int step_at(int ch, int token) { return ch * kStepStride + 8 * (ch >> 3) + 2 * token; }

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

// D = A B for one m16n8k8 tile of TF32 operands, the sum in FP32.
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
            w.first_span = w.fresh ? span : first / a.span_tokens;
            w.seq_end = a.cu_seqlens[w.seq + 1];
        }
    } else {
        w.seq = span / a.spans_per_seq;
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

template <int kBlocks, bool kStates, bool kPacked>
__global__ void __launch_bounds__(kThreads) ssm_kernel(SsmArgs a) {
    using Buf = Buffer<kBlocks, kStates>;
    extern __shared__ __align__(16) float smem[];
    wait_for_kernel_before();
    if (kStates) let_next_kernel_come();
    if (kPacked && !offsets_hold(a.cu_seqlens, a.N, a.tokens, a.valid, a.status)) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = lane & 3;
    const int64_t span = blockIdx.x / a.tiles, tile = blockIdx.x - span * a.tiles;
    Part w = part_of<kStates, kPacked>(a, span);
    if (!w.run) return;
    const int64_t group = tile / a.tiles_per_group, per = a.dim / a.groups;
    const int64_t ch0 = group * per + (tile - group * a.tiles_per_group) * kChannels;
    const int channels = static_cast<int>((group + 1) * per - ch0 < kChannels ? (group + 1) * per - ch0 : kChannels);
    const int S = static_cast<int>(a.nstate);

    // ---- staging: 8 channels of a token, a quarter of its rows of B and C
    const int mine = 8 * (tid & 3), tok = tid >> 2;   // first channel within the CTA, token within the tile
    const int count = channels - mine < 8 ? (channels - mine > 0 ? channels - mine : 0) : 8;
    const bool wide = a.vec && count == 8;
    float bias[8], skip[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        bias[i] = a.dt_bias && i < count ? a.dt_bias[ch0 + mine + i] : 0.f;
        skip[i] = !kStates && a.D && i < count ? a.D[ch0 + mine + i] : 0.f;
    }
    auto fetch = [&](int64_t base, Fetched<kBlocks>& f) {
        const int64_t t = base + tok;
        const uint4 none = make_uint4(0, 0, 0, 0);
        f.x = f.z = f.dt[0] = f.dt[1] = none;
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) f.b[k] = f.c[k] = none;
        if (t >= w.end) return;
        const auto x = static_cast<const __nv_bfloat16*>(a.x) + t * a.ldx + ch0 + mine;
        const auto z = static_cast<const __nv_bfloat16*>(a.z) + t * a.ldz + ch0 + mine;
        const int64_t dt_at = t * a.lddt + ch0 + mine;
        if (wide) {
            f.x = *reinterpret_cast<const uint4*>(x);
            if (!kStates && a.z) f.z = *reinterpret_cast<const uint4*>(z);
            if (a.dt_f32) {
                const auto p = reinterpret_cast<const uint4*>(static_cast<const float*>(a.dt) + dt_at);
                f.dt[0] = p[0];
                f.dt[1] = p[1];
            } else {
                f.dt[0] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.dt) + dt_at);
            }
        } else {
            f.x = gather8(x, count);
            if (!kStates && a.z) f.z = gather8(z, count);
            if (a.dt_f32) {
                f.dt[0] = gather4(static_cast<const float*>(a.dt) + dt_at, count);
                f.dt[1] = gather4(static_cast<const float*>(a.dt) + dt_at + 4, count - 4);
            } else {
                f.dt[0] = gather8(static_cast<const __nv_bfloat16*>(a.dt) + dt_at, count);
            }
        }
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int n0 = 16 * k + 4 * (tid & 3);
            const int64_t b_at = t * a.ldb + group * S + n0, c_at = t * a.ldc + group * S + n0;
            const int have = S - n0;
            if (have <= 0) continue;
            if (a.bc_f32) {
                const float *b = static_cast<const float*>(a.B) + b_at, *cc = static_cast<const float*>(a.C) + c_at;
                if (a.vec_bc) {
                    f.b[k] = *reinterpret_cast<const uint4*>(b);
                    if (!kStates) f.c[k] = *reinterpret_cast<const uint4*>(cc);
                } else {
                    f.b[k] = gather4(b, have);
                    if (!kStates) f.c[k] = gather4(cc, have);
                }
            } else {
                const auto b = static_cast<const __nv_bfloat16*>(a.B) + b_at, cc = static_cast<const __nv_bfloat16*>(a.C) + c_at;
                if (a.vec_bc) {
                    const uint2 rb = *reinterpret_cast<const uint2*>(b);
                    f.b[k] = make_uint4(rb.x, rb.y, 0, 0);
                    if (!kStates) {
                        const uint2 rc = *reinterpret_cast<const uint2*>(cc);
                        f.c[k] = make_uint4(rc.x, rc.y, 0, 0);
                    }
                } else {
                    f.b[k] = gather8(b, have < 4 ? have : 4);
                    if (!kStates) f.c[k] = gather8(cc, have < 4 ? have : 4);
                }
            }
        }
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
    auto stage = [&](int64_t base, const Fetched<kBlocks>& f, float* buf) {
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
        const bool here = base + tok < w.end;   // behind the end nothing decays and nothing is added
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float2 dt = make_float2(u[i] + bias[i], u[i + 1] + bias[i + 1]);
            if (a.softplus) dt = softplus(dt);
            if (!here) dt = make_float2(0.f, 0.f);
            *reinterpret_cast<float2*>(buf + step_at(mine + i, tok)) = make_float2(dt.x, dt.x * x[i]);
            *reinterpret_cast<float2*>(buf + step_at(mine + i + 1, tok)) = make_float2(dt.y, dt.y * x[i + 1]);
        }
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int at = tok * Buf::kRow + 16 * k + 4 * (tid & 3);
            *reinterpret_cast<float4*>(buf + Buf::kB + at) = four(f.b[k]);
            if (!kStates) {
                float4 keys = four(f.c[k]);
                if (a.bc_f32) keys = make_float4(tf32(keys.x), tf32(keys.y), tf32(keys.z), tf32(keys.w));
                *reinterpret_cast<float4*>(buf + Buf::kC + at) = keys;
            }
        }
    };
    // A token's outputs from its y: the skip, the gate and one rounding.
    auto finish = [&](int64_t base, const uint4& xr, const uint4& zr, const float* buf) {
        const int64_t t = base + tok;
        if (t >= w.end) return;
        float y[8], x[8], z[8];
        const float4* p = reinterpret_cast<const float4*>(buf + Buf::kY + tok * kYStride + mine);
        const float4 lo = p[0], hi = p[1];
        y[0] = lo.x; y[1] = lo.y; y[2] = lo.z; y[3] = lo.w; y[4] = hi.x; y[5] = hi.y; y[6] = hi.z; y[7] = hi.w;
        unpack8(xr, x);
        unpack8(zr, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (a.D) y[i] = fmaf(skip[i], x[i], y[i]);
            if (a.z) y[i] *= z[i] * sigmoid(z[i]);
        }
        const auto out = static_cast<__nv_bfloat16*>(a.out) + t * a.dim + ch0 + mine;
        if (a.vec && count == 8) {
            store8(out, y);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < count) out[i] = __float2bfloat16_rn(y[i]);
        }
    };

    // ---- the walk: a warp's 8 channels, four lanes each
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
    Fetched<kBlocks> f;
    if (w.begin < w.end) fetch(w.begin, f);
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
    // The states of the sequences that end at token t, and the next one's.
    int64_t seq = w.seq, seq_end = w.seq_end;
    auto close = [&](int64_t t) {
        while (t == seq_end) {
            ending(seq);
            if (!kPacked || ++seq >= a.N) break;
            seq_end = a.cu_seqlens[seq + 1];
            initial(seq);
        }
    };
    if (!kStates) close(w.begin);

    float steps = 0.f;   // the sum of dt
    if (w.begin < w.end) {
        stage(w.begin, f, smem);
        __syncthreads();
    }
    int which = 0;
    for (int64_t base = w.begin; base < w.end; base += kTile) {
        float* buf = smem + which * Buf::kWords;
        const uint4 xr = f.x, zr = f.z;
        const bool more = base + kTile < w.end;
        if (more) fetch(base + kTile, f);
        const float* step = buf + step_at(local, 0);
        const float* rows = buf + Buf::kB + 4 * c;
        const float* keys = buf + Buf::kC + ((lane >> 3) * Buf::kRow) + 4 * c + 2 * ((lane >> 2) & 1);
        const int n = static_cast<int>(w.end - base < kTile ? w.end - base : kTile);
        // Where the sequence ends within the tile (packed).
        int left = kPacked && !kStates && seq_end - base <= kTile ? static_cast<int>(seq_end - base) : kTile + 4;
#pragma unroll 1
        for (int t = 0; t < n; t += 4) {
            float dts[4], dus[4], ck[kBlocks][2], y = 0.f;
            {
                const float4 p = *reinterpret_cast<const float4*>(step + 2 * t), q = *reinterpret_cast<const float4*>(step + 2 * t + 4);
                dts[0] = p.x; dus[0] = p.y; dts[1] = p.z; dus[1] = p.w;
                dts[2] = q.x; dus[2] = q.y; dts[3] = q.z; dus[3] = q.w;
            }
            if (!kStates)
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    const float2 v = *reinterpret_cast<const float2*>(keys + t * Buf::kRow + 16 * k);
                    ck[k][0] = v.x;
                    ck[k][1] = v.y;
                }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint64_t b[kBlocks][2];
                const uint64_t du = pair(dus[j], dus[j]);
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    const float4 v = *reinterpret_cast<const float4*>(rows + (t + j) * Buf::kRow + 16 * k);
                    b[k][0] = mul_pair(du, pair(v.x, v.y));
                    b[k][1] = mul_pair(du, pair(v.z, v.w));
                }
                decay<kBlocks>(s, rate, pair(dts[j], dts[j]), b);
                if (kStates) {
                    steps += dts[j];
                } else {
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int k = 0; k < kBlocks; ++k) {
                        const float2 lo = halves(s.h[k][0]), hi = halves(s.h[k][1]);
                        mma_tf32(acc, lo.x, hi.x, lo.y, hi.y, ck[k][0], ck[k][1]);
                    }
                    // (The columns of the group's other tokens hold nothing of use.)
                    if (c == j) y = acc[0] + acc[3];
                    if (kPacked && t + j + 1 == left) {
                        close(base + left);
                        left = seq_end - base <= kTile ? static_cast<int>(seq_end - base) : kTile + 4;
                    }
                }
            }
            if (!kStates) buf[Buf::kY + (t + c) * kYStride + local] = y;
        }
        if (!kPacked && !kStates && base + n == seq_end) close(seq_end);
        if (more) stage(base + kTile, f, smem + (which ^ 1) * Buf::kWords);
        __syncthreads();
        if (!kStates) finish(base, xr, zr, buf);
        which ^= 1;
    }
    if (kStates && live) {
        store_row<kBlocks>(a.span_states, true, span * a.dim + ch, c, 16 * kBlocks, s);
        if (c == 0) a.span_steps[span * a.dim + ch] = steps;
    }
}

// ---- single tokens: four lanes a channel, kSeqs sequences a thread
template <int kBlocks, int kSeqs>
__global__ void __launch_bounds__(256) ssm_decode_kernel(SsmArgs a) {
    wait_for_kernel_before();
    const int c = threadIdx.x & 3, S = static_cast<int>(a.nstate);
    const int64_t blocks = (a.dim + 63) / 64, part = blockIdx.x / blocks;
    const int64_t ch_raw = (blockIdx.x - part * blocks) * 64 + (threadIdx.x >> 2);
    const bool live = ch_raw < a.dim;
    const int64_t ch = live ? ch_raw : a.dim - 1, group = ch / (a.dim / a.groups);
    int64_t slot[kSeqs];
    State<kBlocks> s[kSeqs];
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int64_t n = part * kSeqs + i;
        slot[i] = n < a.N ? (a.slots ? a.slots[n] : n) : -1;
        if (slot[i] >= a.pool) {
            if (ch_raw == 0 && c == 0) atomicOr(a.status, kDevBadSlots);
            slot[i] = -1;
        }
        if (slot[i] >= 0) load_row<kBlocks>(a.state, a.state_f32, slot[i] * a.dim + ch, c, S, s[i]);
    }
    State<kBlocks> rate;
    load_row<kBlocks>(a.A, true, ch, c, S, rate);
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) rate.h[k][i] = mul_pair(rate.h[k][i], pair(kLog2e, kLog2e));
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f, skip = a.D ? a.D[ch] : 0.f;
    auto bf16_at = [](const void* p, int64_t at) { return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]); };
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int64_t n = part * kSeqs + i;
        if (n >= a.N) break;
        float y = 0.f;
        if (slot[i] >= 0) {   // (the same for the whole CTA)
            const float x = bf16_at(a.x, n * a.ldx + ch);
            float dt = (a.dt_f32 ? static_cast<const float*>(a.dt)[n * a.lddt + ch] : bf16_at(a.dt, n * a.lddt + ch)) + bias;
            if (a.softplus) dt = softplus(make_float2(dt, dt)).x;
            uint64_t b[kBlocks][2];
            const uint64_t du = pair(dt * x, dt * x);
            const int es = a.bc_f32 ? 4 : 2;
            State<kBlocks> bs, cs;
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                const int n0 = 16 * k + 4 * c;
                const auto bp = static_cast<const uint8_t*>(a.B) + (n * a.ldb + group * S) * es,
                           cp = static_cast<const uint8_t*>(a.C) + (n * a.ldc + group * S) * es;
                float v[4], u[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[j] = u[j] = 0.f;
                    if (n0 + j < S) {
                        v[j] = a.bc_f32 ? reinterpret_cast<const float*>(bp)[n0 + j] : bf16_at(bp, n0 + j);
                        u[j] = a.bc_f32 ? reinterpret_cast<const float*>(cp)[n0 + j] : bf16_at(cp, n0 + j);
                    }
                }
                bs.h[k][0] = pair(v[0], v[1]);
                bs.h[k][1] = pair(v[2], v[3]);
                cs.h[k][0] = pair(u[0], u[1]);
                cs.h[k][1] = pair(u[2], u[3]);
                b[k][0] = mul_pair(du, bs.h[k][0]);
                b[k][1] = mul_pair(du, bs.h[k][1]);
            }
            decay<kBlocks>(s[i], rate, pair(dt, dt), b);
            uint64_t sum = 0ull;
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                sum = fma_pair(cs.h[k][0], s[i].h[k][0], sum);
                sum = fma_pair(cs.h[k][1], s[i].h[k][1], sum);
            }
            const float2 both = halves(sum);
            y = both.x + both.y;
            y += __shfl_xor_sync(0xffffffffu, y, 1);
            y += __shfl_xor_sync(0xffffffffu, y, 2);
            if (a.D) y = fmaf(skip, x, y);
            if (a.z) {
                const float z = bf16_at(a.z, n * a.ldz + ch);
                y *= z * sigmoid(z);
            }
            if (live) store_row<kBlocks>(a.state, a.state_f32, slot[i] * a.dim + ch, c, S, s[i]);
        }
        if (live && c == 0) static_cast<__nv_bfloat16*>(a.out)[n * a.dim + ch] = __float2bfloat16_rn(y);
    }
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

template <int kBlocks, int kSeqs>
cudaError_t decode(const SsmArgs& a, cudaStream_t stream) {
    const int64_t blocks = (a.dim + 63) / 64, parts = (a.N + kSeqs - 1) / kSeqs;
    if (parts > 0x7fffffffLL / blocks) return cudaErrorInvalidValue;
    return launch_after(ssm_decode_kernel<kBlocks, kSeqs>, dim3(static_cast<unsigned>(parts * blocks)), dim3(256), 0, stream, a);
}
template <int kBlocks>
cudaError_t pick_decode(const SsmArgs& a, int sms, cudaStream_t stream) {
    // Four sequences a thread share its rates where that still fills the SMs.
    constexpr int kMany = kBlocks == 1 ? 4 : 2;
    if (a.N / kMany * ((a.dim + 63) / 64) >= 4 * static_cast<int64_t>(sms)) return decode<kBlocks, kMany>(a, stream);
    return decode<kBlocks, 1>(a, stream);
}

bool multiple(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

cudaError_t launch_ssm_prefill(SsmArgs a, cudaStream_t stream, int* launches) {
    if (a.N <= 0 || a.dim <= 0) return cudaSuccess;
    const int64_t per = a.dim / a.groups;
    // Rows that can be read 8 channels (4 states) at a time.
    auto rows = [&](const void* p, int64_t ld, int size, int n) {
        return !p || (multiple(p, static_cast<uintptr_t>(size * n)) && (a.tokens < 2 || ld % n == 0));
    };
    a.vec = per % 8 == 0 && rows(a.x, a.ldx, 2, 8) && rows(a.z, a.ldz, 2, 8) &&
            (a.dt_f32 ? rows(a.dt, a.lddt, 4, 4) : rows(a.dt, a.lddt, 2, 8));
    const int size = a.bc_f32 ? 4 : 2;
    a.vec_bc = a.nstate % 4 == 0 && rows(a.B, a.ldb, size, 4) && rows(a.C, a.ldc, size, 4);
    if (a.nstate <= 16) return prefill<1>(a, stream, launches);
    if (a.nstate <= 32) return prefill<2>(a, stream, launches);
    return prefill<4>(a, stream, launches);
}

cudaError_t launch_ssm_decode(const SsmArgs& a, int sms, cudaStream_t stream) {
    if (a.N <= 0 || a.dim <= 0) return cudaSuccess;
    if (a.nstate <= 16) return pick_decode<1>(a, sms, stream);
    if (a.nstate <= 32) return pick_decode<2>(a, sms, stream);
    return pick_decode<4>(a, sms, stream);
}

}  // namespace kda
