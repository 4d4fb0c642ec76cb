// kda_ssm_scan.cuh -- the selective state space scan of prompts (sm_103a).
//
// For each channel d of a sequence, with states n = 0 .. S - 1:
//     dt = softplus(dt_raw + bias_d),  h[n] <- exp(dt A[d][n]) h[n] + dt x B[n],
//     y = sum_n C[n] h[n] + D_d x,  out = y silu(z);
// B and C are shared by a group of channels.
//
// The decays differ in every channel and state, so there is no product of matrices
// in it: 8 S + 20 operations for 8 bytes, of which S exponentials.  A CTA has 32
// channels and a span of tokens, 32 at a time: some of its threads form dt, dt x and the rows of B and C as FP32 in
// shared memory; the warps of the others walk 16 channels and a half (of 64 states
// a quarter) of the states through the tokens, two channels and two states of every eight
// in a lane's registers, so that what a lane reads serves four.  The states lie as the A operand of an
// m16n8k8 product (TF32), four registers that it takes as they are: rows are
// channels, and column j of the B operand is token j's C, so that one instruction
// gives sum_n C[n] h[n] of 16 channels, without shuffles.  That takes h to TF32 on its
// way to out (cut to 10 bits: at most 2^-10 of |C[n] h[n]|, where out's own rounding to
// BF16 is 2^-9 of out); the states themselves stay FP32.
//
// 8192 tokens of 12,288 channels and 16 states: 547 us, where the bytes take 119 and
// the exponentials alone 172.  What bounds it is the schedulers' issue: a walking
// warp takes 29 cycles of it a token (of 4 x 32 elements: two packed and four scalar
// products for dt A and dt x B, 4 exponentials of 4 cycles' worth of a unit, two packed
// multiply-adds, the step's, B's and C's loads, the product), a staging warp 17, the
// exponentials' unit is busy for a third of the time and shared memory for half.
//
// Few (sequence, channel) chains are cut into spans of tokens: a first launch
// forms the state each span ends with (and the sum of its dt: the decay over a
// span is exp(A sum dt)), a second one each span's incoming state from those
// before it, and its outputs.  8192 tokens of 768 channels take 62 us so, 338 uncut.
//
// Many chains that do not fill the SMs evenly are cut too, and their spans run one
// after the other (SsmArgs::relay): a CTA takes up the state that the span before
// it left.  Nothing is computed twice and no bit changes; but a chain's spans run
// on whichever SM has room, where whole chains would stay on an SM that is
// fuller than others: 8192 tokens of 12,288 channels (384 chains on 152 SMs) take 547 us
// so, 602 uncut.
#pragma once

#include <cfloat>
#include <type_traits>

#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kRole = 128;               // threads that stage and finish
// Warps that share the states of 16 channels, and threads that walk.  Four for 64 states:
// 2 x 2000 tokens of 1536 channels 162 us, with two 167 (128 registers); for 32
// (4096 x 12,288) two 436 and four 475.
template <int kBlocks>
constexpr int kSplit = kBlocks == 4 ? 4 : 2;
template <int kBlocks>
constexpr int kWalkers = 64 * kSplit<kBlocks>;
constexpr int kTile = kSsmTile;          // tokens at a time
static_assert(kRole == 4 * kTile && kChannels == 32, "a thread stages 8 channels of one token");

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

// Shared memory of one of two buffers (read at 256 bytes a cycle where neighbouring
// lanes read the same 16 bytes, at 128 else): for each token and two channels
// (dt, dt, dt x, dt x), the rows of B and of C, and y, a sum over each warp's part of
// the states.  Strides that keep the lanes' accesses on different banks.
constexpr int kStepStride = 4 * (kTile + 1), kStepHalf = 8 * kStepStride + 8;
constexpr int kStepWords = 2 * kStepHalf;
constexpr int kYStride = kChannels + 4;
template <int kBlocks, bool kStates>
struct Buffer {
    static constexpr int kRow = 16 * kBlocks, kRowC = kRow + 8;
    static constexpr int kB = kStepWords, kC = kB + kTile * kRow, kY = kC + (kStates ? 0 : kTile * kRowC);
    static constexpr int kHalf = kTile * kYStride;   // of y
    static constexpr int kXZ = kY + (kStates ? 0 : kSplit<kBlocks> * kHalf);   // x and z of each staging thread, for its outputs
    static constexpr int kWords = kXZ + (kStates ? 0 : 8 * kRole);
};
// Channels ch (even) and ch + 1 at a token: (dt, dt, dt x, dt x).
__device__ __forceinline__ int step_at(int ch, int token) { return (ch >> 4) * kStepHalf + (ch >> 1 & 7) * kStepStride + 4 * token; }

// What a staging thread fetches of a tile: of one token eight channels' x, z and dt, and
// four values of every 16 of B and C.
template <int kBlocks>
struct Fetched {
    uint4 x, z, dt[2], b[kBlocks], c[kBlocks];
};
// 16 bytes at once, or 8 and 8.
__device__ __forceinline__ uint4 load16(const uint8_t* p, bool whole) {
    if (whole) return *reinterpret_cast<const uint4*>(p);
    const uint2 lo = *reinterpret_cast<const uint2*>(p), hi = *reinterpret_cast<const uint2*>(p + 8);
    return make_uint4(lo.x, lo.y, hi.x, hi.y);
}

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
// The lane's states of two rows of S (of two channels), from n0 on in steps of kStep.
template <int kStep, int kHold>
__device__ __forceinline__ void load_rows(const void* p, bool f32, int64_t row, int64_t row1, int n0, int S, State<kHold>& s) {
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        float2 a, b;
        if (f32) {
            a = load_two(static_cast<const float*>(p) + row * S, kStep * k + n0, S);
            b = load_two(static_cast<const float*>(p) + row1 * S, kStep * k + n0, S);
        } else {
            a = load_two(static_cast<const __nv_bfloat16*>(p) + row * S, kStep * k + n0, S);
            b = load_two(static_cast<const __nv_bfloat16*>(p) + row1 * S, kStep * k + n0, S);
        }
        s.h[k][0] = pair(a.x, b.x);
        s.h[k][1] = pair(a.y, b.y);
    }
}
template <int kStep, int kHold>
__device__ __forceinline__ void store_rows(void* p, bool f32, int64_t row, bool live, int64_t row1, bool live1, int n0, int S,
                                           const State<kHold>& s) {
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const float2 x = halves(s.h[k][0]), y = halves(s.h[k][1]);
        const float2 a = make_float2(x.x, y.x), b = make_float2(x.y, y.y);
        if (f32) {
            if (live) store_two(static_cast<float*>(p) + row * S, kStep * k + n0, S, a);
            if (live1) store_two(static_cast<float*>(p) + row1 * S, kStep * k + n0, S, b);
        } else {
            if (live) store_two(static_cast<__nv_bfloat16*>(p) + row * S, kStep * k + n0, S, a);
            if (live1) store_two(static_cast<__nv_bfloat16*>(p) + row1 * S, kStep * k + n0, S, b);
        }
    }
}
// A tile's decays are off on average: the exponential comes out 6e-9 too small for
// arguments above -2^-8, and 2.2e-8 below (measured on GB300 in steps of a half octave:
// 5e-9 .. 1e-8 and 1.4e-8 .. 3e-8), which adds up in states that last for hundreds of
// tokens, where roundings cancel.  Once a tile, in its middle, the states get it back,
// by the argument that one token's step gives (none if that is 0: what stands still
// keeps its bits).  1024 tokens with arguments around -0.0014: off
// by 1.5e-6 (as exact exponentials in FP32: 1e-6), without this by 5.6e-6; around -0.014 by
// 3.2e-6 and 2.5e-5.  (Where the state is gone by the tile's end it does not matter.)  2 %
// of the time.
__device__ __forceinline__ float lost(float x) {
    const float part = x > -0x1p-8f ? kTile * 6e-9f : kTile * 2.2e-8f;
    return x > -0x1p-23f ? 0.f : part;   // (the exponential is 1 there)
}
template <int kBlocks>
__device__ __forceinline__ void settle(State<kBlocks>& s, const State<kBlocks>& rate, uint64_t dt) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 x = halves(mul_pair(rate.h[k][i], dt));
            s.h[k][i] = fma_pair(s.h[k][i], pair(lost(x.x), lost(x.y)), s.h[k][i]);
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

// The walking warps' barrier.
template <int kBlocks>
__device__ __forceinline__ void walkers_meet() {
    asm volatile("bar.sync 1, %0;" ::"n"(kWalkers<kBlocks>) : "memory");
}
// A span's state is there: waits for `flag` with one thread, for kWaitBoundCycles at most.
__device__ __forceinline__ void wait_for_state(const int32_t* flag, int* status) {
    const long long start = clock64();
    int32_t there;
    for (;;) {
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(there) : "l"(flag) : "memory");
        if (there) return;
        if (clock64() - start > kWaitBoundCycles) break;
        __nanosleep(100);
    }
    atomicOr(status, kDevPipeTimeout);
}
__device__ __forceinline__ void state_is_there(int32_t* flag) {
    asm volatile("fence.acq_rel.gpu;\n st.release.gpu.global.s32 [%0], 1;" ::"l"(flag) : "memory");
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

// Some warps walk; four others stage the tile ahead and finish the one behind, so that there are warps enough to hide each other's latencies.
// kMode: any inputs (kAny), or, with the types of dt and of B and C known, a softplus,
// rows that can be read four values at a time, and groups of 32 channels or more (of
// which the last CTA then also has some of the one before it, and writes the same
// values).  That leaves out two fifths of the staging's instructions: 8192 x 12288,
// 16 states, uncut 602 us, as kAny 690.
// Registers are short: with three CTAs an SM (80 registers) values that wait in them spill,
// and each spill costs more than it seems (16 of y held for the tile's end: 612 us for 549).
// Two CTAs (128 registers) 615 us, four 686.
constexpr int kAny = 0, kPlain = 1, kDtF32 = 1, kKeysF32 = 2;   // kPlain plus the types that are FP32
template <int kBlocks, bool kStates, bool kPacked, int kMode>
__global__ void __launch_bounds__(kWalkers<kBlocks> + kRole, kBlocks > 1 ? 2 : 3) ssm_kernel(SsmArgs a) {
    using Buf = Buffer<kBlocks, kStates>;
    constexpr bool kFast = kMode != kAny;
    extern __shared__ __align__(16) float smem[];
    wait_for_kernel_before();
    if (kStates) let_next_kernel_come();
    if (kPacked && !offsets_hold(a.cu_seqlens, a.N, a.tokens, a.valid, a.status)) return;
    int64_t span, tile;
    if (!kStates && a.relay) {
        // In the order in which CTAs begin: the span before is under way or done.
        __shared__ int32_t ticket;
        if (threadIdx.x == 0) ticket = atomicAdd(a.relay, 1);
        __syncthreads();
        const int64_t chains = kPacked ? 1 : a.N, each = quotient(ticket, a.tiles * chains), rest = ticket - each * a.tiles * chains;
        const int64_t chain = quotient(rest, a.tiles);
        span = chain * a.spans_per_seq + each;
        tile = rest - chain * a.tiles;
    } else {
        span = quotient(blockIdx.x, a.tiles);
        tile = blockIdx.x - span * a.tiles;
    }
    const Part w = part_of<kStates, kPacked>(a, span);
    if (!w.run) return;
    const int64_t group = quotient(tile, a.tiles_per_group), per = quotient(a.dim, a.groups);
    int64_t ch0 = group * per + (tile - group * a.tiles_per_group) * kChannels;
    if (kFast && ch0 > (group + 1) * per - kChannels) ch0 = (group + 1) * per - kChannels;
    const int channels = kFast || (group + 1) * per - ch0 > kChannels ? kChannels : static_cast<int>((group + 1) * per - ch0);
    const int S = static_cast<int>(a.nstate);
    const int tid = threadIdx.x & (kRole - 1);
    const int total = static_cast<int>(w.end - w.begin);   // tokens; tiles i = 0 .. tiles - 1 of them
    const int tiles = total / kTile + (total % kTile > 0);

    if (threadIdx.x >= kWalkers<kBlocks>) {
        // ---- staging: of one token eight channels, and a quarter of its rows of B and C
        const int tok = tid >> 2, mine = 8 * (tid & 3);
        auto clip = [](int n) { return n < 0 ? 0 : n < 4 ? n : 4; };
        const int count = clip(channels - mine), count4 = clip(channels - mine - 4);
        const bool wide = kFast || (a.vec && count4 == 4), whole = a.vec8, wide_keys = kFast || a.vec_bc, gated = !kStates && a.z;
        const bool dt_f32 = kFast ? ((kMode - kPlain) & kDtF32) != 0 : a.dt_f32, bc_f32 = kFast ? ((kMode - kPlain) & kKeysF32) != 0 : a.bc_f32;
        // The channels' biases and skips, which would take 16 registers.
        float* const of_channel = smem + 2 * Buf::kWords;
        if (tid < kChannels) {
            of_channel[tid] = a.dt_bias && tid < channels ? a.dt_bias[ch0 + tid] : 0.f;
            if (!kStates) of_channel[kChannels + tid] = a.D && tid < channels ? a.D[ch0 + tid] : 0.f;
        }
        asm volatile("bar.sync 2, %0;" ::"n"(kRole) : "memory");
        auto eight_of = [&](const float* p, float (&v)[8]) {
            const float4 lo = *reinterpret_cast<const float4*>(p + mine), hi = *reinterpret_cast<const float4*>(p + mine + 4);
            v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w; v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
        };
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
                    f.x = load16(xp, whole);
                    if (gated) f.z = load16(zp, whole);
                    if (dt_f32) {
                        f.dt[0] = *reinterpret_cast<const uint4*>(dp);
                        f.dt[1] = *reinterpret_cast<const uint4*>(dp + 16);
                    } else {
                        f.dt[0] = load16(dp, whole);
                    }
                } else {
                    auto eight = [&](const uint8_t* p) {
                        const uint4 lo = gather8(reinterpret_cast<const __nv_bfloat16*>(p), count),
                                    hi = gather8(reinterpret_cast<const __nv_bfloat16*>(p + 8), count4);
                        return make_uint4(lo.x, lo.y, hi.x, hi.y);
                    };
                    f.x = eight(xp);
                    if (gated) f.z = eight(zp);
                    if (dt_f32) {
                        f.dt[0] = gather4(reinterpret_cast<const float*>(dp), count);
                        f.dt[1] = gather4(reinterpret_cast<const float*>(dp + 16), count4);
                    } else {
                        f.dt[0] = eight(dp);
                    }
                }
#pragma unroll
                for (int k = 0; k < kBlocks; ++k) {
                    const int have = S - 16 * k - 4 * (tid & 3);
                    const uint8_t *b = bp + 16 * k * es, *cc = cp + 16 * k * es;
                    if (have <= 0) {
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
            float dt[8], x[8], bias[8];
            eight_of(of_channel, bias);
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
                *reinterpret_cast<float4*>(buf + step_at(mine + 2 * j, tok)) =
                    make_float4(dt[2 * j], dt[2 * j + 1], dt[2 * j] * x[2 * j], dt[2 * j + 1] * x[2 * j + 1]);
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
                    const float4 v = *reinterpret_cast<const float4*>(p + 4 * j), u = *reinterpret_cast<const float4*>(p + Buf::kHalf + 4 * j);
                    y[4 * j] = v.x + u.x; y[4 * j + 1] = v.y + u.y; y[4 * j + 2] = v.z + u.z; y[4 * j + 3] = v.w + u.w;
#pragma unroll
                    for (int i = 2; i < kSplit<kBlocks>; ++i) {
                        const float4 w = *reinterpret_cast<const float4*>(p + i * Buf::kHalf + 4 * j);
                        y[4 * j] += w.x; y[4 * j + 1] += w.y; y[4 * j + 2] += w.z; y[4 * j + 3] += w.w;
                    }
                }
                if (a.D) {
                    float skip[8];
                    eight_of(of_channel + kChannels, skip);
                    unpack8(xz[0], x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = fmaf(skip[j], x[j], y[j]);
                }
                if (gated) {
                    unpack8(xz[kRole], z);
                    gate8(z, y);
                }
                if (wide && whole) {
                    store8(op, y);
                } else if (wide) {
                    *reinterpret_cast<uint2*>(op) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                    *reinterpret_cast<uint2*>(op + 4) = make_uint2(pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (mine + j < channels) op[j] = __float2bfloat16_rn(y[j]);
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

    // ---- the walk: 16 channels and eight of every kStep states for each warp
    constexpr int kStep = 8 * kSplit<kBlocks>, kHold = 2 * kBlocks / kSplit<kBlocks>;
    const int walker = kWalkers<kBlocks> == kRole ? tid : threadIdx.x;
    const int warp = walker >> 5, lane = walker & 31, c = lane & 3, part = warp % kSplit<kBlocks>;
    const int local = 16 * (warp / kSplit<kBlocks>) + 2 * (lane >> 2), n0 = 8 * part + 2 * c;
    const bool live = local < channels, live1 = local + 1 < channels;
    const int64_t ch = ch0 + (live ? local : 0), ch1 = ch0 + (live1 ? local + 1 : 0);
    State<kHold> rate, s;
    load_rows<kStep>(a.A, true, ch, ch1, n0, S, rate);
#pragma unroll
    for (int k = 0; k < kHold; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            // (Finite, for the zero steps behind the end; 2^-FLT_MAX is 0 for any other step.)
            const float2 v = halves(mul_pair(rate.h[k][i], pair(kLog2e, kLog2e)));
            rate.h[k][i] = pair(v.x < -FLT_MAX ? -FLT_MAX : v.x, v.y < -FLT_MAX ? -FLT_MAX : v.y);
        }
    auto initial = [&](int64_t seq) {
#pragma unroll
        for (int k = 0; k < kHold; ++k) s.h[k][0] = s.h[k][1] = 0ull;
        if (a.init_state) load_rows<kStep>(a.init_state, a.state_f32, seq * a.dim + ch, seq * a.dim + ch1, n0, S, s);
    };
    auto ending = [&](int64_t seq) {
        if (a.final_state)
            store_rows<kStep>(a.final_state, a.state_f32, seq * a.dim + ch, live, seq * a.dim + ch1, live1, n0, S, s);
    };
    if (w.fresh) {
        initial(w.seq);
    } else {
#pragma unroll
        for (int k = 0; k < kHold; ++k) s.h[k][0] = s.h[k][1] = 0ull;
        if (!kStates && a.relay) {
            if (walker == 0) wait_for_state(a.relay + 1 + (span - 1) * a.tiles + tile, a.status);
            walkers_meet<kBlocks>();
            load_rows<kStep>(a.span_states, true, (span - 1) * a.dim + ch, (span - 1) * a.dim + ch1, n0, 16 * kBlocks, s);
        } else if (!kStates) {
            // The states of the sequence's spans before this one, each decayed over
            // those behind it; the first one's has the initial state in it.
#pragma unroll 4
            for (int64_t i = w.first_span; i < span; ++i) {
                State<kHold> add;
                load_rows<kStep>(a.span_states, true, i * a.dim + ch, i * a.dim + ch1, n0, 16 * kBlocks, add);
                decay<kHold>(s, rate, pair(a.span_steps[i * a.dim + ch], a.span_steps[i * a.dim + ch1]), add.h);
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
    const int keys0 = Buf::kC + (lane >> 2) * Buf::kRowC + n0, y0 = Buf::kY + part * Buf::kHalf + 2 * c * kYStride + local;
    // Eight tokens from t on of the tile at `base`; with `ends`, sequences may end
    // among them.  (Tokens behind the span's end change nothing: only the last span
    // has them, and no sequence behind it.)  y: of tokens 2 c and 2 c + 1, and of
    // the second channel, as the product's accumulators have them.
    auto walk = [&](auto ends, const float* buf, int64_t base, int t, float (&y)[4]) {
        float ck[kHold][2];
        if (!kStates)
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const float2 v = *reinterpret_cast<const float2*>(buf + keys0 + t * Buf::kRowC + kStep * k);
                ck[k][0] = v.x;
                ck[k][1] = v.y;
            }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            uint64_t b[kHold][2];
            const ulonglong2 dd = *reinterpret_cast<const ulonglong2*>(buf + step0 + 4 * (t + j));   // both dt, both dt x
            const float2 du = halves(dd.y);
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                const float2 v = *reinterpret_cast<const float2*>(buf + rows0 + (t + j) * Buf::kRow + kStep * k);
                b[k][0] = pair(du.x * v.x, du.y * v.x);
                b[k][1] = pair(du.x * v.y, du.y * v.y);
            }
            decay<kHold>(s, rate, dd.x, b);
            if (kStates) {
                steps = add_pair(steps, dd.x);
            } else {
                float acc[4];
#pragma unroll
                for (int k = 0; k < kHold; ++k) {
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
        *reinterpret_cast<float2*>(at) = make_float2(y[0], y[2]);
        *reinterpret_cast<float2*>(at + kYStride) = make_float2(y[1], y[3]);
    };
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        float* buf = smem + (i & 1) * Buf::kWords;
        const int64_t base = static_cast<int64_t>(i) * kTile;
        if (base + kTile <= total && (!kPacked || kStates || seq_end >= base + kTile)) {
#pragma unroll
            for (int t = 0; t < kTile; t += 8) {
                if (t == kTile / 2) settle<kHold>(s, rate, *reinterpret_cast<const uint64_t*>(buf + step0 + 4 * t));
                float y[4];
                walk(std::false_type{}, buf, base, t, y);
                if (!kStates) store_y(buf, t, y);
            }
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
    if (kStates || a.relay)
        store_rows<kStep>(a.span_states, true, span * a.dim + ch, live, span * a.dim + ch1, live1, n0, 16 * kBlocks, s);
    if (!kStates && a.relay) {
        walkers_meet<kBlocks>();
        if (walker == 0) state_is_there(a.relay + 1 + span * a.tiles + tile);
    }
    if (kStates) {
        if (c == 0 && part == 0) {
            if (live) a.span_steps[span * a.dim + ch] = halves(steps).x;
            if (live1) a.span_steps[span * a.dim + ch1] = halves(steps).y;
        }
    }
}

template <int kBlocks, bool kStates, bool kPacked, int kMode>
cudaError_t run(const SsmArgs& a, cudaStream_t stream) {
    constexpr int bytes = 8 * Buffer<kBlocks, kStates>::kWords + 4 * 2 * kChannels;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(ssm_kernel<kBlocks, kStates, kPacked, kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    if (a.spans > 0x7fffffffLL / a.tiles) return cudaErrorInvalidValue;
    return launch_after(ssm_kernel<kBlocks, kStates, kPacked, kMode>, dim3(static_cast<unsigned>(a.spans * a.tiles)),
                        dim3(kWalkers<kBlocks> + kRole),
                        bytes, stream, a);
}

template <int kBlocks, int kMode>
cudaError_t prefill(const SsmArgs& a, cudaStream_t stream, int* launches) {
    cudaError_t e;
    if (a.span_states && !a.relay) {
        e = a.cu_seqlens ? run<kBlocks, true, true, kMode>(a, stream) : run<kBlocks, true, false, kMode>(a, stream);
        if (e != cudaSuccess) return e;
        ++*launches;
    }
    e = a.cu_seqlens ? run<kBlocks, false, true, kMode>(a, stream) : run<kBlocks, false, false, kMode>(a, stream);
    if (e == cudaSuccess) ++*launches;
    return e;
}
template <int kBlocks>
cudaError_t prefill(const SsmArgs& a, cudaStream_t stream, int* launches) {
    if (!a.vec || !a.vec_bc || !a.softplus || a.dim / a.groups < kChannels) return prefill<kBlocks, kAny>(a, stream, launches);
    if (a.bc_f32)
        return a.dt_f32 ? prefill<kBlocks, kPlain + kDtF32 + kKeysF32>(a, stream, launches)
                        : prefill<kBlocks, kPlain + kKeysF32>(a, stream, launches);
    return a.dt_f32 ? prefill<kBlocks, kPlain + kDtF32>(a, stream, launches) : prefill<kBlocks, kPlain>(a, stream, launches);
}

}  // namespace
}  // namespace kda
