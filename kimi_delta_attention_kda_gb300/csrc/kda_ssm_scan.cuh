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
// shared memory; the warps of the others walk 8 channels each through the tokens, four lanes a
// channel with a quarter of the states in their registers (64 states: two warps, an eighth).  A lane sums
// its products with C, and every four tokens the four lanes of a channel hand each
// other their sums, so that each ends with one token's.  All of it is FP32.  (Summed on the
// tensor cores, TF32, the call below took 546 us, but cut the states to 10 bits on the
// way to out: outputs too small by 3.5e-4 on average.)
//
// 8192 tokens of 12,288 channels and 16 states: 586 us, where the bytes take 119 and
// the exponentials alone 172.  Of the time shared memory's pipe is busy 80 % (a walking lane reads
// 40 bytes a token), the exponentials' unit 35 %, and 61 % of the issue slots are used; warps
// wait most at the barrier between staging and walking, then for shared memory.

// Few (sequence, channel) chains are cut into spans of tokens: a first launch
// forms the state each span ends with (and the sum of its dt: the decay over a
// span is exp(A sum dt)), a second one each span's incoming state from those
// before it, and its outputs.  8192 tokens of 768 channels take 62 us so, 332 uncut.
//
// Many chains that do not fill the SMs evenly are cut too, and their spans run one
// after the other (SsmArgs::relay): a CTA takes up the state that the span before
// it left.  Nothing is computed twice and no bit changes; but a chain's spans run
// on whichever SM has room, where whole chains would stay on an SM that is
// fuller than others: 8192 tokens of 12,288 channels (384 chains on 152 SMs) take 586 us
// so, 633 uncut.
#pragma once

#include <type_traits>

#include "kda_ssm.cuh"

namespace kda {
namespace {

constexpr int kRole = 128;               // threads that stage and finish
// Warps that share the states of 8 channels, and threads that walk.
template <int kBlocks>
constexpr int kSplit = kBlocks == 4 ? 2 : 1;
template <int kBlocks>
constexpr int kWalkers = 128 * kSplit<kBlocks>;
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

// Shared memory of one of two buffers: for each token (dt, dt x) of every channel, the
// rows of B and of C, and y, a sum over each warp's part of the states.  Strides and
// places that keep the lanes' accesses on different banks.
constexpr int kStepStride = 2 * kChannels + 8, kStepWords = kTile * kStepStride;
constexpr int kNoStep = 2 * kChannels;   // two words of 0 behind every token's
constexpr int kYStride = kChannels + 4;
template <int kBlocks, bool kStates>
struct Buffer {
    static constexpr int kRow = 16 * kBlocks;
    static constexpr int kB = kStepWords, kC = kB + kTile * kRow, kY = kC + (kStates ? 0 : kTile * kRow);
    static constexpr int kHalf = kTile * kYStride;   // of y
    static constexpr int kXZ = kY + (kStates ? 0 : kSplit<kBlocks> * kHalf);   // x and z of each staging thread, for its outputs
    static constexpr int kWords = kXZ + (kStates ? 0 : 8 * kRole);
};
// Channels ch (even) and ch + 1 at a token: (dt, dt x, dt, dt x).
__device__ __forceinline__ int step_at(int ch, int token) {
    return token * kStepStride + (ch >> 3) * 16 + 4 * ((ch >> 1 & 3) ^ (ch >> 4));
}

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

// A lane's states of a row of S: 4 kHold from n0 on.
template <int kHold, typename T>
__device__ __forceinline__ void load_row(const T* row, int n0, int S, State<kHold>& s) {
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int n = n0 + 4 * k;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (S % 4 == 0) {
            if (n < S) load_vec<4>(row + n, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < S) v[i] = static_cast<float>(row[n + i]);
        }
        s.h[k][0] = pair(v[0], v[1]);
        s.h[k][1] = pair(v[2], v[3]);
    }
}
template <int kHold, typename T>
__device__ __forceinline__ void store_row(T* row, int n0, int S, const State<kHold>& s) {
#pragma unroll
    for (int k = 0; k < kHold; ++k) {
        const int n = n0 + 4 * k;
        const float2 a = halves(s.h[k][0]), b = halves(s.h[k][1]);
        const float v[4] = {a.x, a.y, b.x, b.y};
        if (S % 4 == 0) {
            if (n < S) store_vec<4>(row + n, v);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < S) from_f32(row + n + i, v[i]);
        }
    }
}
// Row `row` of states of either type.
template <int kHold>
__device__ __forceinline__ void load_states(const void* p, bool f32, int64_t row, int n0, int S, State<kHold>& s) {
    if (f32)
        load_row(static_cast<const float*>(p) + row * S, n0, S, s);
    else
        load_row(static_cast<const __nv_bfloat16*>(p) + row * S, n0, S, s);
}
template <int kHold>
__device__ __forceinline__ void store_states(void* p, bool f32, int64_t row, int n0, int S, const State<kHold>& s) {
    if (f32)
        store_row(static_cast<float*>(p) + row * S, n0, S, s);
    else
        store_row(static_cast<__nv_bfloat16*>(p) + row * S, n0, S, s);
}
// A tile's decays are off on average, see lost(), which adds up in states that last for hundreds of
// tokens, where roundings cancel.  Once a tile, in its middle, the states get it back, by the
// argument that the least step of the tile's first half gives, below which no token of
// that half is: none if that is 0 (what stands still keeps its bits), and where the second
// half stands still at most twice what was lost, so that it never adds more error than it
// takes away.  1024 tokens with arguments around -0.0014: off
// by 1.5e-6 (as exact exponentials in FP32: 1e-6), without this by 5.6e-6; around -0.014 by
// 3.2e-6 and 2.5e-5.  (Where the state is gone by the tile's end it does not matter.)  3 %
// of the time, most of it for the least step.
template <int kBlocks>
__device__ __forceinline__ void settle(State<kBlocks>& s, const State<kBlocks>& rate, uint64_t dt) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 x = halves(mul_pair(rate.h[k][i], dt));
            s.h[k][i] = fma_pair(s.h[k][i], pair(kTile * lost(x.x), kTile * lost(x.y)), s.h[k][i]);
        }
}

// h <- exp2(A s) h + b over a whole span, s the sum of its steps.  In two factors, each
// finite: a state of zero stays zero whatever it would grow by, and one that grows beyond 2^128
// from far below 1, or comes back from far above it, keeps its value as in the walk.
// (A growth of more than 2^254, cut to that, leaves no normal number finite, and a decay to
// 2^-252 nothing of one; an infinite state stays one.)
template <int kHold>
__device__ __forceinline__ void decay_span(State<kHold>& s, const State<kHold>& rate, float step, const State<kHold>& add) {
#pragma unroll
    for (int k = 0; k < kHold; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 x = halves(mul_pair(rate.h[k][i], pair(0.5f * step, 0.5f * step)));
            const uint64_t e = pair(exp2_fast(fminf(fmaxf(x.x, -126.f), 127.f)), exp2_fast(fminf(fmaxf(x.y, -126.f), 127.f)));
            s.h[k][i] = fma_pair(e, mul_pair(e, s.h[k][i]), add.h[k][i]);
        }
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
// 16 states, uncut 634 us, as kAny 705.
// Three CTAs an SM (80 registers): 587 us; two (128) 645, four (64) 656.
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
        if (tid < 2 * kTile)
            *reinterpret_cast<float2*>(smem + (tid / kTile) * Buf::kWords + tid % kTile * kStepStride + kNoStep) = make_float2(0.f, 0.f);
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
                    make_float4(dt[2 * j], dt[2 * j] * x[2 * j], dt[2 * j + 1], dt[2 * j + 1] * x[2 * j + 1]);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k) {
                const int n0 = 16 * k + 4 * (tid & 3);
                *reinterpret_cast<float4*>(buf + Buf::kB + tok * Buf::kRow + n0) = four(f.b[k]);
                if (!kStates) *reinterpret_cast<float4*>(buf + Buf::kC + tok * Buf::kRow + n0) = four(f.c[k]);
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
                    const float4 v = *reinterpret_cast<const float4*>(p + 4 * j);
                    y[4 * j] = v.x; y[4 * j + 1] = v.y; y[4 * j + 2] = v.z; y[4 * j + 3] = v.w;
#pragma unroll
                    for (int i = 1; i < kSplit<kBlocks>; ++i) {
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

    // ---- the walk: 8 channels a warp, four lanes each, with 4 kHold states
    constexpr int kHold = kBlocks / kSplit<kBlocks>;
    const int walker = kWalkers<kBlocks> == kRole ? tid : threadIdx.x;
    const int warp = walker >> 5, lane = walker & 31, c = lane >> 3, part = warp >> 2;
    const int local = 8 * (warp & 3) + (lane & 7), n0 = 4 * kHold * (4 * part + c);
    const bool live = local < channels;
    const int64_t ch = ch0 + (live ? local : 0);
    State<kHold> rate, s;
    load_states(a.A, true, ch, n0, S, rate);
    to_log2(rate);
    if (!kFast)
#pragma unroll
        for (int k = 0; k < kHold; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) no_rates(rate.h[k][i], n0 + 4 * k + 2 * i, S);
    auto none = [&]() {
#pragma unroll
        for (int k = 0; k < kHold; ++k) s.h[k][0] = s.h[k][1] = 0ull;
    };
    auto initial = [&](int64_t seq) {
        none();
        if (a.init_state) load_states(a.init_state, a.state_f32, seq * a.dim + ch, n0, S, s);
    };
    auto ending = [&](int64_t seq) {
        if (a.final_state && live) store_states(a.final_state, a.state_f32, seq * a.dim + ch, n0, S, s);
    };
    if (w.fresh) {
        initial(w.seq);
    } else {
        none();
        if (!kStates && a.relay) {
            if (walker == 0) wait_for_state(a.relay + 1 + (span - 1) * a.tiles + tile, a.status);
            walkers_meet<kBlocks>();
            load_states(a.span_states, true, (span - 1) * a.dim + ch, n0, 16 * kBlocks, s);
        } else if (!kStates) {
            // The states of the sequence's spans before this one, each decayed over
            // those behind it; the first one's has the initial state in it.
#pragma unroll 4
            for (int64_t i = w.first_span; i < span; ++i) {
                State<kHold> add;
                load_states(a.span_states, true, i * a.dim + ch, n0, 16 * kBlocks, add);
                decay_span(s, rate, a.span_steps[i * a.dim + ch], add);
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
    // States behind S, which the lanes of a short row have, stay 0: an infinite dt x would
    // make NaN of them, and so of y.  Whole lanes of them read steps of 0 (kNoStep).
    const int own0 = step_at(local, 0) + 2 * (local & 1), step0 = n0 < S ? own0 : kNoStep, rows0 = Buf::kB + n0;
    const int keys0 = Buf::kC + n0, y0 = Buf::kY + part * Buf::kHalf + c * kYStride + local;
    auto four_of = [&](const float* p, uint64_t (&v)[2]) {
        const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(p);
        v[0] = r.x;
        v[1] = r.y;
    };
    // Four tokens from t on of the tile at `base`, and their y; with `ends`, sequences
    // may end among them.  (Tokens behind the span's end change nothing: only the last
    // span has them, and no sequence behind it.)
    auto walk = [&](auto ends, float* buf, int64_t base, int t) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint64_t b[kHold][2];
            const float2 dd = *reinterpret_cast<const float2*>(buf + step0 + (t + j) * kStepStride);   // dt, dt x
#pragma unroll
            for (int k = 0; k < kHold; ++k) {
                four_of(buf + rows0 + (t + j) * Buf::kRow + 4 * k, b[k]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int n = n0 + 4 * k + 2 * i;
                    b[k][i] = mul_pair(b[k][i], pair(kFast || n < S ? dd.y : 0.f, kFast || n + 1 < S ? dd.y : 0.f));
                }
            }
            decay<kHold>(s, rate, pair(dd.x, dd.x), b);
            if (kStates) {
                steps += dd.x;
            } else {
                uint64_t sum = 0ull;
#pragma unroll
                for (int k = 0; k < kHold; ++k) {
                    uint64_t key[2];
                    four_of(buf + keys0 + (t + j) * Buf::kRow + 4 * k, key);
                    sum = k == 0 ? mul_pair(key[0], s.h[k][0]) : fma_pair(key[0], s.h[k][0], sum);
                    sum = fma_pair(key[1], s.h[k][1], sum);
                }
                const float2 v = halves(sum);
                y[j] = v.x + v.y;
                if (decltype(ends)::value) close(base + t + j + 1);
            }
        }
        if (!kStates) {
            // Lane c of a channel's four gets the sum of token t + c over them.
            const bool up = c & 2, right = c & 1;
            float keep0 = up ? y[2] : y[0], keep1 = up ? y[3] : y[1];
            keep0 += __shfl_xor_sync(0xffffffffu, up ? y[0] : y[2], 16);
            keep1 += __shfl_xor_sync(0xffffffffu, up ? y[1] : y[3], 16);
            const float keep = right ? keep1 : keep0;
            buf[y0 + t * kYStride] = keep + __shfl_xor_sync(0xffffffffu, right ? keep0 : keep1, 8);
        }
    };
    // The least step of a tile's first half, 0 where there are negative ones: each of a
    // channel's lanes looks at every fourth.
    auto least_step = [&](const float* buf) {
        float least = buf[own0 + c * kStepStride];
#pragma unroll
        for (int t = 4; t < kTile / 2; t += 4) least = fminf(least, buf[own0 + (t + c) * kStepStride]);
        least = fminf(least, __shfl_xor_sync(0xffffffffu, least, 8));
        return fmaxf(fminf(least, __shfl_xor_sync(0xffffffffu, least, 16)), 0.f);
    };
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
        float* buf = smem + (i & 1) * Buf::kWords;
        const int64_t base = static_cast<int64_t>(i) * kTile;
        float least = 0.f;
        if (base + kTile <= total && (!kPacked || kStates || seq_end >= base + kTile)) {
#pragma unroll
            for (int t = 0; t < kTile; t += 4) {
                if (t == kTile / 2 - 4) least = least_step(buf);
                if (t == kTile / 2) settle<kHold>(s, rate, pair(least, least));
                walk(std::false_type{}, buf, base, t);
            }
            if (kPacked && !kStates) close(base + kTile);
        } else {
#pragma unroll 1
            for (int t = 0; t < kTile && base + t < total; t += 4)
                walk(std::integral_constant<bool, kPacked && !kStates>{}, buf, base, t);
        }
        __syncthreads();
    }
    if (!kPacked && !kStates && total == seq_end && total > 0) close(total);
    if ((kStates || a.relay) && live) store_states(a.span_states, true, span * a.dim + ch, n0, 16 * kBlocks, s);
    if (!kStates && a.relay) {
        walkers_meet<kBlocks>();
        if (walker == 0) state_is_there(a.relay + 1 + span * a.tiles + tile);
    }
    if (kStates && live && c == 0 && part == 0) a.span_steps[span * a.dim + ch] = steps;
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
    // (Lanes with states in the row and behind it are kAny's, which keeps those behind at 0: 4096 tokens
    // of 12,288 channels with 20 states 531 us, as the others 467.)
    const bool mixed = a.nstate % (4 * kBlocks / kSplit<kBlocks>) != 0;
    if (!a.vec || !a.vec_bc || !a.softplus || mixed || a.dim / a.groups < kChannels) return prefill<kBlocks, kAny>(a, stream, launches);
    if (a.bc_f32)
        return a.dt_f32 ? prefill<kBlocks, kPlain + kDtF32 + kKeysF32>(a, stream, launches)
                        : prefill<kBlocks, kPlain + kKeysF32>(a, stream, launches);
    return a.dt_f32 ? prefill<kBlocks, kPlain + kDtF32>(a, stream, launches) : prefill<kBlocks, kPlain>(a, stream, launches);
}

}  // namespace
}  // namespace kda
