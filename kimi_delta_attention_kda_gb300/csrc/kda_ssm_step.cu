// kda_ssm_step.cu -- single tokens of the selective state space scan (sm_103a).
#include <type_traits>

#include "kda_ssm.cuh"

namespace kda {
namespace {

// Four values of a single token's state, which nobody reads before the next token:
// a streaming store (128 sequences of 12,288 channels 35 us, with a plain one 40).
template <typename T>
__device__ __forceinline__ void store_four(T* row, const float (&v)[4]) {
    if constexpr (sizeof(T) == 4)
        __stcs(reinterpret_cast<float4*>(row), make_float4(v[0], v[1], v[2], v[3]));
    else
        __stcs(reinterpret_cast<uint2*>(row), make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])));
}
// How a lane reads its values of a row of S, four at a time and 0 behind S: kOnes, one
// by one; kFours, as they are, where S is a multiple of four and the alignment allows;
// kWhole, the same with S = 16 kBlocks known.
enum Rows { kOnes, kFours, kWhole };
template <int kBlocks, typename T>
struct Row {
    using Four = std::conditional_t<sizeof(T) == 4, uint4, uint2>;
    Four r[kBlocks];

    template <Rows kRows>
    __device__ __forceinline__ void load(const T* row, int c, int S) {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int n0 = 16 * k + 4 * c;
            if constexpr (kRows != kOnes) {
                r[k] = Four{};
                if (kRows == kWhole || n0 < S) r[k] = *reinterpret_cast<const Four*>(row + n0);
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
    template <Rows kRows>
    __device__ static __forceinline__ void store(T* row, int c, int S, const State<kBlocks>& s) {
#pragma unroll
        for (int k = 0; k < kBlocks; ++k) {
            const int n0 = 16 * k + 4 * c;
            const float2 a = halves(s.h[k][0]), b = halves(s.h[k][1]);
            const float v[4] = {a.x, a.y, b.x, b.y};
            if constexpr (kRows != kOnes) {
                if (kRows == kWhole || n0 < S) store_four(row + n0, v);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n0 + i < S) from_f32(row + n0 + i, v[i]);
            }
        }
    }
};
// h <- exp2(A s) h + b; with kRepaid, b has what the exponential takes from h on average,
// 6e-6 to 2e-5 of states that last for a thousand tokens (128 sequences of 12,288 channels 34.7 us,
// without 33.9; by the slowest of every four states, with fewer comparisons, 37.4).  BF16 states go
// without: they are rounded by up to 2^-8 a token.
template <int kBlocks, bool kRepaid>
__device__ __forceinline__ void advance(State<kBlocks>& s, const State<kBlocks>& rate, float step, const uint64_t (&b)[kBlocks][2]) {
#pragma unroll
    for (int k = 0; k < kBlocks; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 x = halves(mul_pair(rate.h[k][i], pair(step, step)));
            const uint64_t e = pair(exp2_fast(x.x), exp2_fast(x.y));
            const uint64_t add = kRepaid ? fma_pair(mul_pair(e, pair(lost(x.x), lost(x.y))), s.h[k][i], b[k][i]) : b[k][i];
            s.h[k][i] = fma_pair(e, s.h[k][i], add);
        }
}
// Four lanes have a channel, a thread four sequences.  Lane i of a channel's four loads
// x, dt and z of sequence i, forms its step and its gate and hands the step to the
// other three; the sums over the states come back to it, so that nothing is computed
// four times, and the rates are read once for four sequences.  With up to 16 states
// all loads are issued before the first value is used.
// Bound by HBM: each state is read and written once, 2 x 4 S bytes (FP32) a channel.
// 128 sequences of 12,288 channels and 16 states take 35 us, of which the bytes 31 at
// the rate of a copy; with BF16 states 26 and 17, where the issue binds (441
// instructions a warp, 73 % of the slots; with FP32 states 505 and 65 %).
constexpr int kStepThreads = 4 * kChannels;
template <int kBlocks, Rows kRows, bool kStateF32, bool kKeysF32>
__global__ void __launch_bounds__(kStepThreads, kBlocks == 1 ? 8 : kBlocks == 2 ? 4 : 3) ssm_decode_kernel(SsmArgs a, int blocks) {
    wait_for_kernel_before();
    // Sequences whose states are under way together, and whose rows of B and C are,
    // as far as the registers go.
    constexpr int kTogether = kBlocks == 1 && kRows != kOnes ? 4 : 1, kKeysTogether = kKeysF32 ? 1 : kTogether;
    using StateT = std::conditional_t<kStateF32, float, __nv_bfloat16>;
    using KeyT = std::conditional_t<kKeysF32, float, __nv_bfloat16>;
    const int c = threadIdx.x & 3, S = kRows == kWhole ? 16 * kBlocks : static_cast<int>(a.nstate);
    const int part = static_cast<int>(blockIdx.x / static_cast<uint32_t>(blocks)), n0 = 4 * part;
    const int ch_raw = (static_cast<int>(blockIdx.x) - part * blocks) * kChannels + static_cast<int>(threadIdx.x >> 2);
    const int dim = static_cast<int>(a.dim), N = static_cast<int>(a.N);
    const bool live = ch_raw < dim;
    const int ch = live ? ch_raw : dim - 1;
    const int group = a.groups > 1 ? static_cast<uint32_t>(ch) / static_cast<uint32_t>(dim / static_cast<int>(a.groups)) : 0;

    // The sequences' slots (-1: none) are the same for the whole CTA: a lane reads one.
    const int own = n0 + c;
    int own_slot = own < N ? (a.slots ? a.slots[own] : own) : -1;
    if (own_slot >= a.pool) {
        if (ch_raw == 0) atomicOr(a.status, kDevBadSlots);
        own_slot = -1;
    }
    int slot[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) slot[i] = __shfl_sync(0xffffffffu, own_slot, i, 4);
    // (A state's row is below 2^32 bytes, see kSsmMaxDim.)
    const uint32_t state_bytes = static_cast<uint32_t>(dim) * S * sizeof(StateT);
    uint8_t* base = static_cast<uint8_t*>(a.state) + static_cast<uint64_t>(static_cast<uint32_t>(ch)) * (S * sizeof(StateT));
    auto row_at = [&](int i) { return reinterpret_cast<StateT*>(base + static_cast<uint64_t>(static_cast<uint32_t>(slot[i])) * state_bytes); };
    Row<kBlocks, StateT> states[kTogether];
    Row<kBlocks, KeyT> bs[kKeysTogether], cs[kKeysTogether];
    const KeyT *b_row = static_cast<const KeyT*>(a.B) + n0 * a.ldb + group * S, *c_row = static_cast<const KeyT*>(a.C) + n0 * a.ldc + group * S;
    auto load = [&](int i, int to) {
        if (slot[i] >= 0) states[to].template load<kRows>(row_at(i), c, S);
    };
    auto load_keys = [&](int i, int to) {
        if (slot[i] >= 0) {
            bs[to].template load<kRows>(b_row, c, S);
            cs[to].template load<kRows>(c_row, c, S);
        }
        b_row += a.ldb;
        c_row += a.ldc;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kTogether == 4) load(i, i);
        if (kKeysTogether == 4) load_keys(i, i);
    }
    __nv_bfloat16 x_raw = __float2bfloat16_rn(0.f), z_raw = x_raw;
    uint32_t dt_raw = 0;
    if (own < N) {   // (read for a padding row too, and not used)
        // (n0 times a stride is the same for the whole CTA.)
        auto at = [&](int64_t ld) { return n0 * ld + (c * ld + ch); };
        x_raw = static_cast<const __nv_bfloat16*>(a.x)[at(a.ldx)];
        if (a.z) z_raw = static_cast<const __nv_bfloat16*>(a.z)[at(a.ldz)];
        dt_raw = a.dt_f32 ? static_cast<const uint32_t*>(a.dt)[at(a.lddt)] : static_cast<const uint16_t*>(a.dt)[at(a.lddt)];
    }
    Row<kBlocks, float> rates;
    rates.template load<kRows>(a.A + static_cast<uint64_t>(static_cast<uint32_t>(ch)) * S, c, S);
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f, skip = a.D ? a.D[ch] : 0.f;

    float dt = __uint_as_float(a.dt_f32 ? dt_raw : dt_raw << 16) + bias;
    if (a.softplus) dt = softplus(dt);
    const float x = __bfloat162float(x_raw), z = __bfloat162float(z_raw), du = dt * x;
    State<kBlocks> rate;
    rates.unpack(rate);
    to_log2(rate);
    if (kRows != kWhole)
#pragma unroll
        for (int k = 0; k < kBlocks; ++k)
#pragma unroll
            for (int j = 0; j < 2; ++j) no_rates(rate.h[k][j], 16 * k + 4 * c + 2 * j, S);
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = kTogether == 4 ? i : 0, key_at = kKeysTogether == 4 ? i : 0;
        if (kTogether == 1) load(i, 0);
        if (kKeysTogether == 1) load_keys(i, 0);
        const float step = __shfl_sync(0xffffffffu, dt, i, 4), add = __shfl_sync(0xffffffffu, du, i, 4);
        y[i] = 0.f;
        if (slot[i] >= 0) {
            State<kBlocks> s, b, key;
            states[at].unpack(s);
            bs[key_at].unpack(b);
            cs[key_at].unpack(key);
            uint64_t sum = 0ull;
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // States behind S, which the lanes of a short row have, stay 0: an infinite
                    // dt x would make NaN of them, and so of y.
                    const int n = 16 * k + 4 * c + (kRows == kOnes ? 2 * j : 0);
                    const float lo = kRows == kWhole || n < S ? add : 0.f, hi = kRows != kOnes ? lo : n + 1 < S ? add : 0.f;
                    b.h[k][j] = mul_pair(b.h[k][j], pair(lo, hi));
                }
            advance<kBlocks, kStateF32>(s, rate, step, b.h);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
#pragma unroll
                for (int j = 0; j < 2; ++j) sum = fma_pair(key.h[k][j], s.h[k][j], sum);
            y[i] = halves(sum).x + halves(sum).y;
            if (live) Row<kBlocks, StateT>::template store<kRows>(row_at(i), c, S, s);
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
    if (live && own < N)
        static_cast<__nv_bfloat16*>(a.out)[n0 * a.dim + (c * dim + ch)] = __float2bfloat16_rn(own_slot >= 0 ? sum : 0.f);
}

template <int kBlocks, Rows kRows, bool kStateF32, bool kKeysF32>
cudaError_t decode(const SsmArgs& a, cudaStream_t stream) {
    const int64_t blocks = (a.dim + kChannels - 1) / kChannels, parts = (a.N + 3) / 4;
    if (parts > 0x7fffffffLL / blocks) return cudaErrorInvalidValue;
    return launch_after(ssm_decode_kernel<kBlocks, kRows, kStateF32, kKeysF32>, dim3(static_cast<unsigned>(blocks * parts)),
                        dim3(kStepThreads), 0, stream, a, static_cast<int>(blocks));
}
template <int kBlocks, Rows kRows>
cudaError_t pick_decode(const SsmArgs& a, cudaStream_t stream) {
    if (a.state_f32)
        return a.bc_f32 ? decode<kBlocks, kRows, true, true>(a, stream) : decode<kBlocks, kRows, true, false>(a, stream);
    return a.bc_f32 ? decode<kBlocks, kRows, false, true>(a, stream) : decode<kBlocks, kRows, false, false>(a, stream);
}
template <int kBlocks>
cudaError_t pick_decode(const SsmArgs& a, cudaStream_t stream) {
    // (16 states, 128 x 12288: 35 us as kWhole, 38 as kFours; 64 states, 32 x 12288, 35 and 40; but 32 states,
    // 64 x 12288, 40 and 38.7.)
    if (kBlocks != 2 && a.vec_bc && a.nstate == 16 * kBlocks) return pick_decode<kBlocks, kBlocks != 2 ? kWhole : kFours>(a, stream);
    return a.vec_bc ? pick_decode<kBlocks, kFours>(a, stream) : pick_decode<kBlocks, kOnes>(a, stream);
}

}  // namespace

cudaError_t launch_ssm_decode(SsmArgs a, cudaStream_t stream) {
    if (a.N <= 0 || a.dim <= 0) return cudaSuccess;
    set_ssm_vectors(&a);
    if (a.nstate <= 16) return pick_decode<1>(a, stream);
    return a.nstate <= 32 ? pick_decode<2>(a, stream) : pick_decode<4>(a, stream);
}

}  // namespace kda
