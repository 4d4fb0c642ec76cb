// kda_conv.cu -- the short causal convolution in front of a mixer (sm_103a).
//
// kda_conv_prefill, for each channel d of a sequence:
//     y_t = act(bias_d + sum_{j < W} w[d][j] x_{t - W + 1 + j}),
// with the initial state's W - 1 rows in front of the first token;
// kda_conv_decode: one token of it on a pool of such states.
// Bound by HBM: 4 bytes a token and channel against 2 W + 10 operations.  A
// thread has a few channels and a run of tokens, and keeps the last W - 1 inputs
// in registers as it walks, so that each input is read once but for the W - 1
// before every run, which another thread reads too (and L2 has then).
// All arithmetic is FP32; outputs are rounded once, states are inputs as they are.
#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_seq.cuh"
#include "kda_vec.cuh"

namespace kda {
namespace {

constexpr int kConvThreads = 256;
constexpr int kGroup = 4;   // tokens whose loads are under way together

__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, uint4& r) { r = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, uint32_t& r) { r = *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* p, uint16_t& r) { r = *reinterpret_cast<const uint16_t*>(p); }

// kVec consecutive BF16 values as loaded: 8, or 2 or 1 where rows start at any element.
template <int kVec>
struct Raw;
template <>
struct Raw<8> {
    using type = uint4;
    __device__ static void unpack(const uint4& r, float (&x)[8]) { unpack8(r, x); }
    __device__ static uint4 zero() { return make_uint4(0, 0, 0, 0); }
};
template <>
struct Raw<2> {
    using type = uint32_t;
    __device__ static void unpack(uint32_t r, float (&x)[2]) {
        x[0] = bf16_lo(r);
        x[1] = bf16_hi(r);
    }
    __device__ static uint32_t zero() { return 0; }
};
template <>
struct Raw<1> {
    using type = uint16_t;
    __device__ static void unpack(uint16_t r, float (&x)[1]) { x[0] = bf16_lo(r); }
    __device__ static uint16_t zero() { return 0; }
};

// A thread's filter: kVec channels with kW taps each, and their bias.
template <int kW, int kVec>
struct Filter {
    float w[kW][kVec], b[kVec];

    template <typename T>
    __device__ __forceinline__ void load_as(const void* weight, const void* bias, int64_t ch) {
        float flat[kW * kVec];
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            float part[kVec];
            load_vec<kVec>(static_cast<const T*>(weight) + ch * kW + i * kVec, part);
#pragma unroll
            for (int j = 0; j < kVec; ++j) flat[i * kVec + j] = part[j];
        }
#pragma unroll
        for (int i = 0; i < kW; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) w[i][j] = flat[j * kW + i];
#pragma unroll
        for (int j = 0; j < kVec; ++j) b[j] = 0.f;
        if (bias) load_vec<kVec>(static_cast<const T*>(bias) + ch, b);
    }
    __device__ __forceinline__ void load(const ConvArgs& a, int64_t ch) {
        if (a.weight_f32)
            load_as<float>(a.weight, a.bias, ch);
        else
            load_as<__nv_bfloat16>(a.weight, a.bias, ch);
    }
    // Row kW - 1 of x is the token's own.
    __device__ __forceinline__ void apply(const float (*x)[kVec], bool silu, __nv_bfloat16* out) const {
        float y[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            y[j] = b[j];
#pragma unroll
            for (int i = 0; i < kW; ++i) y[j] = fmaf(w[i][j], x[i][j], y[j]);
            if (silu) y[j] *= sigmoid(y[j]);
        }
        store_vec<kVec>(out, y);
    }
};

template <int kW, int kVec, bool kPacked>
__global__ void __launch_bounds__(kConvThreads) conv_prefill_kernel(ConvArgs a) {
    wait_for_kernel_before();
    if (kPacked && !offsets_hold(a.cu_seqlens, a.N, a.tokens, a.valid, a.status)) return;
    const int64_t vecs = a.D / kVec, at = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
    const int64_t run = at / vecs, ch = (at - run * vecs) * kVec;
    if (run >= a.runs) return;
    using R = Raw<kVec>;
    constexpr int kKeep = kW - 1;
    const auto x = static_cast<const __nv_bfloat16*>(a.x) + ch;
    const auto init = static_cast<const __nv_bfloat16*>(a.init_state) + ch;
    const auto out = static_cast<__nv_bfloat16*>(a.out) + ch;
    const auto final_state = static_cast<__nv_bfloat16*>(a.final_state) + ch;

    int64_t seq, begin, t, end;   // the sequence, its first token, this run's tokens
    int64_t seq_end;
    if (kPacked) {
        t = run * a.run_tokens;
        end = t + a.run_tokens < a.tokens ? t + a.run_tokens : a.tokens;
        // The first run also has the empty sequences before the first token.
        seq = run == 0 ? 0 : ended_by(a.cu_seqlens, a.N, t);
        begin = a.cu_seqlens[seq];
        seq_end = a.cu_seqlens[seq + 1];
    } else {
        seq = run / a.runs_per_seq;
        begin = seq * a.tokens_per_seq;
        t = begin + (run - seq * a.runs_per_seq) * a.run_tokens;
        seq_end = begin + a.tokens_per_seq;
        end = t + a.run_tokens < seq_end ? t + a.run_tokens : seq_end;
    }
    Filter<kW, kVec> filter;
    filter.load(a, ch);

    float win[kKeep + kGroup][kVec];   // the kKeep rows before token t, oldest first, and a group's own
    // Row `back` rows before token t of the sequence.
    auto before = [&](int back, float (&row)[kVec]) {
        typename R::type r = R::zero();
        if (t - back >= begin)
            load_bf16(x + (t - back) * a.ldx, r);
        else if (a.init_state)
            load_bf16(init + (seq * kKeep + kKeep + (t - back - begin)) * a.D, r);
        R::unpack(r, row);
    };
    auto window = [&]() {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) before(kKeep - i, win[i]);
    };
    // The states of the sequences that end at token t; the next one's window.
    auto close = [&]() {
        while (t == seq_end) {
            if (a.final_state)
#pragma unroll
                for (int i = 0; i < kKeep; ++i) store_vec<kVec>(final_state + (seq * kKeep + i) * a.D, win[i]);
            if (!kPacked || ++seq >= a.N) break;
            begin = seq_end;
            seq_end = a.cu_seqlens[seq + 1];
            window();
        }
    };
    window();
    close();
    while (t < end) {
        // A whole group within the sequence, or a token at a time.
        if (t + kGroup <= end && t + kGroup <= seq_end) {
            typename R::type raw[kGroup];
#pragma unroll
            for (int i = 0; i < kGroup; ++i) load_bf16(x + (t + i) * a.ldx, raw[i]);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) R::unpack(raw[i], win[kKeep + i]);
#pragma unroll
            for (int i = 0; i < kGroup; ++i) filter.apply(win + i, a.silu, out + (t + i) * a.D);
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
#pragma unroll
                for (int j = 0; j < kVec; ++j) win[i][j] = win[kGroup + i][j];
            t += kGroup;
        } else {
            typename R::type raw;
            load_bf16(x + t * a.ldx, raw);
            R::unpack(raw, win[kKeep]);
            filter.apply(win, a.silu, out + t * a.D);
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
#pragma unroll
                for (int j = 0; j < kVec; ++j) win[i][j] = win[i + 1][j];
            ++t;
        }
        close();
    }
}

// One token for kSeqs sequences and kVec channels a thread.
template <int kW, int kVec, int kSeqs>
__global__ void __launch_bounds__(kConvThreads) conv_decode_kernel(ConvArgs a) {
    wait_for_kernel_before();
    using R = Raw<kVec>;
    constexpr int kKeep = kW - 1;
    const int64_t vecs = a.D / kVec, at = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
    const int64_t part = at / vecs, ch = (at - part * vecs) * kVec;
    if (part * kSeqs >= a.N) return;
    const auto x = static_cast<const __nv_bfloat16*>(a.x) + ch;
    const auto state = static_cast<__nv_bfloat16*>(a.state) + ch;
    const auto out = static_cast<__nv_bfloat16*>(a.out) + ch;
    int64_t slot[kSeqs];
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int64_t n = part * kSeqs + i;
        slot[i] = n < a.N ? (a.slots ? a.slots[n] : n) : -1;
        if (slot[i] >= a.pool) {
            if (ch == 0) atomicOr(a.status, kDevBadSlots);
            slot[i] = -1;
        }
    }
    typename R::type raw[kSeqs][kW];
#pragma unroll
    for (int i = 0; i < kSeqs; ++i)
        if (slot[i] >= 0) {
#pragma unroll
            for (int j = 0; j < kKeep; ++j) load_bf16(state + (slot[i] * kKeep + j) * a.D, raw[i][j]);
            load_bf16(x + (part * kSeqs + i) * a.ldx, raw[i][kKeep]);
        }
    Filter<kW, kVec> filter;
    filter.load(a, ch);
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int64_t n = part * kSeqs + i;
        if (slot[i] >= 0) {
            float win[kW][kVec];
#pragma unroll
            for (int j = 0; j < kW; ++j) {
                R::unpack(raw[i][j], win[j]);
                if (j > 0) *reinterpret_cast<typename R::type*>(state + (slot[i] * kKeep + j - 1) * a.D) = raw[i][j];
            }
            filter.apply(win, a.silu, out + n * a.D);
        } else if (n < a.N) {
            *reinterpret_cast<typename R::type*>(out + n * a.D) = R::zero();
        }
    }
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool on4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

// The widest vector that every row starts on: 8 channels need rows and filters
// on 16 bytes, 2 on 4 (filters are 16-byte aligned tensors).
int conv_vec(const ConvArgs& a) {
    if (a.D % 8 == 0 && (a.rows < 2 || a.ldx % 8 == 0) && on16(a.x)) return 8;
    return a.D % 2 == 0 && (a.rows < 2 || a.ldx % 2 == 0) && on4(a.x) ? 2 : 1;
}

template <int kW, int kVec>
cudaError_t run_prefill(ConvArgs a, int sms, cudaStream_t stream) {
    // Runs of 32 tokens, and shorter ones where there are too few threads: the
    // rows before a run are read twice, W - 1 for each.
    a.run_tokens = 32;
    while (a.run_tokens > 4 && a.rows / a.run_tokens * (a.D / kVec) < static_cast<int64_t>(sms) * 1024) a.run_tokens /= 2;
    if (a.cu_seqlens) {
        a.runs = (a.rows + a.run_tokens - 1) / a.run_tokens;
        if (a.runs == 0) a.runs = 1;   // no tokens: the states alone
    } else {
        a.runs_per_seq = (a.tokens_per_seq + a.run_tokens - 1) / a.run_tokens;
        if (a.runs_per_seq == 0) a.runs_per_seq = 1;
        a.runs = a.N * a.runs_per_seq;
    }
    const int64_t vecs = a.D / kVec;
    if (a.runs > (int64_t(1) << 40) / vecs) return cudaErrorInvalidValue;
    const int64_t ctas = (a.runs * vecs + kConvThreads - 1) / kConvThreads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_after(a.cu_seqlens ? conv_prefill_kernel<kW, kVec, true> : conv_prefill_kernel<kW, kVec, false>,
                        dim3(static_cast<unsigned>(ctas)), dim3(kConvThreads), 0, stream, a);
}

template <int kW, int kVec, int kSeqs>
cudaError_t run_decode(const ConvArgs& a, cudaStream_t stream) {
    const int64_t vecs = a.D / kVec, parts = (a.N + kSeqs - 1) / kSeqs;
    if (parts > (int64_t(1) << 40) / vecs) return cudaErrorInvalidValue;
    const int64_t ctas = (parts * vecs + kConvThreads - 1) / kConvThreads;
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_after(conv_decode_kernel<kW, kVec, kSeqs>, dim3(static_cast<unsigned>(ctas)), dim3(kConvThreads), 0, stream, a);
}

template <int kW, int kVec>
cudaError_t pick(const ConvArgs& a, bool decode, int sms, cudaStream_t stream) {
    if (!decode) return run_prefill<kW, kVec>(a, sms, stream);
    // Four sequences a thread share its filter where that still fills the SMs.
    if (a.N / 4 * (a.D / kVec) >= static_cast<int64_t>(sms) * 512) return run_decode<kW, kVec, 4>(a, stream);
    return run_decode<kW, kVec, 1>(a, stream);
}
template <int kW>
cudaError_t pick(const ConvArgs& a, bool decode, int sms, cudaStream_t stream) {
    const int vec = conv_vec(a);
    if (vec == 8) return pick<kW, 8>(a, decode, sms, stream);
    return vec == 2 ? pick<kW, 2>(a, decode, sms, stream) : pick<kW, 1>(a, decode, sms, stream);
}
cudaError_t pick(const ConvArgs& a, bool decode, int sms, cudaStream_t stream) {
    if (a.W == 2) return pick<2>(a, decode, sms, stream);
    if (a.W == 3) return pick<3>(a, decode, sms, stream);
    return a.W == 4 ? pick<4>(a, decode, sms, stream) : cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_conv_prefill(const ConvArgs& a, int sms, cudaStream_t stream) {
    if (a.N <= 0 || a.D <= 0) return cudaSuccess;
    return pick(a, false, sms, stream);
}
cudaError_t launch_conv_decode(const ConvArgs& a, int sms, cudaStream_t stream) {
    if (a.N <= 0 || a.D <= 0) return cudaSuccess;
    return pick(a, true, sms, stream);
}

}  // namespace kda
