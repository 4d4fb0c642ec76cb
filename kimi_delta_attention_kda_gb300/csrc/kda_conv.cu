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

// Two groups of eight rows are under way while one is worked on, in five CTAs of 128
// threads (96 registers).  8192 x 12288: 68 us (a copy of as many bytes 62, without the SiLU
// 64); one group ahead 71, in registers instead of shared memory 72, three 70, four 73;
// groups of four and six rows 70 to 76, four CTAs 73, six (spilled) 90.
constexpr int kConvThreads = 128;
constexpr int kConvCtas = 5;   // an SM
constexpr int kGroup = 8;

// kVec consecutive BF16 values as loaded, and as pairs of FP32 values (of one: with
// a zero): 4, or 2 or 1 where rows start at any element.
template <int kVec>
struct Raw;
template <>
struct Raw<4> {
    using type = uint2;
    __device__ __forceinline__ static void unpack(uint2 r, uint64_t (&x)[2]) {
        x[0] = pair(bf16_lo(r.x), bf16_hi(r.x));
        x[1] = pair(bf16_lo(r.y), bf16_hi(r.y));
    }
    __device__ __forceinline__ static uint2 pack(const uint64_t (&x)[2]) {
        const float2 a = halves(x[0]), b = halves(x[1]);
        return make_uint2(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y));
    }
    __device__ __forceinline__ static uint2 zero() { return make_uint2(0, 0); }
};
template <>
struct Raw<2> {
    using type = uint32_t;
    __device__ __forceinline__ static void unpack(uint32_t r, uint64_t (&x)[1]) { x[0] = pair(bf16_lo(r), bf16_hi(r)); }
    __device__ __forceinline__ static uint32_t pack(const uint64_t (&x)[1]) {
        const float2 a = halves(x[0]);
        return pack_bf16(a.x, a.y);
    }
    __device__ __forceinline__ static uint32_t zero() { return 0; }
};
template <>
struct Raw<1> {
    using type = uint16_t;
    __device__ __forceinline__ static void unpack(uint16_t r, uint64_t (&x)[1]) { x[0] = pair(bf16_lo(r), 0.f); }
    __device__ __forceinline__ static uint16_t pack(const uint64_t (&x)[1]) {
        return static_cast<uint16_t>(pack_bf16(halves(x[0]).x, 0.f));
    }
    __device__ __forceinline__ static uint16_t zero() { return 0; }
};
template <int kVec>
using RawT = typename Raw<kVec>::type;
template <int kVec>
__device__ __forceinline__ RawT<kVec> load_raw(const __nv_bfloat16* p) {
    return *reinterpret_cast<const RawT<kVec>*>(p);
}
template <int kVec>
__device__ __forceinline__ void store_raw(__nv_bfloat16* p, RawT<kVec> r) {
    *reinterpret_cast<RawT<kVec>*>(p) = r;
}

// A thread's filter: kVec channels with kW taps each, and their bias.
template <int kW, int kVec>
struct Filter {
    static constexpr int kPairs = (kVec + 1) / 2;
    uint64_t w[kW][kPairs], b[kPairs];

    template <typename T>
    __device__ __forceinline__ void load_as(const T* weight, const T* bias, int64_t ch) {
        float f[2 * kPairs * kW] = {}, c[2 * kPairs] = {};
#pragma unroll
        for (int i = 0; i < kW; ++i) load_vec<kVec>(weight + ch * kW + i * kVec, *reinterpret_cast<float(*)[kVec]>(f + i * kVec));
        if (bias) load_vec<kVec>(bias + ch, *reinterpret_cast<float(*)[kVec]>(c));
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            b[j] = pair(c[2 * j], c[2 * j + 1]);
#pragma unroll
            for (int i = 0; i < kW; ++i) w[i][j] = pair(f[2 * j * kW + i], f[(2 * j + 1) * kW + i]);
        }
    }
    __device__ __forceinline__ void load(const ConvArgs& a, int64_t ch) {
        if (a.weight_f32)
            load_as(static_cast<const float*>(a.weight), static_cast<const float*>(a.bias), ch);
        else
            load_as(static_cast<const __nv_bfloat16*>(a.weight), static_cast<const __nv_bfloat16*>(a.bias), ch);
    }
    // Row kW - 1 of x is the token's own.
    __device__ __forceinline__ RawT<kVec> apply(const uint64_t (*x)[kPairs], bool silu) const {
        uint64_t y[kPairs];
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            y[j] = b[j];
#pragma unroll
            for (int i = 0; i < kW; ++i) y[j] = fma_pair(w[i][j], x[i][j], y[j]);
            if (silu) y[j] = silu_pair(y[j]);
        }
        return Raw<kVec>::pack(y);
    }
};

// A thread's rows on their way, kGroups groups of them in shared memory, which it alone
// copies and reads (asynchronous copies are of four bytes at least: single elements wait
// in registers, one group of them).
template <int kVec>
struct Ring {
    static constexpr int kGroups = kVec > 1 ? 2 : 1;
    RawT<kVec>* mine;   // [kGroups * kGroup][kConvThreads]
    RawT<kVec> held[kVec > 1 ? 1 : kGroup];

    // The rows from p on, the first n of a group, to its place.
    __device__ __forceinline__ void fetch(int group, const __nv_bfloat16* p, int64_t ld, int n) {
        if constexpr (kVec > 1) {
            const uint32_t to = smem_u32(mine + (group % kGroups) * kGroup * kConvThreads);
            if (n >= kGroup) {
#pragma unroll
                for (int i = 0; i < kGroup; ++i)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + i * kConvThreads * 2 * kVec), "l"(p + i * ld), "n"(2 * kVec) : "memory");
            } else {
                for (int i = 0; i < n; ++i)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to + i * kConvThreads * 2 * kVec), "l"(p + i * ld), "n"(2 * kVec) : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        } else if (n >= kGroup) {
#pragma unroll
            for (int i = 0; i < kGroup; ++i) held[i] = load_raw<kVec>(p + i * ld);
        }
    }
    // The oldest group is there.
    __device__ __forceinline__ void wait() {
        if constexpr (kVec > 1) asm volatile("cp.async.wait_group %0;" ::"n"(kGroups - 1) : "memory");
    }
    // Row i of a group, of a whole one; or of any, from p where it is not held.
    __device__ __forceinline__ RawT<kVec> row(int group, int i) const {
        if constexpr (kVec > 1)
            return mine[((group % kGroups) * kGroup + i) * kConvThreads];
        else
            return held[i];
    }
    __device__ __forceinline__ RawT<kVec> any_row(int group, int i, const __nv_bfloat16* p) const {
        if constexpr (kVec > 1)
            return row(group, i);
        else
            return load_raw<kVec>(p);
    }
};

// (Tokens are counted in 32 bits: there are fewer than 2^31.)
template <int kW, int kVec, bool kPacked>
__global__ void __launch_bounds__(kConvThreads, kConvCtas) conv_prefill_kernel(ConvArgs a) {
    __shared__ RawT<kVec> places[Ring<kVec>::kGroups * kGroup * kConvThreads];
    wait_for_kernel_before();
    if (kPacked && !offsets_hold(a.cu_seqlens, a.N, a.tokens, a.valid, a.status)) return;
    const int64_t vecs = a.D / kVec, at = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
    const int64_t run = quotient(at, vecs), ch = (at - run * vecs) * kVec;
    if (run >= a.runs) return;
    using R = Raw<kVec>;
    constexpr int kKeep = kW - 1, kPairs = Filter<kW, kVec>::kPairs;
    const auto x = static_cast<const __nv_bfloat16*>(a.x) + ch;
    const auto init = static_cast<const __nv_bfloat16*>(a.init_state) + ch;
    const auto final_state = static_cast<__nv_bfloat16*>(a.final_state) + ch;

    // The run's tokens [t, end).
    int64_t seq = kPacked ? 0 : quotient(run, a.runs_per_seq);
    int begin = kPacked ? 0 : static_cast<int>(seq * a.tokens_per_seq);
    int t = kPacked ? static_cast<int>(run * a.run_tokens) : begin + static_cast<int>((run - seq * a.runs_per_seq) * a.run_tokens);
    int seq_end = static_cast<int>(kPacked ? a.tokens : begin + a.tokens_per_seq);
    const int end = t + a.run_tokens < seq_end ? static_cast<int>(t + a.run_tokens) : seq_end;
    const __nv_bfloat16* next = x + t * a.ldx;   // of the group to fetch next
    auto out = static_cast<__nv_bfloat16*>(a.out) + ch + t * a.D;
    Ring<kVec> ring;
    ring.mine = places + threadIdx.x;
    int left = end - t;   // tokens from there on
    auto fetch = [&](int group) {
        ring.fetch(group, next, a.ldx, left);
        next += kGroup * a.ldx;
        left -= kGroup;
    };
#pragma unroll
    for (int i = 0; i < Ring<kVec>::kGroups; ++i) fetch(i);
    Filter<kW, kVec> filter;
    filter.load(a, ch);
    if (kPacked) {   // the sequence and its first token; the first run also has the empty ones before that
        seq = run == 0 ? 0 : ended_by(a.cu_seqlens, a.N, t);
        begin = static_cast<int>(a.cu_seqlens[seq]);
        seq_end = static_cast<int>(a.cu_seqlens[seq + 1]);
    }
    uint64_t win[kKeep + kGroup][kPairs];   // the kKeep rows before token t, oldest first, and a group's own
    auto window = [&]() {
#pragma unroll
        for (int i = 0; i < kKeep; ++i) {
            RawT<kVec> r = R::zero();
            const int at = t - kKeep + i;   // below the sequence's first token: the initial state
            if (at >= begin)
                r = load_raw<kVec>(x + at * a.ldx);
            else if (a.init_state)
                r = load_raw<kVec>(init + (seq * kKeep + kKeep + (at - begin)) * a.D);
            R::unpack(r, win[i]);
        }
    };
    // The states of the sequences that end at token t; the next one's window.
    auto close = [&]() {
        while (t == seq_end) {
            if (a.final_state)
#pragma unroll
                for (int i = 0; i < kKeep; ++i) store_raw<kVec>(final_state + (seq * kKeep + i) * a.D, R::pack(win[i]));
            if (!kPacked || ++seq >= a.N) break;
            begin = seq_end;
            seq_end = static_cast<int>(a.cu_seqlens[seq + 1]);
            window();
        }
    };
    auto shift = [&](int n) {
#pragma unroll
        for (int i = 0; i < kKeep; ++i)
#pragma unroll
            for (int j = 0; j < kPairs; ++j) win[i][j] = win[n + i][j];
    };
    window();
    for (int group = 0;; ++group) {
        close();
        if (t >= end) return;
        ring.wait();
        const int last = end < seq_end ? end : seq_end;
        if (last - t >= kGroup) {   // a whole group within the sequence
#pragma unroll
            for (int i = 0; i < kGroup; ++i) R::unpack(ring.row(group, i), win[kKeep + i]);
            fetch(group + Ring<kVec>::kGroups);
            t += kGroup;
#pragma unroll
            for (int i = 0; i < kGroup; ++i) {
                store_raw<kVec>(out, filter.apply(win + i, a.silu));
                out += a.D;
            }
            shift(kGroup);
        } else {   // a token at a time
            const int n = end - t < kGroup ? end - t : kGroup;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
                close();
                R::unpack(ring.any_row(group, i, x + t * a.ldx), win[kKeep]);
                ++t;
                store_raw<kVec>(out, filter.apply(win, a.silu));
                out += a.D;
                shift(1);
            }
            fetch(group + Ring<kVec>::kGroups);
        }
    }
}

// One token for kSeqs sequences and kVec channels a thread.  Bound by HBM: 128 x 36,864
// 12.6 us, of which the bytes 11.0 at the rate of a copy.  The states are stored
// streaming, as nobody reads them before the next token (14.2 without).
template <int kW, int kVec, int kSeqs>
__global__ void __launch_bounds__(kConvThreads) conv_decode_kernel(ConvArgs a) {
    wait_for_kernel_before();
    using R = Raw<kVec>;
    constexpr int kKeep = kW - 1;
    const int64_t vecs = a.D / kVec, at = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
    const int64_t part = quotient(at, vecs), ch = (at - part * vecs) * kVec;
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
    RawT<kVec> raw[kSeqs][kW];
#pragma unroll
    for (int i = 0; i < kSeqs; ++i)
        if (slot[i] >= 0) {
#pragma unroll
            for (int j = 0; j < kKeep; ++j) raw[i][j] = load_raw<kVec>(state + (slot[i] * kKeep + j) * a.D);
            raw[i][kKeep] = load_raw<kVec>(x + (part * kSeqs + i) * a.ldx);
        }
    Filter<kW, kVec> filter;
    filter.load(a, ch);
#pragma unroll
    for (int i = 0; i < kSeqs; ++i) {
        const int64_t n = part * kSeqs + i;
        if (slot[i] >= 0) {
            uint64_t win[kW][Filter<kW, kVec>::kPairs];
#pragma unroll
            for (int j = 0; j < kW; ++j) {
                R::unpack(raw[i][j], win[j]);
                if (j > 0) __stcs(reinterpret_cast<RawT<kVec>*>(state + (slot[i] * kKeep + j - 1) * a.D), raw[i][j]);
            }
            store_raw<kVec>(out + n * a.D, filter.apply(win, a.silu));
        } else if (n < a.N) {
            store_raw<kVec>(out + n * a.D, R::zero());
        }
    }
}

// The widest vector that every row of x starts on (the other tensors start on 16 bytes).
int conv_vec(const ConvArgs& a) {
    auto fits = [&](int n) {
        return a.D % n == 0 && (a.rows < 2 || a.ldx % n == 0) && reinterpret_cast<uintptr_t>(a.x) % (2 * n) == 0;
    };
    return fits(4) ? 4 : fits(2) ? 2 : 1;
}

template <int kW, int kVec>
cudaError_t run_prefill(ConvArgs a, int sms, cudaStream_t stream) {
    // Runs of 64 tokens, and shorter ones, of a group at least, for two waves of threads:
    // a run begins with its filter and the W - 1 rows before it.
    a.run_tokens = 64;
    while (a.run_tokens > kGroup && a.rows / a.run_tokens * (a.D / kVec) < 2 * kConvCtas * kConvThreads * static_cast<int64_t>(sms)) a.run_tokens /= 2;
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
    // Two sequences a thread share its filter where that still fills the SMs: 128 x 36,864
    // 12.6 us, with four 13.1, with one 16.
    if (a.N / 2 * (a.D / kVec) >= static_cast<int64_t>(sms) * 512) return run_decode<kW, kVec, 2>(a, stream);
    return run_decode<kW, kVec, 1>(a, stream);
}
template <int kW>
cudaError_t pick(const ConvArgs& a, bool decode, int sms, cudaStream_t stream) {
    const int vec = conv_vec(a);
    if (vec == 4) return pick<kW, 4>(a, decode, sms, stream);
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
