// kda_norm.cu -- the norms around a block (sm_103a).
//
// kda_gated_norm, per row of 128 channels:
//     y = x / sqrt(mean(x^2) + eps) * w * act(gate), or the norm of x act(gate) times w;
// kda_residual_norm, per row of any width:
//     u = x or x / sqrt(mean(x^2) + eps) * w_post,  r' = r + scale gate u,
//     y = r' / sqrt(mean(r'^2) + eps) * w.
// Both are bound by HBM: every element is read once and written once, and a
// row stays in registers (or shared memory) between its sums and its outputs.
// Sums and all arithmetic are FP32; outputs are rounded once.
//
// Measured on GB300, floors at 6.80 TB/s, the rate of a plain copy of 2 GB: gated
// norm of 8192 x 96 rows 86 to 88 us among other calls (part of the last call's
// output is still in L2 then), 94 from a flushed L2, 6.4 TB/s (floor 89); residual
// norm of 8192 x 12288, FP32 residual and three weights 206 to 213 us either way,
// 5.8 TB/s (floor 178; a plain copy of as many bytes 196), BF16 residual 136 to 140,
// 5.8 TB/s (floor 119).  Rows above 16384 go one to a CTA, at 64 FP32 values a
// thread and 64 registers, spilled: 2048 x 18432 140 us (floor 67), x 32768 229
// (119).
#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_launch.h"
#include "kda_vec.cuh"
#include "kda_wait.cuh"

namespace kda {
namespace {

__device__ __forceinline__ float inv_rms(float mean, float eps) { return rsqrtf(mean + eps); }

// ------------------------------------------------------------- gated norm
// 16 lanes share a row, 8 channels (16 bytes) each; a thread has kRows rows,
// whose loads are all issued before the first sum.  Five CTAs an SM: without the
// bound some forms take 52 registers, four CTAs, and 98 us for 95.
constexpr int kGnThreads = 256;
constexpr int kGnPass = kGnThreads / 16;   // rows of a CTA at a time

template <typename W, int kAct, bool kFirst, int kRows>
__global__ void __launch_bounds__(kGnThreads, 5)
    gated_norm_kernel(const __nv_bfloat16* x, const W* weight, const __nv_bfloat16* gate,
                      __nv_bfloat16* out, int64_t rows, float eps) {
    const int sub = threadIdx.x & 15;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (kGnPass * kRows) + (threadIdx.x >> 4);
    uint4 xr[kRows], zr[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = row0 + i * kGnPass;
        xr[i] = zr[i] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
            xr[i] = *reinterpret_cast<const uint4*>(x + r * kHeadDim + 8 * sub);
            if (kAct != KDA_ACT_NONE) zr[i] = *reinterpret_cast<const uint4*>(gate + r * kHeadDim + 8 * sub);
        }
    }
    float w[8];
    load8(weight + 8 * sub, w);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float a[8], z[8];
        unpack8(xr[i], a);
        unpack8(zr[i], z);
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float s = 1.f;
            if (kAct != KDA_ACT_NONE) s = sigmoid(z[j]);
            if (kAct == KDA_ACT_SILU) s *= z[j];
            z[j] = s;
            if (kFirst) a[j] *= s;
            ss = fmaf(a[j], a[j], ss);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float rms = inv_rms(ss * (1.f / kHeadDim), eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] *= rms * w[j];
            if (!kFirst) a[j] *= z[j];
        }
        const int64_t r = row0 + i * kGnPass;
        if (r < rows) store8(out + r * kHeadDim + 8 * sub, a);
    }
}

template <typename W, int kAct, bool kFirst, int kRows>
cudaError_t run_gated(const void* x, const void* weight, const void* gate, void* out, int64_t rows,
                      float eps, cudaStream_t stream) {
    const int64_t blocks = (rows + kGnPass * kRows - 1) / (kGnPass * kRows);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    gated_norm_kernel<W, kAct, kFirst, kRows><<<static_cast<unsigned>(blocks), kGnThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(x), static_cast<const W*>(weight), static_cast<const __nv_bfloat16*>(gate),
        static_cast<__nv_bfloat16*>(out), rows, eps);
    return cudaGetLastError();
}

// ---------------------------------------------------------- residual norm
// One row per CTA of kThreads threads; a thread holds kGroups groups of eight
// consecutive elements.
template <int kThreads>
__device__ __forceinline__ float block_sum(float x, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (kThreads == 32) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) buf[warp] = x;
    __syncthreads();
    float y = lane < kThreads / 32 ? buf[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    return y;
}

template <typename R, typename W, int kGroups, int kThreads>
__global__ void __launch_bounds__(kThreads) residual_norm_kernel(ResidualNormArgs p) {
    __shared__ float buf[2][32];
    const int64_t D = p.dim, base = static_cast<int64_t>(blockIdx.x) * D;
    const auto x = static_cast<const __nv_bfloat16*>(p.x) + base;
    const auto res = static_cast<const R*>(p.residual) + base;
    const auto post = static_cast<const W*>(p.post_weight);
    const auto gate = static_cast<const W*>(p.gate);
    const auto weight = static_cast<const W*>(p.weight);
    float u[kGroups][8], r[kGroups][8];
    const float inv_d = 1.f / static_cast<float>(D);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int64_t at = (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = r[i][j] = 0.f;
        if (at < D) {
            load8(x + at, u[i]);
            load8(res + at, r[i]);
        }
    }
    if (post) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(u[i][j], u[i][j], ss);
        const float rms = inv_rms(block_sum<kThreads>(ss, buf[0]) * inv_d, p.eps);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int64_t at = (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8;
            if (at < D) {
                float w[8];
                load8(post + at, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] *= rms * w[j];
            }
        }
    }
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int64_t at = (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8;
        if (at < D) {
            if (gate) {
                float w[8];
                load8(gate + at, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[i][j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                r[i][j] = fmaf(p.scale, u[i][j], r[i][j]);
                ss = fmaf(r[i][j], r[i][j], ss);
            }
            store8(static_cast<R*>(p.residual_out) + base + at, r[i]);
        }
    }
    const float rms = inv_rms(block_sum<kThreads>(ss, buf[1]) * inv_d, p.eps);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int64_t at = (static_cast<int64_t>(i) * kThreads + threadIdx.x) * 8;
        if (at < D) {
            float w[8];
            load8(weight + at, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) r[i][j] *= rms * w[j];
            store8(static_cast<__nv_bfloat16*>(p.out) + base + at, r[i]);
        }
    }
}

// Narrow rows: kLanes lanes a row and kGroups vectors a lane, all loaded before
// the first sum; no barrier.  65536 rows of 128, FP32 residual: 25 us, against 60
// with a CTA of 128 threads a row; of 512 68 and 82, of 768 107 and 103: up to 512.
constexpr int kRowsThreads = 256;
constexpr int64_t kRowsMaxDim = 512;
template <typename R, typename W, int kVec, int kGroups, int kLanes>
__global__ void __launch_bounds__(kRowsThreads) residual_norm_rows_kernel(ResidualNormArgs p) {
    const int D = static_cast<int>(p.dim), lane = threadIdx.x % kLanes;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kRowsThreads / kLanes) + threadIdx.x / kLanes, base = row * D;
    const int end = row < p.rows ? D : 0;
    const auto x = static_cast<const __nv_bfloat16*>(p.x) + base;
    const auto res = static_cast<const R*>(p.residual) + base;
    const auto post = static_cast<const W*>(p.post_weight), gate = static_cast<const W*>(p.gate);
    float u[kGroups][kVec], r[kGroups][kVec];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int at = (i * kLanes + lane) * kVec;
#pragma unroll
        for (int j = 0; j < kVec; ++j) u[i][j] = r[i][j] = 0.f;
        if (at < end) {
            load_vec<kVec>(x + at, u[i]);
            load_vec<kVec>(res + at, r[i]);
        }
    }
    auto sum_row = [](float v) {
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    const float inv_d = 1.f / static_cast<float>(D);
    float ss = 0.f;
    if (post) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int j = 0; j < kVec; ++j) ss = fmaf(u[i][j], u[i][j], ss);
        const float rms = inv_rms(sum_row(ss) * inv_d, p.eps);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int at = (i * kLanes + lane) * kVec;
            if (at < end) {
                float w[kVec];
                load_vec<kVec>(post + at, w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) u[i][j] *= rms * w[j];
            }
        }
        ss = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int at = (i * kLanes + lane) * kVec;
        if (at < end) {
            if (gate) {
                float w[kVec];
                load_vec<kVec>(gate + at, w);
#pragma unroll
                for (int j = 0; j < kVec; ++j) u[i][j] *= w[j];
            }
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                r[i][j] = fmaf(p.scale, u[i][j], r[i][j]);
                ss = fmaf(r[i][j], r[i][j], ss);
            }
            store_vec<kVec>(static_cast<R*>(p.residual_out) + base + at, r[i]);
        }
    }
    const float rms = inv_rms(sum_row(ss) * inv_d, p.eps);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int at = (i * kLanes + lane) * kVec;
        if (at < end) {
            float w[kVec];
            load_vec<kVec>(static_cast<const W*>(p.weight) + at, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) r[i][j] *= rms * w[j];
            store_vec<kVec>(static_cast<__nv_bfloat16*>(p.out) + base + at, r[i]);
        }
    }
}

template <typename R, typename W, int kVec, int kGroups, int kLanes>
cudaError_t run_rows(const ResidualNormArgs& p, cudaStream_t stream) {
    constexpr int64_t each = kRowsThreads / kLanes;
    residual_norm_rows_kernel<R, W, kVec, kGroups, kLanes>
        <<<static_cast<unsigned>((p.rows + each - 1) / each), kRowsThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

// Wide rows of a width that is no multiple of 8, for which the streaming
// kernel has too few rows or too little room: one row per CTA, its new
// residual in shared memory until its norm is known.  Elements (pairs, where the
// width is even) one at a time: 300 rows of 5001 take 16 us, launch and latency.
template <typename R, typename W, int kVec, int kThreads>
__global__ void __launch_bounds__(kThreads) residual_norm_odd_kernel(ResidualNormArgs p) {
    extern __shared__ __align__(16) float row_smem[];
    __shared__ float buf[2][32];
    const int D = static_cast<int>(p.dim), t0 = threadIdx.x * kVec;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * D;
    const auto x = static_cast<const __nv_bfloat16*>(p.x) + base;
    const auto res = static_cast<const R*>(p.residual) + base;
    const auto post = static_cast<const W*>(p.post_weight), gate = static_cast<const W*>(p.gate);
    const float inv_d = 1.f / static_cast<float>(D);
    float rms = 1.f;
    if (post) {
        float ss = 0.f;
        for (int at = t0; at < D; at += kThreads * kVec) {
            float v[kVec];
            load_vec<kVec>(x + at, v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) ss = fmaf(v[j], v[j], ss);
        }
        rms = inv_rms(block_sum<kThreads>(ss, buf[0]) * inv_d, p.eps);
    }
    float ss = 0.f;
    for (int at = t0; at < D; at += kThreads * kVec) {
        float u[kVec], r[kVec], w[kVec];
        load_vec<kVec>(x + at, u);
        load_vec<kVec>(res + at, r);
        if (post) {
            load_vec<kVec>(post + at, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) u[j] *= rms * w[j];
        }
        if (gate) {
            load_vec<kVec>(gate + at, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) u[j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            r[j] = fmaf(p.scale, u[j], r[j]);
            ss = fmaf(r[j], r[j], ss);
        }
        store_vec<kVec>(row_smem + at, r);
        store_vec<kVec>(static_cast<R*>(p.residual_out) + base + at, r);
    }
    rms = inv_rms(block_sum<kThreads>(ss, buf[1]) * inv_d, p.eps);
    for (int at = t0; at < D; at += kThreads * kVec) {   // (a thread's own elements)
        float r[kVec], w[kVec];
        load_vec<kVec>(row_smem + at, r);
        load_vec<kVec>(static_cast<const W*>(p.weight) + at, w);
#pragma unroll
        for (int j = 0; j < kVec; ++j) r[j] *= rms * w[j];
        store_vec<kVec>(static_cast<__nv_bfloat16*>(p.out) + base + at, r);
    }
}

template <typename R, typename W, int kVec, int kThreads>
cudaError_t run_odd(const ResidualNormArgs& p, cudaStream_t stream) {
    const int bytes = static_cast<int>(p.dim) * 4;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(residual_norm_odd_kernel<R, W, kVec, kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kMaxNormDim) * 4);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    residual_norm_odd_kernel<R, W, kVec, kThreads><<<static_cast<unsigned>(p.rows), kThreads, bytes, stream>>>(p);
    return cudaGetLastError();
}

// Many wide rows: every SM walks over its rows, whose x and residual a bulk
// copy brings to shared memory two or three rows ahead; a thread keeps the
// weights of its channels in registers (post weight, gate and scale as one
// factor: they only ever meet as a product).  Reading the weights again for
// every row would take as much of L2's bandwidth as the rows take of HBM's: a
// CTA a row takes 336 us for 8192 x 12288 with an FP32 residual, this 209 (768
// threads; 1024 206, but 144 against 133 with a BF16 residual).  Rows of a width
// that is no multiple of 8 gain more, because shared memory has no need of their
// alignment: 8192 x 12281 213 against 343 us, 65536 x 777 111 against 195.  Up to
// 1024, multiples of 8 are as well served by a CTA a row (65536 x 768: 103, 105).
constexpr int kStreamStages = 3;
constexpr int64_t kStreamMaxDim = 16384, kStreamMinRows = 2;
constexpr int kStreamSmem = 226 * 1024;
// A row that does not start on 16 bytes is copied from the boundary before it to
// the one behind it, and read in shared memory at its offset.
template <typename R, int kVec>
__host__ __device__ constexpr uint32_t stream_x_bytes(uint32_t D) { return kVec == 8 ? 2 * D : (2 * D + 30) & ~15u; }
template <typename R, int kVec>
__host__ __device__ constexpr uint32_t stream_stage_bytes(uint32_t D) {
    constexpr uint32_t n = sizeof(R);
    return stream_x_bytes<R, kVec>(D) + (kVec == 8 ? n * D : (n * D + 30) & ~15u);
}
// The span of row `row` that a bulk copy brings, [lo, up): where the tensor
// ends between two boundaries, up to the one before, and the rest is copied here.
__device__ __forceinline__ void stream_span(const uint8_t* base, uint8_t* dst, int64_t row, int64_t rows, uint32_t row_bytes,
                                            int64_t* lo, int64_t* up) {
    const int64_t at = row * row_bytes, end = at + row_bytes;
    *lo = at & ~int64_t(15);
    *up = (end + 15) & ~int64_t(15);
    if (*up > rows * row_bytes) {
        *up = end & ~int64_t(15);
        for (int64_t b = *up; b < end; b += 2)
            *reinterpret_cast<uint16_t*>(dst + (b - *lo)) = *reinterpret_cast<const uint16_t*>(base + b);
    }
}
template <typename R, typename W, int kVec, int kGroups, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
    residual_norm_stream_kernel(ResidualNormArgs p, int stages) {
    extern __shared__ __align__(16) uint8_t stream_smem[];
    __shared__ uint64_t full[kStreamStages];
    __shared__ float red[2][2][32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int D = static_cast<int>(p.dim);
    const uint32_t xb = D * 2, rb = D * static_cast<uint32_t>(sizeof(R));
    const uint32_t xs_bytes = stream_x_bytes<R, kVec>(D), stage_bytes = stream_stage_bytes<R, kVec>(D);
    const auto x = static_cast<const uint8_t*>(p.x), res = static_cast<const uint8_t*>(p.residual);
    auto fetch = [&](int64_t row, int s) {
        uint8_t* dst = stream_smem + s * stage_bytes;
        if constexpr (kVec == 8) {
            mbar_arrive_expect_tx(&full[s], xb + rb);
            bulk_g2s(dst, x + row * xb, xb, &full[s]);
            bulk_g2s(dst + xs_bytes, res + row * rb, rb, &full[s]);
        } else {
            int64_t xlo, xup, rlo, rup;
            stream_span(x, dst, row, p.rows, xb, &xlo, &xup);
            stream_span(res, dst + xs_bytes, row, p.rows, rb, &rlo, &rup);
            const uint32_t xn = static_cast<uint32_t>(xup - xlo), rn = static_cast<uint32_t>(rup - rlo);
            mbar_arrive_expect_tx(&full[s], xn + rn);
            bulk_g2s(dst, x + xlo, xn, &full[s]);
            bulk_g2s(dst + xs_bytes, res + rlo, rn, &full[s]);
        }
    };
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_barrier_init();
        for (int s = 0; s < stages; ++s) {
            const int64_t row = blockIdx.x + static_cast<int64_t>(s) * gridDim.x;
            if (row < p.rows) fetch(row, s);
        }
    }
    float fac[kGroups][kVec], wt[kGroups][kVec];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        const int at = (i * kThreads + tid) * kVec;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            fac[i][j] = p.scale;
            wt[i][j] = 0.f;
        }
        if (at < D) {
            float v[kVec];
            load_vec<kVec>(static_cast<const W*>(p.weight) + at, wt[i]);
            if (p.post_weight) {
                load_vec<kVec>(static_cast<const W*>(p.post_weight) + at, v);
#pragma unroll
                for (int j = 0; j < kVec; ++j) fac[i][j] *= v[j];
            }
            if (p.gate) {
                load_vec<kVec>(static_cast<const W*>(p.gate) + at, v);
#pragma unroll
                for (int j = 0; j < kVec; ++j) fac[i][j] *= v[j];
            }
        }
    }
    const float inv_d = 1.f / static_cast<float>(D);
    __syncthreads();
    auto sum_all = [&](float v, float* buf) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) buf[warp] = v;
        __syncthreads();
        float y = lane < kThreads / 32 ? buf[lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        return y;
    };
    int s = 0;
    uint32_t phase = 0;
    int odd = 0;   // the sums' buffers alternate from row to row
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        if (!mbar_wait_warp(&full[s], phase, p.status)) {
            // Warp 0 starts the copies, so none follows: none may be under way
            // when the CTA ends.
            const int64_t after = (p.rows - row + gridDim.x - 1) / gridDim.x;
            if (warp == 0) drain_ring(full, stages, s, phase, static_cast<int>(after < stages ? after : stages), p.status);
            return;
        }
        const auto xs = reinterpret_cast<const __nv_bfloat16*>(stream_smem + s * stage_bytes + (kVec == 8 ? 0 : row * xb & 15));
        const auto rs = reinterpret_cast<const R*>(stream_smem + s * stage_bytes + xs_bytes + (kVec == 8 ? 0 : row * rb & 15));
        float rms = 1.f;
        if (p.post_weight) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int at = (i * kThreads + tid) * kVec;
                if (at < D) {
                    float v[kVec];
                    load_vec<kVec>(xs + at, v);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) ss = fmaf(v[j], v[j], ss);
                }
            }
            rms = inv_rms(sum_all(ss, red[odd][0]) * inv_d, p.eps);
        }
        float r[kGroups][kVec], ss = 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int at = (i * kThreads + tid) * kVec;
            if (at < D) {
                float v[kVec];
                load_vec<kVec>(xs + at, v);
                load_vec<kVec>(rs + at, r[i]);
#pragma unroll
                for (int j = 0; j < kVec; ++j) {
                    r[i][j] = fmaf(v[j] * rms, fac[i][j], r[i][j]);
                    ss = fmaf(r[i][j], r[i][j], ss);
                }
                store_vec<kVec>(static_cast<R*>(p.residual_out) + row * D + at, r[i]);
            }
        }
        fence_proxy_async_smem();   // this stage is read; a copy may follow the barrier
        rms = inv_rms(sum_all(ss, red[odd][1]) * inv_d, p.eps);
        const int64_t next = row + static_cast<int64_t>(stages) * gridDim.x;
        if (tid == 0 && next < p.rows) fetch(next, s);
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int at = (i * kThreads + tid) * kVec;
            if (at < D) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) r[i][j] *= rms * wt[i][j];
                store_vec<kVec>(static_cast<__nv_bfloat16*>(p.out) + row * D + at, r[i]);
            }
        }
        odd ^= 1;
        if (++s == stages) {
            s = 0;
            phase ^= 1u;
        }
    }
}

template <typename R, typename W, int kVec, int kGroups, int kThreads>
cudaError_t run_stream(const ResidualNormArgs& p, int sms, cudaStream_t stream) {
    const int row = static_cast<int>(stream_stage_bytes<R, kVec>(static_cast<uint32_t>(p.dim))), room = kStreamSmem / (1024 / kThreads);
    const int stages = row * kStreamStages <= room ? kStreamStages : room / row;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
        e = cudaFuncSetAttribute(residual_norm_stream_kernel<R, W, kVec, kGroups, kThreads>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    const int64_t ctas = static_cast<int64_t>(sms) * (1024 / kThreads);
    residual_norm_stream_kernel<R, W, kVec, kGroups, kThreads>
        <<<static_cast<unsigned>(p.rows < ctas ? p.rows : ctas), kThreads, stages * row, stream>>>(p, stages);
    return cudaGetLastError();
}

template <typename R, typename W, int kGroups, int kThreads>
cudaError_t run_residual(const ResidualNormArgs& p, cudaStream_t stream) {
    residual_norm_kernel<R, W, kGroups, kThreads>
        <<<static_cast<unsigned>(p.rows), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename R, typename W, int kVec>
cudaError_t pick_stream(const ResidualNormArgs& p, int sms, cudaStream_t stream) {
    constexpr int n = 8 / kVec;   // vectors in eight elements
    if constexpr (kVec != 8)
        if (p.dim <= 1024) return run_stream<R, W, kVec, n, 128>(p, sms, stream);
    if (p.dim <= 2048) return run_stream<R, W, kVec, n, 256>(p, sms, stream);
    if (p.dim <= 4096) return run_stream<R, W, kVec, n, 512>(p, sms, stream);
    if (p.dim <= 8192) return run_stream<R, W, kVec, n, 1024>(p, sms, stream);
    if (p.dim <= 12288) return run_stream<R, W, kVec, 2 * n, 768>(p, sms, stream);
    return run_stream<R, W, kVec, 2 * n, 1024>(p, sms, stream);
}
template <typename R, typename W, int kVec>
cudaError_t pick_rows(const ResidualNormArgs& p, cudaStream_t stream) {
    constexpr int n = 8 / kVec;
    if (p.dim <= 64) return run_rows<R, W, kVec, n, 8>(p, stream);
    if (p.dim <= 256) return run_rows<R, W, kVec, n, 32>(p, stream);
    if constexpr (kVec != 8)
        if (p.dim > 512) return run_rows<R, W, kVec, 4 * n, 32>(p, stream);
    return run_rows<R, W, kVec, 2 * n, 32>(p, stream);
}
template <typename R, typename W>
cudaError_t pick_residual(const ResidualNormArgs& p, int sms, cudaStream_t stream) {
    const int64_t D = p.dim;
    const int vec = D % 8 == 0 ? 8 : D % 2 == 0 ? 2 : 1;
    const bool walk = D > kRowsMaxDim && D <= kStreamMaxDim && p.rows >= kStreamMinRows * sms;
    if (vec == 8 && D > kRowsMaxDim && D <= 1024) return run_residual<R, W, 1, 128>(p, stream);
    if (D <= kRowsMaxDim || (D <= 1024 && !walk))
        return vec == 8 ? pick_rows<R, W, 8>(p, stream) : vec == 2 ? pick_rows<R, W, 2>(p, stream) : pick_rows<R, W, 1>(p, stream);
    if (walk)
        return vec == 8 ? pick_stream<R, W, 8>(p, sms, stream)
                        : vec == 2 ? pick_stream<R, W, 2>(p, sms, stream) : pick_stream<R, W, 1>(p, sms, stream);
    if (vec == 2) return run_odd<R, W, 2, 512>(p, stream);
    if (vec == 1) return run_odd<R, W, 1, 512>(p, stream);
    if (D <= 4096) return run_residual<R, W, 2, 256>(p, stream);
    if (D <= 12288) return run_residual<R, W, 3, 512>(p, stream);
    return run_residual<R, W, 4, 1024>(p, stream);
}

}  // namespace

cudaError_t launch_gated_norm(const void* x, const void* weight, const void* gate, void* out,
                              int64_t rows, int activation, bool gate_first, bool weight_f32,
                              float eps, cudaStream_t stream) {
    if (rows <= 0) return cudaSuccess;
    constexpr int kRows = 4;
#define KDA_GN(ACT, FIRST)                                                                            \
    return weight_f32 ? run_gated<float, ACT, FIRST, kRows>(x, weight, gate, out, rows, eps, stream)  \
                      : run_gated<__nv_bfloat16, ACT, FIRST, kRows>(x, weight, gate, out, rows, eps, stream)
    if (activation == KDA_ACT_SIGMOID) {
        if (gate_first) KDA_GN(KDA_ACT_SIGMOID, true);
        KDA_GN(KDA_ACT_SIGMOID, false);
    }
    if (activation == KDA_ACT_SILU) {
        if (gate_first) KDA_GN(KDA_ACT_SILU, true);
        KDA_GN(KDA_ACT_SILU, false);
    }
    KDA_GN(KDA_ACT_NONE, false);
#undef KDA_GN
}

cudaError_t launch_residual_norm(const ResidualNormArgs& p, int sms, cudaStream_t stream) {
    if (p.rows <= 0) return cudaSuccess;
    if (p.rows > 0x7fffffffLL) return cudaErrorInvalidValue;
    if (p.residual_f32)
        return p.weight_f32 ? pick_residual<float, float>(p, sms, stream)
                            : pick_residual<float, __nv_bfloat16>(p, sms, stream);
    return p.weight_f32 ? pick_residual<__nv_bfloat16, float>(p, sms, stream)
                        : pick_residual<__nv_bfloat16, __nv_bfloat16>(p, sms, stream);
}

}  // namespace kda
