// kda_ops_api.cu -- the C entry points of the operators around the prefill
// (declared in include/kda.h): argument checks, workspace and launches on the
// caller's stream.  No host <-> device synchronisation, no host reads of
// device data.
#include "../../include/kda.h"
#include "kda_common.cuh"
#include "kda_launch.h"

namespace kda {
namespace {

constexpr int64_t kMaxElems = int64_t(1) << 56;
constexpr int64_t kStateElems = kHeadDim * kHeadDim;

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Span {
    uintptr_t lo, hi;
    Span(const void* p, int64_t bytes)
        : lo(reinterpret_cast<uintptr_t>(p)), hi(p ? lo + static_cast<uintptr_t>(bytes) : lo) {}
    bool meets(const Span& o) const { return lo != hi && o.lo != o.hi && lo < o.hi && o.lo < hi; }
};
template <size_t n>
bool meets_any(const Span& s, const Span (&others)[n]) {
    for (const Span& o : others)
        if (s.meets(o)) return true;
    return false;
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

struct LaPlan {
    bool packed;
    int64_t N, tokens;
    int64_t meta_bytes;   // packed: the verdict on the offsets, and whether there is a cut
};

int plan_la(int64_t B, int64_t T, int64_t H, bool packed, LaPlan* p) {
    if (B < 1 || T < 0 || H < 1) return KDA_ERR_SHAPE;
    if (H > kMaxElems / kStateElems || B > kMaxElems / (H * kStateElems)) return KDA_ERR_SHAPE;
    if (!packed && T > 0 && B > kMaxElems / T) return KDA_ERR_SHAPE;
    p->packed = packed;
    p->N = B;
    p->tokens = packed ? T : B * T;
    if (p->tokens >= (int64_t(1) << 31) || p->tokens > kMaxElems / (H * kHeadDim)) return KDA_ERR_SHAPE;
    if (B * H > 0x7fffffffLL) return KDA_ERR_SHAPE;
    p->meta_bytes = packed ? 256 : 0;
    return KDA_OK;
}

// The cut of a call's sequences into spans (see kda_la_prefill).  A packed
// batch's lengths are on the device, and so is its choice (launch_la_cut).
constexpr int64_t kMinPackedChunks = 16;   // fewer in all: not worth the launches
// Fixed layout, one span of a head to an SM, in microseconds a call among others:
// an uncut chain takes 5 and 2.4 a chunk (8 chunks 23, 16 42, 64 151 to 161, 128
// 313), a cut call 15 and 4.5 for each chunk of a span, in both passes (spans of 1
// chunk 15 to 24, of 3 28, 16 86, 22 114, 32 157 to 165, 64 297 to 313; more heads
// take longer).  So 8 chunks of 2 heads are cut (23 against 16), 4 are not (14
// against 15), nor 64 of 76 heads (161 against 165).
constexpr double kLaFixedChunkUs = 2.4, kLaFixedCutChunkUs = 4.5, kLaFixedCutUs = 10;

struct LaCut {
    int64_t chunks = 0;        // chunks of a span (packed: when forced)
    int64_t segs = 0;          // fixed: spans of each sequence
    int64_t spans = 0;         // in all (0: no cut; packed: the most there can be)
    bool order = false;        // packed: an uncut batch's sequences go longest first
    int64_t init_bytes = 0;    // when final states overwrite initial ones (not in bytes)
    int64_t bytes = 0;         // states, decays, the packed tables and the order
};

LaCut cut_la(const LaPlan& pl, int64_t T, int64_t H, int sms, int allowed, int64_t forced) {
    LaCut c, none;
    if (pl.tokens <= 0) return c;
    const int64_t units = pl.N * H;
    if (pl.packed && pl.N > 1 && pl.N <= kMaxLaOrdered && units > sms && pl.tokens >= kMinPackedChunks * kLaChunk) {
        c.order = none.order = true;
        c.bytes = none.bytes = align256(4 * pl.N);
    }
    if (!allowed) return none;
    if (forced > 0) {
        c.chunks = (forced + kLaChunk / 16 - 1) / (kLaChunk / 16);
        if (c.chunks > (1 << 23)) c.chunks = 1 << 23;   // 2^30 tokens
    }
    if (pl.packed) {
        if (forced > 0) {
            c.spans = (pl.tokens / kLaChunk + pl.N) / c.chunks + 1;
        } else {
            // (A cut costs every SM its part of the chunks; without one, one
            // sequence is the most that a batch can wait for.)
            c.spans = sms / H;
            const double part = static_cast<double>(H) / sms, uncut = part + 0.5 > 1. ? part + 0.5 : 1.;
            if (pl.tokens < kMinPackedChunks * kLaChunk || c.spans < 2 || kLaCutChunkUs >= kLaChunkUs * uncut * c.spans)
                return none;
        }
    } else {
        const int64_t seq_chunks = (T + kLaChunk - 1) / kLaChunk;
        if (forced <= 0) {
            if (2 * units > sms) return none;
            const int64_t want = sms / units;
            c.chunks = (seq_chunks + want - 1) / want;
            const int64_t segs = (seq_chunks + c.chunks - 1) / c.chunks;
            const double cut = kLaFixedCutUs + c.chunks * kLaFixedCutChunkUs;
            if (segs < 2 || cut >= seq_chunks * kLaFixedChunkUs) return none;
        }
        c.segs = (seq_chunks + c.chunks - 1) / c.chunks;
        c.spans = c.segs * pl.N;
    }
    if (units > 0x7fffffffLL / 128 || c.spans > 0x7fffffffLL / H || c.spans > kMaxElems / (H * kStateElems * 4)) return none;
    c.init_bytes = units * kStateElems * 4;
    c.bytes += align256(c.spans * H * kStateElems * 4) + align256(c.spans * H * 4);
    if (pl.packed) c.bytes += align256(16 * (pl.N + c.spans)) + align256(4 * (c.spans + 1)) + align256(8 * pl.N);
    return c;
}

// q, k, v, out, state and slots of a single-token step.
int check_step(const StepArgs& a, int64_t g_bytes, int64_t g_align) {
    if (a.N < 0 || a.H < 1 || a.Hk < 1 || a.H % a.Hk || a.pool < 0) return KDA_ERR_SHAPE;
    if (a.H > kMaxElems / kStateElems || a.pool > kMaxElems / (a.H * kStateElems) ||
        a.N > 0x7fffffffLL / 4 / a.H)
        return KDA_ERR_SHAPE;
    if (!a.slots && a.N > a.pool) return KDA_ERR_SHAPE;
    if (a.N == 0) return KDA_OK;
    if (!a.q || !a.k || !a.v || !a.g || !a.out || (a.pool > 0 && !a.state)) return KDA_ERR_NULL;
    if (!aligned(a.q, 16) || !aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.out, 16) ||
        !aligned(a.state, 16) || !aligned(a.g, g_align) || !aligned(a.slots, 4))
        return KDA_ERR_ALIGN;
    const int64_t hv = a.N * a.H * kHeadDim * 2, hk = a.N * a.Hk * kHeadDim * 2;
    const Span state(a.state, a.pool * a.H * kStateElems * (a.state_f32 ? 4 : 2)), out(a.out, hv);
    const Span in[] = {Span(a.q, hk), Span(a.k, hk), Span(a.v, hv), Span(a.g, g_bytes),
                       Span(a.beta, a.N * a.H * 2), Span(a.slots, a.N * 4)};
    if (meets_any(out, in) || meets_any(state, in) || out.meets(state)) return KDA_ERR_OVERLAP;
    return KDA_OK;
}

int run_step(StepArgs& a, bool delta, void* stream) {
    DeviceView d;
    int rc = device_view(&d);
    if (rc != KDA_OK || a.N == 0) return rc;
    a.status = d.status;
    if (launch_step(a, delta, d.sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    add_launches(1);
    return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int kda_la_prefill(const void* q, const void* k, const void* v, const float* g,
                              const void* init_state, void* out, void* final_state, int64_t B,
                              int64_t T, int64_t H, int64_t Hk, const int64_t* cu_seqlens,
                              float scale, uint32_t flags, void* stream_ptr) {
    reset_launches();
    if (flags & ~(KDA_FLAG_STATE_F32 | KDA_FLAG_G_PER_HEAD)) return KDA_ERR_ARG;
    LaPlan pl;
    int rc = plan_la(B, T, H, cu_seqlens != nullptr, &pl);
    if (rc != KDA_OK) return rc;
    if (Hk < 1 || H % Hk) return KDA_ERR_SHAPE;
    if (pl.tokens > 0 && (!q || !k || !v || !g || !out)) return KDA_ERR_NULL;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 4) ||
        !aligned(out, 16) || !aligned(init_state, 16) || !aligned(final_state, 16) ||
        !aligned(cu_seqlens, 8))
        return KDA_ERR_ALIGN;
    LaArgs a = {};
    a.state_f32 = (flags & KDA_FLAG_STATE_F32) != 0;
    const bool per_head = (flags & KDA_FLAG_G_PER_HEAD) != 0;
    {
        const int64_t hv = pl.tokens * H * kHeadDim * 2, hk = pl.tokens * Hk * kHeadDim * 2;
        const int64_t st = B * H * kStateElems * (a.state_f32 ? 4 : 2);
        const Span so(out, hv), sf(final_state, st), si(init_state, st);
        const Span in[] = {Span(q, hk), Span(k, hk), Span(v, hv),
                           Span(g, per_head ? 4 * H : 4 * pl.tokens * H), Span(cu_seqlens, 8 * (B + 1))};
        if (meets_any(so, in) || meets_any(sf, in) || so.meets(sf) || so.meets(si) ||
            (final_state != init_state && sf.meets(si)))
            return KDA_ERR_OVERLAP;
    }
    DeviceView d;
    rc = device_view(&d);
    if (rc != KDA_OK) return rc;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    a.q = q;
    a.k = k;
    a.v = v;
    a.g = g;
    a.g_stride = per_head ? 0 : H;
    a.init_state = init_state;
    a.out = out;
    a.final_state = final_state;
    a.N = B;
    a.tokens = pl.tokens;
    a.tokens_per_seq = T;
    a.H = H;
    a.Hk = Hk;
    a.scale = scale;
    a.status = d.status;
    const LaCut cut = cut_la(pl, T, H, d.sms, d.segments, d.seg_chunks);
    uint8_t* ws = nullptr;
    const bool in_place = init_state && init_state == final_state;
    const int64_t ws_bytes = pl.meta_bytes + cut.bytes + (in_place ? cut.init_bytes : 0);
    if (ws_bytes > 0 &&
        cudaMallocFromPoolAsync(reinterpret_cast<void**>(&ws), static_cast<size_t>(ws_bytes), d.pool, stream) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    LaSegments sg = {};
    uint8_t* at = ws + pl.meta_bytes;
    auto take = [&at](int64_t bytes) {
        uint8_t* p = at;
        at += align256(bytes);
        return p;
    };
    if (cut.spans > 0) {
        sg.starts = reinterpret_cast<float*>(take(cut.spans * H * kStateElems * 4));
        sg.decay = reinterpret_cast<float*>(take(cut.spans * H * 4));
        if (in_place) sg.inits = reinterpret_cast<float*>(take(cut.init_bytes));
        sg.spans = cut.spans;
        sg.segs = cut.segs;
        sg.seg_tokens_each = cut.chunks * kLaChunk;
    }
    if (pl.packed) {
        int32_t* valid = reinterpret_cast<int32_t*>(ws);
        if (cut.spans > 0) {
            sg.cut = valid + 1;
            sg.part = reinterpret_cast<int4*>(take(16 * (B + cut.spans)));
            sg.first = reinterpret_cast<int32_t*>(take(4 * (cut.spans + 1)));
            sg.inner = reinterpret_cast<int2*>(take(8 * B));
        }
        if (cut.order) sg.order = reinterpret_cast<int32_t*>(take(4 * B));
        a.cu_seqlens = cu_seqlens;
        // With nothing to decide, and few offsets, the prefill kernel checks them itself.
        if (cut.spans > 0 || cut.order || B > kMaxLaOrdered) {
            if (launch_la_cut(cu_seqlens, B, T, H, d.sms, sg, static_cast<int>(cut.chunks), valid, d.status, stream) !=
                cudaSuccess) {
                rc = KDA_ERR_CUDA;
            } else {
                add_launches(1);
                a.valid = valid;
            }
        }
    }
    if (rc == KDA_OK) {
        int launches = 0;
        if (launch_la_prefill(a, sg, d.sms, stream, &launches) != cudaSuccess) rc = KDA_ERR_CUDA;
        add_launches(launches);
    }
    if (ws) cudaFreeAsync(ws, stream);
    if (rc != KDA_OK) cudaGetLastError();
    return rc;
}

extern "C" int kda_la_plan_segments(int64_t B, int64_t T, int64_t H, int packed, int64_t* segs) {
    if (!segs) return KDA_ERR_NULL;
    LaPlan pl;
    int rc = plan_la(B, T, H, packed != 0, &pl);
    if (rc != KDA_OK) return rc;
    DeviceView d;
    rc = device_view(&d);
    if (rc != KDA_OK) return rc;
    const LaCut cut = cut_la(pl, T, H, d.sms, d.segments, d.seg_chunks);
    *segs = pl.packed ? cut.spans : cut.segs;
    return KDA_OK;
}

extern "C" int kda_la_workspace_bytes(int64_t B, int64_t T, int64_t H, int packed, int64_t* bytes) {
    if (!bytes) return KDA_ERR_NULL;
    LaPlan pl;
    int rc = plan_la(B, T, H, packed != 0, &pl);
    if (rc != KDA_OK) return rc;
    // As planned on the current device (on a 152-SM device when there is none).
    DeviceView d;
    if (device_view(&d) != KDA_OK) {
        d.sms = 152;
        segment_settings(&d.segments, &d.seg_chunks);
    }
    const LaCut cut = cut_la(pl, T, H, d.sms, d.segments, d.seg_chunks);
    *bytes = pl.meta_bytes + cut.bytes + cut.init_bytes;
    return KDA_OK;
}

extern "C" int kda_la_decode(const void* q, const void* k, const void* v, const float* g,
                             void* state, const int32_t* slots, void* out, int64_t N, int64_t H,
                             int64_t Hk, int64_t pool, float scale, uint32_t flags, void* stream) {
    reset_launches();
    if (flags & ~(KDA_FLAG_STATE_F32 | KDA_FLAG_G_PER_HEAD)) return KDA_ERR_ARG;
    const bool per_head = (flags & KDA_FLAG_G_PER_HEAD) != 0;
    StepArgs a = {q, k, v, g, per_head ? 0 : H, nullptr, state, slots, out, N, H, Hk, pool, scale,
                  (flags & KDA_FLAG_STATE_F32) != 0, false, nullptr};
    int rc = check_step(a, per_head ? 4 * H : 4 * N * H, 4);
    return rc != KDA_OK ? rc : run_step(a, false, stream);
}

extern "C" int kda_decode(const void* q, const void* k, const void* v, const float* g,
                          const void* beta, void* state, const int32_t* slots, void* out,
                          int64_t N, int64_t H, int64_t pool, uint32_t flags, void* stream) {
    reset_launches();
    if (flags & ~(KDA_FLAG_STATE_F32 | KDA_FLAG_BETA_LOGIT)) return KDA_ERR_ARG;
    StepArgs a = {q, k, v, g, H, beta, state, slots, out, N, H, H, pool, 0.08838834764831845f,
                  (flags & KDA_FLAG_STATE_F32) != 0, (flags & KDA_FLAG_BETA_LOGIT) != 0, nullptr};
    int rc = check_step(a, 4 * N * H * kHeadDim, 16);
    if (rc != KDA_OK) return rc;
    if (N > 0 && !beta) return KDA_ERR_NULL;
    if (!aligned(beta, 2)) return KDA_ERR_ALIGN;
    return run_step(a, true, stream);
}

extern "C" int kda_gated_norm(const void* x, const void* weight, const void* gate, void* out,
                              int64_t rows, int activation, float eps, uint32_t flags,
                              void* stream) {
    reset_launches();
    if (flags & ~(KDA_FLAG_WEIGHT_F32 | KDA_FLAG_GATE_FIRST)) return KDA_ERR_ARG;
    if (activation < KDA_ACT_NONE || activation > KDA_ACT_SILU || !(eps >= 0.f)) return KDA_ERR_ARG;
    if (rows < 0 || rows >= (int64_t(1) << 35)) return KDA_ERR_SHAPE;
    const bool gated = activation != KDA_ACT_NONE;
    const bool w32 = (flags & KDA_FLAG_WEIGHT_F32) != 0;
    if (rows > 0) {
        if (!x || !weight || !out || (gated && !gate)) return KDA_ERR_NULL;
        if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(out, 16) || (gated && !aligned(gate, 16)))
            return KDA_ERR_ALIGN;
        const int64_t b = rows * kHeadDim * 2;
        const Span so(out, b), sx(x, b), sg(gated ? gate : nullptr, b);
        if (so.meets(Span(weight, kHeadDim * (w32 ? 4 : 2))) || (out != x && so.meets(sx)) ||
            (out != gate && so.meets(sg)))
            return KDA_ERR_OVERLAP;
    }
    DeviceView d;
    int rc = device_view(&d);
    if (rc != KDA_OK || rows == 0) return rc;
    if (launch_gated_norm(x, weight, gate, out, rows, activation, (flags & KDA_FLAG_GATE_FIRST) != 0,
                          w32, eps, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    add_launches(1);
    return KDA_OK;
}

extern "C" int kda_residual_norm(const void* x, const void* residual, const void* weight,
                                 const void* post_weight, const void* gate, void* out,
                                 void* residual_out, int64_t rows, int64_t dim, float scale,
                                 float eps, uint32_t flags, void* stream) {
    reset_launches();
    if (flags & ~(KDA_FLAG_WEIGHT_F32 | KDA_FLAG_RESIDUAL_F32)) return KDA_ERR_ARG;
    if (!(eps >= 0.f)) return KDA_ERR_ARG;
    if (rows < 0 || rows > 0x7fffffffLL || dim < 1 || dim > kMaxNormDim) return KDA_ERR_SHAPE;
    ResidualNormArgs a = {x, residual, weight, post_weight, gate, out, residual_out, rows, dim, scale, eps,
                          (flags & KDA_FLAG_WEIGHT_F32) != 0, (flags & KDA_FLAG_RESIDUAL_F32) != 0, nullptr};
    if (rows > 0) {
        if (!x || !residual || !weight || !out || !residual_out) return KDA_ERR_NULL;
        for (const void* p : {x, residual, weight, post_weight, gate, static_cast<const void*>(out),
                              static_cast<const void*>(residual_out)})
            if (!aligned(p, 16)) return KDA_ERR_ALIGN;
        const int64_t n = rows * dim, w = dim * (a.weight_f32 ? 4 : 2), r = n * (a.residual_f32 ? 4 : 2);
        const Span so(out, 2 * n), sro(residual_out, r), sx(x, 2 * n), sr(residual, r);
        const Span in[] = {Span(weight, w), Span(post_weight, w), Span(gate, w)};
        if (meets_any(so, in) || meets_any(sro, in) || so.meets(sro) || so.meets(sr) ||
            sro.meets(sx) || (out != x && so.meets(sx)) || (residual_out != residual && sro.meets(sr)))
            return KDA_ERR_OVERLAP;
    }
    DeviceView d;
    int rc = device_view(&d);
    if (rc != KDA_OK || rows == 0) return rc;
    a.status = d.status;
    if (launch_residual_norm(a, d.sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    add_launches(1);
    return KDA_OK;
}
