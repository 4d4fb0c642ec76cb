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

// Rows of `width` elements that lie `ld` apart, as a range of memory.
int64_t rows_bytes(int64_t rows, int64_t ld, int64_t width, int64_t size) { return rows > 0 ? ((rows - 1) * ld + width) * size : 0; }
bool rows_fit(int64_t rows, int64_t ld, int64_t width) {
    return width <= kMaxElems && (rows < 2 || (ld >= width && ld <= kMaxElems && rows <= kMaxElems / ld));
}

// Scratch of a call from the library's stream-ordered pool, given back in stream order.
struct Scratch {
    uint8_t* p = nullptr;
    int64_t used = 0;
    cudaStream_t stream = nullptr;
    ~Scratch() {
        if (p) cudaFreeAsync(p, stream);
    }
    bool take(int64_t bytes, cudaMemPool_t pool, cudaStream_t s) {
        stream = s;
        if (bytes <= 0) return true;
        if (cudaMallocFromPoolAsync(reinterpret_cast<void**>(&p), static_cast<size_t>(bytes), pool, s) == cudaSuccess) return true;
        cudaGetLastError();
        p = nullptr;
        return false;
    }
    uint8_t* part(int64_t bytes) {
        uint8_t* at = p + used;
        used += align256(bytes);
        return at;
    }
};
// The offsets' check ahead of the kernels that read them, where there are many.
int check_offsets(const int64_t* cu, int64_t N, int64_t tokens, const DeviceView& d, int32_t* valid, cudaStream_t stream) {
    if (launch_la_cut(cu, N, tokens, 1, d.sms, LaSegments{}, 0, valid, d.status, stream) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    add_launches(1);
    return KDA_OK;
}

// Tokens of N sequences, fixed (T each) or packed (T in all).
int count_tokens(int64_t N, int64_t T, bool packed, int64_t* tokens) {
    if (N < 1 || T < 0 || N > 0x7fffffffLL || T >= (int64_t(1) << 31)) return KDA_ERR_SHAPE;
    *tokens = packed ? T : N * T;
    return *tokens < (int64_t(1) << 31) ? KDA_OK : KDA_ERR_SHAPE;
}

int check_conv(const ConvArgs& a, int activation) {
    if (activation != KDA_ACT_NONE && activation != KDA_ACT_SILU) return KDA_ERR_ARG;
    if (a.D < 1 || a.D > kMaxElems / 8 || a.W < 2 || a.W > 4) return KDA_ERR_SHAPE;
    return rows_fit(a.rows, a.ldx, a.D) && a.rows <= kMaxElems / a.D ? KDA_OK : KDA_ERR_SHAPE;
}

// The cut of a call of the scan (see kda_ssm_prefill).
struct SsmCut {
    int64_t tiles_per_group = 0, tiles = 0;
    int64_t spans = 0, spans_per_seq = 1, span_tokens = 0;
    int64_t state_bytes = 0, step_bytes = 0;   // of the spans' states, with more than one
    int64_t relay_bytes = 0;                   // of the flags of spans that run one after the other
    int64_t init_bytes = 0;                    // a copy of initial states that final ones overwrite
    bool cut() const { return state_bytes > 0; }
    int64_t bytes() const { return align256(state_bytes) + align256(step_bytes) + align256(relay_bytes); }
};

// Costs of the scan on GB300, in microseconds for 32 tokens (rows: up to 16, 32 and 64
// states): uncut, of a CTA with one, two and three of them on its SM, of which
// the fullest SM decides; cut, for each CTA's part on every SM, states and outputs.
// T = 8192, uncut and cut: 5,120 channels 458 and 354 us, 6,144 459 and 429, 8,192
// 459 and 559.
constexpr double kSsmTileUs[3][3] = {{1.42, 1.81, 2.47}, {1.69, 2.65, 0}, {2.63, 4.52, 0}};
constexpr double kSsmCutTileUs[3] = {1.27, 2.1, 3.7}, kSsmCutUs = 10;
// Spans one after the other (more chains than SMs), a sixteenth of the tokens each, 512
// at least: for the flags' clearing, and for each span that takes up a state.  Uncut and so:
// 8192 tokens of 12,288 channels 633 and 586 us, of 10,240 632 and 566, two prompts of
// 4096 tokens 627 and 555, 4096 tokens of 12,288 with 64 states 895 and 784.
constexpr double kSsmRelayUs = 10, kSsmRelaySpanUs = 2.2;
constexpr int64_t kSsmRelaySpans = 16, kSsmRelayMin = 16 * kSsmTile;
// A span is this long at least: where that leaves more than one wave of CTAs, whole
// waves of them (a last one that is not full costs as much), the more the better balanced.
constexpr int64_t kSsmMinSpan = 2 * kSsmTile, kSsmGoodSpan = 14 * kSsmTile;

int plan_ssm(int64_t N, int64_t T, int64_t dim, int64_t groups, int64_t nstate, bool packed, bool state_f32, int sms,
             int allowed, int64_t forced, int64_t* tokens, SsmCut* c) {
    *c = SsmCut{};
    int rc = count_tokens(N, T, packed, tokens);
    if (rc != KDA_OK) return rc;
    if (dim < 1 || groups < 1 || dim % groups || nstate < 1 || nstate > kSsmMaxState) return KDA_ERR_SHAPE;
    const int64_t wide = nstate <= 16 ? 16 : nstate <= 32 ? 32 : 64;
    if (dim > kSsmMaxDim || N > kMaxElems / (dim * wide * 4)) return KDA_ERR_SHAPE;
    c->tiles_per_group = (dim / groups + kSsmChannels - 1) / kSsmChannels;
    c->tiles = c->tiles_per_group * groups;
    const int64_t chains = packed ? 1 : N;        // that go on for `length` tokens
    const int64_t length = packed ? *tokens : T;
    c->span_tokens = length > 0 ? length : 1;
    bool relay = false;
    if (allowed && forced > 0 && length > 0) {
        c->span_tokens = forced > length / 16 ? length : (16 * forced + kSsmTile - 1) / kSsmTile * kSsmTile;
    } else if (length > 0) {
        const int row = nstate <= 16 ? 0 : nstate <= 32 ? 1 : 2;
        const int64_t units = c->tiles * chains, resident = row == 0 ? 3 : 2, room = resident * sms;
        const int64_t full = units / room, rest = (units - full * room + sms - 1) / sms;
        const double tiles_each = static_cast<double>(length) / kSsmTile;
        const double uncut = tiles_each * (full * kSsmTileUs[row][resident - 1] + (rest ? kSsmTileUs[row][rest - 1] : 0));
        const double cut = kSsmCutUs + tiles_each * units / sms * kSsmCutTileUs[row];
        const int64_t most = length / kSsmGoodSpan * units / room;   // waves that spans of that length fill
        const int64_t want = (most < 1 ? 1 : most < 8 ? most : 8) * room / units;   // spans of each chain
        double best = uncut;
        if (allowed && want > 1 && length >= 2 * kSsmMinSpan && cut < best) {
            best = cut;
            c->span_tokens = ((length + want - 1) / want + kSsmTile - 1) / kSsmTile * kSsmTile;
            if (c->span_tokens < kSsmMinSpan) c->span_tokens = kSsmMinSpan;
        }
        if (units > sms && length >= 2 * kSsmRelayMin) {
            // Each of an SM's places has a chain that runs with the same probability.
            const double p = units < room ? static_cast<double>(units) / room : 1;
            double rate = 0, ways = 1, with = 1;   // of one SM; places out of those resident; p^n
            for (int64_t n = 1; n <= resident; ++n) {
                ways = ways * (resident - n + 1) / n;
                with *= p;
                double without = 1;
                for (int64_t k = n; k < resident; ++k) without *= 1 - p;
                rate += ways * with * without * n / kSsmTileUs[row][n - 1];
            }
            const int64_t each = length / kSsmRelaySpans / kSsmTile * kSsmTile;
            const int64_t span = each > kSsmRelayMin ? each : kSsmRelayMin;
            const double relays = static_cast<double>(length) / span * (units > room ? static_cast<double>(units) / room : 1);
            if (tiles_each * units / sms / rate + kSsmRelayUs + kSsmRelaySpanUs * relays < 0.97 * best) {
                relay = true;
                c->span_tokens = span;
            }
        }
    }
    c->spans_per_seq = length > 0 ? (length + c->span_tokens - 1) / c->span_tokens : 1;
    c->spans = c->spans_per_seq * chains;
    if (c->spans > 0x7fffffffLL / c->tiles) return KDA_ERR_SHAPE;
    if (c->spans_per_seq > 1) {
        if (c->spans > kMaxElems / (dim * wide * 4)) return KDA_ERR_SHAPE;
        c->state_bytes = c->spans * dim * wide * 4;
        if (relay)
            c->relay_bytes = (1 + c->spans * c->tiles) * 4;
        else
            c->step_bytes = c->spans * dim * 4;
    }
    // (Where a group is no whole 32 channels two CTAs have some of them.)
    if (c->spans_per_seq > 1 || dim / groups % kSsmChannels) c->init_bytes = N * dim * nstate * (state_f32 ? 4 : 2);
    return KDA_OK;
}

// What both forms of the scan read, for `rows` tokens, and where they write.
int check_ssm(const SsmArgs& a, int64_t rows, const Span& read_write, const Span& also_read) {
    const int64_t dt = a.dt_f32 ? 4 : 2, bc = a.bc_f32 ? 4 : 2, w = a.groups * a.nstate;
    if (rows <= 0) return KDA_OK;
    if (!a.x || !a.dt || !a.A || !a.B || !a.C || !a.out) return KDA_ERR_NULL;
    if (!aligned(a.x, 2) || !aligned(a.dt, dt) || !aligned(a.A, 16) || !aligned(a.B, bc) || !aligned(a.C, bc) ||
        !aligned(a.D, 4) || !aligned(a.z, 2) || !aligned(a.dt_bias, 4) || !aligned(a.out, 16))
        return KDA_ERR_ALIGN;
    const Span out(a.out, rows * a.dim * 2);
    const Span in[] = {Span(a.x, rows_bytes(rows, a.ldx, a.dim, 2)), Span(a.dt, rows_bytes(rows, a.lddt, a.dim, dt)),
                       Span(a.B, rows_bytes(rows, a.ldb, w, bc)), Span(a.C, rows_bytes(rows, a.ldc, w, bc)),
                       Span(a.z, rows_bytes(rows, a.ldz, a.dim, 2)), Span(a.A, a.dim * a.nstate * 4), Span(a.D, a.dim * 4),
                       Span(a.dt_bias, a.dim * 4), also_read};
    return meets_any(out, in) || meets_any(read_write, in) || out.meets(read_write) ? KDA_ERR_OVERLAP : KDA_OK;
}
bool ssm_rows_fit(const SsmArgs& a, int64_t rows) {
    const int64_t w = a.groups * a.nstate;
    return rows <= kMaxElems / a.dim && rows_fit(rows, a.ldx, a.dim) && rows_fit(rows, a.lddt, a.dim) && rows_fit(rows, a.ldb, w) &&
           rows_fit(rows, a.ldc, w) && (!a.z || rows_fit(rows, a.ldz, a.dim));
}
constexpr uint32_t kSsmFlags = KDA_FLAG_STATE_F32 | KDA_FLAG_DT_F32 | KDA_FLAG_BC_F32 | KDA_FLAG_DT_SOFTPLUS;
void ssm_flags(SsmArgs* a, uint32_t flags) {
    a->state_f32 = (flags & KDA_FLAG_STATE_F32) != 0;
    a->dt_f32 = (flags & KDA_FLAG_DT_F32) != 0;
    a->bc_f32 = (flags & KDA_FLAG_BC_F32) != 0;
    a->softplus = (flags & KDA_FLAG_DT_SOFTPLUS) != 0;
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

extern "C" int kda_conv_prefill(const void* x, int64_t ldx, const void* weight, const void* bias, const void* init_state,
                                void* out, void* final_state, int64_t B, int64_t T, int64_t D, int W,
                                const int64_t* cu_seqlens, int activation, uint32_t flags, void* stream_ptr) {
    reset_launches();
    if (flags & ~KDA_FLAG_WEIGHT_F32) return KDA_ERR_ARG;
    ConvArgs a = {};
    int rc = count_tokens(B, T, cu_seqlens != nullptr, &a.tokens);
    if (rc != KDA_OK) return rc;
    a.x = x;
    a.ldx = ldx;
    a.weight = weight;
    a.bias = bias;
    a.init_state = init_state;
    a.out = out;
    a.final_state = final_state;
    a.N = B;
    a.rows = a.tokens;
    a.tokens_per_seq = T;
    a.D = D;
    a.W = W;
    a.cu_seqlens = cu_seqlens;
    a.silu = activation == KDA_ACT_SILU;
    a.weight_f32 = (flags & KDA_FLAG_WEIGHT_F32) != 0;
    if ((rc = check_conv(a, activation)) != KDA_OK) return rc;
    if (B > kMaxElems / (8 * D)) return KDA_ERR_SHAPE;
    // (The filter is read without tokens too, by the threads that write the states.)
    if (!weight || (a.tokens > 0 && (!x || !out))) return KDA_ERR_NULL;
    if (!aligned(x, 2) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(init_state, 16) || !aligned(out, 16) ||
        !aligned(final_state, 16) || !aligned(cu_seqlens, 8))
        return KDA_ERR_ALIGN;
    const int64_t state = B * (W - 1) * D * 2, wb = a.weight_f32 ? 4 : 2;
    const Span so(out, a.tokens * D * 2), sf(final_state, state), si(init_state, state);
    const Span in[] = {Span(x, rows_bytes(a.tokens, ldx, D, 2)), Span(weight, D * W * wb), Span(bias, D * wb),
                       Span(cu_seqlens, 8 * (B + 1))};
    if (meets_any(so, in) || meets_any(sf, in) || so.meets(sf) || so.meets(si) || (final_state != init_state && sf.meets(si)))
        return KDA_ERR_OVERLAP;
    DeviceView d;
    if ((rc = device_view(&d)) != KDA_OK) return rc;
    a.status = d.status;
    const auto stream = static_cast<cudaStream_t>(stream_ptr);
    const bool many = cu_seqlens && B > kMaxSelfChecked, in_place = init_state && init_state == final_state;
    Scratch ws;
    if (!ws.take((many ? 256 : 0) + (in_place ? align256(state) : 0), d.pool, stream)) return KDA_ERR_CUDA;
    if (many) {
        const auto valid = reinterpret_cast<int32_t*>(ws.part(256));
        if ((rc = check_offsets(cu_seqlens, B, a.tokens, d, valid, stream)) != KDA_OK) return rc;
        a.valid = valid;
    }
    if (in_place) {   // one thread ends a sequence while another begins it
        void* copy = ws.part(state);
        if (cudaMemcpyAsync(copy, init_state, static_cast<size_t>(state), cudaMemcpyDeviceToDevice, stream) != cudaSuccess) {
            cudaGetLastError();
            return KDA_ERR_CUDA;
        }
        a.init_state = copy;
    }
    if (launch_conv_prefill(a, d.sms, stream) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    add_launches(1);
    return KDA_OK;
}

extern "C" int kda_conv_decode(const void* x, int64_t ldx, const void* weight, const void* bias, void* state,
                               const int32_t* slots, void* out, int64_t N, int64_t D, int W, int64_t pool,
                               int activation, uint32_t flags, void* stream) {
    reset_launches();
    if (flags & ~KDA_FLAG_WEIGHT_F32) return KDA_ERR_ARG;
    ConvArgs a = {};
    a.x = x;
    a.ldx = ldx;
    a.weight = weight;
    a.bias = bias;
    a.state = state;
    a.slots = slots;
    a.out = out;
    a.N = a.rows = N;
    a.D = D;
    a.W = W;
    a.pool = pool;
    a.silu = activation == KDA_ACT_SILU;
    a.weight_f32 = (flags & KDA_FLAG_WEIGHT_F32) != 0;
    if (N < 0 || N > 0x7fffffffLL || pool < 0) return KDA_ERR_SHAPE;
    int rc = check_conv(a, activation);
    if (rc != KDA_OK) return rc;
    if (pool > kMaxElems / (8 * D) || (!slots && N > pool)) return KDA_ERR_SHAPE;
    if (N > 0) {
        if (!x || !weight || !out || (pool > 0 && !state)) return KDA_ERR_NULL;
        if (!aligned(x, 2) || !aligned(weight, 16) || !aligned(bias, 16) || !aligned(state, 16) || !aligned(out, 16) ||
            !aligned(slots, 4))
            return KDA_ERR_ALIGN;
        const int64_t wb = a.weight_f32 ? 4 : 2;
        const Span so(out, N * D * 2), ss(state, pool * (W - 1) * D * 2);
        const Span in[] = {Span(x, rows_bytes(N, ldx, D, 2)), Span(weight, D * W * wb), Span(bias, D * wb), Span(slots, 4 * N)};
        if (meets_any(so, in) || meets_any(ss, in) || so.meets(ss)) return KDA_ERR_OVERLAP;
    }
    DeviceView d;
    rc = device_view(&d);
    if (rc != KDA_OK || N == 0) return rc;
    a.status = d.status;
    if (launch_conv_decode(a, d.sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    add_launches(1);
    return KDA_OK;
}

extern "C" int kda_ssm_prefill(const void* x, int64_t ldx, const void* dt, int64_t lddt, const float* A, const void* Bm,
                               int64_t ldb, const void* Cm, int64_t ldc, const float* D, const void* z, int64_t ldz,
                               const float* dt_bias, const void* init_state, void* out, void* final_state, int64_t B,
                               int64_t T, int64_t dim, int64_t groups, int64_t nstate, const int64_t* cu_seqlens,
                               uint32_t flags, void* stream_ptr) {
    reset_launches();
    if (flags & ~kSsmFlags) return KDA_ERR_ARG;
    SsmArgs a = {};
    ssm_flags(&a, flags);
    SsmCut cut;
    int64_t tokens = 0;
    // (The sizes' check; the device's plan follows.)
    int rc = plan_ssm(B, T, dim, groups, nstate, cu_seqlens != nullptr, a.state_f32, 1, 0, 0, &tokens, &cut);
    if (rc != KDA_OK) return rc;
    a.x = x;
    a.ldx = ldx;
    a.dt = dt;
    a.lddt = lddt;
    a.A = A;
    a.B = Bm;
    a.ldb = ldb;
    a.C = Cm;
    a.ldc = ldc;
    a.D = D;
    a.z = z;
    a.ldz = ldz;
    a.dt_bias = dt_bias;
    a.init_state = init_state;
    a.out = out;
    a.final_state = final_state;
    a.N = B;
    a.tokens = tokens;
    a.tokens_per_seq = T;
    a.dim = dim;
    a.groups = groups;
    a.nstate = nstate;
    a.cu_seqlens = cu_seqlens;
    if (!ssm_rows_fit(a, tokens)) return KDA_ERR_SHAPE;
    // (The rates are read without tokens too.)
    if (!A) return KDA_ERR_NULL;
    if (!aligned(A, 16) || !aligned(init_state, 16) || !aligned(final_state, 16) || !aligned(cu_seqlens, 8)) return KDA_ERR_ALIGN;
    const int64_t state = B * dim * nstate * (a.state_f32 ? 4 : 2);
    const Span sf(final_state, state), si(init_state, state), cu(cu_seqlens, 8 * (B + 1));
    if ((rc = check_ssm(a, tokens, sf, cu)) != KDA_OK) return rc;
    if ((final_state != init_state && sf.meets(si)) || sf.meets(cu) || (tokens > 0 && Span(out, tokens * dim * 2).meets(si)))
        return KDA_ERR_OVERLAP;
    DeviceView d;
    if ((rc = device_view(&d)) != KDA_OK) return rc;
    a.status = d.status;
    if ((rc = plan_ssm(B, T, dim, groups, nstate, cu_seqlens != nullptr, a.state_f32, d.sms, d.segments, d.seg_chunks, &tokens,
                       &cut)) != KDA_OK)
        return rc;
    a.spans = cut.spans;
    a.spans_per_seq = cut.spans_per_seq;
    a.span_tokens = cut.span_tokens;
    a.tiles = cut.tiles;
    a.tiles_per_group = cut.tiles_per_group;
    const auto stream = static_cast<cudaStream_t>(stream_ptr);
    const bool many = cu_seqlens && B > kMaxSelfChecked, copied = cut.init_bytes > 0 && init_state && init_state == final_state;
    Scratch ws;
    if (!ws.take((many ? 256 : 0) + cut.bytes() + (copied ? align256(state) : 0), d.pool, stream)) return KDA_ERR_CUDA;
    if (many) {
        const auto valid = reinterpret_cast<int32_t*>(ws.part(256));
        if ((rc = check_offsets(cu_seqlens, B, tokens, d, valid, stream)) != KDA_OK) return rc;
        a.valid = valid;
    }
    if (cut.cut()) {
        a.span_states = reinterpret_cast<float*>(ws.part(cut.state_bytes));
        a.span_steps = reinterpret_cast<float*>(ws.part(cut.step_bytes));
    }
    if (cut.relay_bytes) {
        a.relay = reinterpret_cast<int32_t*>(ws.part(cut.relay_bytes));
        if (cudaMemsetAsync(a.relay, 0, static_cast<size_t>(cut.relay_bytes), stream) != cudaSuccess) {
            cudaGetLastError();
            return KDA_ERR_CUDA;
        }
    }
    if (copied) {   // one CTA ends a sequence that another has yet to begin
        void* copy = ws.part(state);
        if (cudaMemcpyAsync(copy, init_state, static_cast<size_t>(state), cudaMemcpyDeviceToDevice, stream) != cudaSuccess) {
            cudaGetLastError();
            return KDA_ERR_CUDA;
        }
        a.init_state = copy;
    }
    int launches = 0;
    const cudaError_t e = launch_ssm_prefill(a, stream, &launches);
    add_launches(launches);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

extern "C" int kda_ssm_decode(const void* x, int64_t ldx, const void* dt, int64_t lddt, const float* A, const void* Bm,
                              int64_t ldb, const void* Cm, int64_t ldc, const float* D, const void* z, int64_t ldz,
                              const float* dt_bias, void* state, const int32_t* slots, void* out, int64_t N, int64_t dim,
                              int64_t groups, int64_t nstate, int64_t pool, uint32_t flags, void* stream) {
    reset_launches();
    if (flags & ~kSsmFlags) return KDA_ERR_ARG;
    if (N < 0 || N > 0x7fffffffLL / 4 || pool < 0 || dim < 1 || dim > kSsmMaxDim || groups < 1 || dim % groups || nstate < 1 ||
        nstate > kSsmMaxState || pool > kMaxElems / (dim * nstate * 4) || (!slots && N > pool))
        return KDA_ERR_SHAPE;
    SsmArgs a = {};
    ssm_flags(&a, flags);
    a.x = x;
    a.ldx = ldx;
    a.dt = dt;
    a.lddt = lddt;
    a.A = A;
    a.B = Bm;
    a.ldb = ldb;
    a.C = Cm;
    a.ldc = ldc;
    a.D = D;
    a.z = z;
    a.ldz = ldz;
    a.dt_bias = dt_bias;
    a.state = state;
    a.slots = slots;
    a.out = out;
    a.N = a.tokens = N;
    a.dim = dim;
    a.groups = groups;
    a.nstate = nstate;
    a.pool = pool;
    if (!ssm_rows_fit(a, N)) return KDA_ERR_SHAPE;
    if (N > 0 && pool > 0 && !state) return KDA_ERR_NULL;
    if (!aligned(state, 16) || !aligned(slots, 4)) return KDA_ERR_ALIGN;
    int rc = check_ssm(a, N, Span(state, pool * dim * nstate * (a.state_f32 ? 4 : 2)), Span(slots, 4 * N));
    if (rc != KDA_OK) return rc;
    DeviceView d;
    rc = device_view(&d);
    if (rc != KDA_OK || N == 0) return rc;
    a.status = d.status;
    if (launch_ssm_decode(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return KDA_ERR_CUDA;
    }
    add_launches(1);
    return KDA_OK;
}

extern "C" int kda_ssm_plan_segments(int64_t B, int64_t T, int64_t dim, int64_t groups, int64_t nstate, int packed,
                                     int64_t* segs) {
    if (!segs) return KDA_ERR_NULL;
    SsmCut cut;
    int64_t tokens;
    int rc = plan_ssm(B, T, dim, groups, nstate, packed != 0, true, 1, 0, 0, &tokens, &cut);
    if (rc != KDA_OK) return rc;
    DeviceView d;
    if ((rc = device_view(&d)) != KDA_OK) return rc;
    rc = plan_ssm(B, T, dim, groups, nstate, packed != 0, true, d.sms, d.segments, d.seg_chunks, &tokens, &cut);
    if (rc == KDA_OK) *segs = cut.cut() && !cut.relay_bytes ? cut.spans_per_seq : 0;
    return rc;
}

extern "C" int kda_ssm_workspace_bytes(int64_t B, int64_t T, int64_t dim, int64_t groups, int64_t nstate, int packed,
                                       int64_t* bytes) {
    if (!bytes) return KDA_ERR_NULL;
    // As planned on the current device (on a 152-SM device when there is none).
    DeviceView d;
    if (device_view(&d) != KDA_OK) {
        d.sms = 152;
        segment_settings(&d.segments, &d.seg_chunks);
    }
    SsmCut cut;
    int64_t tokens;
    const int rc = plan_ssm(B, T, dim, groups, nstate, packed != 0, true, d.sms, d.segments, d.seg_chunks, &tokens, &cut);
    if (rc == KDA_OK) *bytes = (packed && B > kMaxSelfChecked ? 256 : 0) + cut.bytes() + align256(cut.init_bytes);
    return rc;
}
