/*
 * kda.h -- C ABI of the GB300 (sm_103a) Kimi Delta Attention prefill library.
 *
 * The operation is the chunkwise KDA forward pass of "FlashKDA column split"
 * (mainlymatmul.com), section 1: for every sequence and head, with the state S
 * a 128 x 128 matrix (rows = value channels, columns = key channels), per
 * token t
 *     S <- S Diag(exp(g_t));  u_t = beta_t (v_t - S khat_t);
 *     S <- S + u_t khat_t^T;  o_t = s S qhat_t,   s = 1/sqrt(128),
 * evaluated 16 tokens at a time through the chunk quantities K^start, Q^start,
 * K^end, D_{0:15}, A^kk = (I + R)^{-1} and A^qk of that section.  q and k are
 * L2-normalised inside the operation, xhat = x / sqrt(sum x^2 + 1e-6)
 * (flashinfer kda_prefill, "Optimized Blackwell prefill subset",
 * use_qk_l2norm_in_kernel).  The log-decay g must lie in [-5, 0] ("K3's KDA
 * precision problem", introduction: the lower bound keeps exp(+-G) of a
 * 16-token chunk inside the FP32/BF16 range).
 *
 * Every pointer argument is a DEVICE pointer on the current CUDA device unless
 * stated otherwise.  The caller owns every buffer; the library keeps no
 * pointer after a call returns.  Calls are asynchronous on `stream` (a
 * cudaStream_t; NULL is the legacy default stream): the host never reads
 * device data and never synchronises.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
#define KDA_OK 0
#define KDA_ERR_NULL (-1)      /* a required pointer is NULL */
#define KDA_ERR_SHAPE (-2)     /* B, T or H out of range, or sizes overflow */
#define KDA_ERR_ALIGN (-3)     /* a pointer is not suitably aligned */
#define KDA_ERR_OVERLAP (-4)   /* an output overlaps an input or another output */
#define KDA_ERR_DEVICE (-5)    /* no CUDA device, or not compute capability 10.3 */
#define KDA_ERR_CUDA (-6)      /* a CUDA call (allocation, launch) failed */
#define KDA_ERR_ARG (-7)       /* an option value is out of range */
#define KDA_ERR_SCRATCH (-8)   /* shape too large for kda_prefill_noalloc's fixed scratch */
#define KDA_ERR_SEQLENS (-9)   /* kda_prefill_host: the host cu_seqlens break their contract */

/* Flags of kda_prefill_ex. */
#define KDA_FLAG_BETA_LOGIT 1u /* beta holds logits; the operation uses sigmoid(beta) */
/* Flags of the operators around the prefill (each lists the ones it takes). */
#define KDA_FLAG_STATE_F32 2u     /* states are FP32 (BF16 without it) */
#define KDA_FLAG_G_PER_HEAD 4u    /* g is [H], one constant decay for each head */
#define KDA_FLAG_WEIGHT_F32 8u    /* norm weights (and a channel gate) are FP32 (BF16 without it) */
#define KDA_FLAG_GATE_FIRST 16u   /* the gate multiplies before the norm */
#define KDA_FLAG_RESIDUAL_F32 32u /* the residual stream is FP32 (BF16 without it) */
#define KDA_FLAG_DT_F32 64u       /* step sizes are FP32 (BF16 without it) */
#define KDA_FLAG_BC_F32 128u      /* the scan's B and C are FP32 (BF16 without it) */
#define KDA_FLAG_DT_SOFTPLUS 256u /* step sizes pass through a softplus */

/* Activations of kda_gated_norm. */
#define KDA_ACT_NONE 0
#define KDA_ACT_SIGMOID 1
#define KDA_ACT_SILU 2

/* Device-side status bits, reported by kda_device_status(). */
#define KDA_DEV_BAD_SEQLENS 1  /* cu_seqlens broke its contract; out/final_state untouched */
#define KDA_DEV_PIPE_TIMEOUT 2 /* an internal pipeline wait hit its bound; results incomplete */
#define KDA_DEV_BAD_CHECKPOINTS 4 /* a checkpoint had no valid row in checkpoint_cu_starts; skipped */
#define KDA_DEV_BAD_SLOTS 8    /* a state slot lay outside the pool; that row's state untouched, out zero */

/*
 * KDA prefill, fixed or packed variable-length layout.
 *
 * Fixed layout (cu_seqlens == NULL): N = B sequences of T tokens each.
 *   q, k, v, out : BF16 [B, T, H, 128], contiguous (head dim innermost)
 *   g            : FP32 [B, T, H, 128], natural-log decay, alpha = exp(g), g in [-5, 0]
 *   beta         : BF16 [B, T, H], beta in [0, 1] (already passed through a sigmoid)
 * Packed layout (cu_seqlens != NULL): tensors are [1, T, H, ...] with T the
 *   total number of tokens, and B is read as the number of sequences N.
 *   cu_seqlens is a device int64 array of N + 1 offsets with cu[0] == 0,
 *   cu[n] <= cu[n+1] and cu[N] == T (flashinfer kda_prefill, "Optimized
 *   Blackwell prefill subset").  Equal neighbours are empty sequences, whose
 *   final state equals their initial state.  The offsets are validated on the
 *   device; a violation leaves out and final_state untouched and sets
 *   KDA_DEV_BAD_SEQLENS (see kda_device_status).
 * init_state  : BF16 [N, H, 128, 128] (value rows x key columns) or NULL for zeros.
 * final_state : BF16 [N, H, 128, 128] or NULL (not written).  final_state may be
 *   the same pointer as init_state (in-place update, as in flashinfer
 *   kda_prefill "State and graph semantics"); any other overlap is refused.
 *
 * Alignment: q, k, v, g, out, init_state and final_state 16 bytes; beta 2
 * bytes; cu_seqlens 8 bytes.  out must not overlap any input.
 * Limits: B >= 1, T >= 0, H >= 1, fewer than 2^31 tokens in total.  With no tokens (T = 0) only final_state is
 * written (a copy of init_state, or zeros) and q, k, v, g, beta and out may be NULL.
 *
 * Scratch: the call takes a workspace of about 13.5 KB per (chunk, head) from
 * a stream-ordered memory pool owned by the library (cudaMallocFromPoolAsync /
 * cudaFreeAsync on `stream`), so it allocates and frees in stream order.
 *
 * Returns KDA_OK or a negative KDA_ERR_* code; on an error nothing is launched.
 */
int kda_prefill(const void* q, const void* k, const void* v, const float* g, const void* beta,
                const void* init_state, void* out, void* final_state, int64_t B, int64_t T,
                int64_t H, const int64_t* cu_seqlens, void* stream);

/*
 * kda_prefill on HOST buffers: the same operation, arguments and layouts as
 * kda_prefill, except that q, k, v, g, beta, init_state, out, final_state and
 * cu_seqlens are HOST pointers (cu_seqlens: host int64 [B + 1] or NULL).  The
 * library copies the inputs to the device, runs the device path and copies
 * out and final_state back, overlapping the copies with the computation: the
 * batch is cut into at most 8 pieces, each a contiguous range of every tensor
 * (token ranges of whole chunks for a single fixed-length sequence, groups of
 * batch rows, or groups of whole packed sequences); while the caller's stream
 * computes one piece, a library stream copies the next one in and another
 * copies the previous piece's outputs back.  A single sequence cut into token
 * ranges carries its state from piece to piece as a BF16 state, as two
 * kda_prefill calls chained through final_state -> init_state would, so its
 * results can differ from one device call by that rounding (within the
 * operation's tolerance); batches cut between sequences give each sequence
 * the results of a device call on its group.
 *
 * Host memory: page-locked buffers (cudaHostAlloc, cudaHostRegister, or a
 * pinned framework tensor) let the copies run asynchronously and overlap;
 * pageable buffers are accepted, but the driver then stages each copy and the
 * overlap is lost (and a CUDA-graph capture of the call fails).
 * Asynchronous on `stream`: the call returns once everything is enqueued; the
 * inputs must stay unchanged and the outputs unread until `stream` has passed
 * the call.  Device memory: images of every tensor, taken from the library's
 * stream-ordered pool for the duration of the call, plus kda_prefill's
 * workspace per piece.  The copy streams are the library's, one pair per
 * device: calls from several host threads enqueue one after another, and
 * while a CUDA-graph capture that contains a kda_prefill_host call is open,
 * those streams belong to it: no other thread may call kda_prefill_host on
 * the device until the capture ends.
 *
 * Returns KDA_OK, kda_prefill's argument codes (shape, NULL, overlap of the
 * host ranges; no alignment rule), KDA_ERR_SEQLENS when the host cu_seqlens
 * break the contract of kda_prefill (nothing is enqueued then), or
 * KDA_ERR_CUDA when a copy or launch could not be enqueued (the copies already
 * enqueued are joined back into `stream` before the call returns).
 */
int kda_prefill_host(const void* q, const void* k, const void* v, const float* g, const void* beta,
                     const void* init_state, void* out, void* final_state, int64_t B, int64_t T,
                     int64_t H, const int64_t* cu_seqlens, void* stream);

/*
 * How many pieces kda_prefill_host cuts a call into: 0 (the default) chooses
 * automatically, 1 .. 8 sets the number (fewer when the batch has fewer
 * chunks, rows or sequences).  Process-wide, for comparing the choices;
 * KDA_ERR_ARG for other values.
 */
int kda_set_host_pieces(int n);

/*
 * Number of kernels (HOST out) that the last kda_prefill, kda_prefill_checkpointed
 * or kda_prefill_host call, or call of the operators at the end of this header, made on this host
 * thread enqueued (memsets and copies
 * are not counted; after a call that returned an error the count may include
 * the launch that failed).
 */
int kda_last_call_launches(int64_t* n);

/* Human-readable text for a KDA_* status code (static storage). */
const char* kda_error_string(int status);

/*
 * Synchronise `stream`, then read and clear this device's KDA_DEV_* status
 * bits into *status (a HOST pointer).  The bits accumulate over every call on
 * the device since the last read.
 */
int kda_device_status(void* stream, int* status);

/*
 * Number of CTAs that share one (sequence, head) in the recurrence: each owns
 * 128 / nsplit value columns (value columns are independent recurrences,
 * "FlashKDA column split" section 3.1).  nsplit is one of 1, 2, 4, 8, 16, or 0
 * for the automatic choice (the largest split whose grid fits the SM count).
 * Process-wide setting; returns KDA_ERR_ARG for other values.
 */
int kda_set_split(int nsplit);

/*
 * Recurrence engine.  0 (default) and 1: the column-split kernel (warp-level
 * m16n8k16 MMAs, state in registers, `nsplit` CTAs per head).  Engine 0 gives
 * each warp 32 value columns at nsplit 1, 8 columns at nsplit 2, and at nsplit
 * 4, 8 and 16 splits each 8-column group's 128 keys over a pair of warps
 * (their partial sums over keys are added in a fixed order, so results agree
 * with the other variants to rounding, not bit for bit).  Engine 1 gives each
 * warp 8 columns and all 128 keys at every split.  2: the tcgen05
 * kernel (one CTA per (sequence, head); the value rows are the MMA's M = 128;
 * the FP32 state, its BF16 operand copy and every accumulator live in tensor
 * memory, the packets are read by the tensor cores from shared memory; the
 * split setting is ignored).
 * Process-wide; returns KDA_ERR_ARG for other values.
 */
int kda_set_engine(int engine);

/*
 * kda_prefill plus native state checkpoints ("flashinfer kda_prefill", Native
 * checkpoints): the recurrent state before each interval of
 * checkpoint_every_n_tokens tokens (a positive multiple of 16).  Every
 * non-empty sequence n contributes ceil(len_n / interval) rows: its initial
 * state (init_state, or zeros), then the states after one, two, ... intervals
 * that strictly precede its end; empty sequences contribute none.
 *
 *   state_checkpoints     BF16 [checkpoint_rows, H, 128 (value), 128 (key)], DEVICE,
 *                         written; 16-byte aligned; must not overlap any other
 *                         argument.
 *   checkpoint_cu_starts  int64 [N + 1], DEVICE, read: sequence n's rows are
 *                         checkpoint_cu_starts[n] ..; N = B (fixed layout) or the
 *                         number of sequences (packed).  Caller-provided and not
 *                         scanned at launch: a checkpoint whose row falls outside
 *                         [cu_starts[n], cu_starts[n + 1]) or [0, checkpoint_rows)
 *                         is not written and sets KDA_DEV_BAD_CHECKPOINTS.
 *
 * Everything else, including results and errors, is as kda_prefill (a call
 * that takes the segmented scan, kda_set_segments, writes the checkpoints
 * from its last pass: those at segment starts are the segments' BF16
 * incoming states); in addition KDA_ERR_ARG for an interval that is not a
 * positive multiple of 16 or negative checkpoint_rows, KDA_ERR_NULL for NULL
 * checkpoint pointers.
 * Under engine 2 (kda_set_engine) such calls run on the column-split kernels.
 */
int kda_prefill_checkpointed(const void* q, const void* k, const void* v, const float* g,
                             const void* beta, const void* init_state, void* out,
                             void* final_state, int64_t B, int64_t T, int64_t H,
                             const int64_t* cu_seqlens, int64_t checkpoint_every_n_tokens,
                             void* state_checkpoints, const int64_t* checkpoint_cu_starts,
                             int64_t checkpoint_rows, void* stream);

/*
 * kda_prefill with options: the same operation, arguments, layouts, results
 * and errors, plus
 *   flags  0, or KDA_FLAG_BETA_LOGIT: beta (BF16 [B, T, H]) holds logits x and
 *          the operation uses beta = sigmoid(x) = 1 / (1 + exp(-x)), formed in
 *          FP32 inside the chunk preparation ("flashinfer kda_prefill",
 *          "Optimized Blackwell prefill subset": beta_is_logit=True).  Other
 *          bits: KDA_ERR_ARG.
 *   checkpoint_every_n_tokens, state_checkpoints, checkpoint_cu_starts,
 *   checkpoint_rows: native checkpoints exactly as kda_prefill_checkpointed;
 *          state_checkpoints NULL for none (the other three are then ignored).
 */
int kda_prefill_ex(const void* q, const void* k, const void* v, const float* g, const void* beta,
                   const void* init_state, void* out, void* final_state, int64_t B, int64_t T,
                   int64_t H, const int64_t* cu_seqlens, uint32_t flags,
                   int64_t checkpoint_every_n_tokens, void* state_checkpoints,
                   const int64_t* checkpoint_cu_starts, int64_t checkpoint_rows, void* stream);

/*
 * Whether kda_prefill may run preparation and recurrence as one cooperative
 * launch (1, the default) or always as two kernels (0).  One launch is used
 * under engine 0 in two forms, each packet behind a ready flag in the
 * workspace: (a) fixed-length batches (cu_seqlens NULL) with few heads, whose
 * recurrence takes a split of 8 or 16 and leaves at least 16 SMs free: those
 * SMs prepare packets while the recurrence consumes them; (b) many heads, one
 * recurrence CTA per (sequence, head) and 3 N H <= 2 x the SM count, at
 * least 64 chunks per sequence (packed: on average), never with checkpoints:
 * one CTA per SM, the first N * H of them each run a head's recurrence and
 * prepare packets on two warp pairs, the others prepare on eight.  The
 * preparation walks the chunks in the order the recurrences consume them:
 * chunk index first across all heads (fixed layout), or, for a packed batch,
 * by each chunk's position relative to its sequence's length (a small kernel
 * ranks the chunks on the device after the offsets are checked), so that
 * every sequence's recurrence gets its packets at the pace its length needs.
 * The results are bit for bit those of the two-kernel path.
 * Process-wide; returns KDA_ERR_ARG for other values.
 */
int kda_set_fusion(int on);

/*
 * Whether kda_prefill would run a call of this shape as one launch on the
 * current device under the current settings (HOST out: 1 or 0).  Errors as
 * kda_prefill's shape checks, or KDA_ERR_DEVICE / KDA_ERR_CUDA without a
 * usable device.
 */
int kda_plan_fused(int64_t B, int64_t T, int64_t H, int packed, int* fused);

/*
 * For a packed call of n_seqs sequences (T tokens in all) and H heads: how
 * many of its longest sequences kda_prefill runs at split 2 in a second,
 * concurrent recurrence launch on a library-owned stream (HOST out; 0 when
 * the call uses a single recurrence launch or the many-head one-launch form).
 * That happens under engine 0 with the automatic split when the
 * one-CTA-per-head grid leaves SMs free and n_seqs <= 1024; the results are
 * bitwise those of split 1.
 */
int kda_plan_long_split(int64_t n_seqs, int64_t T, int64_t H, int64_t* k);

/*
 * Whether kda_prefill may use the segmented scan over chunks (1, the default)
 * or always runs each (sequence, head) as one serial chain of chunk steps (0).
 * The chunkwise state update is affine in the incoming state, so over a run
 * of chunks it is S -> S F + Z (the chunk equations of "FlashKDA column
 * split", section 1: S_{c+1} = S_c D_{0:15} + U_c K^end_c with
 * U_c = (V_c - S_c K^start_c) B_c (A^kk_c)^T affine in S_c).  When there
 * are too few (sequence, head) chains to fill the GPU (engine 0, automatic
 * split; fixed or packed layout; with or without checkpoints, which the last
 * pass writes), each sequence is cut into
 * segments: one launch forms every segment's F and Z, a short chain over the
 * segments forms each segment's incoming state, and one launch reruns every
 * segment from its incoming state and writes O.  The results agree with the
 * serial chain to rounding (the incoming states are rounded to BF16), not bit
 * for bit.  seg_chunks 0 lets a cost estimate decide whether and how to cut;
 * seg_chunks > 0 cuts every eligible call into segments of that many chunks
 * (for tests).  Process-wide; returns KDA_ERR_ARG for on not 0 or 1 or
 * seg_chunks negative or above 2^26.
 */
int kda_set_segments(int on, int64_t seg_chunks);

/*
 * Segments kda_prefill would use for a call of this shape on the current
 * device under the current settings (HOST out; 0: no segmented scan): per
 * sequence for the fixed layout; for the packed layout a bound on all
 * segments (the cut itself is made on the device from cu_seqlens).  Errors as
 * kda_plan_fused.
 */
int kda_plan_segments(int64_t B, int64_t T, int64_t H, int packed, int64_t* segs);

/* The split the automatic rule picks on the current device for N*H units (HOST out). */
int kda_auto_split(int64_t n_seqs, int64_t H, int* nsplit);

/*
 * Bytes of scratch kda_prefill takes for a given shape at most (HOST out);
 * `packed` is nonzero for the packed layout.  The ready flags of a fused
 * launch (kda_set_fusion) are counted whether or not a fixed-length call
 * fuses, and for a packed call, with its chunk order (4 bytes a chunk), when
 * the current device (a 152-SM one when there is none) would run it as the
 * many-head one-launch form; the segmented scan's three state buffers
 * (kda_set_segments) when that device would use it.
 */
int kda_workspace_bytes(int64_t B, int64_t T, int64_t H, int packed, int64_t* bytes);

/*
 * Test hook: run only the chunk preparation and write the per-(chunk, head)
 * packets into `packets` (device, capacity `packets_bytes`).  Packet
 * (chunk, head) starts at byte (chunk * H + head) * kda_packet_bytes(), with
 * chunks numbered sequence by sequence.  The packet layout is documented in
 * kda_common.cuh.  Arguments as for kda_prefill.
 */
int kda_prep_only(const void* q, const void* k, const float* g, const void* beta, int64_t B,
                  int64_t T, int64_t H, const int64_t* cu_seqlens, void* packets,
                  int64_t packets_bytes, void* stream);

/* Size in bytes of one (chunk, head) packet. */
int64_t kda_packet_bytes(void);

/*
 * Per-kernel timing for benchmarks.  kda_profile_begin(max_calls) creates
 * 5 * max_calls CUDA events on the current device; each of the next
 * max_calls kda_prefill calls then records, on its own stream, one event
 * before its preparation kernels, one after them, one after the transition
 * pass and one after the segment chain of a segmented scan (see
 * kda_set_segments; recorded right after the second otherwise), and one after
 * the recurrence.  When a call runs as one launch (see kda_set_fusion), the
 * first interval holds only the reset of the ready flags and the last the
 * fused kernel.  kda_profile_end synchronises those events, writes the summed
 * preparation time and recurrence time (the last three intervals) in
 * milliseconds and the number of calls timed (HOST pointers), and destroys
 * the events; kda_profile_end_detail does the same but writes the four
 * summed intervals to intervals_ms[0..3].  Process-wide; begin while active
 * returns KDA_ERR_ARG.
 */
int kda_profile_begin(int max_calls);
int kda_profile_end(double* prep_ms, double* recurrence_ms, int* calls);
int kda_profile_end_detail(double* intervals_ms, int* calls);

/*
 * Measurement hook: nanoseconds per step of the shortest dependent chain of
 * one chunk step on the current device (HOST out), for the critical-path
 * bound of a serial walk over the chunks ("FlashKDA column split" section 1:
 * chunk c + 1 needs chunk c's state).  One warp runs, 4,096 times, U^T = K'
 * S^T over 128 keys (two interleaved MMA accumulators and an add), the FP16
 * conversion and transpose of U^T, S^T <- D S^T + (K^end)^T U^T and the BF16
 * conversion and transpose of the new state, with operands in registers.
 * Synchronises the device; not for use on a hot path.  KDA_ERR_DEVICE
 * without a compute capability 10.3 device, KDA_ERR_CUDA on a CUDA error.
 */
int kda_chain_step_ns(double* ns);

/*
 * kda_prefill without any allocation.  The pages describe no such entry
 * point; it exists for callers that cannot let a library allocate device
 * memory: code running under an allocator that owns all of the GPU's memory
 * (a serving engine that carves HBM up front, a framework whose caching
 * allocator must account for every byte), callers that forbid driver
 * allocations on their hot path, or processes that have already handed out
 * nearly all HBM.
 *
 * Arguments, alignment and overlap rules and error codes are those of
 * kda_prefill; the caller still passes every input and output.  It runs the
 * plain plan -- the preparation kernel, then one recurrence launch at the
 * split kda_prefill would pick (kda_set_split and kda_set_engine apply) --
 * and never the one-launch form, the segmented scan or the longest-first
 * scheduling of packed sequences, so its results agree with kda_prefill's
 * within the operation's tolerance, not bit for bit.  The
 * scratch kda_prefill would take from its pool lives instead in one fixed
 * device array of kda_noalloc_scratch_bytes() bytes (48 MiB) inside this
 * library, which every GPU that loads the library holds until the process
 * exits.  A shape whose scratch does not fit -- about 13.5 KB per (chunk of
 * 16 tokens, head), plus (N + 1) * 8 + 512 bytes for packed input -- is
 * refused with KDA_ERR_SCRATCH before anything is launched.  No call
 * allocates or frees device or host memory.
 *
 * The first call on a device, with that device current, looks up the
 * array's device address (cudaGetSymbolAddress) once; make that first call
 * before any stream capture.  Every call on a device shares the one array
 * and leaves its contents behind; nothing in it has to start at zero.  Calls
 * whose kernels overlap on the GPU (on different streams, or from different
 * host threads) race on that array and corrupt each other's results: order
 * them on one stream, or with events.
 */
int kda_prefill_noalloc(const void* q, const void* k, const void* v, const float* g,
                        const void* beta, const void* init_state, void* out, void* final_state,
                        int64_t B, int64_t T, int64_t H, const int64_t* cu_seqlens, void* stream);

/* Size in bytes of kda_prefill_noalloc's fixed scratch array. */
int64_t kda_noalloc_scratch_bytes(void);

/* ------------------------------------------------------------------------
 * Operators around the prefill.  As above: DEVICE pointers, asynchronous on
 * `stream`, no host synchronisation, CUDA-graph capturable, contiguous
 * tensors, KDA_OK or a negative KDA_ERR_* code with nothing launched
 * (KDA_ERR_ARG for a flag that the call does not take).
 * ------------------------------------------------------------------------ */

/*
 * Linear attention with one decay per head and token, over whole prompts:
 *     S_t = exp(g_t) S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t
 * with S a 128 x 128 matrix (value rows x key columns) per sequence and head.
 * q and k are taken as they are (no normalisation).
 *
 *   q, k        : BF16 [B, T, Hk, 128]; head h uses key head h / (H / Hk), Hk divides H
 *   v, out      : BF16 [B, T, H, 128]
 *   g           : FP32 [B, T, H], natural-log decay, g <= 0 (-inf forgets the state);
 *                 with KDA_FLAG_G_PER_HEAD FP32 [H], the same for every token
 *   init_state  : [N, H, 128, 128] or NULL for zeros; BF16, or FP32 with KDA_FLAG_STATE_F32
 *   final_state : the same type, or NULL (not written); may be init_state
 * Fixed and packed layouts, cu_seqlens, empty sequences, alignment, overlap
 * rules, limits and the T = 0 rule are those of kda_prefill (g: 4 bytes).
 * The state is held in FP32 throughout (final states are off by 4e-7 of their
 * norm); a NaN or an infinity in a token reaches no earlier token and no other
 * sequence.  On the way to out, the decayed scores (q . k) exp(..) and a copy of
 * the state before each 128 tokens are operands of the tensor cores, rounded to
 * BF16 once each: out is off by 2.4e-3 of its norm, where its own rounding alone
 * is 1.7e-3.  Range: out is formed with a factor of up to 2^48 that its token's
 * decay then takes away, so where the tokens of a chunk of 128 decay, values of
 * out / scale above 2^79 (6e23) may come out infinite.
 * When there are too few (sequence, head) chains to fill the GPU, the tokens
 * are cut into spans of whole 128-token chunks: one launch forms the state each
 * span adds, one chains them, and one forms the outputs from the spans'
 * incoming states.  In the fixed layout each sequence is cut into equal
 * segments.  A packed batch's lengths are known on the device alone, and a
 * launch there decides: its sequences' chunks, one after the other, are cut into
 * one span an SM (and head) where that is sooner done than its longest sequence;
 * else, when there are more (sequence, head) units than SMs, the longest
 * sequences go first.  kda_set_segments governs this too (off: no cut; a forced
 * length is rounded up to whole 128-token chunks).  Equal calls give equal bits.
 * Scratch comes from the library's stream-ordered pool: with a cut, an FP32 state
 * for each span and head, and copies of the initial states where final_state
 * is init_state.
 */
int kda_la_prefill(const void* q, const void* k, const void* v, const float* g,
                   const void* init_state, void* out, void* final_state, int64_t B, int64_t T,
                   int64_t H, int64_t Hk, const int64_t* cu_seqlens, float scale, uint32_t flags,
                   void* stream);

/*
 * One token per sequence of the same operation, on a pool of states:
 *   q, k [N, Hk, 128], v, out [N, H, 128] BF16; g FP32 [N, H] (or [H]);
 *   state : [pool, H, 128, 128], BF16 or FP32 as above, updated in place
 *   slots : int32 [N], the pool row of each sequence, no row twice; negative:
 *           padding (out row zero, no state touched).  NULL: row n is slot n (N <= pool).
 * A slot >= pool sets KDA_DEV_BAD_SLOTS and is treated as padding.  N = 0 does
 * nothing.  Alignment: q, k, v, out, state 16 bytes, g and slots 4.
 */
int kda_la_decode(const void* q, const void* k, const void* v, const float* g, void* state,
                  const int32_t* slots, void* out, int64_t N, int64_t H, int64_t Hk, int64_t pool,
                  float scale, uint32_t flags, void* stream);

/*
 * One token per sequence of kda_prefill's operation (q and k L2-normalised
 * inside, scale 1/sqrt(128)), on a pool of states: q, k, v, out BF16
 * [N, H, 128], g FP32 [N, H, 128], beta BF16 [N, H] (logits with
 * KDA_FLAG_BETA_LOGIT); state, slots and their errors as kda_la_decode
 * (beta 2 bytes, g 16 bytes aligned).
 */
int kda_decode(const void* q, const void* k, const void* v, const float* g, const void* beta,
               void* state, const int32_t* slots, void* out, int64_t N, int64_t H, int64_t pool,
               uint32_t flags, void* stream);

/*
 * The norm after a mixer with its gate, for each row of 128 channels (a token's head):
 *     y = x / sqrt(mean(x^2) + eps) * weight * act(gate),
 * or, with KDA_FLAG_GATE_FIRST, the norm of x act(gate) times weight.
 *   x, gate, out : BF16 [rows, 128]; weight: [128], BF16 or FP32 (KDA_FLAG_WEIGHT_F32)
 *   activation   : KDA_ACT_NONE (gate is not read and may be NULL), KDA_ACT_SIGMOID
 *                  or KDA_ACT_SILU.  out may be x or gate.  eps >= 0.
 */
int kda_gated_norm(const void* x, const void* weight, const void* gate, void* out, int64_t rows,
                   int activation, float eps, uint32_t flags, void* stream);

/*
 * Between two blocks: the norm after a block, its gate and residual scale,
 * the residual sum, and the norm before the next block, for each row:
 *     u = x                                  (post_weight NULL), else
 *     u = x / sqrt(mean(x^2) + eps) * post_weight
 *     r' = residual + scale * gate * u       (gate NULL: 1)
 *     out = r' / sqrt(mean(r'^2) + eps) * weight      (r' before its rounding)
 *   x, out                 : BF16 [rows, dim], 1 <= dim <= 32768
 *   residual, residual_out : [rows, dim], BF16 or FP32 (KDA_FLAG_RESIDUAL_F32)
 *   weight, post_weight, gate : [dim], BF16 or FP32 (KDA_FLAG_WEIGHT_F32)
 * residual_out may be residual, and out may be x; other overlaps are refused.
 * Alignment: 16 bytes for every tensor.
 */
int kda_residual_norm(const void* x, const void* residual, const void* weight,
                      const void* post_weight, const void* gate, void* out, void* residual_out,
                      int64_t rows, int64_t dim, float scale, float eps, uint32_t flags,
                      void* stream);

/*
 * Segments per sequence kda_la_prefill would use for a call of this shape
 * (packed: the most spans it may cut the batch into; 0: no cut), and the bytes
 * of scratch it takes at most (HOST out).  As kda_plan_segments and
 * kda_workspace_bytes.
 */
int kda_la_plan_segments(int64_t B, int64_t T, int64_t H, int packed, int64_t* segs);
int kda_la_workspace_bytes(int64_t B, int64_t T, int64_t H, int packed, int64_t* bytes);

/*
 * The short causal convolution in front of a mixer, for each channel on its own
 * and over whole prompts:
 *     y[t][d] = act(bias[d] + sum_{j < W} weight[d][j] x[t - W + 1 + j][d])
 * where the W - 1 rows before a sequence's first are its initial state.
 *
 *   x           : BF16, a row of D channels for each token, rows ldx elements apart
 *                 (ldx >= D: a part of a wider projection's output; 2-byte aligned).
 *                 Fixed layout: the B sequences' rows one after the other, T each
 *   out         : BF16 [tokens, D], contiguous
 *   weight      : [D, W], W = 2 .. 4; bias: [D] or NULL; BF16, or FP32 (KDA_FLAG_WEIGHT_F32)
 *   init_state  : BF16 [N, W - 1, D], oldest first, or NULL for zeros
 *   final_state : BF16 [N, W - 1, D] or NULL (not written): the last W - 1 inputs,
 *                 the initial state's among them where a sequence is shorter; may
 *                 be init_state (then the call takes a copy of it as scratch)
 *   activation  : KDA_ACT_NONE or KDA_ACT_SILU
 * Packed layout, cu_seqlens, empty sequences, the T = 0 rule (weight is still
 * needed) and the limit on tokens are those of kda_prefill.  Alignment: 16 bytes
 * but for x and cu_seqlens (8).  out may overlap no input; it and final_state no
 * input and not each other.  FP32 inside, one rounding of out.  Rows and
 * channels in multiples of 4 (ldx, D, and x on 8 bytes) are read fastest.
 */
int kda_conv_prefill(const void* x, int64_t ldx, const void* weight, const void* bias,
                     const void* init_state, void* out, void* final_state, int64_t B, int64_t T,
                     int64_t D, int W, const int64_t* cu_seqlens, int activation, uint32_t flags,
                     void* stream);

/*
 * One token per sequence of the same operation, on a pool of states: x [N, D]
 * (rows ldx apart), out [N, D], state BF16 [pool, W - 1, D], updated in place
 * (its rows move up by one and x becomes the last); slots as kda_la_decode.
 */
int kda_conv_decode(const void* x, int64_t ldx, const void* weight, const void* bias, void* state,
                    const int32_t* slots, void* out, int64_t N, int64_t D, int W, int64_t pool,
                    int activation, uint32_t flags, void* stream);

/*
 * The selective state space scan over whole prompts: a linear recurrence whose
 * decay differs in every channel d and state n = 0 .. nstate - 1,
 *     s = softplus(dt[t][d] + dt_bias[d])        (without KDA_FLAG_DT_SOFTPLUS: the sum)
 *     h[d][n] <- exp(s A[d][n]) h[d][n] + s x[t][d] B[t][g][n]
 *     y = sum_n C[t][g][n] h[d][n] + D[d] x[t][d],   out[t][d] = y silu(z[t][d])
 * with g = d / (dim / groups), the channel's group.
 *
 *   x, z        : BF16, a row of dim channels for each token; z may be NULL (no gate)
 *   dt          : BF16 or FP32 (KDA_FLAG_DT_F32), a row of dim for each token
 *   Bm, Cm      : BF16 or FP32 (KDA_FLAG_BC_F32), a row of [groups, nstate] for each token
 *   ldx, lddt, ldb, ldc, ldz : elements between rows, at least a row's width
 *   A           : FP32 [dim, nstate], contiguous, below infinity (minus infinity: a state
 *                 that any step above 1e-36 clears); D, dt_bias: FP32 [dim] or NULL
 *   out         : BF16 [tokens, dim], contiguous
 *   init_state  : [N, dim, nstate] or NULL for zeros; BF16, or FP32 with KDA_FLAG_STATE_F32
 *   final_state : the same type, or NULL (not written); may be init_state
 *   nstate      : 1 .. 64 (16, 32 and 64 waste nothing); dim below 2^24; groups divides dim
 * Fixed and packed layouts, cu_seqlens, empty sequences, the T = 0 rule (A is
 * still needed) and the limit on tokens are those of kda_prefill.  Alignment: A, out
 * and the states 16 bytes, cu_seqlens 8, the rest an element's size (rows on 8
 * bytes, dt, B and C in FP32 on 16, 32 channels or more to a group in multiples of 4, and
 * nstate a multiple of 4 run fastest).
 * out and final_state may overlap no input and not each other.
 * The states and all sums are FP32, and out is rounded once.  The exponential's mean error
 * (6e-9 to 2.2e-8 of a state a token) is made up for by the 32 tokens.  A NaN or an infinity in a token reaches no earlier token, no other
 * channel (but through B and C, its group's) and no other sequence.
 * When there are too few channels to fill the GPU the tokens are cut into
 * spans: one launch forms the state each span ends with, one the outputs from
 * what the spans before leave.  kda_set_segments governs this (off: no cut; a
 * forced length is rounded up to whole 32 tokens).  Where there are more than fill
 * it evenly, spans may run one after the other, which changes no bit, whether cuts are on or
 * off; a forced length takes their place.  Equal calls give equal bits.  Scratch comes from the library's
 * stream-ordered pool: with spans of either kind an FP32 state for each span and
 * channel, and a copy of the initial states where final_state is init_state.
 */
int kda_ssm_prefill(const void* x, int64_t ldx, const void* dt, int64_t lddt, const float* A,
                    const void* Bm, int64_t ldb, const void* Cm, int64_t ldc, const float* D,
                    const void* z, int64_t ldz, const float* dt_bias, const void* init_state,
                    void* out, void* final_state, int64_t B, int64_t T, int64_t dim,
                    int64_t groups, int64_t nstate, const int64_t* cu_seqlens, uint32_t flags,
                    void* stream);

/*
 * One token per sequence of the same operation, on a pool of states: rows are
 * the sequences' tokens, state [pool, dim, nstate] (BF16 or FP32 as above) is updated in
 * place, slots as kda_la_decode.  FP32 states: the exponential's mean error is made up for
 * at every token.
 */
int kda_ssm_decode(const void* x, int64_t ldx, const void* dt, int64_t lddt, const float* A,
                   const void* Bm, int64_t ldb, const void* Cm, int64_t ldc, const float* D,
                   const void* z, int64_t ldz, const float* dt_bias, void* state,
                   const int32_t* slots, void* out, int64_t N, int64_t dim, int64_t groups,
                   int64_t nstate, int64_t pool, uint32_t flags, void* stream);

/*
 * Spans kda_ssm_prefill cuts each sequence of a call of this shape into
 * (packed: the whole batch; 0: no cut, or spans one after the other), and the bytes of scratch it takes at
 * most (HOST out).  As kda_plan_segments and kda_workspace_bytes.
 */
int kda_ssm_plan_segments(int64_t B, int64_t T, int64_t dim, int64_t groups, int64_t nstate,
                          int packed, int64_t* segs);
int kda_ssm_workspace_bytes(int64_t B, int64_t T, int64_t dim, int64_t groups, int64_t nstate,
                            int packed, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */
