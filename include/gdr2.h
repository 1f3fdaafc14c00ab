/*
 * gdr2.h -- C ABI of libgdr2, the MI355X (gfx950) implementation of the
 * Gated Delta Rule-2 sequence-mixing operator.
 *
 * Operator ("Gated DeltaNet-2: Decoupling Erase and Write in Linear
 * Attention", anthology record LIT-802, "Key takeaways", first bullet; paper
 * Sec. 3.1, Eqs. 8-10), for every batch row b and head h independently:
 *
 *     S_t = (I - k_t (b_t * k_t)^T) diag(exp g_t) S_{t-1} + k_t (w_t * v_t)^T
 *     o_t = S_t^T q_t                        (readout after the update)
 *
 * b_t is the channel-wise erase gate on the key axis, w_t the channel-wise
 * write gate on the value axis, g_t the channel-wise log-decay on the key axis
 * (alpha_t = exp g_t). gdr2_fwd / gdr2_bwd / gdr2_step take the gates already
 * activated; the *_logits variants take their logits and activate them inside
 * the kernels (see below). Nothing is normalised inside the operator. The
 * forward pass runs the chunkwise algorithm with the cumulative decay folded
 * into asymmetric erase factors and one shared WY/UT inverse (LIT-802
 * takeaway 2, App. A); the backward pass is the gate-aware one (App. B).
 *
 * Layouts (all contiguous, row-major, in the element type `dtype`):
 *   q, k, g, b and dq, dk, dg, db : [B][T][H][dk]
 *   v, w, o, dout and dv, dw      : [B][T][H][dv]
 *   h0, ht, dht, dh0              : [B][H][dk][dv], always fp32
 * Supported: dtype BF16 with dk, dv in {64, 128}; dtype F32 with dk = dv = 64;
 * chunk = 64; any T >= 0 (a partial last chunk is padded with zero tokens,
 * which leave the recurrence unchanged).
 *
 * Calls without tokens (B, T or H zero): the token tensors are empty, their pointers
 * may be NULL, and no workspace is needed (the size functions return 0, a NULL
 * workspace is accepted). A recurrence over no tokens ends where it starts, so
 * gdr2_fwd writes ht = h0 (zeros when h0 is NULL) and gdr2_bwd writes dh0 = dht
 * (zeros when dht is NULL), when ht / dh0 are given and B * H > 0; gdr2_step leaves
 * the state as it is (the state pointer is still required when B * H > 0). Nothing
 * else is enqueued.
 *
 * Ownership: the caller owns every buffer, including the workspace. All device
 * pointers must stay valid until the stream has passed the enqueued work. The
 * library allocates nothing, keeps no state between calls, never synchronises
 * and enqueues everything on `stream` (a hipStream_t, 0 = null stream). Calls on
 * different streams with different workspaces may run concurrently.
 *
 * Errors: every argument is checked on the host before any HIP call; a failed
 * check returns a negative status and enqueues nothing. A failed launch
 * returns GDR2_ERR_HIP. Non-finite inputs are not checked; they propagate.
 *
 * Decay: g is a log-decay (g <= 0, exp g in (0, 1]) of any finite size. The chunkwise
 * kernels scale their factors by exponentials of the decay summed over 16-token blocks;
 * where a block's decay is strong enough that the diagonal block factor would leave the
 * fp32 range, they form that block from per-element decay products instead, so every
 * finite g <= 0 gives finite results (LIT-802 takeaway 1: the channel-wise decay of
 * KDA, which bounds no decay strength).
 */
#ifndef GDR2_H
#define GDR2_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

enum gdr2_dtype { GDR2_DTYPE_F32 = 0, GDR2_DTYPE_BF16 = 1 };

enum gdr2_status {
    GDR2_OK = 0,
    GDR2_ERR_NULL = -1,        /* a required pointer is NULL */
    GDR2_ERR_SHAPE = -2,       /* B, T or H negative, heads that do not divide, or sizes overflow
                                  (scalar gates and cache: launches of 2^32 threads among them) */
    GDR2_ERR_UNSUPPORTED = -3, /* dk/dv/chunk/dtype combination not built */
    GDR2_ERR_ALIGN = -4,       /* a pointer is not 16-byte aligned */
    GDR2_ERR_WORKSPACE = -5,   /* workspace NULL or smaller than required */
    GDR2_ERR_HIP = -6,         /* a HIP launch failed */
    GDR2_ERR_VALUE = -7,       /* a scalar argument is out of range (gate scales, segments, page size,
                                  attention scale, window) */
    GDR2_ERR_SCRATCH = -8      /* gdr2_fwd_noalloc: the call needs more than the fixed scratch */
};

/* Bytes of workspace gdr2_fwd needs. save_for_bwd = 1 sizes it for a later
 * gdr2_bwd(..., fwd_saved = 1) on the same buffer. Returns 0 for unsupported
 * or invalid arguments, and for calls without tokens, which need none. */
size_t gdr2_fwd_workspace_bytes(int B, int T, int H, int dk, int dv, int chunk, int dtype,
                                int save_for_bwd);

/* Bytes of workspace gdr2_bwd needs (either value of fwd_saved). */
size_t gdr2_bwd_workspace_bytes(int B, int T, int H, int dk, int dv, int chunk, int dtype);

/* Forward pass: writes o and, if ht != NULL, the final state.
 * h0: initial state or NULL (= 0). save_for_bwd = 1 also keeps in the
 * workspace what gdr2_bwd needs (per-chunk states and operands), so the
 * backward does not recompute the forward. */
int gdr2_fwd(const void* q, const void* k, const void* v, const void* g, const void* b, const void* w,
             const float* h0, void* o, float* ht, int B, int T, int H, int dk, int dv, int chunk,
             int dtype, int save_for_bwd, void* workspace, size_t workspace_bytes, void* stream,
             void* const* stage_events);

/* Backward pass: given dout (= dL/do) and dht (= dL/dS_T, NULL = 0), writes
 * dq, dk_, dv_, dg, db, dw (same layouts and dtype as the inputs) and, if
 * dh0 != NULL, dL/dh0. fwd_saved = 1: the workspace holds what
 * gdr2_fwd(..., save_for_bwd = 1) left there for the same inputs and has not
 * been touched since; fwd_saved = 0: the forward quantities are recomputed
 * inside this call (o is not written). */
int gdr2_bwd(const void* q, const void* k, const void* v, const void* g, const void* b, const void* w,
             const float* h0, const void* dout, const float* dht, void* dq, void* dk_, void* dv_,
             void* dg, void* db, void* dw, float* dh0, int B, int T, int H, int dk, int dv, int chunk,
             int dtype, int fwd_saved, void* workspace, size_t workspace_bytes, void* stream,
             void* const* stage_events);

/* Chunk-parallel scan of the state chains. gdr2_fwd / gdr2_bwd walk each sequence's
 * chunks in order, one chain per sequence and 16-column slice of the value axis, so a
 * call with few sequences and many chunks leaves most of the GPU idle. Only the state
 * is carried between chunks ("Gated DeltaNet-2", anthology record LIT-802, "Key
 * takeaways", second bullet; digg thread post 9/), and the carry is affine in it:
 * S_{c+1} = P_c S_c + H_c with P_c = diag(exp gamma_C) - Kd^T Wm and H_c = Kd^T U. These
 * variants cut every sequence into `segments` pieces of ceil(NT / segments) chunks
 * (NT = ceil(T / chunk); fewer pieces if T is short) and walk them at the same time:
 * summaries of each piece (its end state from a zero start and its transition, the
 * product of its P_c), an fp32 scan over the pieces for their true start states, then
 * the usual walk of every piece. The backward does the same in reverse with P^T.
 * Results equal the one-walk chains up to rounding order. The work grows (about 3x the
 * chain's), so it pays only when the sequences are too few to fill the GPU: gdr2_fwd,
 * gdr2_bwd and their _logits variants use it by themselves when B * H * dv / 16 <= 128,
 * with 512 / (B * H * dv / 16) segments, at most 8, of at least 16 chunks each (their
 * workspace sizes include it), and walk the chains whole otherwise; segments = 1 here
 * forces one walk. Workspace: gdr2_seg_workspace_bytes (with
 * save_for_bwd = 1 for the backward; a gdr2_bwd_seg(..., fwd_saved = 1) needs the
 * workspace of a gdr2_fwd_seg(..., save_for_bwd = 1) with the same segments). Errors
 * as gdr2_fwd / gdr2_bwd; segments < 1 returns GDR2_ERR_VALUE. */
size_t gdr2_seg_workspace_bytes(int B, int T, int H, int dk, int dv, int chunk, int segments, int dtype,
                                int save_for_bwd);

int gdr2_fwd_seg(const void* q, const void* k, const void* v, const void* g, const void* b, const void* w,
                 const float* h0, void* o, float* ht, int B, int T, int H, int dk, int dv, int chunk,
                 int segments, int dtype, int save_for_bwd, void* workspace, size_t workspace_bytes,
                 void* stream, void* const* stage_events);

int gdr2_bwd_seg(const void* q, const void* k, const void* v, const void* g, const void* b, const void* w,
                 const float* h0, const void* dout, const float* dht, void* dq, void* dk_, void* dv_,
                 void* dg, void* db, void* dw, float* dh0, int B, int T, int H, int dk, int dv, int chunk,
                 int segments, int dtype, int fwd_saved, void* workspace, size_t workspace_bytes,
                 void* stream, void* const* stage_events);

/* Recurrent step, for decoding: processes the T tokens of q, k, v, g, b, w one at a
 * time, starting from the state in `state` (fp32 [B][H][dk][dv], required), which is
 * read and then overwritten with the state after the last token; writes o (layouts as
 * above). Same recurrence as gdr2_fwd -- for state = h0 it returns the same o and final
 * state up to fp32 rounding order -- computed token by token with each head's state
 * held on chip: constant memory per head however long the sequence (chatpaper.ai
 * abstract of "Gated DeltaNet-2": constant-memory decoding). Supported dk/dv/dtype as
 * gdr2_fwd; no workspace; no backward. Errors as gdr2_fwd (GDR2_ERR_NULL when state
 * is NULL). */
int gdr2_step(const void* q, const void* k, const void* v, const void* g, const void* b, const void* w,
              float* state, void* o, int B, int T, int H, int dk, int dv, int dtype, void* stream);

/* Gates as logits. The erase and write gates are sigmoids of their own projections
 * ("Gated DeltaNet-2", anthology record LIT-802, "Key takeaways", first bullet); these
 * entry points take the projections' outputs (logits) zg, zb, zw (layouts of g, b, w)
 * and apply, inside the kernels,
 *     b = b_scale * sigmoid(zb),   w = sigmoid(zw),   g = -g_scale * softplus(zg),
 * so that no separate elementwise pass over the gates is needed. b_scale = 1 is the
 * plain erase gate, b_scale = 2 the widened [0, 2] erase range of the paper's Table 5
 * ablation; 0 < b_scale <= 2. The log-decay parametrisation (any g_scale > 0, finite)
 * keeps the decay exp g in (0, 1); the pages leave it open and this is the reading
 * taken. The backward variant writes dL/dzg, dL/dzb, dL/dzw into dzg, dzb, dzw (the
 * other outputs as gdr2_bwd). Everything else -- layouts, dtypes, workspace (the same
 * size functions), ownership, events, errors -- is as for gdr2_fwd / gdr2_bwd /
 * gdr2_step; a scale out of range returns GDR2_ERR_VALUE and enqueues nothing.
 * A gdr2_bwd_logits(..., fwd_saved = 1) must follow gdr2_fwd_logits with the same
 * logits and scales. */
int gdr2_fwd_logits(const void* q, const void* k, const void* v, const void* zg, const void* zb,
                    const void* zw, float g_scale, float b_scale, const float* h0, void* o, float* ht,
                    int B, int T, int H, int dk, int dv, int chunk, int dtype, int save_for_bwd,
                    void* workspace, size_t workspace_bytes, void* stream, void* const* stage_events);

int gdr2_bwd_logits(const void* q, const void* k, const void* v, const void* zg, const void* zb,
                    const void* zw, float g_scale, float b_scale, const float* h0, const void* dout,
                    const float* dht, void* dq, void* dk_, void* dv_, void* dzg, void* dzb, void* dzw,
                    float* dh0, int B, int T, int H, int dk, int dv, int chunk, int dtype, int fwd_saved,
                    void* workspace, size_t workspace_bytes, void* stream, void* const* stage_events);

int gdr2_step_logits(const void* q, const void* k, const void* v, const void* zg, const void* zb,
                     const void* zw, float g_scale, float b_scale, float* state, void* o, int B, int T,
                     int H, int dk, int dv, int dtype, void* stream);

/* stage_events (gdr2_fwd and gdr2_bwd, and their _logits and _seg variants): NULL, or
 * an array of hipEvent_t for per-stage timing on `stream`: element 0 marks the start of
 * the first stage and element i the end of the i-th (a NULL element: no event at that
 * boundary). The events are attached to the
 * stages' kernel launches (start of the first kernel, end of the last), so timing puts no
 * extra commands between the kernels; a stage's interval therefore includes the launch
 * gap before its first kernel.
 * gdr2_fwd runs 2 stages (intra-chunk, state chain), so it needs 3 events; gdr2_bwd
 * runs 2 (reverse state chain, intra-chunk gradients) when fwd_saved = 1, and 4 (the
 * two forward stages first) when fwd_saved = 0, so it needs 3 or 5. With segments > 1
 * the chain stage also holds the summary and scan kernels. The events belong to the
 * caller. */

/* For callers that cannot allocate device memory -- code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc: the inference forward (gdr2_fwd with
 * save_for_bwd = 0) without a workspace argument. Its workspace is a fixed array of
 * GDR2_NOALLOC_SCRATCH_BYTES (64 MiB) of device memory inside the library; each GPU the
 * library runs on holds its own copy until the process ends. The call allocates nothing
 * (no hipMalloc, no hipFree, no allocating library routine); the caller still passes
 * every input and output. A call whose workspace, gdr2_fwd_workspace_bytes(B, T, H, dk,
 * dv, chunk, dtype, 0), exceeds the array returns GDR2_ERR_SCRATCH and enqueues nothing
 * (at d_k = d_v = 128 in bf16 about 72.5 KB per chunk of 64 tokens and head, so e.g.
 * B = 1, H = 16, T = 2048 fits); other errors as gdr2_fwd. All calls on one GPU share the
 * array, which keeps the last call's contents: calls that overlap on one GPU (several
 * streams, or several host threads) race on it and must be serialised by the caller.
 * Arguments, layouts and results otherwise as gdr2_fwd (bitwise the same results). */
#define GDR2_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

int gdr2_fwd_noalloc(const void* q, const void* k, const void* v, const void* g, const void* b, const void* w,
                     const float* h0, void* o, float* ht, int B, int T, int H, int dk, int dv, int chunk,
                     int dtype, void* stream);

/* Gated delta rule with scalar gates: one log-decay g and one write strength beta per token and
 * value head instead of a gate per channel,
 *
 *     S_t = exp(g_t) (I - beta_t k_t k_t^T) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t,
 *
 * which is gdr2_fwd's recurrence with b = w = beta and g the same in every channel, at a third of its
 * input bytes. Value heads may share key heads: Hv is a multiple of Hk, and value head h reads the
 * queries and keys of head h / (Hv / Hk); their gradients are summed over the heads that share them.
 *
 * Layouts (contiguous, row-major, element type `dtype` unless said):
 *   q, k and dq, dk_             : [tokens][Hk][dk]
 *   v, o, dout and dv_           : [tokens][Hv][dv]
 *   g, beta and dg, dbeta        : [tokens][Hv]
 *   h0, ht, dht, dh0             : [N][Hv][dk][dv], always fp32
 * Sequences: with cu_seqlens NULL, N sequences of T tokens each, one after another (tokens = N T).
 * Else packed: T tokens in all, sequence s being the tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1;
 * cu_seqlens is an int32 array of N + 1 non-decreasing entries in 0 .. T on the device, lengths may be
 * zero (such a sequence passes its state through). Its entries are data that no check on the host can
 * see: entries out of order or range give wrong results for the sequences concerned, but no access
 * outside the tensors. Tokens of no sequence are not read, and their rows of o (dq, dk_, dv_, dg, dbeta)
 * are left as they were, or set to zero with zero_rest = 1 (N = 0 writes nothing).
 *
 * Precision: with bf16, o and the gradients of the token tensors carry a few bf16 roundings; the
 * states, which are fp32, do not: ht and dh0 are off by less than 1e-5 of what was written into them
 * (Frobenius norm; writes that cancel one another, as of one key again and again, leave their errors
 * behind). g <= 0 may be of any finite size, as for gdr2_fwd. Results repeat bit for bit; few long
 * sequences of one length are walked in segments, so that their last bits differ from those of a call
 * with more sequences, or a packed one.
 *
 * Supported dtype / dk / dv as gdr2_fwd; chunks are of 64 tokens. Ownership, streams, errors and calls
 * without tokens as gdr2_fwd / gdr2_bwd; g, beta, dg and dbeta need only their element's alignment; Hv
 * that is no multiple of Hk, 0 included unless Hk is 0, returns GDR2_ERR_SHAPE. Outputs must not overlap
 * one another or the inputs. The workspace has no content between calls but for what fwd_saved = 1 reads;
 * calls that may overlap need one each:
 * gdr2_scalar_workspace_bytes (packed = 1 when cu_seqlens is given; save_for_bwd = 1 for a forward that
 * a backward follows, and for the backward). gdr2_scalar_bwd(..., fwd_saved = 1) needs the workspace as
 * gdr2_scalar_fwd(..., save_for_bwd = 1) left it for the same inputs; fwd_saved = 0 recomputes. */
size_t gdr2_scalar_workspace_bytes(int N, int T, int Hk, int Hv, int dk, int dv, int packed, int dtype,
                                   int save_for_bwd);

int gdr2_scalar_fwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0,
                    const int* cu_seqlens, void* o, float* ht, int N, int T, int Hk, int Hv, int dk, int dv,
                    int dtype, int zero_rest, int save_for_bwd, void* workspace, size_t workspace_bytes,
                    void* stream);

int gdr2_scalar_bwd(const void* q, const void* k, const void* v, const void* g, const void* beta, const float* h0,
                    const void* dout, const float* dht, const int* cu_seqlens, void* dq, void* dk_, void* dv_,
                    void* dg, void* dbeta, float* dh0, int N, int T, int Hk, int Hv, int dk, int dv, int dtype,
                    int zero_rest, int fwd_saved, void* workspace, size_t workspace_bytes, void* stream);

/* Its recurrent form, for decoding: T tokens for each of B rows (q, k [B][T][Hk][dk], v, o
 * [B][T][Hv][dv], g, beta [B][T][Hv]) on states in a pool, state fp32 [n_states][Hv][dk][dv], updated
 * in place. Row b's state is slots[b] (an int32 array on the device), or b when slots is NULL
 * (n_states >= B then). A row whose slot is outside 0 .. n_states - 1 is padding: its o is zero and
 * no state is touched. Rows that name the same slot are taken one after another in the order of the
 * rows, as one sequence. States that no row names are left as they were. */
int gdr2_scalar_step(const void* q, const void* k, const void* v, const void* g, const void* beta, float* state,
                     const int* slots, void* o, int B, int T, int Hk, int Hv, int dk, int dv, int n_states, int dtype,
                     void* stream);

/* Attention of one new token a sequence over a paged key-value cache, the decode step of the
 * attention layers that a hybrid decoder alternates with the recurrent ones:
 *
 *     o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q . k_t),   lse = log sum_t p_t
 *
 * over the tokens t that the sequence holds (its new token, appended before, included), or the last
 * `window` of them when window > 0.
 *   q, o   : [B][Hq][D] in `dtype`, contiguous;   lse : fp32 [B][Hq], or NULL
 *   caches : [num_pages][page_size][Hkv][D] in `dtype`, the D elements of a row contiguous;
 *            cache_strides = { page, token, head stride of k_cache, the same of v_cache } in elements
 *            (a host array), multiples of 16 bytes; Hq is a multiple of Hkv, query head h reading key
 *            head h / (Hq / Hkv)
 *   block_table : int32 [B][max_pages] on the device; page i of a sequence holds its tokens
 *            i page_size .. (i + 1) page_size - 1. Entries outside 0 .. num_pages - 1 are no page:
 *            their tokens are masked (attention) or dropped (append)
 *   lengths : int32 [B] on the device, tokens held; taken as 0 .. max_pages page_size where outside
 * page_size is a power of two from 16 on (else GDR2_ERR_VALUE), D 64 or 128, dtype BF16 or F32. A row
 * with nothing visible gets o = 0 and lse = -inf. What the cache holds in masked or unused places,
 * infinities and NaN included, does not matter. GDR2_ERR_SHAPE: max_pages page_size of more than
 * 2^31 - 65, or more than 2^31 - 1 places of B Hkv ceil(Hq / Hkv / 16) rows, each of which takes 6 and one for
 * every 32 tokens (fp32: 16) of the table, or of the window and 32 (16) more where that is less. o must not overlap q. Scores, weights' sums and lse are fp32; with bf16 the
 * weights enter the second product in two bf16 parts, 16 bits together. Results do not depend on the other rows of the call beyond
 * the order of fp32 sums, and are repeatable bit for bit. Workspace: gdr2_attn_workspace_bytes, of no
 * content between calls; calls that may overlap need one each. */
size_t gdr2_attn_workspace_bytes(int B, int Hq, int Hkv, int D, int dtype);

int gdr2_attn_step(const void* q, const void* k_cache, const void* v_cache, const long long* cache_strides,
                   const int* block_table, const int* lengths, void* o, float* lse, int B, int Hq, int Hkv, int D,
                   int num_pages, int page_size, int max_pages, float scale, int window, int dtype, void* workspace,
                   size_t workspace_bytes, void* stream);

/* Writes new tokens' keys and values, k and v [tokens][Hkv][D], into the cache behind the starts[s]
 * tokens that sequence s holds: its i-th new token goes to position starts[s] + i. cu_seqlens (int32
 * [B + 1] on the device) gives each sequence's tokens as in gdr2_scalar_fwd, NULL one token a sequence
 * (tokens = B). Tokens whose position lies outside the table or on no page are dropped, and the rest of
 * the cache is left as it was. Two tokens of a call must not share a place. */
int gdr2_kv_append(const void* k, const void* v, void* k_cache, void* v_cache, const long long* cache_strides,
                   const int* block_table, const int* starts, const int* cu_seqlens, int B, int tokens, int Hkv, int D,
                   int num_pages, int page_size, int max_pages, int dtype, void* stream);

/* Static description of a status code. */
const char* gdr2_strerror(int status);

/* Library version as an integer (major * 10000 + minor * 100 + patch). */
int gdr2_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDR2_H */
