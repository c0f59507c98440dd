/*
 * gdn2.h -- C ABI of the MI355X (gfx950) gated delta rule-2 library.
 *
 * The operation (per batch b, head h; state S in R^{dk x dv}, key-by-value:
 * rows are key channels, columns value channels), for each token t:
 *
 *     Sbar = Diag(a_t) S                 decay first; a_t = exp(log_decay_t)
 *     m    = Sbar^T k_t                  the key read of the decayed state
 *     S    = Sbar - (b_t .* k_t) m^T + (w_t .* k_t) v_t^T
 *     o_t  = S^T (q_scale * q_t)         the query read of the updated state
 *
 * Sources: the "Gated DeltaNet-2" blog summary ("Core Mechanism": separate
 * channel-wise erase gate b_t and write gate w_t, channel-wise decay, the
 * chunkwise WY training algorithm and O(1)-memory recurrent inference); the
 * "Gated DeltaNet" page ("Decay first, then compute the write error": the
 * read and the subtraction use the decayed state); the course slides
 * ("Worked case -- full trace": decay, read, correct, then read with q).
 * Both gates act on the key axis.  Tying b = w = beta (scalar) gives Gated
 * DeltaNet, per-channel decay with tied scalar beta gives KDA, a = 1 gives
 * the delta rule (gist.science summary, "Technische Samenvatting", sec. 1).
 *
 * desc->form = GDN2_FORM_VALUE_WRITE selects the update as the gist.science
 * summary writes it ("Methodologie", 1. "Gated Delta-regel-2"):
 *
 *     S    = (I - k_t (b_t .* k_t)^T) Sbar + k_t (w_t .* v_t)^T
 *
 * i.e. the erase gate weights the read (m = Sbar^T (b_t .* k_t)), the erase
 * and the write run along k_t, and the write gate has one factor per VALUE
 * channel.  With scalar gates both forms are the same operation.
 *
 * Conventions shared by every call:
 *  - Every data pointer is DEVICE memory (hipMalloc'd or torch CUDA
 *    tensors) owned by the caller; the library allocates nothing and is
 *    safe to call from several host threads.  Its only global state is the
 *    static scratch of gdn2_chunk_fwd_static and that array's per-GPU
 *    address, looked up once.
 *  - All tensors are contiguous, row-major, last index fastest:
 *        q, k           [B, T, H, dk]    bf16 or fp32 (desc->qkv_dtype)
 *        v              [B, T, H, dv]    same dtype as q, k
 *        o              [B, T, H, dv]    fp32, or bf16 (desc->o_dtype)
 *        log_decay      [B, T, H, dk] fp32 if decay_kind == GDN2_GATE_KEY,
 *                       [B, T, H]     fp32 if GDN2_GATE_HEAD
 *        erase, write   same rule with erase_kind / write_kind (the write
 *                       gate of GDN2_FORM_VALUE_WRITE: [B, T, H, dv] per
 *                       channel)
 *        state tensors  [B, H, dk, dv]   fp32
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the default stream)
 *    and the call returns without synchronising.  Device faults surface at
 *    the caller's next synchronisation.
 *  - Host-side validation runs before any HIP call: on any status other
 *    than GDN2_OK nothing has been enqueued and no output was touched
 *    (GDN2_ERR_HIP aside, which reports a failed launch).
 *  - Input preparation may be fused (desc->gate_logits, desc->qk_l2norm):
 *    the gates then arrive as bf16 logits and q, k unnormalised, and the
 *    kernels apply the activations and the normalisation as they load them
 *    (2048 instead of 2816 bytes per token-head for the full GDN-2 forward).
 *  - Preconditions not checked (they would need a device pass): log_decay
 *    finite and <= 0 (decay gate in (0, 1], course slides "Stability"),
 *    erase/write in [0, 1], all values finite.  These hold for every call
 *    and every path.  The matrix-core forward kernels of gdn2_chunk_fwd,
 *    gdn2_chunk_fwd_static and gdn2_chunk_fwd_varlen (bf16 q/k/v, dk = dv =
 *    128) hold derived operands, intermediates and a copy of the state in
 *    fp16; a chunk whose values would leave fp16's range is recomputed as
 *    the exact fp32 token recurrence instead, with the workspace and without
 *    it, so they ask nothing more (tested with |v| and states of 2^15).  The
 *    backward, the decode step and the fp32 kernels compute in fp32.
 */
#ifndef GDN2_H
#define GDN2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN2_ABI_VERSION 6

typedef enum gdn2_status {
    GDN2_OK = 0,
    GDN2_ERR_NULL = 1,        /* a required pointer (or desc) is NULL            */
    GDN2_ERR_SHAPE = 2,       /* negative / zero / overflowing sizes            */
    GDN2_ERR_DTYPE = 3,       /* unknown qkv_dtype or o_dtype                    */
    GDN2_ERR_UNSUPPORTED = 4, /* valid request no kernel of the library covers  */
    GDN2_ERR_ALIAS = 5,       /* an output overlaps an input (see each call)     */
    GDN2_ERR_WORKSPACE = 6,   /* workspace smaller than the query reported      */
    GDN2_ERR_HIP = 7,         /* a HIP launch or copy failed                     */
    GDN2_ERR_SCRATCH = 8      /* too large for the static scratch of
                                 gdn2_chunk_fwd_static                           */
} gdn2_status;

typedef enum gdn2_dtype { GDN2_F32 = 0, GDN2_BF16 = 1 } gdn2_dtype;

typedef enum gdn2_gate_kind {
    GDN2_GATE_HEAD = 0, /* one value per token-head, shared by all key channels */
    GDN2_GATE_KEY = 1   /* one value per key channel                            */
} gdn2_gate_kind;

typedef enum gdn2_form {
    GDN2_FORM_KEY = 0,         /* erase (b.*k)(k^T Sbar), write (w.*k) v^T  */
    GDN2_FORM_VALUE_WRITE = 1  /* erase k((b.*k)^T Sbar), write k (w.*v)^T;
                                  needs an untied write gate               */
} gdn2_form;

/* Problem description.  For gdn2_recurrent_step `batch` is the number of
 * sequences N and `seqlen` must be 1. */
typedef struct gdn2_desc {
    int64_t batch;      /* B >= 0 */
    int64_t seqlen;     /* T >= 0 */
    int64_t heads;      /* H >= 1 */
    int64_t dk;         /* key channels,   1..128 */
    int64_t dv;         /* value channels, 1..128 */
    int64_t chunk;      /* chunk length C of the chunkwise algorithm: 16, 32 or 64 */
    int32_t qkv_dtype;  /* gdn2_dtype of q, k, v */
    int32_t decay_kind; /* gdn2_gate_kind of log_decay */
    int32_t erase_kind; /* gdn2_gate_kind of erase      */
    int32_t write_kind; /* gdn2_gate_kind of write (ignored when tied) */
    int32_t tie_write_to_erase; /* nonzero: w := b and `write` is ignored */
    float q_scale;      /* multiplies q; 1.0 for the plain read */
    int32_t form;       /* gdn2_form; a tied write gate with
                           GDN2_FORM_VALUE_WRITE is GDN2_ERR_SHAPE */
    int32_t gate_logits; /* nonzero: log_decay, erase and write point at bf16
                            LOGITS x (same shapes, 2 bytes per element; the
                            float* parameters are reinterpreted); the kernels
                            use log a = -softplus(x), b = sigmoid(x),
                            w = sigmoid(x) */
    int32_t qk_l2norm;  /* nonzero: q and k are divided by their L2 norm over
                           the dk channels of each token-head inside the
                           kernels (a zero vector stays zero), before q_scale */
    int32_t o_dtype;    /* gdn2_dtype of the output o of gdn2_chunk_fwd,
                           gdn2_chunk_fwd_varlen and gdn2_recurrent_step:
                           GDN2_F32 (0, the default) or GDN2_BF16, the fp32
                           result rounded to nearest even (2 bytes per element;
                           the float* o parameter is reinterpreted).  Anything
                           else is GDN2_ERR_DTYPE.  The backward's d_o is fp32
                           whatever this says. */
} gdn2_desc;

/* GDN2_ABI_VERSION of the loaded library. */
int gdn2_abi_version(void);

/* Static, human-readable name of a status code. */
const char *gdn2_status_str(int status);

/* Device workspace, in bytes, for the two-pass form of gdn2_chunk_fwd on
 * `desc`; 0 when the request has no two-pass kernel (it then always runs in
 * one pass).  The two-pass form covers bf16 q/k/v, dk = dv = 128, chunk 64
 * and gates per key channel or per head (a per-head decay only with
 * per-head erase and write gates; untied, the write gate of the erase
 * gate's kind); it needs B*H*ceil(T/64) records of about
 * 71 KiB, and, when B*H is small against T (long sequences on few chains,
 * scanned in parallel segments), two 64 KiB states per (chain, segment).
 * Same validation as gdn2_chunk_fwd. */
gdn2_status gdn2_chunk_fwd_workspace(const gdn2_desc *desc, size_t *bytes);

/*
 * Chunkwise-parallel forward over whole sequences (training / prefill).
 *
 * The "Gated DeltaNet-2" blog summary ("Core Mechanism") and the
 * gist.science summary ("Technische Samenvatting", section 3) describe the
 * algorithm: the cumulative per-channel decay of each chunk is absorbed
 * into the erase and write factors, a unit-lower-triangular solve gives the
 * chunk's auxiliary matrices, and dense chunk contractions carry the state
 * from chunk to chunk.  The result equals running the recurrence above
 * token by token (up to rounding); the chunk length only changes speed.
 *
 *   q, k, v      inputs, see layouts above.
 *   log_decay    log of the decay gate (<= 0).
 *   erase        erase gate b.
 *   write        write gate w; ignored (may be NULL) when
 *                desc->tie_write_to_erase is set.
 *   state0       initial state [B,H,dk,dv] fp32, or NULL for zeros.
 *   o            output [B,T,H,dv], fp32 or bf16 per desc->o_dtype (must not overlap
 *                any input).
 *   state_out    final state [B,H,dk,dv] fp32, or NULL to skip.  It may be
 *                exactly state0 (updated in place); any other overlap with
 *                an input is GDN2_ERR_ALIAS.
 *   workspace    NULL (or ws_bytes 0): run in one pass, no scratch.
 *                Otherwise device scratch of ws_bytes >=
 *                gdn2_chunk_fwd_workspace(), 256-byte aligned, else
 *                GDN2_ERR_WORKSPACE; it must not overlap any other argument
 *                (GDN2_ERR_ALIAS).  The two-pass form first computes every
 *                chunk's state-independent products in parallel into it,
 *                then scans the chunks; its contents need no initialisation
 *                and are undefined afterwards.  Calls that share one
 *                workspace must not overlap in time.
 * With T == 0 nothing is read but state0, o is untouched and state_out
 * receives state0 (or zeros).
 */
gdn2_status gdn2_chunk_fwd(const gdn2_desc *desc,
                           const void *q, const void *k, const void *v,
                           const float *log_decay, const float *erase, const float *write,
                           const float *state0, float *o, float *state_out,
                           void *workspace, size_t ws_bytes, void *stream);

/*
 * gdn2_chunk_fwd without any allocation, for callers that cannot allocate
 * device memory: code under HIP graph capture, tight serving loops, harnesses
 * that forbid hipMalloc.  Same arguments, layouts, rules and result as
 * gdn2_chunk_fwd with workspace = NULL, except that requests of the
 * two-pass form keep their per-chunk records in one static device array of
 * the library, 128 MiB per GPU, held from the first such call on a GPU until
 * the process ends.  When the records of all ceil(T/64) chunks of every
 * chain do not fit there, the chunks are processed in consecutive windows
 * that do, the state carried from window to window in the same array
 * (more launches, the same arithmetic).  Each record takes 70.5 KiB and
 * each carried state 64 KiB: a request fits in one window up to
 * B*H*ceil(T/64) = 1859 records, in windows up to B*H = 974 chains; beyond
 * both it returns GDN2_ERR_SCRATCH before anything is enqueued.  Requests without a two-pass
 * kernel run the single-pass kernels, which use no scratch.
 *
 * Every call on one GPU shares that GPU's array: calls that overlap in time
 * on one GPU (other streams, other host threads) race and give undefined
 * results; serialise them.  The array needs no initialisation.  The first
 * call on each GPU looks up the array's device address (hipGetSymbolAddress)
 * and keeps it; no call allocates or frees memory.
 */
gdn2_status gdn2_chunk_fwd_static(const gdn2_desc *desc,
                                  const void *q, const void *k, const void *v,
                                  const float *log_decay, const float *erase, const float *write,
                                  const float *state0, float *o, float *state_out, void *stream);

/* Device workspace, in bytes, for the two-pass form of gdn2_chunk_fwd_varlen
 * on `desc` (batch = N sequences, seqlen = T packed tokens); 0 when the
 * request has no two-pass kernel.  It holds records for ceil(T/64) + N
 * chunks per head (every sequence may end in a partial chunk) and the
 * sequence plan.  Same validation as gdn2_chunk_fwd_varlen. */
gdn2_status gdn2_chunk_fwd_varlen_workspace(const gdn2_desc *desc, size_t *bytes);

/*
 * The chunkwise forward over N sequences of different lengths packed along
 * one token axis (training on packed documents, prefill of a batch of
 * prompts).  The sequences are independent recurrences, each from its own
 * initial state: the result for sequence i equals gdn2_chunk_fwd on its
 * tokens alone.  Chunks never straddle two sequences; each sequence's
 * chunks start at its first token ("Gated DeltaNet" page, "What makes the
 * architecture more than a recurrence": chunkwise training over long
 * sequences, each transition an affine map of the state).
 *
 *   desc         batch = N >= 0 sequences, seqlen = T >= 0 packed tokens
 *                (T <= INT32_MAX), other fields as for gdn2_chunk_fwd.
 *   cu_seqlens   DEVICE int32 [N+1]: sequence i covers packed tokens
 *                cu_seqlens[i] .. cu_seqlens[i+1]-1; required
 *                0 = cu_seqlens[0] <= cu_seqlens[1] <= ... <= cu_seqlens[N]
 *                = T.  Not checked (it would need a device pass): other
 *                offsets give unspecified results, but every offset is
 *                clamped into [0, T] and every range made non-negative, so
 *                no access leaves the tensors or the workspace.
 *   q, k, v, gates, o   [T, H, ...]: the [B, T, H, ...] layouts with B = 1.
 *   state0, state_out   [N, H, dk, dv] fp32, one state per sequence
 *                (state0 NULL: zeros; state_out NULL: skipped; in place as
 *                for gdn2_chunk_fwd).
 *   workspace    as for gdn2_chunk_fwd with gdn2_chunk_fwd_varlen_workspace()
 *                bytes; NULL runs the single-kernel path.
 * Outputs must not overlap cu_seqlens, any other input or the workspace
 * (GDN2_ERR_ALIAS).  Rows of o outside every sequence are untouched; an
 * empty sequence passes its initial state through.
 */
gdn2_status gdn2_chunk_fwd_varlen(const gdn2_desc *desc, const int32_t *cu_seqlens,
                                  const void *q, const void *k, const void *v,
                                  const float *log_decay, const float *erase, const float *write,
                                  const float *state0, float *o, float *state_out,
                                  void *workspace, size_t ws_bytes, void *stream);

/* Device workspace, in bytes, for gdn2_chunk_bwd on `desc`: two fp32 state
 * histories, B*H*ceil(T/Cb)*dk*dv*4 bytes each (Cb = 16 for dk = dv = 128,
 * larger for small heads); for dk = dv = 128 a 37 KiB fp32 record per
 * (chain, internal chunk); with fused input preparation an fp32 copy of the
 * prepared inputs (q, k, v and two norms per token-head when qk_l2norm, the
 * activated gates when gate_logits).  Each region 256-byte aligned.  Same
 * validation as gdn2_chunk_fwd; GDN2_ERR_UNSUPPORTED if no internal chunk
 * fits. */
gdn2_status gdn2_chunk_bwd_workspace(const gdn2_desc *desc, size_t *bytes);

/*
 * Backward of gdn2_chunk_fwd: the gradients of
 *     L = <d_o, o> + <d_state_out, S_T>
 * with respect to q, k, v, the three gates and state0.  Training is why the
 * chunk form exists ("Gated DeltaNet-2" blog summary, "Core Mechanism": the
 * chunkwise algorithm and its kernels serve training; gist.science summary,
 * "Technische Samenvatting" section 3).  The result equals reverse-mode
 * differentiation of the token recurrence (up to rounding).  It is computed
 * chunk by chunk in fp32 (on the matrix cores for dk = dv = 128): a forward
 * scan records the state entering every internal chunk, a reverse scan
 * carries the state gradient back through the chunks, then every chunk
 * forms its gradients in parallel from the two records.  Both forms
 * (desc->form) are covered.  With fused input preparation (desc->gate_logits,
 * desc->qk_l2norm) the gradients are those of the raw inputs: of the gate
 * logits (through -softplus and sigmoid) and of unnormalised q, k (through
 * the L2 normalisation; a zero row gets zero).
 *
 *   q .. state0  the forward's inputs (same layouts and rules as
 *                gdn2_chunk_fwd; state0 NULL means zeros).
 *   d_o          gradient of o, [B,T,H,dv] fp32 (required).
 *   d_state_out  gradient of the final state [B,H,dk,dv] fp32, or NULL for
 *                zeros.
 *   dq, dk, dv   fp32, [B,T,H,dk] / [B,T,H,dv] (fp32 whatever qkv_dtype).
 *   d_log_decay, d_erase, d_write   fp32, shaped like their gate (per key
 *                channel or per token-head; the value-write form's write gate
 *                per value channel), also for bf16 logits; d_write ignored
 *                (may be NULL) when tied, and then d_erase holds the gradient
 *                of the one shared gate.
 *   d_state0     gradient of state0 [B,H,dk,dv] fp32, or NULL to skip.
 *   workspace    device scratch of ws_bytes >= gdn2_chunk_bwd_workspace(),
 *                256-byte aligned, else GDN2_ERR_WORKSPACE; contents need no
 *                initialisation and are undefined afterwards.
 * Outputs must not overlap each other, any input or the workspace
 * (GDN2_ERR_ALIAS).  Every output is written in full.  With T == 0,
 * d_state0 receives d_state_out (or zeros) and nothing else is touched.
 */
gdn2_status gdn2_chunk_bwd(const gdn2_desc *desc,
                           const void *q, const void *k, const void *v,
                           const float *log_decay, const float *erase, const float *write,
                           const float *state0, const float *d_o, const float *d_state_out,
                           float *dq, float *dk, float *dv,
                           float *d_log_decay, float *d_erase, float *d_write,
                           float *d_state0, void *workspace, size_t ws_bytes, void *stream);

/* Device workspace, in bytes, for gdn2_chunk_bwd_varlen on `desc` (batch =
 * N sequences, seqlen = T packed tokens): the regions of
 * gdn2_chunk_bwd_workspace sized for ceil(T/Cb) + N internal chunks per head,
 * and the sequence plan.  Same validation as gdn2_chunk_bwd_varlen. */
gdn2_status gdn2_chunk_bwd_varlen_workspace(const gdn2_desc *desc, size_t *bytes);

/*
 * Backward of gdn2_chunk_fwd_varlen: the gradients of
 *     L = <d_o, o> + <d_state_out, S_T(i) for every sequence i>
 * for N sequences packed along one token axis, each its own recurrence
 * (training on packed documents).  The result for sequence i equals
 * gdn2_chunk_bwd on its tokens alone.
 *
 *   desc, cu_seqlens   as for gdn2_chunk_fwd_varlen (offsets unchecked, but
 *                clamped so that no access leaves the buffers).
 *   q .. write, d_o, the gradients of q .. write   [T, H, ...] (the B = 1
 *                layouts), rules as for gdn2_chunk_bwd.
 *   state0, d_state_out, d_state0   [N, H, dk, dv] fp32.
 *   workspace    as for gdn2_chunk_bwd, gdn2_chunk_bwd_varlen_workspace() bytes.
 * Outputs must not overlap each other, cu_seqlens, any other input or the
 * workspace (GDN2_ERR_ALIAS).  Rows outside every sequence are untouched; an
 * empty sequence passes its state gradient through to d_state0.
 */
gdn2_status gdn2_chunk_bwd_varlen(const gdn2_desc *desc, const int32_t *cu_seqlens,
                                  const void *q, const void *k, const void *v,
                                  const float *log_decay, const float *erase, const float *write,
                                  const float *state0, const float *d_o, const float *d_state_out,
                                  float *dq, float *dk, float *dv,
                                  float *d_log_decay, float *d_erase, float *d_write,
                                  float *d_state0, void *workspace, size_t ws_bytes, void *stream);

/*
 * One recurrent decode step for N = desc->batch sequences (desc->seqlen must
 * be 1): the O(1)-memory inference form ("Gated DeltaNet-2" blog summary,
 * "Core Mechanism"; the fixed-size state of the divagr.com explainer, part
 * 5).  The fp32 state [N,H,dk,dv] is read and rewritten in place.
 *
 *   q, k [N,H,dk], v [N,H,dv] (qkv_dtype); gates [N,H,dk] or [N,H] fp32;
 *   write ignored when tied; state in/out; o [N,H,dv] fp32 or bf16 (o_dtype), must not overlap
 *   the state or any input.
 */
gdn2_status gdn2_recurrent_step(const gdn2_desc *desc,
                                const void *q, const void *k, const void *v,
                                const float *log_decay, const float *erase, const float *write,
                                float *state, float *o, void *stream);

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head: the token mixer without the
 * erase step, beside the gated delta rule.  Per (batch, head), with a state
 * S in R^{dk x dv} (key-by-value, as above):
 *
 *     S_t = a_t S_{t-1} + k_t v_t^T          a_t = exp(log_decay_t)
 *     o_t = q_scale S_t^T q_t                read after the update
 *
 * The delta rule with b = 0, w = 1 and a per-head decay is the same
 * recurrence; these calls do not pay for its triangular solve, take q, k, v
 * of any finite size (no fp16 anywhere) and decays that are one value per
 * token and head or one per head.
 *
 * Conventions are those at the top of this file: contiguous device tensors,
 * host-side validation before anything is enqueued, work on `stream`, no
 * allocation, no synchronisation.  Outputs and gradients of q, k, v have
 * the type of q, k, v (bf16 results are the fp32 ones rounded once, to
 * nearest even); states, decays and their gradients are fp32.
 *
 * Precision, bf16 inputs: the products of inputs are exact, every sum is
 * fp32.  The masked scores enter their product as two bf16 parts (16 bits),
 * the state enters the read of o and dv as two and of dq and dk as three, and
 * the values that update a state as three (all 24 bits), or two where only
 * bf16 results come of it: two parts leave 2^-16 of an operand, a small share
 * of the 2^-8 that the result's own rounding leaves.  States, d_log_decay and
 * d_state0 carry fp32 accuracy.  fp32 inputs: fp32 throughout.
 *
 * d_log_decay is a sum over the tokens behind, so its rounding errors are of
 * the size of what is summed, also where a token's own gradient is next to
 * nothing (a far decay's) or a head's terms cancel.
 *
 * Preconditions not checked: all values finite, log_decay <= 0 (minus
 * infinity is allowed and clears the state; anything below -10000 counts as
 * -10000, whose exponential is 0).
 *
 * GDN2_ERR_UNSUPPORTED: dk or dv above 128, a sequence of 2^31 tokens or
 * more, more than 65535 heads, 2^20 (sequence, head) states or more, and
 * requests of more than 2.7 million (segment, head) pairs backward or 4.1
 * million forward (a segment: at most 1024 tokens backward).
 */
typedef enum gdn2_decay_kind {
    GDN2_DECAY_TOKEN = 0, /* log_decay [B,T,H]: one value per token and head */
    GDN2_DECAY_HEAD = 1   /* log_decay [H]: one value per head               */
} gdn2_decay_kind;

typedef struct gdn2_linear_desc {
    int64_t batch;      /* B >= 0 (packed: N sequences)            */
    int64_t seqlen;     /* T >= 0 (packed: tokens of the one axis) */
    int64_t heads;      /* H >= 1 */
    int64_t dk;         /* key channels,   1..128 */
    int64_t dv;         /* value channels, 1..128 */
    int32_t dtype;      /* gdn2_dtype of q, k, v, o, d_o and the gradients of q, k, v */
    int32_t decay_kind; /* gdn2_decay_kind */
    float q_scale;      /* multiplies q */
    int32_t reserved;   /* 0 */
} gdn2_linear_desc;

/* Device workspace, in bytes, with which gdn2_linear_fwd runs long
 * sequences on few chains in parallel segments; 0 where whole chains fill
 * the GPU.  It holds one fp32 state per (segment, head). */
gdn2_status gdn2_linear_fwd_workspace(const gdn2_linear_desc *desc, size_t *bytes);

/*
 * Chunked forward over whole sequences (training / prefill).
 *
 *   q, k [B,T,H,dk], v [B,T,H,dv]; log_decay fp32 per desc->decay_kind
 *   state0       initial state [B,H,dk,dv] fp32, or NULL for zeros
 *   o            [B,T,H,dv], must not overlap any input
 *   state_out    final state [B,H,dk,dv] fp32, or NULL; it may be exactly
 *                state0 (in place), any other overlap is GDN2_ERR_ALIAS
 *   workspace    NULL (or ws_bytes 0): one pass over each chain, no scratch;
 *                otherwise >= gdn2_linear_fwd_workspace() bytes, 256-byte
 *                aligned (GDN2_ERR_WORKSPACE), overlapping nothing else.
 *                Calls that share one must not overlap in time.
 * T == 0: state_out receives state0 (or zeros), nothing else is touched.
 */
gdn2_status gdn2_linear_fwd(const gdn2_linear_desc *desc, const void *q, const void *k, const void *v,
                            const float *log_decay, const float *state0, void *o, float *state_out,
                            void *workspace, size_t ws_bytes, void *stream);

/* As gdn2_linear_fwd_workspace, for gdn2_linear_fwd_varlen. */
gdn2_status gdn2_linear_fwd_varlen_workspace(const gdn2_linear_desc *desc, size_t *bytes);

/*
 * The forward over N = desc->batch sequences packed along one axis of T =
 * desc->seqlen tokens (q, k [T,H,dk], v, o [T,H,dv], log_decay [T,H] or [H],
 * states [N,H,dk,dv]).  cu_seqlens: DEVICE int32 [N+1], 0 = cu[0] <= .. <=
 * cu[N] = T, not checked but clamped as for gdn2_chunk_fwd_varlen, so no
 * access leaves the buffers.  Rows outside every sequence are untouched; an
 * empty sequence passes its state through.
 */
gdn2_status gdn2_linear_fwd_varlen(const gdn2_linear_desc *desc, const int32_t *cu_seqlens,
                                   const void *q, const void *k, const void *v,
                                   const float *log_decay, const float *state0, void *o, float *state_out,
                                   void *workspace, size_t ws_bytes, void *stream);

/* Device workspace, in bytes, for gdn2_linear_bwd: two fp32 states per
 * (segment of up to 1024 tokens, head), one per chain, and a few fp32 values
 * per token-head. */
gdn2_status gdn2_linear_bwd_workspace(const gdn2_linear_desc *desc, size_t *bytes);

/*
 * Backward of gdn2_linear_fwd: the gradients of <d_o, o> + <d_state_out, S_T>.
 *
 *   q .. state0  the forward's inputs; d_o like o
 *   d_state_out  [B,H,dk,dv] fp32, or NULL for zeros
 *   dq, dk, dv   like q, k, v
 *   d_log_decay  fp32, like log_decay (per head: summed over tokens and
 *                sequences, in a fixed order)
 *   d_state0     [B,H,dk,dv] fp32, or NULL to skip
 *   workspace    >= gdn2_linear_bwd_workspace() bytes, 256-byte aligned
 * Outputs must not overlap each other, any input or the workspace.  The
 * result is the same, bit for bit, on every run.  T == 0 (or B == 0):
 * d_state0 receives d_state_out (or zeros), a per-head d_log_decay zeros.
 */
gdn2_status gdn2_linear_bwd(const gdn2_linear_desc *desc, const void *q, const void *k, const void *v,
                            const float *log_decay, const float *state0, const void *d_o,
                            const float *d_state_out, void *dq, void *dk, void *dv, float *d_log_decay,
                            float *d_state0, void *workspace, size_t ws_bytes, void *stream);

/* As gdn2_linear_bwd_workspace, for gdn2_linear_bwd_varlen. */
gdn2_status gdn2_linear_bwd_varlen_workspace(const gdn2_linear_desc *desc, size_t *bytes);

/* Backward of gdn2_linear_fwd_varlen; rows of dq, dk, dv and of a per-token
 * d_log_decay outside every sequence are untouched. */
gdn2_status gdn2_linear_bwd_varlen(const gdn2_linear_desc *desc, const int32_t *cu_seqlens,
                                   const void *q, const void *k, const void *v, const float *log_decay,
                                   const float *state0, const void *d_o, const float *d_state_out,
                                   void *dq, void *dk, void *dv, float *d_log_decay, float *d_state0,
                                   void *workspace, size_t ws_bytes, void *stream);

/*
 * One decode step for N = desc->batch sequences (desc->seqlen must be 1):
 * q, k [N,H,dk], v [N,H,dv], log_decay [N,H] or [H]; state [N,H,dk,dv] fp32
 * is read and rewritten in place; o [N,H,dv].  fp32 arithmetic.
 */
gdn2_status gdn2_linear_step(const gdn2_linear_desc *desc, const void *q, const void *k, const void *v,
                             const float *log_decay, float *state, void *o, void *stream);

/* ------------------------------------------------------------------------
 * Layer norm over the last axis, which normalises a mixer's output per head
 * or a block's input over the model width:
 *
 *     y = (x - mean) rstd * weight + bias,   rstd = 1 / sqrt(var + eps)
 *
 * Rows [rows, dim] of bf16 or fp32; weight and bias [groups, dim] (fp32 or
 * bf16, one type), row r taking row r % groups: groups = 1 shares them, and
 * groups = H with rows of [B,T,H,dim] gives each head its own.  All sums are
 * fp32 (over rows: then fp64), results rounded once.  dim 1..16384.
 */
typedef struct gdn2_norm_desc {
    int64_t rows;         /* >= 0, a multiple of groups */
    int64_t groups;       /* >= 1 */
    int64_t dim;          /* 1..16384 */
    int32_t dtype;        /* gdn2_dtype of x, y, dy, dx */
    int32_t weight_dtype; /* gdn2_dtype of weight, bias and their gradients */
    float eps;            /* >= 0 */
    int32_t reserved;     /* 0 */
} gdn2_norm_desc;

/* weight NULL: ones; bias NULL: zeros.  mean, rstd: fp32 [rows], what the
 * backward needs, or NULL.  Outputs overlap nothing else. */
gdn2_status gdn2_layer_norm_fwd(const gdn2_norm_desc *desc, const void *x, const void *weight, const void *bias,
                                void *y, float *mean, float *rstd, void *stream);

/* Device workspace, in bytes, for the row sums of gdn2_layer_norm_bwd. */
gdn2_status gdn2_layer_norm_bwd_workspace(const gdn2_norm_desc *desc, size_t *bytes);

/* Gradients of <dy, y>: dx [rows, dim]; d_weight, d_bias [groups, dim]
 * (either may be NULL), each summed in a fixed order.  The workspace
 * (256-byte aligned) may be NULL when both are.  rows == 0: the sums are 0. */
gdn2_status gdn2_layer_norm_bwd(const gdn2_norm_desc *desc, const void *dy, const void *x, const void *weight,
                                const float *mean, const float *rstd, void *dx, void *d_weight, void *d_bias,
                                void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Rotary positions and norms of queries and keys: what stands in front of a
 * mixer.  Every head's first `rotary` channels hold pairs (u, v), which turn
 * by the token's position times the pair's frequency,
 *
 *     u' = m (cos(t) u - sin(t) v),   v' = m (sin(t) u + cos(t) v),
 *     t  = position * freq[j],        m  = magnitude
 *
 * for j = 0 .. rotary/2 - 1; the other channels pass.  The norms divide each
 * token's q and k of each head by r and multiply by a weight first:
 *
 *     GDN2_QK_RMS: r = sqrt(mean x^2 + eps),   GDN2_QK_L2: r = sqrt(sum x^2)
 *
 * over the `dim` channels (eps takes no part in GDN2_QK_L2); a row of zeros
 * stays zero, with a zero gradient where r is 0.
 *
 * q [tokens, q_heads, dim] and k [tokens, k_heads, dim] (k_heads may be 0)
 * are read with q_stride and k_stride elements between tokens, so that they
 * may be slices of one fused projection; everything written is contiguous.
 * Gradients read by gdn2_rotary_bwd take the strides too, those read by
 * gdn2_qk_norm_bwd are contiguous.  Token r stands at position
 *     offset + positions[r % period]     (positions: device int32 [period])
 *     offset + r % period                (positions NULL)
 * so period = tokens gives every token its own and period = T with tokens =
 * B * T shares them among the batch.  freq: device fp64 [rotary/2], radians a
 * position; an angle keeps its part of a turn to 2^-50 for up to 2^50 turns, so
 * far positions lose nothing.
 * Arithmetic is fp32 (a norm's sum of squares that leaves [2^-80, 2^100], and
 * its 1/r, fp64: values of any size), results are rounded once.  A row of zeros
 * without eps stays zero.
 */
typedef enum gdn2_rotary_layout {
    GDN2_ROTARY_HALF = 0,       /* pairs (x[j], x[j + rotary/2]) */
    GDN2_ROTARY_INTERLEAVED = 1 /* pairs (x[2j], x[2j + 1])      */
} gdn2_rotary_layout;

typedef enum gdn2_qk_norm { GDN2_QK_NONE = 0, GDN2_QK_RMS = 1, GDN2_QK_L2 = 2 } gdn2_qk_norm;

typedef struct gdn2_rotary_desc {
    int64_t tokens;       /* 0 .. 2^31 - 1, a multiple of period */
    int64_t period;       /* >= 1 */
    int64_t q_heads;      /* >= 1, up to 65535 */
    int64_t k_heads;      /* >= 0, up to 65535; 0: no k */
    int64_t dim;          /* channels of a head, 1..256 */
    int64_t rotary;       /* channels that turn: even, 0..dim (0: norm alone) */
    int64_t q_stride;     /* elements from token to token, >= q_heads * dim */
    int64_t k_stride;     /* the same of k, >= k_heads * dim */
    int64_t offset;       /* added to every position, within +-2^40 */
    int32_t dtype;        /* gdn2_dtype of q, k, the outputs and their gradients */
    int32_t weight_dtype; /* gdn2_dtype of the weights and their gradients */
    int32_t layout;       /* gdn2_rotary_layout */
    int32_t norm;         /* gdn2_qk_norm: NONE for gdn2_rotary_*, else RMS or L2 */
    float eps;            /* of GDN2_QK_RMS, >= 0 */
    float magnitude;      /* finite */
} gdn2_rotary_desc;

/* The rotation alone.  q_out may be exactly q where q is contiguous
 * (q_stride = q_heads * dim), and k_out k; outputs overlap nothing else. */
gdn2_status gdn2_rotary_fwd(const gdn2_rotary_desc *desc, const void *q, const void *k, const double *freq,
                            const int32_t *positions, void *q_out, void *k_out, void *stream);

/* Its gradients: d_q_out, d_k_out (with the strides) turned back into dq, dk;
 * in place as above. */
gdn2_status gdn2_rotary_bwd(const gdn2_rotary_desc *desc, const void *d_q_out, const void *d_k_out, const double *freq,
                            const int32_t *positions, void *dq, void *dk, void *stream);

/* Norm, weight [dim] (NULL: ones; shared by the heads) and rotation in one
 * pass; in place as above.  freq may be NULL where rotary is 0. */
gdn2_status gdn2_qk_norm_fwd(const gdn2_rotary_desc *desc, const void *q, const void *k, const void *q_weight,
                             const void *k_weight, const double *freq, const int32_t *positions, void *q_out,
                             void *k_out, void *stream);

/* Device workspace, in bytes, for the sums of gdn2_qk_norm_bwd. */
gdn2_status gdn2_qk_norm_bwd_workspace(const gdn2_rotary_desc *desc, size_t *bytes);

/* Gradients of <d_q_out, q_out> + <d_k_out, k_out>: dq, dk (contiguous) and
 * d_q_weight, d_k_weight [dim] (either may be NULL), summed in a fixed order.
 * q, k are the forward's inputs.  The workspace (256-byte aligned) may be NULL
 * when both weight gradients are.  Outputs overlap nothing else.  No tokens:
 * the weight gradients are 0. */
gdn2_status gdn2_qk_norm_bwd(const gdn2_rotary_desc *desc, const void *d_q_out, const void *d_k_out, const void *q,
                             const void *k, const void *q_weight, const void *k_weight, const double *freq,
                             const int32_t *positions, void *dq, void *dk, void *d_q_weight, void *d_k_weight,
                             void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * A gated linear recurrence over channels, the mixer whose state is one value
 * a channel (linear attention without a key axis):
 *
 *     h_t = a_t h_{t-1} + w_t x_t,   y_t = h_t,   a_t = exp(log_decay_t)
 *
 * for each of `dim` channels, with w = 1, or w = 1 - a (desc->complement).
 * With desc->gate_logits the gate holds logits g instead: log a = -softplus(g)
 * as elsewhere in this file, so a = sigmoid(-g), 1 - a = sigmoid(g), and the
 * gradient is that of the logits.
 *
 * x, y [B,T,dim] (dtype), log_decay [B,T,dim] (gate_dtype), states [B,dim]
 * fp32.  Products, sums and states are fp32 in a fixed order, so results are
 * the same, bit for bit, on every run; results of fewer bits are rounded once.
 *
 * For the backward, the forward leaves the state that enters every 128th
 * token (its marks): [B, ceil(T/128), dim] fp32, row j the state that token
 * 128 j multiplies by its decay (token 0: the initial state).  Packed:
 * [ceil(T/128), dim], counted along the packed axis.
 *
 * Preconditions not checked: all values finite, log_decay <= 0 (minus infinity
 * is allowed and clears the state).
 *
 * GDN2_ERR_UNSUPPORTED: a sequence of 2^31 tokens or more, 2^31 or more
 * sequences, 2^21 or more channels, 2^22 - 32 or more blocks of 64 channels over
 * all sequences (packed: over the axis), 2^31 or more of their tiles of 128 tokens, or 2^29
 * or more values in the states of packed sequences.
 */
typedef struct gdn2_scan_desc {
    int64_t batch;       /* B >= 0 (packed: N sequences)            */
    int64_t seqlen;      /* T >= 0 (packed: tokens of the one axis) */
    int64_t dim;         /* channels >= 1 */
    int32_t dtype;       /* gdn2_dtype of x, y and their gradients */
    int32_t gate_dtype;  /* gdn2_dtype of log_decay and its gradient */
    int32_t gate_logits; /* nonzero: log_decay holds logits */
    int32_t complement;  /* nonzero: w = 1 - a, else w = 1 */
} gdn2_scan_desc;

/* Device workspace, in bytes, for gdn2_scan_fwd; 0 where it needs none. */
gdn2_status gdn2_scan_fwd_workspace(const gdn2_scan_desc *desc, size_t *bytes);

/*
 * Forward over whole sequences.
 *   state0     [B,dim] fp32, or NULL for zeros
 *   y          [B,T,dim]
 *   state_out  [B,dim] fp32, or NULL; it may be exactly state0
 *   marks      see above, or NULL
 *   workspace  >= gdn2_scan_fwd_workspace() bytes, 256-byte aligned, its
 *              contents undefined before and after; NULL where that is 0.
 *              Calls that share one must not overlap in time.
 * Outputs overlap nothing else.  T == 0: state_out receives state0 (or zeros).
 */
gdn2_status gdn2_scan_fwd(const gdn2_scan_desc *desc, const void *x, const void *log_decay, const float *state0,
                          void *y, float *state_out, float *marks, void *workspace, size_t ws_bytes, void *stream);

gdn2_status gdn2_scan_fwd_varlen_workspace(const gdn2_scan_desc *desc, size_t *bytes);

/* The forward over N = desc->batch sequences packed along one axis of T
 * tokens: x, log_decay, y [T,dim], states [N,dim], cu_seqlens as for
 * gdn2_linear_fwd_varlen (clamped, so no access leaves the buffers).  Rows of
 * y, and of marks, outside every sequence are untouched; an empty sequence
 * passes its state through. */
gdn2_status gdn2_scan_fwd_varlen(const gdn2_scan_desc *desc, const int32_t *cu_seqlens, const void *x,
                                 const void *log_decay, const float *state0, void *y, float *state_out, float *marks,
                                 void *workspace, size_t ws_bytes, void *stream);

gdn2_status gdn2_scan_bwd_workspace(const gdn2_scan_desc *desc, size_t *bytes);

/*
 * Backward of gdn2_scan_fwd: the gradients of <dy, y> + <d_state_out, h_T>.
 *   marks        as the forward left them
 *   state0       the forward's, or NULL for zeros
 *   d_state_out  [B,dim] fp32, or NULL for zeros
 *   dx           like x;  d_log_decay like log_decay
 *   d_state0     [B,dim] fp32, or NULL to skip
 * Outputs overlap nothing else.  T == 0: d_state0 receives d_state_out (or
 * zeros).
 */
gdn2_status gdn2_scan_bwd(const gdn2_scan_desc *desc, const void *dy, const void *x, const void *log_decay,
                          const float *marks, const float *state0, const float *d_state_out, void *dx,
                          void *d_log_decay, float *d_state0, void *workspace, size_t ws_bytes, void *stream);

gdn2_status gdn2_scan_bwd_varlen_workspace(const gdn2_scan_desc *desc, size_t *bytes);

/* Backward of gdn2_scan_fwd_varlen; rows of dx and d_log_decay outside every
 * sequence are untouched. */
gdn2_status gdn2_scan_bwd_varlen(const gdn2_scan_desc *desc, const int32_t *cu_seqlens, const void *dy, const void *x,
                                 const void *log_decay, const float *marks, const float *state0,
                                 const float *d_state_out, void *dx, void *d_log_decay, float *d_state0,
                                 void *workspace, size_t ws_bytes, void *stream);

/* One decode step for N = desc->batch sequences (desc->seqlen must be 1): x,
 * log_decay, y [N,dim]; state [N,dim] fp32 is read and rewritten in place.  y
 * overlaps nothing else. */
gdn2_status gdn2_scan_step(const gdn2_scan_desc *desc, const void *x, const void *log_decay, float *state, void *y,
                           void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN2_H */
