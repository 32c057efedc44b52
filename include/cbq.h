/*
 * cbq.h -- C ABI of the codebook-4bit quantized matvec library (libcbq.so).
 *
 * The library computes the low-bit quantized matrix-vector product that
 * streams 4-bit codebook weights for single-token decode and for small-batch
 * speculative verification (n = 1..5 activation columns), over dense
 * projections and over top-k routed MoE experts with the SwiGLU split and the
 * router-weighted combine fused in.  Every step runs in CUDA kernels built for
 * sm_103a; there is no CPU fallback.
 *
 * Sources of each operation (pages: the lucebox pull requests about the
 * DeepSeek-V4-Flash "DS4" server):
 *   - quant type + CPU reference conversion: "feat(ds4): add DSpark speculative
 *     runtime + optimizations" #496, summary bullet "ROCmFP4/ROCmFPX quant types
 *     + CPU reference conversions";
 *   - MMVQ vecdot / MMVQ kernel over ne1 columns, MMVQ_MAX_MOE_BATCH_SIZE: same
 *     summary ("CUDA/HIP dequant, copy, getrows, MMVQ vecdot, MMVF ...");
 *   - codebook-16 expander: "fix(ggml): make ROCmFP4 codebook self-contained on
 *     CUDA" (commit on "fix(ds4): correct layer-split HC handoff and per-device
 *     state" #507);
 *   - SwiGLU split for the fused FFN matvec paths: #496 summary, "DS4 SwiGLU
 *     split op plumbing";
 *   - routed-expert top-k and the fused expert-FFN combine: "fix(ds4): keep
 *     ROCmFPX generation byte-safe" #494 (DFLASH_DS4_FFN_FUSED_COMBINE) and
 *     "feat(ds4): add DSpark speculative decoding" (configured routed-expert
 *     top-k, fused batched verification).
 *
 * Weight format ("canonical blocks"): a matrix of M rows x K columns
 * (K % 32 == 0) is M x (K/32) blocks, row-major, 18 bytes per block:
 *   bytes 0-1  fp16 scale dw, little-endian;
 *   bytes 2-17 index bytes qs: byte j holds the codebook index of element j
 *              in its low nibble and of element j+16 in its high nibble;
 *   weight_i = dw * codebook[index_i], codebook = {-127,-104,-83,-65,-49,-35,
 *              -22,-10,1,13,25,38,53,69,89,113}.
 *
 * Activation quantization (per 32 consecutive values of one column):
 *   d = max|x| / 127 (fp32), q = round-half-to-even(x / d) clamped to
 *   [-127,127], q = 0 when d == 0.  Inputs are assumed finite.
 *
 * Conventions for every entry point:
 *   - returns CBQ_OK (0) or a negative cbq_status; argument errors are
 *     reported before anything is launched;
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream); work is enqueued on it and the call returns without waiting,
 *     except where a function says it synchronizes;
 *   - pointers named *_dev are device pointers owned by the caller; the
 *     library only reads inputs and writes outputs within the stated sizes;
 *   - a handle owns its device memory (repacked weights and a workspace) and
 *     remembers its device; calls switch to that device and restore the
 *     caller's current device before returning;
 *   - the workspace of a handle is shared by its calls: two calls on one
 *     handle that overlap on the GPU (different streams without ordering)
 *     race.  Calls on one stream are ordered and safe;
 *   - kernels are launched as programmatic dependents (programmatic stream
 *     serialization) where that hides launch latency: such a kernel may
 *     become resident before the work ahead of it on the stream has ended,
 *     but it reads an input of the call or a counter of a handle only once
 *     all work enqueued before the call has ended (the call's first kernel
 *     waits for it with griddepcontrol.wait before it lets the call's next
 *     kernel start), so results are those of plain stream order, also after
 *     a caller's kernel that signals its dependents early;
 *   - no call allocates or frees device memory except *_create, *_destroy
 *     and cbq_moe_set_shared (which allocates the shared expert's weights the
 *     first time, frees them on removal, and uses a temporary device buffer
 *     for host blocks);
 *   - errors found by a kernel while it runs (an expert id out of range, a
 *     bounded wait that gave up) set bits in an error word that belongs to
 *     the handle; cbq_weights_get_error / cbq_moe_get_error read and clear it
 *     in the order of a stream.  Outputs of a call that set a *_TIMEOUT bit
 *     are undefined.
 */
#ifndef CBQ_H
#define CBQ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CBQ_QK 32            /* weights per block */
#define CBQ_BLOCK_BYTES 18   /* bytes per canonical block */
#define CBQ_MAX_COLS 5       /* activation columns per matvec (decode + verify q<=4) */
#define CBQ_MAX_TOKENS 5     /* tokens per MoE call */
#define CBQ_MAX_TOPK 16      /* routed experts per token */

typedef enum {
    CBQ_OK = 0,
    CBQ_EINVAL = -1,   /* bad argument (null pointer, size, count) */
    CBQ_ECUDA = -2,    /* a CUDA runtime call or a launch failed */
    CBQ_ENOMEM = -3,   /* device allocation failed in a *_create */
    CBQ_EDEVICE = -4   /* no usable sm_103 device */
} cbq_status;

/* Bits of a handle's error word (cbq_weights_get_error, cbq_moe_get_error). */
#define CBQ_DEVERR_BAD_EXPERT_ID 0x1u          /* an id outside [0,E): that slot was skipped */
#define CBQ_DEVERR_PIPE_TIMEOUT 0x100u         /* a weight-stream wait gave up after 1 s */
#define CBQ_DEVERR_DEPENDENCY_TIMEOUT 0x200u   /* a down-projection item gave up waiting 1 s for its
                                                  expert's intermediate; its outputs were not written */

typedef struct cbq_weights cbq_weights; /* one dense M x K matrix, repacked on device */
typedef struct cbq_moe cbq_moe;         /* E experts: gate_up (2F x H) and down (H x F) */

/* Human-readable name of a cbq_status. */
const char *cbq_status_string(int status);

/* Text of the last CUDA error seen by this thread ("" if none). */
const char *cbq_last_cuda_error(void);

/* Create a dense weight handle on the current device from canonical blocks
 * `blocks` (M*(K/32)*18 bytes; host memory if on_device == 0, else device
 * memory).  The blocks are repacked into the device layout (16-byte index
 * stream interleaved by 32-row groups plus a separate fp16 scale stream); the
 * source is not retained.  Synchronizes `stream`.
 * K is bounded by the shared-memory staging of CBQ_MAX_COLS quantized
 * activation columns next to a four-stage weight ring and the partial-sum
 * set: K <= 27,136 on GB300 (227 KB of shared memory per CTA).
 * Errors: EINVAL (null, M < 1, K < 32, K % 32 != 0, K above that bound),
 * ENOMEM, ECUDA, EDEVICE. */
int cbq_weights_create(const void *blocks, int64_t M, int64_t K, int on_device,
                       void *stream, cbq_weights **out);
int cbq_weights_destroy(cbq_weights *W);

/* Shape of a handle and the device bytes it holds (any pointer may be NULL). */
int cbq_weights_info(const cbq_weights *W, int64_t *M, int64_t *K, int64_t *device_bytes);

/* Activation quantization (pages: activation side of the MMVQ vecdot).
 * x_dev: n x K fp32, row-major (column c at x_dev + c*K); K % 32 == 0; n >= 1.
 * qx_dev: n x K int8 out; dx_dev: n x (K/32) fp32 out.
 * Bit-exact with the rule in the header comment. */
int cbq_quantize_act(const float *x_dev, int64_t K, int n, int8_t *qx_dev, float *dx_dev,
                     void *stream);

/* Quantized matvec from already-quantized activations (MMVQ with ne1 = n).
 * qx_dev: n x K int8, dx_dev: n x (K/32) fp32 (layout of cbq_quantize_act);
 * y_dev: n x M fp32 out, y[c][r] = sum_b dw(r,b) * dx[c][b] * s(r,b,c) where
 * s is the exact int32 block dot.  1 <= n <= CBQ_MAX_COLS.  All n columns are
 * computed in one pass over the weights. */
int cbq_matvec_q(const cbq_weights *W, const int8_t *qx_dev, const float *dx_dev, int n,
                 float *y_dev, void *stream);

/* The whole dense path: quantize x_dev (n x K fp32) with the rule of
 * cbq_quantize_act, then the matvec of cbq_matvec_q into y_dev (n x M fp32);
 * the result has the same bits as those two calls.  For n == 1 with x_dev
 * 16-byte aligned this is one kernel launch (the matvec kernel quantizes x
 * while its weight stream starts); otherwise the quantization kernel writes
 * the handle's workspace first and the matvec kernel follows it as a
 * programmatic dependent.  One call at a time per handle. */
int cbq_matvec(const cbq_weights *W, const float *x_dev, int n, float *y_dev, void *stream);

/* Same with HOST buffers: copies x (n x K fp32) to the device, runs
 * cbq_matvec and copies y (n x M fp32) back, then synchronizes `stream`.
 * Pinned host memory makes the copies asynchronous to the host. */
int cbq_matvec_host(const cbq_weights *W, const float *x_host, int n, float *y_host,
                    void *stream);

/* Create an MoE layer handle from canonical blocks of E experts, contiguous
 * per expert: gate_up = E x (2F rows x H cols), rows 0..F-1 the gate
 * projection and rows F..2F-1 the up projection; down = E x (H rows x F cols).
 * H % 32 == 0, F % 32 == 0, E >= 1, H and F <= 1,048,576.  Host memory if
 * on_device == 0.
 * Synchronizes `stream`.  Errors as cbq_weights_create. */
int cbq_moe_create(const void *gate_up, const void *down, int E, int64_t H, int64_t F,
                   int on_device, void *stream, cbq_moe **out);
int cbq_moe_destroy(cbq_moe *L);

/* Give the layer a shared expert: one more gate_up (2F x H) and down (H x F)
 * pair in canonical blocks, the same shapes as a routed expert, that every
 * token passes through with weight 1 in each later cbq_moe_matvec* call:
 *   y_t = sum_j wts[t][j] * o_{ids[t][j]}(h_t) + o_sh(h_t),
 * o_sh computed exactly as a routed slot (SwiGLU split, requantization, down)
 * and added after the routed sum.  The pages name only the routed layer
 * ("feat(ds4): add DSpark speculative decoding" routes each token to its
 * configured top-k); the always-on expert of the DS4 FFN block is read here
 * as one more expert of the same shape.  Its weights are read once per call,
 * in the same layer kernel, like any routed expert.  Host memory if
 * on_device == 0; the blocks are repacked and not retained.  gate_up == down
 * == NULL removes the shared expert.  Synchronizes `stream` first (a call
 * still running on another stream must have ended).
 * Errors: EINVAL (exactly one of gate_up, down NULL), ENOMEM, ECUDA. */
int cbq_moe_set_shared(cbq_moe *L, const void *gate_up, const void *down, int on_device, void *stream);

int cbq_moe_info(const cbq_moe *L, int *E, int64_t *H, int64_t *F, int64_t *device_bytes);

/* Routed-expert FFN (mul_mat_id with the SwiGLU split and the weighted
 * combine fused).  h_dev: n_tok x H fp32; ids_dev: n_tok x topk int32 expert
 * ids; wts_dev: n_tok x topk fp32 router weights; y_dev: n_tok x H fp32 out.
 * For every token t and slot j (slot order), expert e = ids[t][j]:
 *   g,u = gate/up rows of e applied to quantize(h_t);
 *   a = swiglu ? silu(g)*u : g*u (fp32), silu(z) = z/(1+exp(-z));
 *   o = down_e applied to quantize(a);  y_t = sum_j wts[t][j] * o.
 * Tokens are grouped by expert on the device: each distinct expert's bytes
 * are read once per call for all of its tokens.  Ids should be distinct per
 * token; a repeated id is served as an extra column and summed on its own.
 * An id outside [0,E) skips its slot and sets CBQ_DEVERR_BAD_EXPERT_ID.
 * The sum over j runs in slot order (deterministic, no atomics on y).
 * With a shared expert (cbq_moe_set_shared) its output is added last.
 * Three kernel launches on `stream`, each a programmatic dependent of the one
 * before: the token quantization, the layer kernel (gate_up, SwiGLU,
 * requantization, down), the combine.  With one token the layer kernel forms
 * the combine itself (same order, same bits), and with h_dev also 16-byte
 * aligned it quantizes the token itself too (same bits): one launch.  One
 * call at a time per handle (its workspace and counters are shared by the
 * calls).
 * 1 <= n_tok <= CBQ_MAX_TOKENS, 1 <= topk <= min(CBQ_MAX_TOPK, E). */
int cbq_moe_matvec(const cbq_moe *L, const float *h_dev, int n_tok, const int32_t *ids_dev,
                   const float *wts_dev, int topk, int swiglu, float *y_dev, void *stream);

/* Largest expert count of the router entry points (its logits are staged in
 * shared memory). */
#define CBQ_ROUTER_MAX_E 16384

/* Routed-expert selection from router logits: logits_dev n_tok x E fp32;
 * for every token t, ids_dev[t][0..topk) = the indices of the topk largest
 * logits in descending order (equal logits: lower index first) and
 * wts_dev[t][j] = softmax over those topk logits, computed in fp64 and
 * rounded to fp32.  The pages name a "configured routed-expert top-k"
 * ("feat(ds4): add DSpark speculative decoding") without a formula; this is
 * the plain reading.  Logits must be finite.  1 <= n_tok <= 65535,
 * 1 <= E <= CBQ_ROUTER_MAX_E, 1 <= topk <= min(CBQ_MAX_TOPK, E).  One kernel
 * launch on `stream`; the caller owns every buffer. */
int cbq_router_topk(const float *logits_dev, int n_tok, int E, int topk, int32_t *ids_dev, float *wts_dev,
                    void *stream);

/* The weight converter: a row-major M x K fp32 matrix on the device to the
 * M x (K/32) canonical 18-byte blocks that cbq_weights_create and
 * cbq_moe_create read (on_device = 1).  The pages name "CPU reference
 * conversions" of the quant types ("feat(ds4): add DSpark speculative
 * runtime + optimizations" #496) without a rule; this is the plain reading,
 * per block of 32 weights:
 *   m = the weight of largest magnitude (the first among equal ones);
 *   scale = binary16(m / -127): IEEE fp32 division, then rounding to nearest
 *           even (-127 is the codebook level of largest magnitude, so m lands
 *           on it); an all-zero block gives 18 zero bytes;
 *   index_i = the level j whose reconstruction scale * codebook[j] is nearest
 *           to w_i, the lowest j among equal distances (index 0 everywhere
 *           when the scale rounds to zero).
 * The decisions are exact (no rounding can move a weight to another level),
 * so the bytes are the same on every run.  Weights must be finite with
 * |m| < 127 * 65520 (a finite scale).  w_dev 16-byte aligned, blocks_dev
 * 2-byte aligned, both owned by the caller; M >= 1, K >= 32, K % 32 == 0,
 * else CBQ_EINVAL.  One kernel launch on `stream`. */
int cbq_quantize_weights(const float *w_dev, int64_t M, int64_t K, void *blocks_dev, void *stream);

/* Streams of the hyper-connection state (the NHC of the pages' NHC = 4
 * specialisation), and the most normalisation rounds one call accepts. */
#define CBQ_HC_NHC 4
#define CBQ_HC_MAX_ITERS 1024
#define CBQ_HC_MAX_N (1ll << 28)

/* Sinkhorn normalisation of the hyper-connection mixing matrices (the
 * register-resident sinkhorn kernel of the fused DS4 hyper-connection op,
 * "feat(ds4): add DSpark speculative runtime + optimizations" #496, in its
 * NHC = 4 form, "fix(ds4): keep ROCmFPX generation byte-safe" #494).  The
 * pages give neither the iteration count nor the update; the plain reading
 * of a Sinkhorn normalisation is used.  For each of the n row-major
 * CBQ_HC_NHC x CBQ_HC_NHC matrices c of fp32 logits at logits_dev:
 *   P = exp(c - max c);
 *   `iters` rounds of: every row of P scaled to sum 1, then every column
 *   (a sum in index order, times its reciprocal from the hardware
 *   approximation, within 1 ulp);
 *   out_dev = P after the last round (columns sum to 1 within rounding; rows
 *   approach 1 as the rounds converge); iters = 0 gives exp(c - max c).
 * The result agrees with an fp64 evaluation of the same rounds within
 * (8 + 16 * iters) * 2^-24 per entry.  In contract: finite logits whose
 * spread within a matrix (max - min) is at most 80, so every entry stays a
 * normal fp32 number.  Arguments: both pointers 16-byte aligned (out_dev may
 * equal logits_dev: each matrix is read before it is written; otherwise the
 * buffers must not overlap); 1 <= n <= CBQ_HC_MAX_N; 0 <= iters <=
 * CBQ_HC_MAX_ITERS; else CBQ_EINVAL.  One kernel launch on `stream` (a
 * programmatic dependent of the work ahead, like every kernel here), one
 * thread per matrix; the caller owns both buffers. */
int cbq_hc_sinkhorn(const float *logits_dev, int64_t n, int iters, float *out_dev, void *stream);

/* cbq_router_topk into the handle's staging buffers, then cbq_moe_matvec with
 * those ids and weights: the routed layer from router logits with no host
 * round trip (one launch more than cbq_moe_matvec).  Same limits as both. */
int cbq_moe_matvec_logits(const cbq_moe *L, const float *h_dev, int n_tok, const float *logits_dev, int topk,
                          int swiglu, float *y_dev, void *stream);

/* Same with HOST buffers (h, ids, wts in; y out), then synchronizes `stream`. */
int cbq_moe_matvec_host(const cbq_moe *L, const float *h_host, int n_tok,
                        const int32_t *ids_host, const float *wts_host, int topk, int swiglu,
                        float *y_host, void *stream);

/* Stage timing: when set, cbq_moe_matvec records these CUDA events
 * (cudaEvent_t passed as void*) on its stream before its first kernel,
 * before the layer kernel (right after ev_start when the layer kernel
 * quantizes the one token itself; else after the token quantization) and
 * after the call's last kernel (the layer kernel, or the combine).  Recording them separates the kernels (the overlap
 * of a kernel's start with the previous one's end is lost).  Pass NULL for
 * all three to stop; a mix of NULL and non-NULL is CBQ_EINVAL.  The events
 * stay owned by the caller. */
int cbq_moe_set_stage_events(cbq_moe *L, void *ev_start, void *ev_layer, void *ev_end);

/* ---- tensor-core path for larger batches ------------------------------ */

/* Most columns of cbq_matmat. */
#define CBQ_MAX_MMQ_COLS 16

/* The dense product for 1 <= n <= CBQ_MAX_MMQ_COLS columns on the tensor
 * cores (tcgen05): the MMQ tile the pages name for larger batches ("#497
 * RDNA MMQ tile, LUCE_MMQ_DP_MAX_NE1", "fix(ds4): correct layer-split HC
 * handoff and per-device state" #507), read for this format.  Same result
 * definition as cbq_matvec (the activation quantization, exact per-block
 * integer dots, y = sum_b dw*dx*s in fp32 with the same three roundings per
 * block); the blocks, in units of four, alternate between two running sums
 * added at the end of the row: every block dot is exact, so y is within the
 * same bound of the plain definition.  A level enters the MMA as
 * the fp16 value 1152 + level, an int8 activation as fp16; each 32-wide block
 * sum is an integer below 2^24 (exact in the fp32 accumulator), and the bias
 * 1152 * sum q is subtracted exactly.  Arguments as cbq_matvec (x_dev n x K
 * fp32, y_dev n x M fp32, both owned by the caller).  Three launches on
 * `stream`: the quantization, the B tiles, the tiles of W.  One call at a
 * time per handle (its workspace is shared by the calls). */
int cbq_matmat(const cbq_weights *W, const float *x_dev, int n, float *y_dev, void *stream);

/* Checking: the exact block dots s[c][r][b] (n x M x K/32 int32) of W's
 * blocks with the int8 columns qx_dev (n x K), taken by the tensor-core path
 * (cbq_debug_block_dots takes them by the dp4a path).  1 <= n <=
 * CBQ_MAX_MMQ_COLS. */
int cbq_debug_mmq_block_dots(const cbq_weights *W, const int8_t *qx_dev, int n, int32_t *s_dev, void *stream);

/* ---- allocation-free dense path --------------------------------------- */

/* Largest K cbq_matvec_static accepts (its scratch holds CBQ_MAX_COLS columns
 * of this many quantized values plus their scales: 92,160 bytes per device). */
#define CBQ_STATIC_SCRATCH_MAX_K 16384

/* cbq_matvec for callers that must not allocate device memory while they run,
 * e.g. hosts that fix their device memory budget at start-up and forbid
 * allocation afterwards.  The pages describe no counterpart; it is the dense
 * path of cbq_matvec with one difference: with more than one column, or x_dev
 * not 16-byte aligned, the quantized activations go to a scratch array the
 * library declares statically on every device (it lives as long as the
 * library is loaded), not to the handle's workspace; one aligned column is
 * quantized inside the matvec kernel (one launch), as cbq_matvec does, and
 * needs no scratch.  Nothing is allocated or freed, here or in any library
 * routine it calls.  Same bits as cbq_matvec.
 *   - Arguments as cbq_matvec; K of W must be <= CBQ_STATIC_SCRATCH_MAX_K,
 *     else CBQ_EINVAL (checked before anything runs).
 *   - The first call on a device looks the scratch array up on that device
 *     (cudaGetSymbolAddress).
 *   - The scratch is one array per device shared by every call of this entry
 *     point on that device, whatever the handle: calls that may overlap on the
 *     GPU (different streams without ordering) race.  Every call rewrites the
 *     part it reads, so no contents carry over from the previous call. */
int cbq_matvec_static(const cbq_weights *W, const float *x_dev, int n, float *y_dev, void *stream);

/* Read the error word of a handle (bits CBQ_DEVERR_*: every error of the
 * handle's calls since the last read) into *code and clear it.  The copy and
 * the clear are enqueued on `stream`, which is then synchronized (no other
 * stream or device-wide synchronization): calls enqueued on `stream` before
 * this one are covered, and a call on another stream is covered once it is
 * ordered before `stream` (an event, or a synchronization).  Errors: EINVAL
 * (null), ECUDA. */
int cbq_weights_get_error(const cbq_weights *W, void *stream, unsigned int *code);
int cbq_moe_get_error(const cbq_moe *L, void *stream, unsigned int *code);

/* ---- between the products: positions, attention, sampling --------------
 *
 * What a verify step needs between its quantized products: the new tokens'
 * rotary positions and their way into a paged cache, the attention of a tree
 * of drafted tokens over that cache, and a token from each row of logits.
 * These calls take no handle: every buffer, the workspace included, is the
 * caller's, and errors found while a kernel runs are ORed into *err_dev
 * (a caller's device word, zeroed by the caller; NULL: not reported).  They
 * run on the current device.  Strides are in elements. */

typedef enum {
    CBQ_F32 = 0,
    CBQ_BF16 = 1,
    CBQ_F16 = 2
} cbq_dtype;

#define CBQ_DEVERR_BAD_SLOT 0x2u    /* a cache slot or page outside the cache: not written, or not seen */
#define CBQ_DEVERR_BAD_LENGTH 0x4u  /* a sequence's tokens or length beyond the call's limits: cut to them */

/* A paged cache of keys and values, on the device and the caller's.  Token t
 * of page p of kv head h has its head_dim values of k at
 * k + p*page_stride + t*tok_stride + h*head_stride (contiguous), and v alike.
 * dtype CBQ_BF16 or CBQ_F16; 1 <= head_dim <= 256; page_size >= 1;
 * n_pages * page_size < 2^31; strides >= 0. */
typedef struct cbq_kv_cache {
    void *k;
    void *v;
    int dtype;
    int kv_heads;
    int head_dim;
    int page_size;
    int64_t n_pages;
    int64_t page_stride;
    int64_t tok_stride;
    int64_t head_stride;
} cbq_kv_cache;

/* How the rotary frequencies are scaled for contexts longer than orig_len. */
#define CBQ_ROPE_NONE 0
#define CBQ_ROPE_LINEAR 1
#define CBQ_ROPE_BY_TURNS 2
#define CBQ_ROPE_BY_INDEX 3
/* Which values of the rotated part form pair i: (i, i + rot_dim/2), or
 * (2i, 2i + 1). */
#define CBQ_ROPE_HALF 0
#define CBQ_ROPE_PAIRS 1
#define CBQ_ROPE_MAX_DIM 1024 /* largest head_dim of cbq_rope */

/* The table of a rotation, on the host: turns_host[i], i < rot_dim/2, is how
 * many turns pair i makes from one position to the next,
 *   t_i = base^(-2i/rot_dim) / (2 pi), scaled as `scaling` says:
 *   NONE      t_i;
 *   LINEAR    t_i / factor;
 *   BY_TURNS  g t_i + (1-g) t_i/factor, g = clamp((t_i*orig_len - low) /
 *             (high - low), 0, 1): pairs that make `high` turns or more over
 *             orig_len positions stay, those under `low` are divided;
 *   BY_INDEX  the same mix with g falling linearly in the index i, from 1 at
 *             max(floor(i(high)), 0) to 0 at min(ceil(i(low)), rot_dim - 1),
 *             where i(r) = ln(orig_len / (2 pi r)) rot_dim / (2 ln base) is
 *             the index whose pair makes r turns over orig_len (the end may
 *             lie past the rot_dim/2 pairs: then none is divided whole).  The
 *             method is YaRN's (Peng et al., 2023), with its beta_slow as
 *             low, beta_fast as high, and 0.1 ln(factor) + 1 as cbq_rope's
 *             mscale.
 * In fp64.  The unused parameters of a scaling are ignored.
 * Errors: EINVAL (null, rot_dim < 2, odd or > CBQ_ROPE_MAX_DIM, base <= 1 or
 * not finite, factor <= 0, orig_len <= 0, not 0 < low < high). */
int cbq_rope_turns(int rot_dim, double base, int scaling, double factor, double orig_len, double low, double high,
                   double *turns_host);

/* Rotary positions of x_dev: n_tok x heads x head_dim of `dtype`, value d of
 * head h of token t at x_dev + t*x_tok_stride + h*x_head_stride + d; out_dev
 * alike with its strides.  In each head the pairs (a, b) of the rot_dim
 * values from rot_off on become
 *   mscale * (a cos r - b sin r, a sin r + b cos r), r = 2 pi pos_t turns_i,
 * the other values are copied.  pos_dev: n_tok int32; turns_dev: rot_dim/2
 * fp64 (cbq_rope_turns).  The angle is reduced to a part of a turn in fp64,
 * so far positions lose nothing; sine, cosine and the products are fp32,
 * rounded once to `dtype`.  out_dev may be x_dev (with the same strides);
 * otherwise the two must not overlap.  One launch on `stream`.
 * Errors: EINVAL (null; n_tok < 1 or > 2^24; heads < 1 or > 65535; head_dim
 * < 1 or > CBQ_ROPE_MAX_DIM; rot_dim < 2 or odd; rot_off < 0 or rot_off +
 * rot_dim > head_dim; an unknown dtype or layout; negative strides, a pointer
 * not aligned to its type, mscale not finite, in place with other strides),
 * ECUDA, EDEVICE. */
int cbq_rope(const void *x_dev, int dtype, int64_t n_tok, int heads, int head_dim, int64_t x_tok_stride,
             int64_t x_head_stride, const int32_t *pos_dev, const double *turns_dev, int rot_dim, int rot_off,
             int layout, float mscale, void *out_dev, int64_t out_tok_stride, int64_t out_head_stride, void *stream);

/* New tokens on their way to attention, in one launch: the queries q_dev
 * (n_tok x q_heads x head_dim) rotated into qout_dev (contiguous, of the
 * cache's dtype), the keys k_dev (n_tok x kv_heads x head_dim) rotated into
 * the cache, the values v_dev copied into it; all as cbq_rope, from `dtype`
 * (any cbq_dtype), rounded once to the cache's.  k_dev and v_dev share their
 * strides.  slots_dev: n_tok int64, the place of each token in the cache
 * (page * page_size + token within it); a negative slot writes nothing, one
 * beyond the cache writes nothing and sets CBQ_DEVERR_BAD_SLOT.  Two tokens
 * with one slot race.  Errors as cbq_rope (head_dim is the cache's), and
 * EINVAL for a bad cache. */
int cbq_rope_append(const void *q_dev, const void *k_dev, const void *v_dev, int dtype, int64_t n_tok, int q_heads,
                    int64_t q_tok_stride, int64_t q_head_stride, int64_t kv_tok_stride, int64_t kv_head_stride,
                    const int32_t *pos_dev, const int64_t *slots_dev, const double *turns_dev, int rot_dim,
                    int rot_off, int layout, float mscale, const cbq_kv_cache *cache, void *qout_dev,
                    unsigned int *err_dev, void *stream);

#define CBQ_TREE_MAX 64             /* drafted tokens of one sequence per call (bits of a mask) */
#define CBQ_TREE_MAX_LEN (1 << 30)  /* largest max_len */

/* Bytes of workspace cbq_tree_attention needs for these limits (at least 16;
 * the same for every content of the device arrays).  Errors: EINVAL (null or
 * out of the ranges below). */
int cbq_tree_attention_workspace(int n_seq, int64_t total_tok, int max_tok, int64_t max_len, int q_heads,
                                 int kv_heads, int head_dim, int64_t *bytes);

/* Attention of each sequence's tree of drafted tokens over its paged cache.
 * Sequence s has ctx_dev[s] committed tokens and the n_s = start_dev[s+1] -
 * start_dev[s] drafted tokens (packed rows start_dev[s].. of q_dev; n_seq + 1
 * int32 in start_dev); draft j sits in the cache right behind the committed
 * ones, at place ctx_dev[s] + j (cbq_rope_append put it there).  Place p of
 * sequence s is token p % page_size of page table_dev[s*table_width + p /
 * page_size].  Draft i sees every committed token and those drafts j of its
 * sequence whose bit j is set in mask_dev[start_dev[s] + i]:
 *   out[i][h] = sum_p softmax_p(scale * q[i][h].k[p][g]) v[p][g],
 *   g = h / (q_heads / kv_heads);  lse[i][h] = ln sum_p exp(scale * q.k).
 * A row that sees nothing gives zeros and -inf.  What a row does not see,
 * NaN and infinities included, does not touch it; a NaN in its query or in a
 * key that it sees makes out and lse NaN.  q_dev: total_tok x q_heads
 * x head_dim of the cache's dtype, with strides; out_dev: total_tok x q_heads
 * x head_dim, contiguous, out_dtype the cache's dtype or CBQ_F32; lse_dev:
 * total_tok x q_heads fp32 or NULL.  Scores, running maxima and sums are
 * fp32; the weights are rounded to the cache's 16 bits for the product with
 * v.  max_tok and max_len bound n_s and ctx_dev[s] + n_s: they size the
 * launch; a sequence beyond them, or beyond its table, is cut to them and
 * sets CBQ_DEVERR_BAD_LENGTH; a page id outside the cache is not seen and
 * sets CBQ_DEVERR_BAD_SLOT.  The result does not depend on timing (no
 * atomics on it) but a row's last bits depend on the call's limits (n_seq,
 * max_tok, max_len and the heads), by which the work is split.  The many-row
 * kernel's roles wait for one another with a limit; a wait that runs out (1 s)
 * sets CBQ_DEVERR_PIPE_TIMEOUT and leaves its block's rows undefined.  (The
 * barriers of clusters and the allocation of tensor memory, which end as soon
 * as the blocks beside them get on, have none.)  ws_dev: 16-byte
 * aligned, ws_bytes at least what cbq_tree_attention_workspace says, one call
 * at a time.
 * Speed: heads of 64, 128 and 256 whose rows in the cache, and out_dev, begin
 * on 16 bytes take the tensor cores with the keys shared out over the GPU.
 * Every other size, stride or address is taken by a warp a row, one key after
 * another: right, and slow (5 drafts over 8,191 keys 7 to 8 ms for 15 us).
 * Errors: EINVAL (null; n_seq < 1 or > 65535; total_tok < 1 or > 2^24;
 * max_tok outside 1..CBQ_TREE_MAX; max_len outside 1..CBQ_TREE_MAX_LEN;
 * kv_heads < 1, > 256 or no divisor of q_heads; q_heads > 1024; table_width
 * < 1; scale not finite; a bad cache; a workspace too small or misaligned),
 * ECUDA, EDEVICE. */
int cbq_tree_attention(const void *q_dev, int64_t q_tok_stride, int64_t q_head_stride, int q_heads, int64_t total_tok,
                       const cbq_kv_cache *cache, const int32_t *table_dev, int table_width, int n_seq,
                       const int32_t *ctx_dev, const int32_t *start_dev, const int64_t *mask_dev, int max_tok,
                       int64_t max_len, float scale, void *out_dev, int out_dtype, float *lse_dev, void *ws_dev,
                       int64_t ws_bytes, unsigned int *err_dev, void *stream);

#define CBQ_SAMPLE_MAX_V (1 << 18)

/* One token from each of n rows of V logits (row c at logits_dev +
 * c*row_stride, `dtype` any cbq_dtype) and one given number u in [0,1) per
 * row.  With l the row's logits, T = temperature[c] and the order "larger
 * logit first, of equal ones the lower index first":
 *   w_i = exp((l_i - max l) / T);
 *   top-k  keeps the first top_k[c] of the order (<= 0 or >= V: all);
 *   top-p  keeps, of those, the shortest beginning of the order whose mass
 *          reaches top_p[c] of theirs: i stays while the mass before it is
 *          below top_p * mass (always the first; >= 1 or NaN: all);
 *   min-p  keeps, of those, w_i >= min_p[c] (always the first);
 *   ids[c] = the first index i whose cumulated kept mass, in the order of the
 *          indices, exceeds u * (kept mass);  probs[c] = w_i / kept mass.
 * T <= 0 or NaN takes the first of the order, with probability 1.  Logits of
 * -inf and NaN are never taken; if a row has nothing else, ids[c] = -1 and
 * probs[c] = 0.  Where +inf occurs only those logits have weight.  Weights
 * are 2^-45 fixed-point numbers (each within 2^-39 of its value) summed in 64
 * bits, so sums and choices are the same on every run; a weight under 2^-46
 * has no mass.  temperature, top_k, top_p and min_p may be NULL (1, all, all,
 * none); probs_dev may be NULL.  1 <= n <= 65535, 1 <= V <=
 * CBQ_SAMPLE_MAX_V, row_stride >= V or n == 1, else EINVAL. */
int cbq_sample(const void *logits_dev, int dtype, int n, int V, int64_t row_stride, const float *temperature_dev,
               const int32_t *top_k_dev, const float *top_p_dev, const float *min_p_dev, const float *u_dev,
               int32_t *ids_dev, float *probs_dev, void *stream);

/* ---- behind the logits, and the cache -----------------------------------
 *
 * The end of a verify step: the distributions of the target and the drafter,
 * the verification of the drafted trees against them, and what becomes of the
 * cache: the accepted drafts move to the end of their context, pages that are
 * full and old are kept in 8 bits, and the tree attention reads both kinds.
 * No handles, as in the section before. */

/* The distribution that cbq_sample draws from: out[c][i] = w_i / kept mass
 * where i is kept by the row's temperature, top-k, top-p and min-p, else 0
 * (the weights, the order and the cuts are cbq_sample's; a weight under 2^-46
 * has no mass).  T <= 0 or NaN gives 1 to the first of the order; a row of
 * nothing but -inf and NaN gives zeros.  out_dev: n x V fp32, row c at out_dev
 * + c*out_stride; each value is within 2^-23
 * (relative) of its quotient, and that within 2^-38 of the formula's, both
 * plus 2^-46 absolute.  u_dev and
 * ids_dev, both or neither: one token a row is drawn too, the same that
 * cbq_sample draws.  out_dev and ids_dev overlap nothing that the call reads,
 * nor each other (rows that lie in turn, the halves of one tensor's, share no
 * byte and do not).  One launch.  Errors as cbq_sample, and EINVAL (out_dev
 * null, out_stride < V with n > 1 or < 0, one of u_dev and ids_dev alone, an
 * output that overlaps). */
int cbq_probs(const void *logits_dev, int dtype, int n, int V, int64_t row_stride, const float *temperature_dev,
              const int32_t *top_k_dev, const float *top_p_dev, const float *min_p_dev, const float *u_dev,
              float *out_dev, int64_t out_stride, int32_t *ids_dev, void *stream);

/* Verification of each sequence's tree of drafted tokens by given random
 * numbers, such that what comes out is distributed as the target's own tokens.
 * Sequence s has n_s = start_dev[s+1] - start_dev[s] nodes, packed rows
 * start_dev[s].. of the arrays.  Node 0 is the sequence's last token, which is
 * settled already; node i > 0 is a drafted token tokens_dev[row], whose parent
 * is the sequence's node parent_dev[row] < i.  Row r of probs_dev (V fp32 that
 * sum to 1) is the target's distribution p of the token behind node r, and row
 * r of draft_dev the distribution q from which the children of node r were
 * drawn, each by itself.  The walk starts at node 0; at each node
 *   c = 0, S = 1;  for its children i, tokens x, in the order of the indices:
 *     u[i] * q(x) * S < p(x) - c * q(x):  i is accepted, the walk goes on there;
 *     otherwise  c = c + S,  S = sum_x max(p(x) - c * q(x), 0);
 *   where no child is accepted the walk ends with the token
 *     next = the first x with  sum_{y <= x} r(y) > u_next[s] * sum_y r(y),
 *     r(x) = max(p(x) - c * q(x), 0).
 * (Rejection by several rounds: each child is a draw from q that is tried
 * against what the ones before left over.)  draft_dev NULL: the children were
 * chosen, not drawn, and q is 1 at the child's token: it is accepted if u[i] *
 * S < r(x), otherwise x is taken out of r and S = S - r(x).  A token outside
 * [0, V) is never accepted.  If nothing is left of r (the draft equals the
 * target, and rounding refused it) the token is drawn from p; from a row of
 * zeros next is -1.  In a row of probs or draft NaN counts as 0, and so does
 * what is below 0; a u of NaN accepts nothing, and u_next is held in [0, 1) with
 * NaN as 0.  c, S, products, differences and sums are carried as two fp32
 * numbers each (within 2^-46 of their terms), and summed in an order that does
 * not depend on timing.
 * path_dev: n_seq x max_tok int32, the accepted nodes from node 0 on,
 * ascending, then -1; count_dev[s]: how many; next_dev[s]: the token.  A
 * sequence of no nodes gives 0 and -1.  One longer than max_tok is cut to it,
 * one whose rows leave [0, total_tok) counts as empty, and both set
 * CBQ_DEVERR_BAD_LENGTH; a node whose parent is not before it is never
 * reached.  u_dev[row] (total_tok; node 0's is not used) and u_next_dev
 * (n_seq) in [0, 1).  path_dev, count_dev and next_dev overlap nothing that the
 * call reads, nor one another.  One launch; nothing but the rows of the nodes
 * that the walk passes is read.
 * Errors: EINVAL (null; V < 1 or > CBQ_SAMPLE_MAX_V; probs_stride or
 * draft_stride < V with total_tok > 1, or < 0; total_tok < 1 or > 2^24; n_seq
 * < 1 or > 65535; max_tok outside 1..CBQ_TREE_MAX; a pointer not aligned to
 * its type; an output that overlaps), ECUDA, EDEVICE. */
int cbq_verify(const float *probs_dev, int64_t probs_stride, const float *draft_dev, int64_t draft_stride, int V,
               const int32_t *tokens_dev, const int32_t *parent_dev, int64_t total_tok, const int32_t *start_dev,
               int n_seq, int max_tok, const float *u_dev, const float *u_next_dev, int32_t *path_dev,
               int32_t *count_dev, int32_t *next_dev, unsigned int *err_dev, void *stream);

/* The accepted drafts moved to the end of their context, in all layers' caches
 * with one launch: for i < count_dev[s], the key and value at place ctx_dev[s]
 * + path_dev[s*max_tok + i] go to place ctx_dev[s] + i (path and count as
 * cbq_verify gives them), and ctx_out_dev[s] = ctx_dev[s] + count_dev[s].
 * `cache` describes the first of `layers` caches of the same shape, the next
 * one layer_stride elements on.  Places go through table_dev as in
 * cbq_tree_attention.  A path that is not ascending, or leaves 0..max_tok-1,
 * or places beyond the table or CBQ_TREE_MAX_LEN, end the sequence's moves there and set
 * CBQ_DEVERR_BAD_LENGTH, as does a count outside 0..max_tok (which counts as
 * the nearer end) or a negative ctx (nothing is moved); a page outside the
 * cache is not read or written and sets CBQ_DEVERR_BAD_SLOT.  ctx_out_dev is
 * written for every sequence: what counts there is how many entries of the
 * path were good.  Pages that two of the call's sequences name must not lie
 * behind their contexts.  ctx_out_dev may be NULL, and overlaps
 * nothing that the call reads (other sequences' blocks are still at it).
 * Errors: EINVAL (null; a bad cache; layers < 1 or > 65535; layer_stride < 0;
 * table_width < 1; n_seq < 1 or > 65535; max_tok outside 1..CBQ_TREE_MAX;
 * a ctx_out_dev that overlaps; a pointer not aligned to its type), ECUDA, EDEVICE. */
int cbq_kv_commit(const cbq_kv_cache *cache, int layers, int64_t layer_stride, const int32_t *table_dev,
                  int table_width, int n_seq, const int32_t *ctx_dev, const int32_t *path_dev, int max_tok,
                  const int32_t *count_dev, int32_t *ctx_out_dev, unsigned int *err_dev, void *stream);

/* A paged cache in 8 bits: k and v hold e4m3 numbers (four exponent bits, three
 * of the mantissa, no infinities, largest 448), value d of token t of page p of
 * kv head h at p*page_stride + t*tok_stride + h*head_stride + d, and stand for
 * that number times the fp32 scale at k_scale (v_scale) + p*scale_page_stride +
 * (t / block)*scale_block_stride + h*scale_head_stride.  block <= 65536
 * divides page_size; the other limits are those of cbq_kv_cache. */
typedef struct cbq_kv_cache8 {
    void *k;
    void *v;
    float *k_scale;
    float *v_scale;
    int kv_heads;
    int head_dim;
    int page_size;
    int block;
    int64_t n_pages;
    int64_t page_stride;
    int64_t tok_stride;
    int64_t head_stride;
    int64_t scale_page_stride;
    int64_t scale_block_stride;
    int64_t scale_head_stride;
} cbq_kv_cache8;

/* Pages of a 16-bit cache written into an 8-bit one: page src_dev[i] of `from`
 * becomes page dst_dev[i] of `to`, i < n, in each of `layers` pairs of caches
 * (the struct's, and those that the layer strides, in elements, lead to).  For
 * each block of tokens and head, of k and of v:
 *   scale = 2^e, the least with max |x| <= 448 * 2^e, -80 <= e <= 120 (1 where
 *           all are zero), the maximum over the finite values;
 *   number = x / scale, rounded to nearest even (nothing exceeds 448: that
 *           would take a maximum above 448 * 2^120).
 * A scale that is a power of two costs a floating-point number no precision,
 * so the bytes do not depend on how the division rounds.  NaN and infinities
 * become NaN.  The two caches do not overlap.  A negative entry of src_dev or dst_dev skips its pair; one
 * beyond the cache does too and sets CBQ_DEVERR_BAD_SLOT.  Two pairs with one
 * dst page race.  One launch.
 * Errors: EINVAL (null; a bad cache; heads, head_dim or page_size that differ;
 * layers < 1 or > 65535; negative layer strides; n < 1 or > 2^24; n * kv_heads *
 * page_size / block > 2^31 - 1; a pointer not aligned to its type), ECUDA,
 * EDEVICE. */
int cbq_kv_quantize(const cbq_kv_cache *from, int64_t from_layer_stride, const int32_t *src_dev,
                    const cbq_kv_cache8 *to, int64_t to_layer_stride, int64_t scale_layer_stride,
                    const int32_t *dst_dev, int layers, int64_t n, unsigned int *err_dev, void *stream);

/* cbq_tree_attention over a context whose first old_dev[s] places are in the
 * 8-bit cache: place p < old_dev[s] of sequence s is token p % old->page_size
 * of its page table8_dev[s*table8_width + p / old->page_size], and every other
 * place p, the drafts' among them, token p % page_size of page
 * table_dev[s*table_width + p / page_size] of the 16-bit cache as ever (what
 * the table says of old places is not read).  Formulas, masks, drafts, NaN and
 * rows that see nothing are cbq_tree_attention's, with k and v what the 8-bit
 * numbers and their scales stand for.  max_old bounds old_dev[s] and max_new
 * the places behind, ctx_dev[s] + n_s - old_dev[s]: they size the launch.  A
 * sequence beyond them, beyond its tables, or with old_dev[s] outside
 * 0..ctx_dev[s], is cut to them (first the old places, then the ones behind)
 * and sets CBQ_DEVERR_BAD_LENGTH; page ids as in cbq_tree_attention.
 * Scores, maxima and sums are fp32.  Old places' products take their numbers
 * unrounded as fp16, the query as fp16 numbers of its row's own power of two
 * (what is below 2^-30 of the row's largest loses bits), and the weights times
 * the values' scales rounded to fp16 relative to the row's largest: those
 * below 2^-24 of it lose bits.  Scales may be any positive numbers from 2^-80 to
 * 2^112, both ends in one row too (of values above 2^120, which take larger
 * ones, small weights are lost).
 * old->kv_heads and head_dim are the cache's.  max_old = 0 with old_dev all
 * zero is cbq_tree_attention.  Speed: heads of 64, 128 and 256 with k, v, out
 * and all rows of both caches on 16 bytes take the tensor cores; every other
 * layout a warp a row, one key after another.  With many rows a kv head an 8-bit
 * cache saves room but takes longer than one of 16 bits (8 trees of 64 drafts
 * over 16,000 keys 324 us for 252; few rows over long contexts take less, 106 for
 * 175), and twice that where pages and blocks are not of whole 16 tokens.
 * ws_dev, out_dtype, lse_dev,
 * err_dev and the other arguments as cbq_tree_attention.
 * Errors: those of cbq_tree_attention, and EINVAL (a bad 8-bit cache; max_old
 * outside 0..CBQ_TREE_MAX_LEN; max_new outside 1..CBQ_TREE_MAX_LEN; their sum
 * above that; table8_width < 1). */
int cbq_tree_attention8_workspace(int n_seq, int64_t total_tok, int max_tok, int64_t max_old, int64_t max_new,
                                  int q_heads, int kv_heads, int head_dim, int64_t *bytes);
int cbq_tree_attention8(const void *q_dev, int64_t q_tok_stride, int64_t q_head_stride, int q_heads, int64_t total_tok,
                        const cbq_kv_cache8 *old, const int32_t *table8_dev, int table8_width, const int32_t *old_dev,
                        const cbq_kv_cache *cache, const int32_t *table_dev, int table_width, int n_seq,
                        const int32_t *ctx_dev, const int32_t *start_dev, const int64_t *mask_dev, int max_tok,
                        int64_t max_old, int64_t max_new, float scale, void *out_dev, int out_dtype, float *lse_dev,
                        void *ws_dev, int64_t ws_bytes, unsigned int *err_dev, void *stream);

/* ---- checking entry points (used by the parity tests) ---------------- */

/* Per-block int32 dots s_dev[c][r][b] (n x M x K/32) of W with plain int8
 * activations qx_dev (n x K), through the same codebook expander and dp4a
 * sequence as the matvec kernels.  1 <= n <= CBQ_MAX_COLS. */
int cbq_debug_block_dots(const cbq_weights *W, const int8_t *qx_dev, int n, int32_t *s_dev,
                         void *stream);

/* Same for expert e of an MoE layer: which = 0 gate_up, 1 down; e == E
 * names the shared expert (CBQ_EINVAL when there is none). */
int cbq_moe_debug_block_dots(const cbq_moe *L, int e, int which, const int8_t *qx_dev, int n,
                             int32_t *s_dev, void *stream);

/* Keep (1) or stop keeping (0) the intermediate of each slot -- a (fp32) and
 * its quantization (qa int8, da fp32) in plain slot order -- in the workspace
 * during cbq_moe_matvec (costs about 5*F bytes of writes per slot). */
int cbq_moe_set_debug(cbq_moe *L, int keep_intermediate);

/* Give-up test mode of the layer kernel, for the tests of its bounded waits
 * (0 turns it off): mode 1 makes every down-projection item wait for an
 * intermediate count that is never reached, so that wait gives up after its
 * 1 s limit (CBQ_DEVERR_DEPENDENCY_TIMEOUT, or CBQ_DEVERR_PIPE_TIMEOUT when
 * the consumers' own 1 s wait for that stage runs out first) and the CTA
 * stops; mode 2 makes the first CTA's first weight stage never arrive, so its
 * consumers' wait gives up (CBQ_DEVERR_PIPE_TIMEOUT; the down items that
 * need that CTA's gate_up results then give up too).  Either way the CTA
 * issues no copy after giving up and waits (bounded) for those in flight, so
 * none is left running when it exits.  A call in either mode returns after a
 * few seconds with undefined outputs, sets only timeout bits, and leaves the
 * handle usable: the next call is correct. */
int cbq_moe_debug_stall(cbq_moe *L, int mode);

/* Give-up test mode of the tensor-core path (cbq_matmat and its block-dot
 * checking entry; 0 turns it off): with mode 1 the first CTA's producer
 * issues no copy, so the bounded waits of every role of that CTA for its
 * first stage give up after 1 s (CBQ_DEVERR_PIPE_TIMEOUT in the handle's
 * error word); the CTA issues no MMA after giving up, waits (bounded) for
 * those it issued and frees its tensor memory before it exits.  A call in
 * this mode returns after about a second with undefined outputs, sets only
 * that bit, and leaves the handle usable: the next call is correct.
 * Errors: EINVAL (null handle, mode outside 0..1). */
int cbq_debug_mmq_stall(cbq_weights *W, int mode);

/* Give-up test mode of the calling thread's cbq_tree_attention and
 * cbq_tree_attention8 calls (0 turns it off): with mode 1 the first block of
 * the many-row kernel copies no tile, so its roles' bounded waits give up after
 * 1 s (CBQ_DEVERR_PIPE_TIMEOUT in *err_dev), and it frees its tensor memory and
 * ends.  Such a call returns after about a second, sets only that bit, leaves
 * that block's rows (of the first sequence and kv head) undefined and the
 * others as they would be; the next call is correct.  Calls that the other
 * kernels take are not touched.
 * Errors: EINVAL (mode outside 0..1). */
int cbq_debug_tree_stall(int mode);

/* Copy the intermediate of the last cbq_moe_matvec on this handle, for
 * slots p < nslots (at most CBQ_MAX_TOKENS * (CBQ_MAX_TOPK + 1)): routed
 * slots p = t*topk + j, then the shared expert's slots p = n_tok*topk + t;
 * a_dev[p][F] fp32, qa_dev[p][F] int8, da_dev[p][F/32] fp32 (any may be
 * NULL), as kept by the last call made with debug on (cbq_moe_set_debug).
 * Slots whose id was out of range hold stale data. */
int cbq_moe_debug_intermediate(const cbq_moe *L, int nslots, float *a_dev, int8_t *qa_dev,
                               float *da_dev, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* CBQ_H */
