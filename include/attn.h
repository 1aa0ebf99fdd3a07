/*
 * attn.h -- C ABI of libattn.so: the fused exact-attention forward pass for
 * NVIDIA GB300 (sm_103a).
 *
 * Operation (one call):
 *   O[b,h,i,:] = sum_{j in A(i)} softmax_j(scale * Q[b,h,i,:] . K[b,h,j,:]) V[b,h,j,:]
 *   LSE[b,h,i] = ln sum_{j in A(i)} exp(scale * Q[b,h,i,:] . K[b,h,j,:])
 * computed tile by tile with a running row maximum and row sum, the division
 * by the row sum deferred to the end, so the Nq x Nk score matrix never
 * reaches device memory.
 *   - "Fused Self Attention" (AWS Neuron NKI tutorial), sections "Background"
 *     (S = Q K^T, R = softmax(S) V), "Fusion to Save SBUF Space" (one strip of
 *     query rows at a time) and "Softmax implementation" (row maximum, row
 *     sum, division delayed until after the product with V).
 *   - PhotoRoom / xformers memory-efficient attention post ("torch-permute"
 *     copy): Q and K are read in tiles with a running softmax, and only the
 *     end result is written to main GPU memory.
 *   - "Profiling in PyTorch" part 3, "Deconstructing Naive Attention": scores
 *     are scaled, masked positions are filled with -inf before the softmax;
 *     "Introducing Scaled Dot Product Attention": is_causal=True.
 *   - NATTEN issue #142 "circular windowed attention": 2-D neighbourhood
 *     attention (each query attends the keys between its window start and
 *     end), its circular "wrap" mode, and a float32 logsumexp output shaped
 *     like q without its last dimension.
 *
 * Allowed sets A(i):
 *   ATTN_MASK_NONE   every key j < Nk.
 *   ATTN_MASK_CAUSAL j <= i (top-left alignment, also when Nq != Nk).
 *   ATTN_MASK_CAUSAL_BR j <= i + (Nk - Nq) (bottom-right alignment: the queries
 *                    are the last Nq of Nk tokens). With Nq > Nk the first
 *                    Nq - Nk rows see no key: O = 0, LSE = -inf (and zero
 *                    gradients in attn_bwd).
 *   ATTN_MASK_NA2D   tokens are row-major on a grid_h x grid_w grid (Nq = Nk =
 *                    grid_h * grid_w); along each axis the window holds k
 *                    positions (k odd: `window` along the rows, `window_w`
 *                    along the columns, 0 = `window`). A clamped axis shifts a
 *                    full window inward at the borders, start = clamp(c - k/2,
 *                    0, G - k); a wrapped axis takes the positions (c + t)
 *                    mod G, t in [-k/2, k/2]. `wrap`: 0 = neither axis wraps,
 *                    1 = both, 2 = the rows only, 3 = the columns only. With
 *                    dilation dl > 1 (NATTEN's convention): a clamped axis
 *                    keeps the keys of c's residue class modulo dl and applies
 *                    the rule above to the index inside that class; a wrapped
 *                    axis takes (c + dl * t) mod G. k * dl <= the grid side of
 *                    its axis, unless k = 1. A 1 x N grid with window 1 along
 *                    the rows is 1-D neighbourhood attention.
 *   ATTN_MASK_NA3D   tokens are row-major on a grid_d x grid_h x grid_w
 *                    volume (depth slowest; Nq = Nk = the product, the grid
 *                    given explicitly); the key is allowed iff each of the
 *                    three axes allows it by the rule above. `window_d` is the
 *                    window along the depth (0 = `window`), `wrap_d` 1 wraps
 *                    the depth; `window`, `window_w`, `wrap` and `dilation`
 *                    as for NA2D (one dilation for all three axes). The
 *                    NATTEN issue's requester works on such volumes and wraps
 *                    some of their axes.
 *
 * Data layout (device memory, owned and allocated by the caller):
 *   q, o : bf16 [B, H, Nq, d]   k, v : bf16 [B, H, Nk, d]   (contiguous by
 *          default; attn_fwd_ex accepts element strides for b, h and n, the
 *          last dimension always contiguous, e.g. NATTEN's heads-last
 *          [B, X, Y, heads, d] layout without a permute)
 *   lse  : fp32 [B, H, Nq] contiguous, natural log; NULL = not written.
 *   d in {32, 64, 128}. Pointers 16-byte aligned; element strides multiples
 *   of 8 (16 bytes).
 *
 * Execution: every call only enqueues work on a CUDA stream (the one set by
 * attn_set_stream for the calling thread, or attn_params_ex.stream) and
 * returns; it launches exactly one kernel. The library keeps one lazily
 * allocated device status word per device, and for unmasked problems whose
 * work is split across CTAs (see attn_params_ex.schedule) a workspace for
 * partial results: the caller's (attn_params_ex.workspace) or else one per
 * device, allocated on first need and grown when a larger one is needed.
 * Calls that use the library's workspace must not overlap on the device
 * (e.g. on two streams at once); give each concurrent stream its own.
 * Device-side failures (a bounded wait that ran out) are reported by
 * attn_get_device_status() after the caller synchronises the stream.
 *
 * Errors: every entry point returns ATTN_OK (0) or one of the codes below;
 * argument checks happen on the host before any CUDA call, so an invalid call
 * touches no device state. attn_last_error() gives a one-line message for
 * the calling thread's last failure.
 *
 * Logging: with ATTN_LOG=1 in the environment, every forward launch writes one
 * line to stderr: the entry point, head dimension, mask and kernel variant,
 * shapes, the neighbourhood parameters and the schedule (whole tasks or split,
 * persistent grid size, tasks, K/V-tile units).
 */
#ifndef EXACT_ATTENTION_69_ATTN_H
#define EXACT_ATTENTION_69_ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_ABI_VERSION 6

typedef enum {
  ATTN_MASK_NONE = 0,
  ATTN_MASK_CAUSAL = 1,
  ATTN_MASK_NA2D = 2,
  ATTN_MASK_NA3D = 3,
  ATTN_MASK_CAUSAL_BR = 4
} attn_mask_kind;

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1,  /* sizes < 1, scale not finite or <= 0, even or
                                oversized window, wrap without NA2D, NA2D with
                                Nq != Nk or a non-square Nq and no grid, ... */
  ATTN_ERR_UNSUPPORTED = 2,  /* d not in {32,64,128} */
  ATTN_ERR_MISALIGNED = 3,   /* a pointer not 16-byte aligned, a stride not a
                                multiple of 8 elements */
  ATTN_ERR_CUDA = 4,         /* a CUDA runtime or driver call failed; the
                                message names it */
  ATTN_ERR_TIMEOUT = 5       /* a device-side wait ran past its bound; the
                                kernel stopped early, outputs are undefined */
} attn_status;

/* Full parameter block for attn_fwd_ex. Call attn_params_init first: it sets
 * every field to its default (contiguous strides, dilation 1, no extras). */
typedef struct attn_params_ex {
  const void* q;   /* bf16, see layout above */
  const void* k;
  const void* v;
  void* o;         /* bf16 output */
  float* lse;      /* fp32 [B,H,Nq] output, or NULL */
  int B, H, Nq, Nk, d;
  float scale;     /* > 0 and finite, typically 1/sqrt(d) */
  int mask_kind;   /* attn_mask_kind */
  int window;      /* NA2D, NA3D: odd window size along the rows (and the
                      columns / depth unless window_w / window_d is set);
                      others: must be 0 */
  int dilation;    /* NA2D, NA3D: key stride >= 1 along each axis; others: 1 */
  int wrap;        /* NA2D, NA3D: 0 = rows and columns clamp, 1 = both wrap,
                      2 = the rows wrap, 3 = the columns wrap; others: 0 */
  int grid_h, grid_w; /* NA2D, NA3D rows and columns; NA2D 0,0 = square grid
                         of side sqrt(Nq); NA3D: required */
  /* element strides of dims (b, h, n); all zero = contiguous [B,H,N,d] */
  int64_t q_stride[3], k_stride[3], v_stride[3], o_stride[3];
  void* stream;    /* cudaStream_t; NULL = the calling thread's stream */
  int num_ctas;    /* persistent CTAs; 0 = one per SM (smaller values are for tests) */
  uint64_t timeout_ns; /* bound on every device-side wait; 0 = 2 seconds */
  int inject;      /* test hook: 1 = the loader withholds one K tile so that
                      the kernel's bounded wait runs out (ATTN_ERR_TIMEOUT);
                      0 otherwise */
  void* ev_start;  /* optional cudaEvent_t recorded right before the kernel */
  void* ev_stop;   /* optional cudaEvent_t recorded right after the kernel */
  int schedule;    /* work split over the persistent CTAs: 0 = automatic,
                      1 = whole (batch, head, 256-query) tasks round robin,
                      2 = equal shares of K/V tiles, a task cut between CTAs
                          merged by its last part (ATTN_MASK_NONE only) */
  void* workspace; /* optional device buffer for schedule 2, zero-filled
                      before its first use (later calls leave it reusable);
                      NULL = the library's own */
  uint64_t workspace_bytes; /* size of `workspace` */
  int window_w;    /* NA2D, NA3D: odd window size along the columns; 0 =
                      `window`; others: must be 0 */
  int grid_d;      /* NA3D: depth of the volume (>= 1); others: must be 0 */
  int window_d;    /* NA3D: odd window size along the depth; 0 = `window`;
                      others: must be 0 */
  int wrap_d;      /* NA3D: 1 = the depth wraps, 0 = it clamps; others: 0 */
} attn_params_ex;

/* Fill *p with defaults (zero pointers and sizes, dilation 1, contiguous). */
void attn_params_init(attn_params_ex* p);

/*
 * attn_fwd: the fused forward pass over contiguous bf16 [B,H,N,d] tensors.
 * q,k,v,o are device pointers, lse a device pointer or NULL. For
 * ATTN_MASK_NA2D the token grid is square, side sqrt(Nq) (else
 * ATTN_ERR_INVALID_ARG); use attn_fwd_ex for other grids and layouts.
 * Returns an attn_status code. Asynchronous on the thread's stream.
 */
int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
             int B, int H, int Nq, int Nk, int d, float scale,
             int mask_kind, int window, int dilation, int wrap);

/* attn_fwd with every option (strides, grid, stream, events, test hooks). */
int attn_fwd_ex(const attn_params_ex* p);

/* Set the CUDA stream (a cudaStream_t, NULL = legacy default stream) used by
 * the calling thread's later attn_fwd calls. Thread-local; always ATTN_OK. */
int attn_set_stream(void* stream);

/* Read and clear the current device's status words: the library's own (used
 * by attn_fwd, attn_fwd_ex, attn_bwd) and the one inside attn_fwd_noalloc's
 * fixed array. Allocates nothing (a word that does not exist yet reads as
 * zero). Call after synchronising the stream of the calls in question.
 * Returns ATTN_OK, ATTN_ERR_TIMEOUT, or ATTN_ERR_CUDA if a word could not be
 * read. If detail is not NULL it receives 4 words: code, role (0 loader, 1
 * MMA issuer, 2 softmax), KV tile index, CTA index of the first failure (the
 * library's own word first). */
int attn_get_device_status(uint32_t* detail);

/* Static one-line description of a status code. */
const char* attn_error_string(int code);

/* One-line message about the calling thread's last failing call ("" if none). */
const char* attn_last_error(void);

/* Number of SMs the persistent grid would use on the current device, or a
 * negative attn_status on failure. */
int attn_device_sm_count(void);

/* Bytes of workspace the call described by *p needs on the current device (0
 * if its schedule splits no task), or a negative attn_status. */
int64_t attn_workspace_bytes(const attn_params_ex* p);

/* Schedule tuning: the split-KV schedule's work split, chosen per problem by
 * measurement (the pages' kernels tune their tile configuration per problem;
 * here the tiles are fixed per head dimension and the schedule is tuned).
 * For the problem described by *p, times `iters` launches (>= 1) of each
 * candidate: whole (batch, head, 256-query) tasks over every SM, and, without
 * a mask, equal shares of K/V tiles over G CTAs for several G from the SM count
 * down to a quarter of it. Uses p's buffers (o and lse are overwritten) and
 * stream, and is synchronous. p->schedule and p->num_ctas are ignored; the
 * fastest candidate goes to *out, to be set in the params of later calls.
 * Returns an attn_status code. */
typedef struct attn_tune_result {
  int schedule;      /* 1 = whole tasks, 2 = equal K/V shares */
  int num_ctas;      /* persistent CTAs (0 = one per SM) */
  float us;          /* mean time per launch of that candidate */
  int n_tried;       /* candidates timed */
} attn_tune_result;

int attn_tune(const attn_params_ex* p, int iters, attn_tune_result* out);

/* Free the library's per-device state (status words, workspaces, the
 * backward's stream and scratch) and forget the no-alloc array's device
 * addresses. Later calls re-create it; the first attn_fwd_noalloc call on a
 * device after this looks the address up again, so it too must come before
 * any stream capture. */
void attn_shutdown(void);

/* ATTN_ABI_VERSION of the built library. */
int attn_abi_version(void);

/* sizeof(attn_params_ex) in the built library (lets bindings check their
 * copy of the struct layout). */
int attn_params_size(void);

/*
 * Backward pass: the gradients of a scalar loss through attn_fwd, given the
 * loss's gradient dout at the output O. With P the forward's softmax weights
 * (recomputed from Q, K and the saved log-sum-exp) and D_i = dout_i . O_i:
 *   dV = P^T dout,  dS = P * (dout V^T - D),  dQ = scale dS K,  dK = scale dS^T Q
 * (the chain rule through S = Q K^T, the row softmax and R = S V of "Fused Self
 * Attention", section "Background").
 * Layout: q, o, dout, dq: bf16 [B, H, Nq, d]; k, v, dk, dv: bf16 [B, H, Nk, d];
 * lse: fp32 [B, H, Nq] as written by attn_fwd; all contiguous, device memory
 * owned by the caller, 16-byte aligned. mask_kind and the neighbourhood
 * fields as for attn_fwd (the same checks apply). dq, dk and dv are
 * overwritten. Three kernels are enqueued: rowsum(dout * O) and dQ on the
 * stream, dK and dV on a library-owned second stream forked from it after the
 * first kernel and joined back into it (so later work on the stream, and CUDA
 * graph capture, see one ordered call). The library keeps a lazily grown
 * per-device scratch of B*H*Nq floats for D, so calls on one device must not
 * overlap in time.
 */
typedef struct attn_bwd_params {
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* dout;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  int B, H, Nq, Nk, d;
  float scale;          /* the forward's scale */
  int mask_kind;        /* attn_mask_kind */
  void* stream;         /* cudaStream_t; NULL = the calling thread's stream */
  uint64_t timeout_ns;  /* bound on every device-side wait; 0 = 2 seconds */
  int window, window_w, dilation, wrap, grid_h, grid_w;  /* NA2D/NA3D, as attn_params_ex */
  int grid_d, window_d, wrap_d;                          /* NA3D, as attn_params_ex */
} attn_bwd_params;

/* Zero every field of *p, dilation 1. */
void attn_bwd_params_init(attn_bwd_params* p);

/* The backward pass; returns an attn_status code. Asynchronous. */
int attn_bwd(const attn_bwd_params* p);

/*
 * attn_fwd_noalloc: attn_fwd_ex for callers that cannot allocate device
 * memory -- code that runs where cudaMalloc is forbidden or unavailable (an
 * allocator's or memory pool's own internals, an embedded runtime that owns
 * every allocation) or that must never allocate lazily on a first call. The
 * pages describe no such entry point; it has no counterpart there.
 *
 * Computes the unmasked forward pass (mask_kind must be ATTN_MASK_NONE,
 * workspace NULL) with the split schedule, keeping every piece of scratch in
 * one fixed 48 MiB device array inside the library, which each GPU that loads
 * the library holds until the process exits. It calls no cudaMalloc,
 * cudaFree or other allocating routine. The caller passes inputs and outputs
 * as for attn_fwd_ex.
 *  - The first call on a device looks up the array's device address for that
 *    device (cudaGetSymbolAddress); make that first call before any stream
 *    capture.
 *  - A problem that needs more scratch than the array holds is rejected with
 *    ATTN_ERR_INVALID_ARG and a message giving both sizes.
 *  - All calls on a device share its array and each overwrites what the last
 *    one left. Calls that overlap on the GPU (e.g. on two streams at once)
 *    race and give wrong results: serialise them.
 *  - A device-side wait that runs out is recorded in the array's own status
 *    word; attn_get_device_status reads and clears it (allocating nothing).
 */
int attn_fwd_noalloc(const attn_params_ex* p);

/* ------------------------------------------------------------------------
 * Around the attention of a language model: per-head norm with rotary
 * positions (and its gradient), the append to a paged key/value cache, and
 * attention over such a cache with a prefix that the whole batch shares.
 *
 * These calls own no device memory: scratch is the caller's (a size function
 * beside each call that needs some), needs no initialisation and is free again
 * when the call's kernels are done. Calls that overlap on the device, captured
 * graphs among them, each need their own. The first call may be a captured one.
 * ------------------------------------------------------------------------ */

typedef enum { ATTN_TYPE_BF16 = 0, ATTN_TYPE_FP32 = 1 } attn_weight_type;
typedef enum { ATTN_POS_NONE = 0, ATTN_POS_INT32 = 1, ATTN_POS_INT64 = 2 } attn_pos_type;

/*
 * attn_qk_norm_rope: y = R(pos) (x * r * w), r = 1 / sqrt(mean(x^2) + eps), for
 * every head of q and k in one pass; the mean is over the head's d channels
 * and w has d entries, the same for all heads of q (of k).
 *   norm 0: no norm (r * w = 1; the weights must be NULL).
 *   rot: channels of each head that are rotated, the first `rot` of d; 0 =
 *     none, else a multiple of 16 up to d. Pair i turns by
 *     position * inv_freq[i] (radians): (x_i, x_{i + rot/2}), or
 *     (x_{2i}, x_{2i+1}) with `interleaved`. The product is formed modulo a
 *     turn in 64-bit fixed point, exact to position * 2^-64 of a turn: no
 *     position below 2^40 loses anything of the fp32 result. A frequency that
 *     is zero, subnormal or not finite does not rotate.
 *   positions: int32 or int64 [B, N] with element strides pos_stride (0
 *     allowed: shared by the batch), or NULL: token n is at pos_offset + n.
 * q, q_out [B, Hq, N, d]; k, k_out [B, Hk, N, d] bf16; element strides of
 * (b, h, n), all zero = contiguous; inputs may have zero strides; the last
 * dimension contiguous, pointers 16-byte aligned, strides multiples of 8. A
 * stride of a dimension of size 1 is ignored. An output may be its own input; it
 * must not overlap itself (each stride no smaller than what the dimensions of
 * smaller strides reach).
 * d in {32, 64, 128}. Hk 0: queries only (k, k_out NULL). Squares are summed in
 * fp32: a head whose sum of squares passes 3.4e38 gives zeros.
 */
typedef struct attn_rope_params {
  const void* q;
  const void* k;
  const void* v;              /* attn_kv_append only */
  void* q_out;
  void* k_out;                /* attn_qk_norm_rope only */
  int B, N, Hq, Hk, d;
  int rot, interleaved, norm;
  float eps;                  /* >= 0 and finite */
  const void* q_weight;       /* [d] or NULL (ones) */
  const void* k_weight;
  int q_weight_type, k_weight_type; /* attn_weight_type */
  const double* inv_freq;     /* device, [rot / 2]; NULL iff rot is 0 */
  const void* positions;      /* device, or NULL */
  int pos_type;               /* attn_pos_type; NONE iff positions is NULL */
  int64_t pos_stride[2];
  int64_t pos_offset;
  int64_t q_stride[3], k_stride[3], v_stride[3], q_out_stride[3], k_out_stride[3];
  /* attn_kv_append only (else zero) */
  void* k_cache;              /* bf16 [n_pages, Hk, page_size, d] */
  void* v_cache;
  int64_t k_cache_stride[3];  /* elements between pages, heads, slots; zero = contiguous */
  int64_t v_cache_stride[3];
  int n_pages, page_size;     /* page_size: a power of two >= 16 */
  const int32_t* block_table; /* device, [B, table_width] pages of each sequence */
  int table_width;
  int64_t table_stride;       /* elements between sequences */
  const int32_t* starts;      /* device, [B]: tokens that each sequence holds already */
  const int32_t* counts;      /* device, [B]: real tokens of the N new ones, or NULL (all) */
  void* stream;               /* cudaStream_t; NULL = the calling thread's stream */
} attn_rope_params;

/* Zero every field. */
void attn_rope_params_init(attn_rope_params* p);

int attn_qk_norm_rope(const attn_rope_params* p);

/*
 * attn_kv_append: token n of sequence b goes to slot starts[b] + n of the
 * sequence, page block_table[b][slot / page_size], place slot % page_size:
 * keys normed and rotated as by attn_qk_norm_rope, values as they are. With
 * Hq > 0 the queries of the same tokens are normed and rotated into q_out in
 * the same launch (every token, also behind counts[b]). Without `positions`
 * token n is at pos_offset + starts[b] + n. Nothing else of the cache is
 * written: not for tokens n >= counts[b], for a negative start, for slots
 * behind the table's end, nor for entries that are not a page of the cache.
 * Two tokens of one call on the same place of a page leave one or the other,
 * in parts of 16 bytes.
 */
int attn_kv_append(const attn_rope_params* p);

/*
 * attn_qk_norm_rope_bwd: gradients through attn_qk_norm_rope. With g = R^T dy
 * and h = g * w: dx = r h - x r^3 mean(h x), dw = sum over tokens and heads of
 * g x r (without norm dx = g). Sums are fp32 in a fixed order: the same inputs
 * give the same bits. dq, dk as q, k; dq_weight, dk_weight of the weights'
 * types, or NULL. Workspace: attn_qk_norm_rope_bwd_workspace_bytes (0 without
 * weight gradients), 16-byte aligned.
 */
typedef struct attn_rope_bwd_params {
  const void* q;
  const void* k;
  const void* dq_out;         /* gradients at the outputs */
  const void* dk_out;
  void* dq;
  void* dk;
  int B, N, Hq, Hk, d;
  int rot, interleaved, norm;
  float eps;
  const void* q_weight;
  const void* k_weight;
  int q_weight_type, k_weight_type;
  void* dq_weight;
  void* dk_weight;
  const double* inv_freq;
  const void* positions;
  int pos_type;
  int64_t pos_stride[2];
  int64_t pos_offset;
  int64_t q_stride[3], k_stride[3], dq_out_stride[3], dk_out_stride[3], dq_stride[3], dk_stride[3];
  void* workspace;
  uint64_t workspace_bytes;
  void* stream;
} attn_rope_bwd_params;

void attn_rope_bwd_params_init(attn_rope_bwd_params* p);
int attn_qk_norm_rope_bwd(const attn_rope_bwd_params* p);
/* Bytes of workspace, or a negative attn_status. */
int64_t attn_qk_norm_rope_bwd_workspace_bytes(const attn_rope_bwd_params* p);

/*
 * attn_paged: attention of B sequences over a paged cache. The keys of
 * sequence b are the prefix_len tokens of the pages in prefix_table, the same
 * for all sequences, then kv_lens[b] tokens of the pages in block_table[b].
 * Its Nq query rows are the last q_lens[b] of those tokens (rows behind
 * q_lens[b] are padding); with T = prefix_len + kv_lens[b]
 *   ATTN_MASK_CAUSAL_BR  row i sees keys j <= i + T - q_lens[b]
 *   ATTN_MASK_NONE       every row i < q_lens[b] sees all T keys
 *   O[b,h,i,:] = sum_j softmax_j(scale q . k_j) v_j,  LSE the natural-log sum.
 * A row that sees no key, or none whose score is above -inf, gives O = 0,
 * LSE = -inf; one with a score that is NaN or +inf gives NaN for both. Query
 * head h reads key head h / (Hq / Hk). Keys are read once for up to 256 query
 * rows of a key head (a sequence has Nq * Hq / Hk): rows of one sequence, or,
 * for the prefix where that saves enough, rows of all sequences together.
 * Lengths and tables are read on the device when the kernels run. kv_lens is
 * clamped to what the table holds, q_lens to Nq; a table entry that is not a
 * page of the cache reads as zeros. Slots of a page behind a sequence's end
 * may hold anything. Values of keys that only some rows see must be finite.
 * Two kernels are enqueued: attention, and the join of tasks that were cut.
 */
typedef struct attn_paged_params {
  const void* q;              /* bf16 [B, Hq, Nq, d] */
  const void* k_cache;        /* bf16 [n_pages, Hk, page_size, d] */
  const void* v_cache;
  void* o;                    /* bf16 [B, Hq, Nq, d] */
  float* lse;                 /* fp32 [B, Hq, Nq] contiguous, or NULL */
  const int32_t* block_table; /* device, [B, table_width] */
  const int32_t* kv_lens;     /* device, [B] */
  const int32_t* q_lens;      /* device, [B], or NULL (Nq each) */
  const int32_t* prefix_table;/* device, [prefix_pages], or NULL */
  int B, Hq, Hk, Nq, d;       /* Hq a multiple of Hk; d in {32, 64, 128} */
  int n_pages, page_size;     /* page_size: a power of two >= 16 */
  int table_width;
  int64_t table_stride;
  int prefix_len, prefix_pages;
  float scale;                /* > 0 and finite */
  int mask_kind;              /* ATTN_MASK_NONE or ATTN_MASK_CAUSAL_BR */
  int64_t q_stride[3], o_stride[3];             /* elements, (b, h, n); zero = contiguous */
  int64_t k_cache_stride[3], v_cache_stride[3]; /* pages, heads, slots; zero = contiguous */
  void* workspace;            /* attn_paged_workspace_bytes, 16-byte aligned */
  uint64_t workspace_bytes;
  void* stream;
  int num_ctas;               /* 0 = one per SM (smaller values are for tests) */
  uint64_t timeout_ns;        /* bound on every device-side wait; 0 = 2 seconds */
  int inject;                 /* test hook, as attn_params_ex.inject */
} attn_paged_params;

void attn_paged_params_init(attn_paged_params* p);
int attn_paged(const attn_paged_params* p);
/* Bytes of workspace on the current device, or a negative attn_status. Depends
 * on the block's sizes and prefix_len, not on what kv_lens and q_lens hold. */
int64_t attn_paged_workspace_bytes(const attn_paged_params* p);

/* sizeof of attn_rope_params (0), attn_rope_bwd_params (1), attn_paged_params (2). */
int attn_struct_size(int which);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_ATTENTION_69_ATTN_H */
