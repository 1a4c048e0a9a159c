/*
 * fa.h -- C ABI of the GB300 (sm_103a) exact attention forward library.
 *
 * The operation ("FlashAttention: IO-aware attention kernels", table "What
 * goes in, what comes out"; "FlashAttention: Why Tiling Attention Makes
 * Transformers Fast Without Changing the Result", section "The tiled forward
 * pass"): for every batch b and head h,
 *
 *     O   = softmax(scale * Q K^T  restricted to visible keys) V
 *     lse = per-row natural-log sum of exp(scale * q_i . k_j) over visible j
 *
 * computed in one fused pass: key/value tiles stream through on-chip memory
 * while each query row keeps a running max, a running sum and an
 * unnormalised accumulator; the S x S score and probability matrices are
 * never written to device memory.  The result is exact up to floating-point
 * rounding order: inputs are 16-bit, products accumulate in fp32, the
 * probabilities are rounded to the input type before the P V product, and O
 * is rounded to the input type once at the end.
 *
 * Masks (readings of the pages, which name causal and sliding-window masks
 * but not their alignment):
 *   FA_MASK_NONE            every key j < Sk is visible;
 *   FA_MASK_CAUSAL          key j visible to query i iff j <= i (top-left
 *                           aligned: query 0 sees key 0, also when Sq != Sk);
 *   FA_MASK_SLIDING_WINDOW  causal and j > i - window: `window` keys
 *                           including the diagonal.
 * A query row that sees no key (only possible with a window and Sq > Sk)
 * gets O = 0 and lse = -inf, never NaN.  Arbitrary boolean masks are not
 * supported and are rejected, never silently run another way.
 *
 * All entry points are plain C.  No entry point allocates device memory, and
 * none falls back to a slower path: an unsupported request returns an error.
 */
#ifndef FA_GB300_FA_H
#define FA_GB300_FA_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The same type as cudaStream_t (struct CUstream_st*); NULL = legacy stream. */
typedef struct CUstream_st *fa_stream_t;

typedef enum fa_status {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,    /* sizes, pointers, mask/window or scale invalid  */
    FA_ERR_UNSUPPORTED = 2,    /* head dim, dtype, mask kind or GPU not supported */
    FA_ERR_MISALIGNED = 3,     /* q, k, v, o not 16-byte aligned or lse not 4    */
    FA_ERR_CUDA = 4,           /* a CUDA runtime/driver call or the launch failed */
    FA_ERR_DEVICE_TIMEOUT = 5  /* a kernel's pipeline wait ran out (device flag)  */
} fa_status;

enum { FA_MASK_NONE = 0, FA_MASK_CAUSAL = 1, FA_MASK_SLIDING_WINDOW = 2 };
enum { FA_DTYPE_BF16 = 0, FA_DTYPE_FP16 = 1 };
/* fa_rope also takes fp32; the attention entry points do not. */
enum { FA_DTYPE_FP32 = 2 };
/* Pairs of fa_rope: components (i, i + rot_dim/2), or (2i, 2i + 1). */
enum { FA_ROPE_HALF = 0, FA_ROPE_INTERLEAVED = 1 };
enum { FA_ROPE_FORWARD = 0, FA_ROPE_BACKWARD = 1 };
/* Frequency scaling for contexts longer than trained (fa_rope_frequencies). */
enum { FA_ROPE_SCALE_NONE = 0, FA_ROPE_SCALE_LINEAR = 1, FA_ROPE_SCALE_NTK = 2, FA_ROPE_SCALE_BY_PARTS = 3 };
/* Per-request status of fa_paged_update. */
enum { FA_PAGED_OK = 0, FA_PAGED_NO_BLOCKS = 1, FA_PAGED_TOO_LONG = 2, FA_PAGED_NO_ROWS = 3 };
/* Kernel choice of fa_decode_paged / fa_decode_workspace_query. */
enum { FA_DECODE_AUTO = 0, FA_DECODE_TENSOR_CORES = 1, FA_DECODE_CUDA_CORES = 2 };

/*
 * fa_fwd -- fused attention forward, bf16 inputs and output.
 *
 *   q    device pointer, [B, H, Sq, d] bf16, contiguous row-major, 16-B aligned
 *   k, v device pointers, [B, H, Sk, d] bf16, contiguous, 16-B aligned
 *   o    device pointer, [B, H, Sq, d] bf16 output; must not overlap q, k, v
 *   lse  device pointer, [B, H, Sq] fp32 output (natural-log logsumexp of the
 *        scaled scores of each row), 4-B aligned; must not overlap the others
 *   B, H >= 1; Sk >= 1; Sq >= 0 (Sq == 0: FA_OK once the sizes, kinds and scale
 *        are valid; nothing is enqueued and the pointers are not examined)
 *   d    head dimension: 64, 128 or 256 (else FA_ERR_UNSUPPORTED)
 *   scale  multiplies Q K^T; finite and >= 0 (callers usually pass 1/sqrt(d))
 *   mask_kind  FA_MASK_NONE, FA_MASK_CAUSAL or FA_MASK_SLIDING_WINDOW
 *   window  keys per row for FA_MASK_SLIDING_WINDOW (>= 1); ignored otherwise
 *   stream  CUDA stream to enqueue on
 *
 * Ownership: every buffer belongs to the caller; the library keeps no pointer
 * after returning and allocates nothing.  The call validates its arguments
 * synchronously (nothing is enqueued on error), then enqueues one kernel
 * launch and returns; results are ready when the stream reaches that point.
 * Re-entrant: concurrent calls on different streams are independent.
 * A kernel whose internal pipeline wait exceeds its time limit (about 2 s)
 * stops early and raises a device flag read by fa_get_device_error().
 */
fa_status fa_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                 int B, int H, int Sq, int Sk, int d, float scale,
                 int mask_kind, int window, fa_stream_t stream);

/* fa_fwd_fp16 -- identical to fa_fwd with fp16 q, k, v and o. */
fa_status fa_fwd_fp16(const void *q, const void *k, const void *v, void *o, float *lse,
                      int B, int H, int Sq, int Sk, int d, float scale,
                      int mask_kind, int window, fa_stream_t stream);

/*
 * fa_fwd_gqa -- the same forward with grouped-query attention: K and V carry
 * H_kv heads and each run of H / H_kv consecutive query heads shares one, so
 * that query head h reads K/V head h / (H / H_kv).  (The pages name
 * grouped-query attention as a later variant of the method without defining
 * it -- "FlashAttention: Why Tiling...", section "Using it in practice"; this
 * grouping is the reading taken, the one PyTorch's enable_gqa uses.)
 * H_kv == H is fa_fwd / fa_fwd_fp16; H_kv == 1 is multi-query attention.
 *
 *   q, o  [B, H, Sq, d]; k, v [B, H_kv, Sk, d]; lse [B, H, Sq] fp32
 *   H_kv  >= 1 and dividing H, else FA_ERR_INVALID_ARG
 *   dtype FA_DTYPE_BF16 or FA_DTYPE_FP16 (q, k, v and o alike)
 * Every other argument, the ownership, the errors and the device flag are as
 * for fa_fwd; fa_workspace_query with (B, H, ...) answers for this call too
 * once H_kv divides H.  K/V tiles of a shared head are read by all of its
 * query heads from the L2, so DRAM reads of K and V shrink by H / H_kv.
 */
fa_status fa_fwd_gqa(const void *q, const void *k, const void *v, void *o, float *lse,
                     int B, int H, int H_kv, int Sq, int Sk, int d, float scale,
                     int mask_kind, int window, int dtype, fa_stream_t stream);

/*
 * fa_bwd -- attention backward: dQ, dK, dV from Q, K, V, the forward's O and
 * lse, and dO = dLoss/dO ("FlashAttention: Why Tiling...", section "The
 * backward pass: recompute instead of storing").  Each score tile is
 * recomputed on chip from Q and K, its probabilities rebuilt from lse
 * (P = exp(scale q.k - lse)); then dV = P^T dO, dP = dO V^T, the softmax
 * Jacobian gives dS = P (dP - delta) with delta_i = dO_i . O_i, and
 * dQ = scale dS K, dK = scale dS^T Q.  No S x S matrix reaches device memory.
 * Deterministic: no atomics, the same inputs give the same bits.
 *
 *   q, o, dout  [B, H, Sq, d]; k, v [B, H_kv, Sk, d]; lse [B, H, Sq] fp32 as
 *               written by fa_fwd / fa_fwd_gqa for the same q, k, v, scale,
 *               mask and window (-inf marks a row that sees no key)
 *   dq          [B, H, Sq, d] output; dk, dv [B, H_kv, Sk, d] outputs (with
 *               shared K/V heads, summed over the query heads that read them)
 *   workspace   device scratch of at least fa_bwd_workspace_query() bytes,
 *               256-byte aligned; its contents on entry do not matter and on
 *               return are the per-row statistics of this call
 *   d           64, 128 or 256 (for 256 two CTAs share each 128-key tile,
 *               each accumulating half of the dK and dV columns)
 *   dtype       FA_DTYPE_BF16 or FA_DTYPE_FP16 for all 16-bit tensors
 *   the rest    as for fa_fwd_gqa
 * All tensors are contiguous and 16-byte aligned (lse 4-byte).  Outputs may
 * not overlap each other, the inputs or the workspace (FA_ERR_INVALID_ARG).
 * Sq == 0 sets dk and dv to zero; q, o, lse, dout, dq and the workspace are
 * then not examined.  Enqueues three kernels and returns; allocates
 * nothing.  The row statistics and dK/dV run on `stream`; dQ runs on a
 * library stream of the current device (created by the first call, never
 * destroyed), forked from `stream` after the statistics and joined back
 * before any later work on `stream`, both by events: synchronising `stream`
 * covers all three, and a stream capture on `stream` records the fork and
 * join as graph edges.  Calls may come from several host threads on several
 * streams (a lock serialises their enqueue); their dQ kernels then share the
 * library stream and run one after another.  Waits are bounded as in the
 * forward and report through fa_get_device_error().
 */
fa_status fa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                 const void *dout, void *dq, void *dk, void *dv, void *workspace,
                 size_t workspace_bytes, int B, int H, int H_kv, int Sq, int Sk, int d,
                 float scale, int mask_kind, int window, int dtype, fa_stream_t stream);

/*
 * fa_bwd_noalloc -- fa_bwd for callers that cannot provide device memory:
 * the same computation and results, with the workspace taken from a fixed
 * 32 MiB array in the library's device memory instead of the caller.  The
 * pages have no counterpart to this entry point; it exists for the calling
 * convention only.
 *
 *   arguments   as for fa_bwd, without workspace and workspace_bytes
 *   limit       fa_bwd_workspace_query() bytes <= 32 MiB, i.e.
 *               B * H * ceil(Sq / 128) * 128 <= 4,194,304 query rows;
 *               larger problems return FA_ERR_INVALID_ARG (use fa_bwd)
 * The first call on a device looks up the array's device address (with that
 * device current) and should come before any stream capture: under capture
 * that lookup may fail, and the call then returns FA_ERR_CUDA having enqueued
 * nothing; a failed lookup is not remembered, so one plain call made before
 * the capture fixes it.  The address is looked up again in a new context of
 * the device (after cudaDeviceReset).  Nothing is allocated or freed by any
 * call.  Every call on a device uses the same array:
 * calls whose work overlaps in time on one device (another stream, another
 * host thread) race on it and give undefined results.
 */
fa_status fa_bwd_noalloc(const void *q, const void *k, const void *v, const void *o,
                         const float *lse, const void *dout, void *dq, void *dk, void *dv,
                         int B, int H, int H_kv, int Sq, int Sk, int d, float scale,
                         int mask_kind, int window, int dtype, fa_stream_t stream);

/*
 * fa_bwd_workspace_query -- workspace bytes fa_bwd needs (2 x 4 bytes per
 * query row, rows padded per head to a multiple of 128), and the status
 * fa_bwd would return for these sizes on the current device (pointer checks
 * aside).  bytes must be non-NULL; it is 0 whenever the status is not FA_OK.
 */
fa_status fa_bwd_workspace_query(int B, int H, int H_kv, int Sq, int Sk, int d, int mask_kind,
                                 int window, int dtype, size_t *bytes);

/*
 * fa_fwd_fp8 -- the fused forward with 8-bit inputs ("FlashAttention:
 * IO-aware attention kernels", section "Concept", names low-precision paths
 * as a later variant).  Q, K and V are e4m3 codes with one dequantisation
 * factor per tensor (value = code x descale); S = Q K^T and P V run on the
 * 8-bit tensor path with fp32 accumulation, the running max, sum and
 * rescaling are those of fa_fwd, P is rounded to e4m3 (weights of at most
 * 2^4, stored times 2^4) before P V, O is written as bf16 and lse (natural log of the scaled row sums) as
 * fp32.  Exact up to the rounding of P: each output element differs from the
 * exact attention of the dequantised inputs by at most about 2^-4 of
 * sum_j P_ij |v_jc|, plus its bf16 rounding.
 *
 *   q    [B, H, Sq, d] e4m3; k [B, H_kv, Sk, d] e4m3
 *   vt   V transposed, [B, H_kv, d, Sk] e4m3 (both tile products then read
 *        K-major operands); Sk a multiple of 16 (16-byte rows)
 *   o    [B, H, Sq, d] bf16; lse [B, H, Sq] fp32
 *   d    64, 128 or 256 (else FA_ERR_UNSUPPORTED)
 *   scale, q_descale, k_descale, v_descale: finite; descales > 0
 *   the rest as for fa_fwd_gqa (masks, window, H_kv grouping, errors)
 */
fa_status fa_fwd_fp8(const void *q, const void *k, const void *vt, void *o, float *lse, int B,
                     int H, int H_kv, int Sq, int Sk, int d, float scale, float q_descale,
                     float k_descale, float v_descale, int mask_kind, int window,
                     fa_stream_t stream);

/*
 * fa_decode_paged -- attention of the newest Sq rows of each request over its
 * paged K/V cache, as in decoding ("Flash attention and memory-efficient
 * attention variants", sections "A different bottleneck: the KV cache during
 * inference" and "PagedAttention: memory management borrowed from an
 * operating system").  The cache is a pool of physical blocks of block_size
 * tokens; request b's block table maps its logical block n (tokens
 * n*block_size .. (n+1)*block_size - 1) to a physical block.  Exact softmax
 * attention over the gathered tokens; each request's keys are cut into ranges
 * that run in parallel, and the partial results are merged by their lse.
 *
 *   q            [B, H, Sq, d] 16-bit: the new rows (Sq = 1 for one step)
 *   k_cache      [num_blocks, H_kv, block_size, d] 16-bit
 *   v_cache      same layout
 *   block_table  device int32 [B, max_blocks]; entries past a request's last
 *                block are not read; an entry outside [0, num_blocks) reads
 *                zeros
 *   seq_lens     device int32 [B]: cached tokens of each request, the last Sq
 *                of which are the new rows' own; must lie in
 *                [Sq, max_seq_len] (values outside are clamped into it)
 *   o, lse       [B, H, Sq, d] 16-bit and [B, H, Sq] fp32 outputs
 *   workspace    at least fa_decode_workspace_query() bytes, 256-byte aligned
 *   H_kv         K/V heads, dividing H; (H / H_kv) * Sq <= 128
 *   d            64, 128 or 256; block_size 16, 32, 64 or 128
 *   max_seq_len  host bound on seq_lens (it sizes the key ranges)
 *   mask_kind    FA_MASK_NONE (every cached token) or FA_MASK_CAUSAL: row i
 *                sits at position seq_lens[b] - Sq + i and sees tokens up to
 *                it (the reading for decoding: the new rows are the last)
 *   dtype        FA_DTYPE_BF16 or FA_DTYPE_FP16
 *   kernel       FA_DECODE_AUTO: with at most 2 rows per K/V head
 *                ((H / H_kv) * Sq <= 2) the key-range kernel runs on the CUDA
 *                cores (the products are matrix-vector ones), else on the
 *                tensor cores.  FA_DECODE_TENSOR_CORES / FA_DECODE_CUDA_CORES
 *                force one (CUDA cores: at most 2 rows, else
 *                FA_ERR_UNSUPPORTED); other values FA_ERR_UNSUPPORTED.  The
 *                two kernels split the keys differently, so pass the same
 *                choice to fa_decode_workspace_query.
 * Cache slots past a request's length may hold any values, inf and NaN
 * included: they are hidden and never reach O.  Errors and the device flag
 * are as for fa_fwd; the library allocates nothing.  Two launches: the
 * key-range kernel, then the merge.
 */
fa_status fa_decode_paged(const void *q, const void *k_cache, const void *v_cache,
                          const int *block_table, const int *seq_lens, void *o, float *lse,
                          void *workspace, size_t workspace_bytes, int B, int H, int H_kv,
                          int Sq, int d, int block_size, int max_blocks, int num_blocks,
                          int max_seq_len, float scale, int mask_kind, int dtype, int kernel,
                          fa_stream_t stream);

/*
 * fa_decode_workspace_query -- workspace bytes fa_decode_paged needs on the
 * current device with this kernel choice (partial rows of every key range:
 * (d + 1) x 4 bytes per row and range) and the status it would return for
 * these sizes.  bytes must be non-NULL; it is 0 whenever the status is not
 * FA_OK.
 */
fa_status fa_decode_workspace_query(int B, int H, int H_kv, int Sq, int d, int block_size,
                                    int max_blocks, int num_blocks, int max_seq_len,
                                    int mask_kind, int dtype, int kernel, size_t *bytes);

/*
 * fa_rope -- rotary positions on q and k before the attention, or the gradient
 * of that.  The first rot_dim components of every row are pairs (x1, x2); pair
 * i of a row at position n becomes
 *     y1 = a (x1 cos t - x2 sin t),  y2 = a (x1 sin t + x2 cos t),
 *     t = n * f_i,   a = amplitude,
 * and components rot_dim .. d pass through.  The product n * f_i is exact
 * modulo a turn (64-bit fixed point); the f_i of fa_rope_frequencies are fp64, so
 * that an angle is within 2^-53 of its whole size, 2^-22 radians at position
 * 2^31, of the formula's.  Products and sums are fp32, each output is rounded
 * once.
 *
 *   q, q_out   [B, H, S, d] by strides: q_strides[3] are the element strides of
 *              batch, head and token, on the host; components are adjacent.
 *              Rows can so be read out of a packed projection
 *              ([B, S, heads, d]) and written as the contiguous layout the
 *              attention takes.  Any strides >= 0 for inputs (0 repeats a
 *              row); an output's elements must all be distinct
 *   k, k_out   [B, H_kv, S, d] alike; H_kv == 0: no k, the four are not
 *              examined
 *   positions  device int32, row (b, s) at positions[b * position_stride + s]
 *              (stride 0: one row for every batch; at most 2^40), or NULL:
 *              0 .. S-1; negative ones are allowed
 *   offset     added to every position
 *   freq       device array of rot_dim / 2 frequencies, turns per position
 *              times 2^64, as fa_rope_frequencies writes them; 8-byte aligned
 *   direction  FA_ROPE_FORWARD, or FA_ROPE_BACKWARD: q and k are gradients of
 *              the forward's outputs, q_out and k_out those of its inputs
 *   rot_dim    even, 2 <= rot_dim <= d <= 1024
 *   dtype      FA_DTYPE_BF16, FA_DTYPE_FP16 or FA_DTYPE_FP32 (all four tensors)
 * In place is allowed (an output with the base and strides of its own input,
 * also for heads inside one packed tensor); any other overlap of an output
 * with an input, the other output, positions or freq is refused
 * (FA_ERR_INVALID_ARG).  Base addresses are aligned to the element.  S == 0:
 * FA_OK, nothing is enqueued.  One launch on `stream`; no workspace.
 */
fa_status fa_rope(const void *q, const long long *q_strides, void *q_out, const long long *q_out_strides,
                  const void *k, const long long *k_strides, void *k_out, const long long *k_out_strides,
                  const int *positions, long long position_stride, long long offset,
                  const unsigned long long *freq, float amplitude, int B, int H, int H_kv, int S, int d,
                  int rot_dim, int layout, int direction, int dtype, fa_stream_t stream);

/*
 * fa_rope_frequencies -- the frequencies fa_rope reads, computed on the host
 * in fp64: f_i = base^(-2i / rot_dim) radians per position, written to the
 * host array freq[rot_dim / 2] as turns times 2^64, and the amplitude.
 *   FA_ROPE_SCALE_NONE      f_i as it is; amplitude 1
 *   FA_ROPE_SCALE_LINEAR    f_i / factor: positions squeezed by factor
 *   FA_ROPE_SCALE_NTK       base * factor^(rot_dim / (rot_dim - 2)): the
 *                           slowest pair is stretched by factor, the fastest
 *                           left as it is
 *   FA_ROPE_SCALE_BY_PARTS  a pair that makes at least high_turns turns over
 *                           original_length positions keeps f_i, one that
 *                           makes at most low_turns gets f_i / factor, between
 *                           them linear; amplitude 0.1 ln(factor) + 1
 * base >= 1; factor >= 1 (unused for NONE); original_length > 0 and low_turns
 * < high_turns for BY_PARTS (unused otherwise).  No GPU is needed.
 */
fa_status fa_rope_frequencies(int rot_dim, double base, int scaling, double factor, double original_length,
                              double low_turns, double high_turns, unsigned long long *freq,
                              float *amplitude);

/*
 * fa_paged_update -- one step of a paged cache's bookkeeping on the GPU: block
 * tables, slots and positions from the requests' lengths, with the free
 * physical blocks in a ring ("Flash attention and memory-efficient attention
 * variants", section "PagedAttention: memory management borrowed from an
 * operating system").  Nothing is read back to the host, so a step can be
 * captured in a graph and replayed.
 *
 *   seq_lens    device int32 [B]: cached tokens of each request (values outside
 *               [0, max_blocks * block_size] are clamped into it)
 *   delta       device int32 [B]: tokens the step adds (> 0) or takes off the
 *               end (< 0, at most all: rejected drafts, finished requests)
 *   block_table device int32 [B, max_blocks], updated in place: new blocks are
 *               entered; entries past a request's last block are not cleared
 *   free_ring   device int32 [ring_size], updated in place: the free blocks are
 *               entries (head + i) % ring_size, i < count
 *   ring_state  device int32 {head, count}
 *   seq_lens_out, ring_state_out  the new lengths and state; each may be its
 *               input
 *   slot_map, positions  device int32 [max_tokens]: the added tokens, request
 *               by request in index order: the token's slot (physical block *
 *               block_size + place in it) and its position in its request.
 *               Rows past the last token get slot -1 and position 0
 *   status      device int32 [B]: FA_PAGED_OK, or why the request was left as
 *               it was (its rows then have slot -1, position 0):
 *               FA_PAGED_TOO_LONG (past max_blocks * block_size),
 *               FA_PAGED_NO_ROWS (its rows would pass max_tokens),
 *               FA_PAGED_NO_BLOCKS (the free blocks ran out: blocks go to
 *               requests in index order, and once one is short, later ones
 *               that need any are refused too)
 *   block_size  16, 32, 64 or 128, else FA_ERR_UNSUPPORTED
 * New blocks are taken from the ring's head; blocks given back are added
 * behind its tail, in index order, and can be taken from the next call on (a
 * ring of at least the pool's blocks never overflows; blocks past ring_size
 * are dropped).  A row whose table entry is negative, or whose slot would pass
 * 2^31 - 1, gets slot -1 and position 0.
 * Otherwise outputs may not overlap inputs or each other.  One launch; no
 * workspace; the results do not depend on timing.
 */
fa_status fa_paged_update(const int *seq_lens, const int *delta, int *block_table, int *free_ring,
                          const int *ring_state, int *seq_lens_out, int *ring_state_out, int *slot_map,
                          int *positions, int *status, int B, int max_blocks, int ring_size,
                          int block_size, int max_tokens, fa_stream_t stream);

/*
 * fa_paged_update_by_request -- fa_paged_update for batches laid out by request,
 * as fa_decode_paged_fp8 takes q: slot_map and positions are
 * [B, rows_per_request], and the delta tokens that request b adds are the LAST of
 * its rows, so that row i of a request stands at position seq_lens_out[b] -
 * rows_per_request + i.  Rows in front of them, and all rows of a request that
 * adds none (an idle one, a finished one, a padding row of a captured batch), get
 * slot -1 and position 0: nothing is written for them.  FA_PAGED_NO_ROWS: delta
 * > rows_per_request.  rows_per_request >= 1; the rest as above.
 *
 * fa_paged_update's rows, in contrast, follow each other without gaps: row t is
 * the t-th added token of the batch, so request b's are rows b .. only while
 * every request adds exactly one.
 */
fa_status fa_paged_update_by_request(const int *seq_lens, const int *delta, int *block_table,
                                     int *free_ring, const int *ring_state, int *seq_lens_out,
                                     int *ring_state_out, int *slot_map, int *positions, int *status,
                                     int B, int max_blocks, int ring_size, int block_size,
                                     int rows_per_request, fa_stream_t stream);

/*
 * fa_cache_append_fp8 -- writes new K and V rows into a paged cache held in
 * e4m3 codes with one scale per (block, K/V head), K and V apart: the value of
 * a code is code * scale.  For every block the call writes to:
 *     need   = the smallest power of two s >= 2^-126 with |x| <= 448 s for
 *              every finite value x written to it
 *     scale' = need if the block's slot 0 is written (the block starts anew),
 *              else max(scale, need)
 *     where scale' > scale, the codes of the block not written become
 *     e4m3(code * scale / scale'); the written ones are e4m3(x / scale')
 * rounded to nearest even, saturating at +-448 (infinities too; NaN stays
 * NaN).  A stored scale that is no positive finite number counts as none.
 *
 *   k, v        [T, H_kv, d] 16-bit by element strides (token, head); values
 *               of a head adjacent; the strides are >= 0; T <= 2^30
 *   slot_map    device int32 [T], as fa_paged_update writes it: row t goes to
 *               slot s = block * block_size + place; rows whose slot is outside
 *               [0, num_blocks * block_size) are skipped.  Rows of one block
 *               must stand together (skipped rows between them are fine): a
 *               block met again behind another block's rows gives undefined
 *               codes and scale for that block.  A slot named twice in its
 *               block's rows gets the later row
 *   k_cache, v_cache  [num_blocks, H_kv, block_size, d] e4m3, 16-byte aligned
 *   k_scale, v_scale  [num_blocks, H_kv] fp32
 *   d           64, 128 or 256; block_size 16, 32, 64 or 128
 *   dtype       FA_DTYPE_BF16 or FA_DTYPE_FP16 (k and v)
 * Codes and scales of blocks without a row are left as they were, and so are
 * the slots without a row of a block that starts anew.  T == 0: FA_OK.
 * Outputs may not overlap inputs or each other.  One launch; no workspace.
 */
fa_status fa_cache_append_fp8(const void *k, const void *v, long long k_token_stride,
                              long long k_head_stride, long long v_token_stride, long long v_head_stride,
                              const int *slot_map, void *k_cache, void *v_cache, float *k_scale,
                              float *v_scale, int T, int H_kv, int d, int block_size, int num_blocks,
                              int dtype, fa_stream_t stream);

/*
 * fa_decode_paged_fp8 -- fa_decode_paged over the 8-bit cache of
 * fa_cache_append_fp8: exact softmax attention over the dequantised tokens,
 * q and o in 16 bits.  q enters exactly, but for components below 2^-13 of
 * their row's largest: those may be off by 2^-21 of that.  Each weight is
 * rounded to 16 bits before P V with up to four rows per K/V head, else to 8
 * (bf16) or 11 (fp16) bits, as where fa_decode_paged uses the tensor cores;
 * and to no finer than 2^-20 of the row's largest product of a weight and its
 * V scale among up to 256 neighbouring keys.  Sums are fp32.  Deterministic.  Two launches at most; the workspace's
 * contents on entry do not matter.  Arguments as for fa_decode_paged, except:
 *
 *   k_cache, v_cache  [num_blocks, H_kv, block_size, d] e4m3
 *   k_scale, v_scale  [num_blocks, H_kv] fp32, finite (any such scales, powers
 *                     of two or not)
 *   q            finite; a row with an infinity or NaN gives NaN
 *   seq_lens     any length in [0, max_seq_len] (values outside are clamped
 *                into it).  A row that sees no key -- length 0, or with
 *                FA_MASK_CAUSAL a row in front of the request's first token --
 *                gets O = 0 and lse = -inf
 *   block_table  an entry outside [0, num_blocks) reads zeros
 *   workspace    at least fa_decode_fp8_workspace_query() bytes, 256-byte
 *                aligned (may be NULL where that is 0); calls that may overlap in time (other streams, graphs
 *                replayed beside each other) need one each
 *   max_seq_len  at most 2^31 - 513
 * Cache slots past a request's length may hold any codes, NaN included.  A NaN
 * code of V within the length makes its column NaN in all rows of the request
 * and K/V head, also in those that FA_MASK_CAUSAL hides it from (a weight of 0
 * times NaN).
 */
fa_status fa_decode_paged_fp8(const void *q, const void *k_cache, const void *v_cache,
                              const float *k_scale, const float *v_scale, const int *block_table,
                              const int *seq_lens, void *o, float *lse, void *workspace,
                              size_t workspace_bytes, int B, int H, int H_kv, int Sq, int d,
                              int block_size, int max_blocks, int num_blocks, int max_seq_len,
                              float scale, int mask_kind, int dtype, fa_stream_t stream);

/*
 * fa_decode_fp8_workspace_query -- workspace bytes fa_decode_paged_fp8 needs
 * on the current device and the status it would return for these sizes.
 * bytes must be non-NULL; it is 0 whenever the status is not FA_OK.
 */
fa_status fa_decode_fp8_workspace_query(int B, int H, int H_kv, int Sq, int d, int block_size,
                                        int max_blocks, int num_blocks, int max_seq_len, int mask_kind,
                                        int dtype, size_t *bytes);

/*
 * The paged cache in 4 bits.  A cached row of d components is in groups of
 * `group` (32 or 64) adjacent ones: codes c = 0 .. 15, two to a byte (component
 * 2i in the low half of byte i), and one 32-bit word per group: the scale s >= 0
 * (bf16) in its high half, the zero z (a whole number, |z| <= 2048, in fp16) in
 * its low half.  The value of a code is s (c - z).
 *   k_cache, v_cache  [num_blocks, H_kv, block_size, d / 2] bytes of codes
 *   k_scale, v_scale  [num_blocks, H_kv, block_size, d / group] words
 * all 16-byte aligned; d 64, 128 or 256; block_size 16, 32, 64 or 128.  Blocks,
 * tables and slots are those of fa_paged_update.  (0.625 bytes per value with
 * groups of 32, 0.5625 with 64.)
 */

/*
 * fa_cache_append_int4 -- writes new K and V rows into a 4-bit paged cache.  Per
 * group of values x_i of a row, lo and hi the smallest and largest of them:
 *     t   = max((hi - lo) / 15, max |x| / 2048), in fp32 (the difference and
 *           the quotient rounded to nearest), s = t rounded up to bf16
 *     n_i = x_i / s to the nearest whole number, ties to even
 *     c_i = min(n_i - min n, 15), z = -min n
 * so that a value is off by at most s / 2.  All zero: s, c and z are 0.  A group
 * with an infinity or NaN: s is NaN, c and z are 0.
 *
 *   k, v        [T, H_kv, d] 16-bit by element strides (token, head); values
 *               of a head adjacent; the strides are >= 0; T <= 2^30, H_kv <=
 *               65535
 *   slot_map    device int32 [T]: row t goes to slot s = block * block_size +
 *               place; rows whose slot is outside [0, num_blocks * block_size)
 *               are skipped.  Rows may stand in any order.  A slot named twice
 *               gets the later row where the two are less than 128 rows apart;
 *               farther apart, each of its groups is undefined
 *   dtype       FA_DTYPE_BF16 or FA_DTYPE_FP16 (k and v)
 * Slots without a row are left as they were.  T == 0: FA_OK.  Outputs may not
 * overlap inputs or each other.  One launch; no workspace.
 */
fa_status fa_cache_append_int4(const void *k, const void *v, long long k_token_stride,
                               long long k_head_stride, long long v_token_stride, long long v_head_stride,
                               const int *slot_map, void *k_cache, void *v_cache, unsigned *k_scale,
                               unsigned *v_scale, int T, int H_kv, int d, int group, int block_size,
                               int num_blocks, int dtype, fa_stream_t stream);

/*
 * fa_cache_read_int4 -- reads cached rows back in 16 bits, as the forward takes
 * K and V: row i of request b is its token starts[b] + i, each value s (c - z)
 * rounded once.
 *
 *   seq_lens    device int32 [B] (values outside [0, max_blocks * block_size]
 *               are clamped into it)
 *   starts      device int32 [B], or NULL: all 0
 *   k_out, v_out  [B, H_kv, rows, d] by element strides (batch, head, row) in
 *               host arrays of three, >= 0; every element must have an address
 *               of its own.  Rows whose token is below 0 or not below the
 *               request's length are left as they were
 *   block_table device int32 [B, max_blocks]; an entry outside [0, num_blocks)
 *               reads zeros
 *   dtype       FA_DTYPE_BF16 or FA_DTYPE_FP16 (k_out and v_out)
 * rows <= 2^30, H_kv <= 65535; rows == 0: FA_OK.  Outputs may not overlap inputs
 * or each other.  One launch; no workspace.
 */
fa_status fa_cache_read_int4(const void *k_cache, const void *v_cache, const unsigned *k_scale,
                             const unsigned *v_scale, const int *block_table, const int *seq_lens,
                             const int *starts, void *k_out, const long long *k_strides, void *v_out,
                             const long long *v_strides, int B, int H_kv, int rows, int d, int group,
                             int block_size, int max_blocks, int num_blocks, int dtype, fa_stream_t stream);

/*
 * fa_decode_paged_int4 -- fa_decode_paged over a 4-bit cache: exact softmax
 * attention over the values of its codes, q and o in 16 bits.  q enters exactly,
 * but for components below 2^-24 of their row's largest: those may be off by
 * 2^-34 of that.  A weight times its group's V scale is rounded to 11 bits before
 * P V (22 with fp16 q, and in bf16 with up to four rows per K/V head), and to no
 * finer than 2^-23 of the row's largest such product, both relative to a reference
 * of their own group's scales (2^-31 where these are alike).  The reference is
 * within 2^8 of the largest scale of 16 or 32 keys, so that a group whose scales lie
 * that far below it may lose 2^-15 of its own largest product.  Sums are fp32; those
 * of products are cut off, not rounded, at each of at most 512 in a row (2^-15 of
 * the sum of the weights times s (15 + |z|)).  Deterministic.  Two launches at most;
 * the workspace's contents on entry do not matter.  Arguments as for
 * fa_decode_paged, except:
 *
 *   k_cache, v_cache, k_scale, v_scale, group  as above; scales finite and >= 0
 *                or NaN
 *   q            components below 2^112 in size; a row with a larger one, an
 *                infinity or NaN gives NaN.  A row with a score (scale q k) of
 *                2^25 or more in size is undefined
 *   seq_lens     any length in [0, max_seq_len] (values outside are clamped
 *                into it).  A row that sees no key -- length 0, or with
 *                FA_MASK_CAUSAL a row in front of the request's first token --
 *                gets O = 0 and lse = -inf
 *   block_table  an entry outside [0, num_blocks) reads zeros
 *   workspace    at least fa_decode_int4_workspace_query() bytes, 256-byte
 *                aligned (may be NULL where that is 0); calls that may overlap
 *                in time need one each
 *   max_seq_len  at most 2^31 - 513
 * Slots past a request's length may hold anything.  A NaN scale of V within the
 * length makes its group's columns NaN in all rows of the request and K/V head,
 * also in those that FA_MASK_CAUSAL hides it from (a weight of 0 times NaN).
 */
fa_status fa_decode_paged_int4(const void *q, const void *k_cache, const void *v_cache,
                               const unsigned *k_scale, const unsigned *v_scale, const int *block_table,
                               const int *seq_lens, void *o, float *lse, void *workspace,
                               size_t workspace_bytes, int B, int H, int H_kv, int Sq, int d, int group,
                               int block_size, int max_blocks, int num_blocks, int max_seq_len,
                               float scale, int mask_kind, int dtype, fa_stream_t stream);

/*
 * fa_decode_int4_workspace_query -- workspace bytes fa_decode_paged_int4 needs
 * on the current device and the status it would return for these sizes.
 * bytes must be non-NULL; it is 0 whenever the status is not FA_OK.
 */
fa_status fa_decode_int4_workspace_query(int B, int H, int H_kv, int Sq, int d, int group,
                                         int block_size, int max_blocks, int num_blocks,
                                         int max_seq_len, int mask_kind, int dtype, size_t *bytes);

/*
 * fa_fwd_host -- the forward end to end from host memory: Q, K, V are
 * copied into a device workspace, the fused forward of fa_fwd_gqa runs there,
 * and O and lse are copied back to host memory.  The arithmetic and the
 * results are those of fa_fwd_gqa (the method's "what goes in, what comes
 * out" -- "FlashAttention: IO-aware attention kernels" -- with the host
 * copies around it).  The problem is cut into up to 8 chunks of whole K/V
 * heads (with the query heads that read them); chunk c+1's inputs are copied
 * in on a library stream while chunk c's forward runs on one of four library
 * compute streams (round robin, so a chunk too small to fill the GPU leaves
 * its idle SMs to the next one) and chunk c-1's outputs are copied out on a
 * further library stream, so the copies overlap the kernels and each other.
 *
 *   q_host, o_host  host pointers, [B, H, Sq, d] 16-bit (dtype)
 *   k_host, v_host  host pointers, [B, H_kv, Sk, d] 16-bit
 *   lse_host        host pointer, [B, H, Sq] fp32
 *                   Pinned (page-locked) host memory gives asynchronous
 *                   copies; pageable memory works but the copies then
 *                   serialise.  Device pointers are refused
 *                   (FA_ERR_INVALID_ARG): use fa_fwd / fa_fwd_gqa.
 *   workspace       device memory of at least fa_fwd_host_workspace_query()
 *                   bytes (Q, K, V, O and lse), 256-byte aligned; owned by
 *                   the caller; its contents on entry do not matter
 *   the rest        as for fa_fwd_gqa
 * The call returns once everything is enqueued; `stream` reaches its next
 * work only after O and lse have landed in host memory, so synchronising
 * `stream` is enough before reading them.  The host buffers and the
 * workspace must stay valid until then.  The library's copy and compute
 * streams and their events are created by the first call on a device (no
 * device memory is allocated); the enqueue of concurrent calls is
 * serialised by a lock.
 * Sq == 0: FA_OK, nothing is enqueued.  A CUDA error part way through the
 * enqueue returns FA_ERR_CUDA with the earlier chunks already enqueued.
 */
fa_status fa_fwd_host(const void *q_host, const void *k_host, const void *v_host,
                      void *o_host, float *lse_host, void *workspace, size_t workspace_bytes,
                      int B, int H, int H_kv, int Sq, int Sk, int d, float scale,
                      int mask_kind, int window, int dtype, fa_stream_t stream);

/*
 * fa_fwd_host_workspace_query -- device workspace bytes fa_fwd_host needs
 * (the 16-bit Q, K, V and O and the fp32 lse, each rounded up to 256 bytes)
 * and the status it would return for these sizes on the current device
 * (pointer checks aside).  bytes must be non-NULL; 0 unless FA_OK.
 */
fa_status fa_fwd_host_workspace_query(int B, int H, int H_kv, int Sq, int Sk, int d,
                                      int mask_kind, int window, int dtype, size_t *bytes);

/*
 * fa_workspace_query -- device scratch bytes fa_fwd needs for this problem
 * (always 0: the forward keeps every intermediate on chip, so its memory is
 * linear in the sequence length -- "FlashAttention: Why Tiling...", section
 * "The tiled forward pass").  Returns exactly the status fa_fwd would return
 * for these sizes on the current device (pointer checks aside), so it is also
 * the support probe: FA_OK means the fused kernel will run, never a fallback.
 * bytes must be non-NULL.
 */
fa_status fa_workspace_query(int B, int H, int Sq, int Sk, int d, int mask_kind,
                             int window, int dtype, size_t *bytes);

/* Human-readable name of a status code (static string, never NULL). */
const char *fa_status_string(fa_status status);

/*
 * fa_describe -- writes into buf (NUL-terminated, truncated to len) the kernel
 * and tile configuration fa_fwd selects for this head dim / mask / dtype, so
 * a caller can log which kernel ran.  FA_ERR_UNSUPPORTED if none would.
 */
fa_status fa_describe(int d, int mask_kind, int dtype, char *buf, size_t len);

/*
 * fa_get_device_error -- reads and clears the device status word of the
 * current device that kernels set when a pipeline wait times out.  The
 * caller synchronises the stream first.  FA_OK if no kernel raised it,
 * FA_ERR_DEVICE_TIMEOUT if one did, FA_ERR_CUDA if it cannot be read.
 * A kernel that times out stops its pipeline and finishes normally (its O
 * and lse are then undefined); the context stays usable.
 */
fa_status fa_get_device_error(void);

/*
 * fa_set_debug_stall_ms -- test hook for the timeout path.  With ms in
 * 1..10000, every later launch of every entry point makes its first softmax
 * (or compute-warp) wait one that nothing completes, with a limit of ms
 * instead of about 2 s: the wait runs out, the kernel winds down and raises
 * the device flag, without any fault.  0 turns the hook off (the default).
 * Process-wide; FA_ERR_INVALID_ARG outside 0..10000.
 */
fa_status fa_set_debug_stall_ms(int ms);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_H */
