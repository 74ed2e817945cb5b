/*
 * pa.h -- C ABI of libpa.so: single-query paged-attention decode on GB300 (sm_103a).
 *
 * The operation. "vLLM's custom ROCm paged-attention kernel wins all sixty cells"
 * (gqa-gate-costs-nothing), section 1, states the problem: pure decode, one query
 * token per sequence and head, attending over a fully cached context. The context
 * lives in a block-paged K/V cache addressed through a block table. For sequence b
 * of length L = seq_lens[b], query head h and its KV head g(h) = h / G (G = Hq/Hkv):
 *
 *   s_t      = scale * dot(q[b,h,:], K[b,t,g(h),:])            t < L
 *   out[b,h] = sum_t softmax(s)_t * V[b,t,g(h),:]
 *
 * where token t of sequence b is row (t % block_size) of physical block
 * block_tables[b][t / block_size]. Slots at or past L (the unwritten tail of the
 * last block, section 5 of the same page) are never read, so NaN there cannot
 * reach the output. The context is split across CTAs and merged afterwards (the
 * split-KV fix in "Hybrid-SSM decode rate on dual Radeon cards under vLLM"),
 * with fp32 accumulation throughout and one rounding to the output type.
 *
 * Conventions for every call below.
 *  - Pointers named q, k_cache, v_cache, block_tables, seq_lens, out, workspace
 *    are DEVICE pointers, owned by the caller; the library never allocates, frees
 *    or retains them, and keeps no state between calls.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) on the device current to the calling thread inside this library
 *    (see pa_set_device). Host-side argument errors are returned synchronously
 *    and nothing is launched.
 *  - Kernels are launched with programmatic stream serialization. Each one waits
 *    for the kernel before it in the stream to complete (griddepcontrol.wait)
 *    before reading any input, so inputs written by that kernel are safe. Each
 *    one also lets the next kernel in the stream start early: a kernel that the
 *    caller launches after a decode call with the programmatic-serialization
 *    attribute must wait in the same way (cudaGridDependencySynchronize) before
 *    it reads `out`; a kernel launched without the attribute needs nothing.
 *  - Layouts are dense, row-major, with no padding:
 *        q, out        [B, Hq, D]                       (dtype)
 *        k_cache,
 *        v_cache       [num_blocks, block_size, Hkv, D] (dtype, or one byte per element;
 *                      4-bit caches: head after head, see PA_INT4_ROW_BYTES)
 *        block_tables  [B, max_blocks_per_seq]          int32
 *        seq_lens      [B]                              int32
 *    q, k_cache, v_cache and out must be 16-byte aligned.
 *  - Device-side problems (a block table entry outside [0, num_blocks) for a live
 *    token, a seq_len that is negative or above max_seq_len or above
 *    max_blocks_per_seq*block_size) never fault:
 *    the kernel clamps, keeps going, and ORs a PA_DEVERR_* bit into the workspace
 *    header; read it with pa_read_device_errors. The output of such a call is
 *    finite but not meaningful.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_status {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misaligned pointer, Hq % Hkv != 0, G > 16 */
  PA_ERR_UNSUPPORTED = 2,   /* head_dim not 128/256, or an option this build does not implement */
  PA_ERR_WORKSPACE = 3,     /* workspace too small or misaligned */
  PA_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed (the CUDA error is cleared) */
  PA_ERR_OUT_OF_RANGE = 5   /* max_seq_len above max_blocks_per_seq * block_size, or a device error */
} pa_status;

typedef enum pa_dtype { PA_F16 = 0, PA_BF16 = 1 } pa_dtype;

/* Element type of the K/V caches in pa_decode_args.kv_dtype. */
typedef enum pa_kv_dtype {
  PA_KV_AS_DTYPE = 0, /* the caches have the q/out dtype */
  PA_KV_FP8_E4M3 = 1, /* FP8 E4M3 ("fn": bias 7, no infinities, max 448), one byte per
                         element; cache value = stored value * k_scale (K) or v_scale (V) */
  PA_KV_INT4 = 2      /* 4-bit codes in groups of 32, see PA_INT4_ROW_BYTES */
} pa_kv_dtype;

/*
 * A 4-bit cache. The D elements of a row (one token of one KV head) form D / 32 groups
 * of 32 consecutive elements. Group g has a step and a minimum in fp16, and element d of
 * it a code n in 0..15; the cache value is (minimum + step * n) * k_scale (K) or v_scale
 * (V). A row is PA_INT4_ROW_BYTES(D) bytes, 5 bits per element:
 *   D/2 bytes  codes, as 32-bit little-endian words of eight: the word of elements
 *              32 g + 8 t .. 32 g + 8 t + 7 (t = 0..3) is word t * (D/32) + g of the row,
 *              element 32 g + 8 t + j in its bits 4 j .. 4 j + 3
 *   D/16 bytes steps of the groups, then D/16 bytes minima
 * The pages hold head after head: k_cache and v_cache are
 * [num_blocks, Hkv, block_size, PA_INT4_ROW_BYTES(D)], so that a KV head's tokens of a
 * block are contiguous. pa_append writes such rows: the minimum rounded down and the step
 * (a fifteenth of the range above it) rounded up to fp16, and the nearest code. Values
 * beyond +-65280 saturate there. A group that holds a NaN or an infinity reads back as NaN.
 * Rows written otherwise: pa_decode needs steps <= 8734 in the V cache (weights times steps
 * are fp16).
 */
#define PA_INT4_ROW_BYTES(D) ((D) / 8 * 5)

/* Bits of the device error word (workspace header). */
#define PA_DEVERR_BLOCK_INDEX 1u /* a live token's block table entry was outside [0, num_blocks) */
#define PA_DEVERR_SEQ_LEN 2u     /* a seq_len < 0, > max_seq_len or > max_blocks_per_seq*block_size
                                    (pa_decode_shared: or a prefix_len) */
#define PA_DEVERR_COPY 4u        /* a copy into shared memory, or a wait for another part of the kernel,
                                    took over two seconds (pa_cross, pa_decode_shared: and some time for
                                    every token): no meaningful output */
#define PA_DEVERR_ROWS 8u        /* pa_cross, pa_decode_shared: starts or groups that do not ascend, or
                                    reach past the call's rows or sequences */

typedef void* pa_stream_t; /* cudaStream_t */

/* Largest query-head group (Hq / Hkv) a call accepts. */
#define PA_MAX_GQA_GROUP 16

/*
 * Full argument set for pa_decode_ex. Fields beyond those of pa_decode:
 *   splits  0 = choose the split count automatically (fill every SM even at batch 1);
 *           > 0 = use at most this many splits of the context (tests, tuning).
 *   window  0 = attend to the whole context; > 0 = sliding-window decode: each
 *           query attends to the last `window` tokens of its context, t in
 *           [max(0, L - window), L) (the sliding layers of "vLLM's custom ROCm
 *           paged-attention kernel wins all sixty cells", section 4, scan 1024).
 *           Table entries before the window are not read.
 *   kv_dtype  PA_KV_AS_DTYPE (default), PA_KV_FP8_E4M3 or PA_KV_INT4. FP8 caches hold one byte
 *           per element, [num_blocks, block_size, Hkv, D] as before; q and out keep
 *           `dtype`. fp8 K/V are widened exactly to fp16 for the tensor-core
 *           products (the queries are rounded to fp16, so bf16 query elements must
 *           lie within fp16's range, |x| <= 65504; P is kept in fp16) with fp32
 *           accumulation. The pages list an fp8 cache as untested ("vLLM's custom
 *           ROCm paged-attention kernel wins all sixty cells", section 6).
 *           4-bit caches (layout above): the codes enter the tensor-core products exactly
 *           as fp16, the queries rounded to fp16 after scaling by a power of two (any
 *           range up to 2^110 / (scale * k_scale)), the weights rounded to fp16 and once more
 *           after multiplication by the steps, with fp32 accumulation; nothing else is rounded.
 *           v_scale should leave the larger steps above about 2^-10 (values / v_scale
 *           around 1): smaller products with weights lose bits to fp16's 2^-24.
 *   k_scale, v_scale  per-tensor dequantisation scales (finite, > 0) for an fp8 or
 *           4-bit cache; ignored otherwise.
 *   q_len   query rows per sequence (0 or 1 = single-query decode). With R > 1 rows,
 *           q and out are [B, R, Hq, D]: row i is the query of token L - R + i (the
 *           new tokens of a speculative-decode step or a chunked-prefill tail) and
 *           attends causally to the tokens t < L - R + i + 1; a row that sees no
 *           token gets zeros. Every K/V tile is read once for all rows and heads of
 *           its KV head. Limits: G * R <= 32 at head_dim 128, <= 16 at 256; not
 *           combined with a window (PA_ERR_UNSUPPORTED). Cached values must be finite:
 *           a NaN or an infinity in V at one of the sequence's tokens reaches the rows
 *           that do not see it too.
 *   flags   0 or PA_FLAG_DETERMINISTIC. By default, when a long context is split
 *           across CTAs, the splits share out its last eighth tile by tile as
 *           they finish their own shares, so the order of the fp32 sums depends
 *           on timing and repeated calls may differ in the last bit (each within
 *           the usual error). PA_FLAG_DETERMINISTIC keeps fixed splits: repeated
 *           calls give bitwise identical outputs. Other bits: PA_ERR_INVALID_ARG.
 *   total_tokens  0, or the sum of seq_lens over the batch, known on the host like
 *           max_seq_len. It lets the planner estimate how many context splits hold
 *           tokens in a batch of mixed lengths; only the split plan depends on it
 *           (a wrong value costs speed, not correctness). Negative, or above
 *           B * max_seq_len: PA_ERR_INVALID_ARG. Ignored with a window.
 * All other fields mean what the pa_decode parameters of the same name mean.
 */
typedef struct pa_decode_args {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  void* out;
  int32_t B, Hq, Hkv, D;
  int32_t block_size, num_blocks, max_blocks_per_seq, max_seq_len;
  float scale;
  int32_t dtype; /* pa_dtype */
  int32_t splits;
  int32_t window;
  int32_t kv_dtype; /* pa_kv_dtype */
  float k_scale, v_scale;
  int32_t q_len;
  uint32_t flags;
  int64_t total_tokens;
} pa_decode_args;

#define PA_FLAG_DETERMINISTIC 1u

/*
 * Workspace bytes pa_decode needs for these sizes on the current device (the
 * problem's sizes and the host-side bound on seq_lens; the split plan does not
 * depend on the block size, so the query does not take one). The
 * workspace starts with a header of PA_WORKSPACE_HEADER_BYTES that must be zero
 * before the first call (pa_workspace_init or any memset): the device error word
 * (first 4 bytes) and one counter per (sequence, KV head) through which the
 * splits of a sequence share out the tail of its context; every call leaves the
 * counters zero again. After the header come the fp32 split partials (m, l, acc),
 * which every call writes before it reads them. One workspace serves calls of
 * any shape that fit its size; calls that overlap on the GPU must not share one. (Host
 * threads that call on one stream may: the kernels of a call are queued one behind the
 * other.)
 * Returns 0 for invalid sizes (max_seq_len must be > 0 here).
 */
#define PA_WORKSPACE_HEADER_BYTES 8448u
size_t pa_decode_workspace_bytes(int B, int Hq, int Hkv, int D, int max_seq_len);

/* Same, for pa_decode_ex's argument set (pointer fields are ignored). */
size_t pa_decode_ex_workspace_bytes(const pa_decode_args* args);

/*
 * Single-query paged-attention decode: the call of the problem statement in "vLLM's
 * custom ROCm paged-attention kernel wins all sixty cells" (gqa-gate-costs-nothing),
 * section 1 (one query token per sequence and head over a fully cached, block-paged
 * context), with the split-KV partition and reduce of "Hybrid-SSM decode rate on dual
 * Radeon cards under vLLM" (its split-KV paragraph) chosen inside the call.
 *   q             [B, Hq, D] queries (dtype)
 *   k_cache,
 *   v_cache       [num_blocks, block_size, Hkv, D] paged keys / values (dtype)
 *   block_tables  [B, max_blocks_per_seq] int32 physical block of each logical block;
 *                 entries past ceil(seq_lens[b] / block_size) are never read
 *   seq_lens      [B] int32 context length per sequence (0 gives a zero output row)
 *   out           [B, Hq, D] output (dtype), fully written
 *   B             batch (0 is a no-op), Hq and Hkv query and KV heads (Hq % Hkv == 0,
 *                 Hq / Hkv <= PA_MAX_GQA_GROUP), D head_dim (128 or 256)
 *   block_size    tokens per block (any positive size, e.g. 16 or 784)
 *   num_blocks    blocks in each cache tensor
 *   max_seq_len   a host-side upper bound on seq_lens (used to choose the split
 *                 count without reading device memory); <= 0 means
 *                 max_blocks_per_seq * block_size
 *   scale         softmax scale applied to q.k (e.g. 1/sqrt(D))
 *   dtype         PA_F16 or PA_BF16 for q, caches and out
 *   workspace     device scratch of >= pa_decode_workspace_bytes(...) bytes,
 *                 256-byte aligned, its header zero before first use
 * Errors: PA_ERR_INVALID_ARG, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE,
 * PA_ERR_OUT_OF_RANGE (max_seq_len above capacity), PA_ERR_CUDA. On PA_ERR_CUDA a
 * kernel of the call may already be queued; the call then also queues, behind it on
 * `stream`, a clearing of the workspace header (tile counters and device error word),
 * so that the workspace stays usable if the context does.
 */
pa_status pa_decode(const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* seq_lens, void* out,
                    int B, int Hq, int Hkv, int D, int block_size, int num_blocks,
                    int max_blocks_per_seq, int max_seq_len, float scale, pa_dtype dtype,
                    void* workspace, size_t workspace_bytes, pa_stream_t stream);

/* pa_decode with the extra options of pa_decode_args. Same errors. */
pa_status pa_decode_ex(const pa_decode_args* args, void* workspace, size_t workspace_bytes,
                       pa_stream_t stream);

/*
 * The launch plan pa_decode_ex would use on a GPU with `sm_count` SMs: the number
 * of context splits and the tokens per split, a whole number of warp tiles (32
 * tokens at head_dim 128 and for fp8 and 4-bit caches, 16 at head_dim 256). It depends on
 * the sizes, max_seq_len, window, kv_dtype, splits and total_tokens of `args`, and for
 * 4-bit caches on q_len. Pure host arithmetic; needs no GPU. sm_count <= 0 means the
 * current device's SM count.
 */
pa_status pa_decode_plan(const pa_decode_args* args, int sm_count, int* splits,
                         int* partition_tokens);

/*
 * How many kernels pa_decode_ex would launch for `args` on the current device (the
 * plan, and whether the splits merge inside their thread-block clusters, depend on
 * the device): 0 for B == 0, 1 for a context in one split or splits that merge in
 * their cluster, 2 for a decode grid followed by a merge grid. Pointer fields are
 * not read; nothing is launched. The same argument errors as pa_decode_ex.
 */
pa_status pa_decode_kernel_count(const pa_decode_args* args, int* kernels);

/* Zero-fill a workspace on `stream` (asynchronous). */
pa_status pa_workspace_init(void* workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * Wait for `stream`, then copy the device error word (PA_DEVERR_* bits) of
 * `workspace` to *flags and clear it. Synchronous.
 */
pa_status pa_read_device_errors(void* workspace, pa_stream_t stream, uint32_t* flags);

/* Make `device` current for this library's calls on the calling thread. */
pa_status pa_set_device(int device);

/*
 * pa_decode without a workspace, for callers that cannot allocate device memory
 * or pass scratch to the library: for example a plugin inside another runtime
 * that owns all device allocations, code that must not call cudaMalloc because
 * it may synchronise the device, or a binding with no device allocator. The pages
 * describe no such call; it exists only for those callers.
 *
 * Arguments, layouts, validation and results are those of pa_decode. The split
 * partials live in one array of PA_NOALLOC_SCRATCH_BYTES that is part of this
 * library's device image: every GPU that loads it keeps that memory until the
 * process exits, and the call itself allocates nothing (no cudaMalloc, no
 * cudaFree, no allocating library routine).
 *  - Limit: a call whose partials need more than PA_NOALLOC_SCRATCH_BYTES (as
 *    pa_decode_workspace_bytes reports) returns PA_ERR_WORKSPACE and launches
 *    nothing; use pa_decode with your own workspace for it.
 *  - The first call on a device looks up the array's device address (once, kept
 *    for the life of the process) and clears the array's header with an
 *    asynchronous memset on `stream`, ordered before that call's kernels; make that
 *    first call before any stream capture on that device. The address belongs to
 *    the device's current context: after cudaDeviceReset on a device, this entry
 *    point must not be called on it again in the same process.
 *  - Every call on a device shares the one array, which keeps the last call's
 *    contents. Nothing in it needs to start at zero except its header (the tile
 *    counters, which every successful call leaves at zero, and the error word).
 *    Calls that may overlap on the GPU (different streams, concurrent threads)
 *    race on it: serialise them. A call that returns PA_ERR_CUDA queues a clearing
 *    of the header on `stream`, as pa_decode does for its workspace.
 *  - Device-side range errors (PA_DEVERR_*) are recorded in the array's header
 *    and are not readable through this API.
 */
#define PA_NOALLOC_SCRATCH_BYTES (32u << 20)
pa_status pa_decode_noalloc(const void* q, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* seq_lens, void* out,
                            int B, int Hq, int Hkv, int D, int block_size, int num_blocks,
                            int max_blocks_per_seq, int max_seq_len, float scale,
                            pa_dtype dtype, pa_stream_t stream);

/*
 * Rotary positions: how a pair of a head's elements turns with its token's position t.
 * With n = rot_dim / 2 pairs, pair i of the first rot_dim elements is (x[i], x[i + n])
 * (PA_ROPE_HALF) or (x[2 i], x[2 i + 1]) (PA_ROPE_INTERLEAVED); elements past rot_dim
 * stay. It turns by the angle t * f_i and is multiplied by the amplitude a:
 *   (x, y) -> a (x cos - y sin, y cos + x sin)
 * f_i is held as a fraction of a full turn in units of 2^-64, turns[i] = f_i / 2 pi * 2^64
 * (modulo 2^64), so that the angle is exact at far positions.
 */
typedef enum pa_rope_layout { PA_ROPE_HALF = 0, PA_ROPE_INTERLEAVED = 1 } pa_rope_layout;

/*
 * Frequencies for contexts longer than the original_max tokens that a model was trained
 * on, by a factor (>= 1); plain frequencies are f_i = base^(-i / n):
 *   PA_ROPE_LINEAR  f_i / factor: positions interpolated
 *   PA_ROPE_NTK     the base becomes base * factor^(rot_dim / (rot_dim - 2)): the slowest
 *                   pair interpolated, the fastest kept
 *   PA_ROPE_YARN    pairs that make more than `fast` turns over original_max kept, those
 *                   that make fewer than `slow` divided by factor, a linear ramp over the
 *                   pair index between; amplitude 0.1 ln(factor) + 1
 *   PA_ROPE_BANDED  the same two bands, the ramp linear in the number of turns;
 *                   amplitude 1
 */
typedef enum pa_rope_kind {
  PA_ROPE_PLAIN = 0, PA_ROPE_LINEAR = 1, PA_ROPE_NTK = 2, PA_ROPE_YARN = 3, PA_ROPE_BANDED = 4
} pa_rope_kind;
typedef struct pa_rope_scaling {
  int32_t kind; /* pa_rope_kind */
  int32_t original_max;
  double factor, slow, fast;
} pa_rope_scaling;

/*
 * turns[0 .. rot_dim / 2) and the amplitude for a base (> 1) and a scaling (NULL: plain).
 * rot_dim: a multiple of 16 up to 256. Host arithmetic in fp64; needs no GPU. Callers with
 * frequencies of their own fill turns themselves.
 */
pa_status pa_rope_turns(int rot_dim, double base, const pa_rope_scaling* scaling, uint64_t* turns,
                        float* amplitude);

/*
 * Append the keys and values of new tokens to a paged cache, the keys rotated to their
 * positions, and rotate the queries of the same tokens: what precedes pa_decode in a step,
 * with the same block_tables and seq_lens.
 *   q, q_out  queries in and rotated queries out, or both NULL. q_out is dense
 *             [rows, Hq, D]; it may be q itself when q is dense too
 *   k, v      [rows, Hkv, D] keys and values (dtype). Row r of q, k, v starts at element
 *             r * stride (a multiple of 8, e.g. the width of a fused projection whose
 *             slices they are); the heads of a row are dense
 *   starts    NULL: every sequence has `rows` new tokens, row b * rows + i is token i of
 *             sequence b. Else [B + 1] ascending int32 on the device: rows starts[b] to
 *             starts[b + 1] - 1 belong to sequence b, `rows` is the number of rows in all;
 *             rows before starts[0] and from starts[B] on are padding, neither read into
 *             the cache nor written in q_out
 *   seq_lens  [B] context lengths WITH the new tokens: token i of n has position
 *             seq_lens[b] - n + i. A row whose position is negative has no token: nothing
 *             is written to the cache and its q_out row is zero
 *   k_cache, v_cache, block_tables, block_size, num_blocks, max_blocks_per_seq, kv_dtype
 *             as for pa_decode; the table entries of the new positions must be filled
 *   k_scale, v_scale  for fp8 and 4-bit caches: the cache holds value / scale (E4M3
 *             saturates at +-448, nearest even; 4 bits: see PA_INT4_ROW_BYTES)
 *   rot_dim   elements of a head that turn: 0 (none) or a multiple of 16 up to D
 * Angles are rounded to fp32 relative to the nearest quarter turn. Sines and cosines, their
 * products with the amplitude, the rotation and the (correctly rounded) quotients by a scale
 * are fp32; what is stored is rounded once from that. A row with
 * an invalid length or table entry is not written to the cache and raises a PA_DEVERR_*
 * bit. Two rows of one call that name the same cache slot leave either's values there, or
 * a mixture. `workspace`: >= PA_WORKSPACE_HEADER_BYTES, 256-byte aligned; only its error
 * word is used, so it may be the workspace of the decode calls on the stream. Errors as
 * for pa_decode; q, q_out, k, v and the caches must be 16-byte aligned.
 */
typedef struct pa_append_args {
  const void* q;
  void* q_out;
  const void* k;
  const void* v;
  void* k_cache;
  void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* starts;
  const uint64_t* rope_turns; /* [rot_dim / 2] on the device */
  int64_t q_stride, k_stride, v_stride;
  int32_t B, rows, Hq, Hkv, D;
  int32_t block_size, num_blocks, max_blocks_per_seq;
  int32_t dtype;    /* pa_dtype */
  int32_t kv_dtype; /* pa_kv_dtype */
  float k_scale, v_scale;
  int32_t rot_dim;
  int32_t rope_layout; /* pa_rope_layout */
  float rope_amplitude;
} pa_append_args;

pa_status pa_append(const pa_append_args* args, void* workspace, size_t workspace_bytes,
                    pa_stream_t stream);

/*
 * Read rows back from a paged cache into dense k_out, v_out [rows, Hkv, D] (dtype): the
 * reverse of pa_append's writing, with the same meaning of rows, starts and seq_lens (the
 * last n tokens of each sequence; n = seq_lens[b] is the whole context), for attention of a
 * prompt over its cached prefix. fp8 and 4-bit values are multiplied by k_scale, v_scale
 * and rounded once; keys stay rotated. A row without a token, or with an invalid length or
 * table entry, is zero; padding rows are left alone.
 */
typedef struct pa_gather_args {
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* starts;
  void* k_out;
  void* v_out;
  int32_t B, rows, Hkv, D;
  int32_t block_size, num_blocks, max_blocks_per_seq;
  int32_t dtype;    /* pa_dtype */
  int32_t kv_dtype; /* pa_kv_dtype */
  float k_scale, v_scale;
} pa_gather_args;

pa_status pa_gather(const pa_gather_args* args, void* workspace, size_t workspace_bytes,
                    pa_stream_t stream);

/*
 * Cross attention: query rows over a context of another length, for example a decoder's tokens
 * over an encoder's states held in a paged cache. Every row of sequence b sees all seq_lens[b]
 * tokens of its context:
 *   out[r,h] = sum_t softmax(scale * q[r,h] . K[b,t,h / G])_t * V[b,t,h / G]    t < seq_lens[b]
 * Any number of rows: a few (the beams of a search, which share their source), or a prompt's
 * thousands. (One row a sequence is pa_decode_ex's result, which takes half the time over short
 * contexts of few sequences, 5 us instead of 11, and about the same over many.)
 *   q         [rows, Hq, D] (dtype); row r starts at element r * q_stride (a multiple of 8, at
 *             least Hq * D, below 2^39), the heads of a row are dense
 *   starts    as for pa_append: NULL, and sequence b has the `rows` rows b * rows + i; or [B + 1]
 *             ascending int32 on the device, and `rows` is the number of rows in all. Rows of no
 *             sequence are padding, left alone in out
 *   out       dense [rows, Hq, D], apart from q; rows over an empty context (seq_lens[b] = 0) are zero
 *   k_cache, v_cache, block_tables, seq_lens, max_seq_len, kv_dtype, k_scale, v_scale
 *             as for pa_decode_ex, with 16-bit and fp8 caches (with fp8 the queries are rounded to
 *             fp16: |x| <= 65504). 4-bit caches: PA_ERR_UNSUPPORTED
 * G = Hq / Hkv up to PA_MAX_GQA_GROUP; rows * Hq below 2^31. Scores, softmax
 * statistics and sums are fp32; the weights are rounded to the type of the products (dtype, fp16
 * for fp8 caches), the output once. The work is divided among the SMs by the lengths found on the
 * device: the host needs none of them, and repeated calls give the same bits. `workspace`:
 * pa_cross_workspace_bytes, 256-byte aligned, its header zero before first use, as for pa_decode;
 * calls that overlap on the GPU must not share one.
 */
typedef struct pa_cross_args {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* starts;
  void* out;
  int64_t q_stride;
  int32_t B, rows, Hq, Hkv, D;
  int32_t block_size, num_blocks, max_blocks_per_seq, max_seq_len;
  float scale;
  int32_t dtype;    /* pa_dtype */
  int32_t kv_dtype; /* pa_kv_dtype */
  float k_scale, v_scale;
} pa_cross_args;

/* Workspace bytes of a pa_cross call on the current device (pointers are not read, but whether
 * starts is NULL matters); 0 for invalid sizes. */
size_t pa_cross_workspace_bytes(const pa_cross_args* args);

pa_status pa_cross(const pa_cross_args* args, void* workspace, size_t workspace_bytes,
                   pa_stream_t stream);

/*
 * Decode for sequences that share prefixes: pa_decode_ex's result, with the keys and values of a
 * shared prefix read once for all sequences of its group. (Faster than pa_decode_ex on GB300 from
 * about 100 MB of 16-bit keys and values on that are not read again, 200 MB of fp8 ones: 16
 * sequences behind 2048 tokens of 8 heads of 128, or 4 behind 8192.)
 *   args         as for pa_decode_ex, with q_len causal query rows per sequence (any number) and out
 *                apart from q;
 *                16-bit and fp8 caches (4 bits: PA_ERR_UNSUPPORTED); splits and window must be 0
 *   groups       [num_groups + 1] ascending int32 on the device: sequences groups[n] to
 *                groups[n + 1] - 1 are group n. Sequences of no group share nothing
 *   prefix_lens  [num_groups] int32 on the device: how many leading tokens they share. What is
 *                shared is the first min(prefix_lens[n], seq_lens[groups[n]]) tokens, any number
 *                of them, read through the table row of the group's FIRST sequence; the others'
 *                entries, and slots of their own blocks, before that are not used
 * A row sees what it sees in pa_decode_ex: tokens t < seq_lens[b] - q_len + i + 1, the shared ones
 * among them; a row that sees none is zero. Cached values must be finite at the tokens of a group's
 * prefix and of each sequence: a NaN or an infinity in V reaches rows that do not see its token
 * too. Repeated calls give the same bits. Rounding and limits as for pa_cross, with B * q_len
 * rows. `workspace`: pa_decode_shared_workspace_bytes, as for pa_decode.
 */
size_t pa_decode_shared_workspace_bytes(const pa_decode_args* args, int num_groups);

pa_status pa_decode_shared(const pa_decode_args* args, const int32_t* groups,
                           const int32_t* prefix_lens, int num_groups, void* workspace,
                           size_t workspace_bytes, pa_stream_t stream);

/* Static text for a status code. */
const char* pa_status_string(pa_status status);

/* Library version, e.g. "0.1.0". */
const char* pa_version(void);

#ifdef __cplusplus
} /* extern "C" */
#endif

#endif /* PA_H_ */
