/*
 * pkv -- decode attention over a paged KV cache, for GB300 (sm_103a).
 *
 * C ABI.  Every pointer argument is either a host pointer (marked "host") or
 * device memory the caller owns (marked "device"); the library allocates
 * nothing and keeps no state between calls.  Each call that launches work is
 * asynchronous and stream-ordered on `stream` (a cudaStream_t passed as
 * void*), never synchronises the host, and may be captured into a CUDA graph:
 * lengths and segment layout are read from device memory when the kernels
 * run, so one capture serves every length the grid was sized for.
 *
 * Errors come back two ways.  Problems visible on the host (bad sizes, null
 * or misaligned pointers, an unsupported head_dim or dtype) return a negative
 * pkv_status before anything is launched.  Problems only the device sees (a
 * segment whose fields are out of range, a block id outside the pool, ...)
 * set PKV_ERR_* bits in the caller's `err_flags` word with an atomic OR and
 * zero that segment's output; no kernel traps or asserts, and every wait
 * inside a kernel is bounded.
 *
 * Sources, by page and section:
 *   [vllm-omni paged_decode.py]  "Paged KV cache for SenseNova-U1
 *       autoregressive decode" (vLLM-Omni): module constants BLOCK_SIZE,
 *       BUCKETS, TAIL_STEP and _bucket_for; PagedDecodeCache (layout,
 *       attend, grow, load_prefix, reusable_for, to_dynamic_cache);
 *       DecodeGraphRunner.
 *   [tiny-llm kv_cache.py]  causal_kwargs; SlotKVCache.end_step /
 *       advance_host; SlotLayerKV.update.
 *   [ExecuTorch #24072]  triton::sdpa_varlen over a seq_info segment table.
 *   [ExecuTorch #24073]  CudaBatchedSequenceCache: ring rows, scratch column.
 *   [ExecuTorch #24074]  batched-sequence manifest: ring slot formula,
 *       max_segments, per-call causal flag.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens per page ([vllm-omni paged_decode.py] BLOCK_SIZE). */
#define PKV_BLOCK_SIZE 16

typedef enum pkv_status {
    PKV_OK = 0,
    PKV_EMPTY = 1,          /* nothing to do (an empty prefix); not an error */
    PKV_SAME_BUCKET = 2,    /* resize not needed: the length fits the current bucket */
    PKV_EINVAL = -1,        /* an argument is out of range, null or misaligned */
    PKV_EUNSUPPORTED = -2,  /* dtype or head_dim the kernels do not cover */
    PKV_ECUDA = -3,         /* a CUDA launch or copy failed to enqueue */
    PKV_ECAPACITY = -4,     /* the destination cannot hold the requested tokens */
    PKV_ESTALE = -5         /* descriptors that do not describe the same cache shape */
} pkv_status;

/*
 * PKV_FP4 is a cache format: K and V values are e2m1 numbers times a scale
 * shared by 16 consecutive head_dim columns of a token and kv head, 4.5 bits
 * a value.  The scale is an unsigned 8-bit float s of 5 exponent (bias 15)
 * and 3 mantissa bits, the nearest one to max|x| / 6 (ties to even, at most
 * 10240); the code is the nearest e2m1 number to x / s (ties to even, 0 where
 * s is 0, the sign kept).  A group that holds a NaN reads back as NaN, an
 * infinity as its scale's largest value.  Rows (q, k_new, v_new) are bf16.
 */
/*
 * PKV_FP8 is another: values are e4m3 numbers (the finite ones, up to 448) times
 * a scale 2^e shared by the 16 tokens of a page and kv head.  e is the smallest by which
 * every value fits, -126 to 119; the code is the nearest e4m3 number to x / 2^e, ties to
 * even.  A page is filled as tokens come: those that are in it keep e from
 * getting smaller, and where a new one makes it larger, their codes are rounded to the larger one
 * (exact down to 2^-6 times the scale, by at most 2^-10 times it below).  A
 * page whose new rows begin at its first slot starts afresh.  With ring storage the slots that the
 * sequence has not come to hold nothing, whatever an earlier one left there, and
 * e comes down (exactly) where it is more than 6 above what the new rows need and the tokens that the window of the
 * call's first row still reaches; tokens further back, until they are overwritten, saturate then.  A token of a kv head that holds a NaN
 * reads back as NaN, all of it, and an infinity as 448 * 2^119.  Rows are bf16.
 */
typedef enum pkv_dtype { PKV_BF16 = 0, PKV_F32 = 1, PKV_FP4 = 2, PKV_FP8 = 8 } pkv_dtype;

/* Device-side error bits, OR-ed into *err_flags. */
#define PKV_ERR_SEGMENT  (1u << 0)  /* q_start/q_len/col/kv_end out of range, or kv_end < q_len */
#define PKV_ERR_CAPACITY (1u << 1)  /* flat layout: kv_end > max_blocks_per_seq * 16 */
#define PKV_ERR_RING     (1u << 2)  /* ring layout: window <= 0 or window + q_len - 1 > ring_rows */
#define PKV_ERR_BLOCK    (1u << 3)  /* a block-table entry the segment needs is outside [0, num_blocks) */
#define PKV_ERR_QLEN     (1u << 4)  /* q_len above the max_q_len the launch was sized for */
#define PKV_ERR_OVERLAP  (1u << 5)  /* an output row lies in two segments (its value is then unspecified) */
#define PKV_ERR_TIMEOUT  (1u << 6)  /* a bounded wait for a K/V copy inside the kernel gave up; output zeroed */

/* Flags for the attention calls. */
#define PKV_FLAG_SIMT  (1u << 0)  /* bf16: use the CUDA-core kernels instead of the tensor-core ones */
#define PKV_FLAG_PDL   (1u << 1)  /* launch with programmatic dependent launch; see pkv_attend_varlen */
#define PKV_FLAG_PREFETCH_NEXT (1u << 2)  /* warm L2 with layer + 1's pages; see pkv_attend_varlen */
#define PKV_FLAG_MMA_SYNC (1u << 3)  /* bf16, head_dim 128, > 8 rows per kv head: mma.sync tile instead of tcgen05 */
#define PKV_FLAG_OUT_BF16 (1u << 4)  /* PKV_FP4 and PKV_FP8 caches: out is bf16 (it is fp32 otherwise) */

/*
 * One paged K/V cache: per layer, a K pool and a V pool, each
 * (num_blocks, 16, kv_heads, head_dim) of `dtype`, row-major
 * ([vllm-omni paged_decode.py] PagedDecodeCache docstring), plus one block
 * table shared by all layers, int32 (max_seqs, max_blocks_per_seq), row
 * `col` listing the pages of sequence `col` in order.
 *
 * ring_rows = 0 means flat storage: position p lives at page p / 16, offset
 * p % 16 of the sequence's table row, so a sequence holds at most
 * max_blocks_per_seq * 16 tokens.  ring_rows = R > 0 (a multiple of 16, at
 * most max_blocks_per_seq * 16) means ring storage for sliding-window
 * attention: position p lives at slot p % R ([ExecuTorch #24074]), and a
 * window of W keys with steps of up to q_len rows needs
 * R >= W + q_len - 1 ([ExecuTorch #24073]).
 *
 * A PKV_FP4 cache has head_dim 64, 128 or 256 (D below), and pools of bytes,
 * (num_blocks, kv_heads, 9 * D): 8 * D bytes of codes of the page's 16 tokens,
 * then D bytes of scales.  In a K block the code of (token, column) is in byte
 * token * D / 2 + column / 2 (even columns in the low nibble) and its scale at
 * 8 * D + token * D / 16 + column / 16.  In a V block, with token = 8 * hi +
 * 2 * t + n and column = g * D / 8 + 8 * p + i, it is in byte 512 * p +
 * 16 * (4 * g + t) + 2 * i + hi, nibble n, and its scale at 8 * D +
 * 4 * (4 * (column / 16) + t) + 2 * hi + n.
 *
 * A PKV_FP8 cache has the same head_dims, and pools of (num_blocks, kv_heads,
 * 16 * D + 16) bytes: 16 rows of D codes, then 16 bytes: e + 127 (0: no
 * scale yet, every value zero), 0, a 16-bit mask (low byte first) of the tokens that hold a NaN,
 * whose NaN codes are 0, and twelve bytes that are not used.  The
 * 16 codes from column 16 * c on of token t are in place c ^ (((t & 6) ^ (t & 1) << 2)
 * % (D / 16)) of its row.  Pools are zero-filled before their first use.
 *
 * The append and attention calls, pkv_rewind, pkv_advance and
 * pkv_seqinfo_from_seqused take quantised caches (PKV_FP4, PKV_FP8), and
 * pkv_to_contiguous takes PKV_FP8; the other copying calls (pkv_seq_clone,
 * pkv_resize_bucket, pkv_load_prefix) return PKV_EUNSUPPORTED for them.
 *
 * The descriptor is host memory owned by the caller; k and v are host arrays
 * of num_layers device pointers (16-byte aligned).  bucket is the token
 * capacity the buffers were sized for and generation counts reallocations
 * ([vllm-omni paged_decode.py] PagedDecodeCache.generation); the library
 * reads both and writes generation only in pkv_resize_bucket.
 *
 * first_valid (optional, NULL = no padding) is a device int32 array with one
 * entry per table row: the sequence's first valid position, for batches of
 * left-padded sequences ([tiny-llm kv_cache.py] SlotKVCache,
 * padded_causal_mask).  Every query row of that sequence then ignores the
 * keys before it, and a query row whose own position lies before it (a
 * padding row) attends to its own key alone, so no row is empty.  A
 * negative entry counts as 0.  Only the attention calls read it, before the
 * dependency wait like the block table, so the kernel launched just before
 * a PDL attention call must not write it.
 */
typedef struct pkv_cache {
    int32_t num_layers;
    int32_t kv_heads;
    int32_t head_dim;           /* multiple of 8, at most 256 */
    int32_t dtype;              /* pkv_dtype */
    int64_t num_blocks;
    int32_t max_seqs;
    int32_t max_blocks_per_seq;
    int32_t ring_rows;
    int32_t reserved0;
    void *const *k;             /* host array [num_layers] of device pointers */
    void *const *v;             /* host array [num_layers] of device pointers */
    const int32_t *block_table; /* device [max_seqs][max_blocks_per_seq] */
    int64_t bucket;
    int64_t generation;
    const int32_t *first_valid; /* device [max_seqs] or NULL; see above */
} pkv_cache;

/*
 * Growth schedule of the single-sequence decode cache
 * ([vllm-omni paged_decode.py] _bucket_for): the first of 512, 1024, 2048,
 * 4096, 8192 that holds `length`; past 8192, 8192 plus as many 2048-token
 * steps as cover the rest.  length <= 0 returns 512.  Host only.
 */
int64_t pkv_bucket_for(int64_t length);

/* Static string for a pkv_status value. */
const char *pkv_status_str(int status);

/*
 * Append this step's K/V rows ([vllm-omni paged_decode.py]
 * PagedDecodeCache.attend, which writes at length - 1 because the caller has
 * already advanced the length; [tiny-llm kv_cache.py] SlotLayerKV.update).
 *
 * seq_info: device int32 [num_segments][4] = (q_start, q_len, col, kv_end)
 * ([ExecuTorch #24072]).  kv_end counts the sequence's keys after this
 * append, so query row q_start + i (0 <= i < q_len) is the token at position
 * kv_end - q_len + i, and its K and V rows are copied bit for bit into that
 * position's slot of sequence `col`.
 * k_new, v_new: device [total_rows][kv_heads][head_dim] of the cache dtype.
 * window: the attention window the rows will be used with (checked against
 * ring_rows when the cache is a ring; ignored for flat storage).
 *
 * A segment is written only if it is valid as a whole: 0 <= q_start,
 * q_start + q_len <= total_rows, 0 <= col < max_seqs, q_len <= kv_end, the
 * capacity / ring rule above holds and every slot it writes maps to a block
 * id in [0, num_blocks).  Otherwise nothing of it is written and the matching
 * PKV_ERR_* bit is set.  Rows no segment covers are not written.  Two
 * segments that write the same slot race (unspecified result).
 * err_flags: device uint32, OR-ed, never cleared by the library.
 *
 * On a PKV_FP4 cache the rows are bf16 and are quantised on the way (this is
 * pkv_norm_rope_append without a pkv_rope and without q).  A byte of its V
 * pages holds two tokens; calls and segments that write different slots of
 * one page, or the same row to one slot, at the same time do not disturb each
 * other.
 *
 * On a PKV_FP8 cache they are quantised as well, and the page's scale is shared:
 * the segments of one call may write different slots of a page in the same column (the
 * lowest of them writes the page; of rows for one slot the highest segment's counts),
 * and a segment may be in the table twice, but columns whose tables name one page must
 * not both write it, in one call or in two at a time.  An append is at its sequence's
 * end: tokens that such a page holds at kv_end and later are not kept.
 */
int pkv_append(const pkv_cache *cache, int32_t layer,
               const void *k_new, const void *v_new, int32_t total_rows,
               const int32_t *seq_info, int32_t num_segments, int32_t window,
               uint32_t *err_flags, void *stream);

/* Frequency scalings of pkv_rope_inv_freq. */
enum {
    PKV_ROPE_PLAIN = 0,   /* theta^(-2 i / rot_dim) */
    PKV_ROPE_LINEAR = 1,  /* positions divided by factor */
    PKV_ROPE_NTK = 2,     /* theta * factor^(rot_dim / (rot_dim - 2)) in place of theta */
    PKV_ROPE_YARN = 3     /* YaRN: fast pairs kept, slow ones divided by factor, a linear ramp between */
};

/*
 * Rotary frequencies (radians a position) of rot_dim / 2 column pairs, in
 * inv_freq[rot_dim / 2], and the factor on the sines and cosines that goes with them
 * in *mscale (1, or 0.1 ln(factor) + 1 with YaRN).  factor >= 1;
 * trained_len (the context the model was trained on), beta_fast > beta_slow >
 * 0 (turns in that context above which a pair is kept and below which it is
 * stretched; 32 and 1 are usual) are read with YaRN only.  Host only.
 */
int pkv_rope_inv_freq(int32_t rot_dim, double theta, int32_t scaling, double factor, double trained_len,
                      double beta_fast, double beta_slow, double *inv_freq, double *mscale);

/*
 * turns[i] = inv_freq[i] / (2 pi) as a fraction of a turn, in units of 2^-64:
 * the form the kernels read (position * turns, modulo 2^64, is the angle at
 * any position).  Host only; the caller copies the array to the device.
 */
int pkv_rope_turns(const double *inv_freq, int32_t n, uint64_t *turns);

/*
 * What is done to a q or k head: y = x * rsqrt(mean(x^2) + eps) * weight
 * where there is a weight, then the first rot_dim columns are rotated by
 * angle a_i = position * frequency i:
 *   (u, w) -> mscale * (u cos a_i - w sin a_i, w cos a_i + u sin a_i)
 * for column pairs (i, i + rot_dim / 2), or (2 i, 2 i + 1) with interleaved.
 * All in fp32, rounded once at the end.  Host struct, device pointers.
 *
 * num_axes > 1: a row has a position on each of several axes (time, height
 * and width of images and video; at most PKV_ROPE_AXES), positions is
 * [total_rows][num_axes], and pair i is turned by the position on axis[i]
 * (axis: device, values below num_axes; a larger one counts as the last axis).
 * A row without positions, in norm + append, has its cache position on all of them.
 * num_axes 0 or 1 with axis NULL: one axis.
 */
#define PKV_ROPE_AXES 8
typedef struct pkv_rope {
    const uint64_t *turns;      /* device [rot_dim / 2], from pkv_rope_turns; unread if rot_dim is 0 */
    int32_t rot_dim;            /* even, 0 (no rotation) .. head_dim */
    int32_t interleaved;        /* 0 or 1 */
    float mscale;               /* on the rotated columns */
    float eps;
    const void *q_weight;       /* device [head_dim] of the rows' type (16-byte aligned), or NULL: q is not normalised */
    const void *k_weight;       /* the same for k */
    const uint8_t *axis;        /* device [rot_dim / 2], or NULL: one axis */
    int32_t num_axes;           /* positions of a row; 0 counts as 1 */
    int32_t reserved0;
} pkv_rope;

/*
 * This step's rows.  Strides are in elements from one row to the next (at
 * least heads * head_dim, a multiple of 16 bytes), heads of a row are
 * contiguous; q, k and v may be slices of one projection output.  Pointers are
 * 16-byte aligned device memory.  An output may be its own input (same
 * pointer and stride); no other overlap.
 */
typedef struct pkv_rows {
    const void *q, *k, *v;
    void *q_out, *k_out, *v_out;
    int64_t q_stride, k_stride, v_stride;
    int64_t q_out_stride, k_out_stride, v_out_stride;
    int32_t q_heads;
    int32_t total_rows;
    const int32_t *positions;   /* device [total_rows][num_axes], the angles' positions, or NULL */
} pkv_rows;

/*
 * Norm and rotation of rows that go to no cache: q to q_out and k to k_out
 * (either pair may be NULL with q_heads or kv_heads 0), rows of dtype
 * PKV_BF16 or PKV_F32.  v and v_out must be NULL; positions may be NULL only
 * with rot_dim 0.  head_dim: a multiple of 8, at most 256.
 */
int pkv_norm_rope(const pkv_rope *rope, int32_t dtype, int32_t head_dim, int32_t kv_heads,
                  const pkv_rows *rows, void *stream);

/*
 * Norm, rotation and append in one pass: for each row of a segment, q goes to
 * q_out (q NULL with q_heads 0: no queries), k after norm and rotation and v
 * as it is go to the row's cache slot, as pkv_append places and checks them.
 * rope NULL: rows as they are.  The angles' positions are positions[row], or the
 * row's position in the cache (kv_end - q_len + i).  k_out and v_out
 * (optional) get the rows as the cache now holds them; with a PKV_FP4 cache
 * those are the quantised values (k is rounded to bf16 before it is
 * quantised), with PKV_FP8 under the scale that the whole call leaves.  Rows are of
 * the cache's dtype (PKV_FP4, PKV_FP8: bf16).
 *
 * On a bf16 or fp32 cache a row belongs to one segment at most (in two it is
 * unspecified which of them places it).  On a PKV_FP4 cache it goes to its slot
 * in every segment that holds it, turned by positions[row] or by its position
 * in the lowest of them (v_out must not be v then).  On a PKV_FP8 cache it goes to
 * all of them too; its queries are turned once, by positions[row] or by its position in one of them, in place
 * or not, but its k_out and v_out are unspecified (and must not be k and v).  Rows no segment covers, and
 * rows of segments that pkv_append would refuse (the same PKV_ERR_* bits), are
 * not written, in none of the outputs.  A later attention call may be launched
 * with PKV_FLAG_PDL behind this one, unless one segment's rows are older keys
 * of another (two pieces of one sequence in a call).
 */
int pkv_norm_rope_append(const pkv_cache *cache, int32_t layer, const pkv_rope *rope, const pkv_rows *rows,
                         const int32_t *seq_info, int32_t num_segments, int32_t window,
                         uint32_t *err_flags, void *stream);

/*
 * Decode attention over the paged cache ([ExecuTorch #24072]
 * triton::sdpa_varlen semantics over the paged layout of
 * [vllm-omni paged_decode.py]).
 *
 * q: device [total_rows][num_q_heads][head_dim] of the cache dtype; q head h
 * reads kv head h / (num_q_heads / kv_heads) (grouped-query attention; the
 * ratio must be a whole number).  For segment (q_start, q_len, col, kv_end),
 * row q_start + i sits at position p = kv_end - q_len + i and sees keys
 *   causal:     [lo, p + 1),        lo = max(0, p - window + 1) if window > 0 else 0
 *   non-causal: [lo, kv_end),       lo = max(0, kv_end - window) if window > 0 else 0
 * (bottom-right causal alignment, [tiny-llm kv_cache.py] causal_kwargs; for
 * q_len = 1 both are the same).  With cache->first_valid set and
 * f = max(first_valid[col], 0): a row with p < f sees key p alone, any other
 * row has lo raised to at least f.  out[row][h][:] = softmax(softmax_scale *
 * q.k) weighted sum of V, in fp32; lse[row][h] = natural-log sum of
 * exp(softmax_scale * q.k) (may be NULL).  Rows no segment covers, and rows of
 * invalid segments, get out = 0 and lse = -inf.  Keys at or past kv_end and
 * table entries past the keys a segment needs are never read, so they may
 * hold anything (NaN included).
 *
 * max_q_len bounds every segment's q_len and max_kv bounds every segment's
 * kv_end; both only size the launch, so a graph captured once serves every
 * length up to them.  num_splits (0..16) is the number of CTAs that share one
 * (segment, kv head) key range as a thread-block cluster; their partial
 * softmax results are merged by log-sum-exp through distributed shared
 * memory in the same launch, so no workspace is needed (workspace NULL,
 * workspace_bytes 0; see pkv_attend_workspace_bytes for the other mode).  0 picks the count
 * from the launch shape: a power of two aiming at about three waves of
 * resident CTAs (one wave for the tcgen05 tile of wide bf16 groups), the
 * largest cluster the device can co-schedule below it, and, for kernels
 * that fit once per SM with few (segment, kv head) ranges, the cluster size
 * that needs the fewest waves of clusters resident at once.  The tcgen05
 * tile also runs a range of at most 24 groups of 64 keys on one CTA of its
 * cluster, and with up to 64 segments takes the ranges longest first; the
 * results do not depend on either.  A larger count than the segment has
 * 16-token pages leaves CTAs idle.
 *
 * flags: PKV_FLAG_SIMT selects the CUDA-core kernels for bf16 (fp32 always
 * uses them): at most 8 query rows per kv head take the decode kernel's
 * variant with fp32 FMA products, wider groups the general CUDA-core tile.
 * PKV_FLAG_MMA_SYNC keeps wide bf16 groups at head_dim 128 (more than 8
 * rows per kv head) on the mma.sync tile instead of the tcgen05 one.  PKV_FLAG_PDL launches with programmatic dependent launch: the
 * kernel may start reading cache slots of positions below kv_end - q_len,
 * the block table and seq_info while the previous kernel on the stream is
 * still running, so set it only when that previous kernel writes none of
 * those; q, k_new, v_new, out, lse and err_flags are touched only after it
 * has finished.  PKV_FLAG_PREFETCH_NEXT (ignored for the last layer) also
 * brings into L2 the pages of layer + 1 that cover the same key ranges, for
 * a caller whose next call attends layer + 1 with the same block table and
 * segments (one decode step): a hint only, it changes no result.  The
 * prefetch is capped at about 48 MB per call.
 *
 * On a PKV_FP4 or PKV_FP8 cache q is bf16 and out is fp32, or bf16 with
 * PKV_FLAG_OUT_BF16.  Scores are those of the stored values to fp32; the
 * softmax weights are rounded to fp16 for the product with V (each by at most
 * 2^-11 of itself or 2^-32 of its row's largest, whichever is more; with PKV_FP8
 * that is said of a weight times its page's V scale, and sums of such
 * products above 2^100 may overflow).  Weights below 2^-126 of the row's largest may count as zero.  A NaN in V
 * reaches only the rows that see its key.  Without a workspace the splits form
 * a cluster (num_splits 0..16); large launches are faster with one (see
 * pkv_attend_workspace_bytes).  PKV_FLAG_SIMT, PKV_FLAG_MMA_SYNC and
 * PKV_FLAG_PREFETCH_NEXT have no effect.  PKV_FLAG_PDL: pages wholly below
 * position kv_end - q_len may be read before the previous kernel has
 * finished, so it may be the append of this step, unless two segments are
 * pieces of one sequence.  (Most attention launches over quantised caches, and
 * pkv_norm_rope and pkv_norm_rope_append, are programmatic
 * dependent launches without the flag too, which wait for the previous
 * kernel first thing.)
 *
 * Device pointers must be 16-byte aligned (out and lse: 4-byte; with a
 * quantised cache out: 16-byte).
 */
int pkv_attend_varlen(const pkv_cache *cache, int32_t layer,
                      const void *q, int32_t num_q_heads, int32_t total_rows,
                      const int32_t *seq_info, int32_t num_segments,
                      int32_t max_q_len, int64_t max_kv, int32_t num_splits,
                      float softmax_scale, int32_t causal, int32_t window,
                      float *out, float *lse,
                      void *workspace, int64_t workspace_bytes,
                      uint32_t *err_flags, uint32_t flags, void *stream);

/*
 * Attention of whole prompts over their own rows, which are packed one after the
 * other: rows->q [total_rows][q_heads][head_dim], rows->k and rows->v
 * [total_rows][kv_heads][head_dim], bf16, rows apart as their strides say (slices of
 * one projection output); the other pointers of rows are NULL.  No cache is read or
 * written: the step's append (of the same rows and table) and this call may come in either order.
 *
 * seq_info as for pkv_append.  A segment's rows are its sequence from the first
 * position on, so kv_end has to be q_len (else PKV_ERR_SEGMENT: keys before the rows
 * would be in a cache, which pkv_attend_varlen reads); col is not looked at.
 * max_len bounds every segment's q_len (PKV_ERR_QLEN) and sizes the launch.  Which
 * keys a row sees, out, lse, uncovered rows, refused segments and overlaps
 * (PKV_ERR_OVERLAP) are as in pkv_attend_varlen, without padding.  softmax_scale is
 * positive and finite (times log2 e, too); head_dim a multiple of 8, at most 256; q_heads / kv_heads at most 128.  PKV_EINVAL also
 * where num_segments prompts of min(max_len, total_rows) rows would be more than 2^31 tiles.
 *
 * Scores are fp32 sums of exact products; softmax weights are rounded to bf16 (each
 * by at most 2^-8 of itself) for the product with V, whose sums are fp32, and not for the sum that divides it: a
 * row that one key dominates comes out as that key's V times 1 - 2^-8 to 1 + 2^-8 at worst.  A NaN or
 * infinity in k or v reaches the rows that see its key and no others (a
 * call that meets one takes longer).  out: fp32, or bf16 with PKV_FLAG_OUT_BF16, 16-byte
 * aligned, [total_rows][q_heads][head_dim], apart from q, k and v.  The launch is a programmatic dependent one,
 * which waits for the kernel before it first thing; PKV_FLAG_PDL has no effect.
 */
int pkv_attend_prompt(int32_t head_dim, int32_t kv_heads, const pkv_rows *rows,
                      const int32_t *seq_info, int32_t num_segments, int32_t max_len,
                      float softmax_scale, int32_t causal, int32_t window,
                      void *out, float *lse, uint32_t *err_flags, uint32_t flags, void *stream);

/*
 * pkv_append followed by pkv_attend_varlen in one launch: the rows of this
 * step are written into the cache and attended to from k_new / v_new
 * directly.  Same arguments and results as the two calls in sequence, with
 * one extra condition: no two segments of the call may name the same `col`
 * (the two-call sequence has no such limit).  On a quantised cache it is the two
 * calls, one launch each.
 */
int pkv_append_attend(const pkv_cache *cache, int32_t layer,
                      const void *q, const void *k_new, const void *v_new,
                      int32_t num_q_heads, int32_t total_rows,
                      const int32_t *seq_info, int32_t num_segments,
                      int32_t max_q_len, int64_t max_kv, int32_t num_splits,
                      float softmax_scale, int32_t causal, int32_t window,
                      float *out, float *lse,
                      void *workspace, int64_t workspace_bytes,
                      uint32_t *err_flags, uint32_t flags, void *stream);

/*
 * Bytes of workspace the two calls above need for these launch bounds when
 * given one (0: the launch never uses it).  With a workspace, the decode
 * kernel (at most 8 query rows per segment and kv head: G * max_q_len <= 8,
 * bf16, tensor-core path) splits a key range over independent CTAs (up to 64
 * per range, num_splits 0..64) that merge through it: each writes its
 * partial rows, and the last to finish (counted with an atomic it resets)
 * merges them.  Without one (NULL), the splits form a thread-block cluster
 * and merge through distributed shared memory (num_splits 0..16).  The
 * workspace is device memory the caller owns, 16-byte aligned, zero-filled
 * before its first use and not touched by the caller between calls: its
 * first bytes are per-range arrival counters that every call leaves at zero,
 * the rest is scratch.  Used with larger launch bounds (more segments or kv
 * heads) than before, it must be zero-filled again.  Calls that may run
 * concurrently need their own.  A workspace smaller than this size is rejected with
 * PKV_EINVAL.  Returns a negative pkv_status for invalid bounds.
 *
 * With a quantised cache: launches with num_splits 0, at most 512 segments and
 * at most 16 row tiles a kv head, whose bounds make it worth while (at 8 query rows per kv
 * head and head_dim 128, from about half a million (key, kv head) pairs for one
 * sequence and twice that for several; with more rows from fewer).
 * Given a workspace, they run as one wave of CTAs with equal shares of all
 * key ranges and a second launch that merges the shared ones, instead of as a
 * cluster per range; more than 32 rows per kv head at head_dim 128 then take
 * the tcgen05 tile.  The size does not grow with the lengths and is below 25 MB.
 * It need not be zeroed, and may be shared by calls that
 * follow one another on one stream.  A call with a window counts
 * min(max_kv, window + max_q_len) keys in place of max_kv: it uses a workspace where
 * the query for that many keys asks for one, of the same size, and takes any where the
 * query for max_kv asks for none.
 */
int64_t pkv_attend_workspace_bytes(const pkv_cache *cache, int32_t num_q_heads,
                                   int32_t num_segments, int32_t max_q_len,
                                   int64_t max_kv, int32_t num_splits, uint32_t flags);

/*
 * pkv_append_attend with the split-merge workspace taken from a fixed 8 MiB
 * scratch array in the library's device memory instead of the caller: no
 * allocation, no workspace argument.  The pages have no counterpart of this
 * call.  It serves callers that may not allocate device memory at the point
 * of the call: an allocator-free runtime, a custom-op shim that owns no
 * memory pool, or code running while an allocator must not be touched.  The
 * scratch is a file-scope __device__ array (every device that loads the
 * library holds it until the process exits), zero at load; the arrival
 * counters live in an array of their own that every call leaves at zero.
 * Its device address is looked up with cudaGetSymbolAddress on every call
 * (a host-side query, so a new context after cudaDeviceReset is picked up);
 * the first call on a device also loads the library's module there, so make
 * it before any stream capture.  A launch whose merge would need more than
 * 8 MiB (see pkv_attend_workspace_bytes) or more than 4096 (segment, kv
 * head, row tile) ranges is rejected with PKV_ECAPACITY before anything
 * runs; a failed lookup returns PKV_ECUDA.  The scratch is shared by every
 * call on a device and keeps the last call's partials, so calls that overlap
 * on the GPU race: issue them on one stream, or serialise them.  Otherwise
 * the same arguments, results and errors as pkv_append_attend.
 */
int pkv_append_attend_noalloc(const pkv_cache *cache, int32_t layer,
                              const void *q, const void *k_new, const void *v_new,
                              int32_t num_q_heads, int32_t total_rows,
                              const int32_t *seq_info, int32_t num_segments,
                              int32_t max_q_len, int64_t max_kv, int32_t num_splits,
                              float softmax_scale, int32_t causal, int32_t window,
                              float *out, float *lse,
                              uint32_t *err_flags, uint32_t flags, void *stream);

/*
 * Build a segment table from the flash-attention argument form
 * ([vllm-omni paged_decode.py] PagedDecodeCache.attend passes cu_seqlens_q
 * and seqused_k): seq_info[s] = (cu_seqlens_q[s], cu_seqlens_q[s+1] -
 * cu_seqlens_q[s], s, seqused_k[s]) for s < num_seqs.  All device int32.
 */
int pkv_seqinfo_from_seqused(const int32_t *cu_seqlens_q, const int32_t *seqused_k,
                             int32_t num_seqs, int32_t *seq_info_out, void *stream);

/*
 * seq_clone of the batched-sequence cache ([ExecuTorch #24073]
 * CudaBatchedSequenceCache: a device copy of the source prefix), over the
 * paged layout: in every layer, positions 0 .. n-1 of the sequence in
 * block-table row src_col are copied bit for bit (all kv heads) to the same
 * positions of row dst_col, each side mapped through its own table row.
 * With ring storage only the last min(n, ring_rows) positions exist and are
 * copied (slot position % ring_rows on both sides).  Typical use: admit a
 * request that shares a prefix, then set its segment's kv_end to n.
 * All or nothing per layer: if any page either side needs is outside
 * [0, num_blocks), that layer is not written and PKV_ERR_BLOCK is set.  The
 * two rows' pages must not overlap (other than being identical).  Host
 * errors: a column outside [0, max_seqs), n < 0, or (flat layout) n beyond
 * the table's capacity (PKV_ECAPACITY).  Launches one kernel per layer.
 */
int pkv_seq_clone(const pkv_cache *cache, int32_t src_col, int32_t dst_col, int64_t n,
                  uint32_t *err_flags, void *stream);

/*
 * rewind of the batched-sequence cache ([ExecuTorch #24073], bounded by the
 * ring floor), on the device: kv_end -= amount[s] for every segment s
 * (amount: device int32[num_segments]), e.g. the draft tokens a verify step
 * rejected; their slots are simply rewritten by the next append.  On a PKV_FP8
 * cache that does not undo the append of the rejected rows: where tokens before them are in
 * their page, those have been rounded to the scale that the rejected rows needed too (by at most 2^-10 of it; under
 * that of an infinity, 2^119, ordinary values are zero), and a page of a flat cache keeps that scale while it has tokens
 * before the new rows.  In a ring the tokens that the window had passed may be saturated (see PKV_FP8).  A segment
 * keeps its kv_end and sets PKV_ERR_SEGMENT when amount < 0 or
 * amount > kv_end, and PKV_ERR_RING when the cache is a ring of R rows and
 * amount > R - window + 1 (the next step's window would need positions the
 * ring no longer holds; window must be > 0 with rings).  The block table is
 * untouched: removing a sequence (seq_rm) is the caller releasing its table
 * row's pages, which needs no device work.
 */
int pkv_rewind(const pkv_cache *cache, int32_t *seq_info, int32_t num_segments,
               const int32_t *amount, int32_t window, uint32_t *err_flags, void *stream);

/*
 * Advance every segment to the next step on the device: kv_end += q_len
 * ([tiny-llm kv_cache.py] SlotKVCache.end_step does the same for slot
 * lengths inside a captured graph, so a replay needs no host write).
 */
int pkv_advance(int32_t *seq_info, int32_t num_segments, void *stream);

/*
 * Move a cache to a larger bucket, keeping the first old_len tokens
 * ([vllm-omni paged_decode.py] PagedDecodeCache.grow).  new_cache describes
 * buffers the caller has already allocated for the new bucket (same layers,
 * kv_heads, head_dim, dtype, ring_rows = 0, identity-ordered tables); the
 * first old_len flat rows of every layer's K and V are copied from old to
 * new.  Only after every copy has been enqueued is new_cache->generation set
 * to old_cache->generation + 1, so a failure leaves both descriptors as they
 * were and a graph keyed on the old generation is never paired with half-built
 * buffers.  Returns PKV_SAME_BUCKET, copying nothing, when
 * new_cache->bucket == old_cache->bucket; PKV_ESTALE when the shapes differ;
 * PKV_ECAPACITY when old_len exceeds either cache's rows.
 */
int pkv_resize_bucket(const pkv_cache *old_cache, pkv_cache *new_cache,
                      int64_t old_len, void *stream);

/*
 * Copy a prefill cache into the paged buffers ([vllm-omni paged_decode.py]
 * PagedDecodeCache.load_prefix): for every layer l, token s < n and kv head
 * h, keys[l] + s*stride_s + h*stride_h (elements; head_dim contiguous) goes
 * to flat row s of layer l's K pool, and likewise values.  keys / values are
 * host arrays of num_layers device pointers, so a [B, H, S, D] tensor's
 * batch-0 view is passed with stride_s = D, stride_h = S*D.  Rows past n are
 * left as they were.  Returns PKV_EMPTY (and copies nothing) when n == 0 or
 * keys is NULL.
 */
int pkv_load_prefix(const pkv_cache *cache, const void *const *keys,
                    const void *const *values, int64_t n,
                    int64_t stride_s, int64_t stride_h, void *stream);

/*
 * Write-back for a stage that reads an ordinary cache
 * ([vllm-omni paged_decode.py] PagedDecodeCache.to_dynamic_cache): copy the
 * first n flat rows of layer `layer` into keys_out / values_out laid out
 * [kv_heads][n][head_dim] (device, contiguous).  Of a PKV_FP8 cache the rows are
 * bf16, the stored values (exact).
 */
int pkv_to_contiguous(const pkv_cache *cache, int32_t layer, int64_t n,
                      void *keys_out, void *values_out, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
