/*
 * gqa_kv8.h -- C ABI of the 8-bit key/value cache of the same GB300 (sm_103a) library: the
 * cache write (quantising), its read back, grouped-query attention over it for prompts and
 * for single tokens, and the rotary positions that come before it.  Beside gqa_decode.h
 * (one token per sequence over a contiguous bf16 cache), this cache holds one byte per
 * number, so that decode, which is bound by the cache's bytes, reads half as much; it is
 * paged, and a call takes any number of new tokens per sequence.
 *
 * The cache.  Pages of page_size positions; for each of keys and values
 *   codes   uint8 [n_pages][n_kv_heads][page_size][head_size]   e4m3 bytes or int8
 *   scales  fp32  [n_pages][n_kv_heads][page_size / 16]
 * value = code * scale.  Position i of sequence b lives in page page_table[b][i / page_size]
 * at i % page_size.  Every 16 positions of a head (a block) share a scale, and every scale
 * is a power of two between 2^-100 and 2^122: the smallest one under which the block's
 * largest magnitude fits the largest finite code (448 for e4m3, 127 for int8).  A power of
 * two costs e4m3 nothing (its relative step does not depend on the scale) and int8 at most
 * one of its 8 bits; in return the codes do not depend on how a division rounds, and a scale
 * can grow under codes already written: dividing those by a power of two is exact for e4m3
 * numbers that stay normal, and one rounding for the others and for int8.
 *
 * The batch.  Every cache call takes the same description of its sequences: sequence b has
 * lens[b] cached positions, the last offsets[b+1] - offsets[b] of which are the call's
 * tokens (rows offsets[b] .. of q, k, v and the outputs; rows at or past offsets[n_seqs]
 * are neither read nor written).  One decode step is: gqa_rope, gqa_kv8_append,
 * gqa_kv8_attention, with lens already counting the new tokens.  All arrays are in device
 * memory and read when the kernels run, so a captured graph follows their contents.
 *
 * Conventions as in moe_layer.h: device pointers owned by the caller, status codes, no host
 * synchronisation, no allocation inside the library, calls asynchronous on `stream` of the
 * current device.  What only the device can see (a page outside the cache, a length past the
 * page table, offsets out of order, values that are not finite) never faults: the kernels
 * leave out what it concerns and record it in the cache's error word.  Every call leaves
 * out the tokens that a length places past the end of the page table, and a sequence whose
 * offsets are out of order or past the rows; no other position or row stands for them.
 */
#ifndef GQA_KV8_H
#define GQA_KV8_H

#include <stddef.h>
#include <stdint.h>

#include "moe_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { GQA_KV8_E4M3 = 0, GQA_KV8_INT8 = 1 };

typedef struct {
    void* k_codes;              /* uint8 [n_pages][n_kv_heads][page_size][head_size], 16-byte aligned */
    void* v_codes;
    float* k_scales;            /* fp32 [n_pages][n_kv_heads][page_size / 16] */
    float* v_scales;
    uint32_t* error;            /* one device word, zero before the first call */
    int n_pages;                /* n_pages * n_kv_heads * page_size < 2^31 */
    int page_size;              /* a power of two, 16 .. 1024 */
    int n_kv_heads;             /* 1 .. 64 */
    int head_size;              /* 64 or 128 */
    int format;                 /* GQA_KV8_E4M3 or GQA_KV8_INT8 */
} gqa_kv8_cache_t;

typedef struct {
    const int32_t* page_table;  /* [n_seqs][max_pages]; entries past a sequence's length are not read */
    const int32_t* lens;        /* [n_seqs] cached positions, the call's tokens among them */
    const int32_t* offsets;     /* [n_seqs + 1] non-decreasing, offsets[n_seqs] <= n_tokens */
    int n_seqs;                 /* 1 .. 1024 */
    int max_pages;              /* max_pages * page_size <= 2^24 */
    int n_tokens;               /* rows of the call's token tensors, 0 .. 2^20 */
    int max_new;                /* no sequence has more new tokens than this, 1 .. 2^20 */
} gqa_kv8_batch_t;

/* Quantise the call's keys and values and write them into the cache.
 *   k, v     bf16 [n_tokens][n_kv_heads][head_size], 16-byte aligned, row t at
 *            t * k_stride (v_stride) elements, a multiple of 8, at least n_kv_heads *
 *            head_size (k and v may be slices of one projection's output)
 * A block that already holds positions before the new ones keeps its scale if the new rows
 * fit it; otherwise it takes theirs and its codes are rounded again.  An infinity is stored
 * as the largest finite code of its sign and a NaN as zero, neither counts for the scale,
 * and both set MOE_ERR_NONFINITE in the error word: the cache holds finite numbers only.
 * Codes of positions outside the call's tokens and the blocks' earlier positions stay as
 * they are.  The pages that a call writes must belong to one sequence each.
 * Errors: INVALID_ARG, ALIGNMENT, CUDA. */
moe_status_t gqa_kv8_append(const gqa_kv8_cache_t* cache, const gqa_kv8_batch_t* batch, const void* k,
                            long long k_stride, const void* v, long long v_stride, moe_stream_t stream);

/* Read back the rows of the batch's tokens (all of a sequence's positions when its offsets
 * differ by its length): k_out, v_out bf16 [n_tokens][n_kv_heads][head_size], 16-byte
 * aligned; code * scale is exact in bf16 (a magnitude of 2^128, which e4m3 has next to
 * bf16's largest numbers, comes back as the largest).  Errors: INVALID_ARG, ALIGNMENT, CUDA. */
moe_status_t gqa_kv8_gather(const gqa_kv8_cache_t* cache, const gqa_kv8_batch_t* batch, void* k_out, void* v_out,
                            moe_stream_t stream);

/* Bytes of device workspace a gqa_kv8_attention call needs on this cache with n_q_heads
 * query heads and at most max_new new tokens per sequence (0 if those are refused); it does
 * not depend on the number of sequences or their lengths.  Zero-fill it before its first
 * use; every call leaves it ready for the next, of any shape that needs no more bytes. */
size_t gqa_kv8_workspace_bytes(const gqa_kv8_cache_t* cache, int n_q_heads, int max_new);

/* Causal grouped-query attention of the call's tokens over the cache.  Token j of sequence
 * b stands at position p = lens[b] - (offsets[b+1] - offsets[b]) + j and sees positions
 * 0 .. p, its own among them; query head h reads key/value head h / (n_q_heads /
 * n_kv_heads):
 *   o = sum_i softmax_i(scale * q . k_i) v_i
 *   q        bf16 [n_tokens][n_q_heads][head_size], 16-byte aligned, row t at t * q_stride
 *            elements (a multiple of 8, at least n_q_heads * head_size)
 *   out      bf16 [n_tokens][n_q_heads][head_size], 16-byte aligned, no overlap with q
 *   scale    multiplies the scores; 0 means 1 / sqrt(head_size)
 *   workspace  256-byte aligned; two calls that overlap in time need two
 * The products are exact, sums, maxima and the softmax are fp32, its weights are rounded to
 * fp16 for the value product only, and o is rounded once.  A weight counts there with its
 * value's scale.  It is off by at most 2^-11 of itself, and the 32 (in prompts 128) positions
 * that are multiplied together by 2^-11 of the largest of them in all; how small they are
 * beside the row's other positions does not matter down to 2^-40 of the largest, under which
 * they may be lost.  The normaliser counts every weight in full, whatever the scale of its
 * value.  Scores may have any size; one that is past fp32's range (in units of log2) counts
 * as its largest number.  Exactness ends where scales lie very far apart: among 128
 * consecutive positions a block whose scale is under 2^-21 of the largest loses low bits of
 * its codes.  A token that sees no position (its sequence has fewer positions than new
 * tokens, which is recorded as a bad length) gets zeros; a query that is not finite makes
 * its own row NaN and no other.
 * Between 1 and 16 query heads per key/value head.  Results do not depend on timing: the
 * same call gives the same bits.  max_new decides the kernel (one for at most 32 query rows
 * per key/value head, one for more), so a bound that is far too large is right but slow.
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED (heads), CUDA. */
moe_status_t gqa_kv8_attention(const gqa_kv8_cache_t* cache, const gqa_kv8_batch_t* batch, const void* q,
                               long long q_stride, int n_q_heads, float scale, void* out, void* workspace,
                               size_t workspace_bytes, moe_stream_t stream);

/* Synchronise the current device, then read and clear the cache's error word: MOE_OK,
 * MOE_ERR_DEVICE_BOUNDS (a page, length or offset out of range), MOE_ERR_NONFINITE or
 * MOE_ERR_TIMEOUT (a bounded wait gave up). */
moe_status_t gqa_kv8_get_error(const gqa_kv8_cache_t* cache);

/* Rotary positions with one or several axes (time, height, width of images and video).
 * Pair j of a head, elements j and j + rotary / 2, turns by the angle
 * pos[axis(j)][t] * inv_freq[j]; elements from `rotary` on pass through.  The angle is
 * kept as a 64-bit fraction of a turn, so that far positions lose nothing. */
#define GQA_ROPE_MAX_PAIRS 64
#define GQA_ROPE_MAX_AXES 4
typedef struct {
    uint64_t turn[GQA_ROPE_MAX_PAIRS];   /* inv_freq / 2 pi, in units of 2^-64 of a turn, modulo one turn */
    uint8_t axis[GQA_ROPE_MAX_PAIRS];
    int head_size, rotary, n_axes;
} gqa_rope_plan_t;

/* Fill a plan (host memory, no GPU needed).  head_size 64 or 128; rotary a multiple of 16,
 * 16 .. head_size; sections[n_axes] (1 .. 4 axes) are the pairs of each axis and sum to
 * rotary / 2 (NULL: one axis has them all); cyclic 0 gives the axes runs of pairs in
 * order, 1 deals the pairs out in turn to the axes that still lack some.
 * inv_freq: rotary / 2 finite values, or NULL for theta^(-2j / rotary), theta > 0.
 * Errors: INVALID_ARG, UNSUPPORTED. */
moe_status_t gqa_rope_plan_init(gqa_rope_plan_t* plan, int head_size, int rotary, double theta,
                                const double* inv_freq, const int* sections, int n_axes, int cyclic);

/* Rotate the heads of q and k (k may be NULL with n_k_heads 0):
 *   q, k     bf16 [T][heads][head_size], 16-byte aligned, row t at t * stride elements (a
 *            multiple of 8, at least heads * head_size)
 *   pos      int32 [n_axes][T] (device), any sign
 *   q_out, k_out  as q and k with strides of their own; in place (the same pointer and
 *            stride) is allowed, any other overlap is not
 * fp32 arithmetic, one rounding.  T 0 .. 2^20, 1 .. 256 heads each.
 * Errors: INVALID_ARG, ALIGNMENT, CUDA. */
moe_status_t gqa_rope(const gqa_rope_plan_t* plan, const void* q, long long q_stride, int n_q_heads, const void* k,
                      long long k_stride, int n_k_heads, const int32_t* pos, int T, void* q_out,
                      long long q_out_stride, void* k_out, long long k_out_stride, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_KV8_H */
