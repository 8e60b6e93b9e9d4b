/*
 * decode.h -- C ABI of libw4a4's single-token operators (sm_100a): what a
 * model whose linears hold 4-bit weights needs to answer one token at a time.
 *
 *   w4a4_group_*   4-bit weights with one step per group of inputs, and their
 *                  product with a few tokens (no activation quantization: a
 *                  single token's product reads every weight once and is bound
 *                  by that traffic, so 16-bit activations cost nothing)
 *   w4a4_rope_table, w4a4_kv_append
 *                  the rotation table, and new keys and values written into a
 *                  paged cache with the rotation applied on the way
 *   w4a4_kv_attend one new token per sequence against its cached keys and
 *                  values
 *
 * The quantizer is [PTQ] of w4a4.h with N = 4 and one step per group ([GRAN]
 * read at a finer grain); the pages describe neither the cache nor the
 * attention, which are those of any decoder with rotary positions.
 *
 * Conventions are those of w4a4.h: device pointers owned by the caller, 16-byte
 * aligned (arrays of int32 and lse: 4-byte; W4A4_ERR_ALIGN otherwise), argument
 * checks on the host before anything is enqueued, calls that enqueue on `stream` and return,
 * 16-bit data passed as raw patterns: bf16, or IEEE half with W4A4_FLAG_FP16.
 * The current device must be the one that holds the arrays.  Every call may be
 * captured into a CUDA graph.  Sizes named T, M, n_seqs may be 0 (a no-op).
 *
 * Positions, lengths, sequence and page numbers are read on the device.  One
 * that is out of range never leads to an access out of bounds: the token or
 * cache row it names is left out and W4A4_DEV_RANGE is set in the device status
 * word (w4a4_get_device_status).
 */
#ifndef DECODE_H_
#define DECODE_H_

#include <stddef.h>
#include <stdint.h>

#include "w4a4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 16-bit data are IEEE half values instead of bf16 (a flag of the structs
 * below, fixed when they are made). */
#define W4A4_FLAG_FP16 0x200u

/* ------------------------------------------- 4-bit weights with group steps */

/* Weights W [N, K] as codes c in [-8, 7] and steps s, one per group of `group`
 * consecutive inputs of a row: W[n, k] ~ c[n, k] * s[n, k / group], in the order
 * the kernels read (w4a4_group_pack and w4a4_group_quantize write it): rows in
 * tiles of 16 and inputs in blocks of 128, both padded with zeros, one record of
 * 1024 + 4096 / group bytes after another, the blocks of a tile in a row.  In a record, the
 * codes of rows r and r + 8 (r = 0..7) form two runs of 512 bytes; 16 bytes at 64 r
 * + 16 c of a run (c = 0..3) hold four words, word j the 8 codes of inputs 32 j +
 * 8 c + 0..7 of the block, inputs 0, 2, 4, 6, 1, 3, 5, 7 from the lowest nibble up.
 * Then follow, for r = 0..7, the 16-bit steps of rows r and r + 8 for each group. */
typedef struct {
    int32_t N;         /* rows, 1 .. 16777216 */
    int32_t K;         /* inputs, a positive multiple of group, <= 1048576 */
    int32_t group;     /* 32, 64 or 128 */
    uint32_t flags;    /* 0 or W4A4_FLAG_FP16: type of steps, weights and tokens */
    uint8_t *data;
} w4a4_group_weights_t;

/* Bytes of the records; 0 for an N, K or group that is not accepted.  About
 * N K / 2 + 2 N K / group. */
size_t w4a4_group_weights_bytes(int32_t N, int32_t K, int32_t group);

/* Points *out at `base` (16-byte aligned, at least
 * w4a4_group_weights_bytes(N, K, group) bytes, owned by the caller) and fills in
 * the sizes.  flags: 0 or W4A4_FLAG_FP16.  Touches no device memory.
 * W4A4_ERR_UNSUPPORTED for another group or flag, W4A4_ERR_SHAPE for an N, K or
 * `bytes` that is not accepted. */
w4a4_status w4a4_group_bind(void *base, size_t bytes, int32_t N, int32_t K, int32_t group, uint32_t flags,
                            w4a4_group_weights_t *out);

/* The inputs of these three must not overlap the output (W4A4_ERR_ARG).
 *
 * [PTQ] per group: s = round16(max|W| / 7), c = clamp(round-half-even(W / s),
 * -8, 7); a group with s = 0 gets zero codes.  W [N, K] 16-bit, finite. */
w4a4_status w4a4_group_quantize(const uint16_t *W, const w4a4_group_weights_t *w, void *stream);

/* Codes and steps made elsewhere, in plain order: codes [N, K/2], two per byte
 * as in w4a4.h, scales [N, K/group] 16-bit. */
w4a4_status w4a4_group_pack(const uint8_t *codes, const uint16_t *scales, const w4a4_group_weights_t *w,
                            void *stream);

/* W [N, K] 16-bit = round16(c s). */
w4a4_status w4a4_group_dequantize(const w4a4_group_weights_t *w, uint16_t *W, void *stream);

/* Most tokens w4a4_group_gemv takes. */
#define W4A4_GEMV_MAX_TOKENS 16

/* Y [M, N] 16-bit = round16( sum_k X[m, k] c[n, k] s[n, k / group] + bias[n] )
 * for M <= W4A4_GEMV_MAX_TOKENS tokens (W4A4_ERR_SHAPE above) X [M, K]; bias [N]
 * 16-bit or NULL.  Products of codes and activations are exact, sums are fp32:
 * per group first, then times the step.  flags: 0, or W4A4_FLAG_GELU_OUT (bf16
 * only): Y = bf16(GELU(y)) of the rounded y, as in w4a4_linear_ex.  Y must not
 * overlap X, bias or the weights (W4A4_ERR_ARG). */
w4a4_status w4a4_group_gemv(const uint16_t *X, int64_t M, const w4a4_group_weights_t *w, const uint16_t *bias,
                            uint16_t *Y, uint32_t flags, void *stream);

/* ------------------------------------------------------------ the paged cache */

/* Keys and values in pages of page_size tokens.  The element d of head h of a
 * page's token t is at k[page * stride_page + t * stride_token + h * stride_head
 * + d], and the same in v (strides in elements, non-negative multiples of 8, so
 * either order of tokens and heads works).  flags: 0 or W4A4_FLAG_FP16. */
typedef struct {
    uint16_t *k, *v;
    int64_t n_pages;       /* 0 <= n_pages < 2^31 */
    int32_t page_size;     /* >= 1 */
    int32_t n_heads;       /* 1 .. 65535, as the numbers of query heads below */
    int32_t head_dim;      /* 64 or 128 */
    uint32_t flags;
    int64_t stride_page, stride_token, stride_head;
} w4a4_kv_cache_t;

/* w4a4_kv_append: neighbours (2i, 2i + 1) turn together instead of (i, i + rot_dim / 2). */
#define W4A4_FLAG_ROPE_PAIRS 0x400u

/* The usual rotation table, computed on the host in double precision: table
 * (HOST, [n_pos, rot_dim] fp32), row p holding cos(p f_i) then sin(p f_i), f_i =
 * base^(-2i / rot_dim), i < rot_dim / 2.  rot_dim: a positive multiple of 16 up to
 * 128 (W4A4_ERR_UNSUPPORTED otherwise).  Other schemes (two-dimensional positions, scaled
 * frequencies) are tables of the caller's own. */
w4a4_status w4a4_rope_table(int32_t n_pos, int32_t rot_dim, double base, float *table);

/* New tokens for w4a4_kv_append.  Strides are in elements. */
typedef struct {
    const uint16_t *k, *v;    /* [n_tokens, n_heads, head_dim], tokens k_stride / v_stride apart */
    const uint16_t *q;        /* [n_tokens, n_q_heads, head_dim], q_stride apart; or NULL */
    uint16_t *q_out;          /* [n_tokens, n_q_heads, head_dim], contiguous (with q) */
    int64_t k_stride, v_stride, q_stride;
    int64_t n_tokens;
    const int32_t *pages;     /* [n_seqs, max_pages] page numbers */
    const int32_t *seq;       /* [n_tokens] sequence of each token; NULL: token t is sequence t */
    const int32_t *pos;       /* [n_tokens] position of each token in its sequence */
    const int32_t *table_pos; /* [n_tokens] row of the table; NULL: pos */
    const float *table;       /* [n_table, rot_dim] cosines, then sines; NULL when rot_dim = 0 */
    int32_t n_seqs, max_pages, n_q_heads, n_table, rot_dim;
    uint32_t flags;           /* 0 or W4A4_FLAG_ROPE_PAIRS */
} w4a4_kv_append_t;

/* New tokens enter the cache: token t with keys k[t] and values v[t] becomes position pos[t]
 * of sequence seq[t], which lives in page pages[seq, pos / page_size] at row pos %
 * page_size.  Keys, and queries on their way from q to q_out (which may be q itself when
 * q_stride = n_q_heads * head_dim or for one token, and must not overlap it otherwise, nor any
 * other array that is read: W4A4_ERR_ARG), are rotated: with
 * (a, b) elements i and i + rot_dim / 2 (W4A4_FLAG_ROPE_PAIRS: 2i and 2i + 1) of a head and
 * (c, s) elements i and i + rot_dim / 2 of the token's row of the table, a' = a c - b s, b' =
 * b c + a s in fp32, rounded once; elements from rot_dim on, values, and everything when
 * rot_dim = 0 are copied.
 *   - A negative pos[t] marks a padding token: nothing of it is read or written.
 *   - Two tokens of one call must not name the same row of a page: which one stays is
 *     not defined.  A cache whose neighbouring pages, rows or heads share memory (a stride
 *     below head_dim over more than one) is refused (W4A4_ERR_SHAPE), and so is one whose
 *     v begins within a head of its k (W4A4_ERR_ARG).  Other strides are not looked into: no
 *     two rows that a call writes may share memory, and k, v, q and q_out must not lie in them.
 *   - Strides are multiples of 8, at least n_heads * head_dim (q: n_q_heads * head_dim).
 *     rot_dim: a multiple of 16, at most head_dim.  n_tokens < 2^31; n_seqs <= 2^24; n_seqs *
 *     max_pages < 2^31. */
w4a4_status w4a4_kv_append(const w4a4_kv_cache_t *cache, const w4a4_kv_append_t *tokens, void *stream);

/* Device workspace of w4a4_kv_attend: 0 for arguments that it does not accept. */
size_t w4a4_kv_attend_workspace_bytes(int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim);

/* One new token per sequence for w4a4_kv_attend. */
typedef struct {
    const uint16_t *q;        /* [n_seqs, n_q_heads, head_dim], sequences q_stride elements apart */
    uint16_t *out;            /* [n_seqs, n_q_heads, head_dim], contiguous */
    float *lse;               /* [n_seqs, n_q_heads] logarithm of the sum of exponentials, or NULL */
    void *workspace;          /* w4a4_kv_attend_workspace_bytes bytes, contents irrelevant */
    const int32_t *pages;     /* [n_seqs, max_pages] page numbers */
    const int32_t *lens;      /* [n_seqs] tokens of each sequence */
    int64_t q_stride;         /* a multiple of 8, at least n_q_heads * head_dim */
    size_t workspace_bytes;
    int32_t n_seqs, max_pages;
    int32_t n_q_heads;        /* a multiple of the cache's n_heads */
    int32_t window;           /* attend to the last `window` tokens; 0: to all */
    float scale;
} w4a4_kv_attend_t;

/* One new token of every sequence against its cache: for sequence b and query
 * head h, which reads cache head h / (n_q_heads / n_heads),
 *   out[b, h] = sum_t p_t V[t],  p = softmax_t(scale * q[b, h] . K[t])
 * over positions t in [max(0, lens[b] - window), lens[b]) (window 0: all).
 * Statistics and sums are fp32; the weights that multiply values are held to 2^-16 of themselves, in fp16 to
 * 2^-40 of the largest where that is more; the result is rounded once.  A sequence
 * with nothing to attend to (length 0 or negative), or all of whose scores are -inf, gets
 * zeros, and lse = -inf.
 *   - Rows of a page at or behind the length, or in front of the window, are never used,
 *     whatever they hold, nor are the pages that hold only such rows.  Pages may be shared
 *     between sequences.  An infinite value of a token that is attended to gives an infinity
 *     or NaN in its dimension (of the heads that share it); keys follow the formula.
 *   - out may be q itself when q_stride = n_q_heads * head_dim or for one sequence, and must not
 *     overlap it otherwise.  out, lse and the workspace must not overlap one another, pages, lens
 *     or (lse, workspace) q (W4A4_ERR_ARG for all of these), and must not lie in the cache.
 *   - max_pages * page_size is at most 2^30, n_seqs at most 2^24, and n_seqs * n_q_heads *
 *     max_pages * page_size / 16 below 2^31 at the least (W4A4_ERR_SHAPE above).
 *   - A length above max_pages * page_size counts as that many, and a row whose
 *     page number is out of range as absent; both set W4A4_DEV_RANGE.
 *   - How the work is cut follows from the sizes, max_pages * page_size and the window, for the lengths
 *     are on the device: a table no wider than the sequences need is faster for short ones (16 heads of
 *     64, 1 sequence of 128 tokens 4.1 us, 5.5 with room for 16384; 16 of 500 11.6 and 13.9).
 *   - lens and pages are read more than once: they must not change while the call runs.
 *   - Calls that may overlap on the GPU need a workspace each.
 *   - The same inputs give the same bits on every call on one GPU. */
w4a4_status w4a4_kv_attend(const w4a4_kv_cache_t *cache, const w4a4_kv_attend_t *tokens, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_H_ */
