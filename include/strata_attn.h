/*
 * strata_attn.h -- C ABI of the attention step over the 4-bit rotated KV
 * cache: rotary positions, the paged cache (append, copy of pages) and the
 * attention that reads it.
 *
 * Source: "Strata：把 125B 大模型塞进 12GB 显卡，24,576 个专家在内存与 SSD 之间流动",
 * section 长上下文 (the optional 4-bit KV cache: one Hadamard rotation, then
 * 4-bit rounding; the codec is in strata_kv.h) and section 再快一截 (verify
 * steps of 1 + 3 and 1 + 5 tokens). The pages give no interface for the
 * attention: this one is the library's own.
 *
 * Conventions as in strata_moe.h: tensor arguments are device pointers unless
 * marked "host", calls are asynchronous on `stream`, the caller owns every
 * buffer, argument errors return before anything is enqueued, and the reason
 * is in strata_last_error(). All calls may be captured into CUDA graphs. No
 * call keeps device state of its own: calls on different streams may overlap
 * as long as their buffers (the attention's workspace among them) differ.
 * Work runs on the current device, which must own the buffers and the stream.
 */
#ifndef STRATA_ATTN_H
#define STRATA_ATTN_H

#include "strata_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ rotary
 * The first rotary_dim values of a head row are turned in pairs by angles
 * position * f_i, i < rotary_dim / 2; the others stay as they are.
 *   pair i: values (i, i + rotary_dim/2) for STRATA_ROPE_HALF,
 *           values (2i, 2i + 1) for STRATA_ROPE_INTERLEAVED;
 *   (u, v) -> (u c - v s, v c + u s), c = fp32(m cos), s = fp32(m sin).
 * Frequencies f_i = theta^(-2i / rotary_dim) in fp64, by `scaling`:
 *   NONE    as they are;
 *   LINEAR  f_i / factor;
 *   NTK     theta replaced by theta * factor^(rotary_dim / (rotary_dim - 2));
 *   YARN    f_i / factor * r_i + f_i (1 - r_i), r_i = clamp((i - lo) / (hi - lo), 0, 1),
 *           lo = max(floor(p(beta_fast)), 0), hi = min(ceil(p(beta_slow)), rotary_dim - 1)
 *           (hi - lo = 0 reads as 0.001),
 *           p(t) = rotary_dim ln(original_max_position / (2 pi t)) / (2 ln theta).
 * m = attn_factor; when that is 0, m = 0.1 ln(factor) + 1 for YARN, else 1.
 * The turn position * f_i / (2 pi) is taken modulo 1 in 64-bit fixed point, so
 * far positions lose nothing; positions are int32 and may be negative.
 * strata_rope_apply and strata_kv4_append take the cosine and sine in fp64,
 * round them to fp32, round each product and each sum of the pair to fp32 and
 * the result to bf16 (ties to even): their bits are determined by the input.
 */
#define STRATA_ROPE_HALF 0
#define STRATA_ROPE_INTERLEAVED 1
#define STRATA_ROPE_SCALE_NONE 0
#define STRATA_ROPE_SCALE_LINEAR 1
#define STRATA_ROPE_SCALE_NTK 2
#define STRATA_ROPE_SCALE_YARN 3
#define STRATA_ROPE_MAX_HEAD_DIM 256

typedef struct {
    int32_t head_dim;              /* multiple of 8, 8..256 */
    int32_t rotary_dim;            /* even, 2..head_dim */
    int32_t layout;                /* STRATA_ROPE_HALF or STRATA_ROPE_INTERLEAVED */
    int32_t scaling;               /* STRATA_ROPE_SCALE_* */
    double theta;                  /* > 1 */
    double factor;                 /* >= 1; not used by SCALE_NONE */
    int32_t original_max_position; /* YARN: > 0 */
    double beta_fast, beta_slow;   /* YARN: beta_fast > beta_slow > 0 (0, 0: 32 and 1) */
    double attn_factor;            /* m; 0: the scaling's own */
} strata_rope_desc;

typedef struct strata_rope_s *strata_rope;

/* Validate desc and build the table of frequencies (host memory only; the
 * handle is read-only and may be used from any thread, stream and device).
 * Errors: INVALID_ARG, UNSUPPORTED (layout, scaling), OOM. */
strata_status strata_rope_create(const strata_rope_desc *desc, strata_rope *out);
strata_status strata_rope_destroy(strata_rope rope);

/* out[t][h] = rotary(x[t][h], positions[t]) for bf16 rows of head_dim values.
 * Row (t, h) of x starts at x + t * x_token_stride + h * x_head_stride
 * (elements), likewise out. out may be x with the same strides (in place);
 * any other overlap is not allowed. x and out 16-byte aligned, strides
 * multiples of 8 that keep the rows apart: token strides that hold a token's
 * heads, or head strides that hold a head's tokens; positions int32 [n_tokens].
 * n_tokens or n_heads 0: no-op. Errors: INVALID_ARG, CUDA. */
strata_status strata_rope_apply(strata_rope rope, const void *x, int64_t x_token_stride, int64_t x_head_stride,
                                const int32_t *positions, int64_t n_tokens, int32_t n_heads, void *out,
                                int64_t out_token_stride, int64_t out_head_stride, strata_stream_t stream);

/* ------------------------------------------------------------------- cache
 * One layer's paged cache in the format of strata_kv.h. A page holds
 * page_size token slots of every KV head:
 *   codes  [n_pages][n_kv_heads][page_size][head_dim / 2] bytes
 *   scales [n_pages][n_kv_heads][page_size][head_dim / 32] fp16
 * for keys and for values, so (page * n_kv_heads + head) * page_size + slot is
 * the row that strata_kv4_encode and strata_kv4_decode would use.
 */
typedef struct {
    void *k_codes, *k_scales, *v_codes, *v_scales; /* device, 16-byte aligned */
    int64_t n_pages;     /* n_pages * n_kv_heads * page_size < 2^32 - 1 */
    int32_t n_kv_heads;  /* 1.. */
    int32_t page_size;   /* a power of two, 16..1024 */
    int32_t head_dim;    /* 64, 128 or 256 */
} strata_kv4_cache;

/* Append n_tokens key and value rows of every KV head: the key rows pass
 * through `rope` (NULL: none) at positions[t], then both go through the
 * codec's encoder and into slot slots[t] = page * page_size + slot of the
 * cache (int64 [n_tokens]). A token whose slot is negative, or past the last
 * page, is dropped (padding). The slots of the other tokens must differ from
 * one another: rows of two tokens in one slot get mixed. Codes and scales are
 * bit for bit those of strata_rope_apply followed by strata_kv4_encode.
 * Rows (t, h) of k start at k + t * k_token_stride + h * head_dim (elements),
 * likewise v; k and v 16-byte aligned, strides multiples of 8 that hold a
 * token's heads. positions may be NULL when rope is. Inputs must be finite, as for strata_kv4_encode.
 * Errors: INVALID_ARG, UNSUPPORTED (head_dim, page_size), CUDA. */
strata_status strata_kv4_append(const strata_kv4_cache *cache, strata_rope rope, const void *k,
                                int64_t k_token_stride, const void *v, int64_t v_token_stride,
                                const int32_t *positions, const int64_t *slots, int64_t n_tokens,
                                strata_stream_t stream);

/* Copy pages src[i] -> dst[i] (whole pages, all four planes) in each of
 * n_caches caches of one shape (a model's layers): a fork of sequences that
 * share a prefix, or the compaction of a pool. caches, src and dst are HOST
 * arrays, read before the call returns. The destinations must differ from one
 * another, and no page may be both a source and a destination (a source may
 * be named more than once). n_pairs or n_caches 0: no-op. The planes of the
 * caches must not overlap. Errors: INVALID_ARG (a page out of range or named
 * against these rules, caches of different shapes), UNSUPPORTED, OOM, CUDA. */
strata_status strata_kv4_copy_pages(const strata_kv4_cache *caches, int32_t n_caches, const int32_t *src,
                                    const int32_t *dst, int64_t n_pairs, strata_stream_t stream);

/* --------------------------------------------------------------- attention
 * Causal attention of the newest tokens of n_seqs sequences over their cached
 * keys and values (which already hold the new tokens). Sequence b has query
 * rows q_offsets[b] .. q_offsets[b + 1] - 1 (n of them) and kv_lens[b] = L
 * cached tokens; its query i stands at position p = L - n + i and sees the
 * cached positions j <= p, and, with a window w > 0, only p - w < j. Cached
 * position j is slot j % page_size of page block_table[b][j / page_size]. Query
 * head h reads KV head h / (n_q_heads / n_kv_heads).
 *   out[t][h] = sum_j softmax_j(scale * q[t][h] . k_j) v_j,  bf16.
 * A query that sees no key gives zeros. Positions on a page that is negative
 * or >= n_pages (an evicted page) count as masked. Slots that no query of a
 * sequence sees (in front of its first query's window, behind its last token)
 * may hold anything, NaN scales too; the scales of the others must be finite,
 * as the codec leaves them. Lengths are clamped to
 * 0 <= L <= max_pages * page_size and the offsets to 0..n_tokens; query rows
 * outside every sequence, in front of, between or behind them, are not read
 * and their rows of out are left as they were.
 * q passes through `rope` first (NULL: none) at positions[t]; here the rotated
 * row is kept in fp32 instead of being rounded to bf16.
 * Precision: logits, softmax statistics and output sums in fp32; the rotated
 * q, the probabilities (times the values' scales, or beside scaled values) and,
 * with more than 48 rows max_q_len * n_q_heads / n_kv_heads, the scaled keys
 * enter the tensor cores in fp16 (with power-of-two scales, so that no
 * magnitude of the inputs overflows fp16; rotated q and logits times log2(e)
 * have to stay within fp32); the queries' cosines and sines are those of the
 * hardware (2^-20.9). Results do not depend on timing: the same call
 * gives the same bits, another max_q_len may give others.
 * Any n_seqs and lengths >= 0; q and out 16-byte aligned, token strides
 * multiples of 8 that hold a token's heads, heads head_dim apart. out may be q
 * with the same stride (in place); any other overlap is not allowed.
 * workspace: strata_kv4_attention_workspace_bytes() bytes, 16-byte aligned,
 * its contents neither read nor kept between calls; calls that may overlap
 * need one each. Should a wait inside the tensor-core kernel run out (2 s), the
 * rows concerned become NaN. Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
typedef struct {
    int32_t n_seqs;
    int32_t n_q_heads;        /* a multiple of n_kv_heads */
    int32_t max_q_len;        /* the largest n: picks the kernel; larger ones still run */
    int32_t max_pages;        /* entries of a row of block_table */
    int64_t n_tokens;         /* rows of q and out */
    int64_t q_token_stride;   /* elements */
    int64_t out_token_stride; /* elements */
    int32_t window;           /* 0: every earlier position */
    float scale;              /* finite, scale log2(e) too */
} strata_kv4_attn_desc;

/* Workspace of strata_kv4_attention on this cache's shape for n_q_heads query
 * heads, whatever the sequences (partial results of 148 thread blocks: 21 MB
 * for head_dim 64, 40 MB for 128 and 256); 0 for shapes that are not supported.
 * A model's layers, one after the other, can share one. */
size_t strata_kv4_attention_workspace_bytes(const strata_kv4_cache *cache, int32_t n_q_heads);

strata_status strata_kv4_attention(const strata_kv4_cache *cache, const strata_kv4_attn_desc *desc, strata_rope rope,
                                   const int32_t *positions, const void *q, const int32_t *q_offsets,
                                   const int32_t *kv_lens, const int32_t *block_table, void *out, void *workspace,
                                   size_t workspace_bytes, strata_stream_t stream);

/* Failure-detection self test: the attention by its tensor-core kernel without
 * rotary, in which one role of every `every`-th thread block stops signalling
 * from its piece of work number `piece` on (role 0: expanded keys, 1: expanded
 * values, 2: weights, 3: query rows) and waits give up after 5 ms. A query row
 * that such a piece, or one behind it, has part in comes out as NaN, every other
 * as strata_kv4_attention computes it (or NaN, where it was done last before). */
strata_status strata_selftest_attention_timeout(const strata_kv4_cache *cache, const strata_kv4_attn_desc *desc,
                                                const void *q, const int32_t *q_offsets, const int32_t *kv_lens,
                                                const int32_t *block_table, void *out, void *workspace,
                                                size_t workspace_bytes, int32_t role, int32_t every, int32_t piece,
                                                strata_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* STRATA_ATTN_H */
