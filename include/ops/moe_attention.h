/*
 * moe_attention.h -- C ABI of the operators that keep a sequence's keys and
 * values and attend to them at a verify step, MI355X (gfx950).
 *
 * A speculative verify step (bjdmk.com.cn news page, section on the road to
 * 1000 tokens/s: a block of 8 drafted tokens and one more) runs the drafted
 * tokens of a sequence through the model at once.  Each of them attends to
 * the sequence's committed tokens and to its own ancestors among the drafted
 * ones.  The pages keep what is not an expert at FP8; the cache here is in
 * the library's 8-bit format (MXFP8: E4M3 elements, one E8M0 scale per 32
 * consecutive elements, the OCP MX block rule of moe_mxfp8_quantize).
 *
 *   moe_kv_write         keys and values of new tokens, encoded into the cache
 *   moe_kv_read          keys and values of given slots, decoded
 *   moe_tree_attention   attention of drafted tokens over the cache
 *
 * Conventions are those of moe_ops.h: the caller owns every tensor (device
 * memory of the current device) and keeps it alive until the work enqueued on
 * `stream` has completed; arguments are checked before anything is enqueued,
 * a failed check returns a negative MOE_E_* status and enqueues nothing; no
 * call synchronises, allocates or copies to the host, keeps state in the
 * library or needs moe_mxfp4_init; a call may be captured into a HIP graph.
 * Scratch memory is a workspace the caller passes, whose contents need not be
 * initialised and mean nothing after the call; two calls whose work may
 * overlap in time need a workspace each.  num_tokens == 0 is a valid no-op.
 * Inputs must not overlap outputs.
 *
 * What the device holds alone (slots, page numbers, lengths) cannot be
 * refused; each argument says what an entry out of its range does.  No entry
 * makes a call read or write outside the tensors it is given.
 */
#ifndef MOE_ATTENTION_H
#define MOE_ATTENTION_H

#include <stdint.h>

#include "../moe_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------------- cache
 * Keys and values in pages of page_size positions.  In page p, element d of
 * head h at position i has its code at
 *
 *   codes[p * codes_page_stride + (h * page_size + i) * head_dim + d]
 *
 * and its block's scale at
 *
 *   scales[p * scales_page_stride + ((h * page_size + i) * head_dim + d) / 32]
 *
 * A slot is p * page_size + i.  Keys and values of one head have the same
 * number of elements, a position's key and value the same slot. */
typedef struct moe_kv_cache {
    uint8_t* k_codes;           /* [num_pages, kv_heads, page_size, head_dim] E4M3 */
    uint8_t* k_scales;          /* [num_pages, kv_heads, page_size, head_dim / 32] E8M0 */
    uint8_t* v_codes;
    uint8_t* v_scales;
    int64_t codes_page_stride;  /* bytes from page to page, at least one page's, up to 2^31; 0: one page's */
    int64_t scales_page_stride;
    int64_t num_pages;          /* 1 .. 2^31 - 1 */
    int32_t page_size;          /* 16, 32, 64, .. 1024 */
    int32_t kv_heads;           /* 1 .. 1024 */
    int32_t head_dim;           /* a multiple of 32, 32 .. 512 (moe_tree_attention: 64, 128 or 256) */
    int32_t reserved;           /* 0 */
} moe_kv_cache;

/* Codes and scales are 16-byte aligned, and so are their page strides. */

/* ------------------------------------------------------- write and read
 * moe_kv_write:  codes, scales at slots[t] = MXFP8(k[t]), MXFP8(v[t]): the
 *                block rule of moe_mxfp8_quantize, bit for bit.  A token whose
 *                slot is outside 0 .. num_pages * page_size - 1 is not
 *                written (padding: -1).  Two tokens may not share a slot (what
 *                it holds then is any mixture of the two).
 * moe_kv_read:   k[t], v[t] = the values at slots[t], rounded to nearest even
 *                where the type does not hold them; zeros for a slot outside
 *                the cache.  Slots may repeat.  Written to other slots again
 *                the values give the same codes and scales, as long as the
 *                type holds them and they came from moe_kv_write: so a step's
 *                accepted tokens are moved to their places. */
typedef struct moe_kv_rows_args {
    moe_kv_cache cache;
    void* k;                /* [num_tokens, kv_heads, head_dim], heads and elements contiguous */
    void* v;
    int64_t k_stride;       /* elements from token to token; 0: kv_heads * head_dim */
    int64_t v_stride;
    const int64_t* slots;   /* [num_tokens] */
    int64_t num_tokens;     /* 0 .. 2^20 */
    int32_t dtype;          /* of k and v: MOE_DT_BF16 or MOE_DT_F32 */
    int32_t reserved;       /* 0 */
} moe_kv_rows_args;

/* k, v and their tokens' starts are 16-byte aligned, slots 8.  MOE_E_NULL,
 * MOE_E_SHAPE (sizes, strides too short), MOE_E_DTYPE, MOE_E_ALIGN,
 * MOE_E_OPTION (reserved), MOE_E_HIP. */
int moe_kv_write(const moe_kv_rows_args* args, void* stream);
int moe_kv_read(const moe_kv_rows_args* args, void* stream);

/* ------------------------------------------------------------- attention
 * Sequence b has L = context_lens[b] committed positions, held in the cache
 * at positions 0 .. L-1, and n = token_offsets[b+1] - token_offsets[b]
 * drafted tokens, whose keys and values are in the cache at positions
 * L .. L+n-1 (moe_kv_write put them there) and whose queries are tokens
 * token_offsets[b] .. token_offsets[b+1]-1.  Position p is in page
 * block_table[b, p / page_size] at p % page_size.  Drafted token i sees
 *
 *   every position p < L, and
 *   position L + j, j < n, if bit j % 64 of mask[i, j / 64] is set
 *   (bits past the mask's words count as clear; mask == NULL: if j <= i)
 *
 * and for head h, with the keys and values of head h / (num_heads / kv_heads):
 *
 *   out[i, h] = sum_p w_p v_p,   w = softmax over the p it sees of scale * <q[i, h], k_p>
 *
 * zeros if it sees none.  What a token does not see has no part in its
 * result, whatever it holds.  A NaN in a value that it sees makes one of that
 * element of its result; an infinite value (one beyond float32's range) makes
 * an infinity of its sign, a NaN where there are both signs, and may make one
 * where its weight is below 2^-126.  Tokens of no sequence (before the first
 * offset, behind the last) have no result: their rows of `out` are left as
 * they were.
 *
 * Products and sums are float32's (of bf16 factors that hold q, k and v
 * exactly; a query or a cached value below 2^-126 may count as zero, one
 * beyond float32's range counts as infinite); the weights e^(s - m) are
 * rounded to bf16 for the product with v, and the sum they are divided by is
 * that of the rounded ones.  m is the running maximum as it last was where a score passed it by
 * more than 8 powers of two.  Sums are added in an order that the sizes and
 * lengths decide: the same inputs give the same bits.  Scores that leave
 * float32's range give unspecified weights.
 *
 * Out of range: a position whose page number is outside 0 .. num_pages-1, or
 * that is beyond max_pages * page_size, is not seen (and not counted as
 * there); a negative context length counts as 0, one above the table's as the
 * table's; if token_offsets are not ascending within 0 .. num_tokens no
 * result is written at all. */
typedef struct moe_tree_attention_args {
    moe_kv_cache cache;            /* head_dim 64, 128 or 256 */
    const void* q;                 /* [num_tokens, num_heads, head_dim] bf16, heads and elements contiguous */
    int64_t q_stride;              /* elements from token to token, up to 2^31; 0: num_heads * head_dim */
    void* out;                     /* as q */
    int64_t out_stride;
    const int32_t* block_table;    /* [num_seqs, max_pages] */
    int64_t block_table_stride;    /* entries from sequence to sequence; 0: max_pages */
    const int32_t* context_lens;   /* [num_seqs] */
    const int32_t* token_offsets;  /* [num_seqs + 1] */
    const uint64_t* mask;          /* [num_tokens, mask_words] or NULL */
    int64_t mask_words;            /* 1 .. 64; 0 with mask == NULL (without tokens or sequences 0 .. 64) */
    void* workspace;               /* at least moe_tree_attention_workspace() bytes */
    int64_t workspace_bytes;
    int64_t num_tokens;            /* 0 .. 2^20, of q and out */
    int64_t num_seqs;              /* 0 .. 2^16 */
    int64_t max_pages;             /* of a sequence; max_pages * page_size 1 .. 2^30 */
    int32_t num_heads;             /* a multiple of cache.kv_heads, up to 1024 */
    float scale;                   /* finite, > 0 */
} moe_tree_attention_args;

/* Bytes of workspace (0 without tokens or sequences), or a negative status
 * for sizes that moe_tree_attention refuses.  Of the call's own sizes: fewer
 * sequences with more tokens each may need more. */
int64_t moe_tree_attention_workspace(int64_t num_tokens, int64_t num_seqs, int32_t num_heads, int32_t kv_heads,
                                     int32_t head_dim);

/* Pointers 16-byte aligned (context_lens, token_offsets, block_table: 4, mask:
 * 8), and so are the tokens of q and out.  MOE_E_NULL, MOE_E_SHAPE,
 * MOE_E_ALIGN, MOE_E_OPTION (scale, reserved), MOE_E_LIMIT (workspace too
 * small; or num_tokens, num_seqs, kv_heads and max_pages together past 2^30
 * units of 128 positions), MOE_E_HIP. */
int moe_tree_attention(const moe_tree_attention_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTENTION_H */
