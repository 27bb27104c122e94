/*
 * mla_kv8.h -- the 8-bit latent cache of the GB300 (sm_103a) MLA decode library
 * (libmla_decode.so), and the rotary positions of its inputs.
 *
 * The cache holds the same entries as the bf16 cache of mla_decode.h in half
 * the bytes: entry (page, slot, g) is 576 e4m3 codes (512 latent, 64 rope) and
 * one fp32 scale, and stands for K_t = code * scale, V_t = K_t[0:512].
 *
 *   codes   uint8 (e4m3: 4 exponent bits, 3 mantissa bits, no infinities, NaN 0x7f),
 *           entry (page, slot, g) at ((page*64 + slot)*h_kv + g)*stride bytes;
 *           stride >= 576 and a multiple of 16 (576 dense, 640 padded); the pad is
 *           neither read nor written
 *   scales  fp32[num_blocks][h_kv][64], 16-byte aligned
 *
 * The scale covers one token of one head: an entry is then written once and
 * never changed by later tokens.  mla_write_cache_kv8 uses powers of two, so
 * that code * scale is exact in bf16 wherever it is a normal number; the
 * readers take any finite scale that is not negative.
 *
 * Conventions are those of mla_decode.h: device pointers on the current
 * device, owned by the caller; no allocation and no synchronisation; calls
 * enqueue on `stream` and may be captured in a CUDA graph; arguments that the
 * host can check are checked first and a failed check enqueues nothing; what
 * only the device can see goes to the caller's status word.
 */
#ifndef MLA_KV8_H_
#define MLA_KV8_H_

#include "mla_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * New tokens into the 8-bit cache (the counterpart of mla_write_cache): token t
 * with s = slot_mapping[t] >= 0 goes to page s / 64, slot s % 64.  Over its 576
 * values x = [kv_c[t], k_pe[t]],
 *     scale = the smallest 2^e, e >= -126, with max |x| <= 448 * 2^e
 *     code  = x / scale rounded to e4m3, ties to even
 * Values that are not finite are stored as NaN and leave the scale to the
 * others.  Negative slots are skipped (padding tokens); slots outside the
 * cache are skipped and reported as MLA_ERR_BAD_BLOCK_ID.  Two tokens of one
 * call must not share a slot (that entry is then unspecified).
 *   kv_c          bf16 rows of 512, `kv_c_row_stride` elements apart (>= 512, multiple of 8)
 *   k_pe          bf16 rows of 64, `k_pe_row_stride` elements apart (>= 64, multiple of 8)
 *   slot_mapping  int64[num_tokens]
 *   h_kv          1 (MLA caches have one latent head); kv_c, k_pe and codes 16-byte aligned
 */
mla_status_t mla_write_cache_kv8(const void *kv_c, int64_t kv_c_row_stride, const void *k_pe,
                                 int64_t k_pe_row_stride, const int64_t *slot_mapping,
                                 int64_t num_tokens, void *codes, float *scales,
                                 int64_t num_blocks, int block_size, int stride, int32_t *status,
                                 mla_stream_t stream);

/*
 * Entries of b ragged token ranges back as contiguous bf16 rows:
 *     out[cu_tokens[i] + n] = bf16(code * scale) of token starts[i] + n of sequence i
 * for 0 <= n < cu_tokens[i+1] - cu_tokens[i].
 *   block_table   int32[b, max_blocks_per_seq]
 *   cu_tokens     int32[b + 1], device: 0 = cu[0] <= cu[1] <= ... <= cu[b]
 *   starts        int32[b], device, >= 0; NULL means all 0
 *   out           bf16[rows, 576], 16-byte aligned; rows from cu_tokens[b] on stay as they are,
 *                 and rows past `rows` are not written even where cu_tokens asks for them
 * Tokens whose page lies outside the table or the cache leave their row as it
 * is and are reported as MLA_ERR_BAD_BLOCK_ID; a negative token index is
 * reported as MLA_ERR_BAD_SEQLEN.
 */
mla_status_t mla_read_cache_kv8(const void *codes, const float *scales, int64_t num_blocks,
                                int block_size, int stride, const int32_t *block_table,
                                int max_blocks_per_seq, const int32_t *cu_tokens,
                                const int32_t *starts, int b, void *out, int64_t rows,
                                int32_t *status, mla_stream_t stream);

/*
 * Decode over the 8-bit cache: mla_decode_with_kvcache with K_t = code * scale.
 * The schedule (mla_get_metadata) is the same; the part count comes
 * from mla_num_parts_kv8 and the workspace size from mla_workspace_bytes_kv8 (the
 * split-KV scratch, and for more than 64 query rows per KV head the queries in 8
 * bits).  Arguments and results as there, except
 *   codes, scales, stride   as above, codes 16-byte aligned, stride in bytes
 *   q                       bf16; finite values (a row holding others gives NaN)
 * Entries at or past a sequence's length, and with `causal` those a query does
 * not see, never reach that query's result, whatever they hold (NaN included).
 * An entry that a query does see and that holds a NaN, or whose scale is not
 * finite, makes its row NaN.  A weight p_t scale_t is held to 2^-8 of itself (2^-7
 * for more than 64 query rows per KV head) or 2^-16 of its row's largest, as long as
 * the scales of a sequence that are above 2^-60 lie within 2^80 of one another (smaller
 * ones beside them, those of zero entries among them, count in full in the softmax);
 * where all that every query sees is at or below 2^-60, what only some see may be up to
 * 2^75.  For more than 262140 rows s_q h_q, which no decode takes, the part count is
 * MLA_ERR_UNSUPPORTED and the workspace size 0.
 */
int mla_num_parts_kv8(int s_q, int h_q, int h_kv, int device);

size_t mla_workspace_bytes_kv8(int b, int s_q, int h_q, int h_kv, int num_parts);

mla_status_t mla_decode_kv8(const void *q, int b, int s_q, int h_q, int d, const void *codes,
                            const float *scales, int64_t num_blocks, int block_size, int h_kv,
                            int stride, const int32_t *block_table, int max_blocks_per_seq,
                            const int32_t *cache_seqlens, int dv, const int32_t *metadata,
                            int num_parts, const int32_t *num_splits, float softmax_scale,
                            int causal, void *out, float *lse, void *workspace,
                            size_t workspace_bytes, int32_t *status, mla_stream_t stream);

/*
 * Rotary positions: pair i of a row at position p turns by the angle
 * 2 pi p f_i, and the row is multiplied by `gain`:
 *     (u, v) -> gain * (u cos - v sin, u sin + v cos)
 * Pairs are (x[2i], x[2i+1]) with interleaved = 1 and (x[i], x[i + rot_dim/2])
 * with 0.  `inverse` = 1 turns back (the transposed map: also its gradient).
 *   turns      uint64[rot_dim/2], device: f_i in turns per position, as
 *              round(f_i * 2^64) mod 2^64; p * turns wraps at whole turns, so the angle
 *              stays exact to p * 2^-65 turns however far the position
 *   positions  int32[tokens] or int64[tokens] (position_bytes 4 or 8), any sign
 *   x, out     [tokens, heads, rot_dim], strides in elements, last one dense; out may be x
 *              itself with the same strides; one whose rows meet those of x otherwise, of
 *              k or k_out, or one another, is refused (a stride of one token or one head
 *              is not looked at)
 *   k, k_out   a second such pair [tokens, k_heads, rot_dim] turned in the same launch, or
 *              NULL with k_heads = 0
 *   dtype      MLA_BF16, MLA_FP16 or MLA_FP32, of all four; computed in fp32, rounded once
 *   rot_dim    even, 2 .. 256
 */
enum { MLA_BF16 = 0, MLA_FP16 = 1, MLA_FP32 = 2 };

mla_status_t mla_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
                      int64_t out_token_stride, int64_t out_head_stride, int heads, const void *k,
                      int64_t k_token_stride, int64_t k_head_stride, void *k_out,
                      int64_t k_out_token_stride, int64_t k_out_head_stride, int k_heads,
                      int64_t tokens, int rot_dim, const void *positions, int position_bytes,
                      const uint64_t *turns, float gain, int interleaved, int inverse, int dtype,
                      mla_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLA_KV8_H_ */
