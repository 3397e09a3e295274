/*
 * mlra_serving.h -- libmlra's operators around the decode step: the prompt
 * pass that comes before the first token, and the eviction that keeps a long
 * cache small.  They work on the dims, the page pools, the page table and the
 * workspace conventions of mlra.h, which this header includes; read its
 * conventions first (ownership, asynchrony, errors: all hold here).
 *
 * A serving loop strings them together:
 *   latent_store           the prompt's compressed tokens into the cache
 *   mla_prompt             the prompt's attention
 *   mla_decode             (or mlra_attend_partial + mlra_merge_upproj, which
 *                          also give the log-sum-exp) one token at a time
 *   mlra_absorb, mlra_attention_weights
 *                          what each cached token has been worth so far
 *   latent_evict           the tokens worth least leave, whole pages are freed
 *   latent_append          the next token, as before
 *
 * Device and streams: every call enqueues on `stream`, which has to belong to
 * the calling thread's current device, where all buffers lie.  A workspace
 * serves one call at a time: two calls (or two captured graphs) that may run
 * at the same time need one each.
 *
 * Overlap: an output, the workspace among them, shares no byte with an input or
 * another output (MLRA_ERR_INVALID_ARG), but for mlra_attention_weights in
 * place.  A strided input counts from its first element to its last.
 */
#ifndef MLRA_SERVING_H_
#define MLRA_SERVING_H_

#include "mlra.h"

/* The entry points of this header (mlra.h's own carry its own mark). */
#define MLRA_SERVING_API MLRA_API

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * mla_prompt -- causal attention of whole prompts.
 *
 * dims->B sequences are packed: sequence b's queries are rows
 * [cu_q[b], cu_q[b+1]) and its keys and values rows [cu_k[b], cu_k[b+1]).
 * Its keys sit at positions 0 .. Lk-1 and its Lq queries are the last Lq of
 * them (query i at position Lk - Lq + i), so Lk > Lq is a chunk of a prompt
 * whose beginning is cached already.  Unabsorbed form (yololab.net,
 * "超越 GQA 的推理革命…", sections "1. 鍵值聯合低秩壓縮" and "2. 解耦旋轉位置編碼"):
 *   x[i,j]  = scale * (q_nope[i,h] . k_nope[j,g] + RoPE(q_rope[i,h]) . k[j])
 *   out[i,h] = sum_{j <= Lk-Lq+i} softmax_j(x[i,:]) v[j,g]
 *   lse[i,h] = log2 sum_{j <= Lk-Lq+i} 2^(x[i,j] log2(e))     (if lse != NULL)
 * where k_nope = W_UK[h] . c and v = c . W_UV[h] are the up-projected latents
 * (a plain matrix product, the caller's), g = h / (H / kv_heads), and k[j] is
 * the rotated key that latent_store left in rope_cache at position j.  A query
 * with no key (Lq > Lk) gives a zero row and an lse of -inf.
 *
 * Rows of out and lse outside every [cu_q[b], cu_q[b+1]) are not touched.
 * What lies behind a sequence's last key (the next sequence's rows, unused
 * slots of its last page) does not reach its output, and what lies behind a
 * query's last key does not reach that query's, NaN and infinities included
 * (a NaN or an infinity in v costs the queries before it a slower pass).
 *
 *   q_nope [total_q, H, d_h]   q_rope [total_q, H, d_r] (un-rotated)
 *   k_nope [total_k, kv_heads, d_h]   v [total_k, kv_heads, d_v]
 *     strided: the strides (elements) of the token and head axes are in the
 *     shape, the last axis is contiguous; views of the projections' outputs
 *     go in as they are
 *   cu_q, cu_k [B+1] int32, ascending, within [0, total_q] and [0, total_k]
 *   rope_cache [num_pages, page_size, d_r]   page_table [B, max_pages_per_seq]
 *   out [total_q, H, d_v] dense   lse [total_q, H] fp32 dense, or NULL
 * dims: n_branch must be 1; d_c is not used; d_v <= 512.  A sequence whose
 * offsets are out of range, or whose Lk the page table cannot hold, is
 * reported (mlra_check_status) and gets no output; so is a batch whose
 * sequences overlap so far that they have more than total_q rows together, and
 * then its outputs are void.
 * Kernel AUTO runs the tcgen05 kernel for bf16, d_h = 128, d_r = 64,
 * d_v = 128 with every stride a multiple of 8 elements, and the CUDA-core
 * kernel otherwise.
 * ------------------------------------------------------------------------- */
typedef struct {
  int kv_heads;                    /* H is a multiple of it */
  int total_q, total_k;            /* rows of the packed arrays */
  long long q_nope_stride[2];      /* {token, head}, in elements */
  long long q_rope_stride[2];
  long long k_nope_stride[2];
  long long v_stride[2];
} mla_prompt_shape;

MLRA_SERVING_API size_t mla_prompt_workspace_bytes(const mlra_dims* dims, const mla_prompt_shape* shape);
MLRA_SERVING_API mlra_status mla_prompt(const mlra_dims* dims, const mla_prompt_shape* shape, const void* q_nope,
                                        const void* q_rope, const int32_t* cu_q, const void* k_nope, const void* v,
                                        const int32_t* cu_k, const void* rope_cache, const int32_t* page_table,
                                        void* out, float* lse, void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * mlra_absorb -- the decode step's query side by itself (yololab.net, section
 * "矩陣吸收"): what the scores against the cached latent are taken with.
 *   q_abs[b,h,:d_c] = scale * log2(e) * q_nope[b,h] . W_UK[h]
 *   q_abs[b,h,d_c:] = scale * log2(e) * RoPE(q_rope[b,h], q_pos[b])
 * so that q_abs . [c; k] is a base-2 logit.  Arguments as in mla_decode;
 * q_abs [B, H, d_c + d_r] (dtype).  workspace: at least 256 bytes (the device
 * error record), 256-byte aligned.
 *
 * mlra_attention_weights -- each cached token's attention weight, summed over
 * heads and branches and added to what it has gathered so far:
 *   weights[b,t] = weights_in[b,t]
 *                + sum_{br,h} 2^(q_abs[b,h] . [c_br; k][b,t] - lse[b,br,h])
 * for t < seq_lens[b]; weights of later slots are not touched.  lse is the
 * base-2 log-sum-exp of the same scores, as mlra_attend_partial writes it
 * (over several GPUs: the merged one); a head whose lse is -inf attended
 * nothing and adds nothing.
 *   q_abs [B, H, d_c + d_r]   lse [B, n_branch, H] fp32
 *   weights_in [B, max_pages_per_seq * page_size] fp32: NULL for zeros, and
 *     the same buffer as weights to add in place (no partial overlap)
 *   weights [B, max_pages_per_seq * page_size] fp32
 * The same inputs give the same bits.  workspace: at least 256 bytes, 256-byte
 * aligned.  Kernel AUTO runs the tcgen05 kernel for bf16, d_r = 64, branches
 * of a multiple of 64 dims and n_branch * H (H rounded up to 32, at most 128)
 * <= 512, and the CUDA-core kernel otherwise.
 * ------------------------------------------------------------------------- */
MLRA_SERVING_API mlra_status mlra_absorb(const mlra_dims* dims, const void* q_nope, const void* q_rope,
                                         const int32_t* q_pos, const void* W_UK, void* q_abs, void* workspace,
                                         size_t workspace_bytes, cudaStream_t stream);
MLRA_SERVING_API mlra_status mlra_attention_weights(const mlra_dims* dims, const void* q_abs, const float* lse,
                                                    const void* latent_cache, const void* rope_cache,
                                                    const int32_t* page_table, const int32_t* seq_lens,
                                                    const float* weights_in, float* weights, void* workspace,
                                                    size_t workspace_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * latent_evict -- free evict_pages[b] = n pages of each sequence: the 64 n
 * tokens with the least weight leave the cache (of equal weights the later
 * slot leaves first; a NaN weight counts as -inf), except that the last
 * `recent` tokens always stay.  The n pages that the sequence gives up are the
 * first n of its page-table row; those of their tokens that stay move into the
 * slots that tokens leaving the other pages make free, the i-th in slot order
 * into the i-th.  The decode does not depend on the order of cached tokens
 * (rope keys are stored rotated), so nothing else has to move, the most recent
 * tokens keep their places and their order, and no slot is both read and
 * written.
 *   evict_pages [B] int32, 0 <= 64 n <= seq_lens[b] - recent (n = 0: the
 *     sequence stays as it is); another n is reported (mlra_check_status) and
 *     taken as 0
 *   weights [B, max_pages_per_seq * page_size] fp32   (read)
 *   page_table [B, max_pages_per_seq], seq_lens [B]   (read)
 *   latent_cache, rope_cache: written in the slots that tokens move to
 *   weights_out [B, max_pages_per_seq * page_size]: the weights of the tokens
 *     in their new slots, zeros behind them
 *   page_table_out [B, max_pages_per_seq]: the row without its first n
 *     entries, -1 behind it; entries [0, n) of the old row are the pages that
 *     this sequence no longer names (a prefix that it shares with others lies
 *     among them: such a page is free only when no sequence names it)
 *   seq_lens_out [B] = seq_lens[b] - 64 n
 * Decode with page_table_out and seq_lens_out.  Positions do not change: q_pos stays the token's position,
 * and latent_append, which finds a token's slot by its position, keeps taking
 * a table indexed by absolute page (the table from before the first eviction,
 * extended by new pages at both tables' ends).
 * A page that a token moves to has to be this sequence's alone: one that
 * page_table lists more than once (a shared prefix), or whose id is out of
 * range, is reported and not written; that sequence's result is void then.
 * ------------------------------------------------------------------------- */
MLRA_SERVING_API size_t latent_evict_workspace_bytes(const mlra_dims* dims);
MLRA_SERVING_API mlra_status latent_evict(const mlra_dims* dims, int recent, const int32_t* evict_pages,
                                          const float* weights, const int32_t* page_table, const int32_t* seq_lens,
                                          void* latent_cache, void* rope_cache, float* weights_out,
                                          int32_t* page_table_out, int32_t* seq_lens_out, void* workspace,
                                          size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MLRA_SERVING_H_ */
