/*
 * cq_kv8 -- an 8-bit key/value cache in pages and the attention that reads it
 * (part of libcq.so; conventions, status codes and error words as in cq.h).
 *
 * Cache format (one layer).  Keys and values are int8 codes in pages of `page`
 * tokens, Kq and Vq [pages][Hkv][page][D]; 32 consecutive tokens of one head (a
 * block) share one f32 scale, Ks and Vs [pages][Hkv][page/32].  Token p of
 * sequence b is row p % page of page table[b * ldt + p / page].
 *   value = code * scale, code in [-127, 127], scale = 2^e,
 *   e = the smallest integer >= -64 with (largest magnitude) <= 127 * 2^e.
 * A power of two makes every product exact, lets a growing block move to a larger
 * scale by one rounding of its codes, and is reached again only when the block's
 * largest magnitude doubles; against amax / 127 it costs at most one of the
 * code's eight bits.  One scale serves all channels, so a channel that is much larger
 * than the others takes bits from them: attention over 4096 normal keys and values is
 * 2 % (norm) from that over the unrounded ones, 5 % if one key channel in 29 is 5 times
 * as large.  Values whose code rounds up past a type's largest one read as infinite in
 * it (above 65024 in fp16, above 127 * 2^121 in bf16 and f32).  A block that is given
 * a value that is not finite gets the scale NaN (its reading is NaN, not a plausible
 * number) until it is written again from its first token; lengths that go back leave a
 * block its scale as well.
 * Rows past a sequence's length, and scales of blocks past it, are never used:
 * they may hold anything.
 *
 * Ragged batches.  Row r of K, V, Q or O belongs to sequence b with
 * q_start[b] <= r < q_start[b+1]; q_start is a device array of B + 1 ascending
 * entries in [0, T].  Sequences without rows are allowed.
 */
#ifndef CQ_KV8_H
#define CQ_KV8_H

#include "cq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CQ_KV8_BLOCK 32   /* tokens that share a scale */

/* Host descriptor of a cache (the pointers are device pointers; the library reads
 * the descriptor during the call only). */
typedef struct {
    int8_t* Kq;            /* [pages][Hkv][page][D] */
    float* Ks;             /* [pages][Hkv][page/32] */
    int8_t* Vq;
    float* Vs;
    int64_t pages, Hkv, page, D;
    const int32_t* table;  /* [B][ldt] page numbers; entries past a sequence's pages may hold anything and are read only
                              where a length is wrong: all B * ldt must be readable */
    int64_t ldt, B;
} cq_kv8_cache;
/* Shape rules of the descriptor: pages >= 1, 1 <= Hkv <= 1024, page >= 32 and
 * page % 32 == 0, D 64 or 128, pages * Hkv * page < 2^31, ldt >= 1,
 * 1 <= B <= 65536.  Kq, Vq, Ks, Vs 16-byte aligned, table 4-byte aligned.
 * Device-detected (CQ_ERR_INDEX): a length outside [0, ldt * page] (attention: or
 * above 2^31 - 2048), a q_start that descends or leaves [0, T], a page number outside
 * [0, pages).  The rows of a sequence with such an entry are unspecified, nothing
 * outside the tensors is touched. */

/* ---------------------------------------------------------------------------
 * Write:  the rows of K and V become the last tokens of their sequences.
 * Sequence b holds lens[b] tokens after the call; its n_b = q_start[b+1] -
 * q_start[b] rows are tokens lens[b] - n_b .. lens[b] - 1 (n_b <= lens[b], else
 * CQ_ERR_INDEX).  A block that keeps earlier tokens takes the larger of its old
 * scale and the new tokens' own; if that is larger than the old one, the kept codes
 * become rint(code * old / new).  Codes are rint(value / scale), ties to even.
 * K, V: xt fp16, bf16 or f32, [T][Hkv][D] with row pitches ldk, ldv elements
 * (multiples of 16 bytes, >= Hkv * D), 16-byte aligned.  No workspace; one launch.
 * ------------------------------------------------------------------------- */
cq_status cq_kv8_write(const cq_kv8_cache* cache, const void* K, const void* V, int xt, int64_t T, int64_t ldk,
                       int64_t ldv, const int32_t* q_start, const int32_t* lens, void* stream);

/* ---------------------------------------------------------------------------
 * Read back:  rows out_start[b] .. out_start[b+1] - 1 of K and V become the values
 * of tokens first[b] .. of sequence b (first = NULL: from token 0).
 * K, V: yt fp16, bf16 or f32, [T][Hkv][D] with pitches ldk, ldv as above.  Each
 * value is code * scale rounded once to yt (exact in bf16 and f32).  One launch.
 * ------------------------------------------------------------------------- */
cq_status cq_kv8_read(const cq_kv8_cache* cache, const int32_t* first, const int32_t* out_start, void* K, void* V,
                      int yt, int64_t T, int64_t ldk, int64_t ldv, void* stream);

/* ---------------------------------------------------------------------------
 * Attention over the cache:
 *   s_j = scale * q . k_j,  O = sum_j exp(s_j) v_j / sum_j exp(s_j),
 *   lse = log sum_j exp(s_j)       (nullable)
 * over the tokens j that a row sees.  Row i of sequence b (n_b rows, lens[b] tokens)
 * stands at position p = lens[b] - n_b + i.  causal = 1: it sees
 * max(0, p - window + 1) .. p (window = 0: from token 0); causal = 0: it sees all
 * lens[b] tokens (window must be 0).  A row that sees nothing gets O = 0 and
 * lse = -inf; one whose scores are all -inf, or one of them +inf or NaN, gets NaN.
 * Head h of Q reads head h / (Hq / Hkv) of the cache.
 * Q: xt fp16 or bf16 [T][Hq][D], row pitch ldq (a multiple of 8, >= Hq * D),
 * 16-byte aligned.  O: yt fp16, bf16 or f32 [T][Hq][D], row pitch ldo (a multiple
 * of 16 bytes), 16-byte aligned.  lse: f32 [T][Hq].
 * max_q: no sequence has more rows than this (device-checked, CQ_ERR_INDEX); it
 * picks the kernel, so give the batch's own largest n_b.
 * Shape rules: T >= 1, Hq a multiple of Hkv, Hq / Hkv <= 64, 1 <= max_q,
 * T * Hq < 2^31, scale finite and > 0, window >= 0.
 * Arithmetic: products of fp16 operands in f32: queries as given (bf16 queries to
 * fp16 behind a per-row power of two, exact for every value within 2^27 of the
 * row's largest), codes exactly, softmax weights times their value block's scale as
 * one fp16 term for 16-bit outputs (11 bits) and as two for f32 outputs (22 bits), in
 * both cases to 2^-35 of the row's largest such product; tokens that a row does not
 * see, or that have no weight, do not enter, whatever their scale; maxima, sums,
 * scores and accumulators in f32; one rounding to yt.  The tensor cores truncate as
 * they accumulate, so accumulators are added up in windows: f32 outputs lose at most
 * 5e-6 of sums of one sign to that (a few 1e-7 mostly), 16-bit ones 7e-5, whatever
 * the length.  Results do not depend on timing: the same call gives the same bits.
 * Workspace: cq_attn_kv8_workspace_bytes(...) bytes, 256-byte aligned; a buffer for
 * the largest T, B and max_q serves every call with smaller ones.
 * ------------------------------------------------------------------------- */
size_t cq_attn_kv8_workspace_bytes(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q);
cq_status cq_attn_kv8(const void* Q, int xt, int64_t T, int64_t Hq, int64_t ldq, const cq_kv8_cache* cache,
                      const int32_t* q_start, const int32_t* lens, int64_t max_q, float scale, int causal,
                      int64_t window, void* O, int yt, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                      void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CQ_KV8_H */
