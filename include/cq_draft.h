/*
 * cq_draft -- a step of drafting over the 8-bit cache of cq_kv8.h: rotary
 * positions, appending rotated keys, attention for trees of drafted tokens, and the
 * check of drafted tokens against the target's probabilities (part of libcq.so;
 * conventions, status codes and error words as in cq.h, caches and ragged batches as
 * in cq_kv8.h).
 *
 * A tree of drafted tokens.  A sequence's rows of one step are the nodes of a tree:
 * its first row is the last token that stands, every other one a drafted token, after
 * its parent.  The tree is given by mask words [T][ldm]: bit i % 32 of word i / 32 of a
 * row is set where that row sees row i of its sequence (for a tree: its ancestors and
 * itself).  Words hold max_q bits at least: 32 * ldm >= max_q.  mask 4-byte aligned.
 */
#ifndef CQ_DRAFT_H
#define CQ_DRAFT_H

#include "cq_kv8.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------------
 * Rotary positions:  the pair (a, b) of channels at position p becomes
 *   (a cos t - b sin t, b cos t + a sin t) * mag,   t = p * freq[i],  i < rot / 2.
 * CQ_ROPE_HALF: pair i is channels i and i + rot/2; CQ_ROPE_PAIRS: 2i and 2i + 1.
 * Channels from rot on stay as they are.  Contexts beyond the trained one are a matter
 * of freq and mag (cq_rope_freqs).
 * Arithmetic: angles in 64-bit fixed point, exact to 2^-33 of a turn for every position;
 * cosines and sines in f32 (1 ulp; times mag one more rounding); a product each, then
 * their sum in f32; one rounding to yt.
 * Host descriptor (freq is a device pointer, 4-byte aligned).  rot: a multiple of 16,
 * 16 <= rot <= D.  mag finite.  Frequencies that are not finite, or 65536 and more in
 * size, give NaN.
 * ------------------------------------------------------------------------- */
enum { CQ_ROPE_HALF = 0, CQ_ROPE_PAIRS = 1 };
typedef struct {
    const float* freq;     /* [rot/2] radians per position */
    int64_t rot;           /* rotated channels of a head */
    int layout;            /* CQ_ROPE_HALF or CQ_ROPE_PAIRS */
    float mag;             /* factor on the rotated channels */
} cq_rope_spec;

/* X: xt fp16, bf16 or f32 [T][H][D], row pitch ldx elements (a multiple of 16 bytes, >= H * D);
 * Y likewise of type yt.  pos: int32 [T], any values.  Y may be X (same type and
 * pitch) but not overlap it otherwise (CQ_ERR_ARG).  X, Y 16-byte aligned.
 * Shape rules: T >= 1, H >= 1, D a multiple of 16 up to 1024, T * H < 2^31.  One launch. */
cq_status cq_rope(const void* X, int xt, int64_t T, int64_t H, int64_t D, int64_t ldx, const cq_rope_spec* rope,
                  const int32_t* pos, void* Y, int yt, int64_t ldy, void* stream);

/* Fills freq (HOST, [rot/2]) and *mag (HOST) for the angles base^(-2i/rot):
 *   CQ_ROPE_PLAIN   as they are.
 *   CQ_ROPE_LINEAR  divided by factor (positions squeezed into the trained range).
 *   CQ_ROPE_BASE    of the base that divides the slowest one by factor:
 *                   base * factor^(rot / (rot - 2)).
 *   CQ_ROPE_RAMP    divided by factor where a pair turns less than `low` times within
 *                   the trained context, kept where it turns more than `high` times, a
 *                   ramp in i between; mag = 0.1 ln(factor) + 1  ("YaRN").
 *   CQ_ROPE_BANDS   divided by factor where a turn takes more than trained / low
 *                   positions, kept where it takes less than trained / high, between
 *                   them blended by trained / turn.
 * base > 1; factor >= 1; low, high, trained > 0, low < high (the last two kinds only;
 * ignored by the others).  mag is 1 but for CQ_ROPE_RAMP. */
enum { CQ_ROPE_PLAIN = 0, CQ_ROPE_LINEAR = 1, CQ_ROPE_BASE = 2, CQ_ROPE_RAMP = 3, CQ_ROPE_BANDS = 4 };
cq_status cq_rope_freqs(int64_t rot, double base, int kind, double factor, double low, double high, double trained,
                        float* freq, float* mag);

/* ---------------------------------------------------------------------------
 * Write with rotation:  cq_kv8_write of keys that are rotated on the way, in f32
 * before they are rounded to codes.  pos: int32 [T], the rows' positions (drafted
 * siblings share one); NULL: a row's place in its sequence.  One launch.
 * ------------------------------------------------------------------------- */
cq_status cq_kv8_write_rope(const cq_kv8_cache* cache, const void* K, const void* V, int xt, int64_t T, int64_t ldk,
                            int64_t ldv, const int32_t* q_start, const int32_t* lens, const cq_rope_spec* rope,
                            const int32_t* pos, void* stream);

/* ---------------------------------------------------------------------------
 * Attention for drafted trees:  cq_attn_kv8 where row r of sequence b (n_b rows, lens[b]
 * tokens) sees every token before lens[b] - n_b and, of the last n_b tokens, those i
 * whose bit is set in mask row r (bits of tokens that are not there count for nothing).
 * A row that sees nothing gets O = 0 and lse = -inf.  Types, shape rules, workspace and
 * arithmetic are those of cq_attn_kv8.
 * ------------------------------------------------------------------------- */
cq_status cq_attn_kv8_tree(const void* Q, int xt, int64_t T, int64_t Hq, int64_t ldq, const cq_kv8_cache* cache,
                           const int32_t* q_start, const int32_t* lens, int64_t max_q, float scale, const uint32_t* mask,
                           int64_t ldm, void* O, int yt, int64_t ldo, float* lse, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * Check of drafted tokens.  P[r] are the target's probabilities of what follows row r,
 * tokens[r] is row r's token (a first row's is not read), u[r] its random number in [0, 1)
 * (less counts as 0, NaN falls).
 * A row's parent is the last row before it that its mask names (rows without one are
 * left out); mask NULL: a chain, each row after the one before it.
 * The walk begins at the first row, and at each row goes through its children in order:
 *   w = P[row], m = 1; child c with token x stands if
 *     u[c] * Q[row][x] * m < w(x)         (Q: tokens drawn from the draft's Q[row])
 *     u[c] * m < w(x)                     (Q NULL: tokens chosen, not drawn),
 *   and the walk goes on from c; else w becomes max(w - m Q[row], 0) and m its sum
 *   (Q NULL: w(x) becomes 0 and m is lessened by what it was, down to 0).
 * Where no child stands the next token is drawn from what w has become: the smallest x
 * with w(0) + .. + w(x) > u_last[b] * (the sum of w), or the last x with w(x) > 0; if w is
 * nothing, from P[row], and if that is nothing as well the token is -1.  So every
 * token is distributed as the target's, if u and u_last are independent and uniform.
 * Negative entries of P and Q and NaN count as 0; a row with an infinite entry leaves its
 * sequence's outputs unspecified.  Rows of P are taken to sum to 1 and are not normalised.
 * out [B][ldo]: the tokens that stand, then the drawn one; path [B][ldo]: the rows that
 * stand, the first one included; the rest of a row's first max_q entries is -1.  count [B]: drafted tokens that
 * stand (a sequence without rows: 0, and -1 throughout).
 * P, Q: pt fp16, bf16 or f32 [T][V], row pitches ldp, ldq elements (multiples of 16
 * bytes, >= V), 16-byte aligned.  All else int32 or f32, 4-byte aligned.
 * Arithmetic, whatever the type: comparisons as in 64 bits, entries of w exactly after one
 * rejection and to 2^-45 of the larger of P and what was taken off after more, sums of them
 * to 2^-40.  The same call gives the same bits.
 * Shape rules: T >= 1, 1 <= V < 2^30, 1 <= B <= 65536, 1 <= max_q <= 1024, ldo >= max_q;
 * no sequence has more than max_q rows.  One launch, no workspace.
 * Device-detected (CQ_ERR_INDEX): a q_start that descends or leaves [0, T], more than
 * max_q rows, a token outside [0, V) (that sequence's outputs are unspecified).
 * ------------------------------------------------------------------------- */
cq_status cq_verify(const void* P, int pt, int64_t T, int64_t V, int64_t ldp, const void* Q, int64_t ldq,
                    const int32_t* tokens, const uint32_t* mask, int64_t ldm, const int32_t* q_start, int64_t B,
                    int64_t max_q, const float* u, const float* u_last, int32_t* out, int32_t* path, int64_t ldo,
                    int32_t* count, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CQ_DRAFT_H */
