// Which attention kernel serves a call: by the most query rows (tokens x heads of a group) that a
// sequence has for one KV head.
// Up to 16 rows each warp makes its own products out of registers; the legacy tensor path's work grows
// with the rows.  24 sequences of 300 to 9000 tokens, 8 KV heads of 128 channels, bf16 out: 10 rows take
// 74 us there against 77 us in the narrow kernel, 15 rows 80 against 79; f32 out 89 against 98 and 97
// against 99; 16 rows of 3 x 110000 tokens 86 against 97 with f16 out, 105 against 122 with f32.  From 17
// rows on the products are tcgen05's: 20 rows took 108 us of the first kind against 81.  33 rows and more
// no longer fit the narrow kernel's 32 columns.
#include "kv8.cuh"

namespace cq {
namespace kv8 {

size_t attn_workspace(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q) {
    const int64_t G = Hq / Hkv, rows = std::min(max_q, T) * G;
    if (decode_serves(rows)) return decode_workspace(D);
    return narrow_serves(rows) ? narrow_workspace(T, G, D, B) : tiles_workspace(T, G, D, B, std::min(max_q, T));
}

// A batch with fewer rows a sequence may go to another kernel, whose partials are larger: what serves max_q is what any
// smaller one takes too (each kernel's own need grows with T, B and max_q).
size_t attn_workspace_upto(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q) {
    const int64_t G = Hq / Hkv, rows = std::min(max_q, T) * G;
    size_t n = attn_workspace(T, Hq, Hkv, D, B, max_q);
    for (int64_t q = 1; q * G <= 128 && q * G <= rows; ++q) n = std::max(n, attn_workspace(T, Hq, Hkv, D, B, q));
    return n;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.max_q * (a.Hq / a.c.Hkv);
    return decode_serves(rows) ? launch_decode(a, s) : narrow_serves(rows) ? launch_narrow(a, s) : launch_tiles(a, s);
}

}  // namespace kv8
}  // namespace cq
