// Which attention kernel serves a call: by the most query rows (tokens x heads of a group) that a
// sequence has for one KV head.
#include "kv8.cuh"

namespace cq {
namespace kv8 {

size_t attn_workspace(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q) {
    const int64_t G = Hq / Hkv, rows = std::min(max_q, T) * G;
    if (decode_serves(rows)) return decode_workspace(D);
    return narrow_serves(rows) ? narrow_workspace(T, G, D, B) : tiles_workspace(T, G, D, B, std::min(max_q, T));
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
    const int64_t rows = (int64_t)a.max_q * (a.Hq / a.c.Hkv);
    return decode_serves(rows) ? launch_decode(a, s) : narrow_serves(rows) ? launch_narrow(a, s) : launch_tiles(a, s);
}

}  // namespace kv8
}  // namespace cq
