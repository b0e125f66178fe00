// Which attention kernel serves a call.
#include "kv8.cuh"

namespace cq {
namespace kv8 {

size_t attn_workspace(int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t B, int64_t max_q) {
    const int64_t G = Hq / Hkv;
    max_q = std::min(max_q, T);
    return decode_serves(max_q * G) ? decode_workspace(D) : tiles_workspace(T, G, D, B, max_q);
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t s) {
    return decode_serves((int64_t)a.max_q * (a.Hq / a.c.Hkv)) ? launch_decode(a, s) : launch_tiles(a, s);
}

}  // namespace kv8
}  // namespace cq
