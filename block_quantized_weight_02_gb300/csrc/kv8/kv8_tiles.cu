// Many query rows, without a mask.
#include "kv8_tiles.cuh"

namespace cq {
namespace kv8 {
namespace {

template <int D>
size_t space_bytes(int64_t T, int64_t G, int64_t B, int64_t max_q) {
    return max_q * G <= TM ? sizeof(Space<D, 1>) + slots_of(T, G, B, TM) * sizeof(Item)
                           : sizeof(Space<D, 2>) + slots_of(T, G, B, 2 * TM) * sizeof(Item);
}

}  // namespace

size_t tiles_workspace(int64_t T, int64_t G, int64_t D, int64_t B, int64_t max_q) {
    return D == 128 ? space_bytes<128>(T, G, B, max_q) : space_bytes<64>(T, G, B, max_q);
}
cudaError_t launch_tiles(const AttnArgs& a, cudaStream_t s) { return run_tiles<false>(a, s); }

}  // namespace kv8
}  // namespace cq
