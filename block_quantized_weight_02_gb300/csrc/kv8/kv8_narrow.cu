// 17 to 32 query rows, without a mask.
#include "kv8_narrow.cuh"

namespace cq {
namespace kv8 {

bool narrow_serves(int64_t rows) { return rows <= NR; }
size_t narrow_workspace(int64_t T, int64_t G, int64_t D, int64_t B) {
    return (D == 128 ? sizeof(Space<128>) : sizeof(Space<64>)) + slots_of(T, G, B, NR) * sizeof(Item);
}
cudaError_t launch_narrow(const AttnArgs& a, cudaStream_t s) { return run_narrow<false>(a, s); }

}  // namespace kv8
}  // namespace cq
