// Few query rows, without a mask.
#include "kv8_decode.cuh"

namespace cq {
namespace kv8 {

bool decode_serves(int64_t rows) { return rows <= ROWS; }
size_t decode_workspace(int64_t D) { return D == 128 ? sizeof(Space<128>) : sizeof(Space<64>); }
cudaError_t launch_decode(const AttnArgs& a, cudaStream_t s) { return run_decode<false>(a, s); }

}  // namespace kv8
}  // namespace cq
