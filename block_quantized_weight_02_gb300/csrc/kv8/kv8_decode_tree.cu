// Few query rows, with a mask (a translation unit of its own, so that the two compile side by side).
#include "kv8_decode.cuh"

namespace cq {
namespace kv8 {

cudaError_t launch_decode_tree(const AttnArgs& a, cudaStream_t s) { return run_decode<true>(a, s); }

}  // namespace kv8
}  // namespace cq
