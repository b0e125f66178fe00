// 17 to 32 query rows, with a mask.
#include "kv8_narrow.cuh"

namespace cq {
namespace kv8 {

cudaError_t launch_narrow_tree(const AttnArgs& a, cudaStream_t s) { return run_narrow<true>(a, s); }

}  // namespace kv8
}  // namespace cq
