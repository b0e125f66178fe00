// Many query rows, with a mask.
#include "kv8_tiles.cuh"

namespace cq {
namespace kv8 {

cudaError_t launch_tiles_tree(const AttnArgs& a, cudaStream_t s) { return run_tiles<true>(a, s); }

}  // namespace kv8
}  // namespace cq
