// The tile kernel over a list of entries (shared prefixes) for int8 codes
// (fa_cache_tile.cuh).
#include "fa_cache_tile.cuh"

namespace fa {

cudaError_t launch_shared_tiles_int8(const CacheAttnLaunch& a, const SharedGrid& g, int ctas, cudaStream_t stream) {
  return a.c.d == 128 ? launch_tiles<128, true, true>(a, g, ctas, stream) : launch_tiles<64, true, true>(a, g, ctas, stream);
}

}  // namespace fa
