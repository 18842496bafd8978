// The tile kernel of the attention over the cache for int8 codes
// (fa_cache_tile.cuh).
#include "fa_cache_tile.cuh"

namespace fa {

cudaError_t launch_cache_attention_tiles_int8(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  return a.c.d == 128 ? launch_tiles<128, true>(a, g, ctas, stream) : launch_tiles<64, true>(a, g, ctas, stream);
}

}  // namespace fa
