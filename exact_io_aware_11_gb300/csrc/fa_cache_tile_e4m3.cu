// The tile kernel of the attention over the cache for e4m3 codes
// (fa_cache_tile.cuh).
#include "fa_cache_tile.cuh"

namespace fa {

cudaError_t launch_cache_attention_tiles_e4m3(const CacheAttnLaunch& a, const AttnGrid& g, int ctas, cudaStream_t stream) {
  return a.c.d == 128 ? launch_tiles<128, false>(a, g, ctas, stream) : launch_tiles<64, false>(a, g, ctas, stream);
}

}  // namespace fa
