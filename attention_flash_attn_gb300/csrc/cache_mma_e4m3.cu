// cache_mma_e4m3.cu -- the tensor-core attention over e4m3 caches.
#include "cache_mma.cuh"

namespace attn {
namespace cache {

cudaError_t launch_mma_e4m3(const FwdParams &p, int dtype, cudaStream_t st) {
  return launch_kind<ATTN_CACHE_E4M3>(p, dtype, st);
}

}  // namespace cache
}  // namespace attn
