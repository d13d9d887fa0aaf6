// cache_mma_int8.cu -- the tensor-core attention over int8 caches.
#include "cache_mma.cuh"

namespace attn {
namespace cache {

cudaError_t launch_mma_int8(const FwdParams &p, int dtype, cudaStream_t st) {
  return launch_kind<ATTN_CACHE_INT8>(p, dtype, st);
}

}  // namespace cache
}  // namespace attn
