// Chunk attention of few rows, head_dim 256 (tq_chunk_few.cuh).
#include "tq_chunk_few.cuh"

namespace tq {
namespace ck {

cudaError_t launch_few256(const Args& a, int, int vb, int sm_count, cudaStream_t s) {
  return few::launch_v<256, 1>(a, vb, sm_count, s);
}

}  // namespace ck
}  // namespace tq
