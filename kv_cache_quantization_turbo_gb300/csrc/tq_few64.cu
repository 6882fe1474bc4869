// Chunk attention of few rows, head_dim 64 (tq_chunk_few.cuh).
#include "tq_chunk_few.cuh"

namespace tq {
namespace ck {

cudaError_t launch_few64(const Args& a, int rows, int vb, int sm_count, cudaStream_t s) {
  return rows > 8 ? few::launch_v<64, 2>(a, vb, sm_count, s) : few::launch_v<64, 1>(a, vb, sm_count, s);
}

}  // namespace ck
}  // namespace tq
