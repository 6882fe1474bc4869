// Chunk attention of few rows, head_dim 128 (tq_chunk_few.cuh).
#include "tq_chunk_few.cuh"

namespace tq {
namespace ck {

cudaError_t launch_few128(const Args& a, int rows, int vb, int sm_count, cudaStream_t s) {
  return rows > 8 ? few::launch_v<128, 2>(a, vb, sm_count, s) : few::launch_v<128, 1>(a, vb, sm_count, s);
}

}  // namespace ck
}  // namespace tq
