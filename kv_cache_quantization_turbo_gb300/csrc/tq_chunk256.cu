// Chunk attention, head_dim 256 (tq_chunk_tc.cuh).
#include "tq_chunk_tc.cuh"

namespace tq {
namespace ck {

cudaError_t launch_d256(const Args& a, int vb, int sm_count, cudaStream_t s) { return launch_d<256>(a, vb, sm_count, s); }
cudaError_t launch_join256(const Args& a, int sm_count, cudaStream_t s) { return launch_join<256>(a, sm_count, s); }

}  // namespace ck
}  // namespace tq
