// Chunk attention, head_dim 64 (tq_chunk_tc.cuh).
#include "tq_chunk_tc.cuh"

namespace tq {
namespace ck {

cudaError_t launch_d64(const Args& a, int vb, int sm_count, cudaStream_t s) { return launch_d<64>(a, vb, sm_count, s); }
cudaError_t launch_join64(const Args& a, int sm_count, cudaStream_t s) { return launch_join<64>(a, sm_count, s); }

}  // namespace ck
}  // namespace tq
