// Chunk attention over staged f8_block tiles, head_dim 256 (tq_chunk_staged.cuh).
#include "tq_chunk_staged.cuh"

namespace tq {
namespace ck {

cudaError_t launch_staged256(const Args& a, int sm_count, cudaStream_t s) { return staged::launch<256>(a, sm_count, s); }

}  // namespace ck
}  // namespace tq
