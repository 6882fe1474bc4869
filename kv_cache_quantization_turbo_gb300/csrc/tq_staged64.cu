// Chunk attention over staged f8_block tiles, head_dim 64 (tq_chunk_staged.cuh).
#include "tq_chunk_staged.cuh"

namespace tq {
namespace ck {

cudaError_t launch_staged64(const Args& a, int sm_count, cudaStream_t s) { return staged::launch<64>(a, sm_count, s); }

}  // namespace ck
}  // namespace tq
