// Chunk attention over staged f8_block tiles, head_dim 128 (tq_chunk_staged.cuh).
#include "tq_chunk_staged.cuh"

namespace tq {
namespace ck {

cudaError_t launch_staged128(const Args& a, int sm_count, cudaStream_t s) { return staged::launch<128>(a, sm_count, s); }

}  // namespace ck
}  // namespace tq
