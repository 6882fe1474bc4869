// Chunk attention, head_dim 128 (tq_chunk_tc.cuh).
#include "tq_chunk_tc.cuh"

namespace tq {
namespace ck {

cudaError_t launch_d128(const Args& a, int vb, int sm_count, cudaStream_t s) { return launch_d<128>(a, vb, sm_count, s); }

}  // namespace ck
}  // namespace tq
