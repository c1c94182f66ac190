#include "chunk_common.cuh"
namespace qsa {
bool chunk_tc_supported(const ChunkArgs&) { return false; }
int chunk_tc_rows() { return 128; }
cudaError_t launch_chunk_attn_tc(const ChunkArgs&, const ChunkWs&, int, float, float, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace qsa
