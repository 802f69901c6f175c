#include "kda_packed.cuh"
namespace kda {
bool packed_chunk_shape(const PackedParams &, bool) { return false; }
bool packed_chunk_aligned(const PackedParams &) { return false; }
cudaError_t launch_packed_chunk(const PackedParams &, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t read_and_clear_packed_chunk_error(unsigned int *out) { *out = 0; return cudaSuccess; }
}  // namespace kda
