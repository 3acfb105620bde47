// The paged decode kernel (decode_kernel.cuh) over a 4-bit cache.

#include "decode_kernel.cuh"

namespace pa {

cudaError_t launch_decode_int4(const DecodeParams& p, int head_dim, int group, bool split,
                               cudaStream_t stream) {
  if (head_dim == 128) return launch_decode_d<128, 3>(p, group, split, stream);
  if (head_dim == 64) return launch_decode_d<64, 3>(p, group, split, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
