// The evenly cut paged decode (decode_even.cuh) over a bf16 cache with changed
// scores.

#include "decode_even.cuh"

namespace pa {

cudaError_t launch_decode_biased_even(const DecodeParams& p, int head_dim, int group,
                                      cudaStream_t stream) {
  if (head_dim == 128) return launch_even_d<128, 0, true>(p, group, stream);
  if (head_dim == 64) return launch_even_d<64, 0, true>(p, group, stream);
  return cudaErrorInvalidValue;
}

size_t even_floats_biased(int head_dim, int group) {
  return head_dim == 128 ? even_floats_d<128, 0>(group) : even_floats_d<64, 0>(group);
}

}  // namespace pa
