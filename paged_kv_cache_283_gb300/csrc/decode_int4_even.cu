// The evenly cut paged decode (decode_even.cuh) over a 4-bit cache.

#include "decode_even.cuh"

namespace pa {

cudaError_t launch_decode_int4_even(const DecodeParams& p, int head_dim, int group,
                                    cudaStream_t stream) {
  if (head_dim == 128) return launch_even_d<128, 3, false>(p, group, stream);
  if (head_dim == 64) return launch_even_d<64, 3, false>(p, group, stream);
  return cudaErrorInvalidValue;
}

size_t even_floats_int4(int head_dim, int group) {
  return head_dim == 128 ? even_floats_d<128, 3>(group) : even_floats_d<64, 3>(group);
}

}  // namespace pa
