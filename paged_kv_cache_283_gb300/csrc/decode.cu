// The paged decode kernel (decode_kernel.cuh) over bf16, INT8 and FP8 caches.

#include "decode_kernel.cuh"

namespace pa {

bool decode_shape_supported(int head_dim, int group, int block_size) {
  return block_size == kBlockSize && (head_dim == 64 || head_dim == 128) &&
         (group == 2 || group == 4 || group == 8);
}

cudaError_t launch_decode(const DecodeParams& p, int head_dim, int group, bool split,
                          cudaStream_t stream) {
  const int q = p.k8 == nullptr ? 0 : (p.fp8 ? 2 : 1);
  if (head_dim == 128)
    return q == 0 ? launch_decode_d<128, 0>(p, group, split, stream)
                  : q == 1 ? launch_decode_d<128, 1>(p, group, split, stream)
                           : launch_decode_d<128, 2>(p, group, split, stream);
  if (head_dim == 64)
    return q == 0 ? launch_decode_d<64, 0>(p, group, split, stream)
                  : q == 1 ? launch_decode_d<64, 1>(p, group, split, stream)
                           : launch_decode_d<64, 2>(p, group, split, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
