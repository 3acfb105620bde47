// The paged decode kernel (decode_kernel.cuh) over a bf16 cache with changed
// scores: capped, biased by distance, limited to a window.
//
// Bound by bytes, as without the change: 64 windows of 1024 tokens in contexts of
// up to 8192 (32 query / 8 KV heads, D = 128) 48.6 us with the window alone and
// with a cap (37.7 at the copy rate); contexts of up to 65,536 with a bias 64.8
// (62.2).  Groups of 8 at D = 128 (255 registers, two CTAs an SM) are bounded by their
// multiply-adds on the fp32 pipe: the 64 windows with 64 query heads 76.0, a bias over
// 64 contexts of up to 4096 131 (75).  Blocks before the window are not read, and the partitions start at the
// window's first block.

#include "decode_kernel.cuh"

namespace pa {

cudaError_t launch_decode_biased(const DecodeParams& p, int head_dim, int group, bool split,
                                 cudaStream_t stream) {
  if (head_dim == 128) return launch_decode_d<128, 0, true>(p, group, split, stream);
  if (head_dim == 64) return launch_decode_d<64, 0, true>(p, group, split, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
