// The paged decode kernel (decode_kernel.cuh) over a 4-bit cache.
//
// At 4.5 bits a value the bytes come in faster than a warp's steps take them: one of
// 32 tokens for 4 heads is some 350 instructions (Warp4), a third of them the
// unpacking of codes, in dependent chains (scores, maximum, weights, products) that
// three or four warps a scheduler do not hide: issue slots 43 to 52 % used, the tensor
// pipe 18 to 27 %.  Short batches are bounded by a launch's head and tail.  Measured, in us, with the time at the copy rate: 64 contexts of 128
// to 2016 tokens (32 query / 8 KV heads, D = 128) 19.9 (11.7); 256 of up to 4094
// with groups of 8 113.9 (91); 8 of up to 49,796 41.6 (33.0).

#include "decode_kernel.cuh"

namespace pa {

namespace {

// How many blocks a warp takes at a time.  More of them spread what a step costs
// whatever its tokens (waiting, the maximum over the rows, the ring), but hold more
// registers.  D = 128: two blocks with four CTAs an SM (<= 128 registers), or four
// with three (168).  In us, the best partition of each:
//                                        2 blocks  4 blocks
//   groups of 8: 256 x 4083 tokens          111.1     105.5
//                  8 x 43,311                55.2      48.2
//   groups of 4:  64 x 1991                  18.5      19.0
//                500 x 2034                 102.7     113.5
//                  8 x 49,796                54.0      42.4  (4096-token partitions)
//                 12 x 46,911, 4 KV heads    46.7      42.2  (4096)
//                  8 x 131,072              194.1     188.2  (5120)
// So groups of 8 take four, smaller ones from kLongPartition4 tokens on: there one wave of
// three CTAs an SM holds the launch, and its CTAs run long.  One block at a time
// with four CTAs: 22.0 us for the 64, 145 for the 256.  Eight warps a CTA, two CTAs
// an SM, are faster only for whole contexts in one wave (the 64: 17.0; 500: 128),
// which the launch cannot know from lengths in device memory.  D = 64 has the registers
// for four blocks and four CTAs: 64 x 15,763 66.7 us against 74.3 with two,
// 256 x 4094 68.1 against 76.7, 32 x 595 5.3 and 5.3.
// Partitions of up to this many tokens keep each of their warps below kSettleSteps
// steps of four blocks.
constexpr int kShortPartition = kSettleSteps * 4 * 4 * kBlockSize;

template <int D, int G>
cudaError_t launch_g(const DecodeParams& p, bool split, cudaStream_t stream) {
  if (!split) return launch_decode_t<D, G, false, 3, false, D == 64 ? 4 : 2, true>(p, stream);
  if (p.partition_blocks > kShortPartition / kBlockSize)
    return launch_decode_t<D, G, true, 3, false, 4, true>(p, stream);
  if constexpr (D == 128 && G < 8)
    if (p.partition_blocks < kLongPartition4 / kBlockSize)
      return launch_decode_t<D, G, true, 3, false, 2>(p, stream);
  return launch_decode_t<D, G, true, 3, false, 4>(p, stream);
}

template <int D>
cudaError_t launch_d(const DecodeParams& p, int group, bool split, cudaStream_t stream) {
  switch (group) {
    case 2: return launch_g<D, 2>(p, split, stream);
    case 4: return launch_g<D, 4>(p, split, stream);
    case 8: return launch_g<D, 8>(p, split, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_decode_int4(const DecodeParams& p, int head_dim, int group, bool split,
                               cudaStream_t stream) {
  if (head_dim == 128) return launch_d<128>(p, group, split, stream);
  if (head_dim == 64) return launch_d<64>(p, group, split, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
