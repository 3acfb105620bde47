// Internal interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Not installed; not part of the ABI.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <functional>
#include <new>
#include <utility>

#include "../../include/pa.h"

// A checked call, kept to be launched again (pa_prepare_*, pa_run).
struct pa_prepared {
  int device;
  std::function<cudaError_t(cudaStream_t)> launch;
};

namespace pa {

// Changed scores (biased decode and prefill): s = softcap * tanh(scale q.k /
// softcap) (softcap > 0), minus slopes[h] * distance (slopes non-null), over
// the last `window` positions (window > 0).
struct ScoreRule {
  const float* slopes;  // [Hq] fp32
  float softcap;
  int window;
  bool any() const { return slopes != nullptr || softcap > 0.f || window > 0; }
};

// The rule for contexts of up to `capacity` tokens: a window of that many hides
// nothing, and without it no position of the kernels' arithmetic passes 32 bits.
inline ScoreRule within_capacity(ScoreRule r, int64_t capacity) {
  if (r.window >= capacity) r.window = 0;
  return r;
}

// Whether a rule's values make sense beside the score scale (api.cu).
bool score_rule_ok(const ScoreRule& r, float scale);

// The 4-bit split-K step of 128-dim heads in groups of up to 4 takes four blocks at a
// time, three CTAs an SM, from partitions of this many tokens on (launch_decode_int4;
// the partition chooser counts with it).
constexpr int kLongPartition4 = 4096;

// Arguments of the decode kernels (plain and split-K).  Pointers are device
// pointers, already validated on the host.
struct DecodeParams {
  __nv_bfloat16* out;  // pa_decode: [B, Hq, D]
  float* ws_o;         // split-K: [B, Hq, max_partitions, D]
  float* ws_m;         // split-K: [B, Hq, max_partitions]
  float* ws_l;         // split-K: [B, Hq, max_partitions]
  const __nv_bfloat16* q;
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  const int8_t* k8;        // int8 cache: codes [NB, Hkv, bs, D] (null for a bf16 cache)
  const int8_t* v8;
  const uint8_t* k4;       // 4-bit cache: tiles of codes and parameters (int4_row.cuh)
  const uint8_t* v4;
  const float* k_scales;   // int8 / fp8 cache: one scale per (block, head, token)
  const float* v_scales;
  int fp8;                 // 1-byte cache: codes are FP8 (E4M3), not INT8
  const int32_t* block_tables;
  const int32_t* context_lens;
  unsigned* err;
  int max_blocks_per_seq;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int num_blocks;
  int max_partitions;    // split-K only
  int partition_blocks;  // split-K only: blocks per partition
  float scale_log2;      // scale * log2(e): scores are kept in base-2 units
  // Fused decode step (pa_decode_step*), null when off.  The pools above are
  // then written as well (the CTA reading each new token's position writes
  // that token's K and V rows first).
  const __nv_bfloat16* new_key;    // [B, Hkv, D]: each sequence's new token
  const __nv_bfloat16* new_value;
  const int64_t* slot_mapping;     // [B]: the slot of position context_lens[b] - 1, or < 0
  unsigned* counters;              // split-K: [B, Hkv] arrivals; the last CTA merges
  // split-K, optional: the order in which the (sequence, partition) items run,
  // a permutation of [0, B * max_partitions) (item = part * B + b); null: grid order
  const int32_t* order;
  // Tables, lengths, order and pools are not written by the preceding kernel:
  // they may be read before waiting for it (programmatic dependent launch).
  int early_read;
  // split-K: partitions below first_partition are not computed here (a
  // shared prefix's prefix_blocks blocks, computed by launch_prefix_partials,
  // which also checks that every sequence holds them); the others hold
  // partition_blocks blocks each from block prefix_blocks on.
  int first_partition;
  int prefix_blocks;
  ScoreRule rule;        // RULE kernels only
};

struct ReduceParams {
  __nv_bfloat16* out;
  const float* ws_o;
  const float* ws_m;
  const float* ws_l;
  const int32_t* context_lens;
  unsigned* err;
  int num_seqs;
  int num_q_heads;
  int max_partitions;
  int partition_size;
  int window;            // > 0: the partitions cover the blocks of the last `window` tokens
};

struct CacheWriteParams {
  const __nv_bfloat16* key;
  const __nv_bfloat16* value;
  __nv_bfloat16* k_cache;
  __nv_bfloat16* v_cache;
  const int64_t* slot_mapping;
  unsigned* err;
  int num_tokens;
  int num_kv_heads;
  int head_dim;
  int block_size;
  int64_t num_slots;  // num_blocks * block_size
  int8_t* k8;         // int8 / fp8 cache (null for bf16): codes [NB, Hkv, bs, D]
  int8_t* v8;
  float* k_scales;    // [NB, Hkv, bs]
  float* v_scales;
  int fp8;            // codes are FP8 (E4M3), not INT8
};

// Rotary embedding + cache write (rope_append.cu).  Also the plain 4-bit
// cache write: no q, rotary_dim 0, positions and cos_sin null.
struct RopeAppendParams {
  __nv_bfloat16* q_out;           // [T, Hq, D]
  const __nv_bfloat16* q;         // [T] rows of Hq * D at q_stride
  const __nv_bfloat16* key;       // [T] rows of Hkv * D at key_stride
  const __nv_bfloat16* value;
  int64_t q_stride, key_stride, value_stride;  // elements from token to token
  __nv_bfloat16* k_cache;         // kind 0: bf16 pools
  __nv_bfloat16* v_cache;
  int8_t* k8;                     // kinds 1 (INT8), 2 (FP8): codes and scales
  int8_t* v8;
  float* k_scales;
  float* v_scales;
  uint8_t* k4;                    // kind 3: 4-bit tiles (int4_row.cuh)
  uint8_t* v4;
  const int64_t* slot_mapping;
  const int32_t* positions;
  const float* cos_sin;           // [max_position, R]: R / 2 cosines, R / 2 sines
  unsigned* err;
  int64_t num_slots;
  int kind;
  int max_position;
  int rotary_dim;
  int interleaved;
  int num_tokens;
  int num_q_heads;
  int num_kv_heads;
  int block_size;
  int row_slots;                  // thread groups per token (set by the launcher)
};

inline bool aligned_ptr(const void* p, uintptr_t a) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % a == 0;
}

inline bool ranges_meet(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + static_cast<uintptr_t>(b_bytes) &&
         y < x + static_cast<uintptr_t>(a_bytes);
}

// Whether rows of two tensors of one shape, `rows` of row_bytes, row_stride apart, share
// bytes.  (Rows may alternate, as views of one tensor.)
inline bool rows_meet(const void* a, const void* b, int64_t rows, int64_t row_bytes,
                      int64_t row_stride) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const uintptr_t apart = x < y ? y - x : x - y;
  const uintptr_t row = static_cast<uintptr_t>(row_bytes);
  const uintptr_t stride = static_cast<uintptr_t>(row_stride);
  if (apart >= static_cast<uintptr_t>(rows - 1) * stride + row) return false;
  const uintptr_t past = apart % stride;  // into a row's stride
  const bool last = apart / stride == static_cast<uintptr_t>(rows - 1);
  return past < row || (!last && stride - past < row);
}

// Positions of a cache read back (read_cache.cu).
struct ReadCacheParams {
  __nv_bfloat16* k_out;           // rows of Hkv * D at out_stride, or (slots) a bf16 pool
  __nv_bfloat16* v_out;
  const void* k_cache;            // kind 0 bf16, 1 INT8, 2 FP8, 3 4-bit tiles
  const void* v_cache;
  const float* k_scales;
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* first;           // [B] first position read (null: 0)
  const int32_t* row_start;       // [B + 1]
  const int64_t* slots;           // [T] slots of the bf16 pool (null: rows)
  unsigned* err;
  int64_t out_stride;
  int64_t num_out_slots;
  int64_t total_rows;
  int kind;
  int max_rows;
  int max_blocks_per_seq;
  int num_kv_heads;
  int num_blocks;
};

// States reordered in place (reorder_states.cu), up to kReorderMaxTensors a launch.
constexpr int kReorderMaxTensors = 64;
constexpr int kReorderMaxBeams = 32;
struct ReorderParams {
  void* states[kReorderMaxTensors];
  const int32_t* parents;  // [groups * beams]
  unsigned* err;
  int64_t row_bytes;
  int64_t row_stride;      // bytes
  int beams;
  int chunk;               // bytes of a row that a CTA moves (set by the launcher)
};

// Beam search's selection (beam_select.cu).
constexpr int kBeamMaxBeams = 32;
constexpr int kBeamMaxKeep = 64;
constexpr int kBeamMaxVocab = 1 << 27;
struct BeamParams {
  float* out_scores;       // [searches, keep]
  int32_t* out_parents;
  int32_t* out_tokens;
  uint8_t* out_finished;   // may be null
  const void* logits;      // [searches * beams] rows of vocab at row_stride
  const float* scores;     // [searches * beams]
  const uint8_t* finished; // may be null
  uint64_t* ws_keys;       // [searches * beams, parts, keep]
  float2* ws_sums;         // [searches * beams, parts]: maximum, sum of exp
  unsigned* counters;      // [searches]
  unsigned* err;
  int64_t row_stride;      // elements
  int searches, beams, vocab, keep, eos, in_place;
  int parts;
  int part_len;            // (set by the launcher)
  int groups;              // (set by the launcher)
};

// Pools of up to kCopyMaxLayers layers go to one copy_blocks launch.
constexpr int kCopyMaxLayers = 64;

struct CopyBlocksParams {
  void* k_caches[kCopyMaxLayers];
  void* v_caches[kCopyMaxLayers];
  const int64_t* block_mapping;  // [num_pairs, 2]: (src, dst)
  unsigned* err;
  int64_t block_bytes;  // Hkv * bs * D * 2
  int64_t num_blocks;
};

// Shapes with a compiled decode kernel.
bool decode_shape_supported(int head_dim, int group, int block_size);

cudaError_t launch_decode(const DecodeParams& p, int head_dim, int group, bool split,
                          cudaStream_t stream);
// The same over a 4-bit cache, and over a bf16 cache with changed scores.
cudaError_t launch_decode_int4(const DecodeParams& p, int head_dim, int group, bool split,
                               cudaStream_t stream);
cudaError_t launch_decode_biased(const DecodeParams& p, int head_dim, int group, bool split,
                                 cudaStream_t stream);
cudaError_t launch_splitk_reduce(const ReduceParams& p, int head_dim, cudaStream_t stream);
// prefill.cu: the split-K partials of a decode batch's queries over a shared
// prefix, partitions [0, splits) of split_blocks blocks each (head_dim 128);
// sets PA_DEVERR_PREFIX for a sequence not holding the prefix's blocks or not
// going past them.
cudaError_t launch_prefix_partials(const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int max_blocks_per_seq,
                                   const int32_t* context_lens, int num_seqs, int num_q_heads,
                                   int num_kv_heads, int num_blocks, float scale,
                                   int split_blocks, int splits, float* ws_o, float* ws_m,
                                   float* ws_l, int max_partitions, unsigned* err,
                                   cudaStream_t stream);
cudaError_t launch_reshape_and_cache(const CacheWriteParams& p, cudaStream_t stream);
cudaError_t launch_reshape_and_cache_int8(const CacheWriteParams& p, cudaStream_t stream);
cudaError_t launch_rope_append(const RopeAppendParams& p, int head_dim, cudaStream_t stream);
cudaError_t launch_read_cache(const ReadCacheParams& p, int head_dim, int num_seqs,
                              cudaStream_t stream);
// vec: bytes of one access, 1, 2, 4 or 16.
cudaError_t launch_reorder_states(ReorderParams p, int groups, int tensors, int vec,
                                  cudaStream_t stream);
// Parts that a row of logits is cut into (dtype 0 bf16, 1 fp16, 2 fp32).
int beam_parts(int rows, int vocab, int dtype);
cudaError_t launch_beam_select(BeamParams p, int dtype, cudaStream_t stream);
cudaError_t launch_copy_blocks(const CopyBlocksParams& p, int num_pairs, int num_layers,
                               cudaStream_t stream);

// The driver's tensor-map encoder (cuTensorMapEncodeTiled), or nullptr (prefill.cu).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Address of the current device's error word (device memory), or nullptr.
unsigned* device_error_word();

// Records e as the calling thread's last CUDA error (pa_last_cuda_error) and
// returns PA_ERR_CUDA.
pa_status cuda_fail(cudaError_t e);

// A checked call's end: launched on `stream`, or (keep non-null) kept.
template <typename Launch>
pa_status launch_or_keep(Launch&& launch, pa_prepared** keep, pa_stream_t stream) {
  if (!keep) {
    const cudaError_t e = launch(reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e);
  }
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  try {
    *keep = new pa_prepared{dev, std::forward<Launch>(launch)};
  } catch (const std::bad_alloc&) {
    return PA_ERR_INVALID_ARG;
  }
  return PA_OK;
}
// The same for a call with nothing to do.
inline pa_status nothing_to_do(pa_prepared** keep) {
  return launch_or_keep([](cudaStream_t) { return cudaSuccess; }, keep, nullptr);
}

}  // namespace pa
