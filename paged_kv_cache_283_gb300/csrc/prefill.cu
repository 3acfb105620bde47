// Paged prefill on the tensor cores: the kernel (prefill_kernel.cuh) without
// changed scores, the shared-prefix partials, and the C entry points.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "../../include/pa.h"
#include "device.cuh"
#include "internal.h"
#include "prefill_kernel.cuh"

namespace pa {

// ---- host side -------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

namespace {

// K or V pool as a 2-D bf16 tensor [num_blocks * Hkv * 16 rows][128], boxes of
// 16 rows x 64 columns, 128-byte swizzle.
bool encode_pool_map(CUtensorMap* map, const void* base, int64_t rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * 2};
  const cuuint32_t box[2] = {64, kBS};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// q as a 3-D bf16 tensor [T][Hq][128], boxes of (128 / G tokens) x G heads x
// 64 columns, 128-byte swizzle: one box is one 64-column half of a CTA's rows.
bool encode_q_map(CUtensorMap* map, const void* base, int total_q, int num_q_heads, int group) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(num_q_heads),
                              static_cast<cuuint64_t>(total_q)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kD) * 2,
                                 static_cast<cuuint64_t>(num_q_heads) * kD * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group),
                             static_cast<cuuint32_t>(kRows / group)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

bool aligned16(const void* ptr) { return ptr && (reinterpret_cast<uintptr_t>(ptr) & 15) == 0; }

}  // namespace

// The shared-prefix partials of a decode batch (see PrefillParams): grid
// (query tiles, KV heads, splits).  Arguments checked by the caller.
cudaError_t launch_prefix_partials(const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_tables, int max_blocks_per_seq,
                                   const int32_t* context_lens, int num_seqs, int num_q_heads,
                                   int num_kv_heads, int num_blocks, float scale,
                                   int split_blocks, int splits, float* ws_o, float* ws_m,
                                   float* ws_l, int max_partitions, unsigned* err,
                                   cudaStream_t stream) {
  const int group = num_q_heads / num_kv_heads;
  const int64_t rows = static_cast<int64_t>(num_blocks) * num_kv_heads * kBS;
  CUtensorMap tq, tk, tv;
  if (!encode_q_map(&tq, q, num_seqs, num_q_heads, group) ||
      !encode_pool_map(&tk, k_cache, rows) || !encode_pool_map(&tv, v_cache, rows))
    return cudaErrorInvalidValue;
  PrefillParams p{};
  p.block_tables = block_tables;
  p.err = err;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.total_q = num_seqs;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.split_blocks = split_blocks;
  p.ws_o = ws_o;
  p.ws_m = ws_m;
  p.ws_l = ws_l;
  p.max_partitions = max_partitions;
  p.context_lens = context_lens;
  switch (group) {
    case 1: return launch_prefill_g<1>(tq, tk, tv, p, num_seqs, splits, stream);
    case 2: return launch_prefill_g<2>(tq, tk, tv, p, num_seqs, splits, stream);
    case 4: return launch_prefill_g<4>(tq, tk, tv, p, num_seqs, splits, stream);
    default: return launch_prefill_g<8>(tq, tk, tv, p, num_seqs, splits, stream);
  }
}

}  // namespace pa

extern "C" int pa_prefill_supported(int head_dim, int group, int block_size) {
  return head_dim == 128 && block_size == 16 && (group == 1 || group == 2 || group == 4 ||
                                                  group == 8);
}

namespace {

// pa_prefill and pa_prefill_biased (rule non-null).
pa_status prefill_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* context_lens, const int32_t* query_start_loc,
                       int max_query_len, int num_seqs, int total_query_tokens, int num_q_heads,
                       int num_kv_heads, int head_dim, int block_size, int num_blocks,
                       float scale, const pa::ScoreRule* rule, const int32_t* prefix_lens,
                       pa_stream_t stream, pa_prepared** keep = nullptr) {
  using namespace pa;
  if (num_seqs < 0 || max_query_len < 0 || total_query_tokens < 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0 || !(scale > 0.f) || num_seqs > 65535)
    return PA_ERR_INVALID_ARG;
  if (rule && !score_rule_ok(*rule, scale)) return PA_ERR_INVALID_ARG;
  const int group = num_q_heads / num_kv_heads;
  if (!pa_prefill_supported(head_dim, group, block_size)) return PA_ERR_UNSUPPORTED_SHAPE;
  if (num_seqs == 0 || max_query_len == 0 || total_query_tokens == 0)
    return keep ? nothing_to_do(keep) : PA_OK;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !block_tables || !context_lens || !query_start_loc)
    return PA_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(num_blocks) * num_kv_heads * kBS;
  if (rows > 0x7fffffffll || static_cast<int64_t>(max_blocks_per_seq) * kBS > 0x7fffffffll)
    return PA_ERR_INVALID_ARG;
  CUtensorMap tq, tk, tv;
  if (!encode_q_map(&tq, q, total_query_tokens, num_q_heads, group) ||
      !encode_pool_map(&tk, k_cache, rows) || !encode_pool_map(&tv, v_cache, rows))
    return cuda_fail(cudaErrorInvalidValue);  // tensor-map encoding refused the pools
  PrefillParams p{};
  p.out = static_cast<__nv_bfloat16*>(out);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start_loc;
  p.err = device_error_word();
  if (!p.err) return cuda_fail(cudaGetLastError());
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.total_q = total_query_tokens;
  p.scale_log2 = scale * 1.4426950408889634f;
  if (rule) {
    p.rule = within_capacity(*rule, static_cast<int64_t>(max_blocks_per_seq) * block_size);
    p.prefix_lens = prefix_lens;
    p.cap_in = rule->softcap > 0.f ? scale / rule->softcap : 0.f;
  }
  const bool ruled = p.rule.any() || p.prefix_lens != nullptr;
  return launch_or_keep(
      [=](cudaStream_t s) {
        if (ruled) return launch_prefill_biased(tq, tk, tv, p, group, max_query_len, num_seqs, s);
        switch (group) {
          case 1: return launch_prefill_g<1>(tq, tk, tv, p, max_query_len, num_seqs, s);
          case 2: return launch_prefill_g<2>(tq, tk, tv, p, max_query_len, num_seqs, s);
          case 4: return launch_prefill_g<4>(tq, tk, tv, p, max_query_len, num_seqs, s);
          default: return launch_prefill_g<8>(tq, tk, tv, p, max_query_len, num_seqs, s);
        }
      },
      keep, stream);
}

}  // namespace

extern "C" pa_status pa_prefill(void* out, const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_tables, int max_blocks_per_seq,
                                const int32_t* context_lens, const int32_t* query_start_loc,
                                int max_query_len, int num_seqs, int total_query_tokens,
                                int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                int num_blocks, float scale, pa_stream_t stream) {
  return prefill_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start_loc, max_query_len, num_seqs, total_query_tokens, num_q_heads,
                      num_kv_heads, head_dim, block_size, num_blocks, scale, nullptr, nullptr,
                      stream);
}

extern "C" pa_status pa_prefill_biased(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* query_start_loc, int max_query_len, int num_seqs, int total_query_tokens,
    int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    float softcap, const float* alibi_slopes, int window, const int32_t* prefix_lens,
    pa_stream_t stream) {
  if (reinterpret_cast<uintptr_t>(prefix_lens) % 4 != 0) return PA_ERR_INVALID_ARG;
  const pa::ScoreRule rule{alibi_slopes, softcap, window};
  return prefill_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start_loc, max_query_len, num_seqs, total_query_tokens, num_q_heads,
                      num_kv_heads, head_dim, block_size, num_blocks, scale, &rule, prefix_lens,
                      stream);
}

extern "C" pa_status pa_prepare_prefill(
    pa_prepared** prepared, void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    const int32_t* query_start_loc, int max_query_len, int num_seqs, int total_query_tokens,
    int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    float softcap, const float* alibi_slopes, int window, const int32_t* prefix_lens) {
  if (!prepared || reinterpret_cast<uintptr_t>(prefix_lens) % 4 != 0) return PA_ERR_INVALID_ARG;
  *prepared = nullptr;
  const pa::ScoreRule rule{alibi_slopes, softcap, window};
  const bool ruled = softcap != 0.f || alibi_slopes != nullptr || window != 0 || prefix_lens;
  return prefill_impl(out, q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                      query_start_loc, max_query_len, num_seqs, total_query_tokens, num_q_heads,
                      num_kv_heads, head_dim, block_size, num_blocks, scale,
                      ruled ? &rule : nullptr, prefix_lens, nullptr, prepared);
}
