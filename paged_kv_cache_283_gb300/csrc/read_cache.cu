// Positions of a paged cache read back as bf16 rows (pa_read_cache*): the
// inverse of the cache writes, for every cache type.  What the chunked prefill
// of a prompt whose earlier tokens lie in an INT8, FP8 or 4-bit cache reads,
// and what a cache is exported or re-quantised from.
//
// Value of a row: the bf16 value itself; INT8 / FP8: code * scale of the (token,
// KV head) row; 4-bit: offset + scale * code of the row's 64-dim group; taken in
// fp32 and rounded to bf16 once.
//
// Bytes bound it.  One warp per (16-token block, KV head): a block's K tile and
// V tile are runs of memory, loaded in 16-byte pieces that are all in flight
// before the first is used; 4-bit tiles and V tiles, whose codes lie transposed
// for the decode's tensor-core steps, go through shared memory (a warp's own
// part: no barrier wider than the warp), from which a lane reads the 32-bit
// words that hold four tokens of a dim, so that each lane ends with runs of 8 or
// 16 dims of four tokens and stores them in 16-byte pieces.  Neighbouring warps
// take neighbouring heads: their rows are contiguous in a [T, Hkv, D] output.
// 16 prefixes of 512 to 8192 tokens (8 heads of 128): a 4-bit cache 61.7 us, 0.96 of the
// copy rate; INT8 and FP8 69, bf16 86, each some 2 us more into slots.  Three short
// ranges of an INT8 cache 3.0 us: round trips to memory (range, block id, then tile and
// slots together).

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache_row.cuh"
#include "device.cuh"
#include "int4_row.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kWarps = 4;
constexpr int kBS = 16;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte `i` of w as an exact float: 2^23 + byte, less 2^23 (and less 128, the
// offset of INT8 V codes, where `bias` is 2^23 + 128).
__device__ __forceinline__ float byte_minus(uint32_t w, int i, float bias) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7650 + i)) - bias;
}

// Where a warp's rows go: row r of the call, of KV head h.
template <int D>
struct Rows {
  const ReadCacheParams& p;
  int h, t_lo, t_hi;  // tokens [t_lo, t_hi) of the block are asked for
  int64_t row0;       // row of token 0 of the block (may be before the first row)
  int64_t slot_at;    // with slots: the offset of token lane % 16's row

  // The slots of the block's rows, a lane each, fetched with its tiles.
  __device__ __forceinline__ void read_slots(int lane) {
    slot_at = -1;
    const int t = lane % kBS;
    if (!p.slots || t < t_lo || t >= t_hi) return;
    const int64_t s = load_after_wait(p.slots + row0 + t);
    if (s < 0) return;
    if (s >= p.num_out_slots)
      raise_error(p.err, PA_DEVERR_SLOT);
    else
      slot_at = ((s / kBS * p.num_kv_heads + h) * kBS + s % kBS) * D;
  }
  // Element offset of token t's row in the outputs, or -1: not asked for, or no slot.
  // (By the whole warp.)
  __device__ __forceinline__ int64_t at(int t) const {
    if (p.slots) return __shfl_sync(kFullMask, slot_at, t);
    return t < t_lo || t >= t_hi ? -1 : (row0 + t) * p.out_stride + h * D;
  }
};

// kind 0: bf16, 1: INT8, 2: FP8, 3: 4-bit.  grid (items / kWarps, sequences):
// item = block of the sequence's range * Hkv + head.
template <int D, int KIND>
__global__ void __launch_bounds__(32 * kWarps) read_cache_kernel(const ReadCacheParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  const int64_t r0 = load_after_wait(p.row_start + b), r1 = load_after_wait(p.row_start + b + 1);
  const int64_t first = p.first ? load_after_wait(p.first + b) : 0;
  if (r0 < 0 || r1 < r0 || r1 > p.total_rows || first < 0 ||
      first + (r1 - r0) > static_cast<int64_t>(p.max_blocks_per_seq) * kBS) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
    return;
  }
  // rows past max_rows are not read (the host sized the grid by it)
  const int64_t n = min(r1 - r0, static_cast<int64_t>(p.max_rows));
  const int item = blockIdx.x * kWarps + warp;
  const int blk = item / p.num_kv_heads, h = item - blk * p.num_kv_heads;
  const int tb = static_cast<int>(first / kBS) + blk;  // block of the sequence
  const int64_t pos0 = static_cast<int64_t>(tb) * kBS;
  if (n <= 0 || pos0 >= first + n) return;
  if (lane == 0 && blk == 0 && h == 0 && n < r1 - r0) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
  int id = load_after_wait(p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq + tb);
  if (id < 0 || id >= p.num_blocks) {  // never dereferenced: block 0 is read instead
    if (lane == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
    id = 0;
  }
  const int64_t tile = static_cast<int64_t>(id) * p.num_kv_heads + h;
  Rows<D> rows{p, h, static_cast<int>(max(first - pos0, static_cast<int64_t>(0))),
               static_cast<int>(min(first + n - pos0, static_cast<int64_t>(kBS))),
               r0 + pos0 - first, -1};
  constexpr int LR = D / 8;        // lanes that hold a row, 8 dims each
  constexpr int RI = 32 / LR;      // rows of one pass of the warp
  constexpr int NI = kBS / RI;     // passes over a tile
  const int j8 = lane % LR * 8, tr = lane / LR;
  auto put = [](__nv_bfloat16* out, int64_t at, const uint4& v) {
    *reinterpret_cast<uint4*>(out + at) = v;
  };

  if constexpr (KIND == 0) {
    const uint4* k = reinterpret_cast<const uint4*>(p.k_cache) + tile * (kBS * LR);
    const uint4* v = reinterpret_cast<const uint4*>(p.v_cache) + tile * (kBS * LR);
    uint4 kr[NI], vr[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      kr[i] = load_after_wait(k + i * 32 + lane);
      vr[i] = load_after_wait(v + i * 32 + lane);
    }
    rows.read_slots(lane);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t at = rows.at(i * RI + tr);
      if (at >= 0) {
        put(p.k_out, at + j8, kr[i]);
        put(p.v_out, at + j8, vr[i]);
      }
    }
  } else if constexpr (KIND == 3) {
    constexpr int TB = int4_tile_bytes(D), PIECES = TB / 16;
    constexpr int PL = (2 * PIECES + 31) / 32;  // pieces of both tiles per lane
    __shared__ uint4 buf[kWarps][2 * PIECES];
    const uint4* k = reinterpret_cast<const uint4*>(p.k_cache) + tile * PIECES;
    const uint4* v = reinterpret_cast<const uint4*>(p.v_cache) + tile * PIECES;
    uint4 w[PL];
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int c = i * 32 + lane;
      if (c < 2 * PIECES) w[i] = load_after_wait(c < PIECES ? k + c : v + (c - PIECES));
    }
    rows.read_slots(lane);
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int c = i * 32 + lane;
      if (c < 2 * PIECES) buf[warp][c] = w[i];
    }
    __syncwarp();
    const uint8_t* ks = reinterpret_cast<const uint8_t*>(buf[warp]);
    const uint8_t* vs = ks + TB;
    constexpr int NG = D / kInt4Group;
    auto value = [](uint32_t code, uint32_t par) {  // offset + scale * code (exact product)
      return fmaf(__uint_as_float(par & 0xffff0000u), static_cast<float>(code),
                  __uint_as_float(par << 16));
    };
    // K: 8 dims of a row are 8 nibbles of one word
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int t = i * RI + tr;
      const uint32_t c = *reinterpret_cast<const uint32_t*>(ks + t * (D / 2) +
                                                            k4_nibble<D>(j8) / 2);
      const uint32_t par =
          *reinterpret_cast<const uint32_t*>(ks + 8 * D + 4 * (t * NG + j8 / kInt4Group));
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = pack_bf16(value((c >> (8 * e)) & 15u, par), value((c >> (8 * e + 4)) & 15u, par));
      const int64_t at = rows.at(t);
      if (at >= 0) put(p.k_out, at + j8, make_uint4(o[0], o[1], o[2], o[3]));
    }
    // V: a word holds dims 16 c + i (low nibbles) and 16 c + i + 8 of four tokens
    // (bytes 0 .. 3: 2 tig, 2 tig + 8, 2 tig + 1, 2 tig + 9)
    const int tig = lane & 3, c = lane >> 2;
    int64_t to[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = rows.at(2 * tig + (e >> 1) + 8 * (e & 1));
    if (c < D / 16) {
      uint32_t word[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        word[i] = *reinterpret_cast<const uint32_t*>(vs + v4_byte<D>(2 * tig, c, i));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 2 * tig + (e >> 1) + 8 * (e & 1);
        const uint32_t par =
            *reinterpret_cast<const uint32_t*>(vs + 8 * D + 4 * (t * NG + c * 16 / kInt4Group));
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a = word[2 * i] >> (8 * e), d = word[2 * i + 1] >> (8 * e);
          lo[i] = pack_bf16(value(a & 15u, par), value(d & 15u, par));
          hi[i] = pack_bf16(value((a >> 4) & 15u, par), value((d >> 4) & 15u, par));
        }
        if (to[e] >= 0) {
          put(p.v_out, to[e] + 16 * c, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          put(p.v_out, to[e] + 16 * c + 8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
        }
      }
    }
  } else {
    constexpr int PL = kBS * D / 16 / 32;  // 16-byte pieces of a V tile per lane
    __shared__ uint4 buf[kWarps][kBS * D / 16];
    const uint2* k = reinterpret_cast<const uint2*>(p.k_cache) + tile * (kBS * LR);
    const uint4* v = reinterpret_cast<const uint4*>(p.v_cache) + tile * (kBS * D / 16);
    const float* ksc = p.k_scales + tile * kBS;
    const float* vsc = p.v_scales + tile * kBS;
    uint4 w[PL];
    uint2 kr[NI];
    float kscale[NI];
#pragma unroll
    for (int i = 0; i < PL; ++i) w[i] = load_after_wait(v + i * 32 + lane);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      kr[i] = load_after_wait(k + i * 32 + lane);
      kscale[i] = load_after_wait(ksc + i * RI + tr);
    }
    const int tig = lane & 3;
    float vscale[4];  // of tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9
#pragma unroll
    for (int e = 0; e < 4; ++e)
      vscale[e] = load_after_wait(vsc + 2 * tig + (e & 1) + 8 * (e >> 1));
    rows.read_slots(lane);
#pragma unroll
    for (int i = 0; i < PL; ++i) buf[warp][i * 32 + lane] = w[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t word = e < 2 ? kr[i].x : kr[i].y;
        float2 f;
        if constexpr (KIND == 2) {
          const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
              static_cast<__nv_fp8x2_storage_t>(word >> (16 * (e & 1))), __NV_E4M3);
          f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        } else {
          const uint32_t u = word ^ 0x80808080u;  // codes + 128
          f = make_float2(byte_minus(u, 2 * (e & 1), 8388736.f),
                          byte_minus(u, 2 * (e & 1) + 1, 8388736.f));
        }
        o[e] = pack_bf16(f.x * kscale[i], f.y * kscale[i]);
      }
      const int64_t at = rows.at(i * RI + tr);
      if (at >= 0) put(p.k_out, at + j8, make_uint4(o[0], o[1], o[2], o[3]));
    }
    const uint8_t* vs = reinterpret_cast<const uint8_t*>(buf[warp]);
    // a lane takes dims 8 u .. 8 u + 7 of its four tokens
#pragma unroll
    for (int u = lane >> 2; u < LR; u += 8) {
      uint32_t word[8];  // dim 8 u + i: bytes are the tokens of vscale
#pragma unroll
      for (int i = 0; i < 8; ++i)
        word[i] = *reinterpret_cast<const uint32_t*>(vs + v_tile_pos<D>(2 * tig, 8 * u + i));
      uint32_t o[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[2][4];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const uint32_t wd = word[2 * i + s];
          if constexpr (KIND == 2) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                  static_cast<__nv_fp8x2_storage_t>(wd >> (16 * e)), __NV_E4M3);
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
              x[s][2 * e] = f.x;
              x[s][2 * e + 1] = f.y;
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[s][e] = byte_minus(wd, e, 8388736.f);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e][i] = pack_bf16(x[0][e] * vscale[e], x[1][e] * vscale[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t at = rows.at(2 * tig + (e & 1) + 8 * (e >> 1));
        if (at >= 0) put(p.v_out, at + 8 * u, make_uint4(o[e][0], o[e][1], o[e][2], o[e][3]));
      }
    }
  }
}

template <int D>
cudaError_t launch(const ReadCacheParams& p, dim3 grid, cudaStream_t stream) {
  const dim3 block(32 * kWarps);
  switch (p.kind) {
    case 0: return launch_pdl(read_cache_kernel<D, 0>, grid, block, 0, stream, p);
    case 1: return launch_pdl(read_cache_kernel<D, 1>, grid, block, 0, stream, p);
    case 2: return launch_pdl(read_cache_kernel<D, 2>, grid, block, 0, stream, p);
    default: return launch_pdl(read_cache_kernel<D, 3>, grid, block, 0, stream, p);
  }
}

}  // namespace

cudaError_t launch_read_cache(const ReadCacheParams& p, int head_dim, int num_seqs,
                              cudaStream_t stream) {
  // a range of max_rows positions touches one block more where it starts inside one
  const int64_t blocks = (static_cast<int64_t>(p.max_rows) + kBS - 1) / kBS + (p.first ? 1 : 0);
  const int64_t items = blocks * p.num_kv_heads;
  const dim3 grid(static_cast<unsigned>((items + kWarps - 1) / kWarps), num_seqs);
  return head_dim == 64 ? launch<64>(p, grid, stream) : launch<128>(p, grid, stream);
}

namespace {

pa_status read_impl(int kv_kind, void* k_out, void* v_out, int64_t out_stride,
                    const void* k_cache, const void* v_cache, const float* k_scales,
                    const float* v_scales, const int32_t* block_tables, int max_blocks_per_seq,
                    const int32_t* first_positions, const int32_t* row_start_loc, int max_rows,
                    int num_seqs, int total_rows, const int64_t* slot_mapping,
                    int num_out_blocks, int num_kv_heads, int head_dim, int block_size,
                    int num_blocks, pa_stream_t stream, pa_prepared** keep) {
  using namespace pa;
  if (!(kv_kind == 4 || (kv_kind >= 0 && kv_kind <= 2)) || max_blocks_per_seq <= 0 ||
      max_rows < 0 || num_seqs < 0 || total_rows < 0 || num_kv_heads <= 0 || num_blocks <= 0 ||
      (slot_mapping && num_out_blocks <= 0))
    return PA_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || block_size != 16 || num_seqs > 65535)
    return PA_ERR_UNSUPPORTED_SHAPE;
  if (num_seqs == 0 || max_rows == 0 || total_rows == 0) return keep ? nothing_to_do(keep) : PA_OK;
  const bool scaled = kv_kind == 1 || kv_kind == 2;
  if (!aligned_ptr(k_out, 16) || !aligned_ptr(v_out, 16) || !aligned_ptr(k_cache, 16) ||
      !aligned_ptr(v_cache, 16) || !aligned_ptr(block_tables, 4) ||
      !aligned_ptr(row_start_loc, 4) || (first_positions && !aligned_ptr(first_positions, 4)) ||
      (slot_mapping && !aligned_ptr(slot_mapping, 8)) ||
      (scaled ? !aligned_ptr(k_scales, 16) || !aligned_ptr(v_scales, 16)
              : k_scales != nullptr || v_scales != nullptr))
    return PA_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (!slot_mapping && (out_stride < row || out_stride % 8 != 0 || out_stride >= (1ll << 30)))
    return PA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(max_blocks_per_seq) * kBS > 0x7fffffffll) return PA_ERR_INVALID_ARG;
  ReadCacheParams p{};
  p.max_rows = max_rows < total_rows ? max_rows : total_rows;
  if (static_cast<int64_t>(max_blocks_per_seq) * kBS < p.max_rows)
    p.max_rows = max_blocks_per_seq * kBS;
  // (an item's number stays within 31 bits)
  if ((static_cast<int64_t>(p.max_rows) / kBS + 2) * num_kv_heads > 0x7fffffffll - kWarps)
    return PA_ERR_UNSUPPORTED_SHAPE;
  // outputs that overlap the pools would be read while they are written
  const int64_t tile = kv_kind == 0 ? 2ll * kBS * head_dim
                       : kv_kind == 4 ? int4_tile_bytes(head_dim)
                                      : static_cast<int64_t>(kBS) * head_dim;
  const int64_t pool = tile * num_blocks * num_kv_heads;
  const int64_t written = slot_mapping ? 2 * kBS * row * num_out_blocks
                                       : 2 * ((total_rows - 1) * out_stride + row);
  const void* outs[2] = {k_out, v_out};
  const void* pools[2] = {k_cache, v_cache};
  for (const void* o : outs)
    for (const void* c : pools)
      if (ranges_meet(o, written, c, pool)) return PA_ERR_INVALID_ARG;
  // (K and V rows may alternate, as views of one tensor)
  if (slot_mapping ? ranges_meet(k_out, written, v_out, written)
                   : rows_meet(k_out, v_out, total_rows, 2 * row, 2 * out_stride))
    return PA_ERR_INVALID_ARG;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.block_tables = block_tables;
  p.first = first_positions;
  p.row_start = row_start_loc;
  p.slots = slot_mapping;
  p.err = device_error_word();
  if (!p.err) return cuda_fail(cudaGetLastError());
  p.out_stride = out_stride;
  p.num_out_slots = static_cast<int64_t>(num_out_blocks) * kBS;
  p.total_rows = total_rows;
  p.kind = kv_kind == 4 ? 3 : kv_kind;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  return launch_or_keep(
      [=](cudaStream_t s) { return launch_read_cache(p, head_dim, num_seqs, s); }, keep, stream);
}

}  // namespace

}  // namespace pa

extern "C" pa_status pa_read_cache(int kv_kind, void* k_out, void* v_out, int64_t out_stride,
                                   const void* k_cache, const void* v_cache,
                                   const float* k_scales, const float* v_scales,
                                   const int32_t* block_tables, int max_blocks_per_seq,
                                   const int32_t* first_positions, const int32_t* row_start_loc,
                                   int max_rows, int num_seqs, int total_rows,
                                   const int64_t* slot_mapping, int num_out_blocks,
                                   int num_kv_heads, int head_dim, int block_size,
                                   int num_blocks, pa_stream_t stream) {
  return pa::read_impl(kv_kind, k_out, v_out, out_stride, k_cache, v_cache, k_scales, v_scales,
                       block_tables, max_blocks_per_seq, first_positions, row_start_loc, max_rows,
                       num_seqs, total_rows, slot_mapping, num_out_blocks, num_kv_heads, head_dim,
                       block_size, num_blocks, stream, nullptr);
}

extern "C" pa_status pa_prepare_read_cache(
    pa_prepared** prepared, int kv_kind, void* k_out, void* v_out, int64_t out_stride,
    const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* first_positions,
    const int32_t* row_start_loc, int max_rows, int num_seqs, int total_rows,
    const int64_t* slot_mapping, int num_out_blocks, int num_kv_heads, int head_dim,
    int block_size, int num_blocks) {
  if (!prepared) return PA_ERR_INVALID_ARG;
  *prepared = nullptr;
  return pa::read_impl(kv_kind, k_out, v_out, out_stride, k_cache, v_cache, k_scales, v_scales,
                       block_tables, max_blocks_per_seq, first_positions, row_start_loc, max_rows,
                       num_seqs, total_rows, slot_mapping, num_out_blocks, num_kv_heads, head_dim,
                       block_size, num_blocks, nullptr, prepared);
}
