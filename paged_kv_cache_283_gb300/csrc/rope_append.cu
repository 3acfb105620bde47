// Rotary position embedding of a step's new q and k, and the write of its k
// and v into the paged cache, in one launch.
//
// For a token at position p, the pair (a, b) of dims i < R / 2 of every q and
// k head (a = x[i], b = x[i + R / 2]; interleaved: x[2 i], x[2 i + 1]) becomes
//   a cos(p f_i) - b sin(p f_i),  b cos(p f_i) + a sin(p f_i)
// with the cosines and sines of the caller's table; dims from R on pass
// through.  Products and sums are fp32, each rounded by itself (no fused
// multiply-add), so that a result does not depend on which of a pair's two
// products the compiler would fuse; a rotated value is rounded to bf16 once,
// and quantised caches quantise those bf16 values.
//
// What bounds it: bytes (each value is read and written once; three
// operations per value), or the launch itself for a decode step's few tokens.
// A row of D values belongs to L = D / 16 lanes, each holding two 16-byte
// chunks: the two halves of 8 rotation pairs, so that no value crosses lanes
// (interleaved pairs lie within a chunk).  A thread keeps its cosines and sines
// in registers and takes several rows (heads) of one token.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cache_row.cuh"
#include "device.cuh"
#include "int4_row.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 16;  // tokens of a block of the 1-byte and 4-bit caches
constexpr int64_t kOneRowThreads = 152 * 512;  // two CTAs an SM

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
  const float2 c = bf16x2_to_float2(w.z), d = bf16x2_to_float2(w.w);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ void rotate(float& a, float& b, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = u;
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = load_after_wait(reinterpret_cast<const float4*>(p));
  const float4 b = load_after_wait(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// A 16-byte load that may alias this kernel's stores (q rotated in place).
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The quantisers' codes are defined by the rounded quotient x / scale.  A row's 16
// quotients a lane were most of a quantising launch; here a quotient is x times
// the rounded reciprocal, off by less than 2^-22 of itself, which rounds to the
// same code unless it lies that near a border between two codes, and there (or
// for a scale whose reciprocal is no normal number) the division is made.
constexpr float kMinScale = 1e-30f, kMaxScale = 1e30f;  // of which the reciprocal is used

// round_half_even(x / scale), within +-2^21.
__device__ __forceinline__ float round_quotient(float x, float scale, float inv, bool divide) {
  const float t = __fmul_rn(x, inv);
  const float magic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  float c = __fsub_rn(__fadd_rn(t, magic), magic);
  // (|t| up to 127: an error below 3e-5)
  if (divide || fabsf(fabsf(__fsub_rn(t, c)) - 0.5f) < 1e-4f) c = rintf(__fdiv_rn(x, scale));
  return c;
}

// x / scale as E4M3 takes it: the quotient, exact wherever its E4M3 code could
// depend on its last bits.
__device__ __forceinline__ float e4m3_quotient(float x, float scale, float inv, bool divide) {
  const float t = __fmul_rn(x, inv);
  // a border between two codes: the 20 bits below E4M3's 3 are half a step
  const uint32_t low = __float_as_uint(t) & 0xFFFFFu;
  if (divide || !(fabsf(t) >= 0.015625f) || low - 0x7FFF0u <= 0x20u) return __fdiv_rn(x, scale);
  return t;
}

// Two chunks (ca, cb: 8-dim chunk indices) of one row quantised and stored.
// The L lanes of the row call it together; mask: those lanes.  x: the 16
// values, chunk ca's then chunk cb's.
template <int D, int Q>
__device__ __forceinline__ void store_quantised(const RopeAppendParams& p, bool is_v,
                                                const float (&x)[16], int ca, int cb,
                                                int64_t tile, int off, int j, unsigned mask) {
  constexpr int L = D / 16;
  if constexpr (Q == 3) {
    uint8_t* base = (is_v ? p.v4 : p.k4) + tile * int4_tile_bytes(D);
    constexpr int NG = D / kInt4Group;
    float lo[NG], hi[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      lo[g] = INFINITY;
      hi[g] = -INFINITY;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mn = x[8 * h], mx = x[8 * h];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        mn = fminf(mn, x[8 * h + i]);
        mx = fmaxf(mx, x[8 * h + i]);
      }
      const int g = (h == 0 ? ca : cb) / 8;
#pragma unroll
      for (int k = 0; k < NG; ++k)
        if (k == g) {
          lo[k] = fminf(lo[k], mn);
          hi[k] = fmaxf(hi[k], mx);
        }
    }
    float scale[NG];
    uint32_t par[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
#pragma unroll
      for (int m = L / 2; m >= 1; m >>= 1) {
        lo[g] = fminf(lo[g], __shfl_xor_sync(mask, lo[g], m));
        hi[g] = fmaxf(hi[g], __shfl_xor_sync(mask, hi[g], m));
      }
      par[g] = int4_params(lo[g], hi[g], &scale[g]);
    }
    uint32_t c[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int g = (h == 0 ? ca : cb) / 8;
      const float l = NG == 1 || g == 0 ? lo[0] : lo[NG - 1];
      const float s = NG == 1 || g == 0 ? scale[0] : scale[NG - 1];
      const float inv = __frcp_rn(s);
      const bool divide = !(s >= kMinScale && s <= kMaxScale);
#pragma unroll
      for (int i = 8 * h; i < 8 * h + 8; ++i) {
        // int4_code: clamped to 0..15 (a NaN to 0), 0 where the scale is 0
        const float q = round_quotient(__fsub_rn(x[i], l), s, inv, divide);
        c[i] = s > 0.f ? static_cast<uint32_t>(fminf(15.f, fmaxf(0.f, q))) : 0u;
      }
    }
    if (is_v) {  // chunks 2 j, 2 j + 1: dims 16 j + i and 16 j + i + 8
#pragma unroll
      for (int i = 0; i < 8; ++i)
        base[v4_byte<D>(off, j, i)] = static_cast<uint8_t>(c[i] | (c[8 + i] << 4));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= c[8 * h + i] << (4 * i);
        *reinterpret_cast<uint32_t*>(base + off * (D / 2) +
                                     k4_nibble<D>(8 * (h == 0 ? ca : cb)) / 2) = w;
      }
    }
    if (j < NG)
      reinterpret_cast<uint32_t*>(base + 8 * D)[off * NG + j] = j == 0 ? par[0] : par[NG - 1];
  } else {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int m = L / 2; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(mask, amax, m));
    const float scale = __fmul_rn(amax, Q == 2 ? 1.0f / 448.0f : 1.0f / 127.0f);
    uint32_t w[4] = {0, 0, 0, 0};  // chunk ca's 8 codes, chunk cb's 8 codes
    const float inv = __frcp_rn(scale);
    const bool divide = !(scale >= kMinScale && scale <= kMaxScale);
    if (scale > 0.f) {
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        uint32_t two;
        if constexpr (Q == 2) {
          two = __nv_cvt_float2_to_fp8x2(
              make_float2(e4m3_quotient(x[i], scale, inv, divide),
                          e4m3_quotient(x[i + 1], scale, inv, divide)),
              __NV_SATFINITE, __NV_E4M3);
        } else {
          const int a = static_cast<int>(
              fminf(127.f, fmaxf(-127.f, round_quotient(x[i], scale, inv, divide))));
          const int b = static_cast<int>(
              fminf(127.f, fmaxf(-127.f, round_quotient(x[i + 1], scale, inv, divide))));
          two = (static_cast<uint32_t>(a) & 0xffu) | ((static_cast<uint32_t>(b) & 0xffu) << 8);
        }
        w[i / 4] |= two << (8 * (i % 4));
      }
    }
    const int64_t srow = tile * kBlock + off;
    if (is_v) {
      uint8_t* base = reinterpret_cast<uint8_t*>(p.v8) + tile * kBlock * D;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = 8 * (i < 8 ? ca : cb) + i % 8;
        base[v_tile_pos<D>(off, d)] =
            static_cast<uint8_t>(v_stored<Q == 2>(w[i / 4]) >> (8 * (i % 4)));
      }
      if (j == 0) p.v_scales[srow] = scale;
    } else {
      uint8_t* row = reinterpret_cast<uint8_t*>(p.k8) + srow * D;
      *reinterpret_cast<uint2*>(row + 8 * ca) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(row + 8 * cb) = make_uint2(w[2], w[3]);
      if (j == 0) p.k_scales[srow] = scale;
    }
  }
}

// grid (tokens, thread blocks per token); thread group s of a token (L lanes)
// takes its rows s, s + row_slots, ..., U of them at most, loaded together and
// before the position and the slot are known (their round trips overlap).  All
// L lanes of a row follow the same path.
//
// Four CTAs of 256 threads an SM (64 registers): a quantising thread would take 92,
// and its row's chain of steps wants warps beside it.  8192 tokens of 32 + 16 rows,
// with 92, 80, 64 and 48 registers: 4-bit 55.6, 51.1, 44.2, 55.3 us (26.7 at the
// copy rate), INT8 49.8, 49.9, 43.9, 56.4, FP8 46.9, 47.0, 41.5, 55.0.
template <int D, int Q, int U>
__global__ void __launch_bounds__(kThreads, 4) rope_append_kernel(const RopeAppendParams p) {
  constexpr int L = D / 16;
  griddep_wait();  // the producer of q / key / value is complete
  griddep_launch_dependents();
  const int j = threadIdx.x % L;
  const int64_t t = blockIdx.x;
  const int s = (blockIdx.y * blockDim.x + threadIdx.x) / L;
  const unsigned mask = ((1u << L) - 1u) << (threadIdx.x & 31 & ~(L - 1));
  const int rot_lanes = p.rotary_dim / 16;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  if (s >= p.row_slots) return;

  // this lane's chunks of a rotated row
  const bool rot = j < rot_lanes;
  const int ra = rot ? j : 2 * rot_lanes + 2 * (j - rot_lanes);
  const int rb = rot ? j + rot_lanes : ra + 1;
  uint4 wa[U], wb[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = s + u * p.row_slots;
    if (r >= rows) break;
    const int h = r - p.num_q_heads;
    const bool is_v = h >= p.num_kv_heads;
    const __nv_bfloat16* src =
        h < 0 ? p.q + t * p.q_stride + r * D
              : is_v ? p.value + t * p.value_stride + (h - p.num_kv_heads) * D
                     : p.key + t * p.key_stride + h * D;
    wa[u] = load16(src + 8 * (is_v ? 2 * j : ra));
    wb[u] = load16(src + 8 * (is_v ? 2 * j + 1 : rb));
  }
  const int pos = p.positions != nullptr ? load_after_wait(p.positions + t) : 0;
  const int64_t slot = load_after_wait(p.slot_mapping + t);
  if (pos < 0) return;  // a padding token
  if (pos >= p.max_position) {
    if (s == 0 && j == 0) raise_error(p.err, PA_DEVERR_POSITION);
    return;
  }
  const bool bad_slot = slot >= p.num_slots;
  if (bad_slot && s == 0 && j == 0) raise_error(p.err, PA_DEVERR_SLOT);
  const bool put = slot >= 0 && !bad_slot;
  int64_t blk = slot >> 4;
  int off = static_cast<int>(slot & 15);
  if (p.block_size != 16 && put) {
    blk = slot / p.block_size;
    off = static_cast<int>(slot % p.block_size);
  }

  float cs[8], sn[8];  // the lane's cosines and sines
  if (rot) {
    const float* tab = p.cos_sin + static_cast<int64_t>(pos) * p.rotary_dim;
    const int half = p.rotary_dim / 2;
    if (p.interleaved) {  // chunk c holds pairs 4 c .. 4 c + 3
      const float4 ca4 = load_after_wait(reinterpret_cast<const float4*>(tab + 4 * ra));
      const float4 cb4 = load_after_wait(reinterpret_cast<const float4*>(tab + 4 * rb));
      const float4 sa4 = load_after_wait(reinterpret_cast<const float4*>(tab + half + 4 * ra));
      const float4 sb4 = load_after_wait(reinterpret_cast<const float4*>(tab + half + 4 * rb));
      cs[0] = ca4.x; cs[1] = ca4.y; cs[2] = ca4.z; cs[3] = ca4.w;
      cs[4] = cb4.x; cs[5] = cb4.y; cs[6] = cb4.z; cs[7] = cb4.w;
      sn[0] = sa4.x; sn[1] = sa4.y; sn[2] = sa4.z; sn[3] = sa4.w;
      sn[4] = sb4.x; sn[5] = sb4.y; sn[6] = sb4.z; sn[7] = sb4.w;
    } else {
      load8(tab + 8 * j, cs);
      load8(tab + half + 8 * j, sn);
    }
  }

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = s + u * p.row_slots;
    const int h = r - p.num_q_heads;
    if (r >= rows || (h >= 0 && !put)) continue;
    const bool is_v = h >= p.num_kv_heads;
    if (rot && !is_v) {
      float a[8], b[8];
      unpack8(wa[u], a);
      unpack8(wb[u], b);
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          rotate(a[2 * i], a[2 * i + 1], cs[i], sn[i]);
          rotate(b[2 * i], b[2 * i + 1], cs[4 + i], sn[4 + i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) rotate(a[i], b[i], cs[i], sn[i]);
      }
      wa[u] = pack8(a);
      wb[u] = pack8(b);
    }
    const int ca = is_v ? 2 * j : ra, cb = is_v ? 2 * j + 1 : rb;
    if (h < 0) {
      __nv_bfloat16* dst = p.q_out + (t * p.num_q_heads + r) * static_cast<int64_t>(D);
      *reinterpret_cast<uint4*>(dst + 8 * ca) = wa[u];
      *reinterpret_cast<uint4*>(dst + 8 * cb) = wb[u];
      continue;
    }
    const int64_t tile = blk * p.num_kv_heads + (is_v ? h - p.num_kv_heads : h);
    if constexpr (Q == 0) {
      __nv_bfloat16* dst =
          (is_v ? p.v_cache : p.k_cache) + (tile * p.block_size + off) * static_cast<int64_t>(D);
      *reinterpret_cast<uint4*>(dst + 8 * ca) = wa[u];
      *reinterpret_cast<uint4*>(dst + 8 * cb) = wb[u];
    } else {
      float x[16];
      unpack8(wa[u], *reinterpret_cast<float(*)[8]>(x));
      unpack8(wb[u], *reinterpret_cast<float(*)[8]>(x + 8));
      store_quantised<D, Q>(p, is_v, x, ca, cb, tile, off, j, mask);
    }
  }
}

template <int D, int Q>
cudaError_t launch_t(const RopeAppendParams& p, cudaStream_t stream) {
  constexpr int L = D / 16, U = 3;
  const int rows = p.num_q_heads + 2 * p.num_kv_heads;
  // While one row per thread makes few threads, the call is a chain of round
  // trips and a row to a thread is the shortest; past that a thread takes up to U
  // rows, which share its cosines and sines and overlap their loads.  In us, one
  // row and U (D = 128; bf16 with 32 + 16 rows a token, 4-bit with 16 + 8):
  //   bf16   64 tokens,   25K threads   1.9   2.1      128,  49K  1.9  2.1
  //         256,          98K           2.5   2.3     8192, 3.1M 49.3 34.5
  //   4-bit 400,          77K           3.6   4.0      512,  98K  4.1  4.0
  //        1024,         197K           6.4   4.8     8192, 1.6M 35.2 24.2
  // U: 8192 bf16 tokens take 36.6 us with 2 rows, 34.7 with 3, 34.8 with 4, 35.8
  // with 6; into a 4-bit cache 44.2 with 3, 59.3 with 4.
  const bool one = static_cast<int64_t>(p.num_tokens) * rows * L <= kOneRowThreads;
  RopeAppendParams r = p;
  r.row_slots = one ? rows : (rows + U - 1) / U;
  const int threads = (r.row_slots * L + 31) / 32 * 32;
  const dim3 block(threads < kThreads ? threads : kThreads);
  const dim3 grid(p.num_tokens, (threads + block.x - 1) / block.x);
  return one ? launch_pdl(rope_append_kernel<D, Q, 1>, grid, block, 0, stream, r)
             : launch_pdl(rope_append_kernel<D, Q, U>, grid, block, 0, stream, r);
}

template <int D>
cudaError_t launch_d(const RopeAppendParams& p, cudaStream_t stream) {
  switch (p.kind) {
    case 0: return launch_t<D, 0>(p, stream);
    case 1: return launch_t<D, 1>(p, stream);
    case 2: return launch_t<D, 2>(p, stream);
    default: return launch_t<D, 3>(p, stream);
  }
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int head_dim, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  if (head_dim == 128) return launch_d<128>(p, stream);
  if (head_dim == 64) return launch_d<64>(p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pa
