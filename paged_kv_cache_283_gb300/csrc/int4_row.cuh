// The 4-bit KV cache's storage, shared by the cache writes and the decode.
//
// A (block, KV head) tile of K or V is 9 D bytes: 8 D bytes of codes (16
// tokens x D / 2) and D bytes of parameters (one 32-bit word per token and
// group of 64 dims: the group's offset as bf16 in the low half, its scale as
// bf16 in the high half).  A value is offset + scale * code, code 0..15.
// K and V tiles place their nibbles for the decode's tensor-core steps
// (k4_nibble, v4_byte), so that a lane finds the codes it feeds in one run.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

namespace pa {

constexpr int kInt4Group = 64;  // dims that share one scale and offset

__host__ __device__ constexpr int int4_tile_bytes(int d) { return 9 * d; }

// Nibble of dim d within a K row of D / 2 bytes (even nibbles are low halves):
// lane tig of a decoding quad feeds dims 16 tig .. 16 tig + 15 of every group
// and reads them as one run of D / 8 bytes.
template <int D>
__host__ __device__ __forceinline__ int k4_nibble(int d) {
  const int e = d % kInt4Group;
  return (D / 4) * (e / 16) + e % 16 + 16 * (d / kInt4Group);
}

// Byte of a V tile that holds token t's codes of dims 16 c + i (low nibble)
// and 16 c + i + 8 (high nibble), i < 8.  Lane 4 i + (t % 8) / 2 of a decoding
// warp reads its D / 4 bytes as one 32-bit word per c; the word's bytes are
// tokens 2 tig, 2 tig + 8, 2 tig + 1, 2 tig + 9, so that a mask alone leaves
// two tokens' codes in the halves of a register.  Two tokens never share a
// byte.  At D = 128 the lane's two 16-byte runs swap places in every second
// row of lanes, so that the 8 lanes of a shared-memory phase hit 8 bank groups.
template <int D>
__host__ __device__ __forceinline__ int v4_byte(int t, int c, int i) {
  const int lane = 4 * i + ((t & 7) >> 1);
  const int run = D == 128 ? ((c >> 2) ^ (i & 1)) : 0;
  return lane * (D / 4) + 16 * run + 4 * (c & 3) + (t >> 3) + 2 * (t & 1);
}

// A group's parameters from its least and largest value: the offset is the
// least value (a bf16 value, so stored exactly), the scale the range times the
// float nearest 1 / 15, rounded to bf16 (the codes are taken with the rounded
// scale; at most 2^-8 above or below the exact one, so the largest code stays
// 15).  A range past the largest float counts as that.
__device__ __forceinline__ uint32_t int4_params(float lo, float hi, float* scale) {
  const float range = fminf(__fsub_rn(hi, lo), FLT_MAX);
  const uint32_t sc = __bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(range, 1.0f / 15.0f)));
  *scale = __uint_as_float(sc << 16);
  return (sc << 16) | (__float_as_uint(lo) >> 16);
}

// clamp(round_half_even((x - lo) / scale), 0, 15); 0 where the scale is 0.
// NaN gives 0.
__device__ __forceinline__ uint32_t int4_code(float x, float lo, float scale) {
  if (!(scale > 0.f)) return 0;
  const float c = fminf(15.f, fmaxf(0.f, rintf(__fdiv_rn(__fsub_rn(x, lo), scale))));
  return static_cast<uint32_t>(c);
}

// A row of D values spread over a warp (lane l owns dims [l D / 32, (l + 1) D /
// 32), as bf16 pairs) quantised: returns the lane's codes, 4 bits each, first
// dim lowest, and its group's parameters in *par.  All 32 lanes must call it.
template <int D>
__device__ __forceinline__ uint32_t quantise_row_int4(const uint32_t (&w)[D / 64], int lane,
                                                      uint32_t* par) {
  constexpr int PER = D / 32;
  float f[PER];
#pragma unroll
  for (int i = 0; i < PER / 2; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  float lo = f[0], hi = f[0];
#pragma unroll
  for (int i = 1; i < PER; ++i) {
    lo = fminf(lo, f[i]);
    hi = fmaxf(hi, f[i]);
  }
#pragma unroll
  for (int m = kInt4Group / PER / 2; m >= 1; m >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  float scale;
  *par = int4_params(lo, hi, &scale);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) codes |= int4_code(f[i], lo, scale) << (4 * i);
  return codes;
}

// Stores a quantised K row and V row (quantise_row_int4) as token `off` of a
// K tile and a V tile.  All 32 lanes must call it.
template <int D>
__device__ __forceinline__ void store_row_int4(uint8_t* kt, uint8_t* vt, int off, int lane,
                                               uint32_t kc, uint32_t kp, uint32_t vc,
                                               uint32_t vp) {
  constexpr int PER = D / 32, NG = D / kInt4Group;
  uint8_t* k = kt + off * (D / 2) + k4_nibble<D>(PER * lane) / 2;
  if constexpr (PER == 4)
    *reinterpret_cast<uint16_t*>(k) = static_cast<uint16_t>(kc);
  else
    *k = static_cast<uint8_t>(kc);
  // the lane holding dims 8 above this one's gives the bytes' high nibbles
  const uint32_t up = __shfl_xor_sync(0xffffffffu, vc, 8 / PER);
  const int d = PER * lane;
  if (d % 16 < 8) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      vt[v4_byte<D>(off, d / 16, d % 16 + i)] = static_cast<uint8_t>(
          ((vc >> (4 * i)) & 15u) | (((up >> (4 * i)) & 15u) << 4));
  }
  if (lane % (32 / NG) == 0) {
    const int at = off * NG + lane / (32 / NG);
    reinterpret_cast<uint32_t*>(kt + 8 * D)[at] = kp;
    reinterpret_cast<uint32_t*>(vt + 8 * D)[at] = vp;
  }
}

}  // namespace pa
