// The 4-bit cache's share of the paged decode kernels: q's operands, one step
// over NB blocks of 16 tokens, and a warp's finished sums.
//
// A cached value is lo + sc * code per token and group of 64 dims (int4_row.cuh).
// Everything that does not depend on the head is done once for the warp, and
// everything that does once per (token, head):
//
// QK: S = K q, the f16 MMA's rows the block's 16 tokens.  A mask leaves two codes
// in a register as f16 subnormals: nibbles at bits 0 and 16 stand for code *
// 2^-24, nibbles at bits 4 and 20 for code * 2^-20 (the second kind's q carries a
// factor 2^-4, exact), so five operations make the four operands of eight codes.
// (An E4M3 MMA would take the nibbles of a word by two masks and a shift, codes
// 0..15 being E4M3 values as they are; but mma.sync's E4M3 forms cost 125 ALU
// operations a 32-token step here against 80 -- 416 instructions and 1078 cycles
// against 352 and 1002, one warp alone, G = 4, D = 128.)  q,
// times a power of two that brings the head's largest |q| to [2^13, 2^14), is
// exact in f16 down to 2^-26 of that.  The columns, for G <= 4 and two groups: 2
// h + g holds head h's q of group g and zeros for the other group's dims, so one
// chain of MMAs leaves both groups' sums of head tig, tokens gid and gid + 8, in
// lane (gid, tig); for G = 8 heads tig and tig + 4 are columns 2 tig and 2 tig +
// 1, one chain per group.  With c_g those sums and qs_g the sum of q over group g,
//   s = sum_g sc_g c_g + lo_g qs_g.
//
// PV: out^T = V^T W, V's codes as f16 subnormals in the same way (undone once at
// the end).  W holds p * sc, one f16 each, in units of a power of two per head that
// follows the head's largest product: where one passes f16's range, the unit rises
// until it lies in [2^7, 2^8), and where the softmax reference rises, the unit falls
// with the products so far.  So a product keeps 11 bits (the output's error is about
// 2^-12 of its size, against the 2^-9 of its bf16 rounding) down to 2^-21 of the
// head's largest in the warp's tokens, and only below 2^-32 of it is it lost; a
// scale counts by its weight, however large.  (A unit that followed the largest
// scale alone, whatever its weight, put outputs off by 0.56 with one light token of
// 2^20 times the others' scale, and lost 17 % of a long context.  This one costs
// nothing for groups of 4, 64 contexts 19.8 and 19.9 us, and 3 % for groups of 8, 256
// contexts 110.7 and 113.9.)  The accumulators are fp32, to which the MMA truncates:
// some 2^-25 of a head's sum for every 16 tokens of a warp (settle).  The offsets' share,
// sum p * lo, is summed in fp32 beside them.  W's columns: for G <= 4, 2 h + g; for G = 8,
// heads tig and tig + 4 at 2 tig and 2 tig + 1, one operand per group.
// A lane computes its tokens' row of W; a matrix transpose of 8 x 8 halves
// (movmatrix) makes the operand.  So the lane that weighs head tig also holds
// the columns of head tig of the result, and its own rescale factor.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "decode_tile.cuh"
#include "device.cuh"
#include "int4_row.cuh"

namespace pa {

// LONG: a warp may take more than kSettleSteps steps (settle).
constexpr int kSettleSteps = 32;

template <int D, int G, bool LONG>
struct Warp4 {
  static constexpr int NG = D / kInt4Group;
  static constexpr int H = G == 8 ? 2 : 1;      // heads per lane: tig (+ 4)
  static constexpr int NW = G == 8 ? NG : 1;    // W operands per 16 tokens
  static constexpr int KT = int4_tile_bytes(D);
  // results per lane: its heads' dims 16 c + gid and 16 c + gid + 8
  static constexpr int V = D / 16 * 2 * H;
  static constexpr int NC = G == 8 ? NG : 1;    // QK accumulators

  uint32_t qw[D / 8];      // q's column gid
  float qf[H];             // factor of the MMA sums of the lane's heads
  float qs[H][NG];         // their q summed over each group, times the score scale
  float m[H], l[H];        // softmax reference (base 2), the lane's share of the sum
  float z[H][NG];          // the lane's share of sum p * lo
  float acc[D / 16][4];
  float vb[H];             // unit of the heads' PV weights and sums
  float taken[2];          // what settle() took from columns 2 tig, 2 tig + 1 (of 2^20 codes)

  static __device__ __forceinline__ int head(int tig, int h) { return (tig + 4 * h) % G; }
  // whether no other lane of the row holds the same results
  static __device__ __forceinline__ bool owner(int tig) { return G >= 4 || tig < G; }

  // q: the G heads of the group, D values each.
  __device__ __forceinline__ void begin(const __nv_bfloat16* q, float scale_log2, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
    // the column's head, and the one group of its dims that it holds (-1: all)
    const int hn = G == 8 ? gid / 2 + 4 * (gid % 2) : gid / 2 % G;
    const int only = G < 8 && NG == 2 ? gid % 2 : -1;
    const __nv_bfloat16* qh = q + static_cast<size_t>(hn) * D + 16 * tig;
    float f[D / 4];  // dims 16 tig .. 16 tig + 15 of every group
#pragma unroll
    for (int u = 0; u < D / 32; ++u) {
      const uint4 w =
          __ldg(reinterpret_cast<const uint4*>(qh + kInt4Group * (u / 2) + 8 * (u % 2)));
      const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
      const float2 c = bf16x2_to_float2(w.z), d = bf16x2_to_float2(w.w);
      f[8 * u] = a.x; f[8 * u + 1] = a.y; f[8 * u + 2] = b.x; f[8 * u + 3] = b.y;
      f[8 * u + 4] = c.x; f[8 * u + 5] = c.y; f[8 * u + 6] = d.x; f[8 * u + 7] = d.y;
    }
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < D / 4; ++k) amax = fmaxf(amax, fabsf(f[k]));
    amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
    // biased exponent of amax (0 for 0 and subnormals); k = 13 - unbiased
    const int ebits = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu);
    const int kexp = min(127, max(-126, 140 - ebits));
    const float up = __uint_as_float(static_cast<uint32_t>(kexp + 127) << 23);
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {  // nibbles 0 .. 7 of word w: f[8 w ..]
      const float x = only < 0 || only == w / 2 ? up : 0.f, y = x * 0.0625f;
      qw[4 * w] = f16x2_rn(f[8 * w] * x, f[8 * w + 4] * x);
      qw[4 * w + 1] = f16x2_rn(f[8 * w + 1] * y, f[8 * w + 5] * y);
      qw[4 * w + 2] = f16x2_rn(f[8 * w + 2] * x, f[8 * w + 6] * x);
      qw[4 * w + 3] = f16x2_rn(f[8 * w + 3] * y, f[8 * w + 7] * y);
    }
    // the lane's scores are those of its heads: their factors come from the rows
    // that hold them as columns
    float sum[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) x += f[16 * g + k];
      x += __shfl_xor_sync(kFullMask, x, 1);
      x += __shfl_xor_sync(kFullMask, x, 2);
      sum[g] = x * scale_log2;
    }
    const float factor = ldexpf(scale_log2, 24 - kexp);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const int src = 8 * tig + 4 * h;  // column 2 tig + h
      qf[h] = __shfl_sync(kFullMask, factor, src);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        qs[h][g] = __shfl_sync(kFullMask, sum[g], src);
        z[h][g] = 0.f;
      }
      m[h] = -INFINITY;
      l[h] = 0.f;
      vb[h] = kUnitFloor;
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[c][k] = 0.f;
    taken[0] = taken[1] = 0.f;
  }

  // Every kSettleSteps steps: the sums of a column's weights times codes (0 to 15) grow
  // with its weights, all alike; their mean is taken out of them, so that what the MMA
  // truncates stays small.  (Without, whole contexts of 131,072 tokens were off by 2.9 %
  // of their outputs' norm at D = 128 and 8.9 % at D = 64, now 0.18 and 0.21 %; compiled
  // into the short launches it costs them 1 to 3 %.)
  __device__ __forceinline__ void settle() {
    static_assert(LONG, "the means would be lost");
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float a = 0.f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) a += fmaf(acc[c][k], 16.f, acc[c][2 + k]);
      a *= 8.f / D;
      taken[k] += a;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        acc[c][k] = fmaf(a, -0.0625f, acc[c][k]);
        acc[c][2 + k] -= a;
      }
    }
  }
  // factors of the columns 2 tig and 2 tig + 1
  __device__ __forceinline__ void rescale(float fa, float fb) {
    scale_acc<D>(acc, fa, fb);
    if constexpr (LONG) {
      taken[0] *= fa;
      taken[1] *= fb;
    }
  }

  static __device__ __forceinline__ float hi16(uint32_t w) {
    return __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }

  // d = a . b, the first step of a sum
  static __device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                                   uint32_t a2, uint32_t a3, uint32_t b0,
                                                   uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  }
  static __device__ __forceinline__ uint32_t transpose(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
  }

  // The least unit: p * reciprocal(unit) stays finite for p up to 2^8 (lazy_max), and
  // what is below 2^-32 of a scale of 2^-126 is below any bf16.
  static constexpr float kUnitFloor = 0x1p-118f;
  // 1 / x of a power of two, and the largest power of two up to x (0 below 2^-126)
  static __device__ __forceinline__ float reciprocal(float x) {
    return __uint_as_float((254u << 23) - __float_as_uint(x));
  }
  static __device__ __forceinline__ float power_of_2(float x) {
    return __uint_as_float(__float_as_uint(x) & 0x7F800000u);
  }

  // One step: NB blocks, K tile then V tile each, of which the first nvalid
  // tokens count (FULL: all).  A hidden token's bytes may be anything.
  template <int NB, bool FULL>
  __device__ __forceinline__ void step(const unsigned char* __restrict__ stage, int nvalid,
                                       int lane) {
    const int gid = lane >> 2, tig = lane & 3;
    float2 s[NB][H];  // scores, then weights: tokens gid, gid + 8 of each block
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const unsigned char* kt = stage + u * 2 * KT;
      uint32_t k0[D / 32], k1[D / 32];
      const unsigned char* row = kt + gid * (D / 2) + (D / 8) * tig;
      if constexpr (D == 128) {
        const uint4 x = *reinterpret_cast<const uint4*>(row);
        const uint4 y = *reinterpret_cast<const uint4*>(row + 8 * (D / 2));
        k0[0] = x.x; k0[1] = x.y; k0[2] = x.z; k0[3] = x.w;
        k1[0] = y.x; k1[1] = y.y; k1[2] = y.z; k1[3] = y.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(row);
        const uint2 y = *reinterpret_cast<const uint2*>(row + 8 * (D / 2));
        k0[0] = x.x; k0[1] = x.y;
        k1[0] = y.x; k1[1] = y.y;
      }
      float c[NC][4];
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {  // two words of codes to a group
        const int o = NC == 2 ? w / 2 : 0;
        const uint32_t x0 = k0[w], x1 = k1[w], y0 = k0[w] >> 8, y1 = k1[w] >> 8;
        if (w == 0 || (NC == 2 && w == 2))
          mma_first(c[o], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u,
                    x1 & 0x00F000F0u, qw[4 * w], qw[4 * w + 1]);
        else
          mma_f16(c[o], x0 & 0x000F000Fu, x1 & 0x000F000Fu, x0 & 0x00F000F0u,
                  x1 & 0x00F000F0u, qw[4 * w], qw[4 * w + 1]);
        mma_f16(c[o], y0 & 0x000F000Fu, y1 & 0x000F000Fu, y0 & 0x00F000F0u, y1 & 0x00F000F0u,
                qw[4 * w + 2], qw[4 * w + 3]);
      }
      uint32_t p0[NG], p1[NG];  // parameters of tokens gid, gid + 8
      load_params(kt, gid, p0);
      load_params(kt, gid + 8, p1);
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float2 d, zz;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          // column 2 tig + (G = 8: the head, else the group), both tokens
          const int o = NC == 2 ? g : 0, col = G == 8 ? h : g;
          const float2 e = make_float2(c[o][col], c[o][2 + col]);
          const float2 sc = make_float2(hi16(p0[g]), hi16(p1[g]));
          const float2 lo = make_float2(lo16(p0[g]), lo16(p1[g]));
          const float2 q2 = make_float2(qs[h][g], qs[h][g]);
          d = g == 0 ? __fmul2_rn(e, sc) : __ffma2_rn(e, sc, d);
          zz = g == 0 ? __fmul2_rn(lo, q2) : __ffma2_rn(lo, q2, zz);
        }
        s[u][h] = __ffma2_rn(d, make_float2(qf[h], qf[h]), zz);
        if constexpr (!FULL) {
          if (!(16 * u + gid < nvalid)) s[u][h].x = -INFINITY;
          if (!(16 * u + gid + 8 < nvalid)) s[u][h].y = -INFINITY;
        }
      }
    }
    // each head's maximum over the step: the lane's tokens, then the 8 rows
    float alpha[H];
    bool moved = false;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float mx = fmaxf(s[0][h].x, s[0][h].y);
#pragma unroll
      for (int u = 1; u < NB; ++u) mx = fmaxf(mx, fmaxf(s[u][h].x, s[u][h].y));
      mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 16));
      const float m_new = lazy_max(m[h], mx);
      alpha[h] = 1.f;
      if (m_new != m[h]) {
        alpha[h] = ex2_fast(m[h] - m_new);
        moved |= m[h] != -INFINITY;  // (the sums before the first step are zeros)
        m[h] = m_new;
      }
      const float2 neg = make_float2(-m[h], -m[h]);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        const float2 x = __fadd2_rn(s[u][h], neg);
        s[u][h] = make_float2(ex2_fast(x.x), ex2_fast(x.y));
        sum = u == 0 ? s[u][h] : __fadd2_rn(sum, s[u][h]);
      }
      l[h] = fmaf(l[h], alpha[h], sum.x + sum.y);
    }
    // a risen reference lowers what was summed by alpha; its power of two goes into
    // the unit, so that weights to come keep their range
    if (__any_sync(kFullMask, moved)) {
      float f[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float now = alpha[h] * vb[h];
        vb[h] = fmaxf(power_of_2(now), kUnitFloor);
        f[h] = now * reciprocal(vb[h]);
#pragma unroll
        for (int g = 0; g < NG; ++g) z[h][g] *= alpha[h];
      }
      rescale(f[0], f[H - 1]);  // the columns are the lane's heads
    }
    // V's parameters of the lane's tokens of block u (hidden ones count nothing)
    auto load_v = [&](int u, uint32_t(&w0)[NG], uint32_t(&w1)[NG]) {
      const unsigned char* vt = stage + u * 2 * KT + KT;
      load_params(vt, gid, w0);
      load_params(vt, gid + 8, w1);
      if constexpr (!FULL) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          if (!(16 * u + gid < nvalid)) w0[g] = 0u;
          if (!(16 * u + gid + 8 < nvalid)) w1[g] = 0u;
        }
      }
    };
    // the lane's rows of W: tokens gid (b0) and gid + 8 (b1), before the transpose;
    // returns their largest halves
    uint32_t b0[NB][NW], b1[NB][NW];
    auto weigh = [&](int u, const uint32_t(&w0)[NG], const uint32_t(&w1)[NG], uint32_t top) {
      float2 y[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const float inv = reciprocal(vb[h]);
        y[h] = __fmul2_rn(s[u][h], make_float2(inv, inv));
      }
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        // columns 2 tig and 2 tig + 1: two heads' (G = 8), else one head's two groups
        // (one group: the odd columns are not read)
        const int ga = G == 8 ? n : 0, gb = G == 8 ? n : NG - 1;
        b0[u][n] = f16x2_rn(y[0].x * hi16(w0[ga]), y[H - 1].x * hi16(w0[gb]));
        b1[u][n] = f16x2_rn(y[0].y * hi16(w1[ga]), y[H - 1].y * hi16(w1[gb]));
        top = __vimax3_u16x2(top, b0[u][n], b1[u][n]);
      }
      return top;
    };
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      uint32_t w0[NG], w1[NG];
      load_v(u, w0, w1);
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int g = 0; g < NG; ++g)
          z[h][g] = fmaf(s[u][h].x, lo16(w0[g]), fmaf(s[u][h].y, lo16(w1[g]), z[h][g]));
      top = weigh(u, w0, w1, top);
    }
    // a half of 0x7C00 or more is a product past f16's range (65,504 units): the unit
    // rises, and the step's products are taken again
    if (__any_sync(kFullMask, ((top + 0x04000400u) & 0x80008000u) != 0)) {
      float f[H], w[H];
#pragma unroll
      for (int h = 0; h < H; ++h) w[h] = 0.f;
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        uint32_t w0[NG], w1[NG];
        load_v(u, w0, w1);
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int g = 0; g < NG; ++g)  // (times 2^-16: finite for any p and scale)
            w[h] = fmaxf(w[h], fmaxf(s[u][h].x * 0x1p-16f * hi16(w0[g]),
                                     s[u][h].y * 0x1p-16f * hi16(w1[g])));
      }
#pragma unroll
      for (int h = 0; h < H; ++h) {
        w[h] = fmaxf(w[h], __shfl_xor_sync(kFullMask, w[h], 4));
        w[h] = fmaxf(w[h], __shfl_xor_sync(kFullMask, w[h], 8));
        w[h] = fmaxf(w[h], __shfl_xor_sync(kFullMask, w[h], 16));
        const float nb = fmaxf(vb[h], power_of_2(w[h]) * 0x1p9f);
        f[h] = vb[h] * reciprocal(nb);
        vb[h] = nb;
      }
      rescale(f[0], f[H - 1]);
#pragma unroll
      for (int u = 0; u < NB; ++u) {
        uint32_t w0[NG], w1[NG];
        load_v(u, w0, w1);
        weigh(u, w0, w1, 0u);
      }
    }
#pragma unroll
    for (int u = 0; u < NB; ++u)
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        b0[u][n] = transpose(b0[u][n]);
        b1[u][n] = transpose(b1[u][n]);
      }
#pragma unroll
    for (int u = 0; u < NB; ++u) {
      const unsigned char* base = stage + u * 2 * KT + KT + lane * (D / 4);
#pragma unroll
      for (int v = 0; v < D / 64; ++v) {  // dims of group v
        const uint4 x = *reinterpret_cast<const uint4*>(
            base + 16 * (D == 128 ? (v ^ (gid & 1)) : 0));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        const int o = NW == 2 ? v : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t y = w[k] >> 8;
          mma_f16(acc[4 * v + k], w[k] & 0x000F000Fu, w[k] & 0x00F000F0u, y & 0x000F000Fu,
                  y & 0x00F000F0u, b0[u][o], b1[u][o]);
        }
      }
    }
  }

  // The warp's sums: v[(2 c + j) * H + h] = sum p v of head(tig, h), dim 16 c +
  // gid + 8 j; ml[h] = (m, l).  All 32 lanes must call it.
  __device__ __forceinline__ void finish(int lane, float (&v)[V], float2 (&ml)[H]) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[h] += __shfl_xor_sync(kFullMask, l[h], x);
#pragma unroll
        for (int g = 0; g < NG; ++g) z[h][g] += __shfl_xor_sync(kFullMask, z[h][g], x);
      }
      ml[h] = make_float2(m[h], l[h]);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const int g = c / 4;
        const int col = G == 8 ? h : g;  // 2 tig or 2 tig + 1
        // (the codes' 2^-24 and 2^-20 first: a unit may be near the largest float)
        float a = acc[c][col] * 16.f, b = acc[c][2 + col];
        if constexpr (LONG) {
          a += taken[col];
          b += taken[col];
        }
        v[2 * c * H + h] = fmaf(a * 0x1p20f, vb[h], z[h][g]);
        v[(2 * c + 1) * H + h] = fmaf(b * 0x1p20f, vb[h], z[h][g]);
      }
    }
  }

 private:
  static __device__ __forceinline__ void load_params(const unsigned char* tile, int t,
                                                     uint32_t (&w)[NG]) {
    const unsigned char* par = tile + 8 * D + t * NG * 4;
    if constexpr (NG == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(par);
      w[0] = x.x; w[1] = x.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(par);
    }
  }
};

}  // namespace pa
