// Beam search's selection (pa_beam_select): of a search's beams x vocabulary,
// the K continuations with the largest sums of log-probabilities.
//
//   total(w, v) = score[w] + x[w, v] - log sum_u exp(x[w, u])
//
// Bytes bound it: the logits are read once.  Within a row the order of the
// totals is the order of the logits, so one pass gives both the row's log-sum
// (a running maximum and sum per thread, joined by warps, CTAs and the merge)
// and the K largest logits of each part of the row; the totals are needed for
// those alone.
//
//  * A CTA takes a part of a row, block by block, P pieces of eight logits a thread
//    in flight, and leaves each thread's maximum of each block in shared memory.
//    256 threads form G >= 2 K groups; the K-th largest of the groups' maxima is a
//    bound that at least K logits reach, and hardly more do (of independent values
//    some 1.4 K): only the blocks whose maximum reaches it are read again, and what
//    reaches it goes to shared memory, where each counts how many precede it.
//    Where many are equal more may reach the bound: then the K largest are taken one
//    by one: each of the K passes reads the part again, an element a load.  Rows of equal
//    logits, or all but K of them masked with a finite number, go that way (64 x 4
//    beams of 128,256 tokens, K = 8: 556 us against 17.5; one search 31 to 36 against 16).
//    What is masked with -inf is no candidate (16.5 us).
//  * 64 x 4 beams of 128,256 bf16 tokens, 66 MB that fit L2: 20.7 us, 3.2 TB/s, with new
//    logits each call, 17.4 to 17.8 the same ones again.  The phases after a part's sums
//    cost as much as its logits, so parts are long.
//  * Which thread holds which logit goes by its index in the row alone, not by
//    the row's alignment, so equal rows have equal sums, bit for bit, and equal
//    totals: ties go to the lower beam, then to the lower token.
//  * The last CTA of a search to arrive (a counter, zeroed again by it) joins
//    the parts.  Totals are taken and compared in 64 bits, so that fp32's rounding of a
//    sum (1e-6 of a score of -10) joins no two of them.  Within a row their order is the
//    logits' own, exactly.  Between beams it is as good as the rows' log-sums, of which
//    the exponentials (2^-22), their arguments and the parts' sums are taken in fp32:
//    off by less than 2e-5, by at most 3e-7 in rows of 1000 to 2^20 random logits.
//
// A row whose address is no multiple of 16 bytes (an odd vocabulary) is read in
// aligned 16-byte words, shifted into place in registers.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include <algorithm>

#include "device.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 4;      // an SM
constexpr int kWave = 4 * 152;  // CTAs of a wave
constexpr int kRoom = 1024;   // candidates that a CTA can hold
constexpr int kHits = 512;    // blocks of a thread that can hold candidates
constexpr int kMaxBlocks = 16;  // of a part
constexpr int kGroups = 128;  // at most
constexpr int kRank = 192;    // up to this many are ranked by counting
constexpr float kLog2e = 1.4426950408889634f;

// What candidates are ordered by: the larger value first, then the lower index.
// Value and index: within a row the logit and the token; of a search the total and
// (beam, logit, token) in 5, 32 (the larger first) and 27 bits, because logits of a
// row that differ can have the same total in 64 bits.
struct Key {
  uint64_t v;
  uint64_t i;
};
__device__ __forceinline__ bool before(const Key& a, const Key& b) {
  return a.v > b.v || (a.v == b.v && a.i < b.i);
}
constexpr uint64_t kNone = ~0ull;
constexpr uint32_t kTokenMask = kBeamMaxVocab - 1;
__device__ __forceinline__ Key nothing() { return Key{0, kNone}; }

// Unsigned numbers in the order of the floats (all of them above 0; no NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // (-0 counts as 0)
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t ordered(double x) {
  const uint64_t u = __double_as_longlong(x + 0.0);
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unordered64(uint64_t o) {
  return __longlong_as_double(o & 0x8000000000000000ull ? o ^ 0x8000000000000000ull : ~o);
}

// Eight logits in 32-bit words: unpacked in pairs, and, two in a word where they
// are 16-bit, compared without unpacking.
template <typename T>
struct Words;
template <>
struct Words<float> {
  static constexpr int N = 8;
  static constexpr float kLowest = -FLT_MAX;
  using Top = float;
  __device__ static float2 pair(const uint32_t (&w)[8], int i) {
    return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  __device__ static void lowest(uint32_t (&w)[8], int i) { w[i] = 0xff800000u; }
  // the larger of top and the eight, NaN passed over
  __device__ static void raise(float& top, const uint32_t (&w)[8]) {
#pragma unroll
    for (int k = 0; k < 8; k += 2)
      top = fmaxf(top, fmaxf(__uint_as_float(w[k]), __uint_as_float(w[k + 1])));
  }
  __device__ static float none() { return -INFINITY; }
  __device__ static float value(float top) { return top; }
  // bit i: logit i is at least `bound`
  __device__ static uint32_t reach(const uint32_t (&w)[8], float bound) {
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) bits |= __uint_as_float(w[k]) >= bound ? 1u << k : 0u;
    return bits;
  }
};
template <typename T2>
struct Halves {
  static constexpr int N = 4;
  using Top = T2;
  __device__ static T2 word(uint32_t w) { return *reinterpret_cast<const T2*>(&w); }
  __device__ static void lowest(uint32_t (&w)[4], int i, uint32_t bits) {
    w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | bits << 16 : (w[i / 2] & 0xffff0000u) | bits;
  }
  __device__ static void raise(T2& top, const uint32_t (&w)[4]) {
    top = __hmax2(top, __hmax2(__hmax2(word(w[0]), word(w[1])), __hmax2(word(w[2]), word(w[3]))));
  }
  __device__ static uint32_t reach2(const uint32_t (&w)[4], T2 bound) {
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t m = __hge2_mask(word(w[k]), bound);  // 0xffff in each half that reaches
      bits |= m & (0x00010001u << k);
    }
    // low halves are bits 0 .. 3 (logits 0, 2, 4, 6), high ones bits 16 .. 19
    return bits;
  }
};
template <>
struct Words<__nv_bfloat16> : Halves<__nv_bfloat162> {
  static constexpr float kLowest = -3.38953139e38f;
  __device__ static float2 pair(const uint32_t (&w)[4], int i) { return bf16x2_to_float2(w[i]); }
  __device__ static void lowest(uint32_t (&w)[4], int i) {
    Halves<__nv_bfloat162>::lowest(w, i, 0xff80u);
  }
  __device__ static __nv_bfloat162 none() { return word(0xff80ff80u); }
  __device__ static float value(__nv_bfloat162 t) {
    return fmaxf(__low2float(t), __high2float(t));
  }
  __device__ static uint32_t reach(const uint32_t (&w)[4], float bound) {
    return reach2(w, __float2bfloat162_rn(bound));
  }
};
template <>
struct Words<__half> : Halves<__half2> {
  static constexpr float kLowest = -65504.f;
  __device__ static float2 pair(const uint32_t (&w)[4], int i) { return __half22float2(word(w[i])); }
  __device__ static void lowest(uint32_t (&w)[4], int i) {
    Halves<__half2>::lowest(w, i, 0xfc00u);
  }
  __device__ static __half2 none() { return word(0xfc00fc00u); }
  __device__ static float value(__half2 t) { return fmaxf(__low2float(t), __high2float(t)); }
  __device__ static uint32_t reach(const uint32_t (&w)[4], float bound) {
    return reach2(w, __float2half2_rn(bound));
  }
};
// The logit of a bit of reach().
template <typename T>
__device__ __forceinline__ int logit_of(int bit) {
  return sizeof(T) == 4 ? bit : 2 * (bit & 15) + (bit >> 4);
}

// A logit as it counts: NaN and +inf are hidden.
template <typename T>
__device__ __forceinline__ float visible(T x) {
  const float f = static_cast<float>(x);
  return f < INFINITY ? f : -INFINITY;
}

// 2^(-i / 64)
__constant__ double kPowers[64] = {
    1.0, 0.9892280131939755, 0.9785720620877001, 0.9680308967461472,
    0.9576032806985737, 0.9472879907934828, 0.93708381705515, 0.9269895625416927,
    0.9170040432046712, 0.9071260877501994, 0.8973545375015536, 0.8876882462632606,
    0.8781260801866497, 0.8686669176368531, 0.859309649061239, 0.8500531768592617,
    0.8408964152537145, 0.8318382901633682, 0.8228777390769825, 0.8140137109286739,
    0.8052451659746271, 0.7965710756711335, 0.7879904225539432, 0.7795022001189185,
    0.7711054127039704, 0.7627990753722692, 0.7545822137967114, 0.7464538641456324,
    0.7384130729697497, 0.7304588970903235, 0.7225904034885233, 0.714806669195985,
    0.7071067811865476, 0.6994898362691556, 0.691954940981916, 0.6845012114872953,
    0.6771277734684463, 0.6698337620266515, 0.6626183215798707, 0.6554806057623822,
    0.6484197773255048, 0.6414350080393891, 0.6345254785958666, 0.6276903785123455,
    0.620928906036742, 0.614240268053435, 0.6076236799902345, 0.6010783657263515,
    0.5946035575013605, 0.5881984958251406, 0.5818624293887887, 0.5755946149764913,
    0.5693943173783458, 0.5632608093041209, 0.5571933712979462, 0.5511912916539204,
    0.5452538663326288, 0.5393803988785599, 0.5335702003384118, 0.5278225891802786,
    0.5221368912137069, 0.5165124395106142, 0.5109485743270583, 0.5054446430258502};

// ln(s) of 1 <= s < 2^60 to 1e-11, in a tenth of the time of 64-bit arithmetic all
// through: j / 64 is the binary logarithm to half a 64th, t = s 2^(-j / 64) - 1 is
// within 0.0055 of 0, and ln(1 + t) = t - t^2 / 2 + ..., the terms after t in fp32.
__device__ __forceinline__ double log64(double s) {
  float l;
  asm("lg2.approx.f32 %0, %1;" : "=f"(l) : "f"(static_cast<float>(s)));
  const int j = __float2int_rn(64.f * l);
  const double scaled = __longlong_as_double(__double_as_longlong(s) -
                                             (static_cast<int64_t>(j >> 6) << 52));  // s 2^-(j / 64)
  const double t = scaled * kPowers[j & 63] - 1.0;
  const float f = static_cast<float>(t);
  const float rest = f * f * fmaf(f, fmaf(f, fmaf(f, 0.2f, -0.25f), 1.f / 3.f), -0.5f);
  return fma(static_cast<double>(j), 0.010830424696249145, t + static_cast<double>(rest));
}

struct Shared {
  uint32_t tops[kMaxBlocks][kThreads];  // the maximum of each thread's logits of a block
  uint16_t hit[kHits];
  uint64_t v[kRoom];
  uint64_t i[kRoom];
  Key best[kWarps];
  Key last;
  float group_max[kGroups];
  uint64_t group_key[kGroups], warp_key[kWarps][32];
  float m[kWarps], s[kWarps];
  uint64_t out_v[kBeamMaxKeep];  // the K found, first to last
  uint64_t out_i[kBeamMaxKeep];
  double lse[kBeamMaxBeams], score[kBeamMaxBeams];
  int state[kBeamMaxBeams];  // of a beam: 0 ended in nothing, 1 goes on, 2 finished
  int place[kBeamMaxKeep];
  uint64_t bound;
  int count, hits;
  unsigned arrived;
};
__device__ __forceinline__ Shared& shared() {
  __shared__ Shared sh;
  return sh;
}

// The K first of the CTA's keys, one by one, to sh.out_*: each thread offers
// through scan(prev, first) its first key after `prev`.  For many equal values.
template <typename Scan>
__device__ __forceinline__ void one_by_one(int k, Scan&& scan) {
  Shared& sh = shared();
  Key prev{~0ull, 0};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = 0; r < k; ++r) {
    Key best = scan(prev, r == 0);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) {
      Key o;
      o.v = __shfl_xor_sync(kFullMask, best.v, m);
      o.i = __shfl_xor_sync(kFullMask, best.i, m);
      if (before(o, best)) best = o;
    }
    if (lane == 0) sh.best[warp] = best;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kWarps; ++w)
        if (before(sh.best[w], best)) best = sh.best[w];
      sh.last = best;
      sh.out_v[r] = best.v;
      sh.out_i[r] = best.i;
    }
    __syncthreads();
    prev = sh.last;
    if (prev.i == kNone) {  // no more
      for (int q = r + 1 + threadIdx.x; q < k; q += kThreads) {
        sh.out_v[q] = 0;
        sh.out_i[q] = kNone;
      }
      break;
    }
  }
  __syncthreads();
}

__device__ __noinline__ void one_by_one_of_room(int count, int k) {
  Shared& sh = shared();
  one_by_one(k, [&](const Key& prev, bool first) {
    Key best = nothing();
    for (int c = threadIdx.x; c < count; c += kThreads) {
      const Key x{sh.v[c], sh.i[c]};
      if ((first || before(prev, x)) && before(x, best)) best = x;
    }
    return best;
  });
}

template <typename T>
__device__ __noinline__ void one_by_one_of_row(const T* row, int begin, int end, int k) {
  one_by_one(k, [&](const Key& prev, bool first) {
    Key best = nothing();
    for (int e = begin + threadIdx.x; e < end; e += kThreads) {
      const float x = visible(row[e]);
      const Key key{ordered(x), static_cast<uint64_t>(e)};
      if (x > -INFINITY && (first || before(prev, key)) && before(key, best)) best = key;
    }
    return best;
  });
}

// The K first of sh.v / sh.i[0 .. count), count <= kRoom, to sh.out_*.  Each is
// compared with every other: four neighbouring lanes a candidate, a quarter of
// them each.
__device__ __forceinline__ void best_of_room(int count, int k) {
  Shared& sh = shared();
  if (count <= kRank) {
    const int seg = threadIdx.x & 3;
    for (int c0 = 0; c0 < count; c0 += kThreads / 4) {
      if (c0 + static_cast<int>(threadIdx.x >> 5) * 8 >= count) break;  // none for the warp
      const int c = c0 + static_cast<int>(threadIdx.x >> 2);
      const Key mine = c < count ? Key{sh.v[c], sh.i[c]} : nothing();
      int rank = 0;
#pragma unroll 4
      for (int o = seg; o < count; o += 4) {
        const uint64_t v = sh.v[o], i = sh.i[o];
        rank += (v > mine.v) | ((v == mine.v) & (i < mine.i));
      }
      rank += __shfl_xor_sync(kFullMask, rank, 1);
      rank += __shfl_xor_sync(kFullMask, rank, 2);
      if (seg == 0 && c < count && rank < k) {
        sh.out_v[rank] = mine.v;
        sh.out_i[rank] = mine.i;
      }
    }
    for (int r = count + threadIdx.x; r < k; r += kThreads) {
      sh.out_v[r] = 0;
      sh.out_i[r] = kNone;
    }
    __syncthreads();
  } else {
    one_by_one_of_room(count, k);
  }
}

// The K-th largest (rank K - 1) of the groups' values, by the first warps.
__device__ __forceinline__ uint64_t bits_of(float x) { return __float_as_uint(x); }
__device__ __forceinline__ uint64_t bits_of(uint64_t x) { return x; }
template <typename V>
__device__ __forceinline__ void kth_of_groups(const V* value, int groups, int k, uint64_t* out) {
  if (threadIdx.x < static_cast<unsigned>(groups)) {
    const V x = value[threadIdx.x];
    int rank = 0;
#pragma unroll 8
    for (int g = 0; g < groups; ++g) {
      const V o = value[g];
      rank += o > x || (o == x && g < static_cast<int>(threadIdx.x));
    }
    if (rank == k - 1) *out = bits_of(x);
  }
}

// A part's find (beam w, `key` of the workspace) as a candidate of its search.
__device__ __forceinline__ Key candidate(const BeamParams& p, int w, bool first, uint64_t key) {
  const Shared& sh = shared();
  const int state = sh.state[w];
  const uint64_t beam = static_cast<uint64_t>(w) << 59;
  if (state == 2)  // its one continuation
    return first ? Key{ordered(sh.score[w]), beam | static_cast<uint32_t>(p.eos)} : nothing();
  if (state == 0 || key == 0) return nothing();
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  const double total = sh.score[w] + (static_cast<double>(unordered(o)) - sh.lse[w]);
  return Key{ordered(total), beam | static_cast<uint64_t>(~o) << 27 |
                                 static_cast<uint32_t>(~static_cast<uint32_t>(key))};
}
__device__ __forceinline__ Key candidate(const BeamParams& p, int c, uint64_t key) {
  const int w = c / (p.parts * p.keep);
  return candidate(p, w, c == w * p.parts * p.keep, key);
}

__device__ __noinline__ void one_by_one_of_parts(const BeamParams* p, int search) {
  const int total = p->beams * p->parts * p->keep;
  const uint64_t* parts = p->ws_keys + static_cast<int64_t>(search) * total;
  one_by_one(p->keep, [&](const Key& prev, bool first) {
    Key best = nothing();
    for (int c = threadIdx.x; c < total; c += kThreads) {
      const Key x = candidate(*p, c, __ldcg(parts + c));
      if ((first || before(prev, x)) && before(x, best)) best = x;
    }
    return best;
  });
}

// Joins the parts of a search: the last CTA's work.
__device__ __forceinline__ void merge(const BeamParams& p, int search) {
  Shared& sh = shared();
  const int tid = threadIdx.x, W = p.beams, K = p.keep;
  const int total = W * p.parts * K;
  const uint64_t* parts = p.ws_keys + static_cast<int64_t>(search) * total;
  // Thread t takes candidates t, t + 256, .. of the parts' firsts, then their seconds
  // and so on, and group g of `groups` the threads t = g mod groups.  The list of a
  // part moves on by an odd number of groups, 5/8 of them, from one rank to the next,
  // so that the many finds of one good beam lie in many groups and the bound below is
  // a good one (1910 candidates reach it of 32 beams in 4 parts, K = 64, where lists
  // keep to a group, 77 so).
  const int lists = W * p.parts;
  const int turn = (lists - (p.groups * 5 / 8 | 1)) & (p.groups - 1);
  auto place = [&](int c) {
    const int r = c / lists;
    return (c - r * lists + r * turn) % lists * K + r;
  };
  constexpr int kHeld = 2;  // candidates of a thread that stay in registers
  uint64_t raw[kHeld];
  int at[kHeld];
#pragma unroll
  for (int q = 0; q < kHeld; ++q) {
    const int c = tid + q * kThreads;
    at[q] = place(c);
    raw[q] = c < total ? __ldcg(parts + at[q]) : 0;
  }
  for (int w = tid >> 5; w < W; w += kWarps) {  // each row's log-sum from its parts
    const int64_t row = static_cast<int64_t>(search) * W + w;
    const float2* ms = p.ws_sums + row * p.parts;
    const float score = load_after_wait(p.scores + row);
    const bool finished = p.finished && p.finished[row];
    const float2 mine =
        (tid & 31) < p.parts ? __ldcg(ms + (tid & 31)) : make_float2(-INFINITY, 0.f);
    float top = mine.x;
    for (int c = (tid & 31) + 32; c < p.parts; c += 32) top = fmaxf(top, __ldcg(ms + c).x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, m));
    double s = mine.y > 0.f ? mine.y * ex2((mine.x - top) * kLog2e) : 0.f;
    for (int c = (tid & 31) + 32; c < p.parts; c += 32) {
      const float2 part = __ldcg(ms + c);
      if (part.y > 0.f) s += part.y * ex2((part.x - top) * kLog2e);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(kFullMask, s, m);
    if ((tid & 31) == 0) {
      sh.lse[w] = s > 0.0 ? static_cast<double>(top) + log64(s) : 0.0;
      sh.score[w] = score;
      sh.state[w] = !isfinite(score) ? 0 : finished ? 2 : 1;
    }
  }
  if (tid == 0) sh.count = 0;
  __syncthreads();
  // the K-th largest of the groups' maxima bounds the K-th largest of all
  auto nth = [&](int c) {
    const int a = place(c);
    return candidate(p, a, __ldcg(parts + a));
  };
  Key held[kHeld];
  uint64_t gm = 0;
#pragma unroll
  for (int q = 0; q < kHeld; ++q) {
    held[q] = tid + q * kThreads < total ? candidate(p, at[q], raw[q]) : nothing();
    gm = held[q].v > gm ? held[q].v : gm;
  }
  for (int c = tid + kHeld * kThreads; c < total; c += kThreads) {
    const Key x = nth(c);
    gm = x.v > gm ? x.v : gm;
  }
  for (int m = p.groups; m < 32; m <<= 1) {
    const uint64_t o = __shfl_xor_sync(kFullMask, gm, m);
    gm = o > gm ? o : gm;
  }
  sh.warp_key[tid >> 5][tid & 31] = gm;
  __syncthreads();
  if (tid < p.groups) {  // (above 32 groups: of every second warp, or fourth)
    uint64_t x = 0;
    for (int w = tid >> 5; w < kWarps; w += p.groups > 32 ? p.groups / 32 : 1) {
      const uint64_t o = sh.warp_key[w][tid & 31];
      x = o > x ? o : x;
    }
    sh.group_key[tid] = x;
  }
  __syncthreads();
  kth_of_groups(sh.group_key, p.groups, K, &sh.bound);
  __syncthreads();
  const uint64_t bound = sh.bound;
  auto take = [&](const Key& x) {
    if (x.i != kNone && x.v >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kRoom) {
        sh.v[at] = x.v;
        sh.i[at] = x.i;
      }
    }
  };
#pragma unroll
  for (int q = 0; q < kHeld; ++q) take(held[q]);
  for (int c = tid + kHeld * kThreads; c < total; c += kThreads)
    take(nth(c));
  __syncthreads();
  const int count = sh.count;
  if (count <= kRoom)
    best_of_room(count, K);
  else
    one_by_one_of_parts(&p, search);
  // Places: by rank; or (in_place, K = W) the first child of a beam keeps its
  // parent's place and the others take the free ones in order.
  if (p.in_place && tid == 0) {
    unsigned taken = 0, homes = 0;
    for (int r = 0; r < K; ++r) {
      if (sh.out_i[r] == kNone) continue;
      const unsigned w = static_cast<unsigned>(sh.out_i[r] >> 59);
      if (!(taken >> w & 1u)) {
        taken |= 1u << w;
        homes |= 1u << r;
        sh.place[r] = static_cast<int>(w);
      }
    }
    int next = 0;
    for (int r = 0; r < K; ++r) {
      if (homes >> r & 1u) continue;
      while (taken >> next & 1u) ++next;
      sh.place[r] = next++;
    }
  }
  // (K <= kThreads; the outputs may be the inputs' buffers: read, then written)
  static_assert(kBeamMaxKeep <= kThreads, "a thread per output");
  const bool some = tid < K && sh.out_i[tid] != kNone;
  const int w = some ? static_cast<int>(sh.out_i[tid] >> 59) : 0;
  const int token = some ? static_cast<int>(sh.out_i[tid] & kTokenMask) : -1;
  const int64_t row = static_cast<int64_t>(search) * W + w;
  const bool done = some && (token == p.eos || (p.finished && p.finished[row] != 0));
  __syncthreads();
  if (tid < K) {
    const int64_t at = static_cast<int64_t>(search) * K + (p.in_place ? sh.place[tid] : tid);
    p.out_scores[at] = some ? static_cast<float>(unordered64(sh.out_v[tid])) : -INFINITY;
    p.out_parents[at] = some ? static_cast<int32_t>(row) : -1;
    p.out_tokens[at] = token;
    if (p.out_finished) p.out_finished[at] = done;
  }
}

// Eight logits as words, from a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void load8_aligned(const T* at, uint32_t (&w)[Words<T>::N]) {
#pragma unroll
  for (int k = 0; k < Words<T>::N / 4; ++k) {
    const uint4 q = load_after_wait(reinterpret_cast<const uint4*>(at) + k);
    w[4 * k] = q.x;
    w[4 * k + 1] = q.y;
    w[4 * k + 2] = q.z;
    w[4 * k + 3] = q.w;
  }
}
// Those of a row from element e on, one by one; past its end they are -inf.
template <typename T>
__device__ __forceinline__ void load8_each(const T* row, int e, int end,
                                           uint32_t (&w)[Words<T>::N]) {
  T v[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (e + k < end) v[k] = row[e + k];
#pragma unroll
  for (int k = 0; k < Words<T>::N; ++k) w[k] = reinterpret_cast<const uint32_t*>(v)[k];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (e + k >= end) Words<T>::lowest(w, k);
}
// Those of a row off a 16-byte boundary: aligned words, shifted, where they lie within
// the addresses [lo, hi) that the logits span.
template <typename T>
__device__ __forceinline__ void load8_shifted(const T* row, int e, int end, uintptr_t lo,
                                              uintptr_t hi, uint32_t (&w)[Words<T>::N]) {
  constexpr int N = Words<T>::N;
  const uintptr_t addr = reinterpret_cast<uintptr_t>(row + e);
  const unsigned off = addr & 15u;  // the same for the whole row
  if (e + 8 <= end && addr - off >= lo && addr - off + 4 * N + 16 <= hi) {
    uint32_t u[N + 4];
    const uint4* a = reinterpret_cast<const uint4*>(addr - off);
#pragma unroll
    for (int k = 0; k < N / 4 + 1; ++k) {
      const uint4 q = load_after_wait(a + k);
      u[4 * k] = q.x;
      u[4 * k + 1] = q.y;
      u[4 * k + 2] = q.z;
      u[4 * k + 3] = q.w;
    }
    if (off & 8u) {
#pragma unroll
      for (int k = 0; k < N + 2; ++k) u[k] = u[k + 2];
    }
    if (off & 4u) {
#pragma unroll
      for (int k = 0; k < N + 1; ++k) u[k] = u[k + 1];
    }
    const unsigned sh = 8 * (off & 3u);
#pragma unroll
    for (int k = 0; k < N; ++k) w[k] = __funnelshift_r(u[k], u[k + 1], sh);
  } else {
    load8_each<T>(row, e, end, w);
  }
}

// grid (parts, rows).  P: pieces of eight logits that a thread takes of a block.
template <typename T, int P>
__global__ void __launch_bounds__(kThreads, kCtas)
    beam_select_kernel(const __grid_constant__ BeamParams p) {
  using W = Words<T>;
  Shared& sh = shared();
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = p.keep;
  const int64_t row = blockIdx.y;
  const int part = blockIdx.x, search = static_cast<int>(row / p.beams);
  const float score = load_after_wait(p.scores + row);
  if (part == 0 && tid == 0 && !isfinite(score) && score != -INFINITY)
    raise_error(p.err, PA_DEVERR_LOGITS);
  if (isfinite(score) && !(p.finished && load_after_wait(p.finished + row))) {
    constexpr int kBlock = P * kThreads * 8;
    const int begin = part * p.part_len, end = min(begin + p.part_len, p.vocab);
    const T* logits = static_cast<const T*>(p.logits);
    const T* mine = logits + row * p.row_stride;
    const bool aligned = (reinterpret_cast<uintptr_t>(mine) & 15) == 0;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(logits);
    const uintptr_t hi = reinterpret_cast<uintptr_t>(
        logits + (static_cast<int64_t>(gridDim.y) - 1) * p.row_stride + p.vocab);
    auto load = [&](int e, uint32_t (&w)[W::N]) {  // (begin is a multiple of 8)
      if (!aligned)
        load8_shifted<T>(mine, e, end, lo, hi, w);
      else if (e + 8 <= end)
        load8_aligned<T>(mine + e, w);
      else
        load8_each<T>(mine, e, end, w);
    };
    // the thread's maximum, and its sum of exp(x - maximum); NaN where a logit is NaN
    // or +inf
    float tm = -INFINITY;
    float2 s4[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
    const float2 unit = make_float2(kLog2e, kLog2e);
    const int blocks = (end - begin + kBlock - 1) / kBlock;
    uint32_t w[P][W::N];
#pragma unroll 1
    for (int b = 0; b < blocks; ++b) {
      const int e = begin + b * kBlock + tid * 8;
      if (aligned && begin + (b + 1) * kBlock <= end) {
#pragma unroll
        for (int j = 0; j < P; ++j) load8_aligned<T>(mine + e + j * kThreads * 8, w[j]);
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j) load(e + j * kThreads * 8, w[j]);
      }
      typename W::Top top = W::none();
#pragma unroll
      for (int j = 0; j < P; ++j) W::raise(top, w[j]);
      sh.tops[b][tid] = *reinterpret_cast<const uint32_t*>(&top);
      const float bm = W::value(top);
      if (bm > tm) {
        const float a = ex2((tm - bm) * kLog2e);
#pragma unroll
        for (int i = 0; i < 4; ++i) s4[i] = make_float2(s4[i].x * a, s4[i].y * a);
        tm = bm;
      }
      const float ref = tm == -INFINITY ? 0.f : -tm;
      const float2 ref2 = make_float2(ref, ref);
#pragma unroll
      for (int j = 0; j < P; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 d = __fmul2_rn(__fadd2_rn(W::pair(w[j], i), ref2), unit);
          s4[i] = __fadd2_rn(s4[i], make_float2(ex2(d.x), ex2(d.y)));
        }
    }
    const float2 a2 = __fadd2_rn(__fadd2_rn(s4[0], s4[1]), __fadd2_rn(s4[2], s4[3]));
    // the warp's
    float wm = tm;
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) wm = fmaxf(wm, __shfl_xor_sync(kFullMask, wm, m));
    float ws = a2.x + a2.y;
    if (tm > -INFINITY) ws *= ex2((tm - wm) * kLog2e);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) ws += __shfl_xor_sync(kFullMask, ws, m);
    // the groups' maxima
    const int lanes = kThreads / p.groups;
    float gm = tm;
    for (int m = 1; m < lanes; m <<= 1) gm = fmaxf(gm, __shfl_xor_sync(kFullMask, gm, m));
    if (tid % lanes == 0) sh.group_max[tid / lanes] = gm;
    if (lane == 0) {
      sh.m[warp] = wm;
      sh.s[warp] = ws;
    }
    if (tid == 0) sh.count = sh.hits = 0;
    if (__syncthreads_or(!(ws < INFINITY))) {
      // A NaN or +inf is no token: the part once more from memory, which hides them.
      if (tid == 0) raise_error(p.err, PA_DEVERR_LOGITS);
      tm = -INFINITY;
      for (int e = begin + tid; e < end; e += kThreads) tm = fmaxf(tm, visible(mine[e]));
      wm = tm;
      for (int m = 16; m >= 1; m >>= 1) wm = fmaxf(wm, __shfl_xor_sync(kFullMask, wm, m));
      ws = 0.f;
      if (wm > -INFINITY)
        for (int e = begin + tid; e < end; e += kThreads)
          ws += ex2((visible(mine[e]) - wm) * kLog2e);
      for (int m = 16; m >= 1; m >>= 1) ws += __shfl_xor_sync(kFullMask, ws, m);
      if (lane == 0) {
        sh.m[warp] = wm;
        sh.s[warp] = ws;
      }
      if (tid == 0) sh.count = kRoom + 1;  // (the largest one by one)
      __syncthreads();
    } else {
      // the K-th largest of the groups' maxima, and the logits that reach it
      kth_of_groups(sh.group_max, p.groups, K, &sh.bound);
      __syncthreads();
      // (at least the type's lowest number: what is hidden reaches nothing)
      const float bound =
          fmaxf(__uint_as_float(static_cast<uint32_t>(sh.bound)), Words<T>::kLowest);
      auto find = [&](const uint32_t (&w)[W::N], int e, int found) {
        uint32_t bits = W::reach(w, bound);
        if (bits == 0) return;
        int at = atomicAdd(&sh.count, found > 0 ? found : __popc(bits));
        for (; bits != 0; bits &= bits - 1, ++at)
          if (at < kRoom) {
            const int i = e + logit_of<T>(__ffs(bits) - 1);
            sh.i[at] = static_cast<uint64_t>(i);
            sh.v[at] = ordered(static_cast<float>(mine[i]));
          }
      };
      if constexpr (P == 1) {  // (the part is one piece a thread, still in registers)
        if (tm >= bound) find(w[0], begin + tid * 8, 0);
      } else {
        if (tm >= bound) {
          for (int b = 0; b < blocks; ++b) {
            const uint32_t top = sh.tops[b][tid];
            if (W::value(*reinterpret_cast<const typename W::Top*>(&top)) < bound) continue;
            const int at = atomicAdd(&sh.hits, 1);
            if (at < kHits) sh.hit[at] = static_cast<uint16_t>(b * kThreads + tid);
          }
        }
        __syncthreads();
        // those blocks' pieces once more, a thread each (too many: one by one below)
        const int hits = sh.hits;
        for (int c = tid; c < min(hits, kHits) * P; c += kThreads) {
          const int at_block = sh.hit[c / P], j = c % P;
          const int e = begin + (at_block / kThreads) * kBlock +
                        (j * kThreads + at_block % kThreads) * 8;
          uint32_t again[W::N];
          load(e, again);
          find(again, e, hits > kHits ? kRoom + 1 : 0);
        }
      }
      __syncthreads();
    }
    if (tid == kThreads - 1) {
      float m = sh.m[0];
      for (int q = 1; q < kWarps; ++q) m = fmaxf(m, sh.m[q]);
      float s = 0.f;
      if (m > -INFINITY)
        for (int q = 0; q < kWarps; ++q) s += sh.s[q] * ex2((sh.m[q] - m) * kLog2e);
      p.ws_sums[row * p.parts + part] = make_float2(m, s);
    }
    const int count = sh.count;
    if (count <= kRoom) {
      best_of_room(count, K);
    } else {
      one_by_one_of_row(mine, begin, end, K);
    }
    if (tid < K)
      p.ws_keys[(row * p.parts + part) * K + tid] =
          sh.out_i[tid] == kNone ? 0
                                 : (sh.out_v[tid] << 32) | ~static_cast<uint32_t>(sh.out_i[tid]);
  }
  // the last CTA of the search joins
  __syncthreads();
  if (tid == 0)
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                 : "=r"(sh.arrived)
                 : "l"(p.counters + search)
                 : "memory");
  __syncthreads();
  if (sh.arrived + 1 != static_cast<unsigned>(p.parts) * p.beams) return;
  merge(p, search);
  if (tid == 0) p.counters[search] = 0;
}

template <typename T, int P>
cudaError_t launch(const BeamParams& p, cudaStream_t stream) {
  const dim3 grid(p.parts, p.searches * p.beams);
  return launch_pdl(beam_select_kernel<T, P>, grid, dim3(kThreads), 0, stream, p);
}

template <typename T>
cudaError_t launch_t(const BeamParams& p, cudaStream_t stream) {
  if (p.part_len <= kThreads * 8) return launch<T, 1>(p, stream);
  return launch<T, sizeof(T) == 4 ? 2 : 4>(p, stream);
}

// Length of the parts that a row is cut into: one wave of CTAs, where that leaves a
// thread a piece and no part more than kMaxBlocks blocks.  (64 x 4 beams of 128,256
// tokens in 2 parts a row: 20.7 us; in 1 and 4, as waves of half and of twice as many
// would cut them: 24.6 and 23.8; 33 x 5 of 50,257 fp32 15.9, 21.0 and 17.8.)  Whole
// parts leave steps beside the wave's size: 304 rows 17.7 us, 308 25.4; 608 33.5, 612 46.6
// (0.058, 0.083, 0.055 and 0.076 us a row).
int beam_part_len(int rows, int vocab, int dtype) {
  const int least = kThreads * 8, most = (dtype == 2 ? 2 : 4) * least * kMaxBlocks;
  const int parts = std::max(1, std::min(kWave / std::max(rows, 1), (vocab + least - 1) / least));
  return std::min(((vocab + parts - 1) / parts + 7) / 8 * 8, most);
}

}  // namespace

int beam_parts(int rows, int vocab, int dtype) {
  const int len = beam_part_len(rows, vocab, dtype);
  return (vocab + len - 1) / len;
}

cudaError_t launch_beam_select(BeamParams p, int dtype, cudaStream_t stream) {
  p.part_len = beam_part_len(p.searches * p.beams, p.vocab, dtype);
  // (of G groups' maxima the K-th largest is reached by some G ln(G / (G - K)) logits:
  // twice K, 1.4 K; as many as K, K ln K and more than can be ranked by counting)
  static_assert(2 * kBeamMaxKeep <= kGroups, "groups");
  p.groups = 16;
  while (p.groups < 2 * p.keep) p.groups *= 2;
  switch (dtype) {
    case 0: return launch_t<__nv_bfloat16>(p, stream);
    case 1: return launch_t<__half>(p, stream);
    default: return launch_t<float>(p, stream);
  }
}

namespace {

bool beam_shape_ok(int num_searches, int num_beams, int num_keep, int vocab) {
  return num_beams <= kBeamMaxBeams && num_keep <= kBeamMaxKeep &&
         vocab <= kBeamMaxVocab &&
         static_cast<int64_t>(num_searches) * num_beams <= 65535;
}

pa_status beam_impl(float* scores_out, int32_t* parents_out, int32_t* tokens_out,
                    uint8_t* finished_out, const void* logits, int64_t row_stride, int dtype,
                    const float* scores, const uint8_t* finished, int eos_token,
                    int num_searches, int num_beams, int num_keep, int vocab, void* ws,
                    unsigned* counters, int flags, pa_stream_t stream, pa_prepared** keep) {
  if (num_searches < 0 || num_beams <= 0 || num_keep <= 0 || vocab <= 0 || dtype < 0 ||
      dtype > 2 || row_stride < vocab || row_stride > (1ll << 40) || eos_token < -1 ||
      eos_token >= vocab || (finished && eos_token < 0) || (flags & ~PA_BEAM_IN_PLACE) ||
      ((flags & PA_BEAM_IN_PLACE) && num_keep != num_beams))
    return PA_ERR_INVALID_ARG;
  if (!beam_shape_ok(num_searches, num_beams, num_keep, vocab)) return PA_ERR_UNSUPPORTED_SHAPE;
  if (num_searches == 0) return keep ? nothing_to_do(keep) : PA_OK;
  if (!aligned_ptr(scores_out, 4) || !aligned_ptr(parents_out, 4) || !aligned_ptr(tokens_out, 4) ||
      !aligned_ptr(logits, dtype == 2 ? 4 : 2) || !aligned_ptr(scores, 4) ||
      !aligned_ptr(ws, 16) || !aligned_ptr(counters, 4))
    return PA_ERR_INVALID_ARG;
  // an output may be the input of its kind only where a search's entries take its
  // own beams' places: the searches end at different times
  const int64_t in = static_cast<int64_t>(num_searches) * num_beams;
  const int64_t found = static_cast<int64_t>(num_searches) * num_keep;
  auto clash = [&](const void* o, const void* i, int64_t size) {
    return ranges_meet(o, found * size, i, in * size) && !(o == i && num_keep == num_beams);
  };
  if (clash(scores_out, scores, 4) || clash(finished_out, finished, 1)) return PA_ERR_INVALID_ARG;
  BeamParams p{};
  p.out_scores = scores_out;
  p.out_parents = parents_out;
  p.out_tokens = tokens_out;
  p.out_finished = finished_out;
  p.logits = logits;
  p.scores = scores;
  p.finished = finished;
  const int rows = num_searches * num_beams;
  p.parts = beam_parts(rows, vocab, dtype);
  p.ws_keys = static_cast<uint64_t*>(ws);
  p.ws_sums = reinterpret_cast<float2*>(p.ws_keys + static_cast<int64_t>(rows) * p.parts * num_keep);
  p.counters = counters;
  p.err = device_error_word();
  if (!p.err) return cuda_fail(cudaGetLastError());
  p.row_stride = row_stride;
  p.searches = num_searches;
  p.beams = num_beams;
  p.vocab = vocab;
  p.keep = num_keep;
  p.eos = eos_token;
  p.in_place = (flags & PA_BEAM_IN_PLACE) != 0;
  return launch_or_keep([=](cudaStream_t s) { return launch_beam_select(p, dtype, s); }, keep,
                        stream);
}

}  // namespace

}  // namespace pa

extern "C" size_t pa_beam_select_workspace_bytes(int num_searches, int num_beams, int num_keep,
                                                 int vocab, int dtype) {
  if (num_searches < 0 || num_beams <= 0 || num_keep <= 0 || vocab <= 0 || dtype < 0 ||
      dtype > 2 || !pa::beam_shape_ok(num_searches, num_beams, num_keep, vocab))
    return 0;
  const int rows = num_searches * num_beams;
  const size_t parts =
      static_cast<size_t>(rows) * (rows ? pa::beam_parts(rows, vocab, dtype) : 1);
  return (parts ? parts : 1) * (8 * static_cast<size_t>(num_keep) + 8);
}

extern "C" pa_status pa_beam_select(float* scores_out, int32_t* parents_out, int32_t* tokens_out,
                                    uint8_t* finished_out, const void* logits,
                                    int64_t row_stride, int dtype, const float* scores,
                                    const uint8_t* finished, int eos_token, int num_searches,
                                    int num_beams, int num_keep, int vocab, void* ws,
                                    unsigned* counters, int flags, pa_stream_t stream) {
  return pa::beam_impl(scores_out, parents_out, tokens_out, finished_out, logits, row_stride,
                       dtype, scores, finished, eos_token, num_searches, num_beams, num_keep,
                       vocab, ws, counters, flags, stream, nullptr);
}

extern "C" pa_status pa_prepare_beam_select(
    pa_prepared** prepared, float* scores_out, int32_t* parents_out, int32_t* tokens_out,
    uint8_t* finished_out, const void* logits, int64_t row_stride, int dtype, const float* scores,
    const uint8_t* finished, int eos_token, int num_searches, int num_beams, int num_keep,
    int vocab, void* ws, unsigned* counters, int flags) {
  if (!prepared) return PA_ERR_INVALID_ARG;
  *prepared = nullptr;
  return pa::beam_impl(scores_out, parents_out, tokens_out, finished_out, logits, row_stride,
                       dtype, scores, finished, eos_token, num_searches, num_beams, num_keep,
                       vocab, ws, counters, flags, nullptr, prepared);
}
