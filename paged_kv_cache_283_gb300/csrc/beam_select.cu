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
//  * A CTA takes a part of a row, E logits a thread, all in registers before
//    any is used.  256 threads form G >= K groups; the K-th largest of the
//    groups' maxima is a bound that at least K logits reach, and hardly more do
//    (of independent values some G ln G): those go to shared memory, where each
//    counts how many precede it.  Where many are equal (or G ln G is far above K)
//    more may reach the bound: then the K largest are taken one by one.
//  * Which thread holds which logit goes by its index in the row alone, not by
//    the row's alignment, so equal rows have equal sums, bit for bit, and equal
//    totals: ties go to the lower beam, then to the lower token.
//  * The last CTA of a search to arrive (a counter, zeroed again by it) joins
//    the parts.  Totals are taken and compared in 64 bits: sums of different
//    beams lie closer than fp32's 1e-6 often enough to be seen.
//
// A row whose address is no multiple of 16 bytes (an odd vocabulary) is read in
// aligned 16-byte words, shifted into place in registers.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "device.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRoom = 1024;   // candidates that a CTA can hold
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

template <typename T>
struct Words;  // eight logits in 32-bit words
template <>
struct Words<float> {
  static constexpr int N = 8;
  __device__ static float get(const uint32_t (&w)[8], int i) { return __uint_as_float(w[i]); }
  __device__ static void set(uint32_t (&w)[8], int i, float x) { w[i] = __float_as_uint(x); }
};
template <>
struct Words<__nv_bfloat16> {
  static constexpr int N = 4;
  __device__ static float get(const uint32_t (&w)[4], int i) {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
  __device__ static void set(uint32_t (&w)[4], int i, float x) {
    const uint32_t u = __bfloat16_as_ushort(__float2bfloat16_rn(x));
    w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | (u << 16) : (w[i / 2] & 0xffff0000u) | u;
  }
};
template <>
struct Words<__half> {
  static constexpr int N = 4;
  __device__ static float get(const uint32_t (&w)[4], int i) {
    const __half2 h = *reinterpret_cast<const __half2*>(&w[i / 2]);
    return i & 1 ? __high2float(h) : __low2float(h);
  }
  __device__ static void set(uint32_t (&w)[4], int i, float x) {
    const uint32_t u = __half_as_ushort(__float2half_rn(x));
    w[i / 2] = i & 1 ? (w[i / 2] & 0xffffu) | (u << 16) : (w[i / 2] & 0xffff0000u) | u;
  }
};

struct Shared {
  uint64_t v[kRoom];
  uint64_t i[kRoom];
  Key best[kWarps];
  Key last;
  float group_max[64];
  uint64_t group_key[64];
  float m[kWarps], s[kWarps];
  uint64_t bound;
  int count;
  unsigned arrived;
};

// The K largest of the CTA's keys, one by one: each thread offers through
// scan(prev) its largest key after `prev`.  For few threads' many equal values.
template <typename Scan, typename Emit>
__device__ void one_by_one(Shared& sh, int k, Scan&& scan, Emit&& emit) {
  Key prev{~0ull, 0};
  bool first = true;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = 0; r < k; ++r) {
    Key best = scan(prev, first);
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
      emit(r, best);
    }
    __syncthreads();
    prev = sh.last;
    first = false;
    if (prev.i == kNone) {  // no more
      for (int q = r + 1 + threadIdx.x; q < k; q += kThreads) emit(q, nothing());
      break;
    }
  }
  __syncthreads();
}

// The K first of sh.v / sh.i[0 .. count), count <= kRoom, to emit(rank, key).
template <typename Emit>
__device__ void best_of_room(Shared& sh, int count, int k, Emit&& emit) {
  if (count <= kRank) {
    for (int c = threadIdx.x; c < count; c += kThreads) {
      const Key mine{sh.v[c], sh.i[c]};
      int rank = 0;
      for (int o = 0; o < count; ++o) rank += before(Key{sh.v[o], sh.i[o]}, mine);
      if (rank < k) emit(rank, mine);
    }
    for (int r = count + threadIdx.x; r < k; r += kThreads) emit(r, nothing());
    __syncthreads();
  } else {
    one_by_one(
        sh, k,
        [&](const Key& prev, bool first) {
          Key best = nothing();
          for (int c = threadIdx.x; c < count; c += kThreads) {
            const Key x{sh.v[c], sh.i[c]};
            if ((first || before(prev, x)) && before(x, best)) best = x;
          }
          return best;
        },
        emit);
  }
}

// Joins the parts of a search: the last CTA's work.
__device__ void merge(const BeamParams& p, Shared& sh, int search) {
  __shared__ double lse[kBeamMaxBeams];
  __shared__ uint64_t out_v[kBeamMaxKeep];
  __shared__ uint64_t out_i[kBeamMaxKeep];
  const int tid = threadIdx.x, W = p.beams, K = p.keep;
  for (int w = tid >> 5; w < W; w += kWarps) {  // each row's log-sum from its parts
    const float2* ms = p.ws_sums + (static_cast<int64_t>(search) * W + w) * p.parts;
    float top = -INFINITY;
    for (int c = tid & 31; c < p.parts; c += 32) top = fmaxf(top, __ldcg(ms + c).x);
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, m));
    double s = 0.0;
    for (int c = tid & 31; c < p.parts; c += 32) {
      const float2 part = __ldcg(ms + c);
      if (part.y > 0.f)
        s += static_cast<double>(part.y) * exp(static_cast<double>(part.x) - top);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(kFullMask, s, m);
    if ((tid & 31) == 0) lse[w] = s > 0.0 ? static_cast<double>(top) + log(s) : 0.0;
  }
  if (tid == 0) sh.count = 0;
  __syncthreads();
  const int per_row = p.parts * K, total = W * per_row;
  auto candidate = [&](int c) -> Key {
    const int w = c / per_row;
    const int64_t row = static_cast<int64_t>(search) * W + w;
    const float score = p.scores[row];
    if (!isfinite(score)) return nothing();
    const uint64_t beam = static_cast<uint64_t>(w) << 59;
    if (p.finished && p.finished[row])  // its one continuation
      return c % per_row == 0
                 ? Key{ordered(static_cast<double>(score)), beam | static_cast<uint32_t>(p.eos)}
                 : nothing();
    const uint64_t key = __ldcg(p.ws_keys + row * per_row + c % per_row);
    if (key == 0) return nothing();
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    const double total = static_cast<double>(score) + (static_cast<double>(unordered(o)) - lse[w]);
    return Key{ordered(total), beam | static_cast<uint64_t>(~o) << 27 |
                                   static_cast<uint32_t>(~static_cast<uint32_t>(key))};
  };
  // the K-th largest of the groups' maxima bounds the K-th largest of all
  Key mine = nothing();
  for (int c = tid; c < total; c += kThreads) {
    const Key x = candidate(c);
    if (before(x, mine)) mine = x;
  }
  uint64_t gm = mine.v;
  const int lanes = kThreads / p.groups;
  for (int m = 1; m < lanes; m <<= 1) {
    const uint64_t o = __shfl_xor_sync(kFullMask, gm, m);
    gm = o > gm ? o : gm;
  }
  if (tid % lanes == 0) sh.group_key[tid / lanes] = gm;
  __syncthreads();
  if (tid < p.groups) {
    const uint64_t x = sh.group_key[tid];
    int rank = 0;
    for (int g = 0; g < p.groups; ++g)
      rank += sh.group_key[g] > x || (sh.group_key[g] == x && g < tid);
    if (rank == K - 1) sh.bound = x;
  }
  __syncthreads();
  const uint64_t bound = sh.bound;
  for (int c = tid; c < total; c += kThreads) {
    const Key x = candidate(c);
    if (x.i != kNone && x.v >= bound) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kRoom) {
        sh.v[at] = x.v;
        sh.i[at] = x.i;
      }
    }
  }
  __syncthreads();
  auto emit = [&](int r, const Key& k) {
    out_v[r] = k.v;
    out_i[r] = k.i;
  };
  if (sh.count <= kRoom) {
    best_of_room(sh, sh.count, K, emit);
  } else {
    one_by_one(
        sh, K,
        [&](const Key& prev, bool first) {
          Key best = nothing();
          for (int c = tid; c < total; c += kThreads) {
            const Key x = candidate(c);
            if ((first || before(prev, x)) && before(x, best)) best = x;
          }
          return best;
        },
        emit);
  }
  __syncthreads();
  // Places: by rank; or (in_place, K = W) the first child of a beam keeps its
  // parent's place and the others take the free ones in order.
  __shared__ int place[kBeamMaxKeep];
  if (tid == 0) {
    unsigned taken = 0, homes = 0;
    if (p.in_place) {
      for (int r = 0; r < K; ++r) {
        if (out_i[r] == kNone) continue;
        const unsigned w = static_cast<unsigned>(out_i[r] >> 59);
        if (!(taken >> w & 1u)) {
          taken |= 1u << w;
          homes |= 1u << r;
          place[r] = static_cast<int>(w);
        }
      }
      int next = 0;
      for (int r = 0; r < K; ++r) {
        if (homes >> r & 1u) continue;
        while (taken >> next & 1u) ++next;
        place[r] = next++;
      }
    } else {
      for (int r = 0; r < K; ++r) place[r] = r;
    }
  }
  __syncthreads();
  // (K <= kThreads; the outputs may be the inputs' buffers: read, then written)
  static_assert(kBeamMaxKeep <= kThreads, "a thread per output");
  const bool some = tid < K && out_i[tid] != kNone;
  const int w = some ? static_cast<int>(out_i[tid] >> 59) : 0;
  const int token = some ? static_cast<int>(out_i[tid] & kTokenMask) : -1;
  const int64_t row = static_cast<int64_t>(search) * W + w;
  const bool done = some && (token == p.eos || (p.finished && p.finished[row] != 0));
  __syncthreads();
  if (tid < K) {
    const int64_t at = static_cast<int64_t>(search) * K + place[tid];
    p.out_scores[at] = some ? static_cast<float>(unordered64(out_v[tid])) : -INFINITY;
    p.out_parents[at] = some ? static_cast<int32_t>(row) : -1;
    p.out_tokens[at] = token;
    if (p.out_finished) p.out_finished[at] = done;
  }
}

// Eight logits of a row from element e on, as words; those past the row's end
// are -inf.  lo / hi: the addresses that the logits' tensor spans.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int64_t e, int64_t end, uintptr_t lo,
                                      uintptr_t hi, uint32_t (&w)[Words<T>::N]) {
  constexpr int N = Words<T>::N;
  const uintptr_t addr = reinterpret_cast<uintptr_t>(row + e);
  const unsigned off = addr & 15u;  // the same for the whole row
  if (e + 8 <= end && off == 0) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(addr) + k);
      w[4 * k] = q.x;
      w[4 * k + 1] = q.y;
      w[4 * k + 2] = q.z;
      w[4 * k + 3] = q.w;
    }
  } else if (e + 8 <= end && addr - off >= lo && addr - off + 4 * N + 16 <= hi) {
    uint32_t u[N + 4];
    const uint4* a = reinterpret_cast<const uint4*>(addr - off);
#pragma unroll
    for (int k = 0; k < N / 4 + 1; ++k) {
      const uint4 q = __ldg(a + k);
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
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float x = -INFINITY;
      if (e + k < end) x = static_cast<float>(row[e + k]);
      Words<T>::set(w, k, x);
    }
  }
}

// grid (parts, rows).  V: pieces of eight logits a thread.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) beam_select_kernel(const BeamParams p) {
  using W = Words<T>;
  __shared__ Shared sh;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, K = p.keep;
  const int64_t row = blockIdx.y;
  const int part = blockIdx.x, search = static_cast<int>(row / p.beams);
  uint64_t* keys = p.ws_keys + (row * p.parts + part) * K;
  auto emit = [&](int r, const Key& k) {
    keys[r] = k.i == kNone ? 0 : (k.v << 32) | ~static_cast<uint32_t>(k.i);
  };
  const float score = p.scores[row];
  if (part == 0 && tid == 0 && !isfinite(score) && score != -INFINITY)
    raise_error(p.err, PA_DEVERR_LOGITS);
  if (isfinite(score) && !(p.finished && p.finished[row])) {
    const int64_t begin = static_cast<int64_t>(part) * p.part_len;
    const int64_t end = min(begin + p.part_len, static_cast<int64_t>(p.vocab));
    const T* logits = static_cast<const T*>(p.logits);
    const T* mine = logits + row * p.row_stride;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(logits);
    const uintptr_t hi = reinterpret_cast<uintptr_t>(
        logits + (static_cast<int64_t>(gridDim.y) - 1) * p.row_stride + p.vocab);
    uint32_t w[V][W::N];
#pragma unroll
    for (int j = 0; j < V; ++j)
      load8<T>(mine, begin + (j * kThreads + tid) * 8, end, lo, hi, w[j]);
    float tm = -INFINITY;  // the thread's maximum (NaN is passed over)
    auto maximum = [&]() {
      float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) m4[i & 3] = fmaxf(m4[i & 3], W::get(w[j], i));
      tm = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    };
    maximum();
    // sum of exp(x - m), m the warp's maximum; NaN where a logit is NaN or +inf
    float wm, ws;
    auto sum = [&]() {
      wm = tm;
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) wm = fmaxf(wm, __shfl_xor_sync(kFullMask, wm, m));
      const float ref = wm == -INFINITY ? 0.f : -wm;
      const float2 ref2 = make_float2(ref, ref), unit = make_float2(kLog2e, kLog2e);
      float2 s4[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float2 d = __fmul2_rn(
              __fadd2_rn(make_float2(W::get(w[j], i), W::get(w[j], i + 1)), ref2), unit);
          s4[i >> 1] = __fadd2_rn(s4[i >> 1], make_float2(ex2(d.x), ex2(d.y)));
        }
      const float2 a = __fadd2_rn(__fadd2_rn(s4[0], s4[1]), __fadd2_rn(s4[2], s4[3]));
      ws = a.x + a.y;
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) ws += __shfl_xor_sync(kFullMask, ws, m);
    };
    sum();
    if (!(ws < INFINITY)) {  // (the whole warp) a NaN or +inf: no token of the row's
      if (lane == 0) raise_error(p.err, PA_DEVERR_LOGITS);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (!(W::get(w[j], i) < INFINITY)) W::set(w[j], i, -INFINITY);
      maximum();
      sum();
    }
    // the groups' maxima, and their K-th largest
    const int lanes = kThreads / p.groups;
    float gm = tm;
    for (int m = 1; m < lanes; m <<= 1) gm = fmaxf(gm, __shfl_xor_sync(kFullMask, gm, m));
    if (tid % lanes == 0) sh.group_max[tid / lanes] = gm;
    if (lane == 0) {
      sh.m[warp] = wm;
      sh.s[warp] = ws;
    }
    if (tid == 0) sh.count = 0;
    __syncthreads();
    if (tid < p.groups) {
      const float x = sh.group_max[tid];
      int rank = 0;
      for (int g = 0; g < p.groups; ++g) {
        const float o = sh.group_max[g];
        rank += o > x || (o == x && g < tid);
      }
      if (rank == K - 1) sh.bound = __float_as_uint(x);
    }
    if (tid == kThreads - 1) {
      float m = sh.m[0];
      for (int q = 1; q < kWarps; ++q) m = fmaxf(m, sh.m[q]);
      float s = 0.f;
      if (m > -INFINITY)
        for (int q = 0; q < kWarps; ++q) s += sh.s[q] * ex2((sh.m[q] - m) * kLog2e);
      p.ws_sums[row * p.parts + part] = make_float2(m, s);
    }
    __syncthreads();
    const float bound = __uint_as_float(static_cast<uint32_t>(sh.bound));
    if (tm >= bound) {
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = W::get(w[j], i);
          if (x >= bound && x > -INFINITY) {
            const int at = atomicAdd(&sh.count, 1);
            if (at < kRoom) {
              sh.v[at] = ordered(x);
              sh.i[at] = static_cast<uint64_t>(begin + (j * kThreads + tid) * 8 + i);
            }
          }
        }
    }
    __syncthreads();
    if (sh.count <= kRoom) {
      best_of_room(sh, sh.count, K, emit);
    } else {
      one_by_one(
          sh, K,
          [&](const Key& prev, bool first) {
            Key best = nothing();
#pragma unroll
            for (int j = 0; j < V; ++j)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float x = W::get(w[j], i);
                const Key k{ordered(x),
                            static_cast<uint64_t>(begin + (j * kThreads + tid) * 8 + i)};
                if (x > -INFINITY && (first || before(prev, k)) && before(k, best)) best = k;
              }
            return best;
          },
          emit);
    }
  }
  // the last CTA of the search joins
  __threadfence();
  __syncthreads();
  if (tid == 0)
    sh.arrived = atomicAdd(p.counters + search, 1u);
  __syncthreads();
  if (sh.arrived + 1 != static_cast<unsigned>(p.parts) * p.beams) return;
  __threadfence();
  merge(p, sh, search);
  if (tid == 0) p.counters[search] = 0;
}

template <typename T, int V>
cudaError_t launch(const BeamParams& p, cudaStream_t stream) {
  const dim3 grid(p.parts, p.searches * p.beams);
  return launch_pdl(beam_select_kernel<T, V>, grid, dim3(kThreads), 0, stream, p);
}

template <typename T>
cudaError_t launch_t(const BeamParams& p, int pieces, cudaStream_t stream) {
  switch (pieces) {
    case 1: return launch<T, 1>(p, stream);
    case 2: return launch<T, 2>(p, stream);
    case 4: return launch<T, 4>(p, stream);
    default:
      if constexpr (sizeof(T) == 2) return launch<T, 8>(p, stream);
      return launch<T, 4>(p, stream);
  }
}

}  // namespace

// Pieces of eight logits a thread: as many as leave the GPU enough CTAs.
int beam_pieces(int rows, int vocab, int dtype) {
  const int most = dtype == 2 ? 4 : 8;
  int v = 1;
  while (v < most && static_cast<int64_t>(rows) * ((vocab + kThreads * 16 * v - 1) /
                                                    (kThreads * 16 * v)) >= 608)
    v *= 2;
  return v;
}

int beam_parts(int rows, int vocab, int dtype) {
  const int per = kThreads * 8 * beam_pieces(rows, vocab, dtype);
  return (vocab + per - 1) / per;
}

cudaError_t launch_beam_select(BeamParams p, int dtype, cudaStream_t stream) {
  const int rows = p.searches * p.beams;
  const int pieces = beam_pieces(rows, p.vocab, dtype);
  // parts of equal length, whole pieces
  p.part_len = (((p.vocab + p.parts - 1) / p.parts) + 7) / 8 * 8;
  p.groups = 8;
  while (p.groups < p.keep) p.groups *= 2;
  switch (dtype) {
    case 0: return launch_t<__nv_bfloat16>(p, pieces, stream);
    case 1: return launch_t<__half>(p, pieces, stream);
    default: return launch_t<float>(p, pieces, stream);
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
  if (num_keep != num_beams &&
      (scores_out == scores || (finished_out && finished_out == finished)))
    return PA_ERR_INVALID_ARG;
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
