// Rows of state tensors moved to where their parents went, in place
// (pa_reorder_states): after a beam search's selection, row i of each group of
// `beams` rows becomes what row parents[i] of the group was.
//
// Pure data movement: each row that changes is written once and each distinct
// parent of such a row is read once; rows that keep their place are not touched.
// A CTA owns a column of a group: it first brings the parents' parts of the column
// in (registers for few beams, shared memory for many), all loads in flight
// together, and only then writes, so that a row may be the parent of one and the
// child of another.

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <new>
#include <utility>
#include <vector>

#include "device.cuh"
#include "internal.h"

namespace pa {

namespace {

constexpr int kThreads = 256;

template <int V>
struct Piece;
template <>
struct Piece<16> {
  using type = uint4;
};
template <>
struct Piece<4> {
  using type = uint32_t;
};
template <>
struct Piece<2> {
  using type = uint16_t;
};
template <>
struct Piece<1> {
  using type = uint8_t;
};

// The parents of a group's rows: parent_of[w] is -1 for a row that stays, and
// children[w] the rows that row w goes to.  By the first warp.
__device__ __forceinline__ void read_parents(const ReorderParams& p, int64_t group, bool report,
                                             int* parent_of, unsigned* children) {
  const int lane = threadIdx.x, W = p.beams;
  int par = -1;
  if (lane < W) {
    const int64_t g = load_after_wait(p.parents + group * W + lane);
    const int64_t local = g - group * W;
    if (g >= 0) {
      if (local < 0 || local >= W) {  // another group's row, or none: left as it is
        if (report) raise_error(p.err, PA_DEVERR_PARENT);
      } else if (local != lane) {
        par = static_cast<int>(local);
      }
    }
  }
  if (parent_of) parent_of[lane] = par;
  for (int w = 0; w < W; ++w) {
    const unsigned mask = __ballot_sync(kFullMask, par == w);
    if (lane == w) children[w] = mask;
  }
}

// Up to M beams in registers: a thread has its pieces of every parent before it
// stores any, and its pieces are no other thread's.  grid (columns, groups, tensors);
// V: bytes of a piece.  (8 x 64 rows of 512 KiB, 4 beams: 26.8 us, 0.94 of the copy rate,
// against the 78 of the kernel below; tables of 64 x 4 rows of 2 KiB 3.0 against 2.6.)
//
// Rows whose addresses, sizes and strides share 16 bytes go in pieces of 16, others in
// pieces of 4, 2 or 1.  8 x 512 rows of 64 KiB, of the copy rate, by what they share,
// 16, 8 or 4, 2 and 1 bytes: 0.98, 0.95, 0.74, 0.44 in groups of 4; 0.98, 0.96, 0.70, 0.39
// of 8; by the kernel below 0.84, 0.71, 0.45, 0.37 of 16; 0.54, 0.44, 0.28, 0.28 of 32.
template <int V, int M, int U>
__global__ void __launch_bounds__(kThreads) reorder_few_kernel(const ReorderParams p) {
  using T = typename Piece<V>::type;
  __shared__ unsigned children[kReorderMaxBeams];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t group = blockIdx.y;
  if (threadIdx.x < 32)
    read_parents(p, group, blockIdx.x == 0 && blockIdx.z == 0, nullptr, children);
  __syncthreads();
  unsigned to[M];
#pragma unroll
  for (int w = 0; w < M; ++w) to[w] = w < p.beams ? children[w] : 0;
  const int64_t n = p.row_bytes / V;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (U * kThreads) + threadIdx.x;
  char* base = static_cast<char*>(p.states[blockIdx.z]) + group * p.beams * p.row_stride;
  T v[M][U];
#pragma unroll
  for (int w = 0; w < M; ++w) {
    if (to[w] == 0) continue;
    const T* src = reinterpret_cast<const T*>(base + w * p.row_stride);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (first + u * kThreads < n) v[w][u] = src[first + u * kThreads];
  }
#pragma unroll
  for (int w = 0; w < M; ++w) {
    for (unsigned mask = to[w]; mask != 0; mask &= mask - 1) {
      T* dst = reinterpret_cast<T*>(base + (__ffs(mask) - 1) * p.row_stride);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (first + u * kThreads < n) dst[first + u * kThreads] = v[w][u];
    }
  }
}

// Any number of beams.  grid (columns, groups, tensors); V: bytes of a piece.
template <int V>
__global__ void __launch_bounds__(kThreads) reorder_states_kernel(const ReorderParams p) {
  using T = typename Piece<V>::type;
  extern __shared__ uint4 smem4[];
  T* buf = reinterpret_cast<T*>(smem4);  // [beams][chunk]
  __shared__ int parent_of[kReorderMaxBeams];
  __shared__ unsigned children[kReorderMaxBeams];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, W = p.beams;
  const int64_t group = blockIdx.y;
  if (tid < 32)
    read_parents(p, group, blockIdx.x == 0 && blockIdx.z == 0, parent_of, children);
  __syncthreads();
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.chunk), p.row_bytes - c0)) / V;
  char* base = static_cast<char*>(p.states[blockIdx.z]) + group * W * p.row_stride + c0;
  const int per_row = p.chunk / V;
  for (int w = 0; w < W; ++w) {
    if (children[w] == 0) continue;
    const T* src = reinterpret_cast<const T*>(base + w * p.row_stride);
    if constexpr (V >= 4) {
      for (int i = tid; i < n; i += kThreads)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(
                         smem_u32(buf + w * per_row + i)),
                     "l"(src + i), "n"(V)
                     : "memory");
    } else {  // too narrow for an asynchronous copy: eight loads in flight
      for (int i0 = tid; i0 < n; i0 += 8 * kThreads) {
        T v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i0 + k * kThreads < n) v[k] = src[i0 + k * kThreads];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (i0 + k * kThreads < n) buf[w * per_row + i0 + k * kThreads] = v[k];
      }
    }
  }
  if constexpr (V >= 4) asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  for (int w = 0; w < W; ++w) {
    const int par = parent_of[w];
    if (par < 0) continue;
    T* dst = reinterpret_cast<T*>(base + w * p.row_stride);
    for (int i = tid; i < n; i += kThreads) dst[i] = buf[par * per_row + i];
  }
}

}  // namespace

namespace {

template <int V>
cudaError_t launch(ReorderParams p, int groups, int tensors, cudaStream_t stream) {
  if (p.beams <= 8) {
    // 4 pieces a thread of up to 4 rows, 2 of up to 8
    const int64_t per = static_cast<int64_t>(V) * kThreads * (p.beams <= 4 ? 4 : 2);
    const dim3 grid(static_cast<unsigned>((p.row_bytes + per - 1) / per), groups, tensors);
    return p.beams <= 4
               ? launch_pdl(reorder_few_kernel<V, 4, 4>, grid, dim3(kThreads), 0, stream, p)
               : launch_pdl(reorder_few_kernel<V, 8, 2>, grid, dim3(kThreads), 0, stream, p);
  }
  // 32 KiB of shared memory: seven CTAs an SM
  int beams = 16;
  while (beams < p.beams) beams *= 2;
  p.chunk = 32768 / beams;
  const dim3 grid(static_cast<unsigned>((p.row_bytes + p.chunk - 1) / p.chunk), groups, tensors);
  const size_t smem = static_cast<size_t>(p.beams) * p.chunk;
  return launch_pdl(reorder_states_kernel<V>, grid, dim3(kThreads), smem, stream, p);
}

}  // namespace

cudaError_t launch_reorder_states(ReorderParams p, int groups, int tensors, int vec,
                                  cudaStream_t stream) {
  switch (vec) {
    case 16: return launch<16>(p, groups, tensors, stream);
    case 4: return launch<4>(p, groups, tensors, stream);
    case 2: return launch<2>(p, groups, tensors, stream);
    default: return launch<1>(p, groups, tensors, stream);
  }
}

namespace {

// One launch for each kReorderMaxTensors tensors, kept whole by a prepared call.
struct Launches {
  std::vector<std::pair<ReorderParams, int>> parts;  // (parameters, tensors)
  int groups, vec;
  cudaError_t operator()(cudaStream_t stream) const {
    for (const auto& part : parts) {
      const cudaError_t e = launch_reorder_states(part.first, groups, part.second, vec, stream);
      if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
  }
};

// Whether two tensors' rows, or a row and the parents, share bytes: each tensor is
// moved by CTAs of its own, and none may change what another still reads.
bool any_meet(void* const* states, int num_tensors, const int32_t* parents, int64_t rows,
              int64_t row_bytes, int64_t row_stride) {
  const int64_t extent = (rows - 1) * row_stride + row_bytes;
  std::vector<uintptr_t> at(num_tensors);
  for (int t = 0; t < num_tensors; ++t) {
    at[t] = reinterpret_cast<uintptr_t>(states[t]);
    if (ranges_meet(states[t], extent, parents, 4 * rows)) return true;
  }
  std::sort(at.begin(), at.end());
  for (int i = 0; i < num_tensors; ++i)
    for (int j = i + 1; j < num_tensors && at[j] - at[i] < static_cast<uintptr_t>(extent); ++j)
      if (rows_meet(reinterpret_cast<void*>(at[i]), reinterpret_cast<void*>(at[j]), rows,
                    row_bytes, row_stride))
        return true;
  return false;
}

pa_status reorder_impl(void* const* states, int num_tensors, const int32_t* parents,
                       int num_groups, int num_beams, int64_t row_bytes, int64_t row_stride,
                       pa_stream_t stream, pa_prepared** keep) {
  if (num_tensors < 0 || num_groups < 0 || num_beams <= 0 || row_bytes < 0 ||
      row_stride < row_bytes)
    return PA_ERR_INVALID_ARG;
  if (num_beams > kReorderMaxBeams || num_groups > 65535 || row_bytes > (1ll << 40) ||
      row_stride > (1ll << 40))
    return PA_ERR_UNSUPPORTED_SHAPE;
  if (num_tensors == 0 || num_groups == 0 || row_bytes == 0)
    return keep ? nothing_to_do(keep) : PA_OK;
  if (!states || !aligned_ptr(parents, 4)) return PA_ERR_INVALID_ARG;
  uintptr_t bits = static_cast<uintptr_t>(row_bytes) | static_cast<uintptr_t>(row_stride);
  for (int t = 0; t < num_tensors; ++t) {
    if (!states[t]) return PA_ERR_INVALID_ARG;
    bits |= reinterpret_cast<uintptr_t>(states[t]);
  }
  try {
    if (any_meet(states, num_tensors, parents, static_cast<int64_t>(num_groups) * num_beams,
                 row_bytes, row_stride))
      return PA_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return PA_ERR_INVALID_ARG;
  }
  ReorderParams p{};
  p.parents = parents;
  p.err = device_error_word();
  if (!p.err) return cuda_fail(cudaGetLastError());
  p.row_bytes = row_bytes;
  p.row_stride = row_stride;
  p.beams = num_beams;
  try {
    Launches all;
    all.groups = num_groups;
    all.vec = bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : bits % 2 == 0 ? 2 : 1;
    for (int t0 = 0; t0 < num_tensors; t0 += kReorderMaxTensors) {
      const int n = num_tensors - t0 < kReorderMaxTensors ? num_tensors - t0 : kReorderMaxTensors;
      for (int t = 0; t < n; ++t) p.states[t] = states[t0 + t];
      all.parts.emplace_back(p, n);
    }
    return launch_or_keep(std::move(all), keep, stream);
  } catch (const std::bad_alloc&) {
    return PA_ERR_INVALID_ARG;
  }
}

}  // namespace

}  // namespace pa

extern "C" pa_status pa_reorder_states(void* const* states, int num_tensors,
                                       const int32_t* parents, int num_groups, int num_beams,
                                       int64_t row_bytes, int64_t row_stride,
                                       pa_stream_t stream) {
  return pa::reorder_impl(states, num_tensors, parents, num_groups, num_beams, row_bytes,
                          row_stride, stream, nullptr);
}

extern "C" pa_status pa_prepare_reorder_states(pa_prepared** prepared, void* const* states,
                                               int num_tensors, const int32_t* parents,
                                               int num_groups, int num_beams, int64_t row_bytes,
                                               int64_t row_stride) {
  if (!prepared) return PA_ERR_INVALID_ARG;
  *prepared = nullptr;
  return pa::reorder_impl(states, num_tensors, parents, num_groups, num_beams, row_bytes,
                          row_stride, nullptr, prepared);
}
