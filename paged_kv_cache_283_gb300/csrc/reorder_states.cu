// Rows of state tensors moved to where their parents went, in place
// (pa_reorder_states): after a beam search's selection, row i of each group of
// `beams` rows becomes what row parents[i] of the group was.
//
// Pure data movement: each row that changes is written once and each distinct
// parent of such a row is read once; rows that keep their place are not touched.
// A CTA owns a column of a group (its rows' bytes [c0, c0 + chunk)): it first
// brings the parents' parts of the column into shared memory, all copies in
// flight together, and only then writes, so that a row may be the parent of one
// and the child of another.

#include <cuda_runtime.h>
#include <stdint.h>

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

// grid (columns, groups, tensors); V: bytes moved by one instruction.
template <int V>
__global__ void __launch_bounds__(kThreads) reorder_states_kernel(const ReorderParams p) {
  using T = typename Piece<V>::type;
  extern __shared__ uint4 smem4[];
  T* buf = reinterpret_cast<T*>(smem4);  // [beams][chunk]
  __shared__ int parent_of[kReorderMaxBeams];
  __shared__ unsigned needed;  // rows that a changed row comes from
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, W = p.beams;
  const int64_t group = blockIdx.y;
  if (tid < 32) {
    int par = -1;
    if (tid < W) {
      const int64_t g = __ldg(p.parents + group * W + tid);
      const int64_t local = g - group * W;
      if (g >= 0) {
        if (local < 0 || local >= W) {  // another group's row, or none: left as it is
          if (blockIdx.x == 0 && blockIdx.z == 0) raise_error(p.err, PA_DEVERR_PARENT);
        } else if (local != tid) {
          par = static_cast<int>(local);
        }
      }
      parent_of[tid] = par;
    }
    const unsigned bits = __reduce_or_sync(kFullMask, par >= 0 ? 1u << par : 0u);
    if (tid == 0) needed = bits;
  }
  __syncthreads();
  if (needed == 0) return;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.chunk), p.row_bytes - c0)) / V;
  char* base = static_cast<char*>(p.states[blockIdx.z]) + group * W * p.row_stride + c0;
  const int per_row = p.chunk / V;
  for (int w = 0; w < W; ++w) {
    if (!(needed >> w & 1u)) continue;
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

cudaError_t launch_reorder_states(ReorderParams p, int groups, int tensors, int vec,
                                  cudaStream_t stream) {
  // 32 KiB of shared memory: seven CTAs an SM
  int beams = 4;
  while (beams < p.beams) beams *= 2;
  p.chunk = 32768 / beams;
  const int64_t columns = (p.row_bytes + p.chunk - 1) / p.chunk;
  const dim3 grid(static_cast<unsigned>(columns), groups, tensors);
  const size_t smem = static_cast<size_t>(p.beams) * p.chunk;
  switch (vec) {
    case 16: return launch_pdl(reorder_states_kernel<16>, grid, dim3(kThreads), smem, stream, p);
    case 2: return launch_pdl(reorder_states_kernel<2>, grid, dim3(kThreads), smem, stream, p);
    case 4: return launch_pdl(reorder_states_kernel<4>, grid, dim3(kThreads), smem, stream, p);
    default: return launch_pdl(reorder_states_kernel<1>, grid, dim3(kThreads), smem, stream, p);
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
