// Paged decode attention over a 4-bit cache with the batch's work cut evenly
// among the GPU's warps, sm_103a: the launch for large batches of long contexts.
//
// The partitioned kernel (decode_kernel.cuh) gives every CTA a partition of one
// sequence.  A 4-bit cache is quickly read, and what its CTAs cost beside that --
// a second wave, the tail of the longest, each one's start and merge -- grows to
// half of a long launch.  Here the launch is one wave of resident CTAs.  A unit
// is the context of one (sequence, KV head), counted in steps of 64 tokens after
// kEvenUnitSteps more that stand for its beginning and end; the units stand in a
// row, and warp w of N takes the places [w W / N, (w + 1) W / N) of all W: every
// warp the same number, whatever the lengths, with no plan made on the host.
// Warps work alone: each finds its place from the context lengths, copies its
// tiles through its own ring of bulk copies that runs on over the ends of units,
// and keeps its own softmax.
//
// A unit inside one warp's range goes straight to the output.  A unit that
// spans several leaves one partial (m, l, sum p v) per warp in the workspace,
// and the last warp to arrive at it merges them in warp order (so the result
// does not depend on who is last): up to 32 partials at one counter; those of a
// longer unit first inside groups of 16 consecutive warps, then over the groups.
// Nobody waits for another warp, and every counter is left at zero.
//
// Measured (32 query / 8 KV heads, D = 128): 8 contexts of 8K to 50K tokens 47.6
// us against 53.7 in the best partitions (33.0 at the copy rate); 8 of 128K tokens
// 193 us (178); 64 of 128 to 2048 tokens 22.0 against 20.1: a warp's share must
// outweigh its merges, see the binding's rule.  Steps of 64 tokens with three
// CTAs an SM (168 registers a thread); 32 with four (128 registers) take 196 us
// for the 8 x 128K and 69.8 against 66.9 for 8 x 40,000; 96 with two 187 for the
// former, but 122 against 106 for 500 short ones and, with D = 64, 93 against 71
// for 64 of 4K to 16K tokens.
#include "decode_kernel.cuh"

namespace pa {

namespace {

constexpr int kEvenWarps = 4;   // warps of a CTA
// A unit's partials are merged by one warp up to kEvenFlat of them; past that
// first in groups of kEvenGroup consecutive warps, then group by group.
constexpr int kEvenFlat = 32;
constexpr int kEvenGroup = 16;
// fewer steps than this to a warp (while every unit has one) do not pay
constexpr int kEvenMinSteps = 4;
// what beginning a unit (its q, its result) costs a warp, in steps
constexpr int kEvenUnitSteps = 2;
// blocks per step
constexpr int kEvenBlocks = 4;

template <int D, int G>
struct Even {
  static constexpr int S = 2;     // ring stages of a warp
  static constexpr int CTAS = 3;  // per SM
  static constexpr int KT = int4_tile_bytes(D);
  static constexpr int STAGE = kEvenBlocks * 2 * KT;
  static constexpr int RING = S * STAGE;
  static constexpr int PATCH = 512;  // fused step: the new row (fused_cache_write)
  static constexpr int WARP = (RING + PATCH + S * 8 + 127) / 128 * 128;
  static constexpr int SMEM = kEvenWarps * WARP;
  // a lane's share of a unit's result: V sums of p v and (m, l) of H heads
  static constexpr int H = Warp4<D, G>::H, V = Warp4<D, G>::V;
  static constexpr int SLOT = 32 * (V + 2 * H);  // floats of a partial in the workspace
};

struct EvenArgs {
  float* ws;           // [2 * warps][SLOT]
  unsigned* unit_cnt;  // [num_seqs * num_kv_heads]
  unsigned* group_cnt; // [2 * groups]
  int warps;           // of the grid
};

// A result (v and ml: Warp4::finish) written out; o: its unit's first head's row.
template <int D, int G>
__device__ __forceinline__ void even_write_out(__nv_bfloat16* o, int lane,
                                               const float (&v)[Even<D, G>::V],
                                               const float2 (&ml)[Even<D, G>::H]) {
  using E = Even<D, G>;
  float inv[E::H];
#pragma unroll
  for (int h = 0; h < E::H; ++h) inv[h] = 1.0f / ml[h].y;
  const int gid = lane >> 2, tig = lane & 3;
  if (Warp4<D, G>::owner(tig)) {
#pragma unroll
    for (int h = 0; h < E::H; ++h) {
      __nv_bfloat16* oh = o + Warp4<D, G>::head(tig, h) * D + gid;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) oh[8 * c] = __float2bfloat16_rn(v[c * E::H + h] * inv[h]);
    }
  }
}

template <int D, int G>
__device__ __forceinline__ void even_store(float* slot, int lane,
                                           const float (&v)[Even<D, G>::V],
                                           const float2 (&ml)[Even<D, G>::H]) {
  using E = Even<D, G>;
#pragma unroll
  for (int i = 0; i < E::V / 4; ++i)
    __stcg(reinterpret_cast<float4*>(slot) + 32 * i + lane,
           make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
#pragma unroll
  for (int h = 0; h < E::H; ++h)
    __stcg(reinterpret_cast<float2*>(slot + 32 * E::V) + 32 * h + lane, ml[h]);
}

// The slot of warp w's partial of the unit that begins in warp wf.
template <int D, int G>
__device__ __forceinline__ float* even_slot(float* ws, int wf, int w) {
  return ws + static_cast<size_t>(2 * w + (w == wf ? 1 : 0)) * Even<D, G>::SLOT;
}

// `count` partials of one unit, of the warps max(wf, first + i stride), merged in
// order, each weighed against the running maximum; the result goes out (o), or
// (o null) into the first of their slots.  A call of its own, so that the many
// loads it has in flight take no registers from the loop over the steps.
template <int D, int G>
__device__ __noinline__ void even_merge(float* ws, int wf, int first, int stride, int count,
                                        __nv_bfloat16* o) {
  using E = Even<D, G>;
  constexpr int U = 4;  // loaded together
  const int lane = threadIdx.x & 31;
  float v[E::V];
  float2 ml[E::H];
#pragma unroll
  for (int e = 0; e < E::V; ++e) v[e] = 0.f;
#pragma unroll
  for (int h = 0; h < E::H; ++h) ml[h] = make_float2(-INFINITY, 0.f);
  for (int i0 = 0; i0 < count; i0 += U) {
    float4 x[U][E::V / 4];
    float2 y[U][E::H];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // (past the last: the last again, not counted below)
      const int i = min(i0 + u, count - 1);
      const float* slot = even_slot<D, G>(ws, wf, max(wf, first + i * stride));
#pragma unroll
      for (int k = 0; k < E::V / 4; ++k)
        x[u][k] = __ldcg(reinterpret_cast<const float4*>(slot) + 32 * k + lane);
#pragma unroll
      for (int h = 0; h < E::H; ++h)
        y[u][h] = __ldcg(reinterpret_cast<const float2*>(slot + 32 * E::V) + 32 * h + lane);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u >= count) break;
      float a[E::H], c[E::H];
#pragma unroll
      for (int h = 0; h < E::H; ++h) {
        const float m = fmaxf(ml[h].x, y[u][h].x);
        a[h] = ml[h].x == m ? 1.f : exp2f(ml[h].x - m);  // (both -inf: 1)
        c[h] = y[u][h].x == m ? 1.f : exp2f(y[u][h].x - m);
        ml[h] = make_float2(m, ml[h].y * a[h] + y[u][h].y * c[h]);
      }
#pragma unroll
      for (int i = 0; i < E::V / 4; ++i) {
        const float xs[4] = {x[u][i].x, x[u][i].y, x[u][i].z, x[u][i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int e = 4 * i + k, h = e % E::H;
          v[e] = v[e] * a[h] + xs[k] * c[h];
        }
      }
    }
  }
  if (o != nullptr)
    even_write_out<D, G>(o, lane, v, ml);
  else
    even_store<D, G>(even_slot<D, G>(ws, wf, max(wf, first)), lane, v, ml);
}

template <int D, int G>
__global__ void __launch_bounds__(kEvenWarps * 32, (Even<D, G>::CTAS))
    paged_decode_even_kernel(const DecodeParams p, const EvenArgs ev) {
  using E = Even<D, G>;
  constexpr int S = E::S, SB = kEvenBlocks, BS = kBlockSize, WS = 32 / SB;
  constexpr int C = kEvenUnitSteps;
  extern __shared__ __align__(128) unsigned char smem[];
  if (!p.early_read) griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // consecutive ranges go to different SMs: a small batch spreads over them
  const int me = warp * gridDim.x + blockIdx.x;
  unsigned char* wbase = smem + warp * E::WARP;
  unsigned char* tiles = wbase;
  unsigned char* patch = wbase + E::RING;
  uint64_t* bars = reinterpret_cast<uint64_t*>(patch + E::PATCH);
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
  }
  __syncwarp();

  // A sequence's context, clamped to its table, in tokens, blocks and steps.
  const int B = p.num_seqs, hkv = p.num_kv_heads;
  const int cap = p.max_blocks_per_seq * BS;
  struct Seq {
    int ctx, nblk, T;
  };
  auto seq_at = [&](int b) {
    Seq q;
    q.ctx = max(0, min(__ldg(p.context_lens + b), cap));
    q.nblk = (q.ctx + BS - 1) / BS;
    q.T = (q.nblk + SB - 1) / SB;
    return q;
  };
  // Lane l sums the sequences [l K, (l + 1) K): their steps, and how many are
  // not empty.
  const int K = (B + 31) / 32;
  int sum = 0, some = 0;
  bool bad = false;
  for (int i = 0; i < K; ++i) {
    const int b = lane * K + i;
    if (b < B) {
      const int T = seq_at(b).T;
      sum += T > 0 ? T + C : 0;
      some += T > 0;
      if (me == 0) {
        const int c = __ldg(p.context_lens + b);
        bad |= c < 0 || c > cap;
      }
    }
  }
  if (bad) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
  int incl = sum;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int up = __shfl_up_sync(kFullMask, incl, m);
    if (lane >= m) incl += up;
    some += __shfl_xor_sync(kFullMask, some, m);
  }
  const int excl = incl - sum;
  // (W fits 31 bits: the launcher bounds the tables' steps)
  const int W = __shfl_sync(kFullMask, incl, 31) * hkv;
  const int N = min(ev.warps, max(W / kEvenMinSteps, some * hkv));
  auto start_of = [&](int w) {  // warp w's first step (N >= 1)
    return static_cast<int>(static_cast<int64_t>(w) * W / N);
  };
  auto warp_of = [&](int step) {  // the last warp that starts at or before a step
    return static_cast<int>(((step + 1ll) * N - 1) / W);
  };
  const bool work = me < N;  // then W >= N >= 1
  const int v0 = work ? start_of(me) : 0, v1 = work ? start_of(me + 1) : 0;

  // A unit (b, h) in the row: its T steps stand at the places v + C .. v + C + T -
  // 1; rem: its blocks.
  struct Place {
    int b, h, v, T, rem;
  };
  auto set_seq = [&](Place& x) {
    const Seq q = seq_at(x.b);
    x.T = q.T;
    x.rem = q.nblk;
  };
  Place at{};
  if (work) {
    const int tb = v0 / hkv;  // places of one head before it
    const int owner = __ffs(__ballot_sync(kFullMask, excl <= tb && tb < excl + sum)) - 1;
    int run = __shfl_sync(kFullMask, excl, owner);
    at.b = owner * K;
    set_seq(at);
    while (at.T == 0 || tb >= run + at.T + C) {
      run += at.T > 0 ? at.T + C : 0;
      ++at.b;
      set_seq(at);
    }
    at.h = (v0 - run * hkv) / (at.T + C);
    at.v = run * hkv + at.h * (at.T + C);
  }
  // the next unit (b = B past the last)
  auto next_unit = [&](Place& x) {
    x.v += x.T + C;
    if (++x.h < hkv) return;
    x.h = 0;
    do {
      ++x.b;
      if (x.b >= B) return;
      set_seq(x);
    } while (x.T == 0);
  };
  // this warp's steps of a unit: [first_step, end_step), maybe none
  auto first_step = [&](const Place& x) { return max(0, v0 - x.v - C); };
  auto end_step = [&](const Place& x) { return min(x.T, v1 - x.v - C); };

  // The copies run ahead of the sums, over unit ends.  Their block ids come in
  // windows of 32 (lane l: block l of the window), fetched one window ahead.
  // Place of the copies' unit, and the window after the one in use: its first
  // step (within cu) and ids.
  Place cu = at;
  int cs = 0, nids = 0;
  auto fetch_window = [&]() {
    const int j = cs * SB + lane;
    nids = cu.b < B && j < cu.rem
               ? __ldg(p.block_tables + static_cast<size_t>(cu.b) * p.max_blocks_per_seq + j)
               : 0;
  };
  // to the next unit that holds steps of this warp, or past its range
  auto settle = [&]() {
    while (cu.b < B && cu.v + C < v1 && cs >= end_step(cu)) {
      next_unit(cu);
      cs = 0;
    }
  };
  // The window in use: what is left of its steps and blocks; the lane that holds
  // the next block's id; and this lane's source without the block (lanes 2 u and
  // 2 u + 1 copy the K and the V tile of a step's block u).
  int ids = 0, left = 0, blocks = 0, id_at = 0;
  const unsigned char* src = nullptr;
  const uint64_t tile_stride = static_cast<uint64_t>(hkv) * E::KT;
  const unsigned char* pool = (lane & 1) ? p.v4 : p.k4;
  auto take_window = [&]() {
    ids = nids;
    left = min(WS, end_step(cu) - cs);
    blocks = cu.rem - cs * SB;
    id_at = min(lane >> 1, SB - 1);
    src = pool + static_cast<uint32_t>(cu.h) * E::KT;
    cs += left;
    settle();
  };
  const uint64_t policy = l2_policy_evict_first();
  const uint32_t ring_u = smem_u32(wbase) + lane * E::KT, bars_u = smem_u32(bars);
  // whether a step is left to copy
  auto more = [&]() { return left > 0 || (cu.b < B && cu.v + C < v1); };
  if (work) {
    cs = first_step(cu);
    settle();
    if (more()) {
      fetch_window();
      take_window();
      if (cu.b < B) fetch_window();
    }
  }
  auto issue = [&](int st) {
    if (left == 0) {
      take_window();
      if (cu.b < B && cu.v + C < v1) fetch_window();
    }
    int id = __shfl_sync(kFullMask, ids, id_at);
    if (lane < 2 * min(SB, blocks)) {
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(p.num_blocks)) {
        if ((lane & 1) == 0) raise_error(p.err, PA_DEVERR_BLOCK_ID);
        id = 0;  // never dereferenced: block 0 is read instead
      }
      if (lane == 0) mbar_expect_u32(bars_u + 8 * st, min(SB, blocks) * 2 * E::KT);
      bulk_copy_u32(ring_u + st * E::STAGE, src + static_cast<uint32_t>(id) * tile_stride,
                    E::KT, bars_u + 8 * st, policy);
    }
    id_at += SB;
    blocks -= SB;
    --left;
  };
  for (int i = 0; i < S && more(); ++i) issue(i);
  if (p.early_read) griddep_wait();

  // an empty sequence's output is zeros, and a new token has no place there
  for (int b = me; b < B; b += ev.warps) {
    if (__ldg(p.context_lens + b) > 0) continue;
    uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<size_t>(b) * p.num_q_heads * D);
    for (int i = lane; i < p.num_q_heads * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
    if (p.slot_mapping != nullptr && lane == 0 && __ldg(p.slot_mapping + b) >= 0)
      raise_error(p.err, PA_DEVERR_SLOT);
  }

  Warp4<D, G> w4;  // the unit being summed
  bool patched = false;
  int ctx = 0;
  auto begin = [&](bool reaches_end) {
    ctx = seq_at(at.b).ctx;
    w4.begin(p.q + (static_cast<size_t>(at.b) * p.num_q_heads + static_cast<size_t>(at.h) * G) * D,
             p.scale_log2, lane);
    // the warp that reads the unit's last step writes the sequence's new token
    patched = p.slot_mapping != nullptr && reaches_end &&
              fused_cache_write<D, 3>(
                  p, at.b, at.h, ctx,
                  p.block_tables + static_cast<size_t>(at.b) * p.max_blocks_per_seq, lane, patch);
    if (patched) __syncwarp();
  };
  // One arrival of `expected` at a counter, after the warp's writes; the last
  // sees all the others' writes and leaves the counter at zero.
  auto arrive = [&](unsigned* cnt, int expected) -> bool {
    __threadfence();
    __syncwarp();
    unsigned old = 0;
    if (lane == 0) old = atomicAdd(cnt, 1u);
    old = __shfl_sync(kFullMask, old, 0);
    if (old + 1u != static_cast<unsigned>(expected)) return false;
    __threadfence();
    if (lane == 0) *cnt = 0u;
    return true;
  };

  bool ok = true;  // every wait so far succeeded (warp-uniform)
  int st = 0;
  unsigned ph = 0;
  while (work && at.b < B && at.v + C < v1) {
    const int s0 = first_step(at), s1 = end_step(at);
    if (s0 >= s1) {
      next_unit(at);
      continue;
    }
    const bool ends = s1 == at.T;
    begin(ends);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      if (ok) ok = __all_sync(kFullMask, mbar_wait_bounded(&bars[st], ph, p.err));
      if (!ok) continue;
      const int nvalid = min(BS * SB, ctx - s * SB * BS);
      unsigned char* stage = tiles + st * E::STAGE;
      if (patched && s + 1 == s1) {
        patch_tile<D, 3>(stage + (nvalid - 1) / BS * 2 * E::KT, E::KT, patch, (nvalid - 1) % BS,
                         lane);
        __syncwarp();
      }
      if (nvalid == BS * SB)
        w4.template step<SB, true>(stage, nvalid, lane);
      else
        w4.template step<SB, false>(stage, nvalid, lane);
      __syncwarp();  // every lane is done with the stage
      if (more()) issue(st);
      if (++st == S) {
        st = 0;
        ph ^= 1u;
      }
    }
    float v[E::V];
    float2 ml[E::H];
    w4.finish(lane, v, ml);
    __nv_bfloat16* o =
        p.out + (static_cast<size_t>(at.b) * p.num_q_heads + static_cast<size_t>(at.h) * G) * D;
    if (s0 == 0 && ends) {  // the whole unit is this warp's
      even_write_out<D, G>(o, lane, v, ml);
    } else {
      // the unit's warps, and this one's place among them
      const int wf = warp_of(at.v + C), wl = warp_of(at.v + C + at.T - 1);
      const int g0 = wf / kEvenGroup, g1 = wl / kEvenGroup, g = me / kEvenGroup;
      unsigned* unit = ev.unit_cnt + static_cast<size_t>(at.b) * hkv + at.h;
      even_store<D, G>(even_slot<D, G>(ev.ws, wf, me), lane, v, ml);
      if (wl - wf < kEvenFlat) {
        if (arrive(unit, wl - wf + 1))
          even_merge<D, G>(ev.ws, wf, wf, 1, wl - wf + 1, o);
      } else {
        // first this group's warps (a group holds at most one such unit that comes
        // in from the group before, and at most one that begins in it and goes on
        // into the next), then the groups
        const int first = max(wf, g * kEvenGroup);
        const int count = min(wl, g * kEvenGroup + kEvenGroup - 1) - first + 1;
        if (arrive(ev.group_cnt + 2 * g + (g > g0 ? 0 : 1), count)) {
          if (count > 1) even_merge<D, G>(ev.ws, wf, first, 1, count, nullptr);
          if (arrive(unit, g1 - g0 + 1))
            even_merge<D, G>(ev.ws, wf, g0 * kEvenGroup, kEvenGroup, g1 - g0 + 1, o);
        }
      }
    }
    next_unit(at);  // (past this warp's range where the unit goes on)
  }
  // Only after a timed-out wait: copies still in flight land (bounded) before
  // the shared memory can be reused.
  if (!ok)
    for (int i = 0; i < S; ++i) mbar_wait_bounded(&bars[i], ph ^ (i < st ? 1u : 0u), p.err);
}

// Warps of a launch on the current device: one wave of resident CTAs.
template <int D, int G>
cudaError_t even_grid(int* ctas) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) *ctas = sms * Even<D, G>::CTAS;
  return e;
}

template <int D, int G>
cudaError_t launch_even_t(const DecodeParams& p, cudaStream_t stream) {
  using E = Even<D, G>;
  static std::atomic<uint64_t> smem_set{0};
  auto kernel = paged_decode_even_kernel<D, G>;
  cudaError_t e = allow_smem(kernel, E::SMEM, smem_set);
  int ctas = 0;
  if (e == cudaSuccess) e = even_grid<D, G>(&ctas);
  if (e != cudaSuccess) return e;
  // no more CTAs than the tables hold steps
  const int64_t steps = static_cast<int64_t>(p.num_seqs) * p.num_kv_heads *
                        ((p.max_blocks_per_seq + kEvenBlocks - 1) / kEvenBlocks);
  if (steps + static_cast<int64_t>(p.num_seqs) * p.num_kv_heads * kEvenUnitSteps > 0x7fffffff)
    return cudaErrorInvalidValue;
  if (steps < ctas) ctas = static_cast<int>(steps);
  EvenArgs ev;
  ev.ws = p.ws_o;
  ev.unit_cnt = p.counters;
  ev.group_cnt = p.counters + static_cast<size_t>(p.num_seqs) * p.num_kv_heads;
  ev.warps = ctas * kEvenWarps;
  return launch_pdl(kernel, dim3(ctas), dim3(kEvenWarps * 32), E::SMEM, stream, p, ev);
}

}  // namespace

cudaError_t launch_decode_int4_even(const DecodeParams& p, int head_dim, int group,
                                    cudaStream_t stream) {
  if (group != 2 && group != 4) return cudaErrorInvalidValue;
  if (head_dim == 128)
    return group == 2 ? launch_even_t<128, 2>(p, stream) : launch_even_t<128, 4>(p, stream);
  return group == 2 ? launch_even_t<64, 2>(p, stream) : launch_even_t<64, 4>(p, stream);
}

// Floats of workspace a launch may use on the current device (0: no device, no
// such kernel).
size_t even_floats_int4(int head_dim, int group) {
  int ctas = 0;
  if ((group != 2 && group != 4) || even_grid<64, 4>(&ctas) != cudaSuccess) return 0;
  const size_t slot = head_dim == 128 ? Even<128, 4>::SLOT : Even<64, 4>::SLOT;
  static_assert(Even<128, 2>::SLOT == Even<128, 4>::SLOT && Even<64, 2>::SLOT == Even<64, 4>::SLOT,
                "one slot size for both groups");
  return static_cast<size_t>(ctas) * kEvenWarps * 2 * slot;
}

}  // namespace pa
