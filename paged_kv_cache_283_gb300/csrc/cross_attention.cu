// Cross attention over paged source states on the 5th-generation tensor cores,
// sm_103a: decoder queries (prompts, or the beams of a step) against an
// encoder's K and V, which lie in a paged cache like a context's.
//
//   out[t, h] = sum_j softmax_j(scale q[t, h] . K_j) V_j,  0 <= j < source_lens[b]
//
// Every query of a sequence sees the whole source, whatever its position, and
// the source's length has nothing to do with the number of queries.
//
// Design:
//  * A tile is 128 query rows, (token, head) pairs of one GQA group, so the
//    beams of a source and the heads of a group share each K / V tile: a step of
//    W beams reads its source once per KV head, not W times.  S = Q K^T and
//    O += P V are tcgen05.mma with S, P and O in tensor memory; K and V arrive
//    per 16-token block by TMA (the block table is a gather of 16-row boxes), 64
//    keys a chunk.
//  * The batch's work, all (sequence, KV head, tile) units' chunks of keys one after
//    another, is cut evenly among persistent CTAs (two an SM), each taking one run
//    of chunks whatever units it begins and ends in: ragged sources, few long ones
//    and many short ones all keep every SM busy to the end.  A unit's beginning and end
//    count as kUnitCost chunks (four: 64 x 4 beams of sources of 128 to 2048 keys 59.1 us,
//    16 x 512 prompts 424; one: 61.6 and 432), and one CTA an SM takes 72.2 and 532.
//    The lengths are read on the device, so a captured call follows them.
//  * A CTA is 4 softmax warps, a row a thread, and a warp each for the MMAs of
//    Q K^T and of P V and for the copies of K and of V: a warp's waits take it
//    longer than what it waits to issue.  The warps walk their CTA's run on their
//    own, the copy warps ahead of the others, so that the next unit's first tiles
//    are on their way while the last one's are used.
//  * A unit that several CTAs share is joined by the last of them to arrive: each
//    leaves its rows' (m, l, o) in the workspace, where a CTA has two places, one
//    for the unit it begins in and one for the unit it ends in.
//  * The softmax takes a chunk's maximum first and its weights against the row's
//    reference, which follows (and O is rescaled in tensor memory) only where it is
//    more than 2^8 too low.  The weights then go to tensor memory 16 keys at a time
//    and none is held.
//  * The weights enter P V as two bf16 parts, hi + lo, which keep 2^-16 of them;
//    their sum is taken before, in fp32.  One part would be off by up to 2^-9 of
//    the weighted mean of |V|, far more than the rounding of an output whose terms
//    cancel.  It would save a fourth of the time of long prompts.
//  * Few rows (beams of one step): a softmax thread's way through its row of 64
//    scores takes longer than the copies of their keys.  With 32 rows or fewer
//    the tile holds four copies of them, each of which takes a quarter of every
//    chunk's keys (zero weights for the others) and so a quarter of the time, and
//    ends with a share of the row's (m, l, O); with 64, two copies.  (64 x 4 beams
//    59.1 us and 3 x 5 beams of 8K to 64K keys 81.0, against 63.2 and 98.6 of one copy
//    each; one short source 7.9 against 7.6.)  The longest sequence decides for its call:
//    63 x 4 beams beside a prompt of 512 queries, all in full tiles, take 75 us, and 111 in
//    a call for the beams and one for the prompt (61.7 and 32.8 us alone); with a
//    prompt of 40 queries 103 and 99.
//  * Warps whose rows are all past the tile's queries (a step of few beams) do
//    no work but keep the barriers' counts.
//
// What bounds it: copies where rows are few (64 x 4 beams 0.74 of the copy rate, the long
// sources 0.87, with the start and the joins), the softmax threads' chain where tiles are
// full (16 x 512 prompts of 512 to 4096 keys 412 to 424 us, 378 the same call after
// itself: 0.91 to 1.0 PFLOP/s), and for ragged prompts the ends of units (35.5 us).

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/pa.h"
#include "device.cuh"
#include "internal.h"
#include "tensor.cuh"

namespace pa {

struct CrossParams {
  __nv_bfloat16* out;           // [T, Hq, D]
  const int32_t* block_tables;
  const int32_t* source_lens;
  const int32_t* query_start;
  float* ws_o;                  // [CTAs, 2, ws_rows, D]
  float2* ws_ml;                // [CTAs, 2, ws_rows]: reference maximum (base 2), sum
  unsigned* counters;           // [CTAs]
  unsigned* err;
  int max_blocks_per_seq;
  int num_seqs;
  int num_q_heads;
  int num_kv_heads;
  int num_blocks;
  int total_q;
  int max_query_len;
  int group;
  int tile_tokens;              // 128 / group
  int ws_rows;                  // rows of a tile that can hold queries
  float scale_log2;
};

namespace {

constexpr int kRows = 128;    // query rows per tile = MMA M
constexpr int kKeys = 64;     // keys per chunk = MMA N of S = Q K^T
constexpr int kBS = 16;       // tokens per cache block
constexpr int kChunkBlocks = kKeys / kBS;
constexpr int kSoftmaxThreads = 128;
constexpr int kThreads = kSoftmaxThreads + 128;
constexpr int kScoreWarp = 4, kMixWarp = 5, kCopyWarp = 6;  // Q K^T, P V, copies of K and of V
constexpr int kSumFloats = 4 * 32 * 20;  // room for 16 columns of every row's copies
constexpr int kMinChunks = 4;  // of a unit's part, on average: less is not worth a join
constexpr int kAhead = 2;      // batches of block ids that run ahead of their copies
constexpr int kUnitCost = 4;   // of a unit's beginning and end, in chunks
constexpr int kMaxParts = 64;  // CTAs that share a unit, on average at most
constexpr uint32_t kTO = 2 * kKeys;     // O's first column, after two S buffers
constexpr uint32_t kTmemCols = 256;

// mbar_wait_bounded, whose clock and loop stay out of the code of the waits, nearly
// all of which end in a sleeping try: the roles' loops then fit the instruction
// caches that they share (16 x 512 prompts 424 us, 467 with the loops in line).
__device__ __noinline__ bool wait_long(uint64_t* bar, unsigned parity, unsigned* err) {
  return mbar_wait_bounded(bar, parity, err);
}
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, unsigned parity, unsigned* err) {
  if (mbar_try_wait(bar, parity)) return true;
  if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
  return wait_long(bar, parity, err);
}

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;                // 64-column halves of a row
  static constexpr int kQHalf = kRows * 128;            // bytes of a half of Q
  static constexpr int kKVHalf = kKeys * 128;           // of a K or V chunk
  static constexpr int kBox = kBS * 128;                // of a block
  static constexpr int kStage = kHalves * kKVHalf;
  static constexpr int kStages = D == 128 ? 2 : 4;      // chunks in the K and V rings
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + kHalves * kQHalf;
  static constexpr int kV = kK + kStages * kStage;
  static constexpr int kBar = kV + kStages * kStage;
  static constexpr int kSums = kBar + 256;               // the copies' sums (few rows)
  static constexpr int smem(int copies) {                // + alignment
    return kSums + (copies > 1 ? kSumFloats * 4 + kRows * 8 : 0) + 1024;
  }
  static constexpr uint32_t kIdescQK = idesc_bf16(kRows, kKeys, 0, 0);
  static constexpr uint32_t kIdescPV = idesc_bf16(kRows, D, 0, 1);
  static_assert(kTO + D <= kTmemCols, "tensor memory");
  static_assert(2 * (smem(4) + 2048) <= 232448, "two CTAs an SM");
};

// A sequence's lengths, read and checked on the device.
struct Seq {
  int q0, n;     // its rows; 0 for one that is skipped
  int src;       // source length
  int chunks;    // of keys
  int tiles;     // of queries
  bool bad;
};
__device__ __forceinline__ Seq read_seq(const CrossParams& p, int b) {
  Seq s;
  s.q0 = load_after_wait(p.query_start + b);
  const int q1 = load_after_wait(p.query_start + b + 1);
  s.src = load_after_wait(p.source_lens + b);
  s.bad = s.q0 < 0 || q1 < s.q0 || q1 > p.total_q || s.src < 0 ||
          s.src > p.max_blocks_per_seq * kBS;
  s.n = s.bad ? 0 : min(q1 - s.q0, p.max_query_len);
  s.chunks = s.bad ? 0 : (s.src + kKeys - 1) / kKeys;
  s.tiles = (s.n + p.tile_tokens - 1) / p.tile_tokens;
  return s;
}

// a / b of non-negative numbers, most of which fit 32 bits (a 64-bit division
// takes ten times as long).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The list of units is ordered in pairs (tile, sequence), the tile the slower
// (kTileMajor), each with its KV heads: runs that begin at different tiles then
// pass the same keys at the same time, and a source larger than L2 is read from
// memory once for all its tiles, not once for each (16 x 512 queries: 0.31 GB read
// in place of 1.2).  With more pairs than a CTA looks through in a few microseconds
// the pairs are the sequences, each with its heads and their tiles.
constexpr int kMostPairs = 64 * kThreads;

struct Order {
  int num_seqs;
  int pairs;
  bool tile_major;
  __device__ int seq(int pair) const { return tile_major ? pair % num_seqs : pair; }
  __device__ int tile0(int pair) const { return tile_major ? pair / num_seqs : 0; }
  // tiles of a pair, from tile0 on
  __device__ int span(int pair, const Seq& s) const {
    return tile_major ? s.tiles > tile0(pair) : s.tiles;
  }
  __device__ int64_t work(const CrossParams& p, int pair, const Seq& s) const {
    return s.chunks == 0 ? 0
                         : static_cast<int64_t>(s.chunks + kUnitCost) * span(pair, s) *
                               p.num_kv_heads;
  }
};

// What all CTAs agree on: a unit takes kUnitCost + chunks positions of the list, its
// chunk c the position kUnitCost + c of them; CTA c's run has `least` positions, the
// first `rest` CTAs' one more.
struct Plan {
  Order order;
  int ctas;           // that take part
  int64_t least;
  int rest;
  __device__ int64_t begin(int c) const { return c * least + min(c, rest); }
  __device__ int64_t length(int c) const { return c < ctas ? least + (c < rest) : 0; }
  __device__ int owner(int64_t at) const {
    const int64_t longer = rest * (least + 1);
    if (at < longer) return static_cast<int>(quotient(at, least + 1));
    return rest + static_cast<int>(quotient(at - longer, least));
  }
};

// A CTA's run of positions, and the unit that it begins in.
struct Run {
  int64_t left;       // positions
  int64_t unit;       // the unit's first position
  int pair, kvh, inner;
  int offset;         // in the unit
};

// A part of a unit: chunks [first, first + count) of its keys.
struct Part {
  int b, kvh, i0;
  Seq seq;
  int first, count;
  int64_t unit;      // the unit's first position
};

struct Walk {
  const Order& order;  // (in shared memory)
  int64_t left, unit;
  int pair, kvh, inner, offset, span;
  Seq seq;
  __device__ Walk(const CrossParams& p, const Order& o, const Run& r)
      : order(o), left(r.left), unit(r.unit), pair(r.pair), kvh(r.kvh), inner(r.inner),
        offset(r.offset), span(0) {
    if (left > 0) enter(p);
  }
  __device__ void enter(const CrossParams& p) {
    seq = read_seq(p, order.seq(pair));
    span = order.span(pair, seq);
  }
  __device__ bool next(const CrossParams& p, Part& t) {
    while (left > 0) {
      while (span == 0 || seq.chunks == 0 || kvh == p.num_kv_heads) {
        kvh = inner = 0;
        if (++pair >= order.pairs) {  // (the run ends within the units)
          left = 0;
          return false;
        }
        enter(p);
      }
      const int size = seq.chunks + kUnitCost;
      const int taken = static_cast<int>(min(static_cast<int64_t>(size - offset), left));
      t.first = max(0, offset - kUnitCost);
      t.count = max(0, offset + taken - kUnitCost) - t.first;
      t.b = order.seq(pair);
      t.kvh = kvh;
      t.i0 = (order.tile0(pair) + inner) * p.tile_tokens;
      t.seq = seq;
      t.unit = unit;
      left -= taken;
      unit += size;
      offset = 0;
      if (++inner == span) {
        inner = 0;
        ++kvh;
      }
      if (t.count > 0) return true;  // (a run may end before its last unit's first chunk)
    }
    return false;
  }
};

// The even cut: sums of the pairs' work by the whole CTA, each thread taking a run
// of pairs; the thread whose pairs hold the CTA's first position finds it.
__device__ void cut(const CrossParams& p, Plan* plan, Run* out, int64_t* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kThreads / 32;
  int* warp_ints = reinterpret_cast<int*>(warp_sums + kWarps);
  // tiles of the longest sequence (the host knows a bound)
  int tiles = 1;
  if (p.max_query_len > p.tile_tokens) {
    for (int b = tid; b < p.num_seqs; b += kThreads) tiles = max(tiles, read_seq(p, b).tiles);
    tiles = __reduce_max_sync(kFullMask, tiles);
    if (lane == 0) warp_ints[warp] = tiles;
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) tiles = max(tiles, warp_ints[w]);
    __syncthreads();
  }
  Order order;
  order.num_seqs = p.num_seqs;
  order.tile_major = static_cast<int64_t>(tiles) * p.num_seqs <= kMostPairs;
  order.pairs = order.tile_major ? tiles * p.num_seqs : p.num_seqs;
  const int per = (order.pairs + kThreads - 1) / kThreads;
  const int a0 = min(tid * per, order.pairs), a1 = min(a0 + per, order.pairs);
  int64_t sum = 0;
  int units = 0;  // counted as far as it matters
  for (int a = a0; a < a1; ++a) {
    const Seq s = read_seq(p, order.seq(a));
    const int64_t w = order.work(p, a, s);
    sum += w;
    if (w > 0)
      units = static_cast<int>(min(static_cast<int64_t>(order.span(a, s)) * p.num_kv_heads + units,
                                   static_cast<int64_t>(1 << 20)));
  }
  int64_t incl = sum;
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) {
    const int64_t o = __shfl_up_sync(kFullMask, incl, k);
    if (lane >= k) incl += o;
  }
  units = __reduce_add_sync(kFullMask, units);
  if (lane == 31) {
    warp_sums[warp] = incl;
    warp_ints[warp] = units;
  }
  __syncthreads();
  int64_t total = 0, before = 0;
  units = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sums[w];
    total += warp_sums[w];
    units += warp_ints[w];
  }
  before += incl - sum;
  // a CTA for each unit, or for each kMinChunks chunks where those are more
  const int64_t chunks = total - static_cast<int64_t>(units) * kUnitCost;
  int ctas = static_cast<int>(
      max(static_cast<int64_t>(units),
          min(chunks / kMinChunks, static_cast<int64_t>(units) * kMaxParts)));
  ctas = max(1, min(static_cast<int>(min(total, static_cast<int64_t>(gridDim.x))), ctas));
  Plan n;
  n.order = order;
  n.ctas = ctas;
  n.least = quotient(total, ctas);
  n.rest = static_cast<int>(total - n.least * ctas);
  if (tid == 0) *plan = n;
  const int64_t begin = n.begin(blockIdx.x), left = n.length(blockIdx.x);
  if (left > 0 ? before <= begin && begin < before + sum : tid == 0) {
    Run r{left, before, a0, 0, 0, 0};
    if (left > 0) {
      Seq s;
      for (;; ++r.pair) {
        s = read_seq(p, order.seq(r.pair));
        const int64_t w = order.work(p, r.pair, s);
        if (begin < r.unit + w || r.pair + 1 >= a1) break;
        r.unit += w;
      }
      const int size = s.chunks + kUnitCost;
      const int u = static_cast<int>(quotient(begin - r.unit, size));
      const int span = max(1, order.span(r.pair, s));
      r.unit += static_cast<int64_t>(u) * size;
      r.offset = static_cast<int>(begin - r.unit);
      r.kvh = u / span;
      r.inner = u - r.kvh * span;
    }
    *out = r;
  }
  __syncthreads();
}

// The rows of a unit from its parts' (m, l, o): part k lies in the place of CTA
// c0 + k, the first one in that of the unit its CTA ends in; the parts are summed in
// their order, whichever CTA does it.
//
// Full tiles: a thread a row, whose pieces of 4 dims lie beside the other rows' in the
// workspace, and this CTA's own part still in tensor memory.
template <int D>
__device__ __forceinline__ float4* column_piece(const CrossParams& p, int64_t place, int piece,
                                                int row) {
  return reinterpret_cast<float4*>(p.ws_o + place * D) + piece * p.ws_rows + row;
}
template <int D>
__device__ __forceinline__ void join_rows(const CrossParams& p, int c0, int parts, bool row_ok,
                                          int row, float2 own_ml, uint32_t t_o,
                                          __nv_bfloat16* out) {
  const int own = static_cast<int>(blockIdx.x) - c0, r = min(row, p.ws_rows - 1);
  auto place = [&](int k) { return (static_cast<int64_t>(c0 + k) * 2 + (k == 0)) * p.ws_rows; };
  auto stats = [&](int k) { return k == own ? own_ml : __ldcg(p.ws_ml + place(k) + r); };
  float top = own_ml.x;
#pragma unroll 1
  for (int k = 0; k < parts; ++k) top = fmaxf(top, stats(k).x);
  const float ref = top == -INFINITY ? 0.f : top;
  float total = 0.f;
#pragma unroll 1
  for (int k = 0; k < parts; ++k) {
    const float2 ml = stats(k);
    total = fmaf(ml.y, ex2(ml.x - ref), total);
  }
  const float inv = total > 0.f ? 1.f / total : 0.f;
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float acc[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = 0.f;
#pragma unroll 1
    for (int k = 0; k < parts; ++k) {
      const float f = ex2(stats(k).x - ref) * inv;
      if (k == own) {
        uint32_t o[32];
        tmem_ld32(t_o + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(o[j]), f, acc[j]);
      } else {
        float4 o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __ldcg(column_piece<D>(p, place(k), c / 4 + j, r));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[4 * j] = fmaf(o[j].x, f, acc[4 * j]);
          acc[4 * j + 1] = fmaf(o[j].y, f, acc[4 * j + 1]);
          acc[4 * j + 2] = fmaf(o[j].z, f, acc[4 * j + 2]);
          acc[4 * j + 3] = fmaf(o[j].w, f, acc[4 * j + 3]);
        }
      }
    }
    if (row_ok) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h2 =
              __floats2bfloat162_rn(acc[8 * e + 2 * j], acc[8 * e + 2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t*>(&h2);
        }
        reinterpret_cast<uint4*>(out + c)[e] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// Few rows: a thread takes 4 dims of a row at a time, P such pieces and E parts of
// each in flight.
template <int D, int P, int E>
__device__ __forceinline__ void join(const CrossParams& p, const Part& it, int c0, int parts) {
  constexpr int kCols = D / 4;
  const int shift = 31 - __clz(p.group);
  const int rows = min(kRows, (it.seq.n - it.i0) << shift);
  auto at = [&](int k, int row) {
    return (static_cast<int64_t>(c0 + k) * 2 + (k == 0)) * p.ws_rows + row;
  };
  const int pieces = rows * kCols;
#pragma unroll 1
  for (int q0 = threadIdx.x; q0 < pieces; q0 += P * kSoftmaxThreads) {
    float m[P], l[P];
    float4 acc[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      m[j] = -INFINITY;
      l[j] = 0.f;
      acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int k0 = 0; k0 < parts; k0 += E) {
      float2 ml[P][E];
      float4 o[P][E];
      // (loads without conditions, so that none waits for another: past the end the
      // last piece or part again, without weight)
#pragma unroll
      for (int j = 0; j < P; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int q = min(q0 + j * kSoftmaxThreads, pieces - 1);
          const int64_t r = at(min(k0 + e, parts - 1), q / kCols);
          ml[j][e] = __ldcg(p.ws_ml + r);
          o[j][e] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + r * D) + q % kCols);
        }
#pragma unroll
      for (int j = 0; j < P; ++j) {
        float top = m[j];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (k0 + e >= parts) ml[j][e] = make_float2(-INFINITY, 0.f);
          top = fmaxf(top, ml[j][e].x);
        }
        const float ref = top == -INFINITY ? 0.f : top;
        const float a = ex2(m[j] - ref);
        m[j] = top;
        l[j] *= a;
        acc[j] = make_float4(acc[j].x * a, acc[j].y * a, acc[j].z * a, acc[j].w * a);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float b = ex2(ml[j][e].x - ref);
          l[j] = fmaf(ml[j][e].y, b, l[j]);
          acc[j].x = fmaf(o[j][e].x, b, acc[j].x);
          acc[j].y = fmaf(o[j][e].y, b, acc[j].y);
          acc[j].z = fmaf(o[j][e].z, b, acc[j].z);
          acc[j].w = fmaf(o[j][e].w, b, acc[j].w);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int q = q0 + j * kSoftmaxThreads, r = q / kCols;
      if (q >= pieces) continue;
      const float z = l[j] > 0.f ? 1.f / l[j] : 0.f;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[j].x * z, acc[j].y * z);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[j].z * z, acc[j].w * z);
      const int64_t row = static_cast<int64_t>(it.seq.q0 + it.i0 + (r >> shift)) * p.num_q_heads +
                          it.kvh * p.group + (r & (p.group - 1));
      reinterpret_cast<uint2*>(p.out + row * D)[q % kCols] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                     *reinterpret_cast<const uint32_t*>(&hi));
    }
  }
}

// grid: persistent.  Barriers (each wait names one use of one slot):
//   k_full / v_full [stage]: copies landed; k_free / v_free [stage]: the MMA that
//   read the stage is done; s_done [2]: scores of a chunk ready; p_ready [2]:
//   its weights written (an arrival a softmax warp); pv_done [2]: PV read them;
//   q_full / q_free: a unit's Q landed / its last scores taken; o_free: O read.
template <int D, int R>
__global__ void __launch_bounds__(kThreads, 2)
    cross_attention_kernel(const __grid_constant__ CUtensorMap tq,
                           const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv, const CrossParams p) {
  using S = Shape<D>;
  constexpr int kStages = S::kStages;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBar);
  uint64_t* k_full = bars;
  uint64_t* v_full = bars + kStages;
  uint64_t* k_free = bars + 2 * kStages;
  uint64_t* v_free = bars + 3 * kStages;
  uint64_t* s_done = bars + 4 * kStages;
  uint64_t* pv_done = s_done + 2;
  uint64_t* p_ready = s_done + 4;
  uint64_t* q_full = s_done + 6;
  uint64_t* q_free = s_done + 7;
  uint64_t* o_free = s_done + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::kBar + 248);
  unsigned* last_slot = reinterpret_cast<unsigned*>(sm + S::kBar + 252);
  constexpr int kBarriers = 4 * kStages + 9;
  static_assert(kBarriers * 8 <= 248, "barriers");
  float* sums = reinterpret_cast<float*>(sm + S::kSums);                         // R > 1
  float2* stats = reinterpret_cast<float2*>(sm + S::kSums + kSumFloats * 4);  // [128]

  if (tid == 0) {
    for (int i = 0; i < kBarriers; ++i) mbar_init(bars + i, 1);
    for (int i = 0; i < 2; ++i) mbar_init(p_ready + i, kSoftmaxThreads / 32);
    mbar_init(o_free, kSoftmaxThreads / 32);
    fence_mbar_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __shared__ Plan plan;
  __shared__ Run run;
  __shared__ int64_t warp_sums[2 * (kThreads / 32)];
  tc_fence_before();
  cut(p, &plan, &run, warp_sums);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const bool vwarp = warp == kCopyWarp + 1;

  if (warp >= kCopyWarp) {
    // ------------------------------------------------------------ copies
    // One warp for Q and the K ring, one for the V ring.  A part's block ids are
    // fetched a lane each, 32 at a time, kAhead such batches ahead of their copies.
    constexpr int kBatch = 32 / kChunkBlocks;  // chunks
    struct Batch {
      int id;          // lane j: the raw table entry of block j (checked at use)
      int blocks;      // 0: no batch
      int kvh, q_row;  // q_row: of the Q of a part that the batch opens, else -1
    };
    Walk walk(p, plan.order, run);
    Part it;
    bool some = walk.next(p, it);
    int c = 0;  // chunk of `it` that is fetched next
    auto fetch = [&]() -> Batch {
      Batch a{0, 0, 0, -1};
      if (!some) return a;
      const int block = (it.first + c) * kChunkBlocks;
      const int chunks = min(kBatch, it.count - c);
      a.blocks = min(chunks * kChunkBlocks, (it.seq.src + kBS - 1) / kBS - block);
      a.kvh = it.kvh;
      if (c == 0) a.q_row = it.seq.q0 + it.i0;
      if (lane < a.blocks)
        a.id = load_after_wait(p.block_tables +
                               static_cast<int64_t>(it.b) * p.max_blocks_per_seq + block + lane);
      c += chunks;
      if (c == it.count) {
        some = walk.next(p, it);
        c = 0;
      }
      return a;
    };
    const uint32_t leader = elect_lane();
    auto wait = [&](uint64_t* bar, int use) {
      return __all_sync(kFullMask, wait_bounded(bar, use & 1, p.err)) != 0;
    };
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(vwarp ? &tv : &tk))
                   : "memory");
      if (!vwarp)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tq)) : "memory");
    }
    Batch ahead[kAhead];
#pragma unroll 1
    for (int i = 0; i < kAhead; ++i) {
#pragma unroll
      for (int k = 0; k + 1 < kAhead; ++k) ahead[k] = ahead[k + 1];
      ahead[kAhead - 1] = fetch();
    }
    bool ok = true;
    int g = 0, items = 0;
    while (ok && ahead[0].blocks > 0) {
      Batch a = ahead[0];
#pragma unroll
      for (int k = 0; k + 1 < kAhead; ++k) ahead[k] = ahead[k + 1];
      ahead[kAhead - 1] = fetch();
      if (lane < a.blocks && (a.id < 0 || a.id >= p.num_blocks)) {
        raise_error(p.err, PA_DEVERR_BLOCK_ID);  // never dereferenced: block 0 is read instead
        a.id = 0;
      }
      const int row = (a.id * p.num_kv_heads + a.kvh) * kBS;
#pragma unroll 1
      for (int at = 0; at < a.blocks; at += kChunkBlocks) {
        const int blocks = min(kChunkBlocks, a.blocks - at);
        const int st = g % kStages;
        if (g >= kStages) ok = wait(vwarp ? &v_free[st] : &k_free[st], g / kStages - 1);
        if (!ok) break;
        uint64_t* bar = vwarp ? &v_full[st] : &k_full[st];
        mbar_arrive_expect_tx(bar, static_cast<uint32_t>(blocks * S::kHalves * S::kBox), leader);
        ++g;
        unsigned char* dst = sm + (vwarp ? S::kV : S::kK) + st * S::kStage;
#pragma unroll
        for (int j = 0; j < kChunkBlocks; ++j) {
          const int y = __shfl_sync(kFullMask, row, at + j);
          if (j >= blocks) continue;
          if (vwarp) {
            tma_3d(dst + j * S::kHalves * S::kBox, &tv, 0, y, 0, bar, leader);
          } else {
#pragma unroll
            for (int h = 0; h < S::kHalves; ++h)
              tma_2d(dst + h * S::kKVHalf + j * S::kBox, &tk, 64 * h, y, bar, leader);
          }
        }
        if (!vwarp && at == 0 && a.q_row >= 0) {
          if (items > 0) ok = wait(q_free, items - 1);
          if (!ok) break;
          mbar_arrive_expect_tx(q_full, S::kHalves * S::kQHalf, leader);
#pragma unroll
          for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
            for (int r = 0; r < R; ++r)
              tma_3d(sm + S::kQ + h * S::kQHalf + r * (S::kQHalf / R), &tq, 64 * h,
                     a.kvh * p.group, a.q_row, q_full, leader);
          ++items;
        }
      }
    }
    // Copies this warp issued land before the CTA's shared memory is given up
    // (an earlier use of a stage completed before its last copy was issued).
    if (lane == 0) {
      for (int st = 0; st < kStages && st < g; ++st) {
        const int last = g - 1 - (g - 1 - st) % kStages;  // the last chunk in this stage
        wait_bounded(vwarp ? &v_full[st] : &k_full[st], (last / kStages) & 1, p.err);
      }
      if (!vwarp && items > 0) wait_bounded(q_full, (items - 1) & 1, p.err);
    }
  } else if (warp == kScoreWarp) {
    // ------------------------------------------------------------ scores
    // (the whole warp in step: see umma_bf16)
    const uint32_t leader = elect_lane();
    auto wait = [&](uint64_t* bar, int use) {
      return __all_sync(kFullMask, wait_bounded(bar, use & 1, p.err)) != 0;
    };
    const uint64_t qdesc = sw128_desc(smem_u32(sm + S::kQ), 16, 1024);
    const uint32_t sK = smem_u32(sm + S::kK);
    Walk walk(p, plan.order, run);
    Part it;
    bool ok = true;
    int g = 0;
    for (int items = 0; ok && walk.next(p, it); ++items) {
      ok = wait(q_full, items);
      for (int c = 0; c < it.count && ok; ++c) {
        const int sb = g & 1, st = g % kStages;
        ok = wait(&k_full[st], g / kStages);
        // PV of two chunks ago has read the weights in this S buffer
        if (ok && g >= 2) ok = wait(&pv_done[sb], (g - 2) >> 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t kdesc = sw128_desc(sK + st * S::kStage, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t qoff = ((kk >> 2) * S::kQHalf + (kk & 3) * 32) >> 4;
          const uint32_t koff = ((kk >> 2) * S::kKVHalf + (kk & 3) * 32) >> 4;
          umma_bf16(tmem + sb * kKeys, qdesc + qoff, kdesc + koff, S::kIdescQK, kk > 0, leader);
        }
        umma_commit(&s_done[sb], leader);
        umma_commit(&k_free[st], leader);
        if (c + 1 == it.count) umma_commit(q_free, leader);
        ++g;
      }
    }
    // The MMAs issued complete before tensor and shared memory are given up.
    if (g > 0) wait(&s_done[(g - 1) & 1], (g - 1) >> 1);
  } else if (warp == kMixWarp) {
    // ------------------------------------------------------------ O += P V
    const uint32_t leader = elect_lane();
    auto wait = [&](uint64_t* bar, int use) {
      return __all_sync(kFullMask, wait_bounded(bar, use & 1, p.err)) != 0;
    };
    const uint32_t sV = smem_u32(sm + S::kV);
    Walk walk(p, plan.order, run);
    Part it;
    bool ok = true;
    int g = 0;
    for (int items = 0; ok && walk.next(p, it); ++items) {
      for (int c = 0; c < it.count && ok; ++c) {
        const int sb = g & 1, st = g % kStages;
        // the part before has been read out of O
        if (c == 0 && items > 0) ok = wait(o_free, items - 1);
        ok = ok && wait(&v_full[st], g / kStages) && wait(&p_ready[sb], g >> 1);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vdesc = sw128_desc(sV + st * S::kStage, S::kBox, 1024);
#pragma unroll
        for (int kk = 0; kk < kChunkBlocks; ++kk) {
          const uint64_t v = vdesc + kk * (S::kHalves * S::kBox >> 4);
          umma_bf16_ts(tmem + kTO, tmem + sb * kKeys + 8 * kk, v, S::kIdescPV,
                       (c > 0 || kk > 0) ? 1u : 0u, leader);
          umma_bf16_ts(tmem + kTO, tmem + sb * kKeys + kKeys / 2 + 8 * kk, v, S::kIdescPV, 1u,
                       leader);
        }
        umma_commit(&pv_done[sb], leader);
        umma_commit(&v_free[st], leader);
        ++g;
      }
    }
    if (g > 0) wait(&pv_done[(g - 1) & 1], (g - 1) >> 1);
  } else {
    // ------------------------------------------------------------ softmax
    constexpr int kTileRows = kRows / R, kCols = kKeys / R;  // rows; columns of S a thread takes
    const int copy = warp / (4 / R);                         // of the rows: its columns of S
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tO = tmem + lane_base + kTO;
    const int row = tid & (kTileRows - 1);
    const int shift = 31 - __clz(p.group);
    const int tok = row >> shift, head = row & (p.group - 1);  // row: token, head of the group
    const float sl2 = p.scale_log2;
    const float2 sl2x2 = make_float2(sl2, sl2);
    bool ok = true;  // sticky: this thread's waits all succeeded
    int g = 0;
    Walk walk(p, plan.order, run);
    Part it;
    while (walk.next(p, it)) {
      const int qi = it.i0 + tok;
      const bool row_ok = qi < it.seq.n;
      // some row of the warp is
      const bool warp_ok = it.i0 + (((warp * 32) & (kTileRows - 1)) >> shift) < it.seq.n;
      const int64_t orow = static_cast<int64_t>(it.seq.q0 + (row_ok ? qi : 0)) * p.num_q_heads +
                           it.kvh * p.group + head;
      float m_used = -INFINITY;  // reference maximum of the exponentials (base 2)
      float l_sum = 0.f;
      for (int c = 0; c < it.count; ++c, ++g) {
        const int sb = g & 1;
        const uint32_t tS = tmem + lane_base + sb * kKeys;
        const int keys = it.seq.src - (it.first + c) * kKeys;  // of this chunk
        const int valid = keys - copy * kCols;                 // of this thread's columns
        bool lok = ok && wait_bounded(&s_done[sb], (g >> 1) & 1, p.err);
        lok = __all_sync(kFullMask, lok);
        if (lok && warp_ok) {
          tc_fence_after();
          uint32_t sv[kCols];
          if constexpr (kCols >= 32) {
#pragma unroll
            for (int h = 0; h < kCols / 32; ++h)
              tmem_ld32(tS + copy * kCols + 32 * h,
                        *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * h));
          } else {
            tmem_ld16(tS + copy * kCols, *reinterpret_cast<uint32_t(*)[16]>(sv));
          }
          tmem_wait_ld();
          if (valid < kCols) {
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (j >= valid) sv[j] = __float_as_uint(-INFINITY);
          }
          // The chunk's maximum (in threes); the reference follows where it is more
          // than 2^8 too low.
          float m4[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = __uint_as_float(sv[k]);
#pragma unroll
          for (int j = 4; j + 7 < kCols; j += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              m4[k] = fmaxf(fmaxf(m4[k], __uint_as_float(sv[j + k])),
                            __uint_as_float(sv[j + 4 + k]));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], __uint_as_float(sv[kCols - 4 + k]));
          const float mx = fmaxf(fmaxf(m4[0], m4[2]), fmaxf(m4[1], m4[3])) * sl2;
          float alpha = 1.f;
          if (mx > m_used + 8.f || m_used == -INFINITY) {
            alpha = m_used == -INFINITY ? 1.f : ex2(m_used - mx);
            m_used = mx;
          }
          // O is rescaled before this chunk's PV: PV of the chunk before must be
          // done with it (the part's first PV overwrites O)
          if (c > 0 && __any_sync(kFullMask, alpha != 1.f)) {
            lok = wait_bounded(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, p.err);
            lok = __all_sync(kFullMask, lok);
            if (lok) {
              tc_fence_after();
#pragma unroll 1
              for (int q4 = 0; q4 < D / 16; ++q4) {
                uint32_t o[16];
                tmem_ld16(tO + 16 * q4, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                tmem_st16(tO + 16 * q4, o);
              }
            }
          }
          // P over the scores' columns: bf16 pairs, hi parts, then lo; a copy of
          // the rows has weights in its own columns and zeros in the others
          const float neg = m_used == -INFINITY ? 0.f : -m_used;
          const float2 neg2 = make_float2(neg, neg);
          float2 ps[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};
          const uint32_t tH = tS + copy * (kCols / 2), tL = tH + kKeys / 2;
#pragma unroll
          for (int h = 0; h < kCols / 16; ++h) {
            uint32_t wh[8], wl[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int j = 16 * h + 2 * k;
              const float2 x = __ffma2_rn(
                  make_float2(__uint_as_float(sv[j]), __uint_as_float(sv[j + 1])), sl2x2, neg2);
              const float2 e = make_float2(ex2(x.x), ex2(x.y));
              ps[k & 3] = __fadd2_rn(ps[k & 3], e);
              split_p(__float_as_uint(e.x), __float_as_uint(e.y), wh[k], wl[k]);
            }
            tmem_st8(tH + 8 * h, wh);
            tmem_st8(tL + 8 * h, wl);
          }
          if constexpr (R > 1) {
            const uint32_t none[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int h = 0; h < kKeys / 16; ++h)
              if (h / (kCols / 16) != copy) {
                tmem_st8(tS + 8 * h, none);
                tmem_st8(tS + kKeys / 2 + 8 * h, none);
              }
          }
          const float2 pa = __fadd2_rn(__fadd2_rn(ps[0], ps[2]), __fadd2_rn(ps[1], ps[3]));
          l_sum = l_sum * alpha + (pa.x + pa.y);
          tmem_wait_st();
        }
        // V of keys past the source's end may hold anything (a partly filled
        // block, blocks not loaded): P is 0 there, but 0 * NaN is not.
        if (lok && keys < kKeys) {
          const int st = g % kStages;
          lok = wait_bounded(&v_full[st], (g / kStages) & 1, p.err);
          if (lok && tid >= keys && tid < kKeys) {
            const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int hh = 0; hh < S::kHalves; ++hh) {
              uint4* dst = reinterpret_cast<uint4*>(
                  sm + S::kV + st * S::kStage + ((tid / kBS) * S::kHalves + hh) * S::kBox +
                  (tid % kBS) * 128);
#pragma unroll
              for (int k = 0; k < 8; ++k) dst[k] = z;
            }
          }
          fence_proxy_async();
        }
        ok = ok && lok;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_ready[sb]);
      }
      // the rows' result, once the part's last PV is done
      bool lok = ok && wait_bounded(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, p.err);
      lok = __all_sync(kFullMask, lok);
      ok = ok && lok;
      tc_fence_after();
      const bool shared = it.count < it.seq.chunks;  // with other CTAs
      // (a part that opens its unit is its CTA's last, any other its first)
      const int64_t place = (static_cast<int64_t>(blockIdx.x) * 2 + (it.first == 0)) * p.ws_rows;
      // The copies' shares of a row: against their common maximum, summed through
      // shared memory, some columns at a time.
      float factor = 1.f, total = l_sum;
      if constexpr (R > 1) {
        stats[tid] = make_float2(m_used, l_sum);
        asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
        float top = m_used;
#pragma unroll
        for (int r = 0; r < R; ++r) top = fmaxf(top, stats[r * kTileRows + row].x);
        const float ref = top == -INFINITY ? 0.f : top;
        total = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 e = stats[r * kTileRows + row];
          total = fmaf(e.y, ex2(e.x - ref), total);
        }
        factor = ex2(m_used - ref);
        m_used = top;
      }
      const float inv = shared ? factor : total > 0.f ? factor / total : 0.f;
      // four columns of this thread's row
      auto put = [&](int col, const float4& v) {
        if (shared) {
          *reinterpret_cast<float4*>(p.ws_o + (place + row) * D + col) = v;
        } else {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y);
          const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z, v.w);
          *reinterpret_cast<uint2*>(p.out + orow * D + col) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                         *reinterpret_cast<const uint32_t*>(&hi));
        }
      };
      if constexpr (R == 1) {
        if (warp_ok && lok) {
#pragma unroll 1
          for (int q4 = 0; q4 < D / 16; ++q4) {
            uint32_t o[16];
            tmem_ld16(tO + 16 * q4, o);
            tmem_wait_ld();
            if (!row_ok) continue;
            if (shared) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *column_piece<D>(p, place, 4 * q4 + k, row) =
                    make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3]));
            } else {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(
                    __uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                w[e] = *reinterpret_cast<const uint32_t*>(&h2);
              }
              uint4* dst = reinterpret_cast<uint4*>(p.out + orow * D + 16 * q4);
              dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
              dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      } else {
        // columns of a round: what the buffer holds of the rows that there are
        const int rows = min(kTileRows, (it.seq.n - it.i0) << shift);
        int round = 16;
        while (round < D && rows * R * (2 * round + 4) <= kSumFloats) round *= 2;
        const int pitch = round + 4;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += round) {
          if (warp_ok && lok) {
#pragma unroll 1
            for (int q4 = 0; q4 < round / 16; ++q4) {
              uint32_t o[16];
              tmem_ld16(tO + c0 + 16 * q4, o);
              tmem_wait_ld();
              if (!row_ok) continue;
              float4* dst = reinterpret_cast<float4*>(sums + (copy * rows + row) * pitch + 16 * q4);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k] = make_float4(
                    __uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv,
                    __uint_as_float(o[4 * k + 2]) * inv, __uint_as_float(o[4 * k + 3]) * inv);
            }
          }
          asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
          if (row_ok && lok) {
            for (int k = copy; k < round / 4; k += R) {
              float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int r = 0; r < R; ++r) {
                const float4 x = *reinterpret_cast<const float4*>(sums + (r * rows + row) * pitch +
                                                                  4 * k);
                v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
              }
              put(c0 + 4 * k, v);
            }
          }
          asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
        }
      }
      auto leave_o = [&]() {
        __syncwarp();
        tc_fence_before();
        if (lane == 0) mbar_arrive(o_free);
      };
      if (R > 1 || !shared) leave_o();
      if (shared) {
        if (row_ok && lok && copy == 0) p.ws_ml[place + row] = make_float2(m_used, total);
        // the last CTA of the unit joins its parts (counted at its first CTA)
        const int64_t at = it.unit + kUnitCost;
        const int c0 = plan.owner(at);
        const int shares = plan.owner(at + it.seq.chunks - 1) - c0 + 1;
        asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
        if (tid == 0)
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                       : "=r"(*last_slot)
                       : "l"(p.counters + c0)
                       : "memory");
        asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
        if (*last_slot + 1 == static_cast<unsigned>(shares)) {
          if constexpr (R == 1) {
            if (warp_ok && lok)
              join_rows<D>(p, c0, shares, row_ok, row, make_float2(m_used, total), tO,
                           p.out + orow * D);
          } else if (((it.seq.n - it.i0) << shift) * (D / 4) <= kSoftmaxThreads) {
            join<D, 1, 8>(p, it, c0, shares);  // few rows, as of a long source's step
          } else {
            join<D, 4, 2>(p, it, c0, shares);
          }
          if (tid == 0) p.counters[c0] = 0;
        }
        if (R == 1) leave_o();
      }
    }
    // sequences without a source, and bad ones
    for (int b = blockIdx.x; b < p.num_seqs; b += gridDim.x) {
      const Seq s = read_seq(p, b);
      if (s.bad) {
        if (tid == 0) raise_error(p.err, PA_DEVERR_CONTEXT_LEN);
      } else if (s.src == 0) {
        const int64_t row = static_cast<int64_t>(p.num_q_heads) * D / 8;
        uint4* dst = reinterpret_cast<uint4*>(p.out) + s.q0 * row;
        for (int64_t i = tid; i < s.n * row; i += kSoftmaxThreads) dst[i] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

template <int D, int R>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const CrossParams& p, int ctas, cudaStream_t stream) {
  static std::atomic<uint64_t> smem_set{0};
  auto kernel = cross_attention_kernel<D, R>;
  constexpr int smem = Shape<D>::smem(R);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(smem_set.load() & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    smem_set.fetch_or(bit);
  }
  return launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem, stream, tq, tk, tv, p);
}

template <int D>
cudaError_t launch_d(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                     const CrossParams& p, int copies, int ctas, cudaStream_t stream) {
  switch (copies) {
    case 4: return launch<D, 4>(tq, tk, tv, p, ctas, stream);
    case 2: return launch<D, 2>(tq, tk, tv, p, ctas, stream);
    default: return launch<D, 1>(tq, tk, tv, p, ctas, stream);
  }
}

// The K pool as [num_blocks * Hkv * 16 rows][D] bf16, boxes of 16 rows x 64
// columns; the V pool as [D / 64 halves][rows][64], boxes of a block's 16 rows in
// every half; q as [T][Hq][D], tokens q_stride elements apart, boxes of rows / group
// tokens x group heads x 64 columns; 128-byte swizzle.
bool encode_rows(CUtensorMap* map, const void* base, int head_dim, int64_t rows) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(head_dim) * 2};
  const cuuint32_t box[2] = {64, kBS};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}
bool encode_blocks(CUtensorMap* map, const void* base, int head_dim, int64_t rows) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t halves = static_cast<cuuint64_t>(head_dim / 64);
  const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), halves};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2, 128};
  const cuuint32_t box[3] = {64, kBS, static_cast<cuuint32_t>(halves)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}
bool encode_queries(CUtensorMap* map, const void* base, int head_dim, int num_q_heads, int total_q,
                    int64_t q_stride, int group, int rows) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim),
                              static_cast<cuuint64_t>(num_q_heads),
                              static_cast<cuuint64_t>(total_q)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * 2,
                                 static_cast<cuuint64_t>(q_stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group),
                             static_cast<cuuint32_t>(rows / group)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// Rows of a workspace place: what a tile of up to max_query_len queries holds.
int cross_rows(int max_query_len, int group) {
  return max_query_len < kRows / group ? max_query_len * group : kRows;
}

pa_status cross_impl(void* out, const void* q, int64_t q_stride, const void* k_cache,
                     const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
                     const int32_t* source_lens, const int32_t* query_start_loc,
                     int max_query_len, int num_seqs, int total_query_tokens, int num_q_heads,
                     int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
                     float* ws_out, float* ws_ml, unsigned* counters, int ws_ctas,
                     pa_stream_t stream, pa_prepared** keep) {
  if (num_seqs < 0 || max_query_len < 0 || total_query_tokens < 0 || num_q_heads <= 0 ||
      num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || max_blocks_per_seq <= 0 ||
      num_blocks <= 0 || !(scale > 0.f) || ws_ctas < 1 ||
      ws_ctas > (1 << 20))
    return PA_ERR_INVALID_ARG;
  const int group = num_q_heads / num_kv_heads;
  if (!pa_cross_attention_supported(head_dim, group, block_size)) return PA_ERR_UNSUPPORTED_SHAPE;
  if (num_seqs == 0 || max_query_len == 0 || total_query_tokens == 0)
    return keep ? nothing_to_do(keep) : PA_OK;
  if (!aligned_ptr(out, 16) || !aligned_ptr(q, 16) || !aligned_ptr(k_cache, 16) ||
      !aligned_ptr(v_cache, 16) || !aligned_ptr(block_tables, 4) || !aligned_ptr(source_lens, 4) ||
      !aligned_ptr(query_start_loc, 4))
    return PA_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(num_q_heads) * head_dim || q_stride % 8 != 0 ||
      q_stride >= (1ll << 39))
    return PA_ERR_INVALID_ARG;
  // (tiles are read by one CTA after others have written theirs)
  const int64_t row = 2ll * num_q_heads * head_dim;
  if (ranges_meet(out, row * total_query_tokens, q,
                  2 * q_stride * (total_query_tokens - 1ll) + row))
    return PA_ERR_INVALID_ARG;
  if (!aligned_ptr(ws_out, 16) || !aligned_ptr(ws_ml, 16) || !aligned_ptr(counters, 4))
    return PA_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(num_blocks) * num_kv_heads * kBS;
  // (a source's length, rounded up to whole chunks, stays within 31 bits)
  if (rows > 0x7fffffffll ||
      static_cast<int64_t>(max_blocks_per_seq) * kBS > 0x7fffffffll - kKeys)
    return PA_ERR_INVALID_ARG;
  CrossParams p{};
  p.group = group;
  p.max_query_len = max_query_len < total_query_tokens ? max_query_len : total_query_tokens;
  // Copies of the rows in a tile: 4 where a sequence has 32 rows at most, 2 where 64.
  const int rows_each = cross_rows(p.max_query_len, group);
  const int copies = rows_each <= 32 ? 4 : rows_each <= 64 ? 2 : 1;
  p.tile_tokens = kRows / copies / group;
  CUtensorMap tq, tk, tv;
  if (!encode_queries(&tq, q, head_dim, num_q_heads, total_query_tokens, q_stride, group,
                      kRows / copies) ||
      !encode_rows(&tk, k_cache, head_dim, rows) || !encode_blocks(&tv, v_cache, head_dim, rows))
    return cuda_fail(cudaErrorInvalidValue);  // tensor-map encoding refused the buffers
  p.out = static_cast<__nv_bfloat16*>(out);
  p.block_tables = block_tables;
  p.source_lens = source_lens;
  p.query_start = query_start_loc;
  p.ws_o = ws_out;
  p.ws_ml = reinterpret_cast<float2*>(ws_ml);
  p.counters = counters;
  p.err = device_error_word();
  if (!p.err) return cuda_fail(cudaGetLastError());
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.total_q = total_query_tokens;
  p.ws_rows = cross_rows(p.max_query_len, group);
  p.scale_log2 = scale * 1.4426950408889634f;
  // no more CTAs than the longest sources that the tables hold could feed
  const double most = static_cast<double>((max_blocks_per_seq + kChunkBlocks - 1) / kChunkBlocks) *
                      ((p.max_query_len + p.tile_tokens - 1) / p.tile_tokens) * num_seqs *
                      num_kv_heads;
  const int ctas = most < ws_ctas ? static_cast<int>(most) : ws_ctas;
  return launch_or_keep(
      [=](cudaStream_t s) {
        return head_dim == 64 ? launch_d<64>(tq, tk, tv, p, copies, ctas, s)
                              : launch_d<128>(tq, tk, tv, p, copies, ctas, s);
      },
      keep, stream);
}

}  // namespace

}  // namespace pa

extern "C" int pa_cross_attention_supported(int head_dim, int group, int block_size) {
  return (head_dim == 64 || head_dim == 128) && block_size == 16 &&
         (group == 1 || group == 2 || group == 4 || group == 8);
}

extern "C" int pa_cross_attention_ctas(int num_sms) { return num_sms > 0 ? 2 * num_sms : 0; }

extern "C" int pa_cross_attention_rows(int max_query_len, int group) {
  return max_query_len > 0 && group > 0 ? pa::cross_rows(max_query_len, group) : 0;
}

extern "C" pa_status pa_cross_attention(
    void* out, const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* source_lens,
    const int32_t* query_start_loc, int max_query_len, int num_seqs, int total_query_tokens,
    int num_q_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks, float scale,
    float* ws_out, float* ws_ml, unsigned* counters, int ws_ctas, pa_stream_t stream) {
  return pa::cross_impl(out, q, q_stride, k_cache, v_cache, block_tables, max_blocks_per_seq,
                        source_lens, query_start_loc, max_query_len, num_seqs,
                        total_query_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                        num_blocks, scale, ws_out, ws_ml, counters, ws_ctas, stream, nullptr);
}

extern "C" pa_status pa_prepare_cross_attention(
    pa_prepared** prepared, void* out, const void* q, int64_t q_stride, const void* k_cache,
    const void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* source_lens, const int32_t* query_start_loc, int max_query_len, int num_seqs,
    int total_query_tokens, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
    int num_blocks, float scale, float* ws_out, float* ws_ml, unsigned* counters, int ws_ctas) {
  if (!prepared) return PA_ERR_INVALID_ARG;
  *prepared = nullptr;
  return pa::cross_impl(out, q, q_stride, k_cache, v_cache, block_tables, max_blocks_per_seq,
                        source_lens, query_start_loc, max_query_len, num_seqs,
                        total_query_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                        num_blocks, scale, ws_out, ws_ml, counters, ws_ctas, nullptr, prepared);
}
