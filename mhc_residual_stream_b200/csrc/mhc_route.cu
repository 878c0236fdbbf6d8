// Routing to experts on B200 (sm_100a): mhc_moe_route of libmhc.so (declared in
// include/mhc.h).
//
// Two steps. choose_rows: a warp takes a row, a lane every 32nd expert; scores,
// group values and the top-k selection stay in the warp (the winner of a round is
// found with two warp-wide integer reductions on an order-preserving key). Choices
// are computed in fp32; a row in which a decision falls closer than fp32 can tell
// is chosen again in 64 bits. place_pairs: the stable counting sort of the (row,
// slot) pairs by expert. A block owns a run of consecutive rows and has counted its
// pairs per expert; it adds up the other blocks' counts (at most 148 x E words, from
// L2), scans the experts' totals, and walks its pairs in order, 32 at a time, each
// warp its own run of them, ranking equal experts with match_any. No atomics on
// global memory and no order that depends on timing: the permutation is the same in
// every run. Up to 128 rows the two steps are one launch, a cluster of up to 8 blocks
// with a cluster barrier between them; above, two launches.
//
// Bound by latency at every size: 8191 rows x 200 experts are 7.3 MB (1.1 us of HBM
// time).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "../../include/mhc.h"
#include "mhc_device.cuh"
#include "mhc_host.cuh"

namespace mhc {

constexpr int kFewWarps = 16;          // of a block of the one-launch form
constexpr int kManyWarps = 32;         // of a block of the two launches
// Of the first of them, for V experts a lane: a block's choices in 64 bits have to fit
// its shared memory, and 32 experts a lane need more than 64 registers.
__host__ __device__ constexpr int choose_warps(int v) { return v > 16 ? 16 : kManyWarps; }
constexpr int kRouteBlocks = 148;      // most blocks: each reads every block's counts
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteSmem = 225 * 1024;
constexpr int kClusterBlocks = 8;
constexpr int kClusterRows = kClusterBlocks * kFewWarps;

struct RouteParams {
  const void* logits;
  const float* bias;
  float* weights;
  int32_t* ids;
  int32_t* e2p;
  int32_t* prow;
  int32_t* offsets;
  int* counts;  // workspace: [blocks][E] pairs of each block per expert
  int rows, E, k, chunk, blocks;
  int softmax, groups, top_groups, group_top, renorm;
  int group_magic, group_size;
  int lanes_log;  // log2 of the lanes that share a group: 32 over the group count rounded up to a power of two
  float scale;
};

// Order-preserving keys; 0 stands for "cannot be chosen" (-inf and NaN).
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  if (!(v > -INFINITY)) return 0;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ unsigned order_key(float v) {
  if (!(v > -INFINITY)) return 0;
  v += 0.f;  // -0 and +0 are equal
  const unsigned u = __float_as_uint(v);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(unsigned k) {
  return k == 0 ? -INFINITY : __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k);
}

// Whether two fp32 choices are too near to tell apart. A choice is off by at most
// `unit` + its own magnitude, in half steps of fp32 (2^-24): a sigmoid by 7 (__expf is
// within 2 + 1.17 |l| steps of the exponential, which moves the sigmoid by at most a
// quarter of the first and 0.23 of the second; an addition and __fdividef's 2 steps
// follow), an exponential over a sum of up to 1024 by 50 times the largest of the row;
// a bias adds one rounding. mag: the magnitudes that were rounded on both sides.
__device__ __forceinline__ bool too_near(float a, float b, float units, float mag) {
  return !(fabsf(a - b) > 0x1p-24f * (units + mag));
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

// The groups of the top_groups largest values: bit g << lanes_log for group g, whose
// value (key; 0: no expert is available) the lane of that number holds.
template <typename Key>
__device__ __forceinline__ unsigned best_groups(const RouteParams& p, Key value, int lane) {
  const int G = p.groups, g = lane >> p.lanes_log;
  int rank = 0;  // groups ahead of this lane's
  for (int o = 0; o < G; ++o) {
    const Key w = __shfl_sync(kFull, value, o << p.lanes_log);
    rank += w > value || (w == value && o < g) ? 1 : 0;
  }
  return __ballot_sync(kFull, g < G && rank < p.top_groups && value != 0);
}

// Whether expert e's group is in the mask of best_groups. e / S as a product: exact for
// e < 1024 (group_magic = 2^20 / S rounded up).
__device__ __forceinline__ bool in_groups(const RouteParams& p, unsigned mask, int e) {
  return mask >> ((e * p.group_magic >> 20) << p.lanes_log) & 1u;
}

// The groups that stay, choices in 64 bits in shared memory.
__device__ unsigned keep_groups(const RouteParams& p, const double* choice, int lane) {
  const int G = p.groups, S = p.group_size, per = 1 << p.lanes_log;
  const int g = lane >> p.lanes_log, sub = lane & (per - 1);
  uint64_t k1 = 0, k2 = 0;  // keys of the two largest
  double v1 = 0, v2 = 0;
  auto take = [&](uint64_t key, double v) {
    if (key > k1) {
      k2 = k1;
      v2 = v1;
      k1 = key;
      v1 = v;
    } else if (key > k2) {
      k2 = key;
      v2 = v;
    }
  };
  if (g < G)
    for (int e = sub; e < S; e += per) {
      const double v = choice[g * S + e];
      take(order_key(v), v);
    }
  for (int d = per >> 1; d > 0; d >>= 1) {
    const uint64_t o1 = __shfl_xor_sync(kFull, k1, d), o2 = __shfl_xor_sync(kFull, k2, d);
    const double w1 = __shfl_xor_sync(kFull, v1, d), w2 = __shfl_xor_sync(kFull, v2, d);
    take(o1, w1);
    take(o2, w2);
  }
  const uint64_t value = k1 == 0 ? 0 : order_key(p.group_top == 2 && k2 != 0 ? v1 + v2 : v1);
  return best_groups(p, static_cast<unsigned long long>(value), lane);
}

// The same in fp32; sets `near` where the groups that stay and those that do not cannot be
// told apart: where the least that one of the first may be worth does not exceed the most
// that one of the others may be. Each group has an error of its own (two choices of
// opposite sign may cancel, and leave a small value with their rounding), so a group of any
// rank counts. Three warp-wide maxima (8191 rows x 200 experts in 8 groups 25.0 us, as with
// only the two groups at the border compared, which kept wrong groups).
__device__ __forceinline__ unsigned keep_groups(const RouteParams& p, const float* choice, int lane, float unit,
                                                bool* near) {
  const int G = p.groups, S = p.group_size, per = 1 << p.lanes_log;
  const int g = lane >> p.lanes_log, sub = lane & (per - 1);
  float v1 = -INFINITY, v2 = -INFINITY;
  if (g < G)
    for (int e = sub; e < S; e += per) {
      const float v = choice[g * S + e];
      v2 = fmaxf(v2, fminf(v1, v));
      v1 = fmaxf(v1, v);
    }
  for (int d = per >> 1; d > 0; d >>= 1) {
    const float w1 = __shfl_xor_sync(kFull, v1, d), w2 = __shfl_xor_sync(kFull, v2, d);
    v2 = fmaxf(fmaxf(v2, w2), fminf(v1, w1));
    v1 = fmaxf(v1, w1);
  }
  const bool two = p.group_top == 2 && v2 > -INFINITY;
  const float value = two ? v1 + v2 : v1;
  const unsigned mask = best_groups(p, order_key(value), lane);
  if (p.top_groups < G) {
    const bool open = v1 > -INFINITY;  // the group has an expert that can be chosen
    const bool stays = mask >> (g << p.lanes_log) & 1u;
    // Values as their distances from the last group that stays, which are exact where they
    // are small. Their errors: those of the choices (see too_near), a rounding of the sum,
    // and what a larger distance and its bound are rounded by.
    const float d = value + warp_max(open && stays ? -value : -INFINITY);
    const float err = 0x1p-24f * (2.f * unit + fabsf(v1) + (two ? fabsf(v2) + fabsf(value) : 0.f) + 2.f * fabsf(d));
    const float least = -warp_max(open && stays ? err - d : -INFINITY);
    const float most = warp_max(open && !stays ? d + err : -INFINITY);
    // a value outside fp32's range compares with nothing
    *near = !(least > most) || __any_sync(kFull, open && !(fabsf(value) < INFINITY));
  }
  return mask;
}

// A lane's keys in descending order, equal keys by slot: odd-even merge sort.
template <int V>
__device__ __forceinline__ void sort_keys(unsigned (&key)[V], int (&slot)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k > 0; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const int a = i + j, b = i + j + k;
            const bool swap = key[b] > key[a] || (key[b] == key[a] && slot[b] < slot[a]);
            const unsigned ka = key[a];
            const int sa = slot[a];
            key[a] = swap ? key[b] : ka;
            key[b] = swap ? ka : key[b];
            slot[a] = swap ? slot[b] : sa;
            slot[b] = swap ? sa : slot[b];
          }
}

// Top-k in 64 bits: lane t gets the t-th expert (id -1: none left). For rows whose fp32
// choices decide nothing; the logits are read again.
template <typename T, int V>
__device__ __noinline__ int choose_exact(const RouteParams& p, const T* src, int lane, double* choice, float top) {
  const bool any_inf = top == INFINITY;
  const double shift = top == -INFINITY ? 0.0 : static_cast<double>(top);
  double s[V];
  double dsum = 0.0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    const float l = e < p.E ? load_logit(src + e) : -INFINITY;
    s[j] = -INFINITY;
    if (l > -INFINITY) {
      if (!p.softmax) s[j] = 1.0 / (1.0 + exp(-static_cast<double>(l)));
      else s[j] = any_inf ? (l == INFINITY ? 1.0 : 0.0) : exp(static_cast<double>(l) - shift);
      dsum += s[j];
    }
  }
  if (p.softmax) dsum = warp_sum(dsum);
  uint64_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    if (p.softmax) s[j] /= dsum;
    if (p.bias != nullptr && e < p.E) s[j] += static_cast<double>(p.bias[e]);
    key[j] = order_key(s[j]);
    // without a bias the logits order the choices
    if (p.bias == nullptr && key[j] != 0) key[j] = static_cast<uint64_t>(order_key(load_logit(src + e))) << 32;
    if (p.groups > 1 && e < p.E) choice[e] = s[j];
  }
  if (p.groups > 1) {
    __syncwarp();
    const unsigned kept = keep_groups(p, choice, lane);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (lane + 32 * j < p.E && !in_groups(p, kept, lane + 32 * j)) key[j] = 0;
    __syncwarp();  // the next row overwrites `choice`
  }
  int id = -1;
  for (int t = 0; t < p.k; ++t) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const unsigned hi = static_cast<unsigned>(best >> 32), top_hi = __reduce_max_sync(kFull, hi);
    if (top_hi == 0) break;  // nothing is left (a key that can be chosen has a nonzero high word)
    const unsigned lo = hi == top_hi ? static_cast<unsigned>(best) : 0u, top_lo = __reduce_max_sync(kFull, lo);
    const unsigned e = __reduce_min_sync(
        kFull, hi == top_hi && lo == top_lo ? static_cast<unsigned>(lane + 32 * at) : 0xffffffffu);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (static_cast<unsigned>(lane + 32 * j) == e) key[j] = 0;
    if (lane == t) id = static_cast<int>(e);
  }
  return id;
}

// The first n winners of a row (lane t: the t-th), ordered by their choices in 64 bits:
// sigmoid scores need the winners' own logits only. (8191 rows x 200 experts have some
// 16 rows with two winners too near; choosing those again in full took 12 us of 32.)
template <typename T>
__device__ __noinline__ int order_exact(const RouteParams& p, const T* src, int lane, int n, int id) {
  double d = 0.0;
  if (lane < n) d = 1.0 / (1.0 + exp(-static_cast<double>(load_logit(src + id)))) + static_cast<double>(p.bias[id]);
  int rank = 0;
  for (int o = 0; o < n; ++o) {
    const double w = __shfl_sync(kFull, d, o);
    const int e = __shfl_sync(kFull, id, o);
    rank += w > d || (w == d && e < id) ? 1 : 0;
  }
  if (lane >= n) rank = 32;
  int sorted = -1;
  for (int o = 0; o < n; ++o) {
    const int r = __shfl_sync(kFull, rank, o), e = __shfl_sync(kFull, id, o);
    if (r == lane) sorted = e;
  }
  return sorted;
}

// One row: ids and weights; the row's pairs are counted in `count` (shared memory).
template <typename T, int V>
__device__ __forceinline__ void choose_row(const RouteParams& p, int row, int lane, double* choice, int* count) {
  const T* src = static_cast<const T*>(p.logits) + static_cast<size_t>(row) * p.E;
  float l[V];
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane + 32 * j;
    l[j] = e < p.E ? load_logit(src + e) : -INFINITY;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (l[j] != l[j]) l[j] = -INFINITY;  // NaN: not available
    top = fmaxf(top, l[j]);
  }
  top = warp_max(top);
  const bool any_inf = top == INFINITY;
  const float shift = top == -INFINITY ? 0.f : top;
  const bool scored = p.bias != nullptr || p.groups > 1;
  float s[V];  // choices
  float sum = 1.f;
  if (p.softmax && (scored || !p.renorm)) {
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = any_inf ? (l[j] == INFINITY ? 1.f : 0.f) : __expf(l[j] - shift);
      sum += s[j];
    }
    sum = warp_sum(sum);
  }
  unsigned key[V];  // without a bias the logits order the choices
  bool near = false;
  float unit = 7.f;
  if (scored) {
    const float inv = p.softmax ? 1.f / fmaxf(sum, 1e-30f) : 0.f;
    if (p.softmax) unit = 50.f * inv;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane + 32 * j;
      if (p.softmax) s[j] *= inv;
      else s[j] = __fdividef(1.f, 1.f + __expf(-l[j]));
      if (p.bias != nullptr && e < p.E) s[j] += p.bias[e];
      if (l[j] == -INFINITY || s[j] != s[j]) s[j] = -INFINITY;
      key[j] = order_key(p.bias != nullptr ? s[j] : l[j]);
    }
    if (p.groups > 1) {
      float* choice32 = reinterpret_cast<float*>(choice);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (lane + 32 * j < p.E) choice32[lane + 32 * j] = s[j];
      __syncwarp();
      const unsigned kept = keep_groups(p, choice32, lane, unit, &near);
      __syncwarp();  // the next row's choices overwrite these
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (lane + 32 * j < p.E && !in_groups(p, kept, lane + 32 * j)) key[j] = 0;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = order_key(l[j]);
  }
  // top-k: lane t keeps the t-th winner; with a bias further ones, as far as they are too
  // near to the k-th to say which comes first. Up to 8 experts a lane are sorted first, so
  // that a round takes the head of the winning lane's list (39 instructions less).
  constexpr bool kSorted = V <= 8;
  int slot[V];
#pragma unroll
  for (int j = 0; j < V; ++j) slot[j] = j;
  if constexpr (kSorted) sort_keys<V>(key, slot);
  int id = -1;
  float before = 0.f, last = 0.f;  // the previous winner's choice, and the k-th's
  int n = 0;                       // winners kept: k, and those after it that are too near to it
  bool close = false;              // two neighbours are
  for (; n < 32; ++n) {
    unsigned best = key[0];
    int at = slot[0];
    if constexpr (!kSorted) {
#pragma unroll
      for (int j = 1; j < V; ++j)
        if (key[j] > best) {
          best = key[j];
          at = j;
        }
    }
    const unsigned winner = __reduce_max_sync(kFull, best);
    if (winner == 0) break;  // nothing is left
    if (p.bias != nullptr) {
      const float v = key_value(winner);
      if (n >= p.k && !too_near(last, v, 2.f * unit, fabsf(last) + fabsf(v))) break;
      close |= n > 0 && too_near(before, v, 2.f * unit, fabsf(before) + fabsf(v));
      before = v;
      if (n == p.k - 1) last = v;
    } else if (n == p.k) {
      break;
    }
    const unsigned e = __reduce_min_sync(kFull, best == winner ? static_cast<unsigned>(lane + 32 * at) : 0xffffffffu);
    const bool mine = static_cast<unsigned>(lane + 32 * at) == e && best == winner;
    if constexpr (kSorted) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        key[j] = mine ? (j + 1 < V ? key[j + 1 < V ? j + 1 : j] : 0u) : key[j];
        slot[j] = mine && j + 1 < V ? slot[j + 1 < V ? j + 1 : j] : slot[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (mine && j == at) key[j] = 0;
    }
    if (lane == n) id = static_cast<int>(e);
  }
  if (near || (close && (p.softmax || n == 32))) id = choose_exact<T, V>(p, src, lane, choice, top);
  else if (close) id = order_exact<T>(p, src, lane, n, id);
  if (lane >= p.k) id = -1;
  float chosen = id >= 0 ? load_logit(src + id) : -INFINITY;
  float w = 0.f;
  const float most = warp_max(chosen);  // the largest chosen logit
  if (id >= 0) {
    if (!p.softmax) {
      // of a negative logit e^l / (1 + e^l): e^-l leaves fp32's range at -88.7. Renormalised,
      // over the largest e^l (any factor gives the same), so that a weight underflows only
      // where its share does.
      const float t = expf(-fabsf(chosen));
      w = (chosen >= 0.f ? 1.f : p.renorm && most < 0.f ? expf(chosen - most) : t) / (1.f + t);
    } else if (any_inf) {
      w = chosen == INFINITY ? 1.f : 0.f;
    } else {
      w = expf(chosen - (p.renorm ? most : shift));  // renormalised: any shift gives the same
    }
    if (!p.renorm) w /= sum;
  }
  if (p.renorm) {
    float total = warp_sum(w);
    if (!p.softmax && most < -46.f) {
      // scores of less than 1e-20, down to none in 64 bits: the ratio in 64 bits, where
      // the sigmoid of less than -46 is the exponential (1 + e^46 is e^46 to 2^-66), which
      // unlike 1 / e^-l reaches the subnormals
      const double d = id >= 0 ? exp(static_cast<double>(chosen)) : 0.0;
      const double all = warp_sum(d);
      w = all > 0.0 ? static_cast<float>(d / all) : 0.f;
    } else {
      w = total > 0.f ? w / total : 0.f;
    }
  }
  if (lane < p.k) {
    p.weights[static_cast<size_t>(row) * p.k + lane] = w * p.scale;
    p.ids[static_cast<size_t>(row) * p.k + lane] = id;
    if (id >= 0) atomicAdd(&count[id], 1);
  }
}

// A block's rows: its counts per expert go to the workspace.
template <typename T, int V, int W>
__device__ __forceinline__ void choose_rows(const RouteParams& p, unsigned char* smem) {
  int* count = reinterpret_cast<int*>(smem);  // [E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double* choice = reinterpret_cast<double*>(smem + ((p.E * 4 + 15) & ~15)) + static_cast<size_t>(warp) * p.E;
  for (int e = threadIdx.x; e < p.E; e += W * 32) count[e] = 0;
  __syncthreads();
  griddep_wait();
  const int r0 = blockIdx.x * p.chunk, r1 = min(p.rows, r0 + p.chunk);
  for (int r = r0 + warp; r < r1; r += W) choose_row<T, V>(p, r, lane, choice, count);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += W * 32) p.counts[blockIdx.x * p.E + e] = count[e];
}

// The places of a block's pairs.
template <int W>
__device__ __forceinline__ void place_pairs(const RouteParams& p, unsigned char* smem) {
  constexpr int kThreads = W * 32;
  int* total = reinterpret_cast<int*>(smem);  // [E] pairs of each expert, then the expert's first place
  int* before = total + p.E;                  // [E] of them in the blocks before this one
  int* base = before + p.E;                   // [warps][E] next place of the warp's pairs of each expert
  __shared__ int part[W], used;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = p.E;
  const int r0 = blockIdx.x * p.chunk, r1 = min(p.rows, r0 + p.chunk);
  const int n = max(0, r1 - r0) * p.k;  // the block's pairs
  const int run = ((n + W - 1) / W + 31) & ~31;
  const int i0 = min(n, warp * run), i1 = min(n, i0 + run);
  const int32_t* ids = p.ids + static_cast<size_t>(r0) * p.k;
  for (int i = tid; i < (W + 2) * E; i += kThreads) total[i] = 0;
  __syncthreads();
  // totals over all blocks, and over the blocks before this one: the blocks are
  // divided over as many threads per expert as there are, 8 loads in flight each
  {
    const int parts = max(1, kThreads / E), each = (p.blocks + parts - 1) / parts;
    for (int w = tid; w < parts * E; w += kThreads) {
      const int e = w % E, b0 = w / E * each, b1 = min(p.blocks, b0 + each);
      int all = 0, less = 0;
      for (int b = b0; b < b1; b += 8) {
        int c[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) c[q] = b + q < b1 ? __ldcg(p.counts + (b + q) * E + e) : 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          all += c[q];
          if (b + q < static_cast<int>(blockIdx.x)) less += c[q];
        }
      }
      if (parts == 1) {
        total[e] = all;
        before[e] = less;
      } else if (b0 < b1) {
        atomicAdd(&total[e], all);
        atomicAdd(&before[e], less);
      }
    }
  }
  for (int i = i0 + lane; i < i1; i += 32) {
    const int e = __ldcg(ids + i);
    if (e >= 0) atomicAdd(&base[warp * E + e], 1);
  }
  __syncthreads();
  // exclusive scan of the totals: a warp scans a run of experts
  const int per = ((E + W - 1) / W + 31) & ~31;
  const int e0 = min(E, warp * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0 + lane; e < e1; e += 32) sum += total[e];
  sum = __reduce_add_sync(kFull, sum);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  int at = __reduce_add_sync(kFull, lane < warp ? part[lane] : 0);
  for (int e = e0; e < e1; e += 32) {
    const int c = e + lane < e1 ? total[e + lane] : 0;
    int scan = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, scan, d);
      if (lane >= d) scan += o;
    }
    if (e + lane < e1) {
      const int first = at + scan - c;
      if (blockIdx.x == 0) p.offsets[e + lane] = first;
      int next = first + before[e + lane];
#pragma unroll 8
      for (int w = 0; w < W; ++w) {
        const int d = base[w * E + e + lane];
        base[w * E + e + lane] = next;
        next += d;
      }
    }
    at += __shfl_sync(kFull, scan, 31);
  }
  if (warp == W - 1 && lane == 0) {  // the last warp's scan ends at the number of pairs
    used = at;
    if (blockIdx.x == 0) p.offsets[E] = at;
  }
  __syncthreads();
  for (int i = i0; i < i1; i += 32) {
    const int e = i + lane < i1 ? __ldcg(ids + i + lane) : -1;
    const unsigned peers = __match_any_sync(kFull, e);
    int place = -1;
    if (e >= 0) {
      place = base[warp * E + e] + __popc(peers & ((1u << lane) - 1u));
      p.prow[place] = r0 + (i + lane) / p.k;
    }
    __syncwarp();
    if (e >= 0 && lane == 31 - __clz(peers)) base[warp * E + e] = place + 1;
    if (i + lane < i1) p.e2p[static_cast<size_t>(r0) * p.k + i + lane] = place;
    __syncwarp();
  }
  // places behind the last pair
  const int pairs = p.rows * p.k;
  for (int i = used + blockIdx.x * kThreads + tid; i < pairs; i += p.blocks * kThreads) p.prow[i] = -1;
}

template <typename T, int V>
__global__ void __launch_bounds__(choose_warps(V) * 32) choose_kernel(const RouteParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  choose_rows<T, V, choose_warps(V)>(p, smem);
  griddep_launch_dependents();
}

__global__ void __launch_bounds__(kManyWarps * 32) place_kernel(const RouteParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  place_pairs<kManyWarps>(p, smem);
}

// Both steps, one cluster: the blocks' counts and ids pass through L2, ordered by
// the cluster barrier.
template <typename T, int V>
__global__ void __launch_bounds__(kFewWarps * 32) route_kernel(const RouteParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  choose_rows<T, V, kFewWarps>(p, smem);
  griddep_launch_dependents();
  __threadfence();
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  place_pairs<kFewWarps>(p, smem);
}

}  // namespace mhc

// =====================================================================================
// Host side
// =====================================================================================

namespace {

using namespace mhc;

template <typename Kern>
mhc_status launch(Kern kern, const RouteParams& p, int blocks, int threads, int cluster, size_t smem,
                  std::atomic<int>* configured, cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MHC_ERR_CUDA;
  if (configured[dev].load(std::memory_order_acquire) == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRouteSmem) != cudaSuccess) {
      (void)cudaGetLastError();
      return MHC_ERR_CUDA;
    }
    configured[dev].store(1, std::memory_order_release);
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MHC_ERR_CUDA;
  }
  return MHC_OK;
}

template <typename T, int V>
mhc_status run(RouteParams& p, cudaStream_t stream) {
  static std::atomic<int> c_fused[64], c_choose[64];
  static std::atomic<int> c_place[64];
  // a row's choices, in 64 bits where the fp32 ones decide nothing
  const size_t count = (p.E * 4 + 15) & ~15;
  const size_t choice = p.bias != nullptr || p.groups > 1 ? static_cast<size_t>(p.E) * 8 : 0;
  if (p.rows <= kClusterRows) {
    const size_t choose = count + kFewWarps * choice, place = static_cast<size_t>(kFewWarps + 2) * p.E * 4;
    p.blocks = (p.rows + kFewWarps - 1) / kFewWarps;
    p.chunk = kFewWarps;
    return launch(route_kernel<T, V>, p, p.blocks, kFewWarps * 32, p.blocks, choose > place ? choose : place, c_fused,
                  stream);
  }
  p.chunk = (p.rows + kRouteBlocks - 1) / kRouteBlocks;
  p.blocks = (p.rows + p.chunk - 1) / p.chunk;
  mhc_status st = launch(choose_kernel<T, V>, p, p.blocks, choose_warps(V) * 32, 1,
                         count + choose_warps(V) * choice, c_choose, stream);
  if (st != MHC_OK) return st;
  return launch(place_kernel, p, p.blocks, kManyWarps * 32, 1, static_cast<size_t>(kManyWarps + 2) * p.E * 4, c_place,
                stream);
}

template <typename T>
mhc_status dispatch(RouteParams& p, cudaStream_t stream) {
  if (p.E <= 64) return run<T, 2>(p, stream);
  if (p.E <= 128) return run<T, 4>(p, stream);
  if (p.E <= 256) return run<T, 8>(p, stream);
  if (p.E <= 512) return run<T, 16>(p, stream);
  return run<T, 32>(p, stream);
}

}  // namespace

extern "C" {

size_t mhc_moe_route_workspace_bytes(int rows, int experts, int top_k) {
  if (rows < 1 || rows > 65535 || experts < 1 || experts > kRouteMaxExperts || top_k < 1 || top_k > 16 ||
      top_k > experts)
    return 0;
  return kWsHeader + static_cast<size_t>(kRouteBlocks) * experts * 4;
}

mhc_status mhc_moe_route(const void* logits, int logits_bf16, const float* bias, const mhc_route_args* args,
                         float* expert_weights, int32_t* expert_ids, int32_t* expanded_idx_to_permuted_idx,
                         int32_t* permuted_rows, int32_t* expert_offsets, int rows, int experts, void* workspace,
                         size_t ws_bytes, mhc_stream stream) {
  if (!args) return MHC_ERR_INVALID_ARG;
  const size_t need = mhc_moe_route_workspace_bytes(rows, experts, args->top_k);
  if (need == 0 || args->num_groups < 1 || args->num_groups > 32 || experts % args->num_groups != 0 ||
      args->top_groups < 1 || args->top_groups > args->num_groups || args->group_top < 1 || args->group_top > 2)
    return MHC_ERR_UNSUPPORTED_SHAPE;
  if (args->score != MHC_SCORE_SOFTMAX && args->score != MHC_SCORE_SIGMOID) return MHC_ERR_INVALID_ARG;
  if (!std::isfinite(args->weight_scale)) return MHC_ERR_INVALID_ARG;
  if (!logits || !expert_weights || !expert_ids || !expanded_idx_to_permuted_idx || !permuted_rows || !expert_offsets)
    return MHC_ERR_INVALID_ARG;
  if (!aligned(logits, logits_bf16 ? 2 : 4) || !aligned(bias, 4) || !aligned(expert_weights, 4) ||
      !aligned(expert_ids, 4) || !aligned(expanded_idx_to_permuted_idx, 4) || !aligned(permuted_rows, 4) ||
      !aligned(expert_offsets, 4))
    return MHC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < need) return MHC_ERR_WORKSPACE;
  RouteParams p{};
  p.logits = logits;
  p.bias = bias;
  p.weights = expert_weights;
  p.ids = expert_ids;
  p.e2p = expanded_idx_to_permuted_idx;
  p.prow = permuted_rows;
  p.offsets = expert_offsets;
  p.counts = reinterpret_cast<int*>(static_cast<char*>(workspace) + kWsHeader);
  p.rows = rows;
  p.E = experts;
  p.k = args->top_k;
  p.softmax = args->score == MHC_SCORE_SOFTMAX;
  p.groups = args->num_groups;
  p.group_size = experts / args->num_groups;
  p.group_magic = ((1 << 20) + p.group_size - 1) / p.group_size;
  p.lanes_log = 5;
  for (int g = 1; g < p.groups; g <<= 1) --p.lanes_log;
  p.top_groups = args->top_groups;
  p.group_top = args->group_top;
  p.renorm = args->renormalize != 0;
  p.scale = args->weight_scale;
  return logits_bf16 ? dispatch<__nv_bfloat16>(p, stream) : dispatch<float>(p, stream);
}

}  // extern "C"
