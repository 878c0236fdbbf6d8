// Routing to experts on B200 (sm_100a): mhc_moe_route of libmhc.so (declared in
// include/mhc.h).
//
// Two steps. choose_rows: a warp takes a row, a lane every 32nd expert; scores,
// group values and the top-k selection stay in the warp (the winner of a round is
// found with three warp-wide integer reductions on an order-preserving key).
// place_pairs: the stable counting sort of the (row, slot) pairs by expert. A
// block owns a run of consecutive rows and has counted its pairs per expert; it
// adds up the other blocks' counts (at most 148 x E words, from L2), scans the
// experts' totals, and walks its pairs in order, 32 at a time, each warp its own
// run of them, ranking equal experts with match_any. No atomics on global memory
// and no order that depends on timing: the permutation is the same in every run.
// Up to 128 rows the two steps are one launch, a cluster of up to 8 blocks with a
// cluster barrier between them; above, two launches.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "../../include/mhc.h"
#include "mhc_device.cuh"
#include "mhc_host.cuh"

namespace mhc {

constexpr int kRouteWarps = 16;
constexpr int kRouteThreads = kRouteWarps * 32;
constexpr int kRouteBlocks = 148;      // most blocks: each reads every block's counts
constexpr int kRouteMaxExperts = 1024;
constexpr int kClusterBlocks = 8;
constexpr int kClusterRows = kClusterBlocks * kRouteWarps;

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
  float scale;
};

// Order-preserving keys; 0 stands for "cannot be chosen" (-inf and NaN).
__device__ __forceinline__ uint64_t order_key(double v) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  if (!(v > -INFINITY)) return 0;
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ uint64_t order_key(float v) {
  if (!(v > -INFINITY)) return 0;
  v += 0.f;  // -0 and +0 are equal
  const unsigned u = __float_as_uint(v);
  return static_cast<uint64_t>((u >> 31) ? ~u : (u | 0x80000000u)) << 32;
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

// The groups that stay, as a bit mask: choice[E] are the row's choices in shared
// memory (NaN or -inf: not available).
__device__ __forceinline__ unsigned keep_groups(const RouteParams& p, const double* choice, int lane) {
  const int G = p.groups, S = p.E / G;
  int per = 32;  // lanes per group: 32 over the group count rounded up to a power of two
  for (int g = 1; g < G; g <<= 1) per >>= 1;
  const int g = lane / per, sub = lane % per;
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
  int rank = 0;  // groups ahead of this lane's
  for (int o = 0; o < G; ++o) {
    const uint64_t w = __shfl_sync(kFull, value, o * per);
    rank += w > value || (w == value && o < g) ? 1 : 0;
  }
  const bool kept = g < G && rank < p.top_groups && value != 0;
  unsigned mask = 0;
  const unsigned lanes = __ballot_sync(kFull, kept);
  for (int o = 0; o < G; ++o) mask |= (lanes >> (o * per) & 1u) << o;
  return mask;
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
    if (l[j] != l[j]) l[j] = -INFINITY;  // NaN: not available
    top = fmaxf(top, l[j]);
  }
  top = warp_max(top);
  const bool any_inf = top == INFINITY;
  const float shift = top == -INFINITY ? 0.f : top;
  float sum = 1.f;
  if (p.softmax && !p.renorm) {
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) sum += any_inf ? (l[j] == INFINITY ? 1.f : 0.f) : expf(l[j] - shift);
    sum = warp_sum(sum);
  }
  uint64_t key[V];  // without a bias the logits order the choices
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = order_key(l[j]);
  if (p.bias != nullptr || p.groups > 1) {
    // score + bias in 64 bits: which of two near choices is larger must not
    // depend on the rounding of the exponential
    double s[V];
    double dsum = 0.0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (p.softmax) {
        s[j] = any_inf ? (l[j] == INFINITY ? 1.0 : 0.0) : exp(static_cast<double>(l[j]) - static_cast<double>(shift));
        dsum += s[j];
      } else {
        s[j] = 1.0 / (1.0 + exp(-static_cast<double>(l[j])));
      }
    }
    if (p.softmax) dsum = warp_sum(dsum);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane + 32 * j;
      if (p.softmax) s[j] = dsum > 0.0 ? s[j] / dsum : 0.0;
      if (p.bias != nullptr && e < p.E) s[j] += static_cast<double>(p.bias[e]);
      if (l[j] == -INFINITY) s[j] = -INFINITY;
      if (p.bias != nullptr) key[j] = order_key(s[j]);
    }
    if (p.groups > 1) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (lane + 32 * j < p.E) choice[lane + 32 * j] = s[j];
      __syncwarp();
      const unsigned kept = keep_groups(p, choice, lane);
      __syncwarp();  // the next row's choices overwrite these
      const int S = p.E / p.groups;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (lane + 32 * j < p.E && !(kept >> ((lane + 32 * j) / S) & 1u)) key[j] = 0;
    }
  }
  // top-k: lane t keeps the t-th winner
  int id = -1;
  float chosen = -INFINITY;
  for (int t = 0; t < p.k; ++t) {
    uint64_t best = 0;
    int at = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (key[j] > best) {
        best = key[j];
        at = j;
      }
    const unsigned hi = static_cast<unsigned>(best >> 32);
    const unsigned top_hi = __reduce_max_sync(kFull, hi);
    if (top_hi == 0) break;  // nothing is left (a key that can be chosen has a nonzero high word)
    const unsigned lo = hi == top_hi ? static_cast<unsigned>(best) : 0u;
    const unsigned top_lo = __reduce_max_sync(kFull, lo);
    const bool tied = hi == top_hi && lo == top_lo;
    const unsigned e = __reduce_min_sync(kFull, tied ? static_cast<unsigned>(lane + 32 * at) : 0xffffffffu);
    float v = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (static_cast<unsigned>(lane + 32 * j) == e) {
        key[j] = 0;
        v = l[j];
      }
    v = __shfl_sync(kFull, v, e & 31);
    if (lane == t) {
      id = static_cast<int>(e);
      chosen = v;
    }
  }
  float w = 0.f;
  const float most = warp_max(chosen);  // the largest chosen logit
  if (id >= 0) {
    if (!p.softmax) w = 1.f / (1.f + expf(-chosen));
    else if (any_inf) w = chosen == INFINITY ? 1.f : 0.f;
    else w = expf(chosen - (p.renorm ? most : shift));  // renormalised: any shift gives the same
    if (!p.renorm) w /= sum;
  }
  if (p.renorm) {
    float total = warp_sum(w);
    if (!p.softmax && total < 1e-20f) {
      // every chosen sigmoid is near or below fp32's range: the ratio in 64 bits
      double d = id >= 0 ? 1.0 / (1.0 + exp(-static_cast<double>(chosen))) : 0.0;
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
template <typename T, int V>
__device__ __forceinline__ void choose_rows(const RouteParams& p, unsigned char* smem) {
  int* count = reinterpret_cast<int*>(smem);  // [E]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double* choice = reinterpret_cast<double*>(smem + ((p.E * 4 + 15) & ~15)) + static_cast<size_t>(warp) * p.E;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) count[e] = 0;
  __syncthreads();
  const int r0 = blockIdx.x * p.chunk, r1 = min(p.rows, r0 + p.chunk);
  for (int r = r0 + warp; r < r1; r += kRouteWarps) choose_row<T, V>(p, r, lane, choice, count);
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) p.counts[blockIdx.x * p.E + e] = count[e];
}

// The places of a block's pairs.
__device__ __forceinline__ void place_pairs(const RouteParams& p, unsigned char* smem) {
  int* total = reinterpret_cast<int*>(smem);  // [E] pairs of each expert, then the expert's first place
  int* base = total + p.E;                    // [warps][E] next place of the warp's pairs of each expert
  __shared__ int part[kRouteWarps], used;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int E = p.E;
  const int r0 = blockIdx.x * p.chunk, r1 = min(p.rows, r0 + p.chunk);
  const int n = max(0, r1 - r0) * p.k;  // the block's pairs
  const int run = ((n + kRouteWarps - 1) / kRouteWarps + 31) & ~31;
  const int i0 = min(n, warp * run), i1 = min(n, i0 + run);
  const int32_t* ids = p.ids + static_cast<size_t>(r0) * p.k;
  for (int i = tid; i < kRouteWarps * E; i += kRouteThreads) base[i] = 0;
  __syncthreads();
  for (int i = i0 + lane; i < i1; i += 32) {
    const int e = __ldcg(ids + i);
    if (e >= 0) atomicAdd(&base[warp * E + e], 1);
  }
  // totals over all blocks, and over the blocks before this one
  int before[2] = {0, 0};  // E <= 2 * threads
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = tid + h * kRouteThreads;
    if (e < E) {
      int all = 0;
      for (int b0 = 0; b0 < p.blocks; b0 += 8) {
        int c[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) c[q] = b0 + q < p.blocks ? __ldcg(p.counts + (b0 + q) * E + e) : 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          all += c[q];
          if (b0 + q < static_cast<int>(blockIdx.x)) before[h] += c[q];
        }
      }
      total[e] = all;
    }
  }
  __syncthreads();
  // exclusive scan of the totals: warp w scans a run of E / warps experts
  const int per = ((E + kRouteWarps - 1) / kRouteWarps + 31) & ~31;
  const int e0 = min(E, warp * per), e1 = min(E, e0 + per);
  int sum = 0;
  for (int e = e0 + lane; e < e1; e += 32) sum += total[e];
  sum = __reduce_add_sync(kFull, sum);
  if (lane == 0) part[warp] = sum;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < warp; ++w) at += part[w];
  for (int e = e0; e < e1; e += 32) {
    const int c = e + lane < e1 ? total[e + lane] : 0;
    int scan = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, scan, d);
      if (lane >= d) scan += o;
    }
    if (e + lane < e1) total[e + lane] = at + scan - c;
    at += __shfl_sync(kFull, scan, 31);
  }
  if (warp == kRouteWarps - 1 && lane == 0) used = at;  // the last warp's scan ends at the number of pairs
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = tid + h * kRouteThreads;
    if (e < E) {
      if (blockIdx.x == 0) p.offsets[e] = total[e];
      int next = total[e] + before[h];
      for (int w = 0; w < kRouteWarps; ++w) {
        const int c = base[w * E + e];
        base[w * E + e] = next;
        next += c;
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[E] = used;
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
  for (int i = used + blockIdx.x * kRouteThreads + tid; i < pairs; i += p.blocks * kRouteThreads) p.prow[i] = -1;
}

template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) choose_kernel(const RouteParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  griddep_wait();
  choose_rows<T, V>(p, smem);
  griddep_launch_dependents();
}

__global__ void __launch_bounds__(kRouteThreads) place_kernel(const RouteParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  place_pairs(p, smem);
}

// Both steps, one cluster: the blocks' counts and ids pass through L2, ordered by
// the cluster barrier.
template <typename T, int V>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  griddep_wait();
  griddep_launch_dependents();
  choose_rows<T, V>(p, smem);
  __threadfence();
  __syncthreads();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  place_pairs(p, smem);
}

}  // namespace mhc

// =====================================================================================
// Host side
// =====================================================================================

namespace {

using namespace mhc;

template <typename Kern>
mhc_status launch(Kern kern, const RouteParams& p, int blocks, int cluster, size_t smem, std::atomic<int>* configured,
                  cudaStream_t stream) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MHC_ERR_CUDA;
  if (configured[dev].load(std::memory_order_acquire) == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) != cudaSuccess) {
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
  cfg.blockDim = dim3(kRouteThreads);
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
  const size_t choose = ((p.E * 4 + 15) & ~15) + (p.groups > 1 ? static_cast<size_t>(kRouteWarps) * p.E * 8 : 0);
  const size_t place = static_cast<size_t>(kRouteWarps + 1) * p.E * 4;
  if (p.rows <= kClusterRows) {
    p.blocks = (p.rows + kRouteWarps - 1) / kRouteWarps;
    p.chunk = kRouteWarps;
    return launch(route_kernel<T, V>, p, p.blocks, p.blocks, choose > place ? choose : place, c_fused, stream);
  }
  p.chunk = (p.rows + kRouteBlocks - 1) / kRouteBlocks;
  p.blocks = (p.rows + p.chunk - 1) / p.chunk;
  mhc_status st = launch(choose_kernel<T, V>, p, p.blocks, 1, choose, c_choose, stream);
  if (st != MHC_OK) return st;
  return launch(place_kernel, p, p.blocks, 1, place, c_place, stream);
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
  p.top_groups = args->top_groups;
  p.group_top = args->group_top;
  p.renorm = args->renormalize != 0;
  p.scale = args->weight_scale;
  return logits_bf16 ? dispatch<__nv_bfloat16>(p, stream) : dispatch<float>(p, stream);
}

}  // extern "C"
