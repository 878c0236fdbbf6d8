// The products of a decode step's sublayers on B200 (sm_100a): mhc_linear and
// mhc_moe_experts of libmhc.so (declared in include/mhc.h).
//
// One kernel serves both. Weights are the M side of the tensor-core product and
// tokens the N side: D[128 output features, bn tokens] = W[128, K] x[bn, K]^T
// with the accumulator in tensor memory. A decode batch has few tokens and its
// time is that of reading the weights, so a tile is 128 weight rows wide and
// only as many token columns as there are tokens; a long prompt takes up to 256
// token columns a tile. Per CTA (one per SM, persistent over its tiles):
//   warp 0     copies the operands by tensor map into a ring of shared-memory
//              stages, 128 bytes of K per stage and row, 128-byte swizzle (the
//              experts' first product gathers its token rows, four per copy);
//   warp 1     one thread issues tcgen05.mma over the stages (MXFP8: the scale
//              tiles are copied to tensor memory beside them);
//   warps 2-5  read a finished accumulator (a thread owns one output feature)
//              and write act(acc + bias) + residual.
// Dividing the work. A product of at least a tile per SM gives whole tiles to its
// persistent CTAs. A dense product of fewer divides each tile's K over a cluster of up
// to 8 CTAs: each sends its sums of every token column to the CTA of the cluster that
// finishes the column, through distributed shared memory. The experts' products, whose
// tiles only the device knows, divide the tiles that are left after the full waves
// evenly over all CTAs along the flattened (tile, K) axis; a tile shared by several
// CTAs is joined by whichever of them finishes last: all write their fp32 sums to the
// workspace and count up, the last adds them and runs the epilogue. Sums are added in
// K order in every form, so results do not depend on timing, and no CTA waits for
// another outside its own cluster. Many token rows go to the pair kernel
// (mhc_pair.cuh), two CTAs on one tile.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>


#include "../../include/mhc.h"
#include "mhc_device.cuh"
#include "mhc_host.cuh"
#include "mhc_tcgen05.cuh"

namespace mhc {

constexpr int kGemmThreads = 192;
constexpr int kTileM = 128;          // weight rows of a tile
constexpr int kMaxStages = 12;
constexpr int kGemmSmem = 227 * 1024;
constexpr int kStaticSmem = 1024;    // the barriers
// Two CTAs on an SM: (228 KB - 2 x 1 KB that the system takes) / 2, less the barriers.
constexpr int kHalfSmem = 112 * 1024;
constexpr int kMaxGrid = 160;        // CTAs the workspace has room for
constexpr int kMaxExperts = 1024;
constexpr int64_t kMinBudgetNs = 100000;  // least time limit of a bounded wait
constexpr int kMaxShares = 5;        // CTAs that share a grouped tile: up to 4 shares' worth, unaligned
constexpr int kMinShare = 24;        // K blocks
constexpr int kATile = kTileM * 128;  // bytes of a weight tile in a stage
// Workspace: the status word at byte 0, the join counters at 256, the partial sums at
// 2048. The counters must be zero when a call begins, and a call leaves them so: they lie in
// the header, which no other operator writes behind its status word, so that one
// workspace may serve several operators.
constexpr size_t kGemmCounters = 256;
constexpr size_t kGemmHeader = 2048;
static_assert(kGemmCounters + kMaxGrid * sizeof(unsigned) <= kWsHeader, "the counters lie in the header");

enum Source { kDense = 0, kGather = 1, kGrouped = 2 };

struct GemmParams {
  int rows;      // token rows of x (dense), permuted rows (grouped)
  int x_rows;    // rows that may be gathered
  int n;         // output features
  int kblocks;   // K in blocks of 128 bytes
  int m_tiles, bn, stages, nbuf, tmem_cols, experts;
  int apart;      // a cluster's sums have shared memory of their own, beside the ring
  int max_split;  // grouped: CTAs that may share a tile; dense: CTAs of a cluster, all on one tile
  unsigned idesc;
  const int32_t* offsets;  // [experts + 1]
  const int32_t* prow;     // source row of each permuted row
  const __nv_bfloat16* x;  // permute_rows_kernel: rows of k elements, x_stride apart
  int64_t x_stride;
  int k;
  const uint8_t* x_scale;
  const uint8_t* w_scale;
  const float* bias;
  const __nv_bfloat16* residual;
  int64_t res_stride;
  void* out;
  int64_t out_stride;
  int out_fp32, act;
  int read_ahead;  // the weights are not the preceding kernel's to write
  int paired;  // bf16 output (and residual) whose rows allow 4-byte accesses
  unsigned* status;
  unsigned* counters;
  float* partials;
  int64_t budget_ns;
  unsigned extra_tx;
};

// ---------------------------------------------------------------- schedule

// The tiles of a CTA: `waves` whole tiles (wave * grid + cta), then its share
// [a, b) of the remaining tiles' K blocks, flattened.
struct Schedule {
  int kb, grid, cta, waves, base, parts, total, a, b;

  // One tile per cluster of `split` CTAs, its K divided evenly.
  __device__ static Schedule by_cluster(int kblocks, int split) {
    Schedule s{kblocks, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x), 0, 0, split, 0, 0, 0};
    const int r = s.cta % split, t0 = s.cta / split * s.kb;
    s.a = t0 + static_cast<int>(static_cast<int64_t>(r) * s.kb / split);
    s.b = t0 + static_cast<int>(static_cast<int64_t>(r + 1) * s.kb / split);
    return s;
  }
  __device__ static Schedule by_tile(int tiles, int kblocks, int max_split) {
    Schedule s{kblocks, static_cast<int>(gridDim.x), static_cast<int>(blockIdx.x), 0, 0, 0, 0, 0, 0};
    s.waves = tiles / s.grid;
    s.base = s.waves * s.grid;
    const int rest = tiles - s.base;
    s.total = rest * s.kb;
    // A share of less than kMinShare K blocks is not worth the join (both products of 37
    // rows by 24 experts' 328 x 712: 30 us with shares of 2 and more, 20 without); none
    // is empty.
    s.parts = min(min(s.grid, rest * max_split), max(rest, s.total / kMinShare));
    if (s.cta < s.parts) {
      s.a = s.start_of(s.cta);
      s.b = s.start_of(s.cta + 1);
    }
    return s;
  }
  __device__ int start_of(int c) const { return static_cast<int>(static_cast<int64_t>(c) * total / parts); }
  // the CTA whose share holds flattened block w
  __device__ int owner(int w) const {
    return static_cast<int>((static_cast<int64_t>(w + 1) * parts - 1) / total);
  }
};

struct Segment {
  int tile, k0, k1;
};

struct Segments {  // iterates over a CTA's segments
  const Schedule& s;
  int wave, w;
  __device__ explicit Segments(const Schedule& s_) : s(s_), wave(0), w(s_.a) {}
  __device__ bool next(Segment& g) {
    if (wave < s.waves) {
      g.tile = wave++ * s.grid + s.cta;
      g.k0 = 0;
      g.k1 = s.kb;
      return true;
    }
    if (w >= s.b) return false;
    const int t = w / s.kb;
    g.tile = s.base + t;
    g.k0 = w - t * s.kb;
    g.k1 = min(s.kb, g.k0 + (s.b - w));
    w += g.k1 - g.k0;
    return true;
  }
};

// Token columns that each CTA of a cluster of `split` finishes, in fours.
__host__ __device__ constexpr int columns_each(int cols, int split) {
  return ((cols + split - 1) / split + 3) / 4 * 4;
}

struct TileAt {
  int m, expert, tok0, ntok;
};

// Tile index -> weight rows and tokens. Token tiles are innermost, so that the
// tiles that read the same weights are neighbours in time.
template <int SRC>
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, const int* first, const int* off, int tile,
                                          const int* order = nullptr) {
  TileAt t;
  if constexpr (SRC == kDense) {
    const int tt = (p.rows + p.bn - 1) / p.bn;
    t.m = tile / tt;
    t.expert = 0;
    t.tok0 = (tile - t.m * tt) * p.bn;
    t.ntok = min(p.bn, p.rows - t.tok0);
  } else {
    int lo = 0, hi = p.experts;  // first[lo] <= tile < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (first[mid] <= tile) lo = mid;
      else hi = mid;
    }
    const int tt = (first[lo + 1] - first[lo]) / p.m_tiles;
    const int r = tile - first[lo];
    t.expert = order != nullptr ? order[lo] : lo;
    t.m = r / tt;
    const int begin = off[t.expert], end = off[t.expert + 1];
    t.tok0 = begin + (r - t.m * tt) * p.bn;
    t.ntok = min(p.bn, end - t.tok0);
  }
  return t;
}

__host__ __device__ constexpr int round32(int v) { return (v + 31) / 32 * 32; }

// Rows of an expert's tiles in the pair kernel: nearly equal, multiples of 32 but the last.
__device__ __forceinline__ int even_rows(int n, int bn) {
  const int tt = (n + bn - 1) / bn;
  return n > 0 ? round32((n + tt - 1) / tt) : 0;
}

// Grouped, by one warp: the first permuted row of each expert (off), the experts in the
// order their tiles are taken in (`order`, or as they lie where it is null) and the first
// tile of each place of that order.
__device__ __forceinline__ void expert_tiles(const GemmParams& p, int* first, int* off, int* order, int lane) {
  const int E = p.experts;
  bool bad = false;
  for (int e = lane; e < E; e += 32) {
    const int lo = __ldcg(p.offsets + e), hi = __ldcg(p.offsets + e + 1);
    bad |= lo < 0 || hi < lo || hi > p.rows;
    off[e] = lo;
    if (e == E - 1) off[E] = hi;
  }
  __syncwarp();
  if (__any_sync(kFull, bad)) {  // offsets out of range: nothing is computed
    if (lane == 0) record_error(p.status, MHC_ERR_DEVICE_INDEX);
    for (int e = lane; e <= E; e += 32) first[e] = 0;
    return;
  }
  if (order != nullptr) {  // by falling rows of a tile, experts without rows last
    int n = 0;
    for (int c = p.bn / 32; c >= 0; --c)
      for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        const bool in = e < E && even_rows(off[min(e, E - 1) + 1] - off[min(e, E - 1)], p.bn) == 32 * c;
        const unsigned lanes = __ballot_sync(kFull, in);
        if (in) order[n + __popc(lanes & ((1u << lane) - 1u))] = e;
        n += __popc(lanes);
      }
    __syncwarp();
  }
  int run = 0;
  for (int i0 = 0; i0 < E; i0 += 32) {
    const int i = i0 + lane, e = i < E ? (order != nullptr ? order[i] : i) : 0;
    const int t = i < E ? (off[e + 1] - off[e] + p.bn - 1) / p.bn * p.m_tiles : 0;
    int scan = t;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kFull, scan, d);
      if (lane >= d) scan += o;
    }
    if (i < E) first[i] = run + scan - t;
    run += __shfl_sync(kFull, scan, 31);
  }
  if (lane == 0) first[E] = run;
}

// tile_at with an expert's rows in nearly equal tiles.
template <int SRC>
__device__ __forceinline__ TileAt tile_even(const GemmParams& p, const int* first, const int* off, const int* order,
                                            int tile) {
  TileAt t = tile_at<SRC>(p, first, off, tile, order);
  if constexpr (SRC != kDense) {
    const int begin = off[t.expert], each = even_rows(off[t.expert + 1] - begin, p.bn);
    t.tok0 = begin + (t.tok0 - begin) / p.bn * each;
    t.ntok = min(each, off[t.expert + 1] - t.tok0);
  }
  return t;
}

// A bounded mbarrier wait: false (and the status recorded) once the budget is
// used up; the roles then leave their loops.
__device__ __forceinline__ bool wait_for(uint64_t* bar, unsigned parity, const GemmParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  if (mbar_wait_bounded(bar, parity, wait_deadline(p.budget_ns))) return true;
  record_error(p.status, MHC_ERR_DEVICE_TIMEOUT);
  return false;
}

// A bounded wait on a barrier that other CTAs of the cluster arrive on, `more_ns` longer
// than the others.
__device__ __forceinline__ bool wait_for_cluster(uint64_t* bar, unsigned parity, const GemmParams& p,
                                                 int64_t more_ns = 0) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const long long deadline = wait_deadline(p.budget_ns + more_ns);
  while (!mbar_try_wait_cluster(bar, parity))
    if (clock64() > deadline) {
      record_error(p.status, MHC_ERR_DEVICE_TIMEOUT);
      return false;
    }
  return true;
}

__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same barrier, true where `ok` holds in every epilogue thread: its warps leave
// their loop together or not at all.
template <int kThreads = 128>
__device__ __forceinline__ bool epilogue_all(bool ok) {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "n"(kThreads)
      : "memory");
  return r != 0;
}

// No copy into the ring is left in flight when the CTA ends: a role that gave up waits
// (bounded) for the ring's uses first..last-1, in the order of their requests. The copying
// warp waits for those that it requested last, the issuing one for those it did not come to.
__device__ __forceinline__ void drain_ring(uint64_t* full, int stages, int first, int last, const GemmParams& p) {
  const long long deadline = wait_deadline(p.budget_ns);
  for (int i = max(first, 0); i < last; ++i)
    mbar_wait_bounded(&full[i % stages], static_cast<unsigned>(i / stages) & 1u, deadline);
}

// Every thread of the cluster: what was written before its arrival is seen after
// the wait. Whole warps.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Of the warps that have no part in a cluster's epilogue: its two barriers but the
// second one's wait, which ends the kernel.
__device__ __forceinline__ void pass_cluster_barriers(bool apart) {
  __syncwarp();
  if (!apart) cluster_arrive();
  cluster_wait();
  cluster_arrive();
}
__device__ __forceinline__ unsigned cluster_address(unsigned addr, int rank) {
  unsigned r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Shared memory to the shared memory of a CTA of the cluster, counted on its barrier.
__device__ __forceinline__ void bulk_s2cluster(unsigned dst, unsigned src, unsigned bytes, unsigned bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// Below -88.7 the exponential is infinite and the result 0 (the value is less than 3e-37 in magnitude).
__device__ __forceinline__ float silu(float v) { return v / (1.f + __expf(-v)); }

// C token columns of a warp's 32 output features (thread: feature f), from the
// sums: bias, activation, residual, one rounding, stores. Whole warps.
template <bool GATED, int C>
__device__ __forceinline__ void store_columns(const GemmParams& p, float (&v)[C], float (&u)[C], float bg, float bu,
                                              int64_t tok, int f, int ntok) {
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] += bg;
  if constexpr (GATED) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = silu(v[i]) * (u[i] + bu);
  } else if (p.act == MHC_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = silu(v[i]);
  } else if (p.act == MHC_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = 0.5f * v[i] * (1.f + erff(v[i] * 0.70710678118654752f));
  } else if (p.act == MHC_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];  // NaN stays
  }
  const int odd = f & 1;
  if (p.paired) {
    // neighbouring features exchange a value, so that a thread holds two features of
    // every other token: 4-byte accesses, half as many
    f &= ~1;
    const int64_t at = (tok + odd) * p.out_stride + f;
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + at;
    float2 y[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      const float got = __shfl_xor_sync(kFull, odd ? v[2 * i] : v[2 * i + 1], 1);
      y[i] = odd ? make_float2(got, v[2 * i + 1]) : make_float2(v[2 * i], got);
    }
    const int n = f < p.n ? ntok - odd : 0;  // this thread's tokens: 0, 2, 4, ... below n
    if (p.residual != nullptr) {
      const __nv_bfloat16* res = p.residual + (tok + odd) * p.res_stride + f;
      unsigned r[C / 2];
#pragma unroll
      for (int i = 0; i < C / 2; ++i)
        r[i] = 2 * i < n ? *reinterpret_cast<const unsigned*>(res + 2 * i * p.res_stride) : 0u;
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        y[i].x += __uint_as_float(r[i] << 16);
        y[i].y += __uint_as_float(r[i] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int i = 0; i < C / 2; ++i)
      // fp32 sums throughout; a bf16 output is rounded here, once
      if (2 * i < n) *reinterpret_cast<unsigned*>(dst + 2 * i * p.out_stride) = pack_bf16x2(y[i].x, y[i].y);
    return;
  }
  if (f >= p.n) return;
  if (p.residual != nullptr) {
    const __nv_bfloat16* res = p.residual + tok * p.res_stride + f;
    float r[C];
#pragma unroll
    for (int i = 0; i < C; ++i) r[i] = i < ntok ? __bfloat162float(res[i * p.res_stride]) : 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] += r[i];
  }
  const int64_t at = tok * p.out_stride + f;
  if (p.out_fp32) {
    float* dst = static_cast<float*>(p.out) + at;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < ntok) dst[i * p.out_stride] = v[i];
  } else {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (i < ntok) dst[i * p.out_stride] = __float2bfloat16(v[i]);
  }
}

// 16 columns of a thread's feature.
template <bool GATED>
__device__ __forceinline__ void read_sums(unsigned src, int bn, float (&v)[16], float (&u)[16]) {
  tmem_ld16(src, v);
  if constexpr (GATED) tmem_ld16(src + bn, u);
  tmem_ld_wait();
}

__device__ __forceinline__ void add4(float (&v)[4], const float4 a) {
  v[0] += a.x;
  v[1] += a.y;
  v[2] += a.z;
  v[3] += a.w;
}

// The epilogue of a tile that a cluster computes, K divided over its CTAs: token
// column c is finished by CTA c / each. A CTA lays its sums out by that CTA in the
// first part of its drained ring, [CTA][gate, up][column / 4][feature][4], and one
// bulk copy per CTA takes them to that CTA: to memory of their own beside the ring, or
// to the second part of its ring once all rings are drained; the columns that arrive
// are added in CTA order, which is K order. A CTA whose products did not come sends NaN:
// every CTA that finishes columns then gets all its bytes and waits for them, so that no
// CTA of the cluster ends while a copy still reads or writes its shared memory.
template <bool GATED>
__device__ __forceinline__ void finish_in_cluster(const GemmParams& p, const Schedule& sched, unsigned char* raw,
                                                  unsigned smem0, unsigned tmem, unsigned ring_bytes,
                                                  uint64_t* acc_full, uint64_t* sums_in, int q, int lane) {
  constexpr int kAcc = GATED ? 2 : 1;
  const int S = p.max_split, r = sched.cta % S;
  const TileAt t = tile_at<kDense>(p, nullptr, nullptr, sched.cta / S);
  const int each = columns_each(t.ntok, S), n = min(each, t.ntok - r * each);
  const int owners = (t.ntok + each - 1) / each;
  const int row = q * 32 + lane, f = t.m * kTileM + row;
  const unsigned block = kAcc * each * kTileM * 4;  // bytes of the sums for one CTA
  const unsigned sums0 = smem0 + (p.apart ? ring_bytes : columns_each(p.bn, S) * S * kAcc * kTileM * 4);
  const unsigned peer = min(lane, S - 1);
  const unsigned dst = cluster_address(sums0 + r * block, peer), bar = cluster_address(smem_u32(sums_in), peer);
  float bg = 0.f, bu = 0.f;
  if (p.bias != nullptr && f < p.n) {
    bg = p.bias[f];
    if constexpr (GATED) bu = p.bias[p.n + f];
  }
  unsigned char* out = raw + (smem0 - smem_u32(raw)) + row * 16;
  const bool ok = epilogue_all(wait_for(&acc_full[0], 0, p));
  __syncwarp();
  if (!p.apart) cluster_arrive();  // this CTA's ring is drained
  tcgen05_fence_after();
  const unsigned src = tmem + (static_cast<unsigned>(q * 32) << 16);
  int at = 0;
  unsigned to = 0;  // offset of the CTA's block
  for (int c = 0; c < t.ntok; c += 16) {
    float v[16], u[16];
    read_sums<GATED>(src + c, p.bn, v, u);
    if (!ok) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = u[i] = __int_as_float(0x7fffffff);
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      if (c + i < t.ntok) {
        *reinterpret_cast<float4*>(out + to + at * (kTileM * 4)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        if constexpr (GATED)
          *reinterpret_cast<float4*>(out + to + (each + at) * (kTileM * 4)) =
              make_float4(u[i], u[i + 1], u[i + 2], u[i + 3]);
        if ((at += 4) == each) {
          at = 0;
          to += block;
        }
      }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  epilogue_barrier();
  cluster_wait();
  if (q == 2 && lane < owners) bulk_s2cluster(dst, smem0 + lane * block, block, bar);
  __syncwarp();
  // A CTA sends at the latest when its own wait has run out, and that began no later than
  // this one: twice the limit, and the copies' own time, are enough in every case.
  const bool got = n > 0 && __all_sync(kFull, wait_for_cluster(sums_in, 0, p, p.budget_ns + kMinBudgetNs));
  if (got && ok) {
    const float4* from = reinterpret_cast<const float4*>(raw + (sums0 - smem_u32(raw))) + row;
    for (int c = 0; c < n; c += 4) {
      float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int k = 0; k < S; ++k) {
        const float4* a = from + (k * kAcc * each + c) / 4 * kTileM;
        add4(v, a[0]);
        if constexpr (GATED) add4(u, a[each / 4 * kTileM]);
      }
      store_columns<GATED, 4>(p, v, u, bg, bu, t.tok0 + r * each + c, f, n - c);
    }
  }
  __syncwarp();
  cluster_arrive();  // what was sent to this CTA is there
}

// ---------------------------------------------------------------- kernel

template <bool FP8, bool GATED, int SRC, int CTAS>
__global__ void __launch_bounds__(kGemmThreads, CTAS)
    gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_x) {
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], sums_in;
  __shared__ unsigned tmem_slot, join_slot;
  __shared__ __align__(16) int rows[SRC == kGather ? 32 : 4];  // gathered token rows of the tile being copied
  constexpr int kAcc = GATED ? 2 : 1;
  constexpr int kElems = FP8 ? 128 : 64;  // K elements of a stage's 128-byte rows
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // uniform
  const int x_bytes = p.bn * 128;
  const int sf_bytes = FP8 ? (kAcc + 1) * 512 : 0;
  const unsigned smem0 = (smem_u32(raw) + 1023u) & ~1023u;
  const unsigned x0 = smem0 + p.stages * (kAcc * kATile);
  // bn is a multiple of 16 rows, so a stage's token rows start on the 1024-byte
  // boundary that the swizzle pattern repeats at
  const unsigned sf0 = x0 + p.stages * x_bytes;
  int* first = nullptr;  // grouped: first tile of each expert, and its first permuted row
  int* off = nullptr;
  if constexpr (SRC != kDense) {
    first = reinterpret_cast<int*>(raw + (sf0 - smem_u32(raw)) + p.stages * sf_bytes);
    off = first + p.experts + 1;
  }

  if (tid == 0) {
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 128);
    }
    mbar_init(&sums_in, 1);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  int tiles;
  if constexpr (SRC == kDense) {
    tiles = p.m_tiles * ((p.rows + p.bn - 1) / p.bn);
  } else {
    // The offsets are the preceding kernel's. The second product's preceding kernel is
    // the first, which let it start only after it had itself waited for the offsets:
    // they are there (and read from L2), and the second product can ask for its
    // weights while the first ends.
    if constexpr (SRC == kGather) griddep_wait();
    if (warp == 0) expert_tiles(p, first, off, nullptr, lane);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const bool clustered = SRC == kDense && p.max_split > 1;
  if (clustered) {
    if (tid == 0) {  // the sums that the cluster will send for this CTA's columns
      const TileAt t = tile_at<SRC>(p, first, off, blockIdx.x / p.max_split);
      const int r = blockIdx.x % p.max_split, each = columns_each(t.ntok, p.max_split);
      mbar_arrive_expect_tx(&sums_in, r * each < t.ntok ? p.max_split * (kAcc * each * kTileM * 4) : 0);
    }
    __syncwarp();  // the copying warp issues from uniform registers only while it is converged
    if (p.apart) cluster_arrive();  // this CTA runs and its barriers are set
  }
  // The next kernel may start once this one has itself waited for the one before: what
  // it reads ahead of its own wait is then older than its direct predecessor.
  if constexpr (SRC == kGather) griddep_launch_dependents();
  if constexpr (SRC != kDense) tiles = first[p.experts];
  const unsigned tmem = tmem_slot;
  const Schedule sched =
      clustered ? Schedule::by_cluster(p.kblocks, p.max_split) : Schedule::by_tile(tiles, p.kblocks, p.max_split);
  const int acc_cols = kAcc * p.bn;  // of one tile

  if (warp == 0) {
    // ------------------------------------------------ copies
    const unsigned stage_bytes = kAcc * kATile + x_bytes + sf_bytes;
    auto load_w = [&](int s, const TileAt& t, int kb) {  // one lane
      mbar_arrive_expect_tx(&full[s], stage_bytes + p.extra_tx);
      const int row = (SRC == kDense ? 0 : t.expert * (kAcc * p.n)) + t.m * kTileM;
      const unsigned dst = smem0 + s * (kAcc * kATile);
      tma_load_2d(dst, &tm_w, kb * kElems, row, &full[s]);
      if constexpr (GATED) tma_load_2d(dst + kATile, &tm_w, kb * kElems, row + p.n, &full[s]);
      if constexpr (FP8) {
        unsigned char* sf = raw + (sf0 - smem_u32(raw)) + s * sf_bytes;
        bulk_g2s(sf, p.w_scale + (static_cast<size_t>(t.m) * p.kblocks + kb) * 512, 512, &full[s]);
        if constexpr (GATED)
          bulk_g2s(sf + 512, p.w_scale + (static_cast<size_t>(t.m + p.n / kTileM) * p.kblocks + kb) * 512, 512,
                   &full[s]);
      }
    };
    int ahead = 0;  // stages whose weights were requested before the wait
    if constexpr (SRC != kGather) {
      // The weights are not the preceding kernel's to write (p.read_ahead): the first
      // stages' are requested before waiting for it. (More of them asked into L2 there made every
      // product slower: 32 gated rows 15.5 us, 17.0 with 8 blocks a CTA, 18.1 with 32. The
      // gathering product, which has waited by now, is slower with its first weights asked
      // before its row numbers: experts of 1 row 121.0 us, 122.2.)
      Segments it(sched);
      Segment g;
      while (p.read_ahead && ahead < p.stages && it.next(g)) {
        const TileAt t = tile_at<SRC>(p, first, off, g.tile);
        for (int kb = g.k0; kb < g.k1 && ahead < p.stages; ++kb, ++ahead)
          if (elect_one()) load_w(ahead, t, kb);
      }
      __syncwarp();
      griddep_wait();
      griddep_launch_dependents();
    }
    Segments it(sched);
    Segment g;
    int i = 0, s = 0;
    unsigned ph = 1;
    bool ok = true;
    while (ok && it.next(g)) {
      const TileAt t = tile_at<SRC>(p, first, off, g.tile);
      if constexpr (SRC == kGather) {
        // the tile's token rows; what lies behind the last row, or names no row of
        // x, reads row 0 and is not stored, or is recorded as an error
        __syncwarp();
        for (int c = lane; c < p.bn; c += 32) {
          int r = c < t.ntok ? p.prow[t.tok0 + c] : 0;
          if (r < 0 || r >= p.x_rows) {
            record_error(p.status, MHC_ERR_DEVICE_INDEX);
            r = 0;
          }
          rows[c] = r;
        }
        __syncwarp();
      }
      for (int kb = g.k0; kb < g.k1; ++kb, ++i) {
        if (i >= ahead) {
          ok = wait_for(&empty[s], ph, p);
          if (!__all_sync(kFull, ok)) {
            ok = false;
            break;
          }
          if (elect_one()) load_w(s, t, kb);
          __syncwarp();
        }
        const unsigned dst = x0 + s * x_bytes;
        if constexpr (SRC == kGather) {
          if (elect_one())
            for (int j = 0; j < p.bn / 4; ++j)
              tma_gather4(dst + j * 512, &tm_x, kb * kElems, reinterpret_cast<const int4*>(rows)[j], &full[s]);
        } else if (elect_one()) {
          tma_load_2d(dst, &tm_x, kb * kElems, t.tok0, &full[s]);
          if constexpr (FP8)
            bulk_g2s(raw + (sf0 - smem_u32(raw)) + s * sf_bytes + kAcc * 512,
                     p.x_scale + (static_cast<size_t>(t.tok0 / 128) * p.kblocks + kb) * 512, 512, &full[s]);
        }
        __syncwarp();
        if (++s == p.stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (!ok) drain_ring(full, p.stages, i - p.stages, i, p);
    __syncwarp();
    if (clustered) pass_cluster_barriers(p.apart);
  } else if (warp == 1) {
    // ------------------------------------------------ products
    // The bounded waits start with the operands' copies: the kernel before may take long.
    if constexpr (SRC != kGather) griddep_wait();
    const unsigned a_lo = desc_lo(smem0), b_lo = desc_lo(x0), idesc = p.idesc;
    Segments it(sched);
    Segment g;
    int i = 0, s = 0, buf = 0;
    unsigned ph = 0, aph = 1;
    bool ok = true;
    while (ok && it.next(g)) {
      if (!(ok = __all_sync(kFull, wait_for(&acc_empty[buf], aph, p)))) break;
      tcgen05_fence_after();
      const unsigned d = tmem + buf * acc_cols;
      for (int kb = g.k0; kb < g.k1; ++kb, ++i) {
        if (!(ok = __all_sync(kFull, wait_for(&full[s], ph, p)))) break;
        tcgen05_fence_after();
        if (elect_one()) {
          const unsigned a = a_lo + s * (kAcc * kATile / 16), b = b_lo + s * (x_bytes / 16);
          unsigned sf = 0;
          if constexpr (FP8) {
            // one set of scale columns per stage: a set is rewritten only after
            // the products that read it have released the stage
            sf = tmem + p.nbuf * acc_cols + s * ((kAcc + 1) * 4);
            const unsigned src = sf0 + s * sf_bytes;
#pragma unroll
            for (int q = 0; q <= kAcc; ++q) tmem_copy_scales(sf + 4 * q, desc_scales(src + 512 * q));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int q = 0; q < kAcc; ++q) {
              const unsigned da = a + q * (kATile / 16) + 2 * k;
              if constexpr (FP8)
                mma_mxf8(d + q * p.bn, da, b + 2 * k, idesc | (k << 4) | (k << 29), sf + 4 * q, sf + 4 * kAcc,
                         k > 0 || kb > g.k0);
              else
                mma_bf16(d + q * p.bn, da, b + 2 * k, idesc, k > 0 || kb > g.k0);
            }
          mma_commit(&empty[s]);
          if (kb == g.k1 - 1) mma_commit(&acc_full[buf]);
        }
        __syncwarp();
        if (++s == p.stages) {
          s = 0;
          ph ^= 1;
        }
      }
      if (!ok) break;
      if (++buf == p.nbuf) {
        buf = 0;
        aph ^= 1;
      }
    }
    if (!ok) drain_ring(full, p.stages, i, i + p.stages, p);
    __syncwarp();
    if (clustered) pass_cluster_barriers(p.apart);
  } else {
    // ------------------------------------------------ epilogue
    if constexpr (SRC != kGather) griddep_wait();
    const int q = warp & 3;  // the quarter of the accumulator's lanes this warp can read
    if (clustered) finish_in_cluster<GATED>(p, sched, raw, smem0, tmem, p.stages * (kAcc * kATile + x_bytes + sf_bytes),
                                             acc_full, &sums_in, q, lane);
    Segments it(sched);
    Segment g;
    int buf = 0;
    unsigned ph = 0;
    while (!clustered && it.next(g)) {
      const TileAt t = tile_at<SRC>(p, first, off, g.tile);
      const int f = t.m * kTileM + q * 32 + lane;
      float bg = 0.f, bu = 0.f;
      if (p.bias != nullptr && f < p.n) {
        bg = p.bias[f];
        if constexpr (GATED) bu = p.bias[p.n + f];
      }
      if (!epilogue_all(wait_for(&acc_full[buf], ph, p))) break;
      tcgen05_fence_after();
      const unsigned src = tmem + buf * acc_cols + (static_cast<unsigned>(q * 32) << 16);
      const bool whole = g.k0 == 0 && g.k1 == p.kblocks;
      const size_t slot_floats = static_cast<size_t>(kAcc) * p.bn * kTileM;
      // partial sums of a shared tile in the workspace, [column][feature]
      const size_t own = static_cast<size_t>(sched.cta) * 2 + (g.k0 > 0 ? 0 : 1);
      float* slot = p.partials + own * slot_floats + q * 32 + lane;
      for (int c = 0; c < t.ntok; c += 16) {
        float v[16], u[16];
        read_sums<GATED>(src + c, p.bn, v, u);
        if (whole) {
          store_columns<GATED, 16>(p, v, u, bg, bu, t.tok0 + c, f, t.ntok - c);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < t.ntok) {
              slot[(c + i) * kTileM] = v[i];
              if constexpr (GATED) slot[(p.bn + c + i) * kTileM] = u[i];
            }
        }
      }
      tcgen05_fence_before();
      mbar_arrive(&acc_empty[buf]);
      if (++buf == p.nbuf) {
        buf = 0;
        ph ^= 1;
      }
      if (whole) continue;
      if constexpr (SRC != kDense) {
        // the tile is shared: the CTA that counts last joins the sums
        const int w0 = (g.tile - sched.base) * p.kblocks;
        const int c0 = sched.owner(w0), c1 = sched.owner(w0 + p.kblocks - 1);
        __threadfence();
        epilogue_barrier();
        if (warp == 2 && lane == 0) join_slot = atomicAdd(&p.counters[c0], 1u);
        epilogue_barrier();
        const bool last = join_slot == static_cast<unsigned>(c1 - c0);
        epilogue_barrier();  // join_slot is rewritten by the next shared tile
        if (!last) continue;
        __threadfence();
        if (warp == 2 && lane == 0) p.counters[c0] = 0;  // for the next launch
        const float* from[kMaxShares];
#pragma unroll
        for (int k = 0; k < kMaxShares; ++k) {
          const int o = min(c0 + k, c1);
          const size_t theirs = static_cast<size_t>(o) * 2 + (sched.start_of(o) > w0 ? 0 : 1);
          from[k] = p.partials + theirs * slot_floats + q * 32 + lane;
        }
        const int shares = c1 - c0 + 1;
        for (int c = 0; c < t.ntok; c += 4) {
          float v[kMaxShares][4], u[kMaxShares][4];
#pragma unroll
          for (int k = 0; k < kMaxShares; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool has = k < shares && c + i < t.ntok;
              v[k][i] = has ? __ldcg(from[k] + (c + i) * kTileM) : 0.f;
              if constexpr (GATED) u[k][i] = has ? __ldcg(from[k] + (p.bn + c + i) * kTileM) : 0.f;
            }
#pragma unroll
          for (int k = 1; k < kMaxShares; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[0][i] += v[k][i];
              if constexpr (GATED) u[0][i] += u[k][i];
            }
          store_columns<GATED, 4>(p, v[0], u[0], bg, bu, t.tok0 + c, f, t.ntok - c);
        }
      }
    }
  }
  if (clustered) {
    __syncwarp();
    cluster_wait();  // no CTA leaves while another may still send to it
  }
  tcgen05_fence_before();
  __syncthreads();
  if (warp == 1) {
    tcgen05_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

}  // namespace mhc

#include "mhc_pair.cuh"

// =====================================================================================
// Host side
// =====================================================================================

namespace {

using namespace mhc;

constexpr int kMaxTokens = 65535;
constexpr int kMaxK = 65536;
constexpr int kMaxFeatures = 1 << 20;
constexpr int kSplitCols = 32;  // most token columns of a grouped tile, which several CTAs may share

// Partial sums of the experts' shared tiles: two per CTA, gate and up.
constexpr size_t kPartialBytes = static_cast<size_t>(kMaxGrid) * 2 * kTileM * 2 * kSplitCols * 4;

// A row-major matrix as a 2-D map: rows of `cols` elements, `stride` bytes apart;
// boxes of 128 bytes x box_rows in the 128-byte swizzle. What lies outside reads
// as zero.
bool make_map2(CUtensorMap* m, const void* base, bool bytes, uint64_t cols, uint64_t rows, uint64_t stride,
               uint32_t box_rows) {
  EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return false;
  cuuint64_t d[2] = {cols, rows}, st[1] = {stride};
  cuuint32_t b[2] = {bytes ? 128u : 64u, box_rows}, e[2] = {1, 1};
  return enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), d,
             st, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles of 512 bytes (128 words), one a row; rows behind the last read as zero.
bool make_scale_map(CUtensorMap* m, const void* base, uint64_t tiles) {
  EncodeTiledFn enc = encode_tiled();
  if (enc == nullptr) return false;
  cuuint64_t d[2] = {128, tiles}, st[1] = {512};
  cuuint32_t b[2] = {128, 1}, e[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), d, st, b, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// mhc_debug_set_wait's limit, but no less than what leaves the copies and products issued
// before a wait, which take microseconds, the time to end before it gives up.
int64_t wait_budget() { return g_budget_ns > kMinBudgetNs ? g_budget_ns : kMinBudgetNs; }

// Bytes of a CTA's sums as it lays them out for its cluster, and of those it receives.
int sums_bytes(int bn, int acc, int split) { return columns_each(bn, split) * split * acc * kTileM * 4; }

// bn, kblocks and the operand types are set: the ring, tensor memory and
// instruction descriptor that go with them, and the launch.
template <bool FP8, bool GATED, int SRC, int CTAS>
mhc_status launch_gemm(GemmParams& p, const CUtensorMap& w, const CUtensorMap& x, int grid, int cluster,
                       cudaStream_t stream) {
  constexpr int acc = GATED ? 2 : 1;
  const int fixed = 1024 + (SRC == kDense ? 0 : 8 * (p.experts + 1));
  const int stage = acc * kATile + p.bn * 128 + (FP8 ? (acc + 1) * 512 : 0);
  // Tensor memory: an allocation never waits for a CTA of another launch. A kernel of one
  // CTA an SM takes more than half of the shared memory (12 stages or what fits), so it
  // shares no SM; of the others at most two fit, with half of the columns each. (Two
  // clusters that waited for each other's columns would wait for good.)
  const int limit = CTAS == 2 ? kHalfSmem : kGemmSmem - kStaticSmem;
  // A cluster's sums: apart from the ring where one CTA has the SM's memory (0.25 us
  // less than in the drained ring, which takes a barrier more on the way), in the ring
  // where two share it (three stages of 36 KB against two: 160 gated rows 17.4 us
  // against 18.6).
  const int sums = cluster > 1 ? sums_bytes(p.bn, acc, cluster) : 0;
  p.apart = CTAS == 1;
  const int beside = p.apart ? sums : 0;
  p.stages = (limit - fixed - beside) / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const int smem = fixed + p.stages * stage + beside;
  if (p.stages * stage < (p.apart ? 1 : 2) * sums) return MHC_ERR_UNSUPPORTED_SHAPE;
  auto cols = [&](int nbuf) { return nbuf * acc * p.bn + (FP8 ? p.stages * (acc + 1) * 4 : 0); };
  p.nbuf = cluster == 1 && cols(2) <= 512 / CTAS ? 2 : 1;
  p.tmem_cols = 32;
  while (p.tmem_cols < cols(p.nbuf)) p.tmem_cols *= 2;
  if (p.stages < 2 || p.tmem_cols > 512 / CTAS) return MHC_ERR_UNSUPPORTED_SHAPE;
  p.idesc = (static_cast<unsigned>(p.bn >> 3) << 17) | (static_cast<unsigned>(kTileM >> 4) << 24) |
            (FP8 ? (1u << 23) : (1u << 4) | (1u << 7) | (1u << 10));
  p.budget_ns = wait_budget();
  p.extra_tx = static_cast<unsigned>(g_extra_tx) * 16;
  auto kern = gemm_kernel<FP8, GATED, SRC, CTAS>;
  static std::atomic<int> configured[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MHC_ERR_CUDA;
  if (configured[dev].load(std::memory_order_acquire) == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem - kStaticSmem) !=
            cudaSuccess) {
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
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, p, w, x) != cudaSuccess) {
    (void)cudaGetLastError();
    return MHC_ERR_CUDA;
  }
  return MHC_OK;
}

int gemm_grid() {
  const int sms = sm_count();
  return sms < kMaxGrid ? sms : kMaxGrid;
}

int round16(int v) { return (v + 15) / 16 * 16; }

struct Plan {
  int bn, split, per_sm, grid;
  bool pair;
};

// CTAs that are resident at once in clusters of 1..8, at one and two CTAs an SM, as
// cudaOccupancyMaxActiveClusters counts them on a B200 (148 SMs in clusters of SMs
// that larger clusters do not fill).
constexpr int kRoom[2][8] = {{148, 148, 135, 132, 130, 132, 105, 120}, {296, 296, 279, 284, 280, 270, 259, 264}};

// Token columns of a tile and CTAs per tile of a dense product: the least of an
// estimate of the time, in SM cycles, over a few candidates. Its constants fit the
// times of 32 products (1-2048 rows, K 512-7168, 128-16000 features, plain, gated
// and MXFP8) with every candidate; the candidate it picks takes 2.3% more than the
// best one on average, 14% more at worst. A K block costs the largest of
//   its products, 128 x bn x 64 multiply-adds at 4096 a cycle;
//   kIssue, the least a K block takes on one SM (its copies, waits and issue);
//   its copies: what the ring holds per kLatency, at most kCopyRate bytes a cycle on
//   an SM and kL2Rate over all of them.
// A tile adds kEpilogue cycles a column, one shared by a cluster kJoinColumn. A pair
// of CTAs (mhc_pair.cuh) halves the token rows that each copies.
Plan plan_linear(const GemmParams& p, int rows, bool fp8, bool gated) {
  constexpr double kLatency = 3000, kCopyRate = 45, kL2Rate = 8600, kIssue = 600, kEpilogue = 5, kJoinColumn = 160;
  constexpr int kSplits[] = {1, 2, 3, 4, 5, 6, 8};
  const int sms = gemm_grid();
  const int acc = gated ? 2 : 1;
  const int cap = fp8 || gated ? 128 : 256;
  const int most = round16(rows < cap ? rows : cap);
  Plan best{0, 1, 1, 1, false};
  double least = 0;
  for (int c = 0; c < 6; ++c) {
    const int bn = c == 0 ? most : 8 << c;  // 16, 32, 64, 128, 256
    if (c > 0 && bn >= most) break;
    if (fp8 && rows > bn && bn != 128) continue;  // a token tile starts at a scale tile's first row
    const int tiles = p.m_tiles * ((rows + bn - 1) / bn);
    const int stage = acc * kATile + bn * 128 + (fp8 ? (acc + 1) * 512 : 0);
    const int cols = acc * bn + (fp8 ? kMaxStages * (acc + 1) * 4 : 0);
    const double bytes = acc * kATile + bn * 128;
    for (int per_sm = 1; per_sm <= 2; ++per_sm) {
      for (int split : kSplits) {
        if (split > p.kblocks || tiles * split > (split > 1 ? kRoom[per_sm - 1][split - 1] : 1 << 30)) break;
        if (split == 1 && per_sm == 2) continue;
        const int sums = split > 1 ? sums_bytes(bn, acc, split) : 0;
        const int room = per_sm == 2 ? kHalfSmem - 1024 : kGemmSmem - kStaticSmem - 1024 - sums;
        int stages = room / stage < kMaxStages ? room / stage : kMaxStages;
        if (stages < 2 || cols > 512 / per_sm || stages * stage < per_sm * sums) continue;
        const int ctas = split > 1 ? tiles * split : (tiles < sms ? tiles : sms);
        const int waves = split > 1 ? 1 : (tiles + sms - 1) / sms;
        const int blocks = (p.kblocks + split - 1) / split;
        if (waves == 1 && stages > blocks) stages = blocks;
        const double shared = ctas > sms ? static_cast<double>(ctas) / sms : 1.0;  // CTAs on one SM
        double rate = stages * bytes / kLatency;
        if (rate > kCopyRate / shared) rate = kCopyRate / shared;
        if (rate > kL2Rate / ctas) rate = kL2Rate / ctas;
        double block = (2.0 * acc * bn > kIssue ? 2.0 * acc * bn : kIssue) * shared;
        if (block < bytes / rate) block = bytes / rate;
        const double t = waves * blocks * block +
                         (split > 1 ? kJoinColumn : kEpilogue) * acc * bn;
        if (best.bn == 0 || t < least) {
          least = t;
          best = Plan{bn, split, per_sm, ctas, false};
        }
      }
    }
  }
  if (fp8 ? !gated && rows > 128 : rows > 64) {
    const int bn = rows < 256 && !fp8 ? round32(rows) : 256;  // MXFP8: tiles start at a scale tile's first row
    const int waves = ((p.n + kPairTileM - 1) / kPairTileM * ((rows + bn - 1) / bn) + sms / 2 - 1) / (sms / 2);
    const double copies = (acc * kATile + bn / 2 * 128) / kCopyRate, products = 2.0 * acc * bn;
    double block = copies > products ? copies : products;
    if (block < kIssue) block = kIssue;
    if (waves * p.kblocks * block + kEpilogue * acc * bn < least) best = Plan{bn, 1, 1, sms / 2 * 2, true};
  }
  return best;
}

template <bool FP8, bool GATED, int SRC>
mhc_status launch_pair(GemmParams& p, const CUtensorMap& w, const CUtensorMap& x, const CUtensorMap& ws,
                       const CUtensorMap& xs, cudaStream_t stream) {
  constexpr int acc = GATED ? 2 : 1;
  const int fixed = 1024 + (SRC == kDense ? 0 : 12 * (p.experts + 1));
  const int stage = acc * kATile + p.bn / 2 * 128 + (FP8 ? 3 * 512 : 0);
  p.stages = (kGemmSmem - kStaticSmem - fixed) / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const int scale_cols = FP8 ? p.stages * 12 : 0;
  p.nbuf = 2 * acc * p.bn + scale_cols <= 512 ? 2 : 1;
  if (p.stages < 2 || p.bn % 32 != 0 || acc * p.bn + scale_cols > 512) return MHC_ERR_UNSUPPORTED_SHAPE;
  p.m_tiles = (p.n + kPairTileM - 1) / kPairTileM;
  p.idesc = (static_cast<unsigned>(kPairTileM >> 4) << 24) | (FP8 ? 1u << 23 : (1u << 4) | (1u << 7) | (1u << 10));
  p.budget_ns = wait_budget();
  p.extra_tx = static_cast<unsigned>(g_extra_tx) * 16;
  auto kern = pair_kernel<FP8, GATED, SRC>;
  static std::atomic<int> configured[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MHC_ERR_CUDA;
  if (configured[dev].load(std::memory_order_acquire) == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem - kStaticSmem) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return MHC_ERR_CUDA;
    }
    configured[dev].store(1, std::memory_order_release);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gemm_grid() / 2 * 2);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = fixed + p.stages * stage;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p, w, x, ws, xs) != cudaSuccess) {
    (void)cudaGetLastError();
    return MHC_ERR_CUDA;
  }
  return MHC_OK;
}

template <bool FP8, bool GATED>
mhc_status launch_linear(GemmParams& p, const Plan& plan, const CUtensorMap& w, const CUtensorMap& x,
                         cudaStream_t stream) {
  return plan.per_sm == 2 ? launch_gemm<FP8, GATED, kDense, 2>(p, w, x, plan.grid, plan.split, stream)
                          : launch_gemm<FP8, GATED, kDense, 1>(p, w, x, plan.grid, plan.split, stream);
}

bool linear_shape(int rows, int in_features, int out_features, bool fp8, bool gated) {
  return rows >= 1 && rows <= kMaxTokens && in_features >= 1 && in_features <= kMaxK && out_features >= 1 &&
         out_features <= kMaxFeatures && in_features % (fp8 ? 32 : 8) == 0 &&
         !(fp8 && gated && out_features % kTileM != 0);
}

GemmParams linear_sizes(int rows, int in_features, int out_features, bool fp8) {
  GemmParams p{};
  p.rows = rows;
  p.n = out_features;
  p.kblocks = fp8 ? (in_features + 127) / 128 : (in_features + 63) / 64;
  p.m_tiles = (out_features + kTileM - 1) / kTileM;
  return p;
}

}  // namespace

extern "C" {

mhc_status mhc_debug_linear_form(int rows, int in_features, int out_features, int mxfp8, int gated, int* form) {
  if (!form) return MHC_ERR_INVALID_ARG;
  const bool fp8 = mxfp8 != 0;
  if (!linear_shape(rows, in_features, out_features, fp8, gated != 0)) return MHC_ERR_UNSUPPORTED_SHAPE;
  const Plan plan = plan_linear(linear_sizes(rows, in_features, out_features, fp8), rows, fp8, gated != 0);
  form[0] = plan.pair;
  form[1] = plan.split;
  form[2] = plan.per_sm;
  form[3] = plan.bn;
  return MHC_OK;
}

size_t mhc_linear_workspace_bytes(int rows) {
  if (rows < 1 || rows > kMaxTokens) return 0;
  return kGemmHeader;
}

mhc_status mhc_linear(const void* x, const uint8_t* x_scale, int64_t x_stride, const void* weight,
                      const uint8_t* weight_scale, const float* bias, mhc_activation activation,
                      const mhc_bf16* residual, int64_t residual_stride, void* out, int out_fp32, int64_t out_stride,
                      int rows, int in_features, int out_features, int read_ahead, void* workspace,
                      size_t ws_bytes, mhc_stream stream) {
  const bool fp8 = weight_scale != nullptr;
  const bool gated = activation == MHC_ACT_SWIGLU;
  if (!linear_shape(rows, in_features, out_features, fp8, gated)) return MHC_ERR_UNSUPPORTED_SHAPE;
  if (activation < MHC_ACT_NONE || activation > MHC_ACT_SWIGLU) return MHC_ERR_INVALID_ARG;
  if (!x || !weight || !out || (x_scale != nullptr) != fp8) return MHC_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(x_scale, 16) || !aligned(weight_scale, 16) ||
      !aligned(bias, 4) || !aligned(residual, 2) || !aligned(out, out_fp32 ? 4 : 2))
    return MHC_ERR_INVALID_ARG;
  const int64_t row_bytes = fp8 ? 1 : 2;
  if (x_stride < in_features || (x_stride * row_bytes) % 16 != 0 || out_stride < out_features ||
      (residual && residual_stride < out_features))
    return MHC_ERR_INVALID_ARG;
  if (static_cast<const void*>(residual) == out && (out_fp32 || residual_stride != out_stride))
    return MHC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < mhc_linear_workspace_bytes(rows)) return MHC_ERR_WORKSPACE;
  GemmParams p = linear_sizes(rows, in_features, out_features, fp8);
  p.x_scale = x_scale;
  p.w_scale = weight_scale;
  p.bias = bias;
  p.residual = reinterpret_cast<const __nv_bfloat16*>(residual);
  p.res_stride = residual_stride;
  p.out = out;
  p.out_stride = out_stride;
  p.out_fp32 = out_fp32 != 0;
  p.act = activation;
  p.read_ahead = read_ahead != 0;
  p.paired = !out_fp32 && aligned(out, 4) && out_stride % 2 == 0 && out_features % 2 == 0 && aligned(residual, 4) &&
             residual_stride % 2 == 0;
  p.status = static_cast<unsigned*>(workspace);
  const Plan plan = plan_linear(p, rows, fp8, gated);
  const bool pair = plan.pair;
  p.bn = plan.bn;
  p.max_split = plan.split;
  CUtensorMap mw, mx;
  const uint64_t wrows = static_cast<uint64_t>(out_features) * (gated ? 2 : 1);
  if (!make_map2(&mw, weight, fp8, in_features, wrows, static_cast<uint64_t>(in_features) * row_bytes, kTileM) ||
      !make_map2(&mx, x, fp8, in_features, rows, static_cast<uint64_t>(x_stride) * row_bytes, pair ? p.bn / 2 : p.bn))
    return MHC_ERR_CUDA;
  if (pair && fp8) {
    CUtensorMap ms, mt;
    if (!make_scale_map(&ms, weight_scale, (out_features + 127) / 128 * p.kblocks) ||
        !make_scale_map(&mt, x_scale, (rows + 127) / 128 * p.kblocks))
      return MHC_ERR_CUDA;
    return launch_pair<true, false, kDense>(p, mw, mx, ms, mt, stream);
  }
  if (pair) return gated ? launch_pair<false, true, kDense>(p, mw, mx, mw, mx, stream)
                         : launch_pair<false, false, kDense>(p, mw, mx, mw, mx, stream);
  if (fp8) return gated ? launch_linear<true, true>(p, plan, mw, mx, stream)
                        : launch_linear<true, false>(p, plan, mw, mx, stream);
  return gated ? launch_linear<false, true>(p, plan, mw, mx, stream)
               : launch_linear<false, false>(p, plan, mw, mx, stream);
}

size_t mhc_moe_experts_workspace_bytes(int rows, int num_permuted, int intermediate) {
  if (rows < 1 || rows > kMaxTokens || num_permuted < 1 || intermediate < 1) return 0;
  return kGemmHeader + kPartialBytes + static_cast<size_t>(num_permuted) * intermediate * 2;
}

mhc_status mhc_moe_experts(const mhc_bf16* x, int64_t x_stride, const mhc_bf16* w13, const mhc_bf16* w2,
                           const int32_t* permuted_rows, const int32_t* expert_offsets, mhc_bf16* gemm2_permuted,
                           int rows, int num_permuted, int experts, int hidden, int intermediate, void* workspace,
                           size_t ws_bytes, mhc_stream stream) {
  if (rows < 1 || rows > kMaxTokens || num_permuted < 1 || num_permuted > kMaxTokens * 16 || experts < 1 ||
      experts > kMaxExperts || hidden < 8 || hidden > kMaxK || hidden % 8 != 0 || intermediate < 8 ||
      intermediate > kMaxK || intermediate % 8 != 0)
    return MHC_ERR_UNSUPPORTED_SHAPE;
  if (!x || !w13 || !w2 || !permuted_rows || !expert_offsets || !gemm2_permuted) return MHC_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(gemm2_permuted, 16) ||
      !aligned(permuted_rows, 4) || !aligned(expert_offsets, 4) || x_stride < hidden || x_stride % 8 != 0)
    return MHC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      ws_bytes < mhc_moe_experts_workspace_bytes(rows, num_permuted, intermediate))
    return MHC_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  __nv_bfloat16* inner = reinterpret_cast<__nv_bfloat16*>(ws + kGemmHeader + kPartialBytes);
  GemmParams p{};
  p.rows = num_permuted;
  p.x_rows = rows;
  p.experts = experts;
  p.paired = 1;
  p.read_ahead = 1;  // of w2, while the first product ends
  p.offsets = expert_offsets;
  p.prow = permuted_rows;
  p.status = reinterpret_cast<unsigned*>(ws);
  p.counters = reinterpret_cast<unsigned*>(ws + kGemmCounters);
  p.partials = reinterpret_cast<float*>(ws + kGemmHeader);
  // By the mean number of an expert's rows. From 12, or from 8 where the weights make
  // two waves of pair tiles, the pair kernel, whose tile takes up to 256 rows of an
  // expert (B200, us against tiles of 16-128 rows gathered by tensor map, best of
  // them; E x 7168 x 2048 unless given): mean 8 786 / 803, 16 816 / 841, 48 865 / 1018,
  // 64 891 / 1185, 50 (8 experts, 4096 x 1024) 57 / 69; mean 8 (24 experts, 4096 x
  // 1024, 1.3 waves) 114 / 103, mean 4 245 / 227. Below, tiles of 16 or 32 rows: 18.5
  // against 20.5 at a mean of 4.6, equal at 8.
  const int mean = num_permuted / experts;
  const bool pair = mean >= 12 || (mean >= 8 && static_cast<int64_t>(experts) * ((intermediate + 255) / 256) >=
                                                    gemm_grid());
  const int bn = pair ? 256 : mean < 6 || rows <= 16 ? 16 : 32;
  p.bn = bn;
  p.k = hidden;
  p.x = reinterpret_cast<const __nv_bfloat16*>(x);
  p.x_stride = x_stride;
  p.max_split = kMaxShares - 1;
  const int grid = gemm_grid();
  CUtensorMap mw, mx;
  // first product: gate and up rows of an expert's w13, token rows gathered
  p.n = intermediate;
  p.kblocks = (hidden + 63) / 64;
  p.m_tiles = (intermediate + kTileM - 1) / kTileM;
  p.out = inner;  // in bf16, the tensor cores' operand type: each value is off by 2^-8 of itself at most
  p.out_stride = intermediate;
  p.act = MHC_ACT_SWIGLU;
  if (!make_map2(&mw, w13, false, hidden, static_cast<uint64_t>(experts) * 2 * intermediate,
                 static_cast<uint64_t>(hidden) * 2, kTileM))
    return MHC_ERR_CUDA;
  mhc_status st;
  if (pair) {
    // the permuted rows stand in gemm2_permuted until the second product writes it
    if (!make_map2(&mx, gemm2_permuted, false, hidden, num_permuted, static_cast<uint64_t>(hidden) * 2, 16))
      return MHC_ERR_CUDA;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid * 8);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, permute_rows_kernel, p, reinterpret_cast<__nv_bfloat16*>(gemm2_permuted)) !=
        cudaSuccess) {
      (void)cudaGetLastError();
      return MHC_ERR_CUDA;
    }
    st = launch_pair<false, true, kGrouped>(p, mw, mx, mw, mx, stream);
  } else {
    if (!make_map2(&mx, x, false, hidden, rows, static_cast<uint64_t>(x_stride) * 2, 1)) return MHC_ERR_CUDA;
    st = launch_gemm<false, true, kGather, 1>(p, mw, mx, grid, 1, stream);
  }
  if (st != MHC_OK) return st;
  // second product: the intermediate rows as they lie
  p.n = hidden;
  p.kblocks = (intermediate + 63) / 64;
  p.m_tiles = (hidden + kTileM - 1) / kTileM;
  p.out = gemm2_permuted;
  p.out_stride = hidden;
  p.act = MHC_ACT_NONE;
  if (!make_map2(&mw, w2, false, intermediate, static_cast<uint64_t>(experts) * hidden,
                 static_cast<uint64_t>(intermediate) * 2, kTileM) ||
      !make_map2(&mx, inner, false, intermediate, num_permuted, static_cast<uint64_t>(intermediate) * 2,
                 pair ? 16 : p.bn))
    return MHC_ERR_CUDA;
  if (pair) return launch_pair<false, false, kGrouped>(p, mw, mx, mw, mx, stream);
  return launch_gemm<false, false, kGrouped, 1>(p, mw, mx, grid, 1, stream);
}

}  // extern "C"
