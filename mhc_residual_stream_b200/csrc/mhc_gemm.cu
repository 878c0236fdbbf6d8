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
// Tiles: as many full waves as there are take whole tiles; the rest is divided
// evenly over the CTAs along the flattened (tile, K) axis, so a product of few
// tiles still reads its weights with every SM. A tile shared by several CTAs is
// joined by whichever of them finishes last: all write their fp32 sums to the
// workspace and count up; the last adds them in K order (the result does not
// depend on who is last) and runs the epilogue. Nobody waits for anybody.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstring>

#include "../../include/mhc.h"
#include "mhc_device.cuh"
#include "mhc_host.cuh"
#include "mhc_tcgen05.cuh"

namespace mhc {

constexpr int kGemmThreads = 192;
constexpr int kTileM = 128;          // weight rows of a tile
constexpr int kMaxStages = 12;
constexpr int kGemmSmem = 227 * 1024;
constexpr int kMaxGrid = 160;        // CTAs the workspace has room for
constexpr int kMaxExperts = 1024;
constexpr int kATile = kTileM * 128;  // bytes of a weight tile in a stage
// Workspace: the status word at byte 0, the join counters at 1024, the partial
// sums at 2048.
constexpr size_t kGemmCounters = 1024;
constexpr size_t kGemmHeader = 2048;

enum Source { kDense = 0, kGather = 1, kGrouped = 2 };

struct GemmParams {
  int rows;      // token rows of x (dense), permuted rows (grouped)
  int x_rows;    // rows that may be gathered
  int n;         // output features
  int kblocks;   // K in blocks of 128 bytes
  int m_tiles, bn, stages, nbuf, tmem_cols, experts, max_split;
  unsigned idesc;
  const int32_t* offsets;  // [experts + 1]
  const int32_t* prow;     // source row of each permuted row
  const uint8_t* x_scale;
  const uint8_t* w_scale;
  const float* bias;
  const __nv_bfloat16* residual;
  int64_t res_stride;
  void* out;
  int64_t out_stride;
  int out_fp32, act;
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

  __device__ Schedule(int tiles, int kblocks, int max_split) {
    kb = kblocks;
    grid = gridDim.x;
    cta = blockIdx.x;
    waves = tiles / grid;
    base = waves * grid;
    const int rest = tiles - base;
    total = rest * kb;
    // at least two K blocks a share (and so none is empty), unless a tile has but one
    parts = min(min(grid, rest * max_split), max(rest, total / 2));
    a = cta < parts ? static_cast<int>(static_cast<int64_t>(cta) * total / parts) : 0;
    b = cta < parts ? static_cast<int>(static_cast<int64_t>(cta + 1) * total / parts) : 0;
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

struct TileAt {
  int m, expert, tok0, ntok;
};

// Tile index -> weight rows and tokens. Token tiles are innermost, so that the
// tiles that read the same weights are neighbours in time.
template <int SRC>
__device__ __forceinline__ TileAt tile_at(const GemmParams& p, const int* first, const int* off, int tile) {
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
    t.expert = lo;
    t.m = r / tt;
    const int begin = off[lo], end = off[lo + 1];
    t.tok0 = begin + (r - t.m * tt) * p.bn;
    t.ntok = min(p.bn, end - t.tok0);
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

__device__ __forceinline__ void epilogue_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The same barrier, true where `ok` holds in every epilogue thread: the four warps
// leave their loop together or not at all.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  unsigned r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float silu(float v) { return v / (1.f + __expf(-v)); }

__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MHC_ACT_RELU: return v > 0.f ? v : (v == v ? 0.f : v);
    case MHC_ACT_SILU: return silu(v);
    case MHC_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    default: return v;
  }
}

// 16 token columns of a thread's output feature: activation, residual, store.
template <bool GATED>
__device__ __forceinline__ void store16(const GemmParams& p, float (&v)[16], float (&u)[16], float bg, float bu,
                                        int64_t tok, int f, int ntok) {
  float res[16];
  if (p.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      res[i] = i < ntok ? __bfloat162float(p.residual[(tok + i) * p.res_stride + f]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float y = v[i] + bg;
    y = GATED ? silu(y) * (u[i] + bu) : activate(y, p.act);
    if (p.residual != nullptr) y += res[i];
    if (i < ntok) {
      const int64_t at = (tok + i) * p.out_stride + f;
      // fp32 sums throughout; a bf16 output is rounded here, once
      if (p.out_fp32) static_cast<float*>(p.out)[at] = y;
      else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(y);
    }
  }
}

// ---------------------------------------------------------------- kernel

template <bool FP8, bool GATED, int SRC>
__global__ void __launch_bounds__(kGemmThreads, 1)
    gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_x) {
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  __shared__ unsigned tmem_slot, join_slot;
  constexpr int kAcc = GATED ? 2 : 1;
  constexpr int kElems = FP8 ? 128 : 64;  // K elements of a stage's 128-byte rows
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, p.tmem_cols);
    tmem_relinquish();
  }
  int tiles;
  if constexpr (SRC == kDense) {
    tiles = p.m_tiles * ((p.rows + p.bn - 1) / p.bn);
  } else {
    griddep_wait();  // the offsets are the preceding kernel's
    if (warp == 0) {
      int run = 0;
      bool bad = false;
      for (int e0 = 0; e0 < p.experts; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < p.experts) {
          lo = p.offsets[e];
          hi = p.offsets[e + 1];
          bad |= lo < 0 || hi < lo || hi > p.rows;
          lo = min(max(lo, 0), p.rows);
          hi = min(max(hi, lo), p.rows);
        }
        int t = (hi - lo + p.bn - 1) / p.bn * p.m_tiles;
        int scan = t;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(kFull, scan, d);
          if (lane >= d) scan += o;
        }
        if (e < p.experts) {
          first[e] = run + scan - t;
          off[e] = lo;
          if (e == p.experts - 1) off[p.experts] = hi;
        }
        run += __shfl_sync(kFull, scan, 31);
      }
      if (lane == 0) first[p.experts] = run;
      if (__any_sync(kFull, bad)) {  // offsets out of range: nothing is computed
        if (lane == 0) record_error(p.status, MHC_ERR_DEVICE_INDEX);
        __syncwarp();
        for (int e = lane; e <= p.experts; e += 32) first[e] = 0;
      }
    }
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  if constexpr (SRC != kDense) tiles = first[p.experts];
  const unsigned tmem = tmem_slot;
  const Schedule sched(tiles, p.kblocks, p.max_split);
  const int acc_cols = kAcc * p.bn;

  if (warp == 0) {
    // ------------------------------------------------ copies
    const unsigned stage_bytes = kAcc * kATile + x_bytes + sf_bytes;
    auto load_w = [&](int s, const TileAt& t, int kb) {  // lane 0
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
    if constexpr (SRC == kDense) {
      // The weights are not the preceding kernel's to write: the first stages'
      // are requested before waiting for it.
      if (lane == 0) {
        Segments it(sched);
        Segment g;
        while (ahead < p.stages && it.next(g)) {
          const TileAt t = tile_at<SRC>(p, first, off, g.tile);
          for (int kb = g.k0; kb < g.k1 && ahead < p.stages; ++kb) load_w(ahead++, t, kb);
        }
      }
      ahead = __shfl_sync(kFull, ahead, 0);
      griddep_wait();
    }
    Segments it(sched);
    Segment g;
    int i = 0, s = 0;
    unsigned ph = 1;
    bool ok = true;
    while (ok && it.next(g)) {
      const TileAt t = tile_at<SRC>(p, first, off, g.tile);
      int4 idx = make_int4(0, 0, 0, 0);
      if constexpr (SRC == kGather) {
        // lane l gathers rows 4l..4l+3 of the tile; what lies behind the last
        // row, or names no row of x, reads row 0 and is not stored, or is
        // recorded as an error
        int r[4];
        bool bad = false;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = 4 * lane + q;
          r[q] = c < t.ntok ? p.prow[t.tok0 + c] : 0;
          if (r[q] < 0 || r[q] >= p.x_rows) {
            bad = true;
            r[q] = 0;
          }
        }
        if (bad) record_error(p.status, MHC_ERR_DEVICE_INDEX);
        idx = make_int4(r[0], r[1], r[2], r[3]);
      }
      for (int kb = g.k0; kb < g.k1; ++kb, ++i) {
        if (i >= ahead) {
          ok = wait_for(&empty[s], ph, p);
          if (!__all_sync(kFull, ok)) {
            ok = false;
            break;
          }
          if (lane == 0) load_w(s, t, kb);
          __syncwarp();
        }
        const unsigned dst = x0 + s * x_bytes;
        if constexpr (SRC == kGather) {
          if (lane < p.bn / 4) tma_gather4(dst + lane * 512, &tm_x, kb * kElems, idx, &full[s]);
        } else if (lane == 0) {
          tma_load_2d(dst, &tm_x, kb * kElems, t.tok0, &full[s]);
          if constexpr (FP8)
            bulk_g2s(raw + (sf0 - smem_u32(raw)) + s * sf_bytes + kAcc * 512,
                     p.x_scale + (static_cast<size_t>(t.tok0 / 128) * p.kblocks + kb) * 512, 512, &full[s]);
        }
        if (++s == p.stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    griddep_launch_dependents();
    if (!ok) {  // leave no copy in flight behind: wait (bounded) for the requested stages
      const long long deadline = wait_deadline(p.budget_ns);
      for (int q = 0; q < p.stages && q < i; ++q) {
        const unsigned n = static_cast<unsigned>((i - 1 - q) / p.stages);  // uses of stage q completed or in flight
        mbar_wait_bounded(&full[q], n & 1u, deadline);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------ products
    if (lane == 0) {
      Segments it(sched);
      Segment g;
      int s = 0, buf = 0;
      unsigned ph = 0, aph = 1;
      bool ok = true;
      while (ok && it.next(g)) {
        if (!(ok = wait_for(&acc_empty[buf], aph, p))) break;
        tcgen05_fence_after();
        const unsigned d = tmem + buf * acc_cols;
        for (int kb = g.k0; kb < g.k1; ++kb) {
          if (!(ok = wait_for(&full[s], ph, p))) break;
          tcgen05_fence_after();
          const unsigned a = smem0 + s * (kAcc * kATile), b = x0 + s * x_bytes;
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
          for (int q = 0; q < kAcc; ++q) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint64_t da = desc_sw128(a + q * kATile) + 2 * k, db = desc_sw128(b) + 2 * k;
              const bool accumulate = kb > g.k0 || k > 0;
              if constexpr (FP8)
                mma_mxf8(d + q * p.bn, da, db, p.idesc | (k << 4) | (k << 29), sf + 4 * q, sf + 4 * kAcc, accumulate);
              else
                mma_bf16(d + q * p.bn, da, db, p.idesc, accumulate);
            }
          }
          mma_commit(&empty[s]);
          if (++s == p.stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        mma_commit(&acc_full[buf]);
        if (++buf == p.nbuf) {
          buf = 0;
          aph ^= 1;
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue
    if constexpr (SRC == kDense) griddep_wait();
    const int q = warp & 3;  // the quarter of the accumulator's lanes this warp can read
    Segments it(sched);
    Segment g;
    int buf = 0;
    unsigned ph = 0;
    while (it.next(g)) {
      const TileAt t = tile_at<SRC>(p, first, off, g.tile);
      const int f = t.m * kTileM + q * 32 + lane;
      const bool mine = f < p.n;
      float bg = 0.f, bu = 0.f;
      if (p.bias != nullptr && mine) {
        bg = p.bias[f];
        if constexpr (GATED) bu = p.bias[p.n + f];
      }
      if (!epilogue_all(wait_for(&acc_full[buf], ph, p))) break;
      tcgen05_fence_after();
      const unsigned src = tmem + buf * acc_cols + (static_cast<unsigned>(q * 32) << 16);
      const bool whole = g.k0 == 0 && g.k1 == p.kblocks;
      const size_t slot_floats = static_cast<size_t>(acc_cols) * kTileM;
      float* slot = p.partials + (static_cast<size_t>(sched.cta) * 2 + (g.k0 > 0 ? 0 : 1)) * slot_floats + q * 32 + lane;
      for (int c = 0; c < t.ntok; c += 16) {
        float v[16], u[16];
        tmem_ld16(src + c, v);
        if constexpr (GATED) tmem_ld16(src + p.bn + c, u);
        tmem_ld_wait();
        if (whole) {
          if (mine) store16<GATED>(p, v, u, bg, bu, t.tok0 + c, f, t.ntok - c);
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
      for (int c = 0; c < t.ntok; c += 16) {
        float v[16], u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = u[i] = 0.f;
        for (int k = c0; k <= c1; ++k) {
          const float* from = p.partials +
                              (static_cast<size_t>(k) * 2 + (sched.start_of(k) > w0 ? 0 : 1)) * slot_floats + q * 32 +
                              lane;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < t.ntok) {
              v[i] += __ldcg(from + (c + i) * kTileM);
              if constexpr (GATED) u[i] += __ldcg(from + (p.bn + c + i) * kTileM);
            }
        }
        if (mine) store16<GATED>(p, v, u, bg, bu, t.tok0 + c, f, t.ntok - c);
      }
    }
  }
  tcgen05_fence_before();
  __syncthreads();
  if (warp == 1) {
    tcgen05_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

}  // namespace mhc

// =====================================================================================
// Host side
// =====================================================================================

namespace {

using namespace mhc;

constexpr int kMaxTokens = 65535;
constexpr int kMaxK = 65536;
constexpr int kMaxFeatures = 1 << 20;
constexpr int kMaxSplit = 16;

size_t partial_bytes(int rows) {
  const int cols = rows >= 128 ? 256 : 2 * ((rows + 15) / 16 * 16);
  return static_cast<size_t>(kMaxGrid) * 2 * kTileM * cols * 4;
}

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

// bn, kblocks and the operand types are set: the ring, tensor memory and
// instruction descriptor that go with them, and the launch.
template <bool FP8, bool GATED, int SRC>
mhc_status launch_gemm(GemmParams& p, const CUtensorMap& w, const CUtensorMap& x, int grid, cudaStream_t stream) {
  constexpr int acc = GATED ? 2 : 1;
  const int fixed = 1024 + (SRC == kDense ? 0 : 8 * (p.experts + 1));
  const int stage = acc * kATile + p.bn * 128 + (FP8 ? (acc + 1) * 512 : 0);
  const int static_smem = 1024;  // the barriers
  p.stages = (kGemmSmem - static_smem - fixed) / stage;
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const int smem = fixed + p.stages * stage;
  auto cols = [&](int nbuf) { return nbuf * acc * p.bn + (FP8 ? p.stages * (acc + 1) * 4 : 0); };
  p.nbuf = cols(2) <= 512 ? 2 : 1;
  p.tmem_cols = 32;
  while (p.tmem_cols < cols(p.nbuf)) p.tmem_cols *= 2;
  if (p.stages < 2 || p.tmem_cols > 512) return MHC_ERR_UNSUPPORTED_SHAPE;
  p.idesc = (static_cast<unsigned>(p.bn >> 3) << 17) | (static_cast<unsigned>(kTileM >> 4) << 24) |
            (FP8 ? (1u << 23) : (1u << 4) | (1u << 7) | (1u << 10));
  p.budget_ns = g_budget_ns;
  p.extra_tx = static_cast<unsigned>(g_extra_tx) * 16;
  auto kern = gemm_kernel<FP8, GATED, SRC>;
  static std::atomic<int> configured[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MHC_ERR_CUDA;
  if (configured[dev].load(std::memory_order_acquire) == 0) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kGemmSmem - static_smem) !=
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
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGemmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
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

}  // namespace

extern "C" {

size_t mhc_linear_workspace_bytes(int rows) {
  if (rows < 1 || rows > kMaxTokens) return 0;
  return kGemmHeader + partial_bytes(rows);
}

mhc_status mhc_linear(const void* x, const uint8_t* x_scale, int64_t x_stride, const void* weight,
                      const uint8_t* weight_scale, const float* bias, mhc_activation activation,
                      const mhc_bf16* residual, int64_t residual_stride, void* out, int out_fp32, int64_t out_stride,
                      int rows, int in_features, int out_features, void* workspace, size_t ws_bytes,
                      mhc_stream stream) {
  const bool fp8 = weight_scale != nullptr;
  const bool gated = activation == MHC_ACT_SWIGLU;
  if (rows < 1 || rows > kMaxTokens || in_features < 1 || in_features > kMaxK || out_features < 1 ||
      out_features > kMaxFeatures || in_features % (fp8 ? 32 : 8) != 0 || (fp8 && gated && out_features % kTileM != 0))
    return MHC_ERR_UNSUPPORTED_SHAPE;
  if (activation < MHC_ACT_NONE || activation > MHC_ACT_SWIGLU) return MHC_ERR_INVALID_ARG;
  if (!x || !weight || !out || (x_scale != nullptr) != fp8) return MHC_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(x_scale, 16) || !aligned(weight_scale, 16) ||
      !aligned(bias, 4) || !aligned(residual, 2) || !aligned(out, out_fp32 ? 4 : 2))
    return MHC_ERR_INVALID_ARG;
  const int64_t row_bytes = fp8 ? 1 : 2;
  if (x_stride < in_features || (x_stride * row_bytes) % 16 != 0 || out_stride < out_features ||
      (residual && residual_stride < out_features))
    return MHC_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < mhc_linear_workspace_bytes(rows)) return MHC_ERR_WORKSPACE;
  GemmParams p{};
  p.rows = rows;
  p.n = out_features;
  p.kblocks = fp8 ? (in_features + 127) / 128 : (in_features + 63) / 64;
  p.m_tiles = (out_features + kTileM - 1) / kTileM;
  p.max_split = kMaxSplit;
  p.x_scale = x_scale;
  p.w_scale = weight_scale;
  p.bias = bias;
  p.residual = reinterpret_cast<const __nv_bfloat16*>(residual);
  p.res_stride = residual_stride;
  p.out = out;
  p.out_stride = out_stride;
  p.out_fp32 = out_fp32 != 0;
  p.act = activation;
  p.status = static_cast<unsigned*>(workspace);
  p.counters = reinterpret_cast<unsigned*>(static_cast<char*>(workspace) + kGemmCounters);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + kGemmHeader);
  // Token columns of a tile: all tokens if one tile can hold them, else tiles of
  // 128 (MXFP8, whose scale tiles are 128 rows, and gated products, which hold
  // two accumulators) or of nearly equal parts of up to 256.
  const int cap = fp8 || gated ? 128 : 256;
  if (rows <= cap) {
    p.bn = round16(rows);
  } else if (fp8) {
    p.bn = 128;
  } else {
    const int tt = (rows + cap - 1) / cap;
    p.bn = round16((rows + tt - 1) / tt);
  }
  const int tiles = p.m_tiles * ((rows + p.bn - 1) / p.bn);
  int grid = gemm_grid();
  if (tiles < grid) {  // as many CTAs as the schedule makes shares
    int64_t most = static_cast<int64_t>(tiles) * kMaxSplit;
    const int64_t pairs = static_cast<int64_t>(tiles) * p.kblocks / 2;
    if (pairs < most) most = pairs > tiles ? pairs : tiles;
    if (most < grid) grid = static_cast<int>(most);
  }
  CUtensorMap mw, mx;
  const uint64_t wrows = static_cast<uint64_t>(out_features) * (gated ? 2 : 1);
  if (!make_map2(&mw, weight, fp8, in_features, wrows, static_cast<uint64_t>(in_features) * row_bytes, kTileM) ||
      !make_map2(&mx, x, fp8, in_features, rows, static_cast<uint64_t>(x_stride) * row_bytes, p.bn))
    return MHC_ERR_CUDA;
  if (fp8) return gated ? launch_gemm<true, true, kDense>(p, mw, mx, grid, stream)
                        : launch_gemm<true, false, kDense>(p, mw, mx, grid, stream);
  return gated ? launch_gemm<false, true, kDense>(p, mw, mx, grid, stream)
               : launch_gemm<false, false, kDense>(p, mw, mx, grid, stream);
}

size_t mhc_moe_experts_workspace_bytes(int rows, int num_permuted, int intermediate) {
  if (rows < 1 || rows > kMaxTokens || num_permuted < 1 || intermediate < 1) return 0;
  return kGemmHeader + partial_bytes(rows) + static_cast<size_t>(num_permuted) * intermediate * 2;
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
  __nv_bfloat16* inner = reinterpret_cast<__nv_bfloat16*>(ws + kGemmHeader + partial_bytes(rows));
  GemmParams p{};
  p.rows = num_permuted;
  p.x_rows = rows;
  p.experts = experts;
  p.max_split = kMaxSplit;
  p.offsets = expert_offsets;
  p.prow = permuted_rows;
  p.status = reinterpret_cast<unsigned*>(ws);
  p.counters = reinterpret_cast<unsigned*>(ws + kGemmCounters);
  p.partials = reinterpret_cast<float*>(ws + kGemmHeader);
  // Token columns of a tile: about twice the mean number of an expert's rows
  // (its tokens then mostly fit one tile, which reads the weights once), never
  // more than there are rows.
  const int mean = (num_permuted + experts - 1) / experts;
  int bn = mean <= 4 ? 16 : mean <= 16 ? 32 : mean <= 48 ? 64 : 128;
  if (bn > round16(rows)) bn = round16(rows);
  p.bn = bn;
  const int grid = gemm_grid();
  CUtensorMap mw, mx;
  // first product: gate and up rows of an expert's w13, token rows gathered
  p.n = intermediate;
  p.kblocks = (hidden + 63) / 64;
  p.m_tiles = (intermediate + kTileM - 1) / kTileM;
  p.out = inner;
  p.out_stride = intermediate;
  p.act = MHC_ACT_SWIGLU;
  if (!make_map2(&mw, w13, false, hidden, static_cast<uint64_t>(experts) * 2 * intermediate,
                 static_cast<uint64_t>(hidden) * 2, kTileM) ||
      !make_map2(&mx, x, false, hidden, rows, static_cast<uint64_t>(x_stride) * 2, 1))
    return MHC_ERR_CUDA;
  mhc_status st = launch_gemm<false, true, kGather>(p, mw, mx, grid, stream);
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
      !make_map2(&mx, inner, false, intermediate, num_permuted, static_cast<uint64_t>(intermediate) * 2, p.bn))
    return MHC_ERR_CUDA;
  return launch_gemm<false, false, kGrouped>(p, mw, mx, grid, stream);
}

}  // extern "C"
