// The product of many token rows: two CTAs of a cluster (a pair of SMs) on one
// tile. Included by mhc_gemm.cu, whose parameters, schedule and epilogue it uses.
//
// With one CTA per tile of 128 x 256 every K block brings 48 KB to an SM for 512
// cycles of products; the SMs together then ask L2 for more than it gives (about
// 14.5 TB/s, 52 bytes a cycle and SM, measured with every tile shape tried). A pair
// computes 256 weight rows x up to 256 token rows: each CTA loads its 128 weight
// rows (gated: 128 gate and 128 up rows) and half of the token rows, 32 KB per 512
// cycles (gated: 48 KB per 1024), and the tensor cores of both SMs read the other
// half from the neighbour's shared memory (tcgen05 cta_group::2). The accumulator
// of a CTA's weight rows lies in its own tensor memory and its own warps finish it.
//
//   warp 0      each CTA: copies by tensor map, counted on the first CTA's barrier
//   warp 1      first CTA: issues the products for both
//   warps 2-9   each CTA: epilogue of its 128 weight rows, two warps to a quarter of them
//               (a gated tile of 256 columns fills tensor memory, so nothing hides it)
// The experts' first product reads its token rows from a copy in permuted order
// (permute_rows_kernel): the tensor-map gather moves four rows per 65 cycles, a quarter
// of what a tile of 128 columns needs (2.16 ms against 0.82 for the product of 16384
// rows by 32 experts' 4096 x 7168), and 16-byte asynchronous copies by four more warps
// kept too few bytes in flight (1.67 ms). The copy takes 0.05 ms.
#pragma once

namespace mhc {

constexpr int kPairTileM = 256;
constexpr int kPairWarps = 8;  // of the epilogue
constexpr int kPairThreads = 64 + 32 * kPairWarps;

__device__ __forceinline__ void tmem_alloc2(unsigned* slot, unsigned cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_dealloc2(unsigned addr, unsigned cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
// As tma_load_2d, counted on a barrier of the pair (a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(unsigned dst, const void* map, int x, int y, unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// D[256 x N] (+)= A[256 x 16] B[N x 16]^T over the pair: each CTA holds 128 rows of A
// and N / 2 rows of B at the same shared-memory addresses.
__device__ __forceinline__ void mma_bf16_pair(unsigned d, unsigned a, unsigned b, unsigned idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "n"(kDescHi)
      : "memory");
}
// The same with E4M3 operands and E8M0 scales (K 32): each CTA's tensor memory holds
// the scales of its 128 rows of A at sa and of all N rows of B at sb.
__device__ __forceinline__ void mma_mxf8_pair(unsigned d, unsigned a, unsigned b, unsigned idesc, unsigned sa,
                                              unsigned sb, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, [%5], [%6], p;\n\t}" ::"r"(
          d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate ? 1u : 0u), "r"(sa), "r"(sb), "n"(kDescHi)
      : "memory");
}
// tmem_copy_scales in both CTAs, each from its own shared memory at the same address.
__device__ __forceinline__ void tmem_copy_scales_pair(unsigned addr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(addr), "l"(desc) : "memory");
}
// Arrive on the barrier at this address in both CTAs once the products are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<unsigned short>(3))
      : "memory");
}
// Arrive on a barrier of the cluster, releasing what this thread (and, ordered by a
// warp barrier, its warp) wrote before.
__device__ __forceinline__ void mbar_arrive_cluster(unsigned addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
// x [x_rows, k] rows in permuted order: out[q] = x[permuted_rows[q]] for the places
// that an expert owns. A warp copies 4 KB of a row at a time.
__global__ void __launch_bounds__(256) permute_rows_kernel(const GemmParams p, __nv_bfloat16* out) {
  griddep_wait();
  griddep_launch_dependents();
  bool bad = false;
  for (int e = threadIdx.x; e < p.experts; e += 256) {
    const int lo = p.offsets[e], hi = p.offsets[e + 1];
    bad |= lo < 0 || hi < lo || hi > p.rows;
  }
  if (__syncthreads_or(bad)) return;  // nothing is computed; the products record it
  const int first = p.offsets[0], used = p.offsets[p.experts];
  const int lane = threadIdx.x & 31;
  const int units = p.k / 8, pieces = (units + 255) / 256;  // 16-byte units of a row, 256 a piece
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8, total = static_cast<int64_t>(used - first) * pieces;
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); w < total; w += warps) {
    const int q = first + static_cast<int>(w / pieces), u0 = static_cast<int>(w % pieces) * 256 + lane;
    int r = p.prow[q];
    if (r < 0 || r >= p.x_rows) {
      record_error(p.status, MHC_ERR_DEVICE_INDEX);
      r = 0;
    }
    const uint4* src = reinterpret_cast<const uint4*>(p.x + r * p.x_stride);
    uint4* dst = reinterpret_cast<uint4*>(out + static_cast<int64_t>(q) * p.k);
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (u0 + 32 * i < units) v[i] = src[u0 + 32 * i];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (u0 + 32 * i < units) dst[u0 + 32 * i] = v[i];
  }
}

// A pair's tile of a wave. The experts' tiles come in falling size and the waves run
// forth and back, so that the pairs' sums of sizes are nearly equal: of 16384 rows by 32
// uneven experts the longest has 8% more than the mean, 22% in the experts' own order.
__device__ __forceinline__ int pair_tile(int wave, int pair, int pairs) {
  return wave * pairs + (wave & 1 ? pairs - 1 - pair : pair);
}

template <bool FP8, bool GATED, int SRC>
__global__ void __cluster_dims__(2) __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_ws,
                const __grid_constant__ CUtensorMap tm_xs) {
  static_assert(!FP8 || (!GATED && SRC == kDense), "MXFP8: plain dense products only");
  extern __shared__ unsigned char raw[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2];
  __shared__ unsigned tmem_slot;
  constexpr int kAcc = GATED ? 2 : 1;
  constexpr int kElems = FP8 ? 128 : 64;             // K elements of a stage's 128-byte rows
  constexpr int kScales = FP8 ? (1 + 2) * 512 : 0;   // a stage's scale tiles: 128 weight rows, 256 token rows
  constexpr int kScaleCols = FP8 ? (1 + 2) * 4 : 0;  // and their columns of tensor memory
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);  // uniform
  const int rank = blockIdx.x & 1;
  const int x_bytes = p.bn / 2 * 128;  // bn is a multiple of 32: whole 8-row swizzle groups
  const unsigned smem0 = (smem_u32(raw) + 1023u) & ~1023u;
  const unsigned x0 = smem0 + p.stages * (kAcc * kATile);
  const unsigned sf0 = x0 + p.stages * x_bytes;
  int* first = nullptr;
  int* off = nullptr;
  int* order = nullptr;
  if constexpr (SRC != kDense) {
    first = reinterpret_cast<int*>(raw + (sf0 - smem_u32(raw)));
    off = first + p.experts + 1;
    order = off + p.experts + 1;
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
      mbar_init(&acc_empty[i], 2 * kPairWarps);  // both CTAs' epilogue warps
    }
  }
  if (warp == 1) {
    tmem_alloc2(&tmem_slot, 512);
    tmem_relinquish2();
  }
  int tiles;
  if constexpr (SRC == kDense) {
    tiles = p.m_tiles * ((p.rows + p.bn - 1) / p.bn);
  } else {
    // As in gemm_kernel: the kernel before waited for the offsets before it let this
    // one start.
    if (warp == 0) expert_tiles(p, first, off, order, lane);
  }
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  cluster_arrive();
  if constexpr (SRC != kDense) tiles = first[p.experts];
  const unsigned tmem = tmem_slot;
  cluster_wait();  // the other CTA's barriers are set

  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int acc_cols = kAcc * p.bn;

  if (warp == 0) {
    // ------------------------------------------------ copies
    const unsigned bar0 = cluster_address(smem_u32(&full[0]), 0);
    griddep_wait();
    griddep_launch_dependents();
    int i = 0, s = 0;
    unsigned ph = 1;
    bool ok = true;
    for (int wave = 0, tile = pair; ok && tile < tiles; tile = pair_tile(++wave, pair, pairs)) {
      const TileAt t = tile_even<SRC>(p, first, off, order, tile);
      const int half = round32(t.ntok) / 2;
      const int wrow = (SRC == kDense ? 0 : t.expert * (kAcc * p.n)) + t.m * kPairTileM + rank * kTileM;
      const int xrow = t.tok0 + rank * half;
      const unsigned bytes = kAcc * kATile + (SRC == kDense ? x_bytes : half * 128) + kScales;
      for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
        if (!(ok = __all_sync(kFull, wait_for_cluster(&empty[s], ph, p)))) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * bytes + p.extra_tx);
          const unsigned bar = bar0 + s * 8, dst = smem0 + s * (kAcc * kATile), xdst = x0 + s * x_bytes;
          tma_load_2d_pair(dst, &tm_w, kb * kElems, wrow, bar);
          if constexpr (GATED) tma_load_2d_pair(dst + kATile, &tm_w, kb * kElems, wrow + p.n, bar);
          if constexpr (SRC == kDense) tma_load_2d_pair(xdst, &tm_x, kb * kElems, xrow, bar);
          if constexpr (FP8) {  // scale tiles are 128 rows; of the token rows each CTA needs all
            const unsigned sf = sf0 + s * kScales;
            tma_load_2d_pair(sf, &tm_ws, 0, (t.m * 2 + rank) * p.kblocks + kb, bar);
            for (int r = 0; r < 2; ++r)
              tma_load_2d_pair(sf + 512 + r * 512, &tm_xs, 0, (t.tok0 / 128 + r) * p.kblocks + kb, bar);
          }
          if constexpr (SRC == kGrouped)
            for (int r = 0; r < half; r += 16) tma_load_2d_pair(xdst + r * 128, &tm_x, kb * kElems, xrow + r, bar);
        }
        __syncwarp();
        if (++s == p.stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // Both CTAs' copies are counted on the first one's barriers, and the pair ends together.
    // Not counted are stages that the second CTA requests after the first has given up: the
    // products then wait for a stage that the first did not request, for at least
    // kMinBudgetNs from when the second's last request became possible.
    if (!ok && rank == 0) drain_ring(full, p.stages, i - p.stages, i, p);
  } else if (warp == 1) {
    // ------------------------------------------------ products
    griddep_wait();  // as in gemm_kernel, before the first bounded wait
    if (rank == 0) {
      const unsigned a_lo = desc_lo(smem0), b_lo = desc_lo(x0);
      int i = 0, s = 0, buf = 0;
      unsigned ph = 0, aph = 1;
      bool ok = true;
      for (int wave = 0, tile = pair; ok && tile < tiles; tile = pair_tile(++wave, pair, pairs)) {
        const TileAt t = tile_even<SRC>(p, first, off, order, tile);
        const unsigned idesc = p.idesc | (static_cast<unsigned>(round32(t.ntok) >> 3) << 17);
        if (!(ok = __all_sync(kFull, wait_for_cluster(&acc_empty[buf], aph, p)))) break;
        tcgen05_fence_after();
        const unsigned d = tmem + buf * acc_cols;
        for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
          if (!(ok = __all_sync(kFull, wait_for_cluster(&full[s], ph, p)))) break;
          tcgen05_fence_after();
          if (elect_one()) {
            const unsigned a = a_lo + s * (kAcc * kATile / 16), b = b_lo + s * (x_bytes / 16);
            const unsigned sf = tmem + p.nbuf * acc_cols + s * kScaleCols;
            if constexpr (FP8) {
#pragma unroll
              for (int q = 0; q < 3; ++q)
                tmem_copy_scales_pair(sf + 4 * q, desc_scales(sf0 + s * kScales + 512 * q));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int q = 0; q < kAcc; ++q)
                if constexpr (FP8)
                  mma_mxf8_pair(d, a + 2 * k, b + 2 * k, idesc | (k << 4) | (k << 29), sf, sf + 4, k > 0 || kb > 0);
                else
                  mma_bf16_pair(d + q * p.bn, a + q * (kATile / 16) + 2 * k, b + 2 * k, idesc, k > 0 || kb > 0);
            mma_commit_pair(&empty[s]);
            if (kb == p.kblocks - 1) mma_commit_pair(&acc_full[buf]);
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
    }
  } else {
    // ------------------------------------------------ epilogue
    griddep_wait();
    const int q = warp & 3, part = (warp - 2) >> 2;
    int buf = 0;
    unsigned ph = 0;
    for (int wave = 0, tile = pair; tile < tiles; tile = pair_tile(++wave, pair, pairs)) {
      const TileAt t = tile_even<SRC>(p, first, off, order, tile);
      const int f = t.m * kPairTileM + rank * kTileM + q * 32 + lane;
      float bg = 0.f, bu = 0.f;
      if (p.bias != nullptr && f < p.n) {
        bg = p.bias[f];
        if constexpr (GATED) bu = p.bias[p.n + f];
      }
      if (!epilogue_all<32 * kPairWarps>(wait_for_cluster(&acc_full[buf], ph, p))) break;
      tcgen05_fence_after();
      const unsigned src = tmem + buf * acc_cols + (static_cast<unsigned>(q * 32) << 16);
      for (int c = 16 * part; c < t.ntok; c += 32) {
        float v[16], u[16];
        read_sums<GATED>(src + c, p.bn, v, u);
        store_columns<GATED, 16>(p, v, u, bg, bu, t.tok0 + c, f, t.ntok - c);
      }
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_address(smem_u32(&acc_empty[buf]), 0));
      if (++buf == p.nbuf) {
        buf = 0;
        ph ^= 1;
      }
    }
  }
  tcgen05_fence_before();
  __syncthreads();
  cluster_arrive();
  cluster_wait();  // the pair's products are done and nobody will arrive here any more
  if (warp == 1) {
    tcgen05_fence_after();
    tmem_dealloc2(tmem, 512);
  }
}

}  // namespace mhc
