// skg_gemm_mx on CTA pairs: persistent clusters of two CTAs, 256 x 256 tiles of C
// with one M = 256 MMA (tcgen05 cta_group::2). Each CTA loads its 128 rows of A
// and half of B's 256 rows per stage, with its rows' scales and all of B's; the
// leader issues the scale copies (which run in both CTAs) and the MMAs.
//
// TMEM holds two accumulators and two buffers of scale columns, which together
// need more than its 512 columns (2 x 256, and 24 to 96 for the scales), so the
// accumulators overlap: number 1 starts inside number 0's last columns. The
// epilogue takes half of a tile, the shared columns in it, to registers first, and
// with them out the next tile's MMAs run while it writes the tile.
//
// What it measured on GB300 (each step at 8192 x 28672 x 8192 in mxfp4): the first
// form 903 us; one elected thread issuing (the compiler had wrapped every tcgen05
// instruction behind `lane == 0` in a loop over the lanes, 1540 cycles per stage of
// nvfp4 against 650) 560 us; TMA stores and a hand-over of the accumulator without a
// release at cluster scope (1200 cycles a tile) 517 us; 490 us now in short runs, 560
// in long ones: 6.9 to 7.9 PFLOP/s, 3.6 to 4.1 times the card's bf16 burst rate. In
// mxfp8 4096 x 8192 x 8192 takes 151 us (3.6 PFLOP/s). The tensor pipe is busy 85 % of
// the time in 8 bits, and the clock falls to 1.65 GHz under that load (with the loads
// left out of a copy of the kernel, at the same cycles per stage, it stays at 1.9 GHz):
// power bounds these. In 4 bits the pipe is busy 76 % of the time and what the rest
// waits for has not been shown; the MMAs are those of K = 64 (the K = 96 ones of 4 bits
// have not been tried). With beta, or rows of C off 16-byte boundaries, C does not go
// through TMA and the epilogue takes longer than the MMAs: 4096 x 8192 x 8192 with
// beta = 1 279 us in mxfp8 and 273 in nvfp4 (79 without beta), 358 and 345 into fp32;
// n = 8191 without beta 178 and 142.
#include "skg_mx_gemm.cuh"

namespace skg {
namespace {

template <int FMT>
struct PairCfg : MxStage<FMT> {
  using MxStage<FMT>::CHUNKS;
  using MxStage<FMT>::SF_BYTES;
  static constexpr int SFA_OFF = 2 * kMxOperand;
  static constexpr int SFB_OFF = SFA_OFF + SF_BYTES;
  static constexpr int LOAD_BYTES = 2 * kMxOperand + 3 * SF_BYTES;  // per CTA
  static constexpr int STAGE_BYTES = (LOAD_BYTES + 1023) / 1024 * 1024;
  static constexpr int STAGING = 4 * 8192;  // per epilogue warp: two boxes of 32 rows x 128 bytes
  static constexpr int FIT = ((int)kSmemLimit - 1024 - STAGING - 512) / STAGE_BYTES;
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr uint32_t SMEM = 1024 + STAGES * STAGE_BYTES + STAGING + 512;
  static constexpr int SF_COLS = 3 * CHUNKS * 4;       // one buffer of scale columns
  static constexpr int SF_BASE = 512 - 2 * SF_COLS;
  static constexpr int ACC1 = SF_BASE - 256;           // first column of accumulator 1
  static_assert(256 - ACC1 <= 128, "the overlap lies in half of a tile");
  static_assert(STAGES >= 4 && SMEM <= kSmemLimit, "shared memory");
  static_assert(sizeof(MxAux) <= 512, "aux size");
};

// 32 columns of a warp's 32 rows of the accumulator (v: this lane's row) to C,
// for any alignment and beta.
template <typename T>
__device__ __forceinline__ void pair_write_chunk(const MxParams& p, uint8_t* staging, int lane,
                                                 const uint32_t (&v)[32], int row0, int col0,
                                                 float alpha) {
  float* st = reinterpret_cast<float*>(staging);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    *reinterpret_cast<uint4*>(st + lane * 36 + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  __syncwarp();
  for (int j = 0; j < 8; ++j) {
    const int r = j * 4 + (lane >> 3), c = (lane & 7) * 4;
    if (row0 + r < p.m && col0 + c < p.n)
      mx_write4<T>(p, row0 + r, col0 + c, *reinterpret_cast<const float4*>(st + r * 36 + c), alpha);
  }
}

// 64 columns: scaled, rounded and stored by TMA (beta = 0, rows of C on 16-byte
// boundaries) from boxes of 32 rows x 128 bytes in the 128-byte swizzle, two
// boxes per warp in turn; the engine clips what is past m and the last whole 16
// bytes of n, and the columns behind those are stored one by one.
template <typename T>
__device__ __forceinline__ void pair_store_half(const MxParams& p, const CUtensorMap* tmC,
                                                uint8_t* staging, uint32_t& box, int lane,
                                                const uint32_t (&v)[2][32], int row0, int col0,
                                                float alpha) {
  if (!p.c_tma) {
    pair_write_chunk<T>(p, staging, lane, v[0], row0, col0, alpha);
    if (col0 + 32 < p.n) pair_write_chunk<T>(p, staging, lane, v[1], row0, col0 + 32, alpha);
    return;
  }
  constexpr int PER = 16 / (int)sizeof(T);        // elements of a 16-byte piece
  constexpr int BOXES = sizeof(T) == 4 ? 2 : 1;   // 128-byte boxes of 64 columns
#pragma unroll
  for (int b = 0; b < BOXES; ++b) {
    uint8_t* st = staging + (box & 1) * 4096;
    ++box;
    if (lane == 0) bulk_wait_read<1>();  // the box's last store has read it
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      union {
        T e[PER];
        uint4 q;
      } u;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = b * (64 / BOXES) + j * PER + i;
        u.e[i] = mx_from_f32<T>(alpha * __uint_as_float(v[c >> 5][c & 31]));
      }
      *reinterpret_cast<uint4*>(st + lane * 128 + ((j ^ (lane & 7)) << 4)) = u.q;
    }
    fence_proxy_async_smem();
    __syncwarp();
    const int col = col0 + b * 32, whole = p.n & ~(PER - 1);
    if (lane == 0) {
      if (col < whole) tma_store_2d(tmC, st, col, row0);
      bulk_commit();
    }
    if (whole < p.n && col + 8 * PER > whole)
      store_rest<T>(p.c, p.ldc, p.m, p.n, st, lane, col, row0);
  }
}

// Tile t in an order that keeps the tiles in flight close together: bands of
// eight rows of tiles, column by column within a band (2048 rows of A stay in L2
// while B passes).
__device__ __forceinline__ void pair_tile(const MxParams& p, int t, int& tm, int& tn) {
  constexpr int kBand = 8;
  const int band = t / (kBand * p.tiles_n);
  const int rows = min(kBand, p.tiles_m - band * kBand);
  const int i = t - band * kBand * p.tiles_n;
  tn = i / rows;
  tm = band * kBand + i % rows;
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kMxThreads, 1)
mx_gemm_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA,
                    const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ CUtensorMap tmC, const MxParams p) {
  using C = PairCfg<FMT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* staging = ring + C::STAGES * C::STAGE_BYTES;
  MxAux* aux = reinterpret_cast<MxAux*>(staging + C::STAGING);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const int tiles = p.tiles_m * p.tiles_n;
  const int first = (int)blockIdx.x >> 1, stride = (int)gridDim.x >> 1;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmSA);
    prefetch_tmap(&tmSB);
    prefetch_tmap(&tmC);
    aux->abort_flag = 0;
    aux->limit = p.limit;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&aux->full[i], 1);
      mbar_init(&aux->empty[i], 1);
    }
    mbar_init(&aux->tfull[0], 1);
    mbar_init(&aux->tfull[1], 1);
    mbar_init(&aux->tempty, 8);  // the epilogue warps of both CTAs
    mbar_init(&aux->drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&aux->tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = aux->tmem_slot;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();

  uint32_t issued = 0;  // the loading thread: stages loaded
  if (warp == 0) {
    if (elect_one()) {
      int st = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += stride) {
        int tm, tn;
        pair_tile(p, t, tm, tn);
        const int rt = 2 * tm + rank;
        for (int kb = 0; kb < p.ksteps; ++kb) {
          if (issued >= p.stages) {
            ok = false;
            break;
          }
          if (!mx_wait(&aux->empty[st], phase ^ 1u, aux)) {
            mx_fail(p, aux);
            ok = false;
            break;
          }
          uint8_t* s = ring + st * C::STAGE_BYTES;
          const uint32_t bar = cluster_addr(&aux->full[st], 0);
          if (rank == 0) mbar_arrive_expect_tx(&aux->full[st], 2 * C::LOAD_BYTES);
          tma_load_2d_pair(s, &tmA, bar, kb * kMxRowBytes, rt * kMxTile);
          tma_load_2d_pair(s + kMxOperand, &tmB, bar, kb * kMxRowBytes, (2 * tn + rank) * kMxTile);
          tma_load_2d_pair(s + C::SFA_OFF, &tmSA, bar, 0, rt * p.groups + kb * C::CHUNKS);
          tma_load_2d_pair(s + C::SFB_OFF, &tmSB, bar, 0, 2 * tn * p.groups + kb * C::CHUNKS);
          tma_load_2d_pair(s + C::SFB_OFF + C::SF_BYTES, &tmSB, bar, 0,
                           (2 * tn + 1) * p.groups + kb * C::CHUNKS);
          ++issued;
          if (++st == C::STAGES) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one() && rank == 0) {
      int st = 0, n = 0;
      uint32_t phase = 0, it = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += stride, ++n) {
        // The last tile's shared columns are out of its accumulator (and all of
        // the one before's, whose columns this tile's accumulator reuses).
        if (n > 0 && !mx_wait(&aux->tempty, (uint32_t)(n - 1) & 1u, aux)) {
          mx_fail(p, aux);
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + ((n & 1) ? C::ACC1 : 0);
        for (int kb = 0; kb < p.ksteps; ++kb, ++it) {
          if (!mx_wait(&aux->full[st], phase, aux)) {
            mx_fail(p, aux);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sf = tmem + C::SF_BASE + (it & 1) * C::SF_COLS;
          mx_stage_mmas<FMT, true, 2, kMxOperand>(
              d, sf, sf + C::CHUNKS * 4, smem_u32(ring + st * C::STAGE_BYTES), C::SFA_OFF,
              C::SFB_OFF, p.k - kb * C::STEP, kb == 0);
          umma_commit_pair(&aux->empty[st]);
          if (++st == C::STAGES) {
            st = 0;
            phase ^= 1u;
          }
        }
        if (ok) umma_commit_pair(&aux->tfull[n & 1]);
      }
      if (it > 0) {
        umma_commit_pair(&aux->drain);
        mx_wait(&aux->drain, 0, aux, true);
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    uint8_t* mine = staging + q * 8192;
    uint32_t box = 0;
    float alpha = p.alpha;
    if (p.ga) alpha *= *p.ga;
    if (p.gb) alpha *= *p.gb;
    const uint32_t release = cluster_addr(&aux->tempty, 0);
    int n = 0;
    for (int t = first; t < tiles; t += stride, ++n) {
      int tm, tn;
      pair_tile(p, t, tm, tn);
      const int row0 = (2 * tm + rank) * kMxTile + q * 32, col0 = tn * 256;
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + ((n & 1) ? C::ACC1 : 0);
      // Accumulator 0 shares its last columns, accumulator 1 its first.
      const int start = (n & 1) ? 0 : 192, step = (n & 1) ? 64 : -64;
      const bool got = mx_wait(&aux->tfull[n & 1], (uint32_t)(n >> 1) & 1u, aux);
      if (!got) mx_fail(p, aux);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      uint32_t v[2][2][32];  // two quarters of the tile
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) tmem_ld32_async(acc + start + h * step + i * 32, v[h][i]);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) tmem_ld_wait32(v[h][i]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(release);
      if (row0 >= p.m) continue;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int c = start + s * step;
        if (s >= 2) {
          tmem_ld_wait32(v[s & 1][0]);
          tmem_ld_wait32(v[s & 1][1]);
        }
        if (col0 + c < p.n)
          pair_store_half<T>(p, &tmC, mine, box, lane, v[s & 1], row0, col0 + c, alpha);
        if (s < 2)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tmem_ld32_async(acc + start + (s + 2) * step + i * 32, v[s & 1][i]);
      }
    }
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // Copies that no MMA waited for land before the pair parts (the leader's
  // barriers count both CTAs' bytes), and the leader's last commit has reached the
  // other CTA's barrier; then no CTA leaves while the other may still signal its
  // barriers (the last hand-over of an accumulator is a remote arrival, which the
  // cluster barrier's release waits for). After a wait that ran out the other CTA may
  // have loaded stages that the leader did not come to, whose barriers no longer
  // complete: it gives those copies a millisecond, some thousand times what one takes.
  if (warp == 1 && rank == 1 && first < tiles && elect_one()) mx_wait(&aux->drain, 0, aux, true);
  if (warp == 0 && rank == 0 && issued > 0 && mx_aborted(aux))
    for (uint32_t i = issued > C::STAGES ? issued - C::STAGES : 0; i < issued; ++i)
      mx_wait(&aux->full[i % C::STAGES], (i / C::STAGES) & 1u, aux, true);
  if (warp == 0 && rank == 1 && issued > 0 && mx_aborted(aux))
    for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < 1000000ull;) __nanosleep(1000);
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(&p.report->launches, 1u);
}

template <int FMT, typename T>
cudaError_t launch_pair(const CUtensorMap (&t)[5], const MxParams& p, int clusters,
                        cudaStream_t stream) {
  using C = PairCfg<FMT>;
  static std::atomic<uint64_t> done_mask{0};
  const cudaError_t e = opt_in_smem((const void*)mx_gemm_pair_kernel<FMT, T>, done_mask, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(mx_gemm_pair_kernel<FMT, T>, dim3((unsigned)(2 * clusters)),
                            dim3(kMxThreads), C::SMEM, stream, 2, t[0], t[1], t[2], t[3], t[4], p);
}

}  // namespace

template <int FMT>
cudaError_t launch_mx_pair(const CUtensorMap (&t)[5], const MxParams& p, int out, int clusters,
                           cudaStream_t stream) {
  if (out == SKG_OUT_F32) return launch_pair<FMT, float>(t, p, clusters, stream);
  if (out == SKG_OUT_F16) return launch_pair<FMT, __half>(t, p, clusters, stream);
  return launch_pair<FMT, __nv_bfloat16>(t, p, clusters, stream);
}

template cudaError_t launch_mx_pair<SKG_MXFP8>(const CUtensorMap (&)[5], const MxParams&, int, int,
                                               cudaStream_t);
template cudaError_t launch_mx_pair<SKG_MXFP4>(const CUtensorMap (&)[5], const MxParams&, int, int,
                                               cudaStream_t);
template cudaError_t launch_mx_pair<SKG_NVFP4>(const CUtensorMap (&)[5], const MxParams&, int, int,
                                               cudaStream_t);

int mx_pair_clusters_resident() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int have = cached[dev].load(std::memory_order_acquire);
  if (have != 0) return have > 0 ? have : 0;
  using C = PairCfg<SKG_NVFP4>;  // the kernels' resources differ by the formats' stages alone
  auto kernel = mx_gemm_pair_kernel<SKG_NVFP4, __nv_bfloat16>;
  int n = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM) ==
      cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 256);
    cfg.blockDim = dim3(kMxThreads);
    cfg.dynamicSmemBytes = C::SMEM;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  cached[dev].store(n > 0 ? n : -1, std::memory_order_release);
  return n;
}

}  // namespace skg
