// skg_gemm_mx: C = alpha * A B^T + beta * C of two microscaled matrices (A m x k,
// B n x k, codes and block scales as skgemm.h lays them out), fp32 accumulation,
// on the block-scaled tensor-core instructions of sm_103a.
//
//   C[i][j] = sum over blocks b of sA[i][b] sB[j][b] (sum over l in b of a[i][l] b[j][l]),
//
// the scales applied by the MMA. A CTA runs one 128 x 128 tile of C over a range of
// k: warp 0 fills a ring of stages by TMA (128 bytes of k for each of 128 rows of
// A and of B, and their scale tiles), warp 1 copies each stage's scales to TMEM
// (tcgen05.cp, in the order of the MMAs behind it) and issues four MMAs, warps 2-5
// take the accumulator to C through shared memory.
//
// When the tiles are fewer than the CTAs that fit the GPU, the S CTAs of a
// cluster share a tile, a range of k each: every one leaves its partial sums in
// its own shared memory, and after a cluster barrier each adds the rows r, r + S,
// ... of all of them in rank order through distributed shared memory. No
// workspace, no atomics, the same result every time.
//
// What bounds it: a few rows of A (decode) stream B once, so memory does (1 x 28672
// x 8192 in nvfp4, 132 MB: 22.7 us, 5.8 TB/s; in mxfp8 37.9 us, 6.4 TB/s); small
// products the fixed cost of a launch, a first load and the sum over the cluster
// (333 x 1000 x 2200 in mxfp8: 6.3 us). Larger ones run on CTA pairs
// (skg_mx_gemm_pair.cu).
//
// Every wait is bounded; when one runs out the CTA records
// SKG_ERR_PIPELINE_TIMEOUT in the report, waits for its own copies and MMAs,
// still meets the cluster's barriers, frees its TMEM and leaves.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_mx_gemm.cuh"

namespace skg {
namespace {

constexpr int kMxPitch = 132;                 // floats per row of the partial tile
constexpr int kMxSplitMax = 8;

// FEW: at most 16 rows of A. Its stages hold 16 rows of A (the MMA reads 128 from
// there: what follows in the stage, for rows of the accumulator that nothing
// reads), so that five stages of B fit where three do otherwise.
template <int FMT, bool FEW>
struct MxCfg : MxStage<FMT> {
  using MxStage<FMT>::CHUNKS;
  using MxStage<FMT>::SF_BYTES;
  static constexpr int B_OFF = FEW ? 16 * kMxRowBytes : kMxOperand;
  static constexpr int SFA_OFF = B_OFF + kMxOperand;
  static constexpr int SFB_OFF = SFA_OFF + SF_BYTES;
  static constexpr int STAGE_BYTES = SFA_OFF + 2 * SF_BYTES;
  static constexpr int STAGES = FEW ? 5 : 3;  // two CTAs share an SM
  static_assert(STAGE_BYTES % 1024 == 0 && STAGE_BYTES >= kMxOperand,
                "swizzle atoms; A's 128 rows end inside the ring");
  static constexpr uint32_t SMEM = 1024 + STAGES * STAGE_BYTES + 256;
  // TMEM: the accumulator, then two buffers of scale columns (A's, B's).
  static constexpr int SF_COLS = 2 * CHUNKS * 4;
  static constexpr int TMEM_COLS = 256;
  static_assert(kMxTile + 2 * SF_COLS <= TMEM_COLS, "TMEM columns");
  static_assert(kMxTile * kMxPitch * 4 <= STAGES * STAGE_BYTES, "the partial tile fits the ring");
};

// Rows rank, rank + S, ... of the tile: the S CTAs' partial sums in rank order.
// The loads of several rows are in flight together. Every value that is loaded is
// stored, so no load is still on its way to another CTA's shared memory when a thread
// comes to the barrier that lets that CTA leave.
template <typename T, int S>
__device__ __forceinline__ void mx_reduce_rows(const MxParams& p, const float* part, int warp,
                                               int lane, int rank, int tm, int tn, float alpha) {
  constexpr int R = 16 / S;  // rows at a time
  constexpr int WARPS = kMxThreads / 32;
  const int rows = min(kMxTile, p.m - tm * kMxTile);
  const int col = tn * kMxTile + lane * 4;
  if (col >= p.n) return;
  uint32_t base[S];
#pragma unroll
  for (int s = 0; s < S; ++s) base[s] = cluster_addr(part + lane * 4, (uint32_t)s);
#pragma unroll 1
  for (int i = warp * R; rank + i * S < rows; i += WARPS * R) {
    float4 u[R][S];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int r = rank + (i + j) * S;
      if (r < rows) {
#pragma unroll
        for (int s = 0; s < S; ++s)
          u[j][s] = ld_shared_cluster_f32x4(base[s] + (uint32_t)r * (kMxPitch * 4));
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int r = rank + (i + j) * S;
      if (r >= rows) break;
      float4 v = u[j][0];
#pragma unroll
      for (int s = 1; s < S; ++s) {
        v.x += u[j][s].x;
        v.y += u[j][s].y;
        v.z += u[j][s].z;
        v.w += u[j][s].w;
      }
      mx_write4<T>(p, tm * kMxTile + r, col, v, alpha);
    }
  }
}

template <int FMT, bool FEW, typename T>
__global__ void __launch_bounds__(kMxThreads, 2)
mx_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
               const MxParams p) {
  using C = MxCfg<FMT, FEW>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  MxAux* aux = reinterpret_cast<MxAux*>(ring + C::STAGES * C::STAGE_BYTES);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = (int)blockIdx.x / p.split;
  const int tm = tile / p.tiles_n, tn = tile % p.tiles_n;
  const int kb0 = (int)((int64_t)p.ksteps * rank / p.split);
  const int kb1 = (int)((int64_t)p.ksteps * (rank + 1) / p.split);

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmSA);
    prefetch_tmap(&tmSB);
    aux->abort_flag = 0;
    aux->limit = p.limit;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&aux->full[i], 1);
      mbar_init(&aux->empty[i], 1);
    }
    mbar_init(&aux->tfull[0], 1);
    mbar_init(&aux->drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&aux->tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = aux->tmem_slot;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();

  auto factor = [&]() {
    float a = p.alpha;
    if (p.ga) a *= *p.ga;
    if (p.gb) a *= *p.gb;
    return a;
  };
  float alpha = 0.f;
  const bool direct = !FEW && p.direct != 0;
  bool fine = true;  // epilogue threads: the accumulator is there
  int issued = 0;    // the loading thread: stages loaded
  if (warp == 0) {
    if (elect_one()) {
      const uint32_t tx = (uint32_t)p.a_rows * kMxRowBytes + kMxOperand + 2 * C::SF_BYTES;
      for (int kb = kb0; kb < kb1 && (uint32_t)issued < p.stages; ++kb, ++issued) {
        const int st = issued % C::STAGES;
        if (!mx_wait(&aux->empty[st], (uint32_t)((issued / C::STAGES) & 1) ^ 1u, aux)) {
          mx_fail(p, aux);
          break;
        }
        uint8_t* s = ring + st * C::STAGE_BYTES;
        mbar_arrive_expect_tx(&aux->full[st], tx);
        tma_load_2d(s, &tmA, &aux->full[st], kb * kMxRowBytes, tm * kMxTile);
        tma_load_2d(s + C::B_OFF, &tmB, &aux->full[st], kb * kMxRowBytes, tn * kMxTile);
        tma_load_2d(s + C::SFA_OFF, &tmSA, &aux->full[st], 0, tm * p.groups + kb * C::CHUNKS);
        tma_load_2d(s + C::SFB_OFF, &tmSB, &aux->full[st], 0, tn * p.groups + kb * C::CHUNKS);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      bool ok = true, any = false;
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int st = it % C::STAGES;
        if (!mx_wait(&aux->full[st], (uint32_t)((it / C::STAGES) & 1), aux)) {
          mx_fail(p, aux);
          ok = false;
          break;
        }
        tc_fence_after();
        // Two buffers of scale columns: the copy for this stage does not
        // touch the ones that the last stage's MMAs read.
        const uint32_t sfa = tmem + kMxTile + (it & 1) * C::SF_COLS;
        mx_stage_mmas<FMT, false, 1, C::B_OFF>(
            tmem, sfa, sfa + C::CHUNKS * 4, smem_u32(ring + st * C::STAGE_BYTES), C::SFA_OFF,
            C::SFB_OFF, p.k - kb * C::STEP, it == 0);
        any = true;
        umma_commit(&aux->empty[st]);
      }
      if (ok) umma_commit(&aux->tfull[0]);
      if (any) {
        umma_commit(&aux->drain);
        mx_wait(&aux->drain, 0, aux, true);
      }
    }
    __syncwarp();
  } else {
    // What the way out needs is read while the accumulator is on its way.
    alpha = factor();
    asm volatile("" ::"l"(p.c), "l"(p.ldc), "f"(alpha), "f"(p.beta), "r"(p.m), "r"(p.n),
                 "r"(p.c_vec));
    fine = mx_wait(&aux->tfull[0], 0, aux);
    if (!fine) mx_fail(p, aux);
    fine = epi_all(fine);
    tc_fence_after();
    const int q = warp & 3;
    const int r = q * 32 + lane;
    float* part = reinterpret_cast<float*>(ring);
    if (fine && direct && tm * kMxTile + q * 32 < p.m) {
      // A lane's row, 16 bytes at a time (see plan_and_launch).
      T* out = reinterpret_cast<T*>(p.c) + (int64_t)(tm * kMxTile + r) * p.ldc + tn * kMxTile;
      const int left = tm * kMxTile + r < p.m ? p.n - tn * kMxTile : 0;
#pragma unroll 1
      for (int c = 0; c < kMxTile; c += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c, v);
        constexpr int PER = 16 / (int)sizeof(T);
#pragma unroll
        for (int i = 0; i < 32; i += PER) {
          union {
            T e[PER];
            uint4 u;
          } o;
#pragma unroll
          for (int j = 0; j < PER; ++j) o.e[j] = mx_from_f32<T>(alpha * __uint_as_float(v[i + j]));
          if (c + i + PER <= left) {
            *reinterpret_cast<uint4*>(out + c + i) = o.u;
          } else {
#pragma unroll
            for (int j = 0; j < PER; ++j)
              if (c + i + j < left) out[c + i + j] = o.e[j];
          }
        }
      }
    } else if (fine && tm * kMxTile + q * 32 < p.m) {
      // The ring is idle: every stage was read by MMAs that are complete.
#pragma unroll
      for (int c = 0; c < kMxTile; c += 64) {
        uint32_t v[2][32];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          tmem_ld32_async(tmem + ((uint32_t)(q * 32) << 16) + c + h * 32, v[h]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tmem_ld_wait32(v[h]);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(part + r * kMxPitch + c + h * 32 + i) =
                make_uint4(v[h][i], v[h][i + 1], v[h][i + 2], v[h][i + 3]);
        }
      }
    }
    __syncwarp();
  }
  if (warp < 2) alpha = factor();
  const float* part = reinterpret_cast<const float*>(ring);
  if (p.split == 1) {
    // A warp writes the 32 rows that its own lanes stored.
    const int row0 = tm * kMxTile + (warp & 3) * 32, col = tn * kMxTile + lane * 4;
    if (warp >= 2 && fine && !direct && col < p.n) {
      const float* src = part + (warp & 3) * 32 * kMxPitch + lane * 4;
#pragma unroll 1
      for (int i = 0; i < 32 && row0 + i < p.m; i += 4) {
        float4 u[4];  // read before the stores, which the compiler would keep them behind
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = *reinterpret_cast<const float4*>(src + (i + j) * kMxPitch);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (row0 + i + j < p.m) mx_write4<T>(p, row0 + i + j, col, u[j], alpha);
      }
    }
  } else {
    cluster_sync();
    if (fine) {
      if (p.split == 2) mx_reduce_rows<T, 2>(p, part, warp, lane, rank, tm, tn, alpha);
      else if (p.split == 4) mx_reduce_rows<T, 4>(p, part, warp, lane, rank, tm, tn, alpha);
      else mx_reduce_rows<T, 8>(p, part, warp, lane, rank, tm, tn, alpha);
    }
    __syncwarp();
    cluster_meet();  // no CTA leaves while another reads its partial sums
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  // Copies that no MMA waited for land before the CTA leaves.
  if (warp == 0 && issued > 0 && mx_aborted(aux))
    for (int i = issued > C::STAGES ? issued - C::STAGES : 0; i < issued; ++i)
      mx_wait(&aux->full[i % C::STAGES], (uint32_t)((i / C::STAGES) & 1), aux, true);
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(&p.report->launches, 1u);
}

template <int FMT, bool FEW, typename T>
cudaError_t launch_mx(const CUtensorMap (&t)[5], const MxParams& p, cudaStream_t stream) {
  using C = MxCfg<FMT, FEW>;
  static std::atomic<uint64_t> done_mask{0};
  const cudaError_t e = opt_in_smem((const void*)mx_gemm_kernel<FMT, FEW, T>, done_mask, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  return launch_pdl_cluster(mx_gemm_kernel<FMT, FEW, T>, dim3((unsigned)(tiles * p.split)),
                            dim3(kMxThreads), C::SMEM, stream, p.split, t[0], t[1], t[2], t[3], p);
}

template <int FMT, bool FEW>
cudaError_t launch_mx_out(const CUtensorMap (&t)[5], const MxParams& p, int out,
                          cudaStream_t stream) {
  if (out == SKG_OUT_F32) return launch_mx<FMT, FEW, float>(t, p, stream);
  if (out == SKG_OUT_F16) return launch_mx<FMT, FEW, __half>(t, p, stream);
  return launch_mx<FMT, FEW, __nv_bfloat16>(t, p, stream);
}

// Single CTAs: how many share a 128 x 128 tile (S), and the estimated time (us).
// Up to 16 rows of A the sum over the cluster is a few rows, and S is what fits the
// GPU at once (two CTAs per SM): 1 x 1024 x 8192 in mxfp8 takes 19.8, 9.3, 6.0,
// 4.6 us with S = 1, 2, 4, 8. Else a CTA's 64 KB of partial sums cross the
// SM-to-SM network, S = 8 never pays (512 x 512 x 8192 nvfp4: 12.3, 8.8, 7.0,
// 8.9), and the estimate decides: a fixed cost plus the CTA's stages of k, both
// higher where two CTAs share an SM.
struct SinglePlan {
  int split;
  double us;
};
SinglePlan single_plan(int64_t m, int64_t n, int ksteps, int sms) {
  const int64_t tiles = ((m + 127) / 128) * ((n + 127) / 128);
  SinglePlan best = {1, 1e30};
  for (int s = 1; s <= (m <= 16 ? kMxSplitMax : 4); s *= 2) {
    if (s > 1 && (tiles * s > 2 * sms || s > ksteps)) break;
    const int64_t waves = (tiles * s + 2 * sms - 1) / (2 * sms);
    const int stages = (ksteps + s - 1) / s;
    const double us = tiles * s <= sms ? (s > 1 ? 4.2 : 3.2) + 0.36 * stages
                                       : (s > 1 && m > 64 ? 6.5 : 5.2) + 0.48 * waves * stages;
    if (m <= 16 || us < best.us) best = {s, us};
  }
  return best;
}

// Whether a product runs on CTA pairs: 256 x 256 tiles halve what each SM reads
// per product, but cannot share a tile's k. Up to 128 rows the single CTAs win at
// every n and k (1 x 8192 x 8192 in nvfp4: 9.6 against 17.9 us); beyond, the lower
// estimate (512 x 512 x 8192 in nvfp4: 12.4 us paired, 6.7 single; 2048 x 2048 x
// 2048: 6.5 paired, 8.9 single).
bool wants_pairs(int64_t m, int64_t n, int ksteps, int clusters, double single_us) {
  if (m <= kMxTile) return false;
  const int64_t tiles = ((m + 255) / 256) * ((n + 255) / 256);
  return 4.2 + 0.29 * (double)((tiles + clusters - 1) / clusters) * ksteps <= single_us;
}

template <int FMT>
cudaError_t plan_and_launch(const void* A, int64_t lda, const void* SA, const void* B, int64_t ldb,
                            const void* SB, MxParams p, int out, int sms, cudaStream_t stream,
                            bool* unsupported) {
  using C = MxStage<FMT>;
  p.groups = (int)mx_groups(p.k, FMT);
  p.ksteps = (p.k + C::STEP - 1) / C::STEP;
  const int64_t rt_a = (p.m + kMxTile - 1) / kMxTile, rt_b = (p.n + kMxTile - 1) / kMxTile;
  const int resident = mx_pair_clusters_resident();
  const SinglePlan single = single_plan(p.m, p.n, p.ksteps, sms);
  const bool pair = resident > 0 && wants_pairs(p.m, p.n, p.ksteps, resident, single.us);
  const int64_t tm = pair ? (rt_a + 1) / 2 : rt_a, tn = pair ? (rt_b + 1) / 2 : rt_b;
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.split = pair ? 1 : single.split;
  // A CTA that has a tile and an SM to itself writes it from its registers: half
  // sectors, but without the way through shared memory (128 x 8192 x 512 in mxfp8 4.1
  // against 5.0 us). With more tiles, or one row of 32 lanes in use, whole sectors are
  // faster (128 x 28672 x 2048 14.5 against 15.1, 1 x 28672 x 1024 7.8 against 8.5).
  p.direct = !pair && p.split == 1 && p.c_tma && p.m > 16 && tm * tn <= sms;
  p.a_rows = !pair && p.m < kMxTile ? (p.m + 7) / 8 * 8 : kMxTile;
  const uint64_t bytes = ((uint64_t)p.k * mx_bits(FMT) + 7) / 8;
  const uint64_t chunks_a = (uint64_t)rt_a * p.groups, chunks_b = (uint64_t)rt_b * p.groups;
  // Tile and scale-tile numbers are 32-bit, one tile past the end included.
  *unsupported = tm * tn * p.split > INT32_MAX || chunks_a + 2 * (uint64_t)p.groups > INT32_MAX ||
                 chunks_b + 2 * (uint64_t)p.groups > INT32_MAX;
  if (*unsupported) return cudaErrorInvalidValue;
  CUtensorMap t[5];
  if (encode_tensor_map(&t[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, A, bytes, (uint64_t)p.m,
                        (uint64_t)lda, kMxRowBytes, (uint32_t)p.a_rows,
                        CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tensor_map(&t[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, B, bytes, (uint64_t)p.n,
                        (uint64_t)ldb, kMxRowBytes, kMxTile,
                        CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS ||
      encode_tensor_map(&t[2], CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, SA, kMxTileBytes / 4, chunks_a,
                        kMxTileBytes / 4, kMxTileBytes / 4, C::CHUNKS,
                        CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS ||
      encode_tensor_map(&t[3], CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, SB, kMxTileBytes / 4, chunks_b,
                        kMxTileBytes / 4, kMxTileBytes / 4, C::CHUNKS,
                        CU_TENSOR_MAP_SWIZZLE_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  t[4] = t[0];
  const int es = out == SKG_OUT_F32 ? 4 : 2;
  if (pair && p.n < 16 / es) p.c_tma = 0;  // (no whole 16 bytes to store)
  if (pair && p.c_tma) {
    const CUtensorMapDataType dt = out == SKG_OUT_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : out == SKG_OUT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    if (encode_tensor_map(&t[4], dt, es, p.c, (uint64_t)(p.n / (16 / es) * (16 / es)),
                          (uint64_t)p.m, (uint64_t)p.ldc, (uint32_t)(128 / es), 32,
                          CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (pair)
    return launch_mx_pair<FMT>(t, p, out, (int)(tm * tn < resident ? tm * tn : resident), stream);
  return p.m <= 16 ? launch_mx_out<FMT, true>(t, p, out, stream)
                   : launch_mx_out<FMT, false>(t, p, out, stream);
}

}  // namespace
}  // namespace skg

using namespace skg;

namespace {

// skg_mx_test_stall's settings.
std::atomic<uint32_t> g_test_stages{0};
std::atomic<uint64_t> g_test_limit{0};

}  // namespace

extern "C" {

skg_status_t skg_mx_test_stall(int32_t stages, uint64_t timeout_ns) {
  if (stages < 0) return SKG_ERR_ARG;
  g_test_stages.store((uint32_t)stages, std::memory_order_relaxed);
  g_test_limit.store(timeout_ns, std::memory_order_relaxed);
  return SKG_OK;
}

size_t skg_workspace_size_mx(int64_t m, int64_t n, int64_t k, int32_t format) {
  if (m < 0 || n < 0 || k < 0 || format < SKG_MXFP8 || format > SKG_NVFP4) return 0;
  return fixed_header_bytes();
}

skg_status_t skg_gemm_mx(int64_t m, int64_t n, int64_t k, float alpha, const void* A, int64_t lda,
                         const void* scales_a, const float* tensor_scale_a, const void* B,
                         int64_t ldb, const void* scales_b, const float* tensor_scale_b,
                         float beta, void* C, int64_t ldc, int32_t format, int32_t out_dtype,
                         void* workspace, size_t ws_bytes, void* stream_v) {
  if (m < 0 || n < 0 || k < 0) return SKG_ERR_ARG;
  if (format < SKG_MXFP8 || format > SKG_NVFP4) return SKG_ERR_ARG;
  if (out_dtype < SKG_OUT_F32 || out_dtype > SKG_OUT_BF16) return SKG_ERR_ARG;
  if (m == 0 || n == 0) return SKG_OK;
  if (!C || ldc < n) return SKG_ERR_ARG;
  const int64_t ld = skg_mx_codes_ld(k, format);
  if (k > 0 && (!A || !B || !scales_a || !scales_b || lda < ld || ldb < ld)) return SKG_ERR_ARG;
  if (m > INT32_MAX / 4 || n > INT32_MAX / 4 || k > INT32_MAX / 4) return SKG_ERR_UNSUPPORTED;
  const int es = out_dtype == SKG_OUT_F32 ? 4 : 2;
  if ((uintptr_t)C & (es - 1)) return SKG_ERR_UNSUPPORTED;
  cudaStream_t stream = (cudaStream_t)stream_v;
  if (k == 0)
    return launch_scale(out_dtype, C, ldc, (int)m, (int)n, beta, stream) == cudaSuccess
               ? SKG_OK
               : SKG_ERR_CUDA;
  // The TMA engine's rule.
  if (((uintptr_t)A & 15) || ((uintptr_t)B & 15) || ((uintptr_t)scales_a & 15) ||
      ((uintptr_t)scales_b & 15) || (lda & 15) || (ldb & 15) || ((uintptr_t)tensor_scale_a & 3) ||
      ((uintptr_t)tensor_scale_b & 3))
    return SKG_ERR_UNSUPPORTED;
  if (!workspace || ((uintptr_t)workspace & 255) ||
      ws_bytes < skg_workspace_size_mx(m, n, k, format))
    return SKG_ERR_WORKSPACE;
  const int sms = skg_device_sm_count();
  if (sms <= 0) return SKG_ERR_CUDA;
  MxParams p = {};
  p.m = (int)m;
  p.n = (int)n;
  p.k = (int)k;
  p.alpha = alpha;
  p.beta = beta;
  p.ga = tensor_scale_a;
  p.gb = tensor_scale_b;
  p.c = C;
  p.ldc = ldc;
  p.c_vec = ((uintptr_t)C & (4 * es - 1)) == 0 && ldc % 4 == 0;
  p.c_tma = ((uintptr_t)C & 15) == 0 && (ldc * es) % 16 == 0 && beta == 0.f;
  p.report = workspace_report(workspace);
  const uint32_t stages = g_test_stages.load(std::memory_order_relaxed);
  const uint64_t limit = g_test_limit.load(std::memory_order_relaxed);
  p.stages = stages ? stages : UINT32_MAX;
  p.limit = limit ? limit : kMxTimeoutNs;
  bool unsupported = false;
  cudaError_t e;
  if (format == SKG_MXFP8)
    e = plan_and_launch<SKG_MXFP8>(A, lda, scales_a, B, ldb, scales_b, p, out_dtype, sms, stream,
                                   &unsupported);
  else if (format == SKG_MXFP4)
    e = plan_and_launch<SKG_MXFP4>(A, lda, scales_a, B, ldb, scales_b, p, out_dtype, sms, stream,
                                   &unsupported);
  else
    e = plan_and_launch<SKG_NVFP4>(A, lda, scales_a, B, ldb, scales_b, p, out_dtype, sms, stream,
                                   &unsupported);
  if (unsupported) return SKG_ERR_UNSUPPORTED;
  return e == cudaSuccess ? SKG_OK : SKG_ERR_CUDA;
}

}  // extern "C"
