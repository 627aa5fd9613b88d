// Gradients' products of a layer in one launch: dX = DPRE W (or any K-major A) and the weight
// gradients DPRE^T X and dY^T H, up to three products with N-major B on single CTAs
// (skg_lin_single.cu's tiles). Each alone leaves most of the GPU idle at small sizes, and a
// launch costs 3 us at least; their tiles do not depend on one another.
//
// The first product's tiles, whose sums are the longest (k = 2 hidden), are shared by the CTAs
// of a cluster as there; in the clusters behind, every CTA has a tile of the others of its own.
// The whole gradient of 323 tokens, width 520, hidden 256 takes 11.9 us with this launch and 21.6
// with three in its place; of 2 tokens, width 528, hidden 136 from a given dH 5.8 and 9.1. Where
// the tiles go round more than once, the pairs or a cluster for each tile are faster apart.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_lin_single.cuh"

namespace skg {
namespace {

constexpr int kStages = 3;  // two CTAs share an SM
constexpr int kStageBytes = 2 * kLinOperand;
constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + 256;
static_assert(sizeof(LinAux) <= 256, "aux size");
static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs per SM");
static_assert(kLinTile * kLinPitch * 4 <= kStages * kStageBytes, "the partial tile fits the ring");

template <typename T>
__global__ void __launch_bounds__(kLinThreads, 2)
lin_group_kernel(const __grid_constant__ LinGroupMaps maps, const __grid_constant__ LinGroup p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  LinAux* aux = reinterpret_cast<LinAux*>(ring + kStages * kStageBytes);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int cluster = (int)blockIdx.x / p.split;
  const int job = (cluster >= p.first[1]) + (cluster >= p.first[2]);
  const LinJob& w = p.job[job];
  const bool share = job == 0 && p.split > 1;
  const int local = cluster - p.first[job];
  const int tile = job == 0 ? local : local * p.split + rank;
  const bool live = tile < w.tiles_m * w.tiles_n;  // else a CTA behind the last tile
  const int tm = tile % w.tiles_m, tn = tile / w.tiles_m;
  const int ks = live ? w.ksteps * w.terms : 0;
  const int kb0 = share ? (int)((int64_t)ks * rank / p.split) : 0;
  const int kb1 = share ? (int)((int64_t)ks * (rank + 1) / p.split) : ks;
  LinParams q = {};
  q.m = w.m;
  q.n = w.n;
  q.c = w.c;
  q.ldc = w.ldc;
  q.split = share ? p.split : 1;
  q.report = p.report;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&maps.a[job]);
    prefetch_tmap(&maps.b[job]);
    aux->abort_flag = 0;
    aux->limit = p.limit;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&aux->full[i], 1);
      mbar_init(&aux->empty[i], 1);
    }
    mbar_init(&aux->tfull[0], 1);
    mbar_init(&aux->drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&aux->tmem_slot, kLinTile);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = aux->tmem_slot;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();

  bool fine = live;  // the accumulator is there
  int seq = 0;       // loading threads: stages gone through, every other one by this thread
  const int me = warp == kLinLoader;
  const bool amn = w.a_mn != 0;
  if (warp == 0 || warp == kLinLoader) {
    if (elect_one()) {
      int st = 0;
      uint32_t phase = 0;
      for (int i = kb0; i < kb1; ++i, ++seq) {
        if ((seq & 1) == me) {
          if ((uint32_t)seq >= p.stages) break;
          if (!mx_wait(&aux->empty[st], phase ^ 1u, aux)) {
            lin_fail(q, aux);
            break;
          }
          uint64_t* bar = &aux->full[st];
          mbar_arrive_expect_tx(bar, kStageBytes);
          const bool lo = w.terms == 2 && (i & 1);
          const int k0 = (w.terms == 2 ? i >> 1 : i) * kLinK;
          const CUtensorMap* ma = lo && !w.lo_b ? &maps.lo[job] : &maps.a[job];
          const CUtensorMap* mb = lo && w.lo_b ? &maps.lo[job] : &maps.b[job];
          uint8_t* s = ring + st * kStageBytes;
          if (amn) {
            tma_load_2d(s, ma, bar, tm * kLinTile, k0);
            tma_load_2d(s + kLinBox, ma, bar, tm * kLinTile + 64, k0);
          } else {
            tma_load_2d(s, ma, bar, k0, tm * kLinTile);
          }
          tma_load_2d(s + kLinOperand, mb, bar, tn * kLinTile, k0);
          tma_load_2d(s + kLinOperand + kLinBox, mb, bar, tn * kLinTile + 64, k0);
        }
        if (++st == kStages) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      LinRing<kStages> r = {aux, aux->full};
      const uint64_t a0 = amn ? lin_desc<true>(smem_u32(ring)) : lin_desc<false>(smem_u32(ring));
      const uint64_t b0 = lin_desc<true>(smem_u32(ring) + kLinOperand);
      bool ok = true;
      for (int i = kb0; i < kb1; ++i) {
        const int st = r.take();
        ok = st >= 0;
        if (!ok) break;
        const uint64_t at = (uint64_t)((st * kStageBytes) >> 4);
        const int left = w.k - (w.terms == 2 ? i >> 1 : i) * kLinK;
        if (amn)
          lin_stage_mmas<false, true, true>(tmem, a0 + at, b0 + at, w.idesc, left, i == kb0);
        else
          lin_stage_mmas<false, false, true>(tmem, a0 + at, b0 + at, w.idesc, left, i == kb0);
        umma_commit(&aux->empty[st]);
      }
      if (!ok) lin_fail(q, aux);
      // (A CTA without a tile commits nothing: it would leave before the arrival.)
      if (ok && live) umma_commit(&aux->tfull[0]);
      if (r.used > 0) {
        umma_commit(&aux->drain);
        mx_wait(&aux->drain, 0, aux, true);
      }
    }
    __syncwarp();
  } else if (live) {
    fine = mx_wait(&aux->tfull[0], 0, aux);
    if (!fine) lin_fail(q, aux);
    fine = epi_all(fine);
    tc_fence_after();
    // The ring is idle: every stage was read by MMAs that are complete.
    const int quarter = warp & 3;
    if (fine && tm * kLinTile + quarter * 32 < q.m)
      keep_rows(tmem, quarter, lane, reinterpret_cast<float*>(ring));
    __syncwarp();
  }
  tile_out<kLinPlain, T>(q, reinterpret_cast<const float*>(ring), warp, lane, rank, tm, tn, fine);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kLinTile);
  }
  // Copies that no MMA waited for land before the CTA leaves.
  if (seq > 0 && mx_aborted(aux))
    for (int i = seq > kStages ? seq - kStages : 0; i < seq; ++i)
      if ((i & 1) == me)
        mx_wait(&aux->full[i % kStages], (uint32_t)((i / kStages) & 1), aux, true);
  __syncwarp();
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(&p.report->launches, 1u);
}

template <typename T>
cudaError_t launch(const LinGroupMaps& t, const LinGroup& p, int clusters, cudaStream_t stream) {
  static std::atomic<uint64_t> done_mask{0};
  const cudaError_t e = opt_in_smem((const void*)lin_group_kernel<T>, done_mask, (int)kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(lin_group_kernel<T>, dim3((unsigned)(clusters * p.split)),
                            dim3(kLinThreads), kSmem, stream, p.split, t, p);
}

}  // namespace

cudaError_t launch_lin_group(int out, const LinGroupMaps& t, const LinGroup& p, int clusters,
                             cudaStream_t stream) {
  return out == SKG_OUT_F16 ? launch<__half>(t, p, clusters, stream)
                            : launch<__nv_bfloat16>(t, p, clusters, stream);
}

}  // namespace skg
