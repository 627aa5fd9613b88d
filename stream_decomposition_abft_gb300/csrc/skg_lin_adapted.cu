// A projection with low-rank adapters in one kernel, where a tile's rows can have few: y =
// x W^T + t B^T and t = scale (x A^T) from the same stages.
//
// As in skg_lin_single.cu a CTA runs a 128 x 128 tile of y over a range of k; its stages also
// hold the rows of A_s of every adapter that the tile's rows use (at most 128 in all), behind
// W's rows, so that the MMAs form x A^T beside x W^T: up to 128 more columns (16 adapters of
// rank 8, one of 128). Then
//   - each row keeps its own adapter's columns; the CTAs of a cluster add up their ranges of k
//     through distributed shared memory,
//   - t in high and low parts becomes an operand in shared memory, and one CTA of the cluster
//     for each adapter adds t B_s^T to its accumulator, other adapters' rows left out
//     (skg_lin_single.cu), with B_s brought to shared memory meanwhile,
//   - the tile goes out as any other.
//
// This reads A once per column of tiles (from L2) and multiplies more columns, but is one
// launch where skg_lora.cu and the product behind it are two that wait for one another: 1 x
// 8192 x 8192 with one adapter of rank 16 25.9 us (two launches 29; without adapters 23), 1 x
// 2200 x 1000 6.8 (9.7; 4.1), 333 x 2200 x 1000 with five of rank 8 13.1 (15; 8.7). One token
// is bound by W's bytes; small sizes by the two exchanges over the cluster behind one another.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_lin_single.cuh"

namespace skg {
namespace {

// FEW: at most 16 rows (see SingleCfg), two CTAs to an SM; else one.
template <bool FEW>
struct AdaptedCfg {
  static constexpr int B_OFF = FEW ? 16 * 128 : kLinOperand;
  static constexpr int D_OFF = B_OFF + kLinOperand;
  static constexpr int ROWS = FEW ? 16 : kLinTile;  // of a tile
  static constexpr int SLOTS = 16;                  // adapters of a tile (their ranks: 8 at least)
  static constexpr int MAX_STAGES = 8;
  // Once the stages are idle: t's operand (up to four pieces of 128 rows x 128 bytes), then the
  // partial tile in its place; the partial sums of t.
  static constexpr int PART = 68 * 1024;
  static constexpr int RING = FEW ? 100 * 1024 : 184 * 1024;
  static_assert(4 * kLinOperand <= PART && kLinTile * kLinPitch * 4 <= PART, "t's operand, the tile");
  static_assert(PART + ROWS * kLinPitch * 4 <= RING, "the partial sums of t");
};

struct AdaptedAux : LinAux {
  uint64_t ups;  // B_s is there
};

struct AdaptedPlan {
  int32_t ids[kLinTile], slot[kLinTile];
  uint32_t lead[4];
  int32_t id[16];
  float scale[16];
  uint32_t rows[16][4];
};

constexpr int kAux = 256;
static_assert(sizeof(AdaptedAux) <= kAux, "aux size");
constexpr int adapted_smem(int ring, int ups) {
  return 1024 + ring + ups + kAux + (int)sizeof(AdaptedPlan);
}
static_assert(2 * (adapted_smem(100 * 1024, 8192) + 1024) <= 233472, "two adapters of rank 16");
static_assert(adapted_smem(184 * 1024, kUpsMax) <= (int)kSmemLimit, "shared memory");

template <bool FEW, typename T>
__global__ void __launch_bounds__(kLinThreads, FEW ? 2 : 1)
lin_adapted_kernel(const __grid_constant__ LinMaps maps, const __grid_constant__ CUtensorMap tmD,
                   const LinParams p, const AdaptedParams a) {
  using C = AdaptedCfg<FEW>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int rp = p.rank_pad, per = lora_stages(rp), one = lora_bytes(rp);
  const int mine_most = (a.most + p.split - 1) / p.split;  // adapters to a CTA of the cluster
  uint8_t* ups = ring + C::RING;
  AdaptedAux* aux = reinterpret_cast<AdaptedAux*>(ups + mine_most * per_ups(rp));
  AdaptedPlan* pl = reinterpret_cast<AdaptedPlan*>(reinterpret_cast<uint8_t*>(aux) + kAux);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = (int)blockIdx.x / p.split;
  const int tm = tile % p.tiles_m, tn = tile / p.tiles_m;
  const int kb0 = (int)((int64_t)p.ksteps * rank / p.split);
  const int kb1 = (int)((int64_t)p.ksteps * (rank + 1) / p.split);
  const int rows = min(kLinTile, p.m - tm * kLinTile);
  const int stages = a.stages;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.up);
    prefetch_tmap(&tmD);
    aux->abort_flag = 0;
    aux->limit = p.limit;
    for (int i = 0; i < stages; ++i) {
      mbar_init(&aux->full[i], 1);
      mbar_init(&aux->empty[i], 1);
    }
    mbar_init(&aux->tfull[0], 1);
    mbar_init(&aux->tfull[1], 1);
    mbar_init(&aux->drain, 1);
    mbar_init(&aux->ups, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&aux->tmem_slot, 256);
    tmem_relinquish();
  }
  if (threadIdx.x < 64) (&pl->rows[0][0])[threadIdx.x] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = aux->tmem_slot;
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();

  const bool loader = warp == 0 || warp == kLinLoader;
  const int me = warp == kLinLoader;  // a loading thread takes every other stage
  const uint32_t tx = (uint32_t)p.a_rows * 128 + kLinOperand;
  int seq = 0, early = 0, ups_loaded = 0;
  auto load = [&](int i, int st) {  // x and W of stage i
    uint8_t* s = ring + st * a.stage_bytes;
    tma_load_2d(s, &maps.a, &aux->full[st], (kb0 + i) * kLinK, tm * kLinTile);
    tma_load_2d(s + C::B_OFF, &maps.b, &aux->full[st], (kb0 + i) * kLinK, tn * kLinTile);
  };
  // The first stages' x and W are under way while the rows' adapters are found.
  if (loader && elect_one()) {
    early = min(min(stages, kb1 - kb0), (int)min(p.stages, (uint32_t)C::MAX_STAGES));
    for (int i = me; i < early; i += 2) {
      mbar_expect_tx(&aux->full[i], tx);
      load(i, i);
    }
  }
  __syncwarp();
  const int count = number_adapters<kLinThreads>(
      a.index, a.count, tm * kLinTile, rows, (int)threadIdx.x, pl->ids, pl->slot, pl->lead,
      [&](int s, int id) {
        pl->id[s] = id;
        pl->scale[s] = a.scale ? a.scale[id] : 1.f;
      },
      [&](int s, int w, uint32_t m) { pl->rows[s][w] = m; });

  bool fine = true;
  if (loader) {
    if (elect_one()) {
      if (me) {  // B_s of this CTA's adapters
        const int here = count > rank ? (count - rank + p.split - 1) / p.split : 0;
        if (here > 0) {
          const int pieces = rp <= 32 ? 1 : per / 2;
          mbar_arrive_expect_tx(&aux->ups, (uint32_t)(here * pieces * one));
          for (int e = 0; e < here; ++e)
            for (int j = 0; j < pieces; ++j)
              tma_load_3d(ups + (e * pieces + j) * one, &maps.up, &aux->ups, j * 64, tn * kLinTile,
                          pl->id[rank + e * p.split]);
          ups_loaded = 1;
        }
      }
      int id[C::SLOTS];
#pragma unroll
      for (int j = 0; j < C::SLOTS; ++j) id[j] = j < count ? pl->id[j] : 0;
      int st = 0;
      uint32_t phase = 0;
      const int ks = kb1 - kb0;
      for (; seq < ks; ++seq) {
        if ((seq & 1) == me) {
          if ((uint32_t)seq >= p.stages) break;
          if (!mx_wait(&aux->empty[st], phase ^ 1u, aux)) {
            lin_fail(p, aux);
            break;
          }
          mbar_arrive_expect_tx(&aux->full[st],
                                (seq < early ? 0 : tx) + (uint32_t)(count * a.rank) * 128);
          if (seq >= early) load(seq, st);
          uint8_t* d = ring + st * a.stage_bytes + C::D_OFF;
#pragma unroll
          for (int j = 0; j < C::SLOTS; ++j)
            if (j < count)
              tma_load_3d(d + j * a.rank * 128, &tmD, &aux->full[st], (kb0 + seq) * kLinK, 0, id[j]);
        }
        if (++st == stages) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      const uint64_t a0 = lin_desc<false>(smem_u32(ring));
      const uint64_t b0 = lin_desc<false>(smem_u32(ring) + C::B_OFF);
      int st = 0;
      uint32_t phase = 0;
      bool ok = true, ready = false;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!ready && !mx_wait(&aux->full[st], phase, aux)) {
          lin_fail(p, aux);
          ok = false;
          break;
        }
        tc_fence_after();
        const int mine = st;
        if (++st == stages) {
          st = 0;
          phase ^= 1u;
        }
        ready = mbar_test_wait(&aux->full[st], phase);  // (as LinRing does)
        const uint64_t at = (uint64_t)((mine * a.stage_bytes) >> 4);
        lin_stage_mmas<false, false, false>(tmem, a0 + at, b0 + at, p.idesc, p.k - kb * kLinK,
                                            kb == kb0);
        umma_commit(&aux->empty[mine]);
      }
      if (ok) umma_commit(&aux->tfull[0]);
    }
    __syncwarp();
  } else {
    fine = mx_wait(&aux->tfull[0], 0, aux);
    if (!fine) lin_fail(p, aux);
    fine = epi_all(fine);
    tc_fence_after();
    // The ring is idle. Each row keeps its own adapter's columns of t.
    const int q = warp & 3, r = q * 32 + lane;
    float* tp = reinterpret_cast<float*>(ring + C::PART) + r * kLinPitch;
    if (fine && q * 32 < rows) {
      const int from = r < rows && pl->ids[r] >= 0 ? pl->slot[r] * a.rank : -1;
      for (int c = 0; c < count * a.rank; c += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + kLinTile + c, v);
#pragma unroll
        for (int h = 0; h < 32; h += 8)
          if (from >= 0 && c + h >= from && c + h < from + a.rank) {
#pragma unroll
            for (int i = 0; i < 8; i += 4)
              *reinterpret_cast<uint4*>(tp + c + h - from + i) =
                  make_uint4(v[h + i], v[h + i + 1], v[h + i + 2], v[h + i + 3]);
          }
      }
    }
    __syncwarp();
    tc_fence_before();
  }
  if (p.split > 1) cluster_sync();
  else __syncthreads();
  // t of the rows whose adapter is this CTA's: the sum over the cluster, scaled, in two parts,
  // in the order of a K-major operand with the 128-byte swizzle.
  if (!mx_aborted(aux)) {
    const float* tp = reinterpret_cast<const float*>(ring + C::PART);
    const int quads = rp / 4;
    for (int i = (int)threadIdx.x; i < rows * quads; i += kLinThreads) {
      const int r = i / quads, c = (i - r * quads) * 4;
      const int s = pl->slot[r];
      if (pl->ids[r] < 0 || s % p.split != rank) continue;
      const float* src = tp + r * kLinPitch + c;
      float4 u[8];  // the loads in flight together
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < p.split)
          u[e] = p.split > 1 ? ld_shared_cluster_f32x4(cluster_addr(src, (uint32_t)e))
                             : *reinterpret_cast<const float4*>(src);
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < p.split) {
          v[0] += u[e].x;
          v[1] += u[e].y;
          v[2] += u[e].z;
          v[3] += u[e].w;
        }
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = c + e < a.rank ? pl->scale[s] * v[e] : 0.f;
      // The pieces of A that lora_stage_mmas reads: one with both parts, or each part's 64s.
      auto at = [&](int part) {
        const int piece = rp <= 32 ? 0 : (c >> 6) * 2 + part;
        const int col = rp <= 32 ? part * rp + c : c & 63;
        return reinterpret_cast<T*>(ring + piece * kLinOperand + r * 128 +
                                    (((col >> 3) ^ (r & 7)) << 4) + (col & 7) * 2);
      };
      store_parts<T>(at(0), at(1), v);
    }
  }
  fence_proxy_async_smem();
  __syncthreads();
  if (warp == 1) {
    if (elect_one()) {
      bool ok = !mx_aborted(aux);
      if (ok && count > rank) {
        ok = mx_wait(&aux->ups, 0, aux);
        if (!ok) lin_fail(p, aux);
        tc_fence_after();
        const int pieces = rp <= 32 ? 1 : per / 2;
        const uint32_t t0 = smem_u32(ring), u0 = smem_u32(ups);
        for (int u = rank, e = 0; ok && u < count; u += p.split, ++e) {
          const uint32_t off[4] = {~pl->rows[u][0], ~pl->rows[u][1], ~pl->rows[u][2],
                                   ~pl->rows[u][3]};
          for (int j = 0; j < per; ++j)
            lora_stage_mmas<false>(tmem, t0 + j * kLinOperand,
                                   u0 + (e * pieces + (rp <= 32 ? 0 : j >> 1)) * one, a.idesc_up,
                                   rp, j, 0, off);
        }
      }
      if (ok) umma_commit(&aux->tfull[1]);
      umma_commit(&aux->drain);
      mx_wait(&aux->drain, 0, aux, true);
    }
    __syncwarp();
  } else if (!loader) {
    fine = fine && mx_wait(&aux->tfull[1], 0, aux);
    if (!fine) lin_fail(p, aux);
    fine = epi_all(fine);
    tc_fence_after();
    const int q = warp & 3;
    if (fine && q * 32 < rows) keep_rows(tmem, q, lane, reinterpret_cast<float*>(ring));
    __syncwarp();
  }
  tile_out<kLinPlain, T>(p, reinterpret_cast<const float*>(ring), warp, lane, rank, tm, tn, fine);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
  // Copies land before the CTA leaves: early ones of stages not come to, whose barriers lack
  // the arrival, and those that no MMA waited for.
  if (mx_aborted(aux)) {
    for (int i = 0; i < early; ++i)
      if ((i & 1) == me && i >= seq) {
        mbar_arrive(&aux->full[i]);
        mx_wait(&aux->full[i], 0, aux, true);
      }
    for (int i = seq > stages ? seq - stages : 0; i < seq; ++i)
      if ((i & 1) == me)
        mx_wait(&aux->full[i % stages], (uint32_t)((i / stages) & 1), aux, true);
    if (ups_loaded) mx_wait(&aux->ups, 0, aux, true);
  }
  __syncwarp();
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(&p.report->launches, 1u);
}

template <bool FEW, typename T>
cudaError_t launch(const LinMaps& t, const CUtensorMap& down, const LinParams& p, AdaptedParams a,
                   cudaStream_t stream) {
  using C = AdaptedCfg<FEW>;
  auto kernel = lin_adapted_kernel<FEW, T>;
  const int ups = (a.most + p.split - 1) / p.split * per_ups(p.rank_pad);
  const int smem = adapted_smem(C::RING, ups);
  static std::atomic<uint64_t> done_mask{0};
  const cudaError_t e =
      opt_in_smem((const void*)kernel, done_mask, adapted_smem(C::RING, kUpsMax));
  if (e != cudaSuccess) return e;
  a.stage_bytes = C::D_OFF + a.most * a.rank * 128;
  a.stages = C::RING / a.stage_bytes;
  if (a.stages > C::MAX_STAGES) a.stages = C::MAX_STAGES;
  return launch_pdl_cluster(kernel, dim3((unsigned)((int64_t)p.tiles_m * p.tiles_n * p.split)),
                            dim3(kLinThreads), (size_t)smem, stream, p.split, t, down, p, a);
}

}  // namespace

cudaError_t launch_lin_adapted(int out, const LinMaps& t, const CUtensorMap& down,
                               const LinParams& p, AdaptedParams a, cudaStream_t stream) {
  if (out == SKG_OUT_F16)
    return p.m <= 16 ? launch<true, __half>(t, down, p, a, stream)
                     : launch<false, __half>(t, down, p, a, stream);
  return p.m <= 16 ? launch<true, __nv_bfloat16>(t, down, p, a, stream)
                   : launch<false, __nv_bfloat16>(t, down, p, a, stream);
}

}  // namespace skg
