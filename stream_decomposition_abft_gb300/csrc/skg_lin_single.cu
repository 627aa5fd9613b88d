// A layer's projections on single CTAs: 128 x 128 tiles of the accumulator over a range of
// k. Two threads fill a ring of stages by TMA, one issues the MMAs, warps 2-5 take the
// accumulator out. In the gated mode a tile's columns are 64 of the gate's projection and
// the same 64 of the other.
//
// When the tiles are fewer than the CTAs that fit the GPU, the S CTAs of a cluster share a
// tile, a range of k each: every one leaves its partial sums in its own shared memory, and
// after a cluster barrier each adds the rows r, r + S, ... of all of them in rank order
// through distributed shared memory. No workspace, no atomics, the same result every time.
//
// Adapters. t = scale_s (x A_s^T) of all rows comes from the kernel before (skg_lora.cu),
// and y's low-rank part is a few more stages of k on the same accumulator: for each adapter
// s that a tile's rows use, the stage's A is t and its B is B_s, and the MMA leaves out the
// rows (TMEM lanes) of other adapters. So rows of any mixture share a tile, an adapter with
// infinities or NaN reaches its own rows alone, and y is written once. The stages over W
// need nothing of the kernel before: a warp that has nothing else to do yet waits for it
// (griddepcontrol.wait) and brings the tile's adapters to shared memory, so t is formed while
// W streams.
//
// What bounds it: with few rows the weights' bytes (1 x 8192 -> 28672 gated, 940 MB: 135 to
// 139 us, 6.8 to 7.0 TB/s; 1 x 8192 x 8192 23 us, 5.8 TB/s with the ramp and the tail of one
// wave); with more rows and few tiles launch, first loads and the sum over the cluster (128 x
// 1024 x 1024 5.6 us, of which two stages of k alone take 5.3); long k a stage's MMAs, 0.19 us
// for 64 of k where 256 cycles would be 0.13 (both operands of an M = N = 128 MMA come from
// shared memory; the pairs' M = N = 256 do not wait for them). Rows of k that are not whole
// 32-byte sectors take 0.43 us a stage (k = 2200 against 2208: 16.4 and 11.3 us with 35).
//
// Every wait is bounded; when one runs out the CTA records SKG_ERR_PIPELINE_TIMEOUT in the
// report, waits for its own copies and MMAs, still meets the cluster's barriers, frees its
// TMEM and leaves.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_lin_single.cuh"

namespace skg {
namespace {

constexpr int kPitch = kLinPitch;

// The ring. kFew: at most 16 rows of A. Its stages hold 16 rows of A (the MMA reads 128 from
// there: what follows in the stage, for rows of the accumulator that nothing reads), so that
// six stages of B fit where three do otherwise. kDeep: no more CTAs than SMs, so one has the
// shared memory of both.

// An adapter of a tile, and the lanes of the tile's rows that do not have it.
struct alignas(4) TilePlan {
  uint32_t off[4];
  int32_t id;
};

enum Ring { kFull = 0, kFew = 1, kDeep = 2 };
struct SingleAux : LinAux {
  uint64_t planned;  // the tile's adapters are in shared memory
  int32_t slots;     // their number
};

template <int RING>
struct SingleCfg {
  static constexpr int B_OFF = RING == kFew ? 16 * 128 : kLinOperand;
  static constexpr int STAGE_BYTES = B_OFF + kLinOperand;
  static constexpr int STAGES = RING == kFull ? 3 : 6;  // (but kDeep) two CTAs share an SM
  static_assert(STAGE_BYTES % 1024 == 0 && STAGE_BYTES >= kLinOperand,
                "swizzle atoms; A's 128 rows end inside the ring");
  static constexpr int SLOTS = RING == kFew ? 16 : kLinTile;  // adapters that a tile's rows have
  static constexpr uint32_t SMEM = 1024 + STAGES * STAGE_BYTES + 256 + SLOTS * sizeof(TilePlan);
  static_assert(kLinTile * kPitch * 4 <= STAGES * STAGE_BYTES, "the partial tile fits the ring");
  static_assert(sizeof(SingleAux) <= 256, "aux size");
  static_assert(RING == kDeep || 2 * (SMEM + 1024) <= 233472, "two CTAs per SM");
};

// One warp: the adapters that this tile's rows have, every split-th of them from `rank` on,
// from the 256 rows' plan to shared memory. All loads of 32 adapters are in flight together.
__device__ __forceinline__ void tile_plan(const LoraPlan* plan, int half, int split, int rank,
                                          int lane, TilePlan* out, SingleAux* aux) {
  // (The first 32 entries are read beside their number: what lies past it is not used.)
  uint4 r = *reinterpret_cast<const uint4*>(&plan->rows[lane][half * 4]);
  int id = plan->id[lane];
  const int count = plan->count;
  int n = 0;
  for (int u0 = 0; u0 < count; u0 += 32) {
    const int u = u0 + lane;
    if (u0 > 0 && u < count) {
      r = *reinterpret_cast<const uint4*>(&plan->rows[u][half * 4]);
      id = plan->id[u];
    }
    if (u >= count) r = make_uint4(0, 0, 0, 0);
    const bool some = (r.x | r.y | r.z | r.w) != 0;
    const uint32_t b = __ballot_sync(0xffffffffu, some);
    const int at = n + __popc(b & ((1u << lane) - 1));
    if (some && at % split == rank) {
      TilePlan& o = out[at / split];
      o.off[0] = ~r.x;
      o.off[1] = ~r.y;
      o.off[2] = ~r.z;
      o.off[3] = ~r.w;
      o.id = id;
    }
    n += __popc(b);
  }
  if (lane == 0) aux->slots = n > rank ? (n - rank + split - 1) / split : 0;
  __syncwarp();
  if (lane == 0) mbar_arrive(&aux->planned);
}

template <int MODE, int RING, bool AMN, bool BMN, typename T>
__global__ void __launch_bounds__(kLinThreads, 2)
lin_single_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
  using C = SingleCfg<RING>;
  constexpr bool G = MODE == kLinGated;
  constexpr bool LORA = MODE == kLinPlain && !AMN && !BMN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  SingleAux* aux = reinterpret_cast<SingleAux*>(ring + C::STAGES * C::STAGE_BYTES);
  TilePlan* slots = reinterpret_cast<TilePlan*>(ring + C::STAGES * C::STAGE_BYTES + 256);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int tile = (int)blockIdx.x / p.split;
  // Few rows: one row of tiles. Else a column of tiles after another, so that the CTAs in
  // flight share B.
  const int tm = tile % p.tiles_m, tn = tile / p.tiles_m;
  const int ks = p.ksteps * p.terms;
  const int kb0 = (int)((int64_t)ks * rank / p.split);
  const int kb1 = (int)((int64_t)ks * (rank + 1) / p.split);
  const LoraPlan* plan = LORA && p.plan ? p.plan + (tm >> 1) : nullptr;
  // The adapters' stages come last, or before the last eight of a long range of k: reading
  // the plan and t then passes under stages in flight.
  const int kx = kb1 - kb0 >= 24 ? kb1 - 8 : kb1;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    aux->abort_flag = 0;
    aux->limit = p.limit;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&aux->full[i], 1);
      mbar_init(&aux->empty[i], 1);
    }
    mbar_init(&aux->tfull[0], 1);
    mbar_init(&aux->drain, 1);
    mbar_init(&aux->planned, 1);
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
  // With adapters the kernel before is the one that forms t, which itself has waited for
  // all that ran before it: x and w are there, and y is free.
  if (!(LORA && plan)) {
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
  }

  bool fine = true;  // epilogue threads: the accumulator is there
  int seq = 0;       // loading threads: stages gone through, every other one by this thread
  const int me = warp == kLinLoader;
  if (warp == 0 || warp == kLinLoader) {
    if (elect_one()) {
      bool ok = true;
      int st = 0;
      uint32_t phase = 0;
      // One stage of so many bytes: when it is this thread's and free, load(address, barrier).
      auto step = [&](uint32_t bytes, auto load) {
        if ((seq & 1) == me) {
          if ((uint32_t)seq >= p.stages) {
            ok = false;
            return;
          }
          if (!mx_wait(&aux->empty[st], phase ^ 1u, aux)) {
            lin_fail(p, aux);
            ok = false;
            return;
          }
          mbar_arrive_expect_tx(&aux->full[st], bytes);
          load(ring + st * C::STAGE_BYTES, &aux->full[st]);
        }
        ++seq;
        if (++st == C::STAGES) {
          st = 0;
          phase ^= 1u;
        }
      };
      auto adapters = [&]() {
        if (!mx_wait(&aux->planned, 0, aux)) {
          lin_fail(p, aux);
          ok = false;
          return;
        }
        const int rp = p.rank_pad, pack = lora_pack(rp), per = lora_stages(rp);
        const uint32_t one = (uint32_t)lora_bytes(rp);
        const int count = aux->slots;
        for (int u = 0; u < count; u += pack) {
          const int here = min(pack, count - u);
          for (int j = 0; ok && j < per; ++j)
            step((uint32_t)p.a_rows * 128 + here * one, [&](uint8_t* s, uint64_t* bar) {
              tma_load_2d(s, &maps.t, bar, lora_col_t(rp, j), tm * kLinTile);
              for (int e = 0; e < here; ++e)
                tma_load_3d(s + C::B_OFF + e * one, &maps.up, bar, lora_col_b(rp, j),
                            tn * kLinTile, slots[u + e].id);
            });
        }
      };
      const uint32_t tx = (AMN ? (uint32_t)kLinOperand : (uint32_t)p.a_rows * 128) + kLinOperand;
      for (int i = kb0; ok && i < kb1; ++i) {
        if (LORA && plan && i == kx) {
          adapters();
          if (!ok) break;
        }
        step(tx, [&](uint8_t* s, uint64_t* bar) {
          const bool lo = p.terms == 2 && (i & 1);
          const int k0 = (p.terms == 2 ? i >> 1 : i) * kLinK;
          const CUtensorMap* ma = lo && !p.lo_b ? &maps.lo : &maps.a;
          const CUtensorMap* mb = lo && p.lo_b ? &maps.lo : &maps.b;
          if constexpr (AMN) {
            tma_load_2d(s, ma, bar, tm * kLinTile, k0);
            tma_load_2d(s + kLinBox, ma, bar, tm * kLinTile + 64, k0);
          } else {
            tma_load_2d(s, ma, bar, k0, tm * kLinTile);
          }
          if constexpr (G) {
            tma_load_2d(s + C::B_OFF, mb, bar, k0, tn * 64);
            tma_load_2d(s + C::B_OFF + kLinOperand / 2, mb, bar, k0, p.n + tn * 64);
          } else if constexpr (BMN) {
            tma_load_2d(s + C::B_OFF, mb, bar, tn * kLinTile, k0);
            tma_load_2d(s + C::B_OFF + kLinBox, mb, bar, tn * kLinTile + 64, k0);
          } else {
            tma_load_2d(s + C::B_OFF, mb, bar, k0, tn * kLinTile);
          }
        });
      }
      if (LORA && plan && ok && kx == kb1) adapters();
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      LinRing<C::STAGES> r = {aux, aux->full};
      const uint64_t a0 = lin_desc<AMN>(smem_u32(ring));
      const uint64_t b0 = lin_desc<BMN>(smem_u32(ring) + C::B_OFF);
      bool ok = true;
      auto adapters = [&]() {
        ok = mx_wait(&aux->planned, 0, aux);
        const int rp = p.rank_pad, pack = lora_pack(rp), per = lora_stages(rp);
        const int count = ok ? aux->slots : 0;
        for (int u = 0; u < count; u += pack) {
          const int here = min(pack, count - u);
          for (int j = 0; ok && j < per; ++j) {
            const int st = r.take();
            ok = st >= 0;
            if (!ok) break;
            const uint32_t s = smem_u32(ring + st * C::STAGE_BYTES);
            for (int e = 0; e < here; ++e) {
              const uint32_t off[4] = {slots[u + e].off[0], slots[u + e].off[1],
                                       slots[u + e].off[2], slots[u + e].off[3]};
              lora_stage_mmas<false>(tmem, s, s + C::B_OFF, p.idesc, rp, j, e, off);
            }
            umma_commit(&aux->empty[st]);
          }
        }
      };
      const int terms = p.terms, k = p.k;
      const uint32_t idesc = p.idesc;
      for (int i = kb0; i < kb1; ++i) {
        if (LORA && plan && i == kx) adapters();
        if (!ok) break;
        const int st = r.take();
        ok = st >= 0;
        if (!ok) break;
        const uint64_t at = (uint64_t)((st * C::STAGE_BYTES) >> 4);
        lin_stage_mmas<false, AMN, BMN>(tmem, a0 + at, b0 + at, idesc,
                                        k - (terms == 2 ? i >> 1 : i) * kLinK, i == kb0);
        umma_commit(&aux->empty[st]);
      }
      if (LORA && plan && ok && kx == kb1) adapters();
      if (!ok) lin_fail(p, aux);
      if (ok) umma_commit(&aux->tfull[0]);
      if (r.used > 0) {
        umma_commit(&aux->drain);
        mx_wait(&aux->drain, 0, aux, true);
      }
    }
    __syncwarp();
  } else {
    if (LORA && plan && warp == 2) {
      griddep_wait();
      if (lane == 0) griddep_launch_dependents();
      tile_plan(plan, tm & 1, p.split, rank, lane, slots, aux);
    }
    fine = mx_wait(&aux->tfull[0], 0, aux);
    if (!fine) lin_fail(p, aux);
    fine = epi_all(fine);
    tc_fence_after();
    // The ring is idle: every stage was read by MMAs that are complete.
    const int q = warp & 3;
    if (fine && tm * kLinTile + q * 32 < p.m)
      keep_rows(tmem, q, lane, reinterpret_cast<float*>(ring));
    __syncwarp();
  }
  tile_out<MODE, T>(p, reinterpret_cast<const float*>(ring), warp, lane, rank, tm, tn, fine);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kLinTile);
  }
  // Copies that no MMA waited for land before the CTA leaves.
  if (seq > 0 && mx_aborted(aux))
    for (int i = seq > C::STAGES ? seq - C::STAGES : 0; i < seq; ++i)
      if ((i & 1) == me)
        mx_wait(&aux->full[i % C::STAGES], (uint32_t)((i / C::STAGES) & 1), aux, true);
  __syncwarp();
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(&p.report->launches, 1u);
}

template <int MODE, int RING, bool AMN, bool BMN, typename T>
cudaError_t launch(const LinMaps& t, const LinParams& p, cudaStream_t stream) {
  using C = SingleCfg<RING>;
  auto kernel = lin_single_kernel<MODE, RING, AMN, BMN, T>;
  static std::atomic<uint64_t> done_mask{0};
  const cudaError_t e = opt_in_smem((const void*)kernel, done_mask, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t)p.tiles_m * p.tiles_n * p.split;
  return launch_pdl_cluster(kernel, dim3((unsigned)ctas), dim3(kLinThreads), C::SMEM, stream,
                            p.split, t, p);
}

template <int MODE, bool AMN, bool BMN, typename T>
cudaError_t launch_ring(const LinMaps& t, const LinParams& p, cudaStream_t stream) {
  if constexpr (!AMN && !BMN)
    if (p.m <= 16) return launch<MODE, kFew, AMN, BMN, T>(t, p, stream);
  return p.deep ? launch<MODE, kDeep, AMN, BMN, T>(t, p, stream)
                : launch<MODE, kFull, AMN, BMN, T>(t, p, stream);
}

template <typename T>
cudaError_t launch_type(const LinVariant& v, const LinMaps& t, const LinParams& p,
                        cudaStream_t stream) {
  if (v.mode == kLinGated) return launch_ring<kLinGated, false, false, T>(t, p, stream);
  if (v.mode == kLinGrad) return launch_ring<kLinGrad, false, true, T>(t, p, stream);
  if (v.a_mn) return launch_ring<kLinPlain, true, true, T>(t, p, stream);
  if (v.b_mn) return launch_ring<kLinPlain, false, true, T>(t, p, stream);
  return launch_ring<kLinPlain, false, false, T>(t, p, stream);
}

}  // namespace

cudaError_t launch_lin_single(const LinVariant& v, const LinMaps& t, const LinParams& p,
                              cudaStream_t stream) {
  if (v.out == SKG_OUT_F16) return launch_type<__half>(v, t, p, stream);
  return launch_type<__nv_bfloat16>(v, t, p, stream);
}

int lin_single_clusters(int size) {
  static std::atomic<int> cached[64][9];
  int dev = 0;
  if (size < 1 || size > 8 || cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int have = cached[dev][size].load(std::memory_order_acquire);
  if (have != 0) return have > 0 ? have : 0;
  auto kernel = lin_single_kernel<kLinGated, kDeep, false, false, __nv_bfloat16>;  // all alike
  const int n = clusters_resident((const void*)kernel, SingleCfg<kDeep>::SMEM, size);
  cached[dev][size].store(n > 0 ? n : -1, std::memory_order_release);
  return n;
}

}  // namespace skg
