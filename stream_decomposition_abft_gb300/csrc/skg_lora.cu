// The down-projection of low-rank adapters: t_i = scale_s (x_i A_s^T), s = index[i], for
// rows of any mixture of adapters, and the plans that the product behind it reads.
//
// A cluster takes 128 rows of x and finds the distinct adapters in them (the plan: one pass
// of comparisons over 256 indices). With ranks up to 128 it works on `per` adapters at once,
// at most as many as fit 128 columns of the accumulator (8 of rank 16): a stage is 64 of k
// of the rows and of those adapters' A, one MMA forms every row's product with every one of
// them, and on the way out each row takes the columns of its own. Infinities and NaN in other
// adapters stay in columns that nothing reads. More adapters than that take more passes over
// x (in L2), which `groups` clusters share; larger ranks take a pass for each 128 columns.
// Few rows or few adapters make small stages, and the ring holds up to 16 of them.
//
// The CTAs of a cluster split k; their partial sums are added in rank order through
// distributed shared memory (no atomics, the same result every time). t is stored as the sum
// of two numbers of x's type, so that the product with B_s loses nothing to its rounding.
//
// What bounds it: for prompts x, once from HBM (2048 x 8192, three adapters of rank 64: 23 us
// alone; the product behind it takes 163, and 8192 x 8192 x 8192 with eight adapters in
// segments 609 us against 600 without); for a decode batch latency, much of which passes while
// the product streams W, for which it waits only where it needs t (64 x 8192 x 8192, 64
// adapters of rank 16: 37.8 us against 25.8 without any; their 34 MB alone are 5).
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_lin.cuh"

namespace skg {
namespace {

constexpr int kPitch = kLinPitch;
constexpr int kRing = 6 * kLinOperand;  // two CTAs share an SM
constexpr int kMaxStages = 16;

// The adapters of a tile's rows, and those of the 256 rows that the plan in global memory
// covers.
struct Plan {
  int32_t ids[kLinTile];   // adapter of each row, -1: none
  int32_t slot[kLinTile];  // number of that adapter
  int32_t id[kLinTile];    // adapters by number, in the order of their first rows
  float scale[kLinTile];
  uint32_t lead[4];        // rows that are their adapter's first
  int32_t ids2[kLoraRows], slot2[kLoraRows];
  uint32_t lead2[8];
};

struct LoraAux : LinAux {  // with barriers of its own for the ring
  uint64_t ring_full[kMaxStages], ring_empty[kMaxStages];
};

constexpr uint32_t kSmem = 1024 + kRing + 512 + sizeof(Plan);
static_assert(sizeof(LoraAux) <= 512, "aux size");
static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs per SM");
static_assert(kLinTile * kPitch * 4 <= kRing, "the partial sums fit the ring");

__device__ __forceinline__ void fail(const LoraParams& p, LoraAux* aux) {
  if (atomicExch(&aux->abort_flag, 1) == 0) {
    atomicOr(&p.report->status_bits, 1u << SKG_ERR_PIPELINE_TIMEOUT);
    atomicAdd(&p.report->timeouts, 1u);
  }
}

template <typename T>
__global__ void __launch_bounds__(kLinThreads, 2)
lora_down_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                 const LoraParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  LoraAux* aux = reinterpret_cast<LoraAux*>(ring + kRing);
  Plan* pl = reinterpret_cast<Plan*>(ring + kRing + 512);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int unit = (int)blockIdx.x / p.split;
  const int tm = unit / p.groups, group = unit % p.groups;
  const int kb0 = (int)((int64_t)p.ksteps * rank / p.split);
  const int kb1 = (int)((int64_t)p.ksteps * (rank + 1) / p.split);

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmX);
    prefetch_tmap(&tmA);
    aux->abort_flag = 0;
    aux->limit = p.limit;
    for (int i = 0; i < p.ring_stages; ++i) {
      mbar_init(&aux->ring_full[i], 1);
      mbar_init(&aux->ring_empty[i], 1);
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
  // The product behind reads x and writes y before it waits for this kernel: that is safe
  // once all that ran before is complete, as it is now. (Its loads of W queue with these; to
  // let it start behind the last of these instead took 1 to 3 us more in all.)
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();

  const int rp = p.rank_pad, cols = min(rp, 128), chunks = (rp + 127) / 128;
  const int per = p.per, stages = p.ring_stages;
  int seq = 0, it = 0, n = 0;
  int load_st = 0, mma_st = 0, early = 0;
  uint32_t load_phase = 0, mma_phase = 0;
  bool load_ok = true, mma_ok = true, ready = false;
  const uint64_t a0 = lin_desc<false>(smem_u32(ring));
  const uint64_t b0 = lin_desc<false>(smem_u32(ring) + p.a_rows * 128);
  const bool loader = warp == 0 || warp == kLinLoader;
  const int me = warp == kLinLoader;  // a loading thread takes every other stage
  // The first pass's x is under way while the plan is made.
  if (loader && elect_one()) {
    early = min(min(stages, kb1 - kb0), (int)min(p.stages, (uint32_t)kMaxStages));
    for (int i = me; i < early; i += 2) {
      mbar_expect_tx(&aux->ring_full[i], (uint32_t)p.a_rows * 128);
      tma_load_2d(ring + i * p.stage_bytes, &tmX, &aux->ring_full[i], (kb0 + i) * kLinK,
                  tm * kLinTile);
    }
  }
  __syncwarp();
  const int rows = min(kLinTile, p.m - tm * kLinTile);
  const int count = number_adapters<kLinThreads>(
      p.index, p.count, tm * kLinTile, rows, (int)threadIdx.x, pl->ids, pl->slot, pl->lead,
      [&](int s, int id) {
        pl->id[s] = id;
        pl->scale[s] = p.scale ? p.scale[id] : 1.f;
      },
      [](int, int, uint32_t) {});
  // Passes: `per` adapters each, or (rank over 128) one adapter's next 128 columns.
  const int passes = chunks > 1 ? count * chunks : (count + per - 1) / per;

  // The plan for the product, by the warps that wait for the accumulator anyway.
  if (warp >= 2 && !loader && group == 0 && rank == 0 && (tm & 1) == 0) {
    LoraPlan* out = p.plan + (tm >> 1);
    const int tid = (int)threadIdx.x - 64;
    const int both = min(kLoraRows, p.m - tm * kLinTile);
    for (int i = tid; i < (both + 31) / 32 * 32 * 2; i += 128)
      reinterpret_cast<uint4*>(&out->rows[0][0])[i] = make_uint4(0, 0, 0, 0);
    const int c = number_adapters<128>(
        p.index, p.count, tm * kLinTile, both, tid, pl->ids2, pl->slot2, pl->lead2,
        [&](int s, int id) { out->id[s] = id; },
        [&](int s, int w, uint32_t m) { out->rows[s][w] = m; });
    if (tid == 0) out->count = c;
  }

  for (int pass = group; pass < passes; pass += p.groups, ++n) {
    const int first = chunks > 1 ? pass / chunks : pass * per;
    const int chunk = chunks > 1 ? pass % chunks : 0;
    const int here = chunks > 1 ? 1 : min(per, count - first);
    bool fine = true;
    if (loader) {
      if (elect_one()) {
        int id[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) id[j] = j < here ? pl->id[first + j] : 0;
        for (int kb = kb0; load_ok && kb < kb1; ++kb) {
          if ((seq & 1) == me) {
            if ((uint32_t)seq >= p.stages) {
              load_ok = false;
              break;
            }
            uint64_t* bar = &aux->ring_full[load_st];
            if (!mx_wait(&aux->ring_empty[load_st], load_phase ^ 1u, aux)) {
              fail(p, aux);
              load_ok = false;
              break;
            }
            uint8_t* s = ring + load_st * p.stage_bytes;
            const uint32_t a_bytes = seq < early ? 0 : (uint32_t)p.a_rows * 128;
            mbar_arrive_expect_tx(bar, a_bytes + (uint32_t)(here * cols) * 128);
            if (a_bytes) tma_load_2d(s, &tmX, bar, kb * kLinK, tm * kLinTile);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j < here)
                tma_load_3d(s + (p.a_rows + j * cols) * 128, &tmA, bar, kb * kLinK, chunk * 128,
                            id[j]);
          }
          ++seq;
          if (++load_st == stages) {
            load_st = 0;
            load_phase ^= 1u;
          }
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (elect_one()) {
        for (int kb = kb0; mma_ok && kb < kb1; ++kb) {
          const int st = mma_st;
          if (!ready && !mx_wait(&aux->ring_full[st], mma_phase, aux)) {
            fail(p, aux);
            mma_ok = false;
            break;
          }
          tc_fence_after();
          if (++mma_st == stages) {
            mma_st = 0;
            mma_phase ^= 1u;
          }
          ready = mbar_test_wait(&aux->ring_full[mma_st], mma_phase);  // (as LinRing does)
          const uint64_t at = (uint64_t)((st * p.stage_bytes) >> 4);
          lin_stage_mmas<false, false, false>(tmem, a0 + at, b0 + at, p.idesc, p.k - kb * kLinK,
                                              kb == kb0);
          umma_commit(&aux->ring_empty[st]);
          ++it;
        }
        if (mma_ok) umma_commit(&aux->tfull[0]);
      }
      __syncwarp();
    } else {  // warps 2-5
      fine = mx_wait(&aux->tfull[0], (uint32_t)n & 1u, aux);
      if (!fine) fail(p, aux);
      fine = epi_all(fine);
      tc_fence_after();
      const int q = warp & 3, r = q * 32 + lane;
      float* part = reinterpret_cast<float*>(ring);
      if (fine && q * 32 < rows) {
        // The ring is idle: every stage was read by MMAs that are complete.
#pragma unroll
        for (int c = 0; c < kLinTile; c += 32) {
          if (c >= here * cols) break;
          uint32_t v[32];
          tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c, v);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(part + r * kPitch + c + i) =
                make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      }
      __syncwarp();
      tc_fence_before();
    }
    if (p.split > 1) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (!mx_aborted(aux)) {
      const int quads = min(cols, rp - chunk * 128) / 4;
      const float* part = reinterpret_cast<const float*>(ring);
      const int mine = rank < rows ? (rows - rank + p.split - 1) / p.split : 0;
      for (int i = threadIdx.x; i < mine * quads; i += kLinThreads) {
        const int r = rank + (i / quads) * p.split, c = (i % quads) * 4;
        if (pl->ids[r] < 0) continue;
        const int at = pl->slot[r] - first;
        if (at < 0 || at >= here) continue;
        const float* src = part + r * kPitch + at * cols + c;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        float4 u[8];  // the loads in flight together
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < p.split)
            u[s] = p.split > 1 ? ld_shared_cluster_f32x4(cluster_addr(src, (uint32_t)s))
                               : *reinterpret_cast<const float4*>(src);
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < p.split) {
            v[0] += u[s].x;
            v[1] += u[s].y;
            v[2] += u[s].z;
            v[3] += u[s].w;
          }
        const float f = pl->scale[pl->slot[r]];
        const int col = chunk * 128 + c;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = col + e < p.rank ? f * v[e] : 0.f;
        T* t = reinterpret_cast<T*>(p.t) + (int64_t)(tm * kLinTile + r) * 2 * rp + col;
        store_parts<T>(t, t + rp, v);
      }
    }
    // The ring is written by the next pass's copies, and no CTA leaves while another reads
    // its partial sums (loads whose values are used by now).
    fence_proxy_async_smem();
    __syncwarp();
    if (p.split > 1) cluster_meet();
    else __syncthreads();
  }
  if (warp == 1 && elect_one() && it > 0) {
    umma_commit(&aux->drain);
    mx_wait(&aux->drain, 0, aux, true);
  }
  __syncwarp();
  // Copies land before the CTA leaves: those of x for rows without any adapter (or stages not
  // come to), whose barriers still lack the arrival, and those that no MMA waited for.
  for (int i = 0; i < early; ++i)
    if ((i & 1) == me && i >= seq) {
      mbar_arrive(&aux->ring_full[i]);
      mx_wait(&aux->ring_full[i], 0, aux, true);
    }
  if (seq > 0 && mx_aborted(aux))
    for (int i = seq > stages ? seq - stages : 0; i < seq; ++i)
      if ((i & 1) == me)
        mx_wait(&aux->ring_full[i % stages], (uint32_t)((i / stages) & 1), aux, true);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kLinTile);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(&p.report->launches, 1u);
}

template <typename T>
cudaError_t launch(const CUtensorMap& x, const CUtensorMap& down, LoraParams p,
                   cudaStream_t stream) {
  const int cols = p.rank_pad < 128 ? p.rank_pad : 128;
  p.stage_bytes = (p.a_rows + p.per * cols) * 128;
  // An MMA reads 128 rows from a stage's start, so as many end inside the ring.
  const int last = p.stage_bytes > kLinOperand ? p.stage_bytes : kLinOperand;
  const int fit = (kRing - last) / p.stage_bytes + 1;
  p.ring_stages = fit < kMaxStages ? fit : kMaxStages;
  static std::atomic<uint64_t> done_mask{0};
  const cudaError_t e = opt_in_smem((const void*)lora_down_kernel<T>, done_mask, (int)kSmem);
  if (e != cudaSuccess) return e;
  const int tiles = (p.m + kLinTile - 1) / kLinTile;
  return launch_pdl_cluster(lora_down_kernel<T>, dim3((unsigned)(tiles * p.groups * p.split)),
                            dim3(kLinThreads), kSmem, stream, p.split, x, down, p);
}

}  // namespace

cudaError_t launch_lora_down(int dtype, const CUtensorMap& x, const CUtensorMap& down,
                             const LoraParams& p, cudaStream_t stream) {
  return dtype == SKG_IN_F16 ? launch<__half>(x, down, p, stream)
                             : launch<__nv_bfloat16>(x, down, p, stream);
}

}  // namespace skg
