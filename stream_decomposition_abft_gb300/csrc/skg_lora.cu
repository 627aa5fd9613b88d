// The down-projection of low-rank adapters: t_i = scale_s (x_i A_s^T), s = index[i], for
// rows of any mixture of adapters, and the plans that the product behind it reads.
//
// A cluster takes 128 rows of x and finds the distinct adapters in them (the plan: one pass
// of comparisons over 256 indices). With ranks up to 128 it works on as many adapters at
// once as fit 128 columns of the accumulator (8 of rank 16): a stage is 64 of k of the rows
// and of those adapters' A, one MMA forms every row's product with every one of them, and on
// the way out each row takes the columns of its own. Infinities and NaN in other adapters
// stay in columns that nothing reads. More adapters than that take more passes over x (in
// L2), which `groups` clusters share; larger ranks take a pass for each 128 columns.
//
// The CTAs of a cluster split k; their partial sums are added in rank order through
// distributed shared memory (no atomics, the same result every time). t is stored as the sum
// of two numbers of x's type, so that the product with B_s loses nothing to its rounding.
//
// What bounds it: x once from HBM for prompts (8192 x 8192: 134 MB, 20 us, under the product
// behind it, which takes 20 times as long); a few microseconds of latency for a decode
// batch, which pass while the product streams W (it waits for t only where it needs it).
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_lin.cuh"

namespace skg {
namespace {

constexpr int kPitch = 132;  // floats per row of the partial sums
constexpr int kStages = 3;   // two CTAs share an SM
constexpr int kStageBytes = 2 * kLinOperand;

struct Plan {
  int32_t ids[kLoraRows];   // adapter of each row, -1: none
  int32_t slot[kLoraRows];  // number of that adapter in the plan
  int32_t id[kLoraRows];    // adapters by number
  uint32_t rows[kLoraRows][8];
  int32_t list[kLinTile];   // the adapters (numbers) of this tile's 128 rows
  int32_t place[kLoraRows]; // number -> place in list
  uint32_t lead[8];
  int32_t count, tile_count;
};

constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + 256 + sizeof(Plan);
static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs per SM");
static_assert(kLinTile * kPitch * 4 <= kStages * kStageBytes, "the partial sums fit the ring");

// All threads. Rows row0, ... of the index; `half`: the 128 of them that are this tile's.
__device__ void make_plan(const LoraParams& p, Plan* pl, int row0, int half) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kLoraRows; i += kLinThreads) {
    const int id = row0 + i < p.m ? p.index[row0 + i] : -1;
    pl->ids[i] = id >= 0 && id < p.count ? id : -1;
  }
  for (int i = threadIdx.x; i < kLoraRows * 8; i += kLinThreads) (&pl->rows[0][0])[i] = 0;
  __syncthreads();
  // The first row of each row's adapter, first within its 32 rows, then before them.
  for (int g = warp; g < 8; g += kLinThreads / 32) {
    const int i = g * 32 + lane, id = pl->ids[i];
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    int first = g * 32 + __ffs(same) - 1;
    if (__any_sync(0xffffffffu, id >= 0)) {
      for (int j = g * 32 - 4; j >= 0; j -= 4) {
        const int4 o = *reinterpret_cast<const int4*>(&pl->ids[j]);
        first = o.w == id ? j + 3 : first;
        first = o.z == id ? j + 2 : first;
        first = o.y == id ? j + 1 : first;
        first = o.x == id ? j : first;
      }
    }
    pl->slot[i] = first;  // a row's number, until all are known
    const uint32_t lead = __ballot_sync(0xffffffffu, id >= 0 && first == i);
    if (lane == 0) pl->lead[g] = lead;
  }
  __syncthreads();
  for (int g = warp; g < 8; g += kLinThreads / 32) {
    const int i = g * 32 + lane, id = pl->ids[i], first = pl->slot[i];
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    int s = 0;
    for (int w = 0; w < 8; ++w) {
      const uint32_t below = w < (first >> 5) ? ~0u : (w == (first >> 5) ? (1u << (first & 31)) - 1 : 0u);
      s += __popc(pl->lead[w] & below);
    }
    __syncwarp();
    if (id >= 0) {
      pl->slot[i] = s;
      if (first == i) pl->id[s] = id;
      if (lane == __ffs(same) - 1) pl->rows[s][g] = same;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int count = 0, mine = 0;
    for (int w = 0; w < 8; ++w) count += __popc(pl->lead[w]);
    for (int s = lane; s < (count + 31) / 32 * 32; s += 32) {
      bool here = false;
      if (s < count)
        for (int w = 0; w < 4; ++w) here |= pl->rows[s][half * 4 + w] != 0;
      const uint32_t b = __ballot_sync(0xffffffffu, here);
      if (here) {
        const int at = mine + __popc(b & ((1u << lane) - 1));
        pl->list[at] = s;
        pl->place[s] = at;
      }
      mine += __popc(b);
    }
    if (lane == 0) {
      pl->count = count;
      pl->tile_count = mine;
    }
  }
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ void store_parts(T* hi, T* lo, const float (&v)[4]) {
  union {
    T e[4];
    uint2 d;
  } h, l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h.e[i] = mx_from_f32<T>(v[i]);
    const float r = v[i] - mx_to_f32(h.e[i]);
    l.e[i] = mx_from_f32<T>(isfinite(r) ? r : 0.f);  // an infinite or NaN t is in the high part
  }
  *reinterpret_cast<uint2*>(hi) = h.d;
  *reinterpret_cast<uint2*>(lo) = l.d;
}

template <typename T>
__global__ void __launch_bounds__(kLinThreads, 2)
lora_down_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                 const LoraParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  LinAux* aux = reinterpret_cast<LinAux*>(ring + kStages * kStageBytes);
  Plan* pl = reinterpret_cast<Plan*>(ring + kStages * kStageBytes + 256);
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
  // The product behind reads x and writes y before it waits for this kernel, so it may
  // start only when all that ran before is complete.
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  make_plan(p, pl, (tm >> 1) * kLoraRows, tm & 1);

  if (group == 0 && rank == 0 && (tm & 1) == 0) {
    LoraPlan* out = p.plan + (tm >> 1);
    const int count = pl->count;
    if (threadIdx.x == 0) out->count = count;
    for (int i = threadIdx.x; i < count; i += kLinThreads) out->id[i] = pl->id[i];
    for (int i = threadIdx.x; i < count * 8; i += kLinThreads)
      (&out->rows[0][0])[i] = (&pl->rows[0][0])[i];
  }

  // Passes: `per` adapters each, or (rank over 128) one adapter's next 128 columns.
  const int rp = p.rank_pad, cols = min(rp, 128), chunks = (rp + 127) / 128;
  const int per = 128 / cols;
  const int passes = chunks > 1 ? pl->tile_count * chunks : (pl->tile_count + per - 1) / per;
  const int rows = min(kLinTile, p.m - tm * kLinTile);
  int issued = 0, it = 0, n = 0;
  bool load_ok = true, mma_ok = true;
  for (int pass = group; pass < passes; pass += p.groups, ++n) {
    const int first = chunks > 1 ? pass / chunks : pass * per;
    const int chunk = chunks > 1 ? pass % chunks : 0;
    const int here = chunks > 1 ? 1 : min(per, pl->tile_count - first);
    bool fine = true;
    if (warp == 0) {
      if (elect_one()) {
        for (int kb = kb0; load_ok && kb < kb1; ++kb) {
          const int st = issued % kStages;
          if ((uint32_t)issued >= p.stages) {
            load_ok = false;
            break;
          }
          if (!mx_wait(&aux->empty[st], (uint32_t)((issued / kStages) & 1) ^ 1u, aux)) {
            if (atomicExch(&aux->abort_flag, 1) == 0) {
              atomicOr(&p.report->status_bits, 1u << SKG_ERR_PIPELINE_TIMEOUT);
              atomicAdd(&p.report->timeouts, 1u);
            }
            load_ok = false;
            break;
          }
          uint8_t* s = ring + st * kStageBytes;
          mbar_arrive_expect_tx(&aux->full[st], (uint32_t)(p.a_rows + here * cols) * 128);
          tma_load_2d(s, &tmX, &aux->full[st], kb * kLinK, tm * kLinTile);
          for (int j = 0; j < here; ++j)
            tma_load_3d(s + kLinOperand + j * cols * 128, &tmA, &aux->full[st], kb * kLinK,
                        chunk * 128, pl->id[pl->list[first + j]]);
          ++issued;
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (elect_one()) {
        for (int kb = kb0; mma_ok && kb < kb1; ++kb) {
          const int st = it % kStages;
          if (!mx_wait(&aux->full[st], (uint32_t)((it / kStages) & 1), aux)) {
            if (atomicExch(&aux->abort_flag, 1) == 0) {
              atomicOr(&p.report->status_bits, 1u << SKG_ERR_PIPELINE_TIMEOUT);
              atomicAdd(&p.report->timeouts, 1u);
            }
            mma_ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t s = smem_u32(ring + st * kStageBytes);
          lin_stage_mmas<false, false, false>(tmem, s, s + kLinOperand, p.idesc,
                                              p.k - kb * kLinK, kb == kb0);
          umma_commit(&aux->empty[st]);
          ++it;
        }
        if (mma_ok) umma_commit(&aux->tfull[0]);
      }
      __syncwarp();
    } else {
      fine = mx_wait(&aux->tfull[0], (uint32_t)n & 1u, aux);
      if (!fine && atomicExch(&aux->abort_flag, 1) == 0) {
        atomicOr(&p.report->status_bits, 1u << SKG_ERR_PIPELINE_TIMEOUT);
        atomicAdd(&p.report->timeouts, 1u);
      }
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
        const int row = (tm & 1) * kLinTile + r;
        const int id = pl->ids[row];
        if (id < 0) continue;
        const int at = pl->place[pl->slot[row]] - first;
        if (at < 0 || at >= here) continue;
        const float* src = part + r * kPitch + at * cols + c;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int s = 0; s < p.split; ++s) {
          const float4 u = p.split > 1 ? ld_shared_cluster_f32x4(cluster_addr(src, (uint32_t)s))
                                       : *reinterpret_cast<const float4*>(src);
          v[0] += u.x;
          v[1] += u.y;
          v[2] += u.z;
          v[3] += u.w;
        }
        const float f = p.scale ? p.scale[id] : 1.f;
        const int col = chunk * 128 + c;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = col + e < p.rank ? f * v[e] : 0.f;
        T* t = reinterpret_cast<T*>(p.t) + (int64_t)(tm * kLinTile + r) * 2 * rp + col;
        store_parts<T>(t, t + rp, v);
      }
    }
    // The ring is written by the next pass's copies, and no CTA leaves while another reads
    // its partial sums.
    fence_proxy_async_smem();
    if (p.split > 1) cluster_sync();
    else __syncthreads();
  }
  if (warp == 1 && elect_one() && it > 0) {
    umma_commit(&aux->drain);
    mx_wait(&aux->drain, 0, aux, true);
  }
  __syncwarp();
  if (warp == 0 && issued > 0 && mx_aborted(aux))  // elected lane alone has issued > 0
    for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
      mx_wait(&aux->full[i % kStages], (uint32_t)((i / kStages) & 1), aux, true);
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
cudaError_t launch(const CUtensorMap& x, const CUtensorMap& down, const LoraParams& p,
                   cudaStream_t stream) {
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
