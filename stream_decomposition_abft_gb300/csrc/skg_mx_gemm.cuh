// What the block-scaled product's kernels share: parameters, bounded waits, one
// stage's MMAs, and the way to C.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_internal.h"
#include "skg_mx.cuh"
#include "skgemm.h"

namespace skg {

constexpr int kMxThreads = 192;
constexpr int kMxTile = 128;
constexpr int kMxRowBytes = 128;              // k bytes of a stage row
constexpr int kMxOperand = kMxTile * kMxRowBytes;
constexpr uint64_t kMxTimeoutNs = 2000000000ull;  // bound of a wait

struct MxParams {
  int m, n, k;
  float alpha, beta;
  const float* ga;  // fp32 scales of the matrices (NULL = 1)
  const float* gb;
  void* c;
  int64_t ldc;
  int c_vec;        // four elements of a row are aligned together
  int c_tma;        // rows of C on 16-byte boundaries, beta = 0: pairs store it by TMA
  int ksteps;       // stages of k
  int groups;       // scale tiles along k
  int tiles_m, tiles_n;
  int split;        // single CTAs: CTAs per tile (cluster size)
  int direct;       // single CTAs: C is written from registers
  int a_rows;       // single CTAs: rows of A's box
  uint32_t stages;  // a CTA loads no more stages than this (see skg_mx_test_stall)
  uint64_t limit;   // bound of a wait, ns
  skg_report_t* report;
};

// What the formats ask of a stage of 128 bytes of k.
template <int FMT>
struct MxStage {
  static constexpr int STEP = kMxRowBytes * 8 / mx_bits(FMT);  // elements: 128 or 256
  static constexpr int MMA_K = FMT == SKG_MXFP8 ? 32 : 64;
  static constexpr int CHUNKS = STEP / mx_block(FMT) / 4;      // scale tiles of 128 rows: 1, 2, 4
  static constexpr int SF_BYTES = CHUNKS * kMxTileBytes;
};

struct MxAux {
  uint64_t full[8], empty[8], tfull[2], tempty, drain;
  uint64_t limit;
  uint32_t tmem_slot;
  int32_t abort_flag;
};

__device__ __forceinline__ bool mx_aborted(MxAux* aux) {
  return *(volatile int32_t*)&aux->abort_flag != 0;
}

__device__ __forceinline__ void mx_fail(const MxParams& p, MxAux* aux) {
  if (atomicExch(&aux->abort_flag, 1) == 0) {
    atomicOr(&p.report->status_bits, 1u << SKG_ERR_PIPELINE_TIMEOUT);
    atomicAdd(&p.report->timeouts, 1u);
  }
}

// Wait bounded by aux->limit; `drain` goes on after an abort, for as long as ever (the
// caller's own operations).
__device__ __forceinline__ bool mx_wait(uint64_t* bar, uint32_t parity, MxAux* aux,
                                        bool drain = false) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 31) == 0) {
      if (!drain && mx_aborted(aux)) return false;
      if (globaltimer() - t0 > (drain ? kMxTimeoutNs : aux->limit)) return false;
    }
  }
}

// Four consecutive elements of a row of C: aligned together and beta = 0, or
// (mx_write4_any, out of the way of the instruction cache: a launch runs each line of
// this once) whatever they are.
template <typename T>
__device__ __forceinline__ void mx_write4_plain(T* c, const float4& v, float alpha) {
  union {
    T e[4];
    uint4 q;
    uint2 d;
  } u;
  u.e[0] = mx_from_f32<T>(alpha * v.x);
  u.e[1] = mx_from_f32<T>(alpha * v.y);
  u.e[2] = mx_from_f32<T>(alpha * v.z);
  u.e[3] = mx_from_f32<T>(alpha * v.w);
  if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(c) = u.q;
  else *reinterpret_cast<uint2*>(c) = u.d;
}

template <typename T>
__device__ __noinline__ void mx_write4_any(T* c, float4 v, float alpha, float beta, int left,
                                           bool vec) {
  float o[4] = {alpha * v.x, alpha * v.y, alpha * v.z, alpha * v.w};
  if (vec && left >= 4) {
    union {
      T e[4];
      uint4 q;
      uint2 d;
    } u;
    if (beta != 0.f) {
      if constexpr (sizeof(T) == 4) u.q = *reinterpret_cast<const uint4*>(c);
      else u.d = *reinterpret_cast<const uint2*>(c);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += beta * mx_to_f32(u.e[i]);
    }
    mx_write4_plain<T>(c, make_float4(o[0], o[1], o[2], o[3]), 1.f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i < left) {
        if (beta != 0.f) o[i] += beta * mx_to_f32(c[i]);
        c[i] = mx_from_f32<T>(o[i]);
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void mx_write4(const MxParams& p, int row, int col, const float4& v,
                                          float alpha) {
  T* c = reinterpret_cast<T*>(p.c) + (int64_t)row * p.ldc + col;
  if (p.c_vec && p.beta == 0.f && col + 4 <= p.n) mx_write4_plain<T>(c, v, alpha);
  else mx_write4_any<T>(c, v, alpha, p.beta, p.n - col, p.c_vec != 0);
}

// The MMAs of one stage (A at its start, B at B_OFF): the scales go to TMEM columns sfa,
// sfb (B_TILES scale tiles of 128 rows of B), then up to four MMAs of 32 bytes of k each
// (32 elements of 8 bits, 64 of 4). MMAs wholly past k are left out: their scales need
// not exist. The last one of 4 bits may reach past k's last block of 32: it takes zero
// codes there, with scales that the storage rules have be zero.
template <int FMT, bool PAIR, int B_TILES, int B_OFF>
__device__ __forceinline__ void mx_stage_mmas(uint32_t d, uint32_t sfa, uint32_t sfb,
                                              uint32_t stage, uint32_t sfa_off, uint32_t sfb_off,
                                              int left, bool first) {
  using S = MxStage<FMT>;
#pragma unroll
  for (int c = 0; c < S::CHUNKS; ++c) {
    tmem_cp_scales<PAIR>(sfa + c * 4, sdesc_scales(stage + sfa_off + c * kMxTileBytes));
#pragma unroll
    for (int h = 0; h < B_TILES; ++h)
      tmem_cp_scales<PAIR>(sfb + (c * B_TILES + h) * 4,
                           sdesc_scales(stage + sfb_off + h * S::SF_BYTES + c * kMxTileBytes));
  }
  const uint64_t ad = sdesc_sw128(stage), bd = sdesc_sw128(stage + B_OFF);
  const int mmas = min(4, (left + S::MMA_K - 1) / S::MMA_K);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j >= mmas) break;
    // mxfp8: byte j of the stage's one scale word; mxfp4: half j & 1 of word
    // j / 2; nvfp4: the whole word j.
    constexpr uint32_t F = FMT == SKG_MXFP8 ? 0u : 1u;
    constexpr uint32_t E8 = FMT == SKG_NVFP4 ? 0u : 1u;
    const uint32_t byte = FMT == SKG_MXFP8 ? j : (FMT == SKG_MXFP4 ? (j & 1) * 2 : 0);
    const int word = FMT == SKG_MXFP8 ? 0 : (FMT == SKG_MXFP4 ? j / 2 : j);
    umma_scaled<FMT, PAIR>(d, ad + j * 2, bd + j * 2,
                           idesc_scaled(F, E8, PAIR ? 2 * kMxTile : kMxTile, B_TILES * kMxTile,
                                        byte),
                           sfa + word * 4, sfb + word * B_TILES * 4, (!first || j > 0) ? 1u : 0u);
  }
}

// 256 x 256 tiles on clusters of two CTAs (skg_mx_gemm_pair.cu); t: the maps of
// A, B, their scales and (p.c_tma) C. `clusters` CTA pairs.
template <int FMT>
cudaError_t launch_mx_pair(const CUtensorMap (&t)[5], const MxParams& p, int out, int clusters,
                           cudaStream_t stream);

// CTA pairs of its kernel that can be resident on the current device at once.
int mx_pair_clusters_resident();

}  // namespace skg
