// What the kernels of a layer's projections share: parameters, bounded waits, the
// activations, one stage's MMAs and the plan of the low-rank adapters.
//
// All of them form sums over k of A[i][l] B[j][l] in 16 bits with fp32 accumulation on
// tcgen05 (kind::f16), 64 elements of k (128 bytes of a K-major row) to a stage:
//
//   skg_lin_single.cu  128 x 128 tiles on single CTAs, k split over a cluster where the
//                      tiles are few
//   skg_lin_adapted.cu such tiles with few low-rank adapters in the same launch
//   skg_lin_group.cu   such tiles of up to three products in one launch
//   skg_lin_pair.cu    256 x 256 tiles on CTA pairs
//
// (skg_lora.cu forms what the others take as the adapters' operand,) with these ways out (LinMode):
//   kLinPlain   C = A B^T, and with adapters + scale_s (x A_s^T) B_s^T per row
//   kLinGated   B holds two projections of n rows each; a tile takes half of its columns
//               from either, so one thread holds gate and up of an output:
//               H = act(gate) * up, and PRE = (gate | up) where it is asked for
//   kLinGrad    the product is the gradient of a gated output (N-major B): with PRE,
//               DPRE = the gradients of gate and up, and H formed again
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "skg_internal.h"
#include "skg_mx.cuh"
#include "skg_mx_gemm.cuh"
#include "skgemm.h"

namespace skg {

// Warps 0 and 6 load (issuing a stage takes a thread some 300 cycles, more than the 256 of its
// MMAs on a single CTA: they take every other stage), warp 1 issues the MMAs, warps 2-5
// take the accumulators out.
constexpr int kLinThreads = 224;
constexpr int kLinLoader = 6;
constexpr int kLinTile = 128;
constexpr int kLinK = 64;                      // elements of k in a stage
constexpr int kLinOperand = kLinTile * 128;    // bytes of an operand's 128 rows in a stage
constexpr int kLinPitch = 132;                 // floats per row of a partial tile
constexpr int kLinBox = 64 * 128;              // bytes of an MN-major box: 64 k x 64 elements
constexpr int kLoraRows = 256;                 // rows that one adapter plan covers

// An allocation of TMEM waits while other CTAs of the SM hold too much of it, and CTAs of a
// cluster wait for one another: two clusters that each held what the other wants would never
// end. It cannot come to that: every kernel here (and the block-scaled product's) takes more
// than a third of an SM's shared memory, so two CTAs at most share one, with 256 of the 512
// columns each at most; the pairs, with all columns, take all of the shared memory.
enum LinMode { kLinPlain = 0, kLinGated = 1, kLinGrad = 2 };

// The adapters that 256 rows use, in the order of their first rows, and the rows of each
// (word w, bit b: row 32 w + b).
struct LoraPlan {
  int32_t count;
  int32_t pad[3];
  int32_t id[kLoraRows];
  uint32_t rows[kLoraRows][8];
};

// Pairs, M-major A and N-major B: a second product of the same k in the same launch (its
// tiles behind the first one's; tiles_m = 0: none).
struct LinSecond {
  int m, n, tiles_m, tiles_n, lo_b;
  void* c;
  int64_t ldc;
};

struct LinParams {
  int m, n, k;        // rows and columns of the result (of one projection), length of the sums
  int ksteps;         // stages of k
  int terms;          // 2: one operand is a sum of two (high and low parts): each stage of k runs
                      // once with either
  int lo_b;           // that operand is B, not A
  int tiles_m, tiles_n;
  int split;          // single CTAs: CTAs per tile (cluster size)
  int deep;           // single CTAs: one per SM, with a ring of twice the stages
  int a_rows;         // single CTAs, K-major A: rows of A's box
  uint32_t idesc;
  int act;            // kLinGated, kLinGrad
  void* c;
  int64_t ldc;
  void* pre;          // kLinGated: PRE or NULL; kLinGrad: DPRE
  int64_t ldp;
  const void* pre_in; // kLinGrad: PRE
  int64_t ldp_in;
  void* c_lo;         // kLinGrad: low parts of H and DPRE, or NULL
  void* pre_lo;
  LinSecond second;
  const LoraPlan* plan;  // adapters: one per 256 rows, or NULL
  int rank_pad;          // their rank, rounded up to 16
  uint32_t stages;    // a CTA loads no more stages than this (skg_layers_test_stall)
  uint64_t limit;     // bound of a wait, ns
  skg_report_t* report;
};

// The tensor maps of one launch. Unused ones repeat a.
struct LinMaps {
  CUtensorMap a, b;
  CUtensorMap lo;         // the two-term operand's low parts
  CUtensorMap t, up;      // adapters: scale (x A^T) in high and low parts; their B (3 dimensions)
  CUtensorMap c, gate, pre_up;  // pairs: stores (C or H, the halves of PRE or DPRE);
                                // kLinGrad: t and up are the halves of PRE
  // A second product's a, b, lo and c are t, up, gate and pre_up.
};

struct LinAux : MxAux {
  uint64_t tempty1;
};

__device__ __forceinline__ void lin_fail(const LinParams& p, LinAux* aux) {
  if (atomicExch(&aux->abort_flag, 1) == 0) {
    atomicOr(&p.report->status_bits, 1u << SKG_ERR_PIPELINE_TIMEOUT);
    atomicAdd(&p.report->timeouts, 1u);
  }
}

// ------------------------------------------------------------------ activations
// act(g), and its derivative in d. Relative errors of a few 2^-23, and of 1.2 |x| 2^-23 for an
// exponential e^x that counts: below a 16-bit result's rounding by a hundred times wherever
// that is a normal number.
__device__ __forceinline__ float lin_sigmoid(float x) {
  // (1 / (1 + e^-x) itself would be 0 for all x below -87.3: __fdividef by more than 2^126.)
  const float e = __expf(-fabsf(x)), p = __fdividef(1.f, 1.f + e);
  return x >= 0.f ? p : e * p;
}

// erfc(|x|) = e^-z^2 t Q(t) with z = |x|, t = 1 / (1 + z / 2): Q is the polynomial of degree 8
// with the least relative error for z in [0, 10] (4.3e-8; Remez's exchange on values in 40
// digits), 9e-7 as evaluated here, besides the exponential's error. Half of the instructions
// of the library's function.
__device__ __forceinline__ float lin_erfc(float x) {
  const float z = fabsf(x), t = __fdividef(1.f, fmaf(0.5f, z, 1.f));
  float q = -0.059064567f;
  q = fmaf(q, t, 0.2845551f);
  q = fmaf(q, t, -0.48716226f);
  q = fmaf(q, t, 0.2780283f);
  q = fmaf(q, t, -0.026601857f);
  q = fmaf(q, t, 0.20267805f);
  q = fmaf(q, t, 0.24310568f);
  q = fmaf(q, t, 0.2823751f);
  q = fmaf(q, t, 0.28208643f);
  const float r = q * t * __expf(-z * z);
  return x >= 0.f ? r : 2.f - r;
}

template <int ACT, bool GRAD>
__device__ __forceinline__ float lin_act(float g, float& d) {
  if constexpr (ACT == SKG_ACT_SILU) {
    const float p = lin_sigmoid(g);
    if (GRAD) d = p * (1.f + g * (1.f - p));
    return g * p;
  } else if constexpr (ACT == SKG_ACT_GELU) {
    const float p = 0.5f * lin_erfc(-0.70710678f * g);  // (1 + erf cancels for g < 0)
    if (GRAD) d = p + g * (0.39894228f * __expf(-0.5f * g * g));
    return g * p;
  } else if constexpr (ACT == SKG_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = sigmoid(2 u)
    const float p = lin_sigmoid(1.59576912f * (g + 0.044715f * g * g * g));
    const float q = p * (1.f - p);
    if (GRAD) d = q == 0.f ? p : p + g * q * (1.59576912f * (1.f + 0.134145f * g * g));
    return g * p;
  } else {
    if (GRAD) d = g > 0.f ? 1.f : (g == g ? 0.f : g);
    return g > 0.f ? g : (g == g ? 0.f : g);
  }
}

// f(the activation as a constant): one copy of f's code for each, of which a launch runs one.
// (With the choice inside, at every element, the way out of a tile took 1.5 us longer, most
// of it waiting for instructions.)
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == SKG_ACT_SILU) f(std::integral_constant<int, SKG_ACT_SILU>{});
  else if (act == SKG_ACT_GELU) f(std::integral_constant<int, SKG_ACT_GELU>{});
  else if (act == SKG_ACT_GELU_TANH) f(std::integral_constant<int, SKG_ACT_GELU_TANH>{});
  else f(std::integral_constant<int, SKG_ACT_RELU>{});
}

template <int ACT>
__device__ __forceinline__ float lin_gated(float gate, float up) {
  float d;
  return lin_act<ACT, false>(gate, d) * up;
}

// The gradients of a gated output h = act(g) u: of g and u, from dh; and h.
struct LinGrad {
  float dg, du, h;
};
template <int ACT>
__device__ __forceinline__ LinGrad lin_grad(float dh, float g, float u) {
  float da;
  const float a = lin_act<ACT, true>(g, da);
  return {dh * u * da, dh * a, a * u};
}

// ------------------------------------------------------------------ MMAs
// Masked forms: rows of the accumulator (TMEM lanes) whose bit in `off` is set keep their
// values, whatever the products for them are.
__device__ __forceinline__ void umma_f16_rows(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              const uint32_t (&off)[4]) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
      : "memory");
}

__device__ __forceinline__ void umma_f16_rows_pair(uint32_t d, uint64_t a, uint64_t b,
                                                   uint32_t idesc, const uint32_t (&off)[8]) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, "
      "{%4, %5, %6, %7, %8, %9, %10, %11}, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]),
      "r"(off[5]), "r"(off[6]), "r"(off[7])
      : "memory");
}

// 3D tiled loads (adapter s's rows of a stack): as tma_load_2d and tma_load_2d_pair.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t c0, int32_t c1,
                                                 int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"((uint64_t)map), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Descriptors of an operand in a stage at shared address `at`, and their advance for 16
// elements of k: 32 bytes within a K-major row; two groups of eight k rows (2048 bytes) of an
// MN-major box, whose 64-element boxes lie kLinBox apart (the leading byte offset).
template <bool MN>
__device__ __forceinline__ uint64_t lin_desc(uint32_t at) {
  const uint64_t d = sdesc_sw128(at);
  return MN ? d + ((uint64_t)((kLinBox >> 4) - 1) << 16) : d;
}
template <bool MN>
__host__ __device__ constexpr int lin_step() { return MN ? 2048 >> 4 : 2; }

// The MMAs of one stage (descriptors of its start); those wholly past k are left out.
template <bool PAIR, bool AMN, bool BMN>
__device__ __forceinline__ void lin_stage_mmas(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                               int left, bool first) {
  auto one = [&](int j, uint32_t acc) {
    if constexpr (PAIR) umma_f16_pair(d, a + j * lin_step<AMN>(), b + j * lin_step<BMN>(), idesc, acc);
    else umma_f16(d, a + j * lin_step<AMN>(), b + j * lin_step<BMN>(), idesc, acc);
  };
  one(0, first ? 0u : 1u);
  if (left > 48) {
    one(1, 1u);
    one(2, 1u);
    one(3, 1u);
  } else {
    if (left > 16) one(1, 1u);
    if (left > 32) one(2, 1u);
  }
}

// The MMA thread's way round the ring. The next stage is looked for before the MMAs of this
// one are issued: a look costs some 100 cycles until its answer, which a stage of a single
// CTA (256 cycles of MMAs) has no room for behind them.
template <int STAGES>
struct LinRing {
  LinAux* aux;
  uint64_t* full;
  int st = 0, used = 0;
  uint32_t phase = 0;
  bool ready = false;
  // The next stage's number once it is full; -1: the wait ran out.
  __device__ __forceinline__ int take() {
    if (!ready && !mx_wait(&full[st], phase, aux)) return -1;
    tc_fence_after();
    const int mine = st;
    if (++st == STAGES) {
      st = 0;
      phase ^= 1u;
    }
    ++used;
    ready = mbar_test_wait(&full[st], phase);
    return mine;
  }
};

// ------------------------------------------------------------------ adapters
// The stages that adapters add to a tile. T holds a row's rp high parts, then its rp low
// parts (t = high + low to 16 bits of mantissa in bf16, 22 in fp16: rounding t once would add
// as much error as the rounding of y).
//
// Up to rank 32 both parts lie in one stage's A, and B holds 64 / rp adapters behind one
// another, each 128 rows of rp elements in the 32- or 64-byte swizzle (64 adapters of rank
// 16: 16 stages instead of 64). Beyond, an adapter takes stages s = 0, 1, ... with the parts
// s & 1 of columns 64 (s / 2)... .
__host__ __device__ constexpr int lora_pack(int rp) { return rp <= 32 ? 64 / rp : 1; }
__host__ __device__ constexpr int lora_stages(int rp) {
  return rp <= 32 ? 1 : 2 * ((rp + 63) / 64);
}
__device__ __forceinline__ int lora_col_t(int rp, int s) {
  return rp <= 32 ? 0 : (s & 1) * rp + (s >> 1) * 64;
}
__device__ __forceinline__ int lora_col_b(int rp, int s) { return rp <= 32 ? 0 : (s >> 1) * 64; }
// Bytes of one adapter's part of a stage's B.
__host__ __device__ constexpr int lora_bytes(int rp) {
  return kLinTile * 2 * (rp <= 32 ? rp : 64);
}

// Bytes of an adapter's 128 rows of B_s in shared memory, all of its pieces.
__host__ __device__ constexpr int per_ups(int rp) {
  return lora_bytes(rp) * (rp <= 32 ? 1 : (rp + 63) / 64);
}

// B's descriptor: K-major rows of 32, 64 or 128 bytes (rank 16, 32, more) in the swizzle of
// that width (layout 6, 4, 2 at bits 61-63), groups of eight rows behind one another.
__device__ __forceinline__ uint64_t lora_desc(uint32_t at, int rp) {
  const uint64_t row = rp <= 32 ? rp * 2 : 128, layout = rp == 16 ? 6 : (rp == 32 ? 4 : 2);
  return (uint64_t)((at & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) | ((row * 8 >> 4) << 32) |
         ((uint64_t)1 << 46) | (layout << 61);
}

// The MMAs of adapter number j of a stage (rank over 32: of its stage s), for the rows that
// are not in `off`.
template <bool PAIR, int W>
__device__ __forceinline__ void lora_stage_mmas(uint32_t d, uint32_t a_at, uint32_t b_at,
                                                uint32_t idesc, int rp, int s, int j,
                                                const uint32_t (&off)[W]) {
  const uint64_t a = sdesc_sw128(a_at), b = lora_desc(b_at + j * lora_bytes(rp), rp);
  const int per = (rp <= 32 ? rp : min(64, rp - (s >> 1) * 64)) >> 4;  // 16-column pieces
  const int halves = rp <= 32 ? 2 : 1;
  for (int h = 0; h < halves; ++h)
    for (int i = 0; i < per; ++i) {
      if constexpr (PAIR) umma_f16_rows_pair(d, a + h * (rp >> 3) + i * 2, b + i * 2, idesc, off);
      else umma_f16_rows(d, a + h * (rp >> 3) + i * 2, b + i * 2, idesc, off);
    }
}

template <int THREADS>
__device__ __forceinline__ void plan_sync() {
  if constexpr (THREADS == kLinThreads) __syncthreads();
  else named_bar_sync(3, THREADS);
}

// Numbers the distinct adapters of `rows` rows from row0 on in the order of their first rows
// (THREADS threads, of which this is `tid`): ids and slot of each row, lead (the first rows);
// emit(number, id) once for each, mask(number, word, rows of those 32). Returns their number.
template <int THREADS, typename Emit, typename Mask>
__device__ __forceinline__ int number_adapters(const int32_t* index, int stack, int row0, int rows, int tid,
                                               int32_t* ids, int32_t* slot, uint32_t* lead,
                                               Emit emit, Mask mask) {
  const int warp = tid >> 5, lane = tid & 31, words = (rows + 31) / 32;
  for (int i = tid; i < words * 32; i += THREADS) {
    const int id = i < rows ? index[row0 + i] : -1;
    ids[i] = id >= 0 && id < stack ? id : -1;
  }
  plan_sync<THREADS>();
  // The first row of each row's adapter: within its 32 rows, then before them.
  for (int g = warp; g < words; g += THREADS / 32) {
    const int i = g * 32 + lane, id = ids[i];
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    int first = g * 32 + __ffs(same) - 1;
    for (int j = g * 32 - 4; j >= 0; j -= 4) {
      const int4 o = *reinterpret_cast<const int4*>(&ids[j]);
      first = o.w == id ? j + 3 : first;
      first = o.z == id ? j + 2 : first;
      first = o.y == id ? j + 1 : first;
      first = o.x == id ? j : first;
    }
    slot[i] = first;  // (a row's number, until all are known)
    const uint32_t b = __ballot_sync(0xffffffffu, id >= 0 && first == i);
    if (lane == 0) lead[g] = b;
  }
  plan_sync<THREADS>();
  int count = 0;
  for (int w = 0; w < words; ++w) count += __popc(lead[w]);
  for (int g = warp; g < words; g += THREADS / 32) {
    const int i = g * 32 + lane, id = ids[i], first = slot[i];
    const uint32_t same = __match_any_sync(0xffffffffu, id);
    int s = 0;
    for (int w = 0; w <= first >> 5; ++w)
      s += __popc(lead[w] & (w < (first >> 5) ? ~0u : (1u << (first & 31)) - 1));
    if (id >= 0) {
      slot[i] = s;
      if (first == i) emit(s, id);
      if (lane == __ffs(same) - 1) mask(s, g, same);
    }
  }
  plan_sync<THREADS>();
  return count;
}

// Four values as sums of two of T.
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

// ------------------------------------------------------------------ launches
// The kernels' variants. out: skg_out_t of C (fp16 or bf16).
struct LinVariant {
  int mode;
  bool a_mn, b_mn;  // M-major A, N-major B
  int out;
};

cudaError_t launch_lin_single(const LinVariant& v, const LinMaps& t, const LinParams& p,
                              cudaStream_t stream);
// Plain, K-major operands, adapters in the same kernel (skg_lin_adapted.cu); whether that is
// possible for so many adapters to a tile of a rank.
struct AdaptedParams {
  const int32_t* index;
  const float* scale;  // NULL = 1
  int count;           // adapters in the stack
  int most;            // that a tile's rows can have
  int rank;
  int stage_bytes, stages;
  uint32_t idesc_up;   // of the products with B_s
};
constexpr int kUpsMax = 32768;  // bytes of B_s that a CTA holds: its share of the adapters
inline bool lin_adapted_fits(int most, int rank, int split) {
  return most * rank <= 128 &&
         (most + split - 1) / split * per_ups((rank + 15) / 16 * 16) <= kUpsMax;
}
cudaError_t launch_lin_adapted(int out, const LinMaps& t, const CUtensorMap& down,
                               const LinParams& p, AdaptedParams a, cudaStream_t stream);

// Up to three plain products with N-major B in one launch (skg_lin_group.cu). The tiles of the
// first are shared by the `split` CTAs of a cluster; of the others every CTA has its own.
struct LinJob {
  int m, n, k, ksteps, terms, lo_b, a_mn, tiles_m, tiles_n;
  uint32_t idesc;
  void* c;
  int64_t ldc;
};
struct LinGroup {
  int split;
  int first[3];  // each product's first cluster (none: past the last cluster)
  LinJob job[3];
  uint32_t stages;
  uint64_t limit;
  skg_report_t* report;
};
struct LinGroupMaps {
  CUtensorMap a[3], b[3], lo[3];
};
cudaError_t launch_lin_group(int out, const LinGroupMaps& t, const LinGroup& p, int clusters,
                             cudaStream_t stream);

cudaError_t launch_lin_pair(const LinVariant& v, const LinMaps& t, const LinParams& p,
                            int clusters, cudaStream_t stream);

// CTA pairs of the pair kernel that can be resident on the current device at once, and clusters
// of `size` of the single kernel's CTAs that have an SM each.
int lin_pair_clusters_resident();
int lin_single_clusters(int size);

// Clusters of a kernel of this file's block size that can be resident at once (0: unknown).
inline int clusters_resident(const void* kernel, uint32_t smem, int size) {
  int n = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) ==
      cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(size * 256));
    cfg.blockDim = dim3(kLinThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) n = 0;
  }
  cudaGetLastError();
  return n;
}

// t = scale (x A^T) of every row's adapter, and the plans (skg_lora.cu).
struct LoraParams {
  int m, k, rank, rank_pad, count;  // count: adapters in the stack
  int ksteps, split, groups, a_rows;
  int per;             // adapters to a pass
  int stage_bytes, ring_stages;
  uint32_t idesc;
  const int32_t* index;
  const float* scale;  // NULL = 1
  void* t;             // m x 2 rank_pad: high parts, then low parts
  LoraPlan* plan;
  uint32_t stages;
  uint64_t limit;
  skg_report_t* report;
};
cudaError_t launch_lora_down(int dtype, const CUtensorMap& x, const CUtensorMap& down,
                             const LoraParams& p, cudaStream_t stream);

}  // namespace skg
