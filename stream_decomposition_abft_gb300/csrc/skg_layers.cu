// The entry points of a layer's projections (skgemm.h): checks, the choice of kernel, tensor
// maps and launches; and the elementwise kernel of the gated product's gradient.
//
//   skg_linear                   y = x W^T + t B^T, t = scale (x A^T): one launch where a tile's
//                                rows have few adapters (skg_lin_adapted.cu), else t first
//                                (skg_lora.cu)
//   skg_gated                    one kernel: both projections, the activation, the product
//   skg_gated_backward           dPRE elementwise; dX = dPRE W; dW = dPRE^T X
//   skg_feed_forward_backward    one kernel: dH = dY W_out, dPRE and H from it; dX; dW_in;
//                                dW_out = dY^T H
//
// The products run on skg_lin_single.cu's or skg_lin_pair.cu's kernels, which read operands
// stored along either dimension in place; small gradients' together (skg_lin_group.cu).
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_lin.cuh"

namespace skg {
namespace {

std::atomic<uint32_t> g_test_stages{0};
std::atomic<uint64_t> g_test_limit{0};

// Up to so many rows, dPRE and H are kept as sums of two numbers of dtype. Rounding them
// once adds as much error to a gradient as its own rounding: in the root of the mean square
// sqrt(2) times the latter alone over many elements, and anything over few. The second term
// has every stage loaded (from L2) and multiplied twice: with width and hidden 8192 the
// gradients of 1, 16, 64 and 128 tokens take 119, 116, 123 and 135 us with it and 105, 104,
// 107 and 110 without (through the second projection 167, 162, 172, 192 and 151, 152, 158,
// 160). Beyond one tile's rows it costs more than it gives: 160 tokens 190 and 130, 256
// tokens 208 and 136.
constexpr int64_t kTwoTermRows = 128;

constexpr int64_t kMaxDim = INT32_MAX / 4;

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// ------------------------------------------------------------------ dPRE from a given dH
struct DgateParams {
  int64_t m;
  int f, act;
  const void* dh;
  int64_t lddh;
  const void* pre;
  int64_t ldp;
  void* dpre;     // m x 2 f
  void* dpre_lo;  // its low parts, or NULL
};

template <typename T>
union Eight {
  uint4 q;
  T e[8];
};

template <typename T>
__device__ __forceinline__ void store8(T* hi, T* lo, const float (&v)[8]) {
  Eight<T> h, l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h.e[i] = mx_from_f32<T>(v[i]);
    const float r = v[i] - mx_to_f32(h.e[i]);
    l.e[i] = mx_from_f32<T>(isfinite(r) ? r : 0.f);
  }
  *reinterpret_cast<uint4*>(hi) = h.q;
  if (lo) *reinterpret_cast<uint4*>(lo) = l.q;
}

// Eight elements of a row per thread; reads and writes each element once, so memory bounds it
// (4096 x 8192: 336 MB, 5 % of the gradient that it begins).
template <typename T, int ACT>
__global__ void __launch_bounds__(128) dgate_kernel(const DgateParams p) {
  griddep_wait();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int col = ((int)blockIdx.x * 128 + (int)threadIdx.x) * 8;
  if (col >= p.f) return;
  for (int64_t row = blockIdx.y; row < p.m; row += gridDim.y) {
    Eight<T> d, g, u;
    d.q = *reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(p.dh) + row * p.lddh + col);
    const T* pre = reinterpret_cast<const T*>(p.pre) + row * p.ldp + col;
    g.q = *reinterpret_cast<const uint4*>(pre);
    u.q = *reinterpret_cast<const uint4*>(pre + p.f);
    float dg[8], du[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const LinGrad r = lin_grad<ACT>(mx_to_f32(d.e[i]), mx_to_f32(g.e[i]), mx_to_f32(u.e[i]));
      dg[i] = r.dg;
      du[i] = r.du;
    }
    const int64_t at = row * 2 * p.f + col;
    T *hi = reinterpret_cast<T*>(p.dpre) + at, *lo = reinterpret_cast<T*>(p.dpre_lo);
    lo = lo ? lo + at : lo;
    store8<T>(hi, lo, dg);
    store8<T>(hi + p.f, lo ? lo + p.f : lo, du);
  }
}

template <typename T>
cudaError_t launch_dgate_as(const DgateParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.f / 8 + 127) / 128), (unsigned)(p.m < 32768 ? p.m : 32768));
  const dim3 block(128);
  switch (p.act) {
    case SKG_ACT_SILU: return launch_pdl(dgate_kernel<T, SKG_ACT_SILU>, grid, block, 0, stream, p);
    case SKG_ACT_GELU: return launch_pdl(dgate_kernel<T, SKG_ACT_GELU>, grid, block, 0, stream, p);
    case SKG_ACT_GELU_TANH:
      return launch_pdl(dgate_kernel<T, SKG_ACT_GELU_TANH>, grid, block, 0, stream, p);
    default: return launch_pdl(dgate_kernel<T, SKG_ACT_RELU>, grid, block, 0, stream, p);
  }
}

cudaError_t launch_dgate(int dtype, const DgateParams& p, cudaStream_t stream) {
  return dtype == SKG_IN_F16 ? launch_dgate_as<__half>(p, stream)
                             : launch_dgate_as<__nv_bfloat16>(p, stream);
}

// ------------------------------------------------------------------ the activations alone
template <int ACT>
__global__ void act_kernel(int64_t count, const float* g, float* a, float* d) {
  for (int64_t i = blockIdx.x * 128ll + threadIdx.x; i < count; i += gridDim.x * 128ll)
    a[i] = lin_act<ACT, true>(g[i], d[i]);
}

// ------------------------------------------------------------------ products
struct Operand {
  const void* p;
  int64_t ld;
  bool mn;          // stored k x rows
  const void* lo;   // low parts, or NULL
};

struct Product {
  int mode;
  int64_t m, n, k;
  Operand a, b;
  void* c;
  int64_t ldc;
  int act;
  void* pre;        // kLinGated: PRE, or NULL; kLinGrad: DPRE
  int64_t ldp;
  const void* pre_in;  // kLinGrad: PRE
  int64_t ldp_in;
  void *c_lo, *pre_lo;
  const Product* second;  // a second product of the same k (M-major A, N-major B, pairs)
  const skg_adapters_t* adapters;
  void* t;          // with a plan: t and the plan come from skg_lora.cu's kernel
  LoraPlan* plan;
  int rank_pad;
};

struct Common {
  int dtype, sms;
  skg_report_t* report;
  uint32_t stages;
  uint64_t limit;
  cudaStream_t stream;
};

int out_of(int dtype) { return dtype == SKG_IN_F16 ? SKG_OUT_F16 : SKG_OUT_BF16; }

CUtensorMapDataType tma_type(int dtype) {
  return dtype == SKG_IN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Rows of a matrix of one row lie nowhere: any stride that the engine takes.
int64_t ld_of(int64_t ld, int64_t rows, int64_t inner) {
  return rows > 1 ? ld : (inner + 7) / 8 * 8;
}

bool map2(CUtensorMap* t, int dtype, const void* p, int64_t inner, int64_t rows, int64_t ld,
          int box_inner, int box_rows) {
  return encode_tensor_map(t, tma_type(dtype), 2, p, (uint64_t)inner, (uint64_t)rows,
                           (uint64_t)ld_of(ld, rows, inner), (uint32_t)box_inner,
                           (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

// An operand of `rows` rows: K-major boxes of 64 x box_rows, MN-major ones of 64 x 64.
bool map_operand(CUtensorMap* t, int dtype, const Operand& o, const void* p, int64_t rows,
                 int64_t k, int box_rows) {
  return o.mn ? map2(t, dtype, p, rows, k, o.ld, 64, kLinK)
              : map2(t, dtype, p, k, rows, o.ld, kLinK, box_rows);
}

// Single CTAs: how many share a 128 x 128 tile (S), and the estimated time (us). Up to 16
// rows of A the sum over the cluster is a few rows, and S is what fits the GPU at once (1 x
// 1024 x 8192: 27, 15, 9.1, 6.1 us with S = 1, 2, 4, 8). Else a fixed cost that grows with S,
// and the CTA's stages of k, at 0.2 us where all clusters find an SM for each CTA and 0.44
// where two CTAs share one (333 x 2048 x 2048: 10.4, 8.0, 10.3 with S = 1, 2, 4: 48, 96, 192
// CTAs). Larger clusters find less room, as a GPC's SMs do not divide by them: 128 x 2048 x
// 2048, 16 tiles, takes 6.8, 6.5, 8.6 with S = 4, 6, 8. `out`: what the activations of a whole
// tile take, which the CTAs of a cluster share; `extra`: stages behind k's, which they share too.
struct SinglePlan {
  int split;
  bool deep;
  double us;
};
SinglePlan single_plan(int64_t m, int64_t tiles, int ksteps, int sms, double out, int extra) {
  constexpr double kFixed[9] = {0, 4.4, 4.9, 5.1, 5.3, 0, 5.6, 0, 5.7};
  SinglePlan best = {1, false, 1e30};
  for (int s : {1, 2, 3, 4, 6, 8}) {
    if (s > 1 && (tiles * s > 2 * sms || s > ksteps)) break;
    const bool deep = s == 1 ? tiles <= sms : tiles <= lin_single_clusters(s);
    if ((s == 3 || s == 6) && (m <= 16 || !deep)) continue;
    const int stages = (ksteps + extra + s - 1) / s;
    const int64_t waves = (tiles * s + 2 * sms - 1) / (2 * sms);
    const double us =
        out / s + (deep ? kFixed[s] + 0.2 * stages
                        : (s == 1 ? 3.2 : s == 8 ? 9.0 : 6.5) + 0.436 * (double)waves * stages);
    if (m <= 16 || us < best.us) best = {s, deep, us};
  }
  return best;
}

// The estimate of a product on CTA pairs, whose 256 x 256 tiles halve what each SM reads per
// product but cannot share a tile's k. Up to 128 rows the single CTAs win at every n and k;
// beyond, the lower estimate: 0.262 us a stage, 0.29 where the power limit lowers the clock
// (1024 x 2048 x 2048: 12.9 us paired, 10.8 single; 1024 x 8192 x 1024: 13.8 and 19.9).
double pair_us(int64_t m, int64_t tiles, int ksteps, int clusters, double out) {
  if (m <= kLinTile) return 1e30;
  const int64_t waves = (tiles + clusters - 1) / clusters;
  return 4.2 + out + (waves > 1 ? 0.29 : 0.262) * (double)waves * ksteps;
}

// Adapters that 128 rows can have.
int most_adapters(int64_t m, const skg_adapters_t& ad) {
  const int rows = m < kLinTile ? (int)m : kLinTile;
  return ad.count < rows ? ad.count : rows;
}

// How a product runs.
struct Choice {
  bool pair, deep;
  int64_t tiles_m, tiles_n;
  int split, resident;
  double us;  // the estimate
};
Choice choose(const Product& q, const Common& c) {
  const int64_t cols = q.mode == kLinGated ? 2 * q.n : q.n;  // of the accumulators
  const int64_t tm1 = (q.m + 127) / 128, tn1 = (cols + 127) / 128;
  const int64_t tm2 = (q.m + 255) / 256, tn2 = (cols + 255) / 256;
  const int steps = (int)((q.k + kLinK - 1) / kLinK) * (q.a.lo || q.b.lo ? 2 : 1);
  Choice h = {};
  h.resident = lin_pair_clusters_resident();
  const double out = q.mode == kLinGrad ? 2.0 : q.mode == kLinGated ? 0.5 : 0.0;
  // Adapters' stages: how many of the stack a tile's rows have is not known here; half.
  const int extra = q.adapters ? (most_adapters(q.m, *q.adapters) / 2 + lora_pack(q.rank_pad) - 1) /
                                     lora_pack(q.rank_pad) * lora_stages(q.rank_pad)
                               : 0;
  const SinglePlan single = single_plan(q.m, tm1 * tn1, steps, c.sms, out, extra);
  // (The low parts of H and DPRE are written by single CTAs; up to 128 rows they run.)
  double paired = h.resident > 0 && q.n >= 8 && !q.c_lo
                            ? pair_us(q.m, tm2 * tn2, steps + extra, h.resident, 2.0 * out)
                            : 1e30;
  // With adapters the pairs are two launches, where single CTAs may be one (1087 x 152 x 176, one
  // adapter: 12.4 and 10.6 us).
  if (q.adapters && (q.m <= 16 || single.deep) &&
      lin_adapted_fits(most_adapters(q.m, *q.adapters), q.adapters->rank, single.split))
    paired += 1.5;
  h.pair = paired <= single.us;
  h.tiles_m = h.pair ? tm2 : tm1;
  h.tiles_n = h.pair ? tn2 : tn1;
  h.split = h.pair ? 1 : single.split;
  h.deep = !h.pair && single.deep;
  h.us = h.pair ? paired : single.us;
  return h;
}

// Whether a product with adapters is one launch (skg_lin_adapted.cu). With more than 16 rows
// the columns of x A^T cost a stage up to 0.1 us, which long ranges of k add up to more than
// the second launch takes (64 x 8192 x 8192, adapters of rank 16: one 27.7 in one launch, 29 in
// two; eight 37.9 and 33.1).
bool one_launch(const Product& q, const Choice& h) {
  if (!q.adapters || h.pair) return false;
  const int most = most_adapters(q.m, *q.adapters);
  const int rank = q.adapters->rank;
  if (!lin_adapted_fits(most, rank, h.split)) return false;
  const double stages = (double)((q.k + kLinK - 1) / kLinK) / h.split;
  return q.m <= 16 || (h.deep && 0.1 * stages * most * rank / 128 <= 3.0);
}

// skg_lora.cu's CTAs: to share the rows' k (split), clusters to share the adapters (groups),
// adapters to a pass: the least estimate of passes one behind another, 2.5 us and 0.25 a stage
// each, over what fits the GPU at once (4593 rows, k = 232, 30 adapters of rank 48: 75.8 us with
// k split first, 38 so).
//
// A product behind it whose CTAs take an SM each begins everywhere at once where this kernel
// leaves it as many SMs. That pays while its few CTAs are done by half of the product's time
// (64 x 8192 x 8192, eight adapters of rank 16: 33.1 -> 28.3 us, 25.4 without adapters; 64
// adapters 41.6 -> 53).
void share_out(LoraParams& p, int cols, int most, const Choice& h, int sms) {
  const int64_t tiles = (p.m + kLinTile - 1) / kLinTile;
  const int chunks = (p.rank_pad + 127) / 128;
  auto least = [&](int64_t ctas) {
    double best = 1e30;
    for (int split = 1; split <= 8 && split <= p.ksteps; split *= 2) {
      const int64_t most_ctas = split == 8 && ctas > sms ? sms : ctas;
      if (split > 1 && tiles * split > most_ctas) break;
      int64_t room = most_ctas / (tiles * split);
      if (room < 1) room = 1;
      const int64_t want = (most + room - 1) / room;
      const int per = (int)(want < 128 / cols ? want : 128 / cols);
      const int64_t passes = chunks > 1 ? (int64_t)most * chunks : (most + per - 1) / per;
      const int64_t groups = room < passes ? room : passes;
      const double us = (double)((passes + groups - 1) / groups) *
                        (2.5 + 0.25 * ((p.ksteps + split - 1) / split));
      if (us < best) {
        best = us;
        p.split = split;
        p.per = per;
        p.groups = (int)groups;
      }
    }
    return best;
  };
  const int64_t beside = h.deep ? sms - h.tiles_m * h.tiles_n * h.split : 0;
  if (beside < tiles || least(beside) > 0.5 * h.us) least(2 * (int64_t)sms);
}

bool map_down(CUtensorMap* t, int dtype, const skg_adapters_t& ad, int64_t k, int box_rows) {
  return encode_tensor_map3(t, tma_type(dtype), 2, ad.down, (uint64_t)k, (uint64_t)ad.rank,
                            (uint64_t)ad.count, (uint64_t)ld_of(ad.ld_down, ad.rank, k),
                            (uint64_t)ld_of(ad.stride_down, ad.count, k), kLinK,
                            (uint32_t)box_rows, CU_TENSOR_MAP_SWIZZLE_128B) == CUDA_SUCCESS;
}

skg_status_t run_product(const Product& q, const Common& c) {
  const Choice h = choose(q, c);
  const bool pair = h.pair, gated = q.mode == kLinGated, fused = one_launch(q, h);
  LinParams p = {};
  p.m = (int)q.m;
  p.n = (int)q.n;
  p.k = (int)q.k;
  p.ksteps = (int)((q.k + kLinK - 1) / kLinK);
  p.terms = q.a.lo || q.b.lo ? 2 : 1;
  p.lo_b = q.b.lo != nullptr;
  p.act = q.act;
  p.c = q.c;
  p.ldc = ld_of(q.ldc, q.m, q.n);
  p.pre = q.pre;
  p.ldp = ld_of(q.ldp, q.m, 2 * q.n);
  p.pre_in = q.pre_in;
  p.ldp_in = ld_of(q.ldp_in, q.m, 2 * q.n);
  p.c_lo = q.c_lo;
  p.pre_lo = q.pre_lo;
  p.plan = q.plan;
  p.rank_pad = q.rank_pad;
  p.report = c.report;
  p.stages = c.stages ? c.stages : UINT32_MAX;
  p.limit = c.limit ? c.limit : kMxTimeoutNs;
  if (h.tiles_m * h.tiles_n * h.split > INT32_MAX) return SKG_ERR_UNSUPPORTED;
  p.tiles_m = (int)h.tiles_m;
  p.tiles_n = (int)h.tiles_n;
  p.split = h.split;
  p.deep = h.deep;
  p.a_rows = !pair && q.m < kLinTile ? (p.m + 7) / 8 * 8 : kLinTile;
  const uint32_t bf16 = c.dtype == SKG_IN_BF16;
  p.idesc = idesc_f16(bf16, pair ? 256 : 128, pair ? 256 : 128) | ((uint32_t)q.a.mn << 15) |
            ((uint32_t)q.b.mn << 16);

  // Rows of B, and of its box: a tile's (K-major) columns, or one projection's share of them.
  const int64_t cols = gated ? 2 * q.n : q.n;
  const int b_box = gated && !pair ? 64 : 128;
  LinMaps t;
  if (!map_operand(&t.a, c.dtype, q.a, q.a.p, q.m, q.k, p.a_rows) ||
      !map_operand(&t.b, c.dtype, q.b, q.b.p, cols, q.k, b_box))
    return SKG_ERR_CUDA;
  t.lo = t.t = t.up = t.c = t.gate = t.pre_up = t.a;
  if (p.terms == 2 &&
      !(p.lo_b ? map_operand(&t.lo, c.dtype, q.b, q.b.lo, cols, q.k, b_box)
               : map_operand(&t.lo, c.dtype, q.a, q.a.lo, q.m, q.k, p.a_rows)))
    return SKG_ERR_CUDA;
  if (q.adapters) {
    const skg_adapters_t& ad = *q.adapters;
    if (encode_tensor_map3(&t.up, tma_type(c.dtype), 2, ad.up, (uint64_t)ad.rank, (uint64_t)q.n,
                           (uint64_t)ad.count, (uint64_t)ld_of(ad.ld_up, q.n, ad.rank),
                           (uint64_t)ld_of(ad.stride_up, ad.count, ad.rank),
                           (uint32_t)(q.rank_pad <= 32 ? q.rank_pad : 64), 128,
                           q.rank_pad == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                           : q.rank_pad == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                              : CU_TENSOR_MAP_SWIZZLE_128B) != CUDA_SUCCESS)
      return SKG_ERR_CUDA;
    if (fused) {
      AdaptedParams a = {};
      a.index = ad.index;
      a.scale = ad.scale;
      a.count = ad.count;
      a.rank = ad.rank;
      a.most = most_adapters(q.m, ad);
      a.idesc_up = p.idesc;
      p.idesc = idesc_f16(bf16, 128, (uint32_t)(128 + (a.most * a.rank + 15) / 16 * 16));
      CUtensorMap down;
      if (!map_down(&down, c.dtype, ad, q.k, ad.rank)) return SKG_ERR_CUDA;
      return launch_lin_adapted(out_of(c.dtype), t, down, p, a, c.stream) == cudaSuccess ? SKG_OK
                                                                               : SKG_ERR_CUDA;
    }
    if (!map2(&t.t, c.dtype, q.t, 2 * q.rank_pad, q.m, 2 * q.rank_pad, 64, p.a_rows))
      return SKG_ERR_CUDA;
  }
  if (pair) {
    if (!map2(&t.c, c.dtype, q.c, q.n & ~7, q.m, p.ldc, 64, 32)) return SKG_ERR_CUDA;
    if (q.mode == kLinGrad &&
        (!map2(&t.t, c.dtype, q.pre_in, q.n, q.m, p.ldp_in, 64, 32) ||
         !map2(&t.up, c.dtype, (const uint16_t*)q.pre_in + q.n, q.n, q.m, p.ldp_in, 64, 32)))
      return SKG_ERR_CUDA;
    if (q.pre && (!map2(&t.gate, c.dtype, q.pre, q.n, q.m, p.ldp, 64, 32) ||
                  !map2(&t.pre_up, c.dtype, (const uint16_t*)q.pre + q.n, q.n, q.m, p.ldp, 64, 32)))
      return SKG_ERR_CUDA;
  }
  int64_t tiles = h.tiles_m * h.tiles_n;
  if (pair && q.second) {
    const Product& w = *q.second;
    p.second = {(int)w.m, (int)w.n, (int)((w.m + 255) / 256), (int)((w.n + 255) / 256),
                w.b.lo != nullptr, w.c, ld_of(w.ldc, w.m, w.n)};
    tiles += (int64_t)p.second.tiles_m * p.second.tiles_n;
    if (tiles > INT32_MAX) return SKG_ERR_UNSUPPORTED;
    if (!map_operand(&t.t, c.dtype, w.a, w.a.p, w.m, w.k, 128) ||
        !map_operand(&t.up, c.dtype, w.b, w.b.p, w.n, w.k, 128) ||
        !map2(&t.pre_up, c.dtype, w.c, w.n & ~7, w.m, p.second.ldc, 64, 32) ||
        (p.terms == 2 && !map_operand(&t.gate, c.dtype, w.a.lo ? w.a : w.b, w.a.lo ? w.a.lo : w.b.lo,
                                      w.a.lo ? w.m : w.n, w.k, 128)))
      return SKG_ERR_CUDA;
  }
  const LinVariant v = {q.mode, q.a.mn, q.b.mn, out_of(c.dtype)};
  const cudaError_t e =
      pair ? launch_lin_pair(v, t, p, (int)(tiles < h.resident ? tiles : h.resident), c.stream)
           : launch_lin_single(v, t, p, c.stream);
  return e == cudaSuccess ? SKG_OK : SKG_ERR_CUDA;
}

skg_status_t zero(void* c, int64_t ldc, int64_t m, int64_t n, const Common& k) {
  if (m <= 0 || n <= 0) return SKG_OK;
  return launch_scale(out_of(k.dtype), c, ldc, (int)m, (int)n, 0.f, k.stream) == cudaSuccess
             ? SKG_OK
             : SKG_ERR_CUDA;
}

// A product whose sums may be over nothing.
skg_status_t product_or_zero(const Product& q, const Common& c) {
  if (q.m == 0 || q.n == 0) return SKG_OK;
  if (q.k == 0) return zero(q.c, ld_of(q.ldc, q.m, q.n), q.m, q.n, c);
  return run_product(q, c);
}

// ------------------------------------------------------------------ checks
// A row-major matrix of rows x cols with elements in it: there, and rows that hold cols.
bool there(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return rows == 0 || cols == 0 || (p && (rows <= 1 || ld >= cols));
}

// The TMA engine's rules, of a matrix with elements in it: its base, the rows' distance, which
// has 39 bits, and (of the processor's addresses) its whole extent.
constexpr int64_t kMaxStride = ((int64_t)1 << 39) - 1;  // elements of two bytes
bool spans(int64_t count, int64_t stride) {
  return count <= 1 || (stride <= kMaxStride && stride <= ((int64_t)1 << 55) / count);
}
bool aligned(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return rows == 0 || cols == 0 ||
         (((uintptr_t)p & 15) == 0 && (rows == 1 || ld % 8 == 0) && spans(rows, ld));
}

// Rows of `width` bytes, `pitch` bytes from one to the next (none: rows or width 0).
struct Rows {
  int64_t at, rows, width, pitch;
  int64_t end() const { return at + (rows - 1) * pitch + width; }
};
Rows rows_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int bytes = 2) {
  const bool some = p && rows > 0 && cols > 0;
  return {(int64_t)(uintptr_t)p, some ? rows : 0, cols * bytes, rows > 1 ? ld * bytes : cols * bytes};
}

// Whether some byte is in both. Rows that lie between one another's (columns of one buffer)
// are told apart.
bool overlap(const Rows& a, const Rows& b) {
  if (a.rows == 0 || b.rows == 0 || a.end() <= b.at || b.end() <= a.at) return false;
  // Row i of b and row j of a meet if i b.pitch - j a.pitch is between a.at - b.at - b.width and
  // a.at - b.at + a.width.
  const int64_t low = a.at - b.at - b.width, high = a.at - b.at + a.width;
  auto above = [](int64_t v, int64_t pitch) {  // the least multiple of pitch over v, in pitches
    return v >= 0 ? v / pitch + 1 : -((-v - 1) / pitch);
  };
  if (a.pitch == b.pitch) {
    int64_t t = above(low, a.pitch);
    if (t < 1 - a.rows) t = 1 - a.rows;
    return t < b.rows && t * a.pitch < high;
  }
  if (a.rows > b.rows) return overlap(b, a);
  for (int64_t j = 0; j < a.rows; ++j) {
    int64_t i = above(low + j * a.pitch, b.pitch);
    if (i < 0) i = 0;
    if (i < b.rows && i * b.pitch < high + j * a.pitch) return true;
  }
  return false;
}

// The matrices of a stack, `stride` elements apart.
bool overlap_stack(const Rows& out, const void* p, int64_t count, int64_t stride, int64_t rows,
                   int64_t cols, int64_t ld) {
  Rows one = rows_of(p, rows, cols, ld);
  if (count <= 0 || out.rows == 0 || one.rows == 0 || out.end() <= one.at ||
      one.end() + (count - 1) * stride * 2 <= out.at)
    return false;
  for (int64_t s = 0; s < count; ++s, one.at += stride * 2)
    if (overlap(out, one)) return true;
  return false;
}

// Whether one of the outputs shares memory with an input or another output.
template <int OUTS, int INS>
bool any_overlap(const Rows (&outs)[OUTS], const Rows (&ins)[INS]) {
  for (int i = 0; i < OUTS; ++i) {
    for (const Rows& r : ins)
      if (overlap(outs[i], r)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

skg_status_t check_sizes(int64_t m, int64_t n, int64_t k, int32_t dtype) {
  if (m < 0 || n < 0 || k < 0 || (dtype != SKG_IN_F16 && dtype != SKG_IN_BF16)) return SKG_ERR_ARG;
  if (m > kMaxDim || n > kMaxDim / 2 || k > kMaxDim) return SKG_ERR_UNSUPPORTED;
  return SKG_OK;
}

skg_status_t check_memory(void* workspace, size_t ws_bytes, const void* scratch,
                          size_t scratch_bytes, size_t need) {
  if (!workspace || ((uintptr_t)workspace & 255) || ws_bytes < skg_workspace_size_layers())
    return SKG_ERR_WORKSPACE;
  if (need && (!scratch || ((uintptr_t)scratch & 255) || scratch_bytes < need))
    return SKG_ERR_WORKSPACE;
  return SKG_OK;
}

skg_status_t common(int32_t dtype, void* workspace, void* stream, Common* c) {
  c->dtype = dtype;
  c->sms = skg_device_sm_count();
  if (c->sms <= 0) return SKG_ERR_CUDA;
  c->report = workspace_report(workspace);
  c->stages = g_test_stages.load(std::memory_order_relaxed);
  c->limit = g_test_limit.load(std::memory_order_relaxed);
  c->stream = (cudaStream_t)stream;
  return SKG_OK;
}

// H's scratch rows start on 32-byte sectors (others: half as much again for the loads of a
// stage).
int64_t h_pitch(int64_t f) { return (f + 15) / 16 * 16; }

// Scratch of the gradients, from its start.
struct BackwardScratch {
  size_t dpre, dpre_lo, h, h_lo, total;
};
BackwardScratch backward_scratch(int64_t m, int64_t f, bool block) {
  BackwardScratch s = {};
  const size_t n = (size_t)m * (size_t)f, two = m <= kTwoTermRows ? 1 : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += up256(bytes);
    return a;
  };
  s.dpre = take(n * 4);
  s.dpre_lo = take(two * n * 4);
  const size_t nh = (size_t)m * (size_t)h_pitch(f);
  s.h = take(block ? nh * 2 : 0);
  s.h_lo = take(block ? two * nh * 2 : 0);
  s.total = at;
  return s;
}

// Plain products with N-major B in one launch of single CTAs, the first one's tiles shared by
// `split` CTAs each.
skg_status_t run_group(const Product* const* jobs, int count, int split, const Common& c) {
  LinGroup p = {};
  LinGroupMaps t;
  int64_t clusters = 0;
  p.split = split;
  for (int j = 0; j < 3; ++j) {
    p.first[j] = (int)clusters;
    const Product& q = *jobs[j < count ? j : 0];
    if (j < count) {
      LinJob& w = p.job[j];
      w.m = (int)q.m;
      w.n = (int)q.n;
      w.k = (int)q.k;
      w.ksteps = (int)((q.k + kLinK - 1) / kLinK);
      w.terms = q.a.lo || q.b.lo ? 2 : 1;
      w.lo_b = q.b.lo != nullptr;
      w.a_mn = q.a.mn;
      w.tiles_m = (int)((q.m + 127) / 128);
      w.tiles_n = (int)((q.n + 127) / 128);
      w.idesc = idesc_f16(c.dtype == SKG_IN_BF16, 128, 128) | ((uint32_t)q.a.mn << 15) | (1u << 16);
      w.c = q.c;
      w.ldc = ld_of(q.ldc, q.m, q.n);
      const int64_t tiles = (int64_t)w.tiles_m * w.tiles_n;
      clusters += j == 0 ? tiles : (tiles + split - 1) / split;
    }
    if (!map_operand(&t.a[j], c.dtype, q.a, q.a.p, q.m, q.k, 128) ||
        !map_operand(&t.b[j], c.dtype, q.b, q.b.p, q.n, q.k, 128))
      return SKG_ERR_CUDA;
    t.lo[j] = t.a[j];
    if ((q.a.lo && !map_operand(&t.lo[j], c.dtype, q.a, q.a.lo, q.m, q.k, 128)) ||
        (q.b.lo && !map_operand(&t.lo[j], c.dtype, q.b, q.b.lo, q.n, q.k, 128)))
      return SKG_ERR_CUDA;
  }
  for (int j = count; j < 3; ++j) p.first[j] = (int)clusters;
  p.stages = c.stages ? c.stages : UINT32_MAX;
  p.limit = c.limit ? c.limit : kMxTimeoutNs;
  p.report = c.report;
  return launch_lin_group(out_of(c.dtype), t, p, (int)clusters, c.stream) == cudaSuccess
             ? SKG_OK
             : SKG_ERR_CUDA;
}

// How many CTAs share a tile of the first product if these run in one launch, and the estimate:
// a fixed cost, the longer of its longest CTA and all stages over all SMs, and 3 us for each
// further round of CTAs, whose beginnings and ends nothing covers (512 x 1024 x 2816: 39.7 us
// for the whole gradient in this way, three rounds, 37.5 apart; 323 x 520 x 256 11.9 and 21.6).
double group_us(const Product* const* jobs, int count, const Common& c, int* split) {
  int64_t tiles[3], steps[3], all = 0;
  for (int j = 0; j < count; ++j) {
    const Product& q = *jobs[j];
    tiles[j] = ((q.m + 127) / 128) * ((q.n + 127) / 128);
    steps[j] = (q.k + kLinK - 1) / kLinK * (q.a.lo || q.b.lo ? 2 : 1);
    all += tiles[j] * steps[j];
  }
  double best = 1e30;
  for (int s : {1, 2, 4, 8}) {
    if (s > 1 && (s > steps[0] || tiles[0] * s > 2 * c.sms)) break;
    int64_t ctas = tiles[0] * s, longest = (steps[0] + s - 1) / s;
    for (int j = 1; j < count; ++j) {
      ctas += (tiles[j] + s - 1) / s * s;
      if (steps[j] > longest) longest = steps[j];
    }
    if (ctas > INT32_MAX) return 1e30;
    const double one = (ctas <= c.sms ? 0.2 : 0.44) * (double)longest;
    const double sum = 0.22 * (double)all / c.sms;
    const double waves = (double)((ctas + 2 * c.sms - 1) / (2 * c.sms));
    const double us =
        (s == 1 ? 4.6 : s == 8 ? 6.2 : 5.5) + 3.0 * (waves - 1) + (one > sum ? one : sum);
    if (us < best) {
      best = us;
      *split = s;
    }
  }
  return best;
}

// dX = dPRE W (m x k), dW = dPRE^T X (2 f x k) and a second weight gradient (or NULL): in one
// launch of single CTAs where that is estimated the shortest (a launch less is counted as 2 us),
// else dX by itself and the weight gradients in one launch where both run on pairs.
skg_status_t in_gradients(int64_t m, int64_t f, int64_t k, const void* dpre, const void* dpre_lo,
                          const void* X, int64_t ldx, const void* W, int64_t ldw, void* dX,
                          int64_t lddx, void* dW, int64_t lddw, const Product* other,
                          const Common& c) {
  Product x = {};
  x.m = m;
  x.n = k;
  x.k = 2 * f;
  x.a = {dpre, 2 * f, false, dpre_lo};
  x.b = {W, ldw, true, nullptr};
  x.c = dX;
  x.ldc = lddx;
  Product w = {};
  w.m = 2 * f;
  w.n = k;
  w.k = m;
  w.a = {dpre, 2 * f, true, dpre_lo};
  w.b = {X, ldx, true, nullptr};
  w.c = dW;
  w.ldc = lddw;
  if (m > 0 && f > 0) {
    const Product* jobs[3] = {&x, &w, other};
    const int count = other ? 3 : 2;
    const Choice hx = choose(x, c), hw = choose(w, c);
    double apart = hx.us + hw.us - 2.0;
    bool both = false;
    if (other) {
      const Choice ho = choose(*other, c);
      both = hw.pair && ho.pair;
      apart += both ? ho.us - 4.2 : ho.us - 2.0;
    }
    int split = 1;
    if (group_us(jobs, count, c, &split) < apart) return run_group(jobs, count, split, c);
    if (both) w.second = other;
  }
  skg_status_t st = product_or_zero(x, c);
  if (st == SKG_OK) st = product_or_zero(w, c);
  return st == SKG_OK && other && !w.second ? product_or_zero(*other, c) : st;
}

}  // namespace
}  // namespace skg

using namespace skg;

extern "C" {

skg_status_t skg_layers_test_stall(int32_t stages, uint64_t timeout_ns) {
  if (stages < 0) return SKG_ERR_ARG;
  g_test_stages.store((uint32_t)stages, std::memory_order_relaxed);
  g_test_limit.store(timeout_ns, std::memory_order_relaxed);
  return SKG_OK;
}

skg_status_t skg_layers_test_activation(int32_t act, int64_t count, const float* g, float* a,
                                        float* d, void* stream) {
  if (act < SKG_ACT_SILU || act > SKG_ACT_RELU || count < 0 || (count && (!g || !a || !d)))
    return SKG_ERR_ARG;
  if (count == 0) return SKG_OK;
  const int64_t blocks = (count + 127) / 128;
  const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096)), block(128);
  cudaStream_t st = (cudaStream_t)stream;
  if (act == SKG_ACT_SILU) act_kernel<SKG_ACT_SILU><<<grid, block, 0, st>>>(count, g, a, d);
  else if (act == SKG_ACT_GELU) act_kernel<SKG_ACT_GELU><<<grid, block, 0, st>>>(count, g, a, d);
  else if (act == SKG_ACT_GELU_TANH)
    act_kernel<SKG_ACT_GELU_TANH><<<grid, block, 0, st>>>(count, g, a, d);
  else act_kernel<SKG_ACT_RELU><<<grid, block, 0, st>>>(count, g, a, d);
  return cudaGetLastError() == cudaSuccess ? SKG_OK : SKG_ERR_CUDA;
}

size_t skg_workspace_size_layers(void) { return fixed_header_bytes(); }

size_t skg_scratch_size_linear(int64_t m, int32_t rank) {
  if (m <= 0 || m > kMaxDim || rank <= 0 || rank > 512) return 0;
  const size_t rp = (size_t)(rank + 15) / 16 * 16;
  return up256((size_t)((m + kLoraRows - 1) / kLoraRows) * sizeof(LoraPlan)) +
         up256((size_t)m * 4 * rp);
}

skg_status_t skg_linear(int64_t m, int64_t n, int64_t k, const void* X, int64_t ldx, const void* W,
                        int64_t ldw, const skg_adapters_t* ad, void* Y, int64_t ldy, int32_t dtype,
                        void* workspace, size_t ws_bytes, void* scratch, size_t scratch_bytes,
                        void* stream) {
  skg_status_t st = check_sizes(m, n, k, dtype);
  if (st != SKG_OK) return st;
  if (!there(X, m, k, ldx) || !there(W, n, k, ldw) || !there(Y, m, n, ldy)) return SKG_ERR_ARG;
  if (ad) {
    if (ad->count < 0 || ad->rank < 0 || (m > 0 && !ad->index)) return SKG_ERR_ARG;
    const bool some = ad->count > 0 && ad->rank > 0;
    if (some && (!there(ad->down, ad->rank, k, ad->ld_down) ||
                 !there(ad->up, n, ad->rank, ad->ld_up)))
      return SKG_ERR_ARG;
    if (some && ad->count > 1 && (ad->stride_down <= 0 || ad->stride_up <= 0)) return SKG_ERR_ARG;
    if (ad->rank > 512 || ad->rank % 8) return SKG_ERR_UNSUPPORTED;
    if (some && (!aligned(ad->down, ad->rank, k, ad->ld_down) || !aligned(ad->up, n, ad->rank, ad->ld_up) ||
                 (ad->count > 1 && (ad->stride_down % 8 || ad->stride_up % 8)) ||
                 !spans(ad->count, ad->stride_down) || !spans(ad->count, ad->stride_up) ||
                 ((uintptr_t)ad->index & 3) || ((uintptr_t)ad->scale & 3)))
      return SKG_ERR_UNSUPPORTED;
    if (!some) ad = nullptr;
  }
  if (m == 0 || n == 0) return SKG_OK;
  if (!aligned(X, m, k, ldx) || !aligned(W, n, k, ldw) || !aligned(Y, m, n, ldy)) return SKG_ERR_UNSUPPORTED;
  if (k == 0) ad = nullptr;
  const size_t need = ad ? skg_scratch_size_linear(m, ad->rank) : 0;
  st = check_memory(workspace, ws_bytes, scratch, scratch_bytes, need);
  if (st != SKG_OK) return st;
  const Rows out = rows_of(Y, m, n, ldy);
  if (overlap(out, rows_of(X, m, k, ldx)) || overlap(out, rows_of(W, n, k, ldw))) return SKG_ERR_ARG;
  if (ad && (overlap(out, rows_of(ad->index, 1, m, m, 4)) ||
             overlap(out, rows_of(ad->scale, 1, ad->count, ad->count, 4)) ||
             overlap_stack(out, ad->down, ad->count, ad->stride_down, ad->rank, k, ad->ld_down) ||
             overlap_stack(out, ad->up, ad->count, ad->stride_up, n, ad->rank, ad->ld_up)))
    return SKG_ERR_ARG;
  Common c;
  st = common(dtype, workspace, stream, &c);
  if (st != SKG_OK) return st;
  Product q = {};
  q.m = m;
  q.n = n;
  q.k = k;
  q.a = {X, ldx, false, nullptr};
  q.b = {W, ldw, false, nullptr};
  q.c = Y;
  q.ldc = ldy;
  if (ad) {
    q.adapters = ad;
    q.rank_pad = (ad->rank + 15) / 16 * 16;
  }
  if (ad && !one_launch(q, choose(q, c))) {
    q.plan = reinterpret_cast<LoraPlan*>(scratch);
    q.t = (uint8_t*)scratch +
          up256((size_t)((m + kLoraRows - 1) / kLoraRows) * sizeof(LoraPlan));
    LoraParams p = {};
    p.m = (int)m;
    p.k = (int)k;
    p.rank = ad->rank;
    p.rank_pad = q.rank_pad;
    p.count = ad->count;
    p.ksteps = (int)((k + kLinK - 1) / kLinK);
    p.a_rows = m < kLinTile ? (p.m + 7) / 8 * 8 : kLinTile;
    const int cols = q.rank_pad < 128 ? q.rank_pad : 128;
    p.index = ad->index;
    p.scale = ad->scale;
    p.t = q.t;
    p.plan = q.plan;
    p.stages = c.stages ? c.stages : UINT32_MAX;
    p.limit = c.limit ? c.limit : kMxTimeoutNs;
    p.report = c.report;
    share_out(p, cols, most_adapters(m, *ad), choose(q, c), c.sms);
    p.idesc = idesc_f16(dtype == SKG_IN_BF16, 128, (uint32_t)(p.per * cols));
    CUtensorMap tx, td;
    if (!map2(&tx, dtype, X, k, m, ldx, kLinK, p.a_rows) || !map_down(&td, dtype, *ad, k, cols))
      return SKG_ERR_CUDA;
    if (launch_lora_down(dtype, tx, td, p, c.stream) != cudaSuccess) return SKG_ERR_CUDA;
  }
  return product_or_zero(q, c);
}

skg_status_t skg_gated(int64_t m, int64_t hidden, int64_t k, const void* X, int64_t ldx,
                       const void* W, int64_t ldw, int32_t act, void* H, int64_t ldh, void* PRE,
                       int64_t ldp, int32_t dtype, void* workspace, size_t ws_bytes, void* stream) {
  skg_status_t st = check_sizes(m, hidden, k, dtype);
  if (st != SKG_OK) return st;
  if (act < SKG_ACT_SILU || act > SKG_ACT_RELU) return SKG_ERR_ARG;
  if (!there(X, m, k, ldx) || !there(W, 2 * hidden, k, ldw) || !there(H, m, hidden, ldh) ||
      (PRE && !there(PRE, m, 2 * hidden, ldp)))
    return SKG_ERR_ARG;
  if (hidden % 8) return SKG_ERR_UNSUPPORTED;
  if (m == 0 || hidden == 0) return SKG_OK;
  if (!aligned(X, m, k, ldx) || !aligned(W, 2 * hidden, k, ldw) || !aligned(H, m, hidden, ldh) ||
      (PRE && !aligned(PRE, m, 2 * hidden, ldp)))
    return SKG_ERR_UNSUPPORTED;
  st = check_memory(workspace, ws_bytes, nullptr, 0, 0);
  if (st != SKG_OK) return st;
  if (any_overlap({rows_of(H, m, hidden, ldh), rows_of(PRE, m, 2 * hidden, ldp)},
                  {rows_of(X, m, k, ldx), rows_of(W, 2 * hidden, k, ldw)}))
    return SKG_ERR_ARG;
  Common c;
  st = common(dtype, workspace, stream, &c);
  if (st != SKG_OK) return st;
  if (k == 0) {  // act(0) * 0
    st = zero(H, ld_of(ldh, m, hidden), m, hidden, c);
    return st == SKG_OK && PRE ? zero(PRE, ld_of(ldp, m, 2 * hidden), m, 2 * hidden, c) : st;
  }
  Product q = {};
  q.mode = kLinGated;
  q.m = m;
  q.n = hidden;
  q.k = k;
  q.a = {X, ldx, false, nullptr};
  q.b = {W, ldw, false, nullptr};
  q.c = H;
  q.ldc = ldh;
  q.act = act;
  q.pre = PRE;
  q.ldp = ldp;
  return run_product(q, c);
}

size_t skg_scratch_size_gated_backward(int64_t m, int64_t hidden) {
  if (m <= 0 || hidden <= 0 || m > kMaxDim || hidden > kMaxDim / 2) return 0;
  return backward_scratch(m, hidden, false).total;
}

skg_status_t skg_gated_backward(int64_t m, int64_t hidden, int64_t k, const void* dH, int64_t lddh,
                                const void* X, int64_t ldx, const void* W, int64_t ldw,
                                const void* PRE, int64_t ldp, int32_t act, void* dX, int64_t lddx,
                                void* dW, int64_t lddw, int32_t dtype, void* workspace,
                                size_t ws_bytes, void* scratch, size_t scratch_bytes,
                                void* stream) {
  skg_status_t st = check_sizes(m, hidden, k, dtype);
  if (st != SKG_OK) return st;
  if (act < SKG_ACT_SILU || act > SKG_ACT_RELU) return SKG_ERR_ARG;
  if (!there(dH, m, hidden, lddh) || !there(X, m, k, ldx) || !there(W, 2 * hidden, k, ldw) ||
      !there(PRE, m, 2 * hidden, ldp) || !there(dX, m, k, lddx) || !there(dW, 2 * hidden, k, lddw))
    return SKG_ERR_ARG;
  if (hidden % 8) return SKG_ERR_UNSUPPORTED;
  if (!aligned(dH, m, hidden, lddh) || !aligned(X, m, k, ldx) || !aligned(W, 2 * hidden, k, ldw) ||
      !aligned(PRE, m, 2 * hidden, ldp) || !aligned(dX, m, k, lddx) ||
      !aligned(dW, 2 * hidden, k, lddw))
    return SKG_ERR_UNSUPPORTED;
  if (k == 0 || (m == 0 && hidden == 0)) return SKG_OK;
  st = check_memory(workspace, ws_bytes, scratch, scratch_bytes,
                    skg_scratch_size_gated_backward(m, hidden));
  if (st != SKG_OK) return st;
  if (any_overlap({rows_of(dX, m, k, lddx), rows_of(dW, 2 * hidden, k, lddw)},
                  {rows_of(dH, m, hidden, lddh), rows_of(X, m, k, ldx),
                   rows_of(W, 2 * hidden, k, ldw), rows_of(PRE, m, 2 * hidden, ldp)}))
    return SKG_ERR_ARG;
  Common c;
  st = common(dtype, workspace, stream, &c);
  if (st != SKG_OK) return st;
  const BackwardScratch s = backward_scratch(m, hidden, false);
  uint8_t* base = (uint8_t*)scratch;
  const bool two = m <= kTwoTermRows;
  if (m > 0 && hidden > 0) {
    DgateParams d = {};
    d.m = m;
    d.f = (int)hidden;
    d.act = act;
    d.dh = dH;
    d.lddh = lddh;
    d.pre = PRE;
    d.ldp = ldp;
    d.dpre = base + s.dpre;
    d.dpre_lo = two ? base + s.dpre_lo : nullptr;
    if (launch_dgate(dtype, d, c.stream) != cudaSuccess) return SKG_ERR_CUDA;
  }
  return in_gradients(m, hidden, k, base + s.dpre, two ? base + s.dpre_lo : nullptr, X, ldx, W, ldw,
                      dX, lddx, dW, lddw, nullptr, c);
}

size_t skg_scratch_size_feed_forward_backward(int64_t m, int64_t hidden) {
  if (m <= 0 || hidden <= 0 || m > kMaxDim || hidden > kMaxDim / 2) return 0;
  return backward_scratch(m, hidden, true).total;
}

skg_status_t skg_feed_forward_backward(int64_t m, int64_t hidden, int64_t k, const void* dY,
                                       int64_t lddy, const void* X, int64_t ldx, const void* W_in,
                                       int64_t ldw_in, const void* W_out, int64_t ldw_out,
                                       const void* PRE, int64_t ldp, int32_t act, void* dX,
                                       int64_t lddx, void* dW_in, int64_t lddw_in, void* dW_out,
                                       int64_t lddw_out, int32_t dtype, void* workspace,
                                       size_t ws_bytes, void* scratch, size_t scratch_bytes,
                                       void* stream) {
  skg_status_t st = check_sizes(m, hidden, k, dtype);
  if (st != SKG_OK) return st;
  if (act < SKG_ACT_SILU || act > SKG_ACT_RELU) return SKG_ERR_ARG;
  if (!there(dY, m, k, lddy) || !there(X, m, k, ldx) || !there(W_in, 2 * hidden, k, ldw_in) ||
      !there(W_out, k, hidden, ldw_out) || !there(PRE, m, 2 * hidden, ldp) ||
      !there(dX, m, k, lddx) || !there(dW_in, 2 * hidden, k, lddw_in) ||
      !there(dW_out, k, hidden, lddw_out))
    return SKG_ERR_ARG;
  if (hidden % 8) return SKG_ERR_UNSUPPORTED;
  if (!aligned(dY, m, k, lddy) || !aligned(X, m, k, ldx) ||
      !aligned(W_in, 2 * hidden, k, ldw_in) || !aligned(W_out, k, hidden, ldw_out) ||
      !aligned(PRE, m, 2 * hidden, ldp) || !aligned(dX, m, k, lddx) ||
      !aligned(dW_in, 2 * hidden, k, lddw_in) || !aligned(dW_out, k, hidden, lddw_out))
    return SKG_ERR_UNSUPPORTED;
  if (k == 0 || (m == 0 && hidden == 0)) return SKG_OK;
  st = check_memory(workspace, ws_bytes, scratch, scratch_bytes,
                    skg_scratch_size_feed_forward_backward(m, hidden));
  if (st != SKG_OK) return st;
  if (any_overlap({rows_of(dX, m, k, lddx), rows_of(dW_in, 2 * hidden, k, lddw_in),
                   rows_of(dW_out, k, hidden, lddw_out)},
                  {rows_of(dY, m, k, lddy), rows_of(X, m, k, ldx),
                   rows_of(W_in, 2 * hidden, k, ldw_in), rows_of(W_out, k, hidden, ldw_out),
                   rows_of(PRE, m, 2 * hidden, ldp)}))
    return SKG_ERR_ARG;
  Common c;
  st = common(dtype, workspace, stream, &c);
  if (st != SKG_OK) return st;
  const BackwardScratch s = backward_scratch(m, hidden, true);
  uint8_t* base = (uint8_t*)scratch;
  const bool two = m <= kTwoTermRows;
  if (m > 0 && hidden > 0) {
    Product q = {};
    q.m = m;
    q.n = hidden;
    q.k = k;
    q.a = {dY, lddy, false, nullptr};
    q.b = {W_out, ldw_out, true, nullptr};
    q.mode = kLinGrad;  // dH stays in the accumulator
    q.act = act;
    q.c = base + s.h;
    q.c_lo = two ? base + s.h_lo : nullptr;
    q.ldc = h_pitch(hidden);
    q.pre = base + s.dpre;
    q.pre_lo = two ? base + s.dpre_lo : nullptr;
    q.ldp = 2 * hidden;
    q.pre_in = PRE;
    q.ldp_in = ldp;
    st = run_product(q, c);
    if (st != SKG_OK) return st;
  }
  Product w = {};
  w.m = k;
  w.n = hidden;
  w.k = m;
  w.a = {dY, lddy, true, nullptr};
  w.b = {base + s.h, h_pitch(hidden), true, two ? base + s.h_lo : nullptr};
  w.c = dW_out;
  w.ldc = lddw_out;
  return in_gradients(m, hidden, k, base + s.dpre, two ? base + s.dpre_lo : nullptr, X, ldx, W_in,
                      ldw_in, dX, lddx, dW_in, lddw_in, &w, c);
}

}  // extern "C"
