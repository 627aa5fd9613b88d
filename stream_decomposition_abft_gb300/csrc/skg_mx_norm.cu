// skg_rmsnorm_mx: h = x + residual, y = h / sqrt(mean(h^2) + eps) * weight,
// quantised to a microscaled format as it is formed; and its gradient,
// skg_rmsnorm_backward.
//
// With xhat = h rstd and u = w dy:
//   dx = rstd (u - xhat mean(u xhat)) + dresidual,   dw = sum over rows of dy xhat.
// The quantised output's rounding counts as the identity in the gradient.
//
// Both are bound by memory: 7 bytes per element forward (x and the residual read,
// their sum and the code written), 8 backward. Measured on GB300, bf16, against
// 6.69 TB/s of a copy: 8192 x 8192 forward 75 us (6.3 TB/s); 4096 x 8192 backward
// 48 us (5.6 TB/s: 43 us for dx and the blocks' dw, the rest for the sum of the 152
// partial dw); one row of 8192 3 us forward. Sums and statistics are fp32. Further from
// that rate: 2048 columns (4096 rows: 14 us forward, 17 backward, 4.3 and 3.9 TB/s),
// where a block's barriers, and backward the rows of partial dw, weigh against few
// elements; more than 8192, where no row is fetched ahead (2048 x 28672: 130 and 246 us,
// 3.2 and 1.9 TB/s); rows off 16-byte boundaries (4096 x 8001: 88 and 87 us, 2.6 and 3.0
// TB/s), whose pieces are fetched twice and leave two bytes a lane.
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "skg_internal.h"
#include "skg_mx.cuh"
#include "skgemm.h"

namespace skg {
namespace {

constexpr int kNormMaxThreads = 512;  // threads of one row

struct NormParams {
  const void* x;
  int64_t ldx;
  const void* res;   // may be NULL
  int64_t ldr;
  const void* w;
  int64_t rows;
  int cols;
  float eps;
  void* sum;         // h, may be NULL; may be x or res
  int64_t lds;
  float* rstd;       // may be NULL
  const float* g;
  uint8_t* codes;
  int64_t ldq;
  uint8_t* scales;
  int x_vec, r_vec, w_vec, s_vec;
};

// 1 / sqrt(ss / n + eps): the product with 1 / n and the approximate root, each with
// one Newton step whose remainder a fused multiply-add gives exactly. About half the
// instructions of a rounded division and root, which every warp runs for every row
// (8192 x 8192: 77 us with those, 75 so), and as near (a code is decided by which side
// of a tie its value falls on). Zero and infinity, also of the sum q + eps alone, as the
// plain root has them.
__device__ __forceinline__ float row_rstd(float ss, float n, float inv_n, float eps) {
  const float q = ss * inv_n;
  const float m = fmaf(fmaf(-q, n, ss), inv_n, q) + eps;
  const float r = rsqrtf(m);
  if (!(m > 0.f && m <= 3.402823466e38f)) return rsqrtf(q + eps);
  const float t = m * r, low = fmaf(m, r, -t);
  return fmaf(0.5f * r, fmaf(-t, r, 1.f) - low * r, r);
}

// Sum over the TPR threads (a power of two) that share a row; every thread
// gets it. `red` holds one float per warp.
__device__ __forceinline__ float row_sum(float v, int log_tpr, float* red) {
  const int width = log_tpr < 5 ? (1 << log_tpr) : 32;
  for (int o = width >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (log_tpr <= 5) return v;
  const int warp = threadIdx.x >> 5, nw = 1 << (log_tpr - 5);
  const int first = warp & ~(nw - 1);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[warp] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < nw; ++i) v += red[first + i];
  return v;
}

// Rows that the kernel below does not take (narrow ones on 16-byte boundaries,
// several to a block; more than 8192 elements): 2^log_tpr threads share a row, V
// chunks of 16 elements each, h in registers between the sum and the quantisation;
// V = 0 (over 32768): any width, h formed twice.
template <typename T, int FMT, int V>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_mx_kernel(NormParams p, int log_tpr) {
  __shared__ float red[kNormMaxThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int tpr = 1 << log_tpr;
  const int t = threadIdx.x & (tpr - 1);
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> log_tpr) + (threadIdx.x >> log_tpr);
  const bool here = row < p.rows;
  const int chunks = (p.cols + 31) / 32 * 2;
  const int groups = (int)mx_groups(p.cols, FMT);
  const float g = FMT == SKG_NVFP4 && p.g ? *p.g : 1.f;
  const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
  const T* r = reinterpret_cast<const T*>(p.res) + row * p.ldr;
  const T* w = reinterpret_cast<const T*>(p.w);
  T* sum = reinterpret_cast<T*>(p.sum) + row * p.lds;

  auto count = [&](int c) {
    const int left = p.cols - c * 16;
    return left >= 16 ? 16 : (left > 0 ? left : 0);
  };
  auto load_h = [&](int c, float (&h)[16]) {
    const int n = here ? count(c) : 0;
    mx_load16(x + c * 16, p.x_vec && n == 16, n, h);
    if (p.res) {
      float q[16];
      mx_load16(r + c * 16, p.r_vec && n == 16, n, q);
#pragma unroll
      for (int i = 0; i < 16; ++i) h[i] += q[i];
    }
  };
  auto finish = [&](int c, float (&h)[16], float rstd) {
    const int n = count(c);
    if (here && p.sum) mx_store16(sum + c * 16, p.s_vec && n == 16, n, h);
    float wv[16];
    mx_load16(w + c * 16, p.w_vec && n == 16, n, wv);
#pragma unroll
    for (int i = 0; i < 16; ++i) h[i] = __fmul_rn(__fmul_rn(h[i], rstd), wv[i]);
    uint4 codes;
    uint32_t word;
    const bool live = here && c < chunks;
    mx_quantize_chunk<FMT>(h, mx_absmax16(h), live, lane, g, codes, word);
    if (live) mx_store_codes16<FMT>(p.codes + row * p.ldq, c, codes);
    constexpr int per = mx_group_chunks(FMT);
    if ((lane & (per - 1)) == 0 && c / per < groups)
      *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, c / per, groups)) = word;
  };

  float ss = 0.f, rstd;
  if constexpr (V > 0) {
    float h[V][16];
#pragma unroll
    for (int j = 0; j < V; ++j) load_h(t + j * tpr, h[j]);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) ss += h[j][i] * h[j][i];
    ss = row_sum(ss, log_tpr, red);
    rstd = row_rstd(ss, (float)p.cols, 1.f / (float)p.cols, p.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) finish(t + j * tpr, h[j], rstd);
  } else {
    float h[16];
    for (int c = t; c < chunks; c += tpr) {
      load_h(c, h);
#pragma unroll
      for (int i = 0; i < 16; ++i) ss += h[i] * h[i];
    }
    ss = row_sum(ss, log_tpr, red);
    rstd = row_rstd(ss, (float)p.cols, 1.f / (float)p.cols, p.eps);
    // Whole strides: every lane takes part in the quantiser's shuffles.
    for (int c0 = 0; c0 < chunks; c0 += tpr) {
      load_h(c0 + t, h);
      finish(c0 + t, h, rstd);
    }
  }
  if (here && p.rstd && t == 0) p.rstd[row] = rstd;
}

// ------------------------------------------------------------------ wide rows
// A block per row at a time. A thread owns the pieces of 8 elements t, t + blockDim,
// ... of every row and fetches the next rows' pieces (off 16-byte boundaries the
// aligned ones that cover them) into a ring of its own in shared memory (cp.async): the
// loads of kNormStages rows are in flight whatever the rows in hand wait for, and no
// other thread reads what a thread has fetched, so the ring needs no barriers.
constexpr int kNormStages = 3;
constexpr int kGradStages = 4;

// Sum over the block; `par` alternates from call to call.
__device__ __forceinline__ float block_sum(float v, float (*red)[kNormMaxThreads / 32], int par) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int nw = (int)blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[par][threadIdx.x >> 5] = v;
  __syncthreads();
  v = (threadIdx.x & 31) < nw ? red[par][threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return __shfl_sync(0xffffffffu, v, 0);
}

template <typename T, int FMT, int V, bool VEC>
__global__ void __launch_bounds__(kNormMaxThreads, 2) rmsnorm_mx_wide_kernel(NormParams p) {
  extern __shared__ uint4 ring[];  // stages x (x, residual) x V x threads
  __shared__ uint4 wbuf[VEC ? 1 : kNormMaxThreads / 32][32];
  __shared__ float red[2][kNormMaxThreads / 32];
  const int t = threadIdx.x, lane = t & 31, nt = blockDim.x;
  const int groups = (int)mx_groups(p.cols, FMT);
  const int pieces = (p.cols + 31) / 32 * 4;
  const int64_t rows_pad = (p.rows + 127) / 128 * 128;
  const T* x = reinterpret_cast<const T*>(p.x);
  const T* res = reinterpret_cast<const T*>(p.res);
  griddep_wait();
  griddep_launch_dependents();
  const float g = FMT == SKG_NVFP4 && p.g ? *p.g : 1.f;
  auto count = [&](int c) { return c + 8 <= p.cols ? 8 : (c < p.cols ? p.cols - c : 0); };
  // Off 16-byte boundaries a thread holds the two aligned pieces around its own.
  constexpr int HELD = VEC ? 1 : 2;
  auto fetch = [&](int64_t row, int st) {
    if (row < p.rows) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (t + j * nt) * 8, n = count(c);
        uint4* dst = ring + ((st * 2) * V * HELD + j) * nt + t;
        if constexpr (VEC) {
          cp_async16(dst, x + row * p.ldx + (n ? c : 0), n ? 16u : 0u);
          if (p.res) cp_async16(dst + V * nt, res + row * p.ldr + (n ? c : 0), n ? 16u : 0u);
        } else {
          const MxRow<T> rx(x + row * p.ldx, p.cols, x);
          rx.fetch(dst, t + j * nt);
          rx.fetch(dst + V * nt, t + j * nt + 1);
          if (p.res) {
            const MxRow<T> rr(res + row * p.ldr, p.cols, res);
            rr.fetch(dst + V * HELD * nt, t + j * nt);
            rr.fetch(dst + V * (HELD + 1) * nt, t + j * nt + 1);
          }
        }
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < kNormStages; ++i)
    fetch((int64_t)blockIdx.x + (int64_t)i * gridDim.x, i);
  uint4 wv[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (t + j * nt) * 8;
    wv[j] = mx_load_raw8(reinterpret_cast<const T*>(p.w) + c, VEC && count(c) == 8, count(c)).q[0];
  }
  const float inv_n = 1.f / (float)p.cols;
  int st = 0, par = 0;
  for (int64_t row = blockIdx.x; row < rows_pad; row += gridDim.x) {
    const bool here = row < p.rows;  // the same for the whole block
    float h[V][8], rstd = 0.f;
    cp_async_wait<kNormStages - 1>();
    if (here) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (t + j * nt) * 8, n = count(c);
        const uint4* src = ring + ((st * 2) * V * HELD + j) * nt + t;
        mx_unpack8<T>(VEC ? src[0]
                          : MxRow<T>(x + row * p.ldx, p.cols, x).elements(src, src + V * nt, n),
                      h[j]);
        if (p.res) {
          float r[8];
          mx_unpack8<T>(VEC ? src[V * nt]
                            : MxRow<T>(res + row * p.ldr, p.cols, res)
                                  .elements(src + V * HELD * nt, src + V * (HELD + 1) * nt, n),
                        r);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[j][i] += r[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += h[j][i] * h[j][i];
      }
      rstd = row_rstd(block_sum(ss, red, par), (float)p.cols, inv_n, p.eps);
      par ^= 1;
      if (p.rstd && t == 0) p.rstd[row] = rstd;
    }
    fetch(row + (int64_t)kNormStages * gridDim.x, st);
    if (++st == kNormStages) st = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * nt;
      const bool live = here && c < pieces;
      if (here && p.sum) {
        T* out = reinterpret_cast<T*>(p.sum) + row * p.lds;
        if constexpr (VEC) {
          if (c * 8 < p.cols) *reinterpret_cast<uint4*>(out + c * 8) = mx_pack8<T>(h[j]);
        } else {
          const int c0 = (c - lane) * 8;
          mx_warp_store8(out + c0, p.cols - c0, mx_pack8<T>(h[j]), wbuf[t >> 5], lane);
        }
      }
      float w[8], y[8];
      mx_unpack8<T>(wv[j], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = here ? __fmul_rn(__fmul_rn(h[j][i], rstd), w[i]) : 0.f;
      uint2 codes;
      uint32_t word;
      mx_quantize_piece<FMT>(y, live, lane, g, codes, word);
      if (live) {
        mx_store_codes8<FMT>(p.codes + row * p.ldq, c, codes);
      }
      constexpr int per = 2 * mx_group_chunks(FMT);
      if ((lane & (per - 1)) == 0 && c / per < groups)
        *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, c / per, groups)) = word;
    }
  }
}

template <typename T, int FMT>
cudaError_t launch_norm_wide(const NormParams& p, int v, int threads, bool vec, int sms,
                             cudaStream_t stream) {
  const size_t smem = (size_t)kNormStages * 2 * v * threads * 16 * (vec ? 1 : 2);
  const int64_t rows = (p.rows + 127) / 128 * 128;
  // 1024 threads per SM: two blocks of 512, four of 256 (4096 x 2048: 15 us with
  // two of 256). The double ring of rows off 16-byte boundaries lets three of 256 fit:
  // the last quarter of the blocks starts when the others end (4096 x 2001: 23 us).
  const int64_t most = (int64_t)sms * (1024 / threads < 8 ? 1024 / threads : 8);
  const dim3 grid((unsigned)(rows < most ? rows : most));
  auto run = [&](auto kernel, std::atomic<uint64_t>& done) {
    const cudaError_t e = opt_in_smem((const void*)kernel, done,
                                      kNormStages * 2 * 2 * kNormMaxThreads * 16 * (vec ? 1 : 2));
    return e != cudaSuccess ? e : launch_pdl(kernel, grid, dim3(threads), smem, stream, p);
  };
  static std::atomic<uint64_t> d[4] = {};
  if (v == 1)
    return vec ? run(rmsnorm_mx_wide_kernel<T, FMT, 1, true>, d[0])
               : run(rmsnorm_mx_wide_kernel<T, FMT, 1, false>, d[1]);
  return vec ? run(rmsnorm_mx_wide_kernel<T, FMT, 2, true>, d[2])
             : run(rmsnorm_mx_wide_kernel<T, FMT, 2, false>, d[3]);
}

template <typename T, int FMT>
cudaError_t launch_norm(const NormParams& p, int sms, cudaStream_t stream) {
  // Rows of up to 8192 elements: a block per row with its ring. (Narrow ones on
  // 16-byte boundaries share a block; wider ones need more registers.)
  const int pieces = (p.cols + 31) / 32 * 4;
  const bool vec = p.x_vec && p.w_vec && (!p.res || p.r_vec) && (!p.sum || p.s_vec) &&
                   p.cols % 8 == 0;
  if (pieces <= 2 * kNormMaxThreads && (pieces > 96 || !vec)) {
    const int threads = pieces <= kNormMaxThreads ? (pieces + 31) / 32 * 32
                                                  : (pieces + 63) / 64 * 32;
    return launch_norm_wide<T, FMT>(p, pieces <= kNormMaxThreads ? 1 : 2, threads, vec, sms,
                                    stream);
  }
  const int chunks = (p.cols + 31) / 32 * 2;
  int log_tpr = 3;
  while ((1 << log_tpr) < chunks && (1 << log_tpr) < kNormMaxThreads) ++log_tpr;
  const int v = (chunks + (1 << log_tpr) - 1) >> log_tpr;
  const int threads = log_tpr < 7 ? 128 : (1 << log_tpr);
  const int per = threads >> log_tpr;
  const int64_t rows = (p.rows + 127) / 128 * 128;  // the scale tiles' rows
  const dim3 grid((unsigned)(rows / per));
  if (v <= 1)
    return launch_pdl(rmsnorm_mx_kernel<T, FMT, 1>, grid, dim3(threads), 0, stream, p, log_tpr);
  if (v <= 2)
    return launch_pdl(rmsnorm_mx_kernel<T, FMT, 2>, grid, dim3(threads), 0, stream, p, log_tpr);
  if (v <= 4)
    return launch_pdl(rmsnorm_mx_kernel<T, FMT, 4>, grid, dim3(threads), 0, stream, p, log_tpr);
  return launch_pdl(rmsnorm_mx_kernel<T, FMT, 0>, grid, dim3(threads), 0, stream, p, log_tpr);
}

template <typename T>
cudaError_t launch_norm_fmt(const NormParams& p, int fmt, int sms, cudaStream_t stream) {
  if (fmt == SKG_MXFP8) return launch_norm<T, SKG_MXFP8>(p, sms, stream);
  if (fmt == SKG_MXFP4) return launch_norm<T, SKG_MXFP4>(p, sms, stream);
  return launch_norm<T, SKG_NVFP4>(p, sms, stream);
}

// ------------------------------------------------------------------ gradient
struct GradParams {
  const void* dy;
  int64_t lddy;
  const void* h;
  int64_t ldh;
  const void* w;
  const float* rstd;
  const void* dres;  // may be NULL
  int64_t lddr;
  int64_t rows;
  int cols;
  void* dx;
  int64_t lddx;
  float* partial;    // gridDim.x x cols: dw of each block's rows
  int vec;           // every row is 16-byte aligned
};

// Rows of more than 8192 elements: a row at a time per block of 512 threads, V
// chunks of 16 elements each, in registers between the sum and dx; V = 0 (over 16384):
// any width, the row read twice (and once more for dw by rmsnorm_grad_columns_kernel).
template <typename T, int V>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_grad_long_kernel(GradParams p) {
  __shared__ float red[2][kNormMaxThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x;
  const int chunks = (p.cols + 15) / 16;
  const T* w = reinterpret_cast<const T*>(p.w);
  const float inv_n = 1.f / (float)p.cols;
  auto count = [&](int c) {
    const int left = p.cols - c * 16;
    return left >= 16 ? 16 : (left > 0 ? left : 0);
  };
  constexpr int VV = V > 0 ? V : 1;
  float acc[VV][16];
#pragma unroll
  for (int j = 0; j < VV; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0.f;
  int par = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, par ^= 1) {
    const T* dy = reinterpret_cast<const T*>(p.dy) + row * p.lddy;
    const T* h = reinterpret_cast<const T*>(p.h) + row * p.ldh;
    const T* dr = reinterpret_cast<const T*>(p.dres) + row * p.lddr;
    T* dx = reinterpret_cast<T*>(p.dx) + row * p.lddx;
    const float rstd = p.rstd[row];
    float dot = 0.f;
    auto load = [&](int c, float (&a)[16], float (&b)[16]) {  // dy; xhat
      const int n = count(c);
      mx_load16(dy + c * 16, p.vec && n == 16, n, a);
      mx_load16(h + c * 16, p.vec && n == 16, n, b);
#pragma unroll
      for (int i = 0; i < 16; ++i) b[i] *= rstd;
    };
    auto weigh = [&](int c, float (&a)[16]) {  // dy -> w dy
      const int n = count(c);
      float u[16];
      mx_load16(w + c * 16, p.vec && n == 16, n, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i] *= u[i];
    };
    auto store = [&](int c, const float (&b)[16], const float (&u)[16], float mean) {
      const int n = count(c);
      float o[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = 0.f;
      if (p.dres) mx_load16(dr + c * 16, p.vec && n == 16, n, o);
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] += rstd * (u[i] - b[i] * mean);
      mx_store16(dx + c * 16, p.vec && n == 16, n, o);
    };
    if constexpr (V > 0) {
      float a[V][16], b[V][16];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        load(t + j * kNormMaxThreads, a[j], b[j]);
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][i] += a[j][i] * b[j][i];
        weigh(t + j * kNormMaxThreads, a[j]);
#pragma unroll
        for (int i = 0; i < 16; ++i) dot += a[j][i] * b[j][i];
      }
      const float mean = block_sum(dot, red, par) * inv_n;
#pragma unroll
      for (int j = 0; j < V; ++j) store(t + j * kNormMaxThreads, b[j], a[j], mean);
    } else {
      float a[16], b[16];
      for (int c = t; c < chunks; c += kNormMaxThreads) {
        load(c, a, b);
        weigh(c, a);
#pragma unroll
        for (int i = 0; i < 16; ++i) dot += a[i] * b[i];
      }
      const float mean = block_sum(dot, red, par) * inv_n;
      for (int c = t; c < chunks; c += kNormMaxThreads) {
        load(c, a, b);
        weigh(c, a);
        store(c, b, a, mean);
      }
    }
  }
  if constexpr (V > 0) {
    float* out = p.partial + (int64_t)blockIdx.x * p.cols;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = t + j * kNormMaxThreads, n = count(c);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) out[c * 16 + i] = acc[j][i];
    }
  }
}

// The gradient of rows of up to 8192 elements, with the same ring for dy, h and
// dresidual (off 16-byte boundaries and over 4096 elements a thread also reads the next
// one's piece, behind a barrier). A block takes two rows at a time: the first pass over
// the fetched pieces forms both rows' sums, which cross the block together (a row's sum,
// barriers and all, takes longer than its arithmetic: 4096 x 8192 one row at a time
// 46 us), the second reads them again from shared memory for dx. dw of the block's rows
// stays in registers.
template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(kNormMaxThreads, 1) rmsnorm_grad_wide_kernel(GradParams p) {
  extern __shared__ uint4 ring[];  // stages x (dy, h, dres) x V x threads
  __shared__ float2 red[2][kNormMaxThreads / 32];
  __shared__ uint4 wbuf[VEC ? 1 : kNormMaxThreads / 32][32];
  static_assert(kGradStages == 4, "two rows in hand, two on the way");
  const int t = threadIdx.x, nt = blockDim.x, lane = t & 31;
  const T* in[3] = {reinterpret_cast<const T*>(p.dy), reinterpret_cast<const T*>(p.h),
                    reinterpret_cast<const T*>(p.dres)};
  const int64_t ld[3] = {p.lddy, p.ldh, p.lddr};
  auto count = [&](int c) { return c + 8 <= p.cols ? 8 : (c < p.cols ? p.cols - c : 0); };
  // Pieces of a thread's eight elements in the ring: off 16-byte boundaries the two
  // aligned ones that hold them, or (V = 2: no room) one of its own and the next
  // thread's.
  constexpr bool SHARE = !VEC && V == 2;
  constexpr int HELD = VEC || SHARE ? 1 : 2;
  const int slot = V * HELD * nt + (SHARE ? 1 : 0);
  auto piece = [&](int k, int64_t row, int st, int j) -> uint4 {
    const uint4* src = ring + (st * 3 + k) * slot + j * nt + t;
    if constexpr (VEC) return src[0];
    else return MxRow<T>(in[k] + row * ld[k], p.cols, in[k])
        .elements(src, src + (SHARE ? 1 : nt), count((t + j * nt) * 8));
  };
  griddep_wait();
  griddep_launch_dependents();
  auto fetch = [&](int64_t row, int st) {
    if (row < p.rows) {
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        if (k == 2 && !p.dres) break;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (t + j * nt) * 8;
          uint4* dst = ring + (st * 3 + k) * slot + j * nt + t;
          const int n = count(c);
          if constexpr (VEC) {
            cp_async16(dst, in[k] + row * ld[k] + (n ? c : 0), n ? 16u : 0u);
          } else {
            const MxRow<T> r(in[k] + row * ld[k], p.cols, in[k]);
            r.fetch(dst, t + j * nt);
            if (!SHARE) r.fetch(dst + nt, t + 1);
            else if (j == 0 && t == 0) r.fetch(dst + V * nt, V * nt);
          }
        }
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < kGradStages; ++i)
    fetch((int64_t)blockIdx.x + (int64_t)i * gridDim.x, i);
  uint4 wv[V];
  float acc[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (t + j * nt) * 8;
    wv[j] = mx_load_raw8(reinterpret_cast<const T*>(p.w) + c, VEC && count(c) == 8, count(c)).q[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.f;
  }
  const float inv_n = 1.f / (float)p.cols;
  int st = 0, par = 0;
  float next[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int64_t r = blockIdx.x + (int64_t)q * gridDim.x;
    next[q] = r < p.rows ? p.rstd[r] : 0.f;
  }
  for (int64_t row = blockIdx.x; row < p.rows; row += 2 * (int64_t)gridDim.x) {
    float rstd[2], dot[2] = {0.f, 0.f};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      rstd[q] = next[q];
      const int64_t r = row + (int64_t)(2 + q) * gridDim.x;
      next[q] = r < p.rows ? p.rstd[r] : 0.f;
    }
    cp_async_wait<kGradStages - 2>();
    if constexpr (SHARE) __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      if (row + (int64_t)q * gridDim.x >= p.rows) break;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int64_t r = row + (int64_t)q * gridDim.x;
        float dy[8], h[8], w[8];
        mx_unpack8<T>(piece(0, r, st + q, j), dy);
        mx_unpack8<T>(piece(1, r, st + q, j), h);
        mx_unpack8<T>(wv[j], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = dy[i] * (h[i] * rstd[q]);
          acc[j][i] += a;
          dot[q] += a * w[i];
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      dot[0] += __shfl_xor_sync(0xffffffffu, dot[0], o);
      dot[1] += __shfl_xor_sync(0xffffffffu, dot[1], o);
    }
    if (lane == 0) red[par][t >> 5] = make_float2(dot[0], dot[1]);
    __syncthreads();
    float2 part = lane < (nt >> 5) ? red[par][lane] : make_float2(0.f, 0.f);
    par ^= 1;
#pragma unroll
    for (int o = kNormMaxThreads / 64; o > 0; o >>= 1) {
      part.x += __shfl_xor_sync(0xffffffffu, part.x, o);
      part.y += __shfl_xor_sync(0xffffffffu, part.y, o);
    }
    const float mean[2] = {__shfl_sync(0xffffffffu, part.x, 0) * inv_n,
                           __shfl_sync(0xffffffffu, part.y, 0) * inv_n};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int64_t r = row + (int64_t)q * gridDim.x;
      if (r < p.rows) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = (t + j * nt) * 8;
          float dy[8], h[8], w[8], o[8];
          mx_unpack8<T>(piece(0, r, st + q, j), dy);
          mx_unpack8<T>(piece(1, r, st + q, j), h);
          mx_unpack8<T>(wv[j], w);
          if (p.dres) {
            mx_unpack8<T>(piece(2, r, st + q, j), o);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            o[i] += rstd[q] * (w[i] * dy[i] - h[i] * rstd[q] * mean[q]);
          T* out = reinterpret_cast<T*>(p.dx) + r * p.lddx;
          if constexpr (VEC) {
            if (c < p.cols) *reinterpret_cast<uint4*>(out + c) = mx_pack8<T>(o);
          } else {
            const int c0 = c - lane * 8;
            mx_warp_store8(out + c0, p.cols - c0, mx_pack8<T>(o), wbuf[t >> 5], lane);
          }
        }
      }
      if constexpr (!SHARE) fetch(r + (int64_t)kGradStages * gridDim.x, st + q);
    }
    if constexpr (SHARE) {
      __syncthreads();  // the threads before have read their second pieces
      fetch(row + (int64_t)kGradStages * gridDim.x, st);
      fetch(row + (int64_t)(kGradStages + 1) * gridDim.x, st + 1);
    }
    st ^= 2;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (t + j * nt) * 8;
    mx_store8(p.partial + (int64_t)blockIdx.x * p.cols + c, VEC && count(c) == 8, count(c), acc[j]);
  }
}

// dw of a block's rows, for widths whose sums do not fit the row kernel's
// registers: a thread per column.
template <typename T>
__global__ void __launch_bounds__(256) rmsnorm_grad_columns_kernel(GradParams p, int parts) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float acc = 0.f;
  for (int64_t row = blockIdx.y; row < p.rows; row += parts)
    acc += mx_to_f32(reinterpret_cast<const T*>(p.dy)[row * p.lddy + c]) *
           (mx_to_f32(reinterpret_cast<const T*>(p.h)[row * p.ldh + c]) * p.rstd[row]);
  p.partial[(int64_t)blockIdx.y * p.cols + c] = acc;
}

// dw = the sum of the blocks' partials, in a fixed order: 32 columns per block,
// 32 rows of threads over the partials, four loads in flight each.
__global__ void __launch_bounds__(1024)
rmsnorm_grad_reduce_kernel(const float* partial, int parts, int cols, float* dw) {
  __shared__ float s[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + tx;
  float v = 0.f;
  if (c < cols) {
    const float* src = partial + c;
    for (int i = ty; i < parts; i += 128) {
      float u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = i + 32 * j < parts ? src[(int64_t)(i + 32 * j) * cols] : 0.f;
      v += (u[0] + u[1]) + (u[2] + u[3]);
    }
  }
  s[ty][tx] = v;
  __syncthreads();
  // Warp ty sums column ty of the block.
  v = s[tx][ty];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (tx == 0 && blockIdx.x * 32 + ty < cols) dw[blockIdx.x * 32 + ty] = v;
}

struct GradPlan {
  int v;        // pieces or chunks of a thread
  int threads;  // of rmsnorm_grad_wide_kernel; 0: rmsnorm_grad_long_kernel (512)
  int blocks;
};

GradPlan grad_plan(int64_t rows, int64_t cols, int sms) {
  GradPlan g;
  const int64_t pieces = (cols + 7) / 8, n = sms > 0 ? sms : 152;
  int64_t most = n;
  if (pieces <= 2 * kNormMaxThreads) {
    g.v = pieces <= kNormMaxThreads ? 1 : 2;
    g.threads = (int)((pieces + 32 * g.v - 1) / (32 * g.v) * 32);
    // Blocks of few threads share an SM; each adds a row of partial sums to reduce (4096 x
    // 2048: two 20.4, three 17.1, four 19.5 us). Off 16-byte boundaries two of 192 to 256
    // threads fit with their double rings, and the rest start later (4096 x 2001: 34 us).
    most = g.threads <= 64 ? 4 * n : (g.threads <= 256 ? 3 * n : n);
  } else {
    const int64_t chunks = (cols + 15) / 16, v = (chunks + kNormMaxThreads - 1) / kNormMaxThreads;
    g.v = v <= 2 ? 2 : 0;
    g.threads = 0;
  }
  g.blocks = (int)(rows < most ? rows : most);
  return g;
}

template <typename T>
cudaError_t launch_grad(const GradParams& p, const GradPlan& g, float* dw, cudaStream_t stream) {
  cudaError_t e;
  const dim3 grid(g.blocks), wide(g.threads), block(kNormMaxThreads);
  const bool vec = p.vec && p.cols % 8 == 0;
  if (g.threads) {
    // Off 16-byte boundaries two pieces a thread, or one and one more per row.
    const int pieces = vec ? g.v * g.threads : 2 * g.threads + (g.v == 2 ? 1 : 0);
    const size_t smem = (size_t)kGradStages * 3 * pieces * 16;
    auto run = [&](auto kernel, std::atomic<uint64_t>& done) {
      const cudaError_t r = opt_in_smem((const void*)kernel, done,
                                        kGradStages * 3 * (2 * kNormMaxThreads + 1) * 16);
      return r != cudaSuccess ? r : launch_pdl(kernel, grid, wide, smem, stream, p);
    };
    static std::atomic<uint64_t> d[4] = {};
    if (g.v == 1)
      e = vec ? run(rmsnorm_grad_wide_kernel<T, 1, true>, d[0])
              : run(rmsnorm_grad_wide_kernel<T, 1, false>, d[1]);
    else
      e = vec ? run(rmsnorm_grad_wide_kernel<T, 2, true>, d[2])
              : run(rmsnorm_grad_wide_kernel<T, 2, false>, d[3]);
  } else if (g.v == 2) {
    e = launch_pdl(rmsnorm_grad_long_kernel<T, 2>, grid, block, 0, stream, p);
  } else {
    // dw first: dx may take dy's place.
    e = launch_pdl(rmsnorm_grad_columns_kernel<T>,
                   dim3((unsigned)((p.cols + 255) / 256), (unsigned)g.blocks), dim3(256), 0,
                   stream, p, g.blocks);
    if (e != cudaSuccess) return e;
    e = launch_pdl(rmsnorm_grad_long_kernel<T, 0>, grid, block, 0, stream, p);
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(rmsnorm_grad_reduce_kernel, dim3((unsigned)((p.cols + 31) / 32)), dim3(1024), 0,
                    stream, (const float*)p.partial, g.blocks, p.cols, dw);
}

bool vec_rows(const void* p, int64_t ld) {
  return ((uintptr_t)p & 15) == 0 && (ld * 2) % 16 == 0;
}

}  // namespace
}  // namespace skg

using namespace skg;

extern "C" {

skg_status_t skg_rmsnorm_mx(int64_t rows, int64_t cols, const void* X, int64_t ldx,
                            const void* residual, int64_t ldr, const void* weight, int32_t type,
                            float eps, void* sum, int64_t lds, float* rstd, int32_t format,
                            const float* tensor_scale, void* codes, int64_t ldq, void* scales,
                            void* stream) {
  if (rows < 0 || cols < 0 || !(eps >= 0.f)) return SKG_ERR_ARG;
  if (type != SKG_IN_F16 && type != SKG_IN_BF16) return SKG_ERR_ARG;
  if (format < SKG_MXFP8 || format > SKG_NVFP4) return SKG_ERR_ARG;
  if (rows == 0 || (cols == 0 && !rstd)) return SKG_OK;
  if (cols == 0) {  // the mean over no elements is NaN: all bits set
    if (rows > INT32_MAX / 4 || ((uintptr_t)rstd & 3)) return SKG_ERR_UNSUPPORTED;
    return cudaMemsetAsync(rstd, 0xff, (size_t)rows * 4, (cudaStream_t)stream) == cudaSuccess
               ? SKG_OK
               : SKG_ERR_CUDA;
  }
  if (!X || !weight || !codes || !scales || ldx < cols || (residual && ldr < cols) ||
      (sum && lds < cols) || ldq < skg_mx_codes_ld(cols, format))
    return SKG_ERR_ARG;
  if (cols > INT32_MAX / 4 || rows > INT32_MAX / 4) return SKG_ERR_UNSUPPORTED;
  if (((uintptr_t)codes & 15) || (ldq & 15) || ((uintptr_t)scales & 15) || ((uintptr_t)X & 1) ||
      ((uintptr_t)residual & 1) || ((uintptr_t)weight & 1) || ((uintptr_t)sum & 1) ||
      ((uintptr_t)rstd & 3) || ((uintptr_t)tensor_scale & 3))
    return SKG_ERR_UNSUPPORTED;
  NormParams p;
  p.x = X;
  p.ldx = ldx;
  p.res = residual;
  p.ldr = ldr;
  p.w = weight;
  p.rows = rows;
  p.cols = (int)cols;
  p.eps = eps;
  p.sum = sum;
  p.lds = lds;
  p.rstd = rstd;
  p.g = tensor_scale;
  p.codes = (uint8_t*)codes;
  p.ldq = ldq;
  p.scales = (uint8_t*)scales;
  p.x_vec = vec_rows(X, ldx);
  p.r_vec = vec_rows(residual, ldr);
  p.w_vec = ((uintptr_t)weight & 15) == 0;
  p.s_vec = vec_rows(sum, lds);
  cudaStream_t st = (cudaStream_t)stream;
  const int sms = skg_device_sm_count();
  if (sms <= 0) return SKG_ERR_CUDA;
  const cudaError_t e = type == SKG_IN_F16 ? launch_norm_fmt<__half>(p, format, sms, st)
                                           : launch_norm_fmt<__nv_bfloat16>(p, format, sms, st);
  return e == cudaSuccess ? SKG_OK : SKG_ERR_CUDA;
}

size_t skg_workspace_size_rmsnorm_backward(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  const GradPlan g = grad_plan(rows, cols, skg_device_sm_count());
  return (size_t)g.blocks * (size_t)cols * 4;
}

skg_status_t skg_rmsnorm_backward(int64_t rows, int64_t cols, const void* dY, int64_t lddy,
                                  const void* H, int64_t ldh, const void* weight,
                                  const float* rstd, const void* dresidual, int64_t lddr,
                                  int32_t type, void* dX, int64_t lddx, float* dweight,
                                  void* workspace, size_t ws_bytes, void* stream) {
  if (rows < 0 || cols < 0) return SKG_ERR_ARG;
  if (type != SKG_IN_F16 && type != SKG_IN_BF16) return SKG_ERR_ARG;
  if (cols == 0) return SKG_OK;
  if (!dweight) return SKG_ERR_ARG;
  if (cols > INT32_MAX / 4 || rows > INT32_MAX / 4) return SKG_ERR_UNSUPPORTED;
  if ((uintptr_t)dweight & 3) return SKG_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0)  // an empty sum
    return launch_pdl(rmsnorm_grad_reduce_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024),
                      0, st, (const float*)nullptr, 0, (int)cols, dweight) == cudaSuccess
               ? SKG_OK
               : SKG_ERR_CUDA;
  if (!dY || !H || !weight || !rstd || !dX || lddy < cols || ldh < cols || lddx < cols ||
      (dresidual && lddr < cols))
    return SKG_ERR_ARG;
  if (((uintptr_t)dY & 1) || ((uintptr_t)H & 1) || ((uintptr_t)weight & 1) ||
      ((uintptr_t)dX & 1) || ((uintptr_t)dresidual & 1) || ((uintptr_t)rstd & 3))
    return SKG_ERR_UNSUPPORTED;
  const int sms = skg_device_sm_count();
  if (sms <= 0) return SKG_ERR_CUDA;
  const GradPlan g = grad_plan(rows, cols, sms);
  if (!workspace || ((uintptr_t)workspace & 255) ||
      ws_bytes < skg_workspace_size_rmsnorm_backward(rows, cols))
    return SKG_ERR_WORKSPACE;
  GradParams p;
  p.dy = dY;
  p.lddy = lddy;
  p.h = H;
  p.ldh = ldh;
  p.w = weight;
  p.rstd = rstd;
  p.dres = dresidual;
  p.lddr = lddr;
  p.rows = rows;
  p.cols = (int)cols;
  p.dx = dX;
  p.lddx = lddx;
  p.partial = (float*)workspace;
  p.vec = vec_rows(dY, lddy) && vec_rows(H, ldh) && vec_rows(dX, lddx) &&
          ((uintptr_t)weight & 15) == 0 && (!dresidual || vec_rows(dresidual, lddr));
  const cudaError_t e = type == SKG_IN_F16 ? launch_grad<__half>(p, g, dweight, st)
                                           : launch_grad<__nv_bfloat16>(p, g, dweight, st);
  return e == cudaSuccess ? SKG_OK : SKG_ERR_CUDA;
}

}  // extern "C"
