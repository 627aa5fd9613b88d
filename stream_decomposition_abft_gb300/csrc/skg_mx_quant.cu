// skg_mx_quantize: a matrix to a microscaled format, along its rows or along
// its columns (the transposed operand of a gradient), with the values that
// the codes stand for on request.
//
// Every element is read once and every code, scale and value is written once;
// the kernels are bound by memory.
#include <cuda_runtime.h>
#include <stdint.h>

#include "skg_internal.h"
#include "skg_mx.cuh"
#include "skgemm.h"

namespace skg {
namespace {

constexpr int kQThreads = 256;

struct QuantParams {
  const void* x;
  int64_t ldx;
  int64_t rows, k;         // of the quantised matrix
  const float* g;          // nvfp4: the matrix's fp32 scale (NULL = 1)
  uint8_t* codes;
  int64_t ldq;             // bytes
  uint8_t* scales;
  void* values;            // NULL: not wanted
  int64_t ldv;
  int x_vec, v_vec;        // 16-byte aligned rows
};

// Along the rows. A thread takes 16 consecutive elements; a warp 32 / TX rows
// of TX chunks (TX a power of two of at least 8, so that the lanes of a block
// group sit together). A block of 256 threads takes the rows 32 q + l of one
// scale tile for l in a range of TY / 4: the 16 bytes of scales of each l are
// then written together. Rows past the end only write their zero scales.
template <typename T, int FMT>
__global__ void __launch_bounds__(kQThreads) mx_quantize_rows_kernel(QuantParams p, int log_tx) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int tx = threadIdx.x & ((1 << log_tx) - 1);
  const int ty = threadIdx.x >> log_tx;
  const int ls = (kQThreads >> log_tx) / 4;  // l values of a block
  const int64_t chunk = ((int64_t)blockIdx.x << log_tx) + tx;
  const int64_t chunks = (p.k + 31) / 32 * 2;
  const int groups = (int)mx_groups(p.k, FMT);
  const float g = FMT == SKG_NVFP4 && p.g ? *p.g : 1.f;
  const bool live = chunk < chunks;
  const int64_t left = p.k - chunk * 16;
  const int n = left >= 16 ? 16 : (left > 0 ? (int)left : 0);
  const int64_t tiles = (p.rows + 127) / 128 * 32;  // (scale tile, l) pairs
  for (int64_t u = (int64_t)blockIdx.y * ls; u < tiles; u += (int64_t)gridDim.y * ls) {
    const int64_t ul = u + (ty >> 2);
    const int64_t row = (ul >> 5) * 128 + (ty & 3) * 32 + (ul & 31);
    const bool here = row < p.rows;
    float v[16];
    const T* src = reinterpret_cast<const T*>(p.x) + row * p.ldx + chunk * 16;
    mx_load16(src, here && p.x_vec && n == 16, here ? n : 0, v);
    uint4 codes;
    uint32_t word;
    const MxScale s = mx_quantize_chunk<FMT>(v, here && live, lane, g, codes, word);
    if (here && live) {
      mx_store_codes16<FMT>(p.codes + row * p.ldq, chunk, codes);
      if (p.values) {
        float w[16];
        mx_values16<FMT>(codes, s, g, w);
        mx_store16(reinterpret_cast<T*>(p.values) + row * p.ldv + chunk * 16, p.v_vec && n == 16,
                   n, w);
      }
    }
    constexpr int per = mx_group_chunks(FMT);
    const int64_t grp = chunk / per;
    if ((lane & (per - 1)) == 0 && grp < groups)
      *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, (int)grp, groups)) = word;
  }
}

// Along the columns: X is stored k x rows. A block stages 128 lines of 64
// columns in shared memory; a thread then takes 32 consecutive k of one
// column. Consecutive lanes hold consecutive k ranges of a column, so codes and
// values leave in whole lines; the words of a line are XORed with the line's
// k range, so that those lanes read different banks.
constexpr int kTK = 128, kTC = 64;

template <typename T, int FMT>
__global__ void __launch_bounds__(kQThreads) mx_quantize_cols_kernel(QuantParams p) {
  constexpr int EW = 16 / (int)sizeof(T);         // elements per 16 bytes
  constexpr int VECS = kTC / EW;                  // 16-byte pieces of a line
  constexpr int XOR = 8 * (int)sizeof(T) / 16;    // 16-byte pieces of 8 columns
  __shared__ __align__(16) T tile[kTK * kTC];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t k0 = (int64_t)blockIdx.x * kTK, c0 = (int64_t)blockIdx.y * kTC;
  const T* x = reinterpret_cast<const T*>(p.x);
  for (int i = threadIdx.x; i < kTK * VECS; i += kQThreads) {
    const int line = i / VECS, piece = i % VECS;
    const int64_t kk = k0 + line, c = c0 + piece * EW;
    uint4 u = make_uint4(0u, 0u, 0u, 0u);
    if (kk < p.k) {
      const T* src = x + kk * p.ldx + c;
      if (p.x_vec && c + EW <= p.rows) {
        u = *reinterpret_cast<const uint4*>(src);
      } else {
        T* e = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int j = 0; j < EW; ++j)
          if (c + j < p.rows) e[j] = src[j];
      }
    }
    reinterpret_cast<uint4*>(tile)[line * VECS + (piece ^ ((line >> 5) * XOR))] = u;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int kb = lane & 3, col = (threadIdx.x >> 5) * 8 + (lane >> 2);
  const int piece = (col / EW) ^ (kb * XOR);
  const int64_t row = c0 + col;
  const bool here = row < p.rows;
  const int64_t kfirst = k0 + kb * 32;
  const bool live = here && kfirst < p.k;
  const float g = FMT == SKG_NVFP4 && p.g ? *p.g : 1.f;
  float v[2][16];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      v[h][i] = mx_to_f32(tile[(kb * 32 + h * 16 + i) * kTC + piece * EW + col % EW]);
  uint32_t amax[2] = {mx_absmax16(v[0]), mx_absmax16(v[1])};
  if constexpr (FMT != SKG_NVFP4) amax[0] = amax[1] = max(amax[0], amax[1]);
  MxScale s[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    s[h] = mx_scale<FMT>(amax[h], g);
    if (live) {
      const uint4 codes = mx_codes16<FMT>(v[h], s[h]);
      mx_store_codes16<FMT>(p.codes + row * p.ldq, kfirst / 16 + h, codes);
      if (p.values) {
        float w[16];
        mx_values16<FMT>(codes, s[h], g, w);
        const int64_t left = p.k - (kfirst + h * 16);
        const int n = left >= 16 ? 16 : (left > 0 ? (int)left : 0);
        mx_store16(reinterpret_cast<T*>(p.values) + row * p.ldv + kfirst + h * 16,
                   p.v_vec && n == 16, n, w);
      }
    }
  }
  const int groups = (int)mx_groups(p.k, FMT);
  uint32_t word;
  if constexpr (FMT == SKG_NVFP4) {
    word = live ? (s[0].byte | (s[1].byte << 8)) << (16 * (kb & 1)) : 0u;
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    const int64_t grp = (k0 / 64) + (kb >> 1);
    if ((kb & 1) == 0 && grp < groups)
      *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, (int)grp, groups)) = word;
  } else {
    word = live ? s[0].byte << (8 * kb) : 0u;
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    const int64_t grp = k0 / 128;
    if (kb == 0 && grp < groups)
      *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, (int)grp, groups)) = word;
  }
}

template <typename T, int FMT>
cudaError_t launch_quantize(const QuantParams& p, bool transpose, cudaStream_t stream) {
  if (transpose) {
    const int64_t gx = (p.k + kTK - 1) / kTK, gy = (p.rows + 127) / 128 * 2;
    if (gy > 65535) return cudaErrorInvalidValue;
    return launch_pdl(mx_quantize_cols_kernel<T, FMT>, dim3((unsigned)gx, (unsigned)gy),
                      dim3(kQThreads), 0, stream, p);
  }
  const int64_t chunks = (p.k + 31) / 32 * 2;
  int log_tx = 3;
  while (log_tx < 5 && (1 << log_tx) < chunks) ++log_tx;
  const int ls = (kQThreads >> log_tx) / 4;
  const int64_t gx = (chunks + (1 << log_tx) - 1) >> log_tx;
  int64_t gy = ((p.rows + 127) / 128 * 32 + ls - 1) / ls;
  if (gy > 65535) gy = 65535;
  return launch_pdl(mx_quantize_rows_kernel<T, FMT>, dim3((unsigned)gx, (unsigned)gy),
                    dim3(kQThreads), 0, stream, p, log_tx);
}

template <typename T>
cudaError_t launch_quantize_fmt(const QuantParams& p, int fmt, bool transpose,
                                cudaStream_t stream) {
  if (fmt == SKG_MXFP8) return launch_quantize<T, SKG_MXFP8>(p, transpose, stream);
  if (fmt == SKG_MXFP4) return launch_quantize<T, SKG_MXFP4>(p, transpose, stream);
  return launch_quantize<T, SKG_NVFP4>(p, transpose, stream);
}

}  // namespace
}  // namespace skg

using namespace skg;

extern "C" {

int64_t skg_mx_codes_ld(int64_t k, int32_t format) {
  if (k < 0 || format < SKG_MXFP8 || format > SKG_NVFP4) return 0;
  return (k + 31) / 32 * 32 * mx_bits(format) / 8;
}

size_t skg_mx_scales_size(int64_t rows, int64_t k, int32_t format) {
  if (rows < 0 || k < 0 || format < SKG_MXFP8 || format > SKG_NVFP4) return 0;
  return (size_t)((rows + kMxTileRows - 1) / kMxTileRows) * (size_t)mx_groups(k, format) *
         kMxTileBytes;
}

skg_status_t skg_mx_quantize(int64_t rows, int64_t k, const void* X, int64_t ldx, int32_t type,
                             int32_t transpose, int32_t format, const float* tensor_scale,
                             void* codes, int64_t ldq, void* scales, void* values, int64_t ldv,
                             void* stream) {
  if (rows < 0 || k < 0) return SKG_ERR_ARG;
  if (type < SKG_OUT_F32 || type > SKG_OUT_BF16) return SKG_ERR_ARG;
  if (format < SKG_MXFP8 || format > SKG_NVFP4) return SKG_ERR_ARG;
  if (transpose != 0 && transpose != 1) return SKG_ERR_ARG;
  if (rows == 0 || k == 0) return SKG_OK;
  if (!X || !codes || !scales || ldx < (transpose ? rows : k) ||
      ldq < skg_mx_codes_ld(k, format) || (values && ldv < k))
    return SKG_ERR_ARG;
  // The transposed grid counts column tiles in its second dimension.
  if (k > INT32_MAX / 4 || rows > (transpose ? 65535 * 64 : INT32_MAX / 4))
    return SKG_ERR_UNSUPPORTED;
  const int es = type == SKG_OUT_F32 ? 4 : 2;
  if (((uintptr_t)codes & 15) || (ldq & 15) || ((uintptr_t)scales & 15) ||
      ((uintptr_t)X & (es - 1)) || ((uintptr_t)values & (es - 1)) ||
      ((uintptr_t)tensor_scale & 3))
    return SKG_ERR_UNSUPPORTED;
  QuantParams p;
  p.x = X;
  p.ldx = ldx;
  p.rows = rows;
  p.k = k;
  p.g = tensor_scale;
  p.codes = (uint8_t*)codes;
  p.ldq = ldq;
  p.scales = (uint8_t*)scales;
  p.values = values;
  p.ldv = ldv;
  p.x_vec = ((uintptr_t)X & 15) == 0 && (ldx * es) % 16 == 0;
  p.v_vec = ((uintptr_t)values & 15) == 0 && (ldv * es) % 16 == 0;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (type == SKG_OUT_F32) e = launch_quantize_fmt<float>(p, format, transpose != 0, st);
  else if (type == SKG_OUT_F16) e = launch_quantize_fmt<__half>(p, format, transpose != 0, st);
  else e = launch_quantize_fmt<__nv_bfloat16>(p, format, transpose != 0, st);
  return e == cudaSuccess ? SKG_OK : SKG_ERR_CUDA;
}

}  // extern "C"
