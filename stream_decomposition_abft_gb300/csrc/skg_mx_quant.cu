// skg_mx_quantize: a matrix to a microscaled format, along its rows or along
// its columns (the transposed operand of a gradient), with the values that
// the codes stand for on request.
//
// Every element is read once and every code, scale and value is written once, so
// memory bounds the kernels, with the instructions of the conversion close behind
// (an issue slot is taken in 2 of 3 cycles). Measured on GB300, bf16, against
// 6.69 TB/s of a copy: 8192 x 8192 to mxfp4 with its values 46 us (6.5 TB/s), to
// mxfp8 along the rows 35 us (5.8), along the columns 33 us (6.1), to nvfp4 with its
// values 50 us (6.2); 4096 x 8192 to mxfp8 both ways in one pass 27 us (5.0; the two
// passes take 34). fp32, 8192 x 8192: to mxfp8 along the rows 50 us (6.7), along the
// columns 58 (5.8), to nvfp4 along the columns 66 (4.6: one block of 128 KB per SM).
// Rows off 16-byte boundaries, 4000 x 8191: to mxfp8 28 us (3.5), to nvfp4 with its
// values 47 (3.2).
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

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

// Along the rows. A thread takes 16 consecutive elements (with 8, and four rows'
// loads in flight per thread, the blocks' scales are formed twice as often, and
// the kernel is bound by instructions: 8192 x 8192 in mxfp4 with its values 60 us
// against 50, in nvfp4 86 against 59); a warp 32 / TX rows
// of TX chunks (TX a power of two of at least 8, so that the lanes of a block
// group sit together). A block of 256 threads takes the rows 32 q + l of one
// scale tile for l in a range of TY / 4: the 16 bytes of scales of each l are
// then written together. Rows past the end only write their zero scales.
// VEC: x and the values have their rows on 16-byte boundaries.
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 4 ? 3 : 4)
mx_quantize_rows_kernel(QuantParams p, int log_tx) {
  __shared__ T vbuf[VEC ? 1 : kQThreads / 32][32 * 17];  // a warp's values
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
  const int64_t units = (p.rows + 127) / 128 * 32;  // (scale tile, l) pairs, 32 a tile
  for (int64_t u = (int64_t)blockIdx.y * 2 * ls; u < units; u += (int64_t)gridDim.y * 2 * ls) {
    MxRaw16<T> raw[2];  // both rows' loads in flight
    int64_t row[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t ul = u + h * ls + (ty >> 2);
      row[h] = (ul >> 5) * 128 + (ty & 3) * 32 + (ul & 31);
      const int m = row[h] < p.rows ? n : 0;
      const T* x = reinterpret_cast<const T*>(p.x);
      const T* src = x + row[h] * p.ldx + chunk * 16;
      if constexpr (!VEC && sizeof(T) == 2) {
        const T* end = x + (p.rows - 1) * p.ldx + p.k;
        raw[h].q[0] = mx_load8_any(src, m < 8 ? m : 8, x, end);
        raw[h].q[1] = mx_load8_any(src + 8, m - 8, x, end);
      } else {
        raw[h] = mx_load_raw16(src, VEC && m == 16, m);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool here = live && row[h] < p.rows;
      float v[16];
      mx_unpack_raw16(raw[h], v);
      uint4 codes;
      uint32_t word;
      const MxScale s =
          mx_quantize_chunk<FMT>(v, mx_absmax_raw16(raw[h]), here, lane, g, codes, word);
      if (here) {
        mx_store_codes16<FMT>(p.codes + row[h] * p.ldq, chunk, codes);
        if (p.values) {
          mx_values16<FMT>(codes, s, g, v);
          if (VEC || log_tx < 5)
            mx_store16(reinterpret_cast<T*>(p.values) + row[h] * p.ldv + chunk * 16,
                       VEC && n == 16, n, v);
        }
      }
      // Values of rows off 16-byte boundaries: a warp's 512 of a row leave 32
      // neighbours at a time.
      if (!VEC && p.values && log_tx == 5 && row[h] < p.rows) {
        const int warp = VEC ? 0 : threadIdx.x >> 5;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 16; ++i) vbuf[warp][lane * 17 + i] = mx_from_f32<T>(v[i]);
        __syncwarp();
        const int64_t first = (int64_t)blockIdx.x * 512;
        T* out = reinterpret_cast<T*>(p.values) + row[h] * p.ldv + first;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int e = i * 32 + lane;
          if (first + e < p.k) out[e] = vbuf[warp][(e >> 4) * 17 + (e & 15)];
        }
      }
      constexpr int per = mx_group_chunks(FMT);
      const int64_t grp = chunk / per;
      if ((lane & (per - 1)) == 0 && grp < groups)
        *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row[h], (int)grp, groups)) = word;
    }
  }
}

// Along the columns, or along both. X is stored lines x columns; a block takes
// tiles of 128 x 128 of it in turn, the next one on its way to shared memory
// (cp.async, 8 elements a lane) while it works on one. The row direction (ROWS: the
// quantised X) takes chunks of 16 elements, 8 lanes a line. In the column direction
// (the quantised X^T) a thread takes 32 consecutive lines of two adjacent columns: four
// lanes hold the tile's four line ranges of a column pair, so that codes leave in 64 to
// 128 bytes at a time; the words of a line are XORed with its line range for those
// lanes to read different banks. The tiles of the same columns follow one another,
// so that what is written along a row of X^T is written together.
constexpr int kTile = 128;

template <typename T, int FMT, bool ROWS, bool WIN>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 4 ? 1 : 3)
mx_quantize_tile_kernel(QuantParams p, QuantParams rp, int64_t tiles, int tiles_k) {
  constexpr int W = sizeof(T) / 2;             // 32-bit words of a column pair
  constexpr int LINE = kTile * sizeof(T) / 4;  // words of a line
  // Two tiles of kTile x LINE words; WIN (16-bit lines off 16-byte boundaries): one,
  // and the aligned pieces that cover the next tile's lines.
  static_assert(!WIN || sizeof(T) == 2, "windows of 16-bit elements");
  extern __shared__ __align__(16) uint32_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const T* x = reinterpret_cast<const T*>(p.x);
  const float g = FMT == SKG_NVFP4 && p.g ? *p.g : 1.f;
  const int piece = threadIdx.x & 15, line0 = threadIdx.x >> 4;
  // Where this thread's piece of a line lies: word w of line l at w ^ 8 W (l / 32);
  // pieces of 4 words stay whole.
  auto place = [&](uint32_t* tile, int line, int j) {
    return reinterpret_cast<uint4*>(tile + line * LINE +
                                    ((piece * 4 * W + j * 4) ^ ((line >> 5) * 8 * W)));
  };
  auto fetch = [&](int64_t t, uint32_t* tile) {
    if (t < tiles) {
      const int64_t k0 = t % tiles_k * kTile, c = t / tiles_k * kTile + piece * 8;
      const int64_t left = p.rows - c;
      const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int line = i * 16 + line0;
        const int m = k0 + line < p.k ? n : 0;
        const T* src = x + (k0 + line) * p.ldx + c;
        if (p.x_vec && (m == 8 || m == 0)) {
#pragma unroll
          for (int j = 0; j < W; ++j)
            cp_async16(place(tile, line, j), m ? src + j * (16 / (int)sizeof(T)) : x, m ? 16u : 0u);
        } else {
          const MxRaw8<T> raw = mx_load_raw8(src, false, m);
#pragma unroll
          for (int j = 0; j < W; ++j) *place(tile, line, j) = raw.q[j];
        }
      }
    }
    cp_async_commit();
  };
  constexpr int PIECES = kTile / 8 + 1;  // of a line's window
  uint4* window = reinterpret_cast<uint4*>(smem + kTile * LINE);
  auto fetch_windows = [&](int64_t t) {
    if (t < tiles) {
      const int64_t k0 = t % tiles_k * kTile, c0 = t / tiles_k * kTile;
      const int n = (int)(p.rows - c0 < kTile ? p.rows - c0 : kTile);
      for (int i = threadIdx.x; i < kTile * PIECES; i += kQThreads) {
        const int64_t line = k0 + i / PIECES;
        if constexpr (WIN)
          if (line < p.k) MxRow<T>(x + line * p.ldx + c0, n, x).fetch(window + i, i % PIECES);
      }
    }
    cp_async_commit();
  };
  if constexpr (WIN) fetch_windows(blockIdx.x);
  else fetch(blockIdx.x, smem);
  int buf = 0;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, buf ^= 1) {
    uint32_t* tile = smem + (WIN ? 0 : buf) * (kTile * LINE);
    const int64_t k0 = t % tiles_k * kTile, c0 = t / tiles_k * kTile;
    if constexpr (WIN) {
      cp_async_wait<0>();
      __syncthreads();
      const int64_t left = p.rows - (c0 + piece * 8);
      const int n = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int line = i * 16 + line0;
        const uint4* src = window + line * PIECES + piece;
        *place(tile, line, 0) = MxRow<T>(x + (k0 + line) * p.ldx + c0, n, x)
                                    .elements(src, src + 1, k0 + line < p.k ? n : 0);
      }
      __syncthreads();
      fetch_windows(t + gridDim.x);
    } else {
      fetch(t + gridDim.x, smem + (buf ^ 1) * (kTile * LINE));
      cp_async_wait<1>();
      __syncthreads();
    }
    if constexpr (ROWS) {
      // Chunks of 16 elements, 8 lanes a line.
      const int64_t c = c0 + (threadIdx.x & 7) * 16;
      const int groups = (int)mx_groups(rp.k, FMT);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int line = i * 32 + (threadIdx.x >> 3);
        const int64_t r = k0 + line;
        const bool here = r < rp.rows && c < (rp.k + 31) / 32 * 32;
        MxRaw16<T> raw;
#pragma unroll
        for (int j = 0; j < 2 * W; ++j)
          raw.q[j] = *reinterpret_cast<const uint4*>(
              tile + line * LINE + (((threadIdx.x & 7) * 8 * W + j * 4) ^ ((line >> 5) * 8 * W)));
        float v[16];
        mx_unpack_raw16(raw, v);
        uint4 codes;
        uint32_t word;
        mx_quantize_chunk<FMT>(v, mx_absmax_raw16(raw), here, lane, g, codes, word);
        if (here) mx_store_codes16<FMT>(rp.codes + r * rp.ldq, c / 16, codes);
        constexpr int per = mx_group_chunks(FMT);
        const int64_t grp = c / 16 / per;
        if ((lane & (per - 1)) == 0 && grp < groups)
          *reinterpret_cast<uint32_t*>(rp.scales + mx_scale_word(r, (int)grp, groups)) = word;
      }
    }
    const int kb = lane & 3, pair = (threadIdx.x >> 5) * 8 + (lane >> 2);
    const int64_t kfirst = k0 + kb * 32;
    const int groups = (int)mx_groups(p.k, FMT);
    uint32_t w[32][W];
#pragma unroll
    for (int i = 0; i < 32; ++i)
#pragma unroll
      for (int j = 0; j < W; ++j)
        w[i][j] = tile[(kb * 32 + i) * LINE + ((pair * W + j) ^ (kb * 8 * W))];
    // The values leave by rows of X^T, through the tile (its pieces of 16 bytes
    // XORed for the lanes of a column pair to write different banks).
    auto value_piece = [&](int col, int q) {
      return reinterpret_cast<uint4*>(tile + col * LINE) + (q ^ ((q >> 3) & 1) ^ (((col >> 1) & 1) << 1));
    };
    if (p.values) __syncthreads();  // every thread has its words
    // Largest magnitudes of the two columns' 16-line halves.
    uint32_t top[2][2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t m[W] = {};
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j)
          m[j] = W == 1 ? mx_absmax2(m[j], w[b * 16 + i][j]) : max(m[j], w[b * 16 + i][j] & 0x7fffffffu);
      if constexpr (W == 1) {
        top[0][b] = mx_magnitude<T>(m[0] & 0xffffu);
        top[1][b] = mx_magnitude<T>(m[0] >> 16);
      } else {
        top[0][b] = m[0];
        top[1][b] = m[W - 1];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // the pair's columns
      const int64_t row = c0 + pair * 2 + h;
      const bool live = row < p.rows && kfirst < p.k;
      if constexpr (FMT != SKG_NVFP4) top[h][0] = max(top[h][0], top[h][1]);
      uint32_t bytes[2];
      MxScale s;
#pragma unroll
      for (int b = 0; b < 2; ++b) {  // 16 lines at a time
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t u = w[b * 16 + i][h * (W - 1)];
          if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(u);
          else v[i] = mx_to_f32(reinterpret_cast<const T*>(&u)[h]);
        }
        if (FMT == SKG_NVFP4 || b == 0) s = mx_scale<FMT>(top[h][b], g);
        bytes[b] = s.byte;
        if (live) {
          const uint4 codes = mx_codes16<FMT>(v, s);
          mx_store_codes16<FMT>(p.codes + row * p.ldq, kfirst / 16 + b, codes);
          if (p.values) {
            mx_values16<FMT>(codes, s, g, v);
            MxRaw16<T> o;
            T* e = reinterpret_cast<T*>(o.q);
#pragma unroll
            for (int i = 0; i < 16; ++i) e[i] = mx_from_f32<T>(v[i]);
#pragma unroll
            for (int j = 0; j < 2 * W; ++j)
              *value_piece(pair * 2 + h, (kb * 2 + b) * 2 * W + j) = o.q[j];
          }
        }
      }
      uint32_t word;
      if constexpr (FMT == SKG_NVFP4) {
        word = live ? (bytes[0] | (bytes[1] << 8)) << (16 * (kb & 1)) : 0u;
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        const int64_t grp = (k0 / 64) + (kb >> 1);
        if ((kb & 1) == 0 && grp < groups)
          *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, (int)grp, groups)) = word;
      } else {
        word = live ? bytes[0] << (8 * kb) : 0u;
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        if (kb == 0 && k0 / 128 < groups)
          *reinterpret_cast<uint32_t*>(p.scales + mx_scale_word(row, (int)(k0 / 128), groups)) = word;
      }
    }
    if (p.values) {
      __syncthreads();
      T* values = reinterpret_cast<T*>(p.values);
      if (p.v_vec) {
        constexpr int Q = 16 * W;  // 16-byte pieces of a row
        for (int i = threadIdx.x; i < kTile * Q; i += kQThreads) {
          const int col = i / Q, q = i % Q;
          const int64_t row = c0 + col, k = k0 + q * (16 / (int)sizeof(T));
          if (row >= p.rows || k >= p.k) continue;
          const uint4 u = *value_piece(col, q);
          T* out = values + row * p.ldv + k;
          if (k + 16 / (int)sizeof(T) <= p.k) {
            *reinterpret_cast<uint4*>(out) = u;
          } else {
            const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
            for (int j = 0; j < 16 / (int)sizeof(T); ++j)
              if (k + j < p.k) out[j] = e[j];
          }
        }
      } else {
        constexpr int PER = 16 / (int)sizeof(T);
        for (int i = threadIdx.x; i < kTile * kTile; i += kQThreads) {
          const int col = i / kTile, l = i % kTile;
          const int64_t row = c0 + col;
          if (row < p.rows && k0 + l < p.k)
            values[row * p.ldv + k0 + l] =
                reinterpret_cast<const T*>(value_piece(col, l / PER))[l % PER];
        }
      }
    }
    __syncthreads();  // the tile is free for the one after the next
  }
}

// rp: the row direction of the same matrix too (NULL: columns alone).
template <typename T, int FMT>
cudaError_t launch_tile(const QuantParams& p, const QuantParams* rp, cudaStream_t stream) {
  const int64_t tiles_k = (p.k + kTile - 1) / kTile;
  const int64_t tiles = (p.rows + kTile - 1) / kTile * tiles_k;
  const int64_t most = (int64_t)skg_device_sm_count() * (sizeof(T) == 4 ? 1 : 3);
  if (most <= 0) return cudaErrorNoDevice;
  const dim3 grid((unsigned)(tiles < most ? tiles : most));
  auto run = [&](auto kernel, std::atomic<uint64_t>& done, size_t smem) {
    const cudaError_t e = opt_in_smem((const void*)kernel, done, (int)smem);
    return e != cudaSuccess ? e
                            : launch_pdl(kernel, grid, dim3(kQThreads), smem, stream, p,
                                         rp ? *rp : p, tiles, (int)tiles_k);
  };
  static std::atomic<uint64_t> d[4] = {};
  if constexpr (sizeof(T) == 2) {
    const size_t smem = kTile * kTile * sizeof(T) + kTile * (kTile / 8 + 1) * 16;
    if (!p.x_vec)
      return rp ? run(mx_quantize_tile_kernel<T, FMT, true, true>, d[0], smem)
                : run(mx_quantize_tile_kernel<T, FMT, false, true>, d[1], smem);
  }
  const size_t smem = 2 * kTile * kTile * sizeof(T);
  return rp ? run(mx_quantize_tile_kernel<T, FMT, true, false>, d[2], smem)
            : run(mx_quantize_tile_kernel<T, FMT, false, false>, d[3], smem);
}

template <typename T, int FMT>
cudaError_t launch_rows(const QuantParams& p, cudaStream_t stream) {
  const int64_t chunks = (p.k + 31) / 32 * 2;
  int log_tx = 3;
  while (log_tx < 5 && (1 << log_tx) < chunks) ++log_tx;
  const int ls = (kQThreads >> log_tx) / 4;
  const int64_t gx = (chunks + (1 << log_tx) - 1) >> log_tx;
  int64_t gy = (p.rows + 127) / 128 * 32 / (2 * ls);
  if (gy > 65535) gy = 65535;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  return p.x_vec && (!p.values || p.v_vec)
             ? launch_pdl(mx_quantize_rows_kernel<T, FMT, true>, grid, dim3(kQThreads), 0, stream, p,
                          log_tx)
             : launch_pdl(mx_quantize_rows_kernel<T, FMT, false>, grid, dim3(kQThreads), 0, stream,
                          p, log_tx);
}

template <typename T, int FMT>
cudaError_t launch_one(const QuantParams* rows, const QuantParams* cols, cudaStream_t stream) {
  return cols ? launch_tile<T, FMT>(*cols, rows, stream) : launch_rows<T, FMT>(*rows, stream);
}

template <typename T>
cudaError_t launch_fmt(const QuantParams* rows, const QuantParams* cols, int fmt,
                       cudaStream_t stream) {
  if (fmt == SKG_MXFP8) return launch_one<T, SKG_MXFP8>(rows, cols, stream);
  if (fmt == SKG_MXFP4) return launch_one<T, SKG_MXFP4>(rows, cols, stream);
  return launch_one<T, SKG_NVFP4>(rows, cols, stream);
}

// The quantised matrix (rows), its transpose (cols), or both.
cudaError_t launch_quantize(const QuantParams* rows, const QuantParams* cols, int type, int fmt,
                            cudaStream_t stream) {
  if (type == SKG_OUT_F32) return launch_fmt<float>(rows, cols, fmt, stream);
  if (type == SKG_OUT_F16) return launch_fmt<__half>(rows, cols, fmt, stream);
  return launch_fmt<__nv_bfloat16>(rows, cols, fmt, stream);
}

// Whether codes, scales and the other pointers are aligned as the kernels ask.
bool storage_aligned(const void* codes, int64_t ldq, const void* scales) {
  return !((uintptr_t)codes & 15) && !(ldq & 15) && !((uintptr_t)scales & 15);
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
  if (k > INT32_MAX / 4 || rows > INT32_MAX / 4)
    return SKG_ERR_UNSUPPORTED;
  const int es = type == SKG_OUT_F32 ? 4 : 2;
  if (!storage_aligned(codes, ldq, scales) || ((uintptr_t)X & (es - 1)) ||
      ((uintptr_t)values & (es - 1)) || ((uintptr_t)tensor_scale & 3))
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
  return launch_quantize(transpose ? nullptr : &p, transpose ? &p : nullptr, type, format,
                         (cudaStream_t)stream) == cudaSuccess
             ? SKG_OK
             : SKG_ERR_CUDA;
}

skg_status_t skg_mx_quantize_both(int64_t rows, int64_t cols, const void* X, int64_t ldx,
                                  int32_t type, int32_t format, const float* tensor_scale,
                                  void* codes, int64_t ldq, void* scales, void* codes_t,
                                  int64_t ldq_t, void* scales_t, void* stream) {
  if (rows < 0 || cols < 0) return SKG_ERR_ARG;
  if (type < SKG_OUT_F32 || type > SKG_OUT_BF16) return SKG_ERR_ARG;
  if (format < SKG_MXFP8 || format > SKG_NVFP4) return SKG_ERR_ARG;
  if (rows == 0 || cols == 0) return SKG_OK;
  if (!X || !codes || !scales || !codes_t || !scales_t || ldx < cols ||
      ldq < skg_mx_codes_ld(cols, format) || ldq_t < skg_mx_codes_ld(rows, format))
    return SKG_ERR_ARG;
  if (rows > INT32_MAX / 4 || cols > INT32_MAX / 4) return SKG_ERR_UNSUPPORTED;
  const int es = type == SKG_OUT_F32 ? 4 : 2;
  if (!storage_aligned(codes, ldq, scales) || !storage_aligned(codes_t, ldq_t, scales_t) ||
      ((uintptr_t)X & (es - 1)) || ((uintptr_t)tensor_scale & 3))
    return SKG_ERR_UNSUPPORTED;
  QuantParams r;
  r.x = X;
  r.ldx = ldx;
  r.rows = rows;
  r.k = cols;
  r.g = tensor_scale;
  r.codes = (uint8_t*)codes;
  r.ldq = ldq;
  r.scales = (uint8_t*)scales;
  r.values = nullptr;
  r.ldv = 0;
  r.x_vec = ((uintptr_t)X & 15) == 0 && (ldx * es) % 16 == 0;
  r.v_vec = 0;
  QuantParams c = r;
  c.rows = cols;
  c.k = rows;
  c.codes = (uint8_t*)codes_t;
  c.ldq = ldq_t;
  c.scales = (uint8_t*)scales_t;
  return launch_quantize(&r, &c, type, format, (cudaStream_t)stream) == cudaSuccess ? SKG_OK
                                                                                   : SKG_ERR_CUDA;
}

}  // extern "C"
