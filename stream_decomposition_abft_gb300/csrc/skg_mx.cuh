// Microscaled formats: the block quantiser shared by the quantising kernels,
// and the storage rules of a quantised matrix (rows x k codes and one scale
// per block of consecutive elements along k; see skgemm.h).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "skg_ptx.cuh"
#include "skgemm.h"

namespace skg {

// Elements per scale of a format; bits per code.
__host__ __device__ constexpr int mx_block(int fmt) { return fmt == SKG_NVFP4 ? 16 : 32; }
__host__ __device__ constexpr int mx_bits(int fmt) { return fmt == SKG_MXFP8 ? 8 : 4; }

// Scales lie in tiles of 128 rows x 4 blocks, 512 bytes each (the order in
// which tcgen05.cp reads them): row 32 q + l, block b at byte 16 l + 4 q + b.
constexpr int kMxTileRows = 128;
constexpr int kMxTileBytes = 512;

// Blocks of a row (k rounded up to 32 elements) and tiles along it.
__host__ __device__ constexpr int64_t mx_blocks(int64_t k, int fmt) {
  return (k + 31) / 32 * (32 / mx_block(fmt));
}
__host__ __device__ constexpr int64_t mx_groups(int64_t k, int fmt) {
  return (mx_blocks(k, fmt) + 3) / 4;
}

// Offset of the 4-byte word that holds row r's scales of block group g.
__device__ __forceinline__ int64_t mx_scale_word(int64_t r, int g, int groups) {
  return ((r >> 7) * groups + g) * kMxTileBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// ------------------------------------------------------------------ conversions
__device__ __forceinline__ float mx_to_f32(float v) { return v; }
__device__ __forceinline__ float mx_to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float mx_to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T mx_from_f32(float v);
template <>
__device__ __forceinline__ float mx_from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half mx_from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 mx_from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Sixteen consecutive elements. `vec`: the address is 16-byte aligned and all
// sixteen exist; else the first n (0 .. 16) are read one by one, the rest are 0.
template <typename T>
__device__ __forceinline__ void mx_load16(const T* p, bool vec, int n, float (&v)[16]) {
  if (vec) {
    constexpr int W = 16 * (int)sizeof(T) / 16;
    uint4 u[W];
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = *(reinterpret_cast<const uint4*>(p) + i);
    const T* e = reinterpret_cast<const T*>(u);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = mx_to_f32(e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < n ? mx_to_f32(p[i]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void mx_store16(T* p, bool vec, int n, const float (&v)[16]) {
  if (vec) {
    constexpr int W = 16 * (int)sizeof(T) / 16;
    uint4 u[W];
    T* e = reinterpret_cast<T*>(u);
#pragma unroll
    for (int i = 0; i < 16; ++i) e[i] = mx_from_f32<T>(v[i]);
#pragma unroll
    for (int i = 0; i < W; ++i) *(reinterpret_cast<uint4*>(p) + i) = u[i];
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = mx_from_f32<T>(v[i]);
  }
}

// Four e4m3 codes / eight e2m1 codes, rounded to nearest even, saturating;
// the first element in the lowest bits.
__device__ __forceinline__ uint32_t mx_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ uint32_t mx_e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ float2 mx_half2_f32(uint32_t h2) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}

// The values of four e4m3 codes / eight e2m1 codes (exact in fp16).
__device__ __forceinline__ void mx_e4m3_values(uint32_t c, float* v) {
  uint32_t l, h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(l), "=r"(h)
      : "r"(c));
  const float2 x = mx_half2_f32(l), y = mx_half2_f32(h);
  v[0] = x.x;
  v[1] = x.y;
  v[2] = y.x;
  v[3] = y.y;
}

__device__ __forceinline__ void mx_e2m1_values(uint32_t c, float* v) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = mx_half2_f32(h[i]);
    v[2 * i] = x.x;
    v[2 * i + 1] = x.y;
  }
}

// ------------------------------------------------------------------ the block quantiser
// max |v| as the bits of a float: as unsigned integers, Inf and NaN are above
// every finite magnitude, so neither is lost (fmaxf would drop a NaN).
__device__ __forceinline__ uint32_t mx_absmax16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// The same of 16-bit elements as stored, two at a time (a word's halves apart):
// their magnitudes, too, are ordered as unsigned integers.
__device__ __forceinline__ uint32_t mx_absmax2(uint32_t m, uint32_t w) {
  return __vmaxu2(m, w & 0x7fff7fffu);
}
// A 16-bit magnitude as the bits of a float.
template <typename T>
__device__ __forceinline__ uint32_t mx_magnitude(uint32_t m16);
template <>
__device__ __forceinline__ uint32_t mx_magnitude<__nv_bfloat16>(uint32_t m16) {
  return m16 << 16;
}
template <>
__device__ __forceinline__ uint32_t mx_magnitude<__half>(uint32_t m16) {
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m16)));
}

// One block's scale.
struct MxScale {
  uint32_t byte;  // as stored
  float inv;      // codes = round(x * inv)
  float full;     // value = code * full (nvfp4: the block scale alone, times g last)
  bool bad;       // the block holds an Inf or a NaN: the scale is NaN, the codes 0
};

// e8m0: the least power of two s with amax / s <= most (448 = 1.75 * 2^8 for
// e4m3, 6 = 1.5 * 2^2 for e2m1): amax's exponent less `top`, one more when its
// fraction is above the largest code's; clamped to 2^-127, which an all-zero
// block gets. x * inv is exact. nvfp4: s = e4m3(amax / (6 g)) in fp32.
template <int FMT>
__device__ __forceinline__ MxScale mx_scale(uint32_t amax, float g) {
  MxScale s;
  s.bad = amax >= 0x7f800000u;
  if constexpr (FMT == SKG_NVFP4) {
    const float t = fminf(__fdiv_rn(__uint_as_float(amax), __fmul_rn(6.f, g)), 448.f);
    s.byte = s.bad ? 0x7fu : mx_e4m3x4(t, 0.f, 0.f, 0.f) & 0xffu;
    float v[4];
    mx_e4m3_values(s.byte, v);
    s.full = v[0];
    const float sg = __fmul_rn(v[0], g);
    s.inv = sg > 0.f ? fminf(__frcp_rn(sg), 3.402823466e38f) : 0.f;
  } else {
    constexpr int top = FMT == SKG_MXFP8 ? 8 : 2;
    constexpr uint32_t most = FMT == SKG_MXFP8 ? 0x600000u : 0x400000u;
    const int b = (int)(amax >> 23) - top + ((amax & 0x7fffffu) > most ? 1 : 0);
    s.byte = s.bad ? 0xffu : (uint32_t)max(b, 0);
    s.inv = __uint_as_float((254u - min(s.byte, 253u)) << 23);
    s.full = __uint_as_float(s.byte ? s.byte << 23 : 0x00400000u);
    if (s.bad) s.full = __uint_as_float(0x7fffffffu);
  }
  return s;
}

// Sixteen codes: 16 bytes (e4m3: all of `out`) or 8 (e2m1: out.x, out.y).
template <int FMT>
__device__ __forceinline__ uint4 mx_codes16(const float (&v)[16], const MxScale& s) {
  uint4 o = make_uint4(0u, 0u, 0u, 0u);
  if (s.bad) return o;
  float y[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = __fmul_rn(v[i], s.inv);
  if constexpr (FMT == SKG_MXFP8) {
    o.x = mx_e4m3x4(y[0], y[1], y[2], y[3]);
    o.y = mx_e4m3x4(y[4], y[5], y[6], y[7]);
    o.z = mx_e4m3x4(y[8], y[9], y[10], y[11]);
    o.w = mx_e4m3x4(y[12], y[13], y[14], y[15]);
  } else {
    o.x = mx_e2m1x8(y);
    o.y = mx_e2m1x8(y + 8);
  }
  return o;
}

// Eight codes: 8 bytes (e4m3) or 4 (e2m1: .x).
template <int FMT>
__device__ __forceinline__ uint2 mx_codes8(const float (&v)[8], const MxScale& s) {
  if (s.bad) return make_uint2(0u, 0u);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(v[i], s.inv);
  if constexpr (FMT == SKG_MXFP8)
    return make_uint2(mx_e4m3x4(y[0], y[1], y[2], y[3]), mx_e4m3x4(y[4], y[5], y[6], y[7]));
  else
    return make_uint2(mx_e2m1x8(y), 0u);
}

template <int FMT>
__device__ __forceinline__ void mx_store_codes8(uint8_t* row, int64_t piece, const uint2& o) {
  if constexpr (FMT == SKG_MXFP8)
    *reinterpret_cast<uint2*>(row + piece * 8) = o;
  else
    *reinterpret_cast<uint32_t*>(row + piece * 4) = o.x;
}

// What sixteen codes and their scale stand for (nvfp4: (code * s) * g).
template <int FMT>
__device__ __forceinline__ void mx_values16(const uint4& o, const MxScale& s, float g,
                                            float (&v)[16]) {
  if constexpr (FMT == SKG_MXFP8) {
    mx_e4m3_values(o.x, v);
    mx_e4m3_values(o.y, v + 4);
    mx_e4m3_values(o.z, v + 8);
    mx_e4m3_values(o.w, v + 12);
  } else {
    mx_e2m1_values(o.x, v);
    mx_e2m1_values(o.y, v + 8);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i] = __fmul_rn(v[i], s.full);
    if constexpr (FMT == SKG_NVFP4) v[i] = __fmul_rn(v[i], g);
  }
}

template <int FMT>
__device__ __forceinline__ void mx_store_codes16(uint8_t* row, int64_t chunk, const uint4& o) {
  if constexpr (FMT == SKG_MXFP8)
    *reinterpret_cast<uint4*>(row + chunk * 16) = o;
  else
    *reinterpret_cast<uint2*>(row + chunk * 8) = make_uint2(o.x, o.y);
}

// A warp's lanes hold consecutive 16-element chunks (chunk c in a lane with
// lane % 8 == c % 8; zeros past the row's end), amax the largest magnitude of its
// own: quantise them, and hand back
// in `word` the four scale bytes of the chunk's block group (the OR over the
// group's lanes; the group's first lane writes it). All 32 lanes take part.
template <int FMT>
__device__ __forceinline__ MxScale mx_quantize_chunk(const float (&v)[16], uint32_t amax, bool live,
                                                     int lane, float g, uint4& codes,
                                                     uint32_t& word) {
  if constexpr (FMT != SKG_NVFP4) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  const MxScale s = mx_scale<FMT>(amax, g);
  codes = mx_codes16<FMT>(v, s);
  const int slot = FMT == SKG_NVFP4 ? (lane & 3) : ((lane >> 1) & 3);
  word = live ? s.byte << (8 * slot) : 0u;
  if constexpr (FMT == SKG_NVFP4) word |= __shfl_xor_sync(0xffffffffu, word, 1);
  word |= __shfl_xor_sync(0xffffffffu, word, 2);
  if constexpr (FMT != SKG_NVFP4) word |= __shfl_xor_sync(0xffffffffu, word, 4);
  return s;
}

// The same for pieces of 8 elements (piece c in a lane with lane % 16 == c % 16).
template <int FMT>
__device__ __forceinline__ MxScale mx_quantize_piece(const float (&v)[8], bool live, int lane,
                                                     float g, uint2& codes, uint32_t& word) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  if constexpr (FMT != SKG_NVFP4) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const MxScale s = mx_scale<FMT>(amax, g);
  codes = mx_codes8<FMT>(v, s);
  const int slot = FMT == SKG_NVFP4 ? ((lane >> 1) & 3) : ((lane >> 2) & 3);
  word = live ? s.byte << (8 * slot) : 0u;
  if constexpr (FMT == SKG_NVFP4) word |= __shfl_xor_sync(0xffffffffu, word, 2);
  word |= __shfl_xor_sync(0xffffffffu, word, 4);
  if constexpr (FMT != SKG_NVFP4) word |= __shfl_xor_sync(0xffffffffu, word, 8);
  return s;
}

// Sixteen consecutive elements as they are (see mx_load16), and their largest
// magnitude.
template <typename T>
struct MxRaw16 {
  uint4 q[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ MxRaw16<T> mx_load_raw16(const T* p, bool vec, int n) {
  MxRaw16<T> r;
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) r.q[i] = *(reinterpret_cast<const uint4*>(p) + i);
  } else {
    T* e = reinterpret_cast<T*>(r.q);
#pragma unroll
    for (int i = 0; i < 16; ++i) e[i] = i < n ? p[i] : mx_from_f32<T>(0.f);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void mx_unpack_raw16(const MxRaw16<T>& r, float (&v)[16]) {
  const T* e = reinterpret_cast<const T*>(r.q);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = mx_to_f32(e[i]);
}
template <typename T>
__device__ __forceinline__ uint32_t mx_absmax_raw16(const MxRaw16<T>& r) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.q);
  uint32_t m = 0;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = mx_absmax2(m, w[i]);
    return mx_magnitude<T>(max(m & 0xffffu, m >> 16));
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, w[i] & 0x7fffffffu);
    return m;
  }
}

// Eight consecutive elements as they are. `vec`: the address is 16-byte aligned
// and all eight exist; else the first n are read one by one, the rest are 0.
template <typename T>
struct MxRaw8 {
  uint4 q[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ MxRaw8<T> mx_load_raw8(const T* p, bool vec, int n) {
  MxRaw8<T> r;
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = *(reinterpret_cast<const uint4*>(p) + i);
  } else {
    T* e = reinterpret_cast<T*>(r.q);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = i < n ? p[i] : mx_from_f32<T>(0.f);
  }
  return r;
}

// Elements o .. o + 7 (o < 8) of the sixteen 16-bit ones in a, b; those from n on 0.
__device__ __forceinline__ uint4 mx_shift8(const uint4& a, const uint4& b, int o, int n) {
  uint32_t w[7] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z};
  if (o & 4) {
    w[0] = w[2];
    w[1] = w[3];
    w[2] = w[4];
    w[3] = w[5];
    w[4] = w[6];
    w[5] = b.w;
  }
  if (o & 2) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  const uint32_t odd = (o & 1) * 16;
  uint4 q = make_uint4(__funnelshift_r(w[0], w[1], odd), __funnelshift_r(w[1], w[2], odd),
                       __funnelshift_r(w[2], w[3], odd), __funnelshift_r(w[3], w[4], odd));
  if (n < 8) {
    uint32_t* e = reinterpret_cast<uint32_t*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n < 2 * i + 2) e[i] &= 0xffffu;
      if (n < 2 * i + 1) e[i] = 0u;
    }
  }
  return q;
}

// Eight elements of a 16-bit type from an address that is a multiple of 2 alone:
// the two aligned 16-byte pieces that hold them, shifted together (one load of
// eight would take eight instructions). lo, hi: the matrix; a piece that reaches
// outside of it is read element by element. Elements n .. 7 are 0.
template <typename T>
__device__ __forceinline__ uint4 mx_aligned_piece(uintptr_t at, const T* lo, const T* hi) {
  if (at >= (uintptr_t)lo && at + 16 <= (uintptr_t)hi) return *reinterpret_cast<const uint4*>(at);
  uint4 q = make_uint4(0u, 0u, 0u, 0u);
  T* e = reinterpret_cast<T*>(&q);
  const T* src = reinterpret_cast<const T*>(at);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (src + i >= lo && src + i < hi) e[i] = src[i];
  return q;
}
template <typename T>
__device__ __forceinline__ uint4 mx_load8_any(const T* p, int n, const T* lo, const T* hi) {
  static_assert(sizeof(T) == 2, "16-bit elements");
  if (n <= 0) return make_uint4(0u, 0u, 0u, 0u);
  const uintptr_t at = (uintptr_t)p & ~(uintptr_t)15;
  const int o = (int)(((uintptr_t)p & 15) >> 1);
  const uint4 a = mx_aligned_piece(at, lo, hi);
  const uint4 b = o + n > 8 ? mx_aligned_piece(at + 16, lo, hi) : make_uint4(0u, 0u, 0u, 0u);
  return mx_shift8(a, b, o, n);
}

// A row of 16-bit elements at any address, by the aligned 16-byte pieces that cover
// it: piece c holds elements 8 c - o .. of the row. Only bytes of the row and of the
// elements before it in the matrix are read, nothing before lo, the matrix's start.
template <typename T>
struct MxRow {
  const uint8_t* base;
  const T* lo;
  int o, bytes;  // from base to the row's end
  __device__ __forceinline__ MxRow(const T* row, int n, const T* matrix)
      : base(reinterpret_cast<const uint8_t*>((uintptr_t)row & ~(uintptr_t)15)),
        lo(matrix),
        o((int)(((uintptr_t)row & 15) >> 1)),
        bytes(2 * ((int)(((uintptr_t)row & 15) >> 1) + n)) {}
  // Piece c to shared memory (cp.async).
  __device__ __forceinline__ void fetch(uint4* dst, int c) const {
    const int left = bytes - 16 * c;
    if (left <= 0) return;
    const uint8_t* at = base + 16 * (int64_t)c;
    if (c > 0 || at >= reinterpret_cast<const uint8_t*>(lo))
      cp_async16(dst, at, left < 16 ? (uint32_t)left : 16u);
    else
      *dst = mx_aligned_piece((uintptr_t)at, lo, reinterpret_cast<const T*>(base + bytes));
  }
  // Eight elements from 8 c on, n of them in the row, of pieces c and c + 1.
  __device__ __forceinline__ uint4 elements(const uint4* first, const uint4* second, int n) const {
    if (n <= 0) return make_uint4(0u, 0u, 0u, 0u);
    return mx_shift8(*first, *second, o, n);
  }
};

// A warp's consecutive pieces of 8 elements to a row of any alignment, 32
// neighbouring elements an instruction (a lane's own eight would touch a sector
// each): `total` elements from the first lane's on. buf: 32 pieces of shared memory
// of the warp's own.
template <typename T>
__device__ __forceinline__ void mx_warp_store8(T* first, int total, const uint4& q, uint4* buf,
                                               int lane) {
  __syncwarp();
  buf[lane] = q;
  __syncwarp();
  const T* e = reinterpret_cast<const T*>(buf);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i * 32 + lane < total) first[i * 32 + lane] = e[i * 32 + lane];
}

template <typename T>
__device__ __forceinline__ void mx_store8(T* p, bool vec, int n, const float (&v)[8]) {
  MxRaw8<T> r;
  T* e = reinterpret_cast<T*>(r.q);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = mx_from_f32<T>(v[i]);
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) *(reinterpret_cast<uint4*>(p) + i) = r.q[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = e[i];
  }
}

// Eight elements of a 16-bit type.
template <typename T>
__device__ __forceinline__ void mx_unpack8(const uint4& u, float (&v)[8]) {
  const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = mx_to_f32(e[i]);
}

template <typename T>
__device__ __forceinline__ uint4 mx_pack8(const float (&v)[8]) {
  uint4 u;
  T* e = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = mx_from_f32<T>(v[i]);
  return u;
}

// Chunks of 16 elements per block group.
__host__ __device__ constexpr int mx_group_chunks(int fmt) { return fmt == SKG_NVFP4 ? 4 : 8; }

}  // namespace skg
