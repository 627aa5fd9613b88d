// The way out of a 128 x 128 tile on a single CTA or the CTAs of a cluster.
#pragma once
#include "skg_lin.cuh"

namespace skg {

template <typename T>
__device__ __forceinline__ void write4(T* c, const float (&v)[4], int left) {
  if (left >= 4) {
    mx_write4_plain<T>(c, make_float4(v[0], v[1], v[2], v[3]), 1.f);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) c[i] = mx_from_f32<T>(v[i]);
  }
}

// Four output columns of row r: v as the accumulator has them; gated: gate and up; grad: dH,
// with g and u of PRE.
template <int MODE, int ACT, typename T>
__device__ __forceinline__ void finish4(const LinParams& p, int row, int col, const float4& v,
                                        const float4& u, uint2 g_in, uint2 u_in) {
  T* c = reinterpret_cast<T*>(p.c) + (int64_t)row * p.ldc + col;
  if constexpr (MODE == kLinGated) {
    const float h[4] = {lin_gated<ACT>(v.x, u.x), lin_gated<ACT>(v.y, u.y),
                        lin_gated<ACT>(v.z, u.z), lin_gated<ACT>(v.w, u.w)};
    write4<T>(c, h, p.n - col);
    if (p.pre) {
      T* g = reinterpret_cast<T*>(p.pre) + (int64_t)row * p.ldp + col;
      const float a[4] = {v.x, v.y, v.z, v.w}, b[4] = {u.x, u.y, u.z, u.w};
      write4<T>(g, a, p.n - col);
      write4<T>(g + p.n, b, p.n - col);
    }
  } else if constexpr (MODE == kLinGrad) {  // n is a multiple of 8
    union {
      uint2 q;
      T e[4];
    } g, w;
    g.q = g_in;
    w.q = u_in;
    const float d[4] = {v.x, v.y, v.z, v.w};
    float dg[4], du[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const LinGrad r = lin_grad<ACT>(d[i], mx_to_f32(g.e[i]), mx_to_f32(w.e[i]));
      dg[i] = r.dg;
      du[i] = r.du;
      h[i] = r.h;
    }
    T* o = reinterpret_cast<T*>(p.pre) + (int64_t)row * p.ldp + col;
    if (p.pre_lo) {
      T* l = reinterpret_cast<T*>(p.pre_lo) + (int64_t)row * p.ldp + col;
      store_parts<T>(o, l, dg);
      store_parts<T>(o + p.n, l + p.n, du);
      store_parts<T>(c, reinterpret_cast<T*>(p.c_lo) + (int64_t)row * p.ldc + col, h);
    } else {
      write4<T>(o, dg, 4);
      write4<T>(o + p.n, du, 4);
      write4<T>(c, h, 4);
    }
  } else {
    const float a[4] = {v.x, v.y, v.z, v.w};
    write4<T>(c, a, p.n - col);
  }
}

// Rows `first`, `first` + step, ... of the tile, S CTAs' partial sums in rank order (S = 1:
// this CTA's own). A warp takes a row of 128 columns at once, or two rows of 64 gated
// outputs; the loads of several rows are in flight together. Every value that is loaded is
// used, so no load is still on its way to another CTA's shared memory when a thread comes to
// the barrier that lets that CTA leave.
template <int MODE, int ACT, typename T, int S>
__device__ __forceinline__ void reduce_rows(const LinParams& p, const float* part, int w0,
                                            int warps, int lane, int first, int limit, int tm,
                                            int tn) {
  constexpr bool G = MODE == kLinGated;
  constexpr int PER = G ? 2 : 1;                 // rows that a warp takes at once
  constexpr int R = (G ? 8 : 16) / S > 4 ? 4 : (G ? 8 : 16) / S;  // of those, in flight
  constexpr int TILE_N = G ? 64 : 128;
  const int piece = (G ? lane & 15 : lane) * 4, sub = G ? lane >> 4 : 0;
  const int rows = min(limit, p.m - tm * kLinTile);
  const int col = tn * TILE_N + piece;
  const bool in = col < p.n;
  uint32_t base[S];
#pragma unroll
  for (int s = 0; s < S; ++s) base[s] = S > 1 ? cluster_addr(part + piece, (uint32_t)s) : 0;
#pragma unroll 1
  for (int i = w0 * R * PER; first + i * S < rows; i += warps * R * PER) {
    float4 v[R][S], u[R][S];
    uint2 g_in[R], u_in[R];  // grad: PRE
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int r = first + (i + j * PER + sub) * S;
      if (r < rows && in) {
        if constexpr (MODE == kLinGrad) {
          const T* pre =
              reinterpret_cast<const T*>(p.pre_in) + (int64_t)(tm * kLinTile + r) * p.ldp_in + col;
          g_in[j] = *reinterpret_cast<const uint2*>(pre);
          u_in[j] = *reinterpret_cast<const uint2*>(pre + p.n);
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
          if constexpr (S == 1) {
            v[j][s] = *reinterpret_cast<const float4*>(part + r * kLinPitch + piece);
            if (G) u[j][s] = *reinterpret_cast<const float4*>(part + r * kLinPitch + 64 + piece);
          } else {
            v[j][s] = ld_shared_cluster_f32x4(base[s] + (uint32_t)r * (kLinPitch * 4));
            if (G) u[j][s] = ld_shared_cluster_f32x4(base[s] + (uint32_t)r * (kLinPitch * 4) + 256);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int r = first + (i + j * PER + sub) * S;
      if (r >= rows || !in) break;
      float4 a = v[j][0], b = G ? u[j][0] : a;
#pragma unroll
      for (int s = 1; s < S; ++s) {
        a.x += v[j][s].x;
        a.y += v[j][s].y;
        a.z += v[j][s].z;
        a.w += v[j][s].w;
        if (G) {
          b.x += u[j][s].x;
          b.y += u[j][s].y;
          b.z += u[j][s].z;
          b.w += u[j][s].w;
        }
      }
      finish4<MODE, ACT, T>(p, tm * kLinTile + r, col, a, b, g_in[j], u_in[j]);
    }
  }
}

// A warp's 32 rows of the accumulator (128 columns) to the partial tile.
__device__ __forceinline__ void keep_rows(uint32_t tmem, int q, int lane, float* part) {
#pragma unroll
  for (int c = 0; c < kLinTile; c += 64) {
    uint32_t v[2][32];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      tmem_ld32_async(tmem + ((uint32_t)(q * 32) << 16) + c + h * 32, v[h]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      tmem_ld_wait32(v[h]);
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<uint4*>(part + (q * 32 + lane) * kLinPitch + c + h * 32 + i) =
            make_uint4(v[h][i], v[h][i + 1], v[h][i + 2], v[h][i + 3]);
    }
  }
}

// After each CTA's rows are in its partial tile: the sum over the cluster, and the rows out.
template <int MODE, int ACT, typename T>
__device__ __forceinline__ void tile_out_as(const LinParams& p, const float* part, int warp, int lane,
                                         int rank, int tm, int tn, bool fine) {
  constexpr int W = kLinThreads / 32;
  if (p.split == 1) {
    if constexpr (MODE == kLinPlain) {
      // A warp writes the 32 rows that its own lanes stored.
      const int q = warp & 3;
      if (warp >= 2 && warp < kLinLoader && fine)
        reduce_rows<MODE, ACT, T, 1>(p, part, 0, 1, lane, q * 32, q * 32 + 32, tm, tn);
    } else {
      // The activations take longer than a barrier: all warps share the rows.
      __syncthreads();
      if (fine) reduce_rows<MODE, ACT, T, 1>(p, part, warp, W, lane, 0, kLinTile, tm, tn);
    }
    return;
  }
  cluster_sync();
  if (fine) {
    if (p.split == 2) reduce_rows<MODE, ACT, T, 2>(p, part, warp, W, lane, rank, kLinTile, tm, tn);
    else if (p.split == 3) reduce_rows<MODE, ACT, T, 3>(p, part, warp, W, lane, rank, kLinTile, tm, tn);
    else if (p.split == 6) reduce_rows<MODE, ACT, T, 6>(p, part, warp, W, lane, rank, kLinTile, tm, tn);
    else if (p.split == 4) reduce_rows<MODE, ACT, T, 4>(p, part, warp, W, lane, rank, kLinTile, tm, tn);
    else reduce_rows<MODE, ACT, T, 8>(p, part, warp, W, lane, rank, kLinTile, tm, tn);
  }
  __syncwarp();
  cluster_meet();  // no CTA leaves while another reads its partial sums
}

template <int MODE, typename T>
__device__ __forceinline__ void tile_out(const LinParams& p, const float* part, int warp, int lane,
                                         int rank, int tm, int tn, bool fine) {
  if constexpr (MODE != kLinPlain)
    with_act(p.act, [&](auto act) {
      tile_out_as<MODE, decltype(act)::value, T>(p, part, warp, lane, rank, tm, tn, fine);
    });
  else
    tile_out_as<MODE, 0, T>(p, part, warp, lane, rank, tm, tn, fine);
}

}  // namespace skg
