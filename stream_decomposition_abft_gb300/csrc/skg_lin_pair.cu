// A layer's projections on CTA pairs: persistent clusters of two CTAs, 256 x 256 tiles of
// the accumulator with one M = 256 MMA (tcgen05 cta_group::2). Each CTA loads its 128 rows
// of A and half of B's 256 rows per stage; the leader issues the MMAs. TMEM holds two
// accumulators, so the way out of one tile runs under the MMAs of the next.
//
// In the gated mode the leader's half of B is 128 columns of the gate's projection and the
// other CTA's the same 128 of the other, so every thread finds both of its row in its own
// TMEM lane, 128 columns apart. Adapters as in skg_lin_single.cu: more stages of k for each
// adapter that the tile's 256 rows use, with the other rows left out of the MMA.
//
// Operands stored along k or along their rows are read in place (MN-major boxes of 64 x 64).
// Two weight gradients of the same k share a launch.
//
// What bounds it: the MMAs under the power limit. 4096 x 8192 -> 28672 gated in bf16 takes
// 1.91 to 1.99 ms in short runs and 2.19 in long ones (2.0 and 1.76 PFLOP/s); the tensor pipe
// is busy 93 % of the time at 2048 x 8192 -> 8192 (94 to 97 % in the gradients' products,
// 72 % with PRE, both gradients and H on the way out, whose 256 tiles take four rounds of 76
// pairs where 3.4 would do). Few tiles: a stage of k is 0.262 us, 502 of its 512 cycles MMAs.
//
// What the waits' bounds and the way out share with the block-scaled product's pairs is
// explained there (skg_mx_gemm_pair.cu).
#include "skg_lin.cuh"

namespace skg {
namespace {

struct PairAux : LinAux {
  uint64_t pre[8];  // kLinGrad: a warp's two sets of boxes of PRE are there
};

template <int MODE>
struct PairCfg {
  static constexpr int STAGE_BYTES = 2 * kLinOperand;
  // Boxes of 32 rows x 128 bytes for each epilogue warp: two on their way out; kLinGated: of H,
  // gate and up; kLinGrad: two sets of gate and up, in and out, and one of H.
  static constexpr int WARP_STAGING = 4096 * (MODE == kLinGrad ? 5 : MODE == kLinGated ? 3 : 2);
  static constexpr int STAGING = 4 * WARP_STAGING;
  static constexpr int STAGES = MODE == kLinGrad ? 4 : MODE == kLinGated ? 5 : 6;
  static constexpr uint32_t SMEM = 1024 + STAGES * STAGE_BYTES + STAGING + 512;
  static_assert(SMEM <= kSmemLimit, "shared memory");
  static_assert(sizeof(PairAux) <= 512, "aux size");
};

// A box of 32 rows x 128 bytes (this lane's row: the values f(0), f(1), ...) in the 128-byte
// swizzle, and its store by TMA; two boxes per warp in turn. The engine clips what is past
// the matrix, to whole 16 bytes (store_rest); returns the box.
template <typename T, typename F>
__device__ __forceinline__ uint8_t* store_box(const CUtensorMap* map, uint8_t* staging, uint32_t& box,
                                          int lane, int col, int row, F f) {
  constexpr int PER = 16 / (int)sizeof(T);
  uint8_t* st = staging + (box & 1) * 4096;
  ++box;
  if (lane == 0) bulk_wait_read<1>();  // the box's last store has read it
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    union {
      T e[PER];
      uint4 q;
    } u;
#pragma unroll
    for (int i = 0; i < PER; ++i) u.e[i] = mx_from_f32<T>(f(j * PER + i));
    *reinterpret_cast<uint4*>(st + lane * 128 + ((j ^ (lane & 7)) << 4)) = u.q;
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, st, col, row);
    bulk_commit();
  }
  return st;
}

// 16 values of this lane's row to columns 16 c of its box.
template <typename T>
__device__ __forceinline__ void box_write16(uint8_t* st, int lane, int c, const float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    union {
      T e[8];
      uint4 q;
    } u;
#pragma unroll
    for (int i = 0; i < 8; ++i) u.e[i] = mx_from_f32<T>(v[h * 8 + i]);
    *reinterpret_cast<uint4*>(st + lane * 128 + (((2 * c + h) ^ (lane & 7)) << 4)) = u.q;
  }
}
template <typename T>
__device__ __forceinline__ void box_read16(const uint8_t* st, int lane, int c, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    union {
      T e[8];
      uint4 q;
    } u;
    u.q = *reinterpret_cast<const uint4*>(st + lane * 128 + (((2 * c + h) ^ (lane & 7)) << 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[h * 8 + i] = mx_to_f32(u.e[i]);
  }
}

// The way out of a gated tile and of a gradient's, 16 columns at a time in a loop that is not
// unrolled: the activations are long, and in straight lines of 64 columns a warp waited for
// instructions most of the time (the gradient of a 256 x 256 tile 40 to 60 us). `done` once
// all of the accumulator is read. cols: the tile's columns that are C's.
template <int ACT, typename T, typename Done>
__device__ __forceinline__ void gated_out(const LinParams& p, const LinMaps& maps, uint32_t acc,
                                          uint8_t* mine, uint32_t& box, int lane, int col0,
                                          int row0, int cols, Done done) {
  const int count = (cols + 15) / 16;
  const bool pre = p.pre != nullptr;
  if (count == 0) {
    done();
    return;
  }
  uint32_t g[16], u[16], g2[16], u2[16];
  auto fetch = [&](int i) {
    const uint32_t at = acc + i * 16;
    tmem_ld16_async(at, g2);
    tmem_ld16_async(at + 128, u2);
  };
  uint8_t* hb = mine;
  fetch(0);
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    tmem_ld_wait16(g2);
    tmem_ld_wait16(u2);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      g[j] = g2[j];
      u[j] = u2[j];
    }
    if (i + 1 < count) fetch(i + 1);
    else done();
    if ((i & 3) == 0) {  // boxes whose stores have read them
      if (!pre) hb = mine + (box++ & 1) * 4096;
      if (lane == 0) {
        if (pre) bulk_wait_read<0>();
        else bulk_wait_read<1>();
      }
      __syncwarp();
    }
    float h[16], a[16], b[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      a[j] = __uint_as_float(g[j]);
      b[j] = __uint_as_float(u[j]);
      h[j] = lin_gated<ACT>(a[j], b[j]);
    }
    box_write16<T>(hb, lane, i & 3, h);
    if (pre) {
      box_write16<T>(mine + 4096, lane, i & 3, a);
      box_write16<T>(mine + 8192, lane, i & 3, b);
    }
    if ((i & 3) == 3 || i + 1 == count) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int col = col0 + (i >> 2) * 64;
        tma_store_2d(&maps.c, hb, col, row0);
        if (pre) {
          tma_store_2d(&maps.gate, mine + 4096, col, row0);
          tma_store_2d(&maps.pre_up, mine + 8192, col, row0);
        }
        bulk_commit();
      }
    }
  }
}

// PRE of 64 columns to a warp's set number `pres` & 1 of boxes.
__device__ __forceinline__ void fetch_pre(const LinMaps& maps, PairAux* aux, uint8_t* mine, int q,
                                          uint32_t pres, int col, int row0) {
  uint8_t* set = mine + (pres & 1u) * 8192;
  uint64_t* bar = &aux->pre[q * 2 + (pres & 1u)];
  fence_proxy_async_smem();
  mbar_arrive_expect_tx(bar, 8192);
  tma_load_2d(set, &maps.t, bar, col, row0);
  tma_load_2d(set + 4096, &maps.up, bar, col, row0);
}

template <int ACT, typename T, typename Done>
__device__ __forceinline__ void grad_out(const LinParams& p, const LinMaps& maps, PairAux* aux,
                                         uint32_t acc, uint8_t* mine, uint32_t& pres, int q,
                                         int lane, int col0, int row0, int cols, Done done) {
  const int count = (cols + 15) / 16;
  if (count == 0) {
    done();
    return;
  }
  uint32_t v[16], v2[16];
  uint8_t* set = mine;
  uint8_t* hb = mine + 16384;
  tmem_ld16_async(acc, v2);
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    tmem_ld_wait16(v2);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = v2[j];
    if (i + 1 < count) tmem_ld16_async(acc + (i + 1) * 16, v2);
    else done();
    if ((i & 3) == 0) {
      if (!mx_wait(&aux->pre[q * 2 + (pres & 1u)], (pres >> 1) & 1u, aux, true)) lin_fail(p, aux);
      set = mine + (pres & 1u) * 8192;
      ++pres;
      // The other set and H's box: their stores have read them. PRE of the next 64 columns
      // comes while these are worked on.
      if (lane == 0) {
        bulk_wait_read<0>();
        if (i + 4 < count) fetch_pre(maps, aux, mine, q, pres, col0 + (i >> 2) * 64 + 64, row0);
      }
      __syncwarp();
    }
    float g[16], u[16], h[16];
    box_read16<T>(set, lane, i & 3, g);
    box_read16<T>(set + 4096, lane, i & 3, u);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const LinGrad r = lin_grad<ACT>(__uint_as_float(v[j]), g[j], u[j]);
      g[j] = r.dg;
      u[j] = r.du;
      h[j] = r.h;
    }
    box_write16<T>(set, lane, i & 3, g);
    box_write16<T>(set + 4096, lane, i & 3, u);
    box_write16<T>(hb, lane, i & 3, h);
    if ((i & 3) == 3 || i + 1 == count) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const int col = col0 + (i >> 2) * 64;
        tma_store_2d(&maps.gate, set, col, row0);
        tma_store_2d(&maps.pre_up, set + 4096, col, row0);
        tma_store_2d(&maps.c, hb, col, row0);
        bulk_commit();
      }
    }
  }
}

// Tile t in an order that keeps the tiles in flight close together: bands of eight rows of
// tiles, column by column within a band (2048 rows of A stay in L2 while B passes).
// Returns whether it is the second product's.
template <bool TWO>
__device__ __forceinline__ bool pair_tile(const LinParams& p, int t, int& tm, int& tn) {
  constexpr int kBand = 8;
  const bool second = TWO && t >= p.tiles_m * p.tiles_n;
  const int tiles_m = second ? p.second.tiles_m : p.tiles_m;
  const int tiles_n = second ? p.second.tiles_n : p.tiles_n;
  if (second) t -= p.tiles_m * p.tiles_n;
  const int band = t / (kBand * tiles_n);
  const int rows = min(kBand, tiles_m - band * kBand);
  const int i = t - band * kBand * tiles_n;
  tn = i / rows;
  tm = band * kBand + i % rows;
  return second;
}

template <int MODE, bool AMN, bool BMN, typename T>
__global__ void __launch_bounds__(kLinThreads, 1)
lin_pair_kernel(const __grid_constant__ LinMaps maps, const LinParams p) {
  using C = PairCfg<MODE>;
  constexpr bool G = MODE == kLinGated;
  constexpr bool LORA = MODE == kLinPlain && !AMN && !BMN;
  constexpr int TILE_N = G ? 128 : 256;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* staging = ring + C::STAGES * C::STAGE_BYTES;
  PairAux* aux = reinterpret_cast<PairAux*>(staging + C::STAGING);
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  constexpr bool TWO = AMN && BMN;
  const int tiles = p.tiles_m * p.tiles_n + (TWO ? p.second.tiles_m * p.second.tiles_n : 0);
  const int first = (int)blockIdx.x >> 1, stride = (int)gridDim.x >> 1;
  const bool lora = LORA && p.plan != nullptr;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.c);
    aux->abort_flag = 0;
    aux->limit = p.limit;
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&aux->full[i], 1);
      mbar_init(&aux->empty[i], 1);
    }
    mbar_init(&aux->tfull[0], 1);
    mbar_init(&aux->tfull[1], 1);
    mbar_init(&aux->tempty, 8);  // the epilogue warps of both CTAs
    mbar_init(&aux->tempty1, 8);
    mbar_init(&aux->drain, 1);
    for (int i = 0; i < 8; ++i) mbar_init(&aux->pre[i], 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&aux->tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = aux->tmem_slot;
  if (!lora) {  // see skg_lin_single.cu
    griddep_wait();
    if (threadIdx.x == 0) griddep_launch_dependents();
  }

  uint32_t seq = 0;  // loading threads: stages gone through, every other one by this thread
  const uint32_t me = warp == kLinLoader;
  if (warp == 0 || warp == kLinLoader) {
    if (elect_one()) {
      int st = 0;
      uint32_t phase = 0;
      bool ok = true, waited = false;
      // One stage of so many bytes in either CTA: when it is this thread's and free,
      // load(address, the leader's barrier).
      auto step = [&](uint32_t bytes, auto load) {
        if ((seq & 1u) == me) {
          if (seq >= p.stages) {
            ok = false;
            return;
          }
          if (!mx_wait(&aux->empty[st], phase ^ 1u, aux)) {
            lin_fail(p, aux);
            ok = false;
            return;
          }
          if (rank == 0) mbar_arrive_expect_tx(&aux->full[st], 2 * bytes);
          load(ring + st * C::STAGE_BYTES, cluster_addr(&aux->full[st], 0));
        }
        ++seq;
        if (++st == C::STAGES) {
          st = 0;
          phase ^= 1u;
        }
      };
      // Four adapters of a plan from the u-th on (past their number: anything; past the
      // plan's end its last entry).
      auto read = [](const LoraPlan* plan, int u, int (&id)[4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e) id[e] = plan->id[min(u + e, kLoraRows - 1)];
      };
      int id[4] = {0, 0, 0, 0}, count = 0;
      const int ks = p.ksteps * p.terms;
      for (int t = first; ok && t < tiles; t += stride) {
        int tm, tn;
        const bool second = pair_tile<TWO>(p, t, tm, tn);
        const int lo_b = second ? p.second.lo_b : p.lo_b;
        const CUtensorMap *map_a = second ? &maps.t : &maps.a, *map_b = second ? &maps.up : &maps.b,
                          *map_lo = second ? &maps.gate : &maps.lo;
        const int row = (2 * tm + rank) * kLinTile;
        // The plan is read ahead of its use, the first entries beside their number.
        if (waited) {
          read(p.plan + tm, 0, id);
          count = p.plan[tm].count;
        }
        // Rows of B: this CTA's projection (gated), else its half of the tile's columns.
        const int col = G ? rank * p.n + tn * 128 : tn * 256 + rank * 128;
        for (int i = 0; ok && i < ks; ++i)
          step(C::STAGE_BYTES, [&](uint8_t* s, uint32_t bar) {
            const bool lo = p.terms == 2 && (i & 1);
            const int k0 = (p.terms == 2 ? i >> 1 : i) * kLinK;
            const CUtensorMap* ma = lo && !lo_b ? map_lo : map_a;
            const CUtensorMap* mb = lo && lo_b ? map_lo : map_b;
            if constexpr (AMN) {
              tma_load_2d_pair(s, ma, bar, row, k0);
              tma_load_2d_pair(s + kLinBox, ma, bar, row + 64, k0);
            } else {
              tma_load_2d_pair(s, ma, bar, k0, row);
            }
            if constexpr (BMN) {
              tma_load_2d_pair(s + kLinOperand, mb, bar, col, k0);
              tma_load_2d_pair(s + kLinOperand + kLinBox, mb, bar, col + 64, k0);
            } else {
              tma_load_2d_pair(s + kLinOperand, mb, bar, k0, col);
            }
          });
        if (ok && lora) {
          if (!waited) {
            griddep_wait();
            griddep_launch_dependents();
            waited = true;
            read(p.plan + tm, 0, id);
            count = p.plan[tm].count;
          }
          const int rp = p.rank_pad, pack = lora_pack(rp), per = lora_stages(rp);
          const uint32_t one = (uint32_t)lora_bytes(rp);
          for (int u = 0; ok && u < count; u += pack) {
            const int here = min(pack, count - u);
            int behind[4];
            read(p.plan + tm, u + pack, behind);
            for (int j = 0; ok && j < per; ++j)
              step(kLinOperand + here * one, [&](uint8_t* s, uint32_t bar) {
                tma_load_2d_pair(s, &maps.t, bar, lora_col_t(rp, j), row);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (e < here)
                    tma_load_3d_pair(s + kLinOperand + e * one, &maps.up, bar, lora_col_b(rp, j),
                                     col, id[e]);
              });
#pragma unroll
            for (int e = 0; e < 4; ++e) id[e] = behind[e];
          }
        }
      }
      // A grid ends behind the one that it waits for.
      if (lora && !waited) griddep_wait();
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one() && rank == 0) {
      LinRing<C::STAGES> r = {aux, aux->full};
      const uint64_t a0 = lin_desc<AMN>(smem_u32(ring));
      const uint64_t b0 = lin_desc<BMN>(smem_u32(ring) + kLinOperand);
      int n = 0;
      bool ok = true, waited = false;
      // The rows to leave out for four adapters (as the loading thread reads them).
      auto read = [](const LoraPlan* plan, int u, uint32_t (&off)[4][8]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int w = 0; w < 8; ++w) off[e][w] = ~plan->rows[min(u + e, kLoraRows - 1)][w];
      };
      uint32_t off[4][8];
      int count = 0;
      const int terms = p.terms, k = p.k;
      const uint32_t idesc = p.idesc;
      const int ks = p.ksteps * p.terms;
      for (int t = first; ok && t < tiles; t += stride, ++n) {
        // The accumulator's last tile is out of it.
        if (n > 1 && !mx_wait((n & 1) ? &aux->tempty1 : &aux->tempty, (uint32_t)((n >> 1) - 1) & 1u,
                              aux)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + (n & 1) * 256;
        const LoraPlan* plan = nullptr;
        if (lora) {
          int tm, tn;
          pair_tile<false>(p, t, tm, tn);
          plan = p.plan + tm;
          if (waited) {
            read(plan, 0, off);
            count = plan->count;
          }
        }
        for (int i = 0; i < ks; ++i) {
          const int st = r.take();
          ok = st >= 0;
          if (!ok) break;
          const uint64_t at = (uint64_t)((st * C::STAGE_BYTES) >> 4);
          lin_stage_mmas<true, AMN, BMN>(d, a0 + at, b0 + at, idesc,
                                         k - (terms == 2 ? i >> 1 : i) * kLinK, i == 0);
          umma_commit_pair(&aux->empty[st]);
        }
        if (ok && lora) {
          if (!waited) {
            griddep_wait();
            waited = true;
            read(plan, 0, off);
            count = plan->count;
          }
          const int rp = p.rank_pad, pack = lora_pack(rp), per = lora_stages(rp);
          for (int u = 0; ok && u < count; u += pack) {
            const int here = min(pack, count - u);
            uint32_t behind[4][8];
            read(plan, u + pack, behind);
            for (int j = 0; j < per; ++j) {
              const int st = r.take();
              ok = st >= 0;
              if (!ok) break;
              const uint32_t s = smem_u32(ring + st * C::STAGE_BYTES);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (e < here) lora_stage_mmas<true>(d, s, s + kLinOperand, idesc, rp, j, e, off[e]);
              umma_commit_pair(&aux->empty[st]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int w = 0; w < 8; ++w) off[e][w] = behind[e][w];
          }
        }
        if (ok) umma_commit_pair(&aux->tfull[n & 1]);
      }
      if (!ok) lin_fail(p, aux);
      if (r.used > 0) {
        umma_commit_pair(&aux->drain);
        mx_wait(&aux->drain, 0, aux, true);
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;
    uint8_t* mine = staging + q * C::WARP_STAGING;
    uint32_t box = 0, pres = 0;
    int n = 0;
    for (int t = first; t < tiles; t += stride, ++n) {
      int tm, tn;
      const bool second = pair_tile<TWO>(p, t, tm, tn);
      const int pm = second ? p.second.m : p.m, pn = second ? p.second.n : p.n;
      const int row0 = (2 * tm + rank) * kLinTile + q * 32, col0 = tn * TILE_N;
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (n & 1) * 256;
      const bool live = row0 < pm;
      // (PRE's first 64 columns come while the MMAs are under way.)
      const int cols = live ? min(TILE_N, pn - col0) : 0;
      if (MODE == kLinGrad && cols > 0 && lane == 0)
        fetch_pre(maps, aux, mine, q, pres, col0, row0);
      __syncwarp();
      const bool got = mx_wait(&aux->tfull[n & 1], (uint32_t)(n >> 1) & 1u, aux);
      if (!got) lin_fail(p, aux);
      if (!__all_sync(0xffffffffu, got)) {
        // (What fetch_pre asked for lands before the CTA leaves.)
        if (MODE == kLinGrad && cols > 0)
          mx_wait(&aux->pre[q * 2 + (pres & 1u)], (pres >> 1) & 1u, aux, true);
        break;
      }
      tc_fence_after();
      auto hand_over = [&]() {  // all of the tile is in registers
        tc_fence_before();
        __syncwarp();
        if (lane == 0)
          mbar_arrive_remote(cluster_addr((n & 1) ? &aux->tempty1 : &aux->tempty, 0u));
      };
      if constexpr (G) {
        with_act(p.act, [&](auto act) {
          gated_out<decltype(act)::value, T>(p, maps, acc, mine, box, lane, col0, row0, cols,
                                             hand_over);
        });
      } else if constexpr (MODE == kLinGrad) {
        with_act(p.act, [&](auto act) {
          grad_out<decltype(act)::value, T>(p, maps, aux, acc, mine, pres, q, lane, col0, row0,
                                            cols, hand_over);
        });
      } else {
        // Four pieces of 64 columns.
        uint32_t v[2][2][32];
        auto fetch = [&](int s) {
#pragma unroll
          for (int i = 0; i < 2; ++i) tmem_ld32_async(acc + s * 64 + i * 32, v[s & 1][i]);
        };
        fetch(0);
        fetch(1);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          tmem_ld_wait32(v[s & 1][0]);
          tmem_ld_wait32(v[s & 1][1]);
          const int col = col0 + s * 64;
          if (s == 3) hand_over();
          if (live && col < pn) {
            const uint8_t* st =
                store_box<T>(second ? &maps.pre_up : &maps.c, mine, box, lane, col, row0,
                             [&](int i) { return __uint_as_float(v[s & 1][i >> 5][i & 31]); });
            if ((pn & 7) && col + 64 > (pn & ~7))
              store_rest<T>(second ? p.second.c : p.c, second ? p.second.ldc : p.ldc, pm, pn, st,
                            lane, col, row0);
          }
          if (s < 2) fetch(s + 2);
        }
      }
    }
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  // As in skg_mx_gemm_pair.cu: copies that no MMA waited for land before the pair parts, the
  // leader's last commit has reached the other CTA's barrier, and no CTA leaves while the
  // other may still signal its barriers.
  if (warp == 1 && rank == 1 && first < tiles && elect_one()) mx_wait(&aux->drain, 0, aux, true);
  if (rank == 0 && seq > 0 && mx_aborted(aux))
    for (uint32_t i = seq > C::STAGES ? seq - C::STAGES : 0; i < seq; ++i)
      if ((i & 1u) == me)
        mx_wait(&aux->full[i % C::STAGES], (i / C::STAGES) & 1u, aux, true);
  if (rank == 1 && seq > 0 && mx_aborted(aux))
    for (const uint64_t t0 = globaltimer(); globaltimer() - t0 < 1000000ull;) __nanosleep(1000);
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(&p.report->launches, 1u);
}

template <int MODE, bool AMN, bool BMN, typename T>
cudaError_t launch(const LinMaps& t, const LinParams& p, int clusters, cudaStream_t stream) {
  auto kernel = lin_pair_kernel<MODE, AMN, BMN, T>;
  static std::atomic<uint64_t> done_mask{0};
  const cudaError_t e = opt_in_smem((const void*)kernel, done_mask, (int)PairCfg<MODE>::SMEM);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(kernel, dim3((unsigned)(2 * clusters)), dim3(kLinThreads),
                            PairCfg<MODE>::SMEM, stream, 2, t, p);
}

template <typename T>
cudaError_t launch_type(const LinVariant& v, const LinMaps& t, const LinParams& p, int clusters,
                        cudaStream_t stream) {
  if (v.mode == kLinGated) return launch<kLinGated, false, false, T>(t, p, clusters, stream);
  if (v.mode == kLinGrad) return launch<kLinGrad, false, true, T>(t, p, clusters, stream);
  if (v.a_mn) return launch<kLinPlain, true, true, T>(t, p, clusters, stream);
  if (v.b_mn) return launch<kLinPlain, false, true, T>(t, p, clusters, stream);
  return launch<kLinPlain, false, false, T>(t, p, clusters, stream);
}

}  // namespace

cudaError_t launch_lin_pair(const LinVariant& v, const LinMaps& t, const LinParams& p,
                            int clusters, cudaStream_t stream) {
  if (v.out == SKG_OUT_F16) return launch_type<__half>(v, t, p, clusters, stream);
  return launch_type<__nv_bfloat16>(v, t, p, clusters, stream);
}

int lin_pair_clusters_resident() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int have = cached[dev].load(std::memory_order_acquire);
  if (have != 0) return have > 0 ? have : 0;
  auto kernel = lin_pair_kernel<kLinGated, false, false, __nv_bfloat16>;  // all alike in resources
  const int n = clusters_resident((const void*)kernel, PairCfg<kLinGated>::SMEM, 2);
  cached[dev].store(n > 0 ? n : -1, std::memory_order_release);
  return n;
}

}  // namespace skg
