// The gated feed-forward block and its gradients, dense, in bf16 or fp16:
//   h = a(x Wg^T) * (x Wu^T)                                (moe_gated_ffn)
//   dg = dh u a'(g), du = dh a(g);  dx = [dg du] W1, dW1 = [dg du]^T x   (the backward)
//
// Every product runs on one kernel: persistent CTA pairs, tcgen05.mma.cta_group::2 on
// 256 x BN tiles, operands staged by TMA (128-byte swizzle) in a ring of mbarriers, two TMEM
// accumulators so that a tile's epilogue overlaps the next tile's main loop.
// * The gate and the up projection are one product of N = 2 x BN/2: the leader of the pair
//   stages BN/2 gate rows of W1 and the other CTA the BN/2 up rows of the same features, so
//   that g and u of an output meet in one thread's TMEM lane and the activation is the
//   epilogue. The backward computes them again instead of reading a stored copy: a stored
//   16-bit g would cost a rounding in a'(g) and 4 T I bytes kept from forward to backward.
// * dx and dW1 read operands whose summed dimension is the strided one (W1 as [2I, H] summed
//   over 2I; dg, du and x summed over tokens). They are staged as they lie, 64 columns x 64
//   summed rows per box, and the MMA reads them MN-major: nothing is transposed in memory.
//   Both products share one launch, so that the second's tiles fill the first's last wave.
#include <algorithm>

#include "activation.cuh"
#include "gated.h"

namespace moe_lora {

constexpr int kGBM = 128;         // rows per CTA (256 per pair)
constexpr int kGBK = 64;          // K per stage: 128 bytes
constexpr int kGEpiWarps = 8;
constexpr int kGThreads = 64 + 32 * kGEpiWarps;  // TMA warp, MMA warp, epilogue warps
constexpr int kGGroup = 8;        // row tiles per raster group
constexpr int kGPairs = 76;       // CTA pairs that the plans are made for (152 SMs)

template <int BN, int kEpi>
struct PairCfg {
  static constexpr int kABytes = kGBM * kGBK * 2;
  static constexpr int kBRows = BN / 2;  // rows (columns of the output) per CTA
  static constexpr int kBBytes = kBRows * kGBK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // 6 stages of 256 columns, 8 of 128, 9 of 64; one less where dh is staged too
  static constexpr int kRing = (kEpi == kEpiGrad ? 160 : 192) * 1024;
  static constexpr int kMostStages = 9;
  static constexpr int kOutOff = kRing;  // per epilogue warp 4 KB, and 4 KB of dh
  static constexpr int kWarpBytes = kEpi == kEpiGrad ? 8192 : 4096;
  static constexpr int kBarOff = kOutOff + kGEpiWarps * kWarpBytes;
  static constexpr int kSmemBytes = kBarOff + 512 + 1024;
  static constexpr uint32_t kTmemCols = 2 * BN;
  static_assert((2 * kMostStages + 5 + kGEpiWarps) * 8 + 16 <= 512, "barrier area");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// One product out[m, n] = sum_k A(m, k) B(n, k).
struct PairProblem {
  int M, N, K;         // N: columns of the output (features, for the gated forms)
  int tiles_m, tiles;  // 256-row tiles; all tiles, times ksplit
  int ksplit, kper;    // shares of the sum, and 64-wide steps per share
  int full, parts;     // gated: tiles from `full` on are cut into `parts` of their features each
  int a_mn, b_mn;      // the operand lies with m (n) contiguous, not k
  int up_off;          // gated: rows of B between gate and up
};

struct PairArgs {
  CUtensorMap tm[2][3];  // [problem][A, B, out]
  CUtensorMap tm_part;   // gated: B for a tile's parts
  CUtensorMap tm_dh;     // kEpiGrad: dh [M, N], 32 rows by 32 columns
  PairProblem p[2];
  int nproblems;
  int stages, stage_bytes;
  int light, extra;      // see unit_tile
  unsigned int* err;
  unsigned long long wait_ns;
};

__device__ unsigned int g_ffn_error;  // sticky MOE_LORA_DEVERR_* bits

// The tiles of pair `u` of `nu`, in order: problem 0's tiles u, u + nu, ...; then problem
// 1's. The pairs that got one tile fewer of problem 0 (the last `light` ones) first take
// `extra` tiles of problem 1 each -- as much work as that tile -- and the rest goes round.
__device__ __forceinline__ bool unit_tile(const PairArgs& a, int u, int nu, int i, int& prob, int& tile) {
  const int n0 = a.p[0].tiles;
  const int mine = u < n0 ? (n0 - 1 - u) / nu + 1 : 0;
  prob = 0;
  tile = u + i * nu;
  if (i < mine) return true;
  if (a.nproblems < 2) return false;
  prob = 1;
  int j = i - mine;
  if (u >= nu - a.light) {
    if (j < a.extra) {
      tile = (u - (nu - a.light)) * a.extra + j;
      return tile < a.p[1].tiles;
    }
    j -= a.extra;
  }
  // the remaining tiles start with the light pairs: the others may still be busy
  tile = a.light * a.extra + (nu - 1 - u) + j * nu;
  return tile < a.p[1].tiles;
}

// Where a tile lies. Row-grouped raster: kGGroup row tiles by every column tile, so that the
// pairs at work share rows of A and of B in L2. Shares of a split sum follow one another as
// whole rasters; the parts of a cut tile follow one another.
struct TilePlace {
  int tm, tn, ks;
  int part, parts;  // parts 1: whole
};
__device__ __forceinline__ TilePlace tile_place(const PairProblem& p, int tile) {
  TilePlace t = {0, 0, 0, 0, 1};
  int whole = p.tiles / p.ksplit;
  if (tile >= p.full) {
    const int s = tile - p.full;
    t.parts = p.parts;
    t.part = s % p.parts;
    tile = p.full + s / p.parts;
  }
  if (p.parts > 1) whole = p.full + (p.tiles - p.full) / p.parts;
  t.ks = tile / whole;
  tile -= t.ks * whole;
  const int tiles_n = whole / p.tiles_m;
  const int per = kGGroup * tiles_n;
  const int grp = tile / per, in = tile - grp * per;
  const int rows = min(kGGroup, p.tiles_m - grp * kGGroup);
  t.tm = grp * kGGroup + in % rows;
  t.tn = in / rows;
  return t;
}

// 16 bytes at unit c of row r of a staging tile in the order that a TMA store of 128- or
// 64-byte rows with the swizzle of that width reads it.
__device__ __forceinline__ uint4* staged(uint8_t* tile, int r, int c, bool wide) {
  return reinterpret_cast<uint4*>(wide ? tile + r * 128 + ((c ^ (r & 7)) << 4)
                                       : tile + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

template <typename T, int kEpi, int kAct, int BN>
__global__ void __launch_bounds__(kGThreads, 1) pair_gemm_kernel(const __grid_constant__ PairArgs a) {
  using C = PairCfg<BN, kEpi>;
  const int stages = a.stages, stage_bytes = a.stage_bytes;
  constexpr bool kGated = kEpi != kEpiStore;
  constexpr int kOutCols = kGated ? BN / 2 : BN;  // output columns per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kMostStages;
  uint64_t* tmem_full = empty + C::kMostStages;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* mma_done = tmem_empty + 2;
  uint64_t* dh_full = mma_done + 1;  // kEpiGrad: one per epilogue warp
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(dh_full + kGEpiWarps);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool leader = crank == 0;
  const int unit = blockIdx.x / 2, units = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);   // the leader's arming; the copies of both CTAs complete on it
      mbar_init(&empty[s], 1);  // the commit, to both CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], 2 * kGEpiWarps);  // of both CTAs, on the leader's
    }
    mbar_init(mma_done, 1);
    for (int i = 0; i < kGEpiWarps; ++i) mbar_init(&dh_full[i], 1);
    *s_abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    if (kEpi == kEpiGrad) tma_prefetch_desc(&a.tm_dh);
    for (int i = 0; i < a.nproblems; ++i) {
      tma_prefetch_desc(&a.tm[i][0]);
      tma_prefetch_desc(&a.tm[i][1]);
      tma_prefetch_desc(&a.tm[i][2]);
    }
  }
  cluster_sync();
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_wait();  // every input may come from the launch before
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now, with the tensor memory in hand: a dependent CTA on this SM may take the rest
  if (threadIdx.x == 0) pdl_trigger();
  const uint32_t tmem = *tmem_slot;

  auto set_abort = [&]() {
    *s_abort = 1;
    st_cluster_u32(smem_in_cta((const void*)s_abort, crank ^ 1u), 1u);
  };

  if (warp == 0) {
    // producer: the whole warp walks the loop (see the MMA issuer), one elected lane copies
    const bool elected = elect_one();
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t full0 = smem_in_cta(full, 0);
    int s = 0, prob, tile;
    uint32_t ph = 1;       // of the stage's emptying; the first round finds every stage empty
    bool filled = false;   // the ring has been filled once
    bool ok = true;
    for (int i = 0; ok && unit_tile(a, unit, units, i, prob, tile); ++i) {
      const PairProblem& p = a.p[prob];
      const TilePlace t = tile_place(p, tile);
      const CUtensorMap *ta = &a.tm[prob][0], *tb = kGated && t.parts > 1 ? &a.tm_part : &a.tm[prob][1];
      const int m0 = t.tm * 256 + (int)crank * kGBM;
      const int cols = kOutCols / t.parts;  // gated: features, as many rows of B in each CTA
      const int n0 = kGated ? t.tn * kOutCols + t.part * cols + (int)crank * p.up_off : t.tn * BN + (int)crank * C::kBRows;
      const uint32_t bytes = 2 * (C::kABytes + (kGated ? (uint32_t)cols * 128 : (uint32_t)C::kBBytes));
      const int k0 = t.ks * p.kper, k1 = min(k0 + p.kper, (p.K + kGBK - 1) / kGBK);
      const bool a_mn = p.a_mn != 0, b_mn = !kGated && p.b_mn != 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (filled) ok = __all_sync(0xffffffffu, mbar_wait_cluster(&empty[s], ph, a.wait_ns) && !*s_abort);
        if (!ok) break;
        if (elected) {
          uint8_t* sa = smem + s * stage_bytes;
          uint8_t* sb = sa + C::kABytes;
          const uint32_t bar = full0 + s * 8;
          if (leader) mbar_arrive_expect_tx(&full[s], bytes);
          if (a_mn) {
            tma_load_2d_pair(sa, ta, bar, m0, kb * kGBK, pol);
            tma_load_2d_pair(sa + 8192, ta, bar, m0 + 64, kb * kGBK, pol);
          } else {
            tma_load_2d_pair(sa, ta, bar, kb * kGBK, m0, pol);
          }
          if (b_mn) {
#pragma unroll
            for (int q = 0; q < C::kBRows / 64; ++q)
              tma_load_2d_pair(sb + q * 8192, tb, bar, n0 + 64 * q, kb * kGBK, pol);
          } else {
            tma_load_2d_pair(sb, tb, bar, kb * kGBK, n0, pol);
          }
        }
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1;
          filled = true;
        }
      }
    }
    if (!ok && lane == 0) set_abort();
  } else if (warp == 1) {
    // MMA issuer of the pair. The whole warp walks the loop, with votes where it branches, so
    // that descriptors and indexes stay in uniform registers; one elected lane issues. With
    // this loop and the producer's inside one-lane branches, every MMA and copy moved its
    // operands over from per-thread registers: 852 thousand cycles for 4096 tokens at
    // 4096/11008 (tensor pipe 70% active) against 689 thousand (87%).
    if (leader) {
      const bool elected = elect_one();
      int s = 0, prob, tile;
      uint32_t ph = 0;
      bool ok = true;
      for (int i = 0; ok && unit_tile(a, unit, units, i, prob, tile); ++i) {
        const PairProblem& p = a.p[prob];
        const TilePlace t = tile_place(p, tile);
        const int nk = min(p.kper, (p.K + kGBK - 1) / kGBK - t.ks * p.kper);
        const uint32_t acc = tmem + (uint32_t)((i & 1) * BN);
        const uint32_t idesc = (1u << 4) | (MmaType<T>::kFmt << 7) | (MmaType<T>::kFmt << 10) |
                               ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16) |
                               ((uint32_t)((BN / t.parts) >> 3) << 17) | ((256u >> 4) << 24);
        const uint32_t s0 = smem_u32(smem);
        const uint64_t da0 = p.a_mn ? smem_desc_mn(s0) : smem_desc_sw128(s0);
        const uint64_t db0 = p.b_mn ? smem_desc_mn(s0 + C::kABytes) : smem_desc_sw128(s0 + C::kABytes);
        // a K-major step of 16 is 32 bytes along the swizzled row; MN-major, 16 rows
        const uint32_t astep = p.a_mn ? 2048 >> 4 : 32 >> 4, bstep = p.b_mn ? 2048 >> 4 : 32 >> 4;
        if (i >= 2) ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tmem_empty[i & 1], ((i >> 1) - 1) & 1, a.wait_ns));
        tc_fence_after();
        for (int kb = 0; ok && kb < nk; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(&full[s], ph, a.wait_ns) && !*s_abort);
          if (!ok) break;
          tc_fence_after();
          if (elected) {
            const uint64_t off = (uint64_t)((uint32_t)(s * stage_bytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kGBK / 16; ++kk)
              tc_mma_bf16_pair(acc, da0 + off + kk * astep, db0 + off + kk * bstep, idesc, (kb | kk) != 0);
            tc_commit_pair_mc(&empty[s]);
          }
          __syncwarp();
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok && elected) tc_commit_pair_mc(&tmem_full[i & 1]);
        __syncwarp();
      }
      if (!ok && lane == 0) set_abort();
    }
  } else {
    // Epilogue: warp w reads TMEM lanes [32 (w % 4), + 32) -- 32 rows of the tile -- and half
    // of its columns, in chunks that it lays out in shared memory and stores with TMA: whole
    // lines reach L2, and rows and columns past the output's end are clipped by the map.
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stage = smem + C::kOutOff + (warp - 2) * C::kWarpBytes;
    // 4 KB hold 32 rows of 64 columns (or of 32 in fp32), or of 32 of dg and 32 of du. Gated,
    // the two warps of a row quarter take every other 32 features, as many as the tile has.
    constexpr int kWCols = kOutCols / 2;
    constexpr int kChunk = kGated ? 32 : 64;
    constexpr bool kWide = !kGated;
    // dh of a tile's chunks, behind the output's staging: fetched by TMA while the tile before is
    // at work. (Loaded straight into registers, a lane's row by itself, its 32 lines per
    // instruction kept the tensor cores from their operands in shared memory: 822 thousand
    // cycles against 711 without dh, at 4096 tokens of 4096/11008.)
    uint64_t* dh_bar = &dh_full[warp - 2];
    auto fetch_dh = [&](int i) {
      int prob, tile;
      if (!unit_tile(a, unit, units, i, prob, tile)) return;
      const TilePlace t = tile_place(a.p[prob], tile);
      const int cols = kOutCols / t.parts, m0 = t.tm * 256 + (int)crank * kGBM + quad * 32;
      const int n0 = t.tn * kOutCols + t.part * cols + half * 32;
      const int chunks = cols == 32 ? 1 - half : cols / 64;
      if (lane == 0 && chunks > 0) {
        const uint64_t pol = l2_policy_evict_first();
        mbar_arrive_expect_tx(dh_bar, (uint32_t)chunks * 2048);
        for (int c = 0; c < chunks; ++c)
          tma_load_2d(stage + 4096 + c * 2048, &a.tm_dh, dh_bar, n0 + c * 64, m0, pol);
      }
    };
    uint32_t dh_ph = 0;
    if (kEpi == kEpiGrad) fetch_dh(0);
    int prob, tile;
    for (int i = 0; unit_tile(a, unit, units, i, prob, tile); ++i) {
      const PairProblem& p = a.p[prob];
      const CUtensorMap* to = &a.tm[prob][2];
      const TilePlace t = tile_place(p, tile);
      const int cols = kOutCols / t.parts;
      const int m0 = t.tm * 256 + (int)crank * kGBM + quad * 32;
      const int n0 = kGated ? t.tn * kOutCols + t.part * cols + half * 32 : t.tn * kOutCols + half * kWCols;
      bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tmem_full[i & 1], (i >> 1) & 1, a.wait_ns) ? 1 : 0);
      if (kEpi == kEpiGrad && half * 32 < cols) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(dh_bar, dh_ph, a.wait_ns) && ok);
        dh_ph ^= 1;
      }
      if (!ok && lane == 0) set_abort();
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)((i & 1) * BN + half * (kGated ? 32 : kWCols)) + ((uint32_t)(quad * 32) << 16);
      if (kEpi == kEpiStore && p.ksplit > 1) {
        // a share of a split sum: fp32, 32 columns a chunk (the map counts 16-bit units)
        for (int c = 0; c < kWCols; c += 32) {
          uint32_t v[2][16];
          __syncwarp();
          tmem_ld_x16(acc + c, v[0]);
          tmem_ld_x16(acc + c + 16, v[1]);
          tmem_ld_wait();
          if (lane == 0) bulk_wait_read();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 8; ++q)
            *staged(stage, lane, q, true) = make_uint4(v[q / 4][4 * (q % 4)], v[q / 4][4 * (q % 4) + 1],
                                                       v[q / 4][4 * (q % 4) + 2], v[q / 4][4 * (q % 4) + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (m0 < p.M && n0 + c < p.N) tma_store_3d(to, stage, 2 * (n0 + c), t.ks, m0);
            bulk_commit();
          }
        }
      } else {
#pragma unroll
        for (int ch = 0; ch < kWCols / kChunk; ++ch) {
          const int c = ch * (kGated ? 64 : kChunk);
          if (kGated && half * 32 + c >= cols) break;
          if (lane == 0) bulk_wait_read();
          __syncwarp();
#pragma unroll
          for (int b = 0; b < kChunk; b += 16) {
            uint32_t v[16], w[16];
            tmem_ld_x16(acc + c + b, v);
            if (kGated) tmem_ld_x16(acc + cols + c + b, w);
            tmem_ld_wait();
            uint32_t o[8], o2[8];
            uint4 d[2] = {};
            if (kEpi == kEpiGrad) {
              d[0] = *staged(stage + 4096 + ch * 2048, lane, b / 8, false);
              d[1] = *staged(stage + 4096 + ch * 2048, lane, b / 8 + 1, false);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float g0 = __uint_as_float(v[2 * q]), g1 = __uint_as_float(v[2 * q + 1]);
              if (kEpi == kEpiStore) {
                o[q] = Elem<T>::r2(g0, g1);
              } else {
                const float u0 = __uint_as_float(w[2 * q]), u1 = __uint_as_float(w[2 * q + 1]);
                float a0, a1, d0, d1;
                activation<kAct>(g0, a0, d0);
                activation<kAct>(g1, a1, d1);
                if (kEpi == kEpiGated) {
                  o[q] = Elem<T>::r2(a0 * u0, a1 * u1);
                } else {
                  const uint4& dd = d[q / 4];
                  const uint32_t dw = q % 4 == 0 ? dd.x : q % 4 == 1 ? dd.y : q % 4 == 2 ? dd.z : dd.w;
                  const float2 e = Elem<T>::f2(dw);
                  o[q] = Elem<T>::r2(e.x * u0 * d0, e.y * u1 * d1);
                  o2[q] = Elem<T>::r2(e.x * a0, e.y * a1);
                }
              }
            }
            *staged(stage, lane, b / 8, kWide) = make_uint4(o[0], o[1], o[2], o[3]);
            *staged(stage, lane, b / 8 + 1, kWide) = make_uint4(o[4], o[5], o[6], o[7]);
            if (kEpi == kEpiGrad) {
              *staged(stage + 2048, lane, b / 8, kWide) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
              *staged(stage + 2048, lane, b / 8 + 1, kWide) = make_uint4(o2[4], o2[5], o2[6], o2[7]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (m0 < p.M && n0 + c < p.N) {
              tma_store_3d(to, stage, n0 + c, 0, m0);
              if (kEpi == kEpiGrad) tma_store_3d(to, stage + 2048, n0 + c, 1, m0);
            }
            bulk_commit();
          }
        }
      }
      tc_fence_before();
      if (kEpi == kEpiGrad) fence_proxy_async_smem();  // dh has been read: its place may be written again
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(smem_in_cta(&tmem_empty[i & 1], 0));
      if (kEpi == kEpiGrad) fetch_dh(i + 1);
    }
    if (lane == 0) bulk_wait_read();  // the stores themselves are over when the grid is
  }
  tc_fence_before();
  __syncwarp();
  cluster_sync();
  // Every role of both CTAs has stopped issuing. After a give-up copies may still be landing
  // and MMAs still running: both are drained before the memory is freed. The two CTAs may have
  // stopped at different stages, so no phase of a full barrier can be awaited exactly; a copy
  // is at most 16 KB, and 100 us is far beyond its flight time.
  const bool aborted = *s_abort != 0;
  if (aborted && threadIdx.x == 0) {
    const unsigned long long t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 100000ull) {
    }
    atomicOr(a.err, MOE_LORA_DEVERR_TIMEOUT);
  }
  if (aborted && warp == 1 && leader) {
    if (elect_one()) tc_commit_pair(mma_done);  // the lane that issued the MMAs
    __syncwarp();
    mbar_wait_bounded(mma_done, 0);
  }
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::kTmemCols);
  }
}

// out = the shares of a split sum [ksplit][n] added in order, for up to two products.
struct SumShares {
  const float* part[2];
  void* out[2];
  int64_t n[2];  // a multiple of 8
  int ksplit[2];
};
template <typename T>
__global__ void __launch_bounds__(256) sum_shares_kernel(const SumShares s) {
  pdl_wait();
  const int64_t n8 = s.n[0] / 8, all = n8 + s.n[1] / 8;
  for (int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x; j < all; j += (int64_t)gridDim.x * 256) {
    const int q = j >= n8;
    const int64_t i = (q ? j - n8 : j) * 8;
    float4 a = {}, b = {};
    for (int k = 0; k < s.ksplit[q]; ++k) {
      const float4* p = reinterpret_cast<const float4*>(s.part[q] + k * s.n[q] + i);
      const float4 u = __ldcg(p), v = __ldcg(p + 1);
      a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
      b.x += v.x; b.y += v.y; b.z += v.z; b.w += v.w;
    }
    *reinterpret_cast<uint4*>(static_cast<T*>(s.out[q]) + i) =
        make_uint4(Elem<T>::r2(a.x, a.y), Elem<T>::r2(a.z, a.w), Elem<T>::r2(b.x, b.y), Elem<T>::r2(b.z, b.w));
  }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
int ffn_error_word(unsigned int** out) {
  static std::atomic<uint64_t> seen[kMaxDevices];
  static std::atomic<unsigned int*> addr[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_LORA_ERR_CUDA;
  const int st = once_per_context(seen, [dev] {
    void* p = nullptr;
    ML_CHECK_CUDA(cudaGetSymbolAddress(&p, g_ffn_error));
    addr[dev].store(static_cast<unsigned int*>(p));
    return MOE_LORA_OK;
  });
  *out = addr[dev].load();
  return st;
}

static thread_local unsigned long long t_wait_ns = kWaitLimitNs;
unsigned long long ffn_wait_ns() { return t_wait_ns; }

int operand_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, bool mn, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, (uint32_t)(mn ? 64 : box_rows)};
  return make_tmap_bf16(m, base, 2, dims, strides, box);  // any 16-bit type: bytes are moved
}

// The 64-wide steps that a tile's epilogue takes as long as: no tile is over sooner.
constexpr int kEpiSteps = 6;

struct ProblemDesc {
  const void *A, *B;
  int M, N, K;
  bool a_mn, b_mn;
  void* out;     // [M, parts, N] of 16-bit elements, or fp32 [ksplit, M, N] of a split sum
  int parts;
  int ksplit;
};

template <typename T, int kEpi, int kAct, int BN>
static int launch_pair(const ProblemDesc* d, int n, const void* dh, cudaStream_t stream) {
  using C = PairCfg<BN, kEpi>;
  constexpr bool kGated = kEpi != kEpiStore;
  auto kernel = pair_gemm_kernel<T, kEpi, kAct, BN>;
  static std::atomic<uint64_t> seen[kMaxDevices];
  static std::atomic<int> resident[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_LORA_ERR_CUDA;
  int st = once_per_context(seen, [&] {
    ML_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)num_sms());
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    ML_CHECK_CUDA(cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg));
    if (clusters < 1) return MOE_LORA_ERR_UNSUPPORTED;
    resident[dev].store(clusters);
    return MOE_LORA_OK;
  });
  if (st != MOE_LORA_OK) return st;
  PairArgs a = {};
  int64_t all = 0;
  for (int i = 0; i < n; ++i) {
    PairProblem& p = a.p[i];
    p.M = d[i].M;
    p.N = d[i].N;
    p.K = d[i].K;
    p.a_mn = d[i].a_mn;
    p.b_mn = d[i].b_mn;
    p.kper = ceil_div(ceil_div(p.K, kGBK), d[i].ksplit);
    p.ksplit = d[i].ksplit;
    p.up_off = kGated ? p.N : 0;
    p.tiles_m = ceil_div(p.M, 256);
    const int64_t tiles = (int64_t)p.tiles_m * ceil_div(p.N, kGated ? BN / 2 : BN) * p.ksplit;
    if (tiles > (1 << 28)) return MOE_LORA_ERR_UNSUPPORTED;
    p.tiles = (int)tiles;
    p.full = p.tiles;
    p.parts = 1;
    if (kGated) {
      // The last wave's tiles are cut into parts of their features where that ends it sooner:
      // half a tile takes about two thirds of its time, a quarter little less (the copies of the
      // rows of A, which every part reads whole, then take longer than the MMAs).
      const int pairs = resident[dev].load(), last = p.tiles % pairs;
      double best = 1.0;
      for (int parts = 2; parts <= 4 && last; parts *= 2) {
        const double cost = ceil_div(last * parts, pairs) * (parts == 2 ? 0.65 : 0.6);
        if (cost < best) {
          best = cost;
          p.parts = parts;
        }
      }
      p.full = p.tiles - (p.parts > 1 ? last : 0);
      p.tiles = p.full + (p.parts > 1 ? last * p.parts : 0);
    }
    all += p.tiles;
    st = operand_map(&a.tm[i][0], d[i].A, p.a_mn ? p.K : p.M, p.a_mn ? p.M : p.K, p.a_mn, kGBM);
    if (st != MOE_LORA_OK) return st;
    const int64_t bn_rows = kGated ? 2 * (int64_t)p.N : p.N;
    st = operand_map(&a.tm[i][1], d[i].B, p.b_mn ? p.K : bn_rows, p.b_mn ? bn_rows : p.K, p.b_mn, C::kBRows);
    if (st != MOE_LORA_OK) return st;
    if (p.parts > 1) {
      st = operand_map(&a.tm_part, d[i].B, bn_rows, p.K, false, BN / 2 / p.parts);
      if (st != MOE_LORA_OK) return st;
    }
    {
      // the output as the epilogue stores it: 32 rows by 64 or 32 columns
      const bool split = p.ksplit > 1;
      const int parts = split ? p.ksplit : d[i].parts;
      const uint64_t cols = (uint64_t)p.N * (split ? 2 : 1);
      const bool narrow = kGated;
      const uint64_t dims[3] = {cols, (uint64_t)parts, (uint64_t)p.M};
      const uint64_t strides[2] = {split ? cols * 2 * p.M : cols * 2, split ? cols * 2 : cols * 2 * parts};
      const uint32_t box[3] = {narrow ? 32u : 64u, 1, 32};
      st = make_tmap_bf16(&a.tm[i][2], d[i].out, 3, dims, strides, box,
                          narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
      if (st != MOE_LORA_OK) return st;
    }
  }
  // with every tile cut, stages are smaller and there are more of them
  a.stage_bytes = kGated && a.p[0].full == 0 ? C::kABytes + C::kBBytes / a.p[0].parts : C::kStageBytes;
  a.stages = std::min(C::kMostStages, C::kRing / a.stage_bytes);
  if (kEpi == kEpiGrad) {
    const uint64_t dims[2] = {(uint64_t)a.p[0].N, (uint64_t)a.p[0].M};
    const uint64_t strides[1] = {(uint64_t)a.p[0].N * 2};
    const uint32_t box[2] = {32, 32};
    if ((st = make_tmap_bf16(&a.tm_dh, dh, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B)) != MOE_LORA_OK) return st;
  }
  a.nproblems = n;
  a.wait_ns = ffn_wait_ns();
  if ((st = ffn_error_word(&a.err)) != MOE_LORA_OK) return st;
  const int units = (int)std::min<int64_t>(all, resident[dev].load());
  if (n == 2 && a.p[0].tiles % units) {
    a.light = units - a.p[0].tiles % units;
    const int c0 = std::max(a.p[0].kper, kEpiSteps), c1 = std::max(a.p[1].kper, kEpiSteps);
    a.extra = (c0 + c1 / 2) / c1;
    a.extra = std::min(a.extra, a.p[1].tiles / a.light);
  }
  return launch_pdl_cluster(kernel, dim3(2 * (unsigned)units), kGThreads, C::kSmemBytes, stream, true, 2, a);
}

// The backward's plan: 256-row tiles of bn columns, each sum in ksplit shares.
struct PairPlan {
  int bn;
  int ksplit[2];
};

// Cycles that a 64-wide step of a tile takes: the MMAs' own at 256 columns; at 128 the copies
// into shared memory take longer than the MMAs.
static double step_cost(int bn) { return bn == 256 ? 512 : 320; }

// The plan of two products (m, n, k each) on kGPairs pairs. A sum is split where one tile's
// exceeds what every pair would do on average, into shares of 8 steps at least; the estimate
// adds half a tile for the last wave and the pass that adds the shares.
static PairPlan plan_products(const int (*mnk)[3]) {
  PairPlan best = {256, {1, 1}};
  double best_cost = 0;
  for (int bn = 256; bn >= 128; bn /= 2) {
    PairPlan pl = {bn, {1, 1}};
    double total = 0, longest = 0, extra = 0, steps[2];
    for (int i = 0; i < 2; ++i) {
      steps[i] = std::max(ceil_div(mnk[i][2], kGBK), kEpiSteps);
      total += (double)ceil_div(mnk[i][0], 256) * ceil_div(mnk[i][1], bn) * steps[i];
    }
    const double mean = total / kGPairs;
    for (int i = 0; i < 2; ++i) {
      int ks = 1;
      if (steps[i] > 1.5 * mean) {
        ks = (int)std::min(steps[i] / std::max(mean, 1.0) + 0.5, steps[i] / 8);
        ks = std::max(1, std::min(ks, 16));
        const int per = ceil_div((int)steps[i], ks);
        ks = ceil_div(ceil_div(mnk[i][2], kGBK), per);
      }
      pl.ksplit[i] = ks;
      longest = std::max(longest, steps[i] / ks);
      if (ks > 1) extra = 4000;
    }
    const double cost = std::max(mean + 0.5 * longest, longest) * step_cost(bn) + extra;
    if (bn == 256 || cost < best_cost) {
      best = pl;
      best_cost = cost;
    }
  }
  return best;
}

// The backward's two products of dy = [dg | du], in the order they run (the longer sums
// first), their plan, and the places of the shares of split sums behind dy in the workspace.
// The plan is the same when only one of them is wanted, and so are its bits.
struct BackwardPlan {
  int mnk[2][3];
  bool is_dx[2];
  PairPlan plan;
  size_t part_off[2], bytes;
};
static BackwardPlan plan_backward(int T, int H, int I) {
  BackwardPlan b = {};
  for (int i = 0; i < 2; ++i) {
    b.is_dx[i] = (i == 0) == (2 * I >= T);
    b.mnk[i][0] = b.is_dx[i] ? T : 2 * I;
    b.mnk[i][1] = H;
    b.mnk[i][2] = b.is_dx[i] ? 2 * I : T;
  }
  b.plan = plan_products(b.mnk);
  b.bytes = round_up((size_t)T * 2 * I * 2, 256);
  for (int i = 0; i < 2; ++i) {
    b.part_off[i] = b.bytes;
    if (b.plan.ksplit[i] > 1) b.bytes += round_up((size_t)b.plan.ksplit[i] * b.mnk[i][0] * b.mnk[i][1] * 4, 256);
  }
  return b;
}

template <typename T>
static int launch_backward_products(const BackwardPlan& b, const void* dy, char* workspace, const void* x,
                                    const void* W1, void* dx, void* dW1, cudaStream_t stream) {
  ProblemDesc d[2];
  SumShares sums = {};
  int n = 0, nsums = 0;
  int64_t work = 0;
  for (int i = 0; i < 2; ++i) {
    void* out = b.is_dx[i] ? dx : dW1;
    if (!out) continue;
    const int ks = b.plan.ksplit[i];
    if (ks > 1) {
      sums.part[nsums] = reinterpret_cast<const float*>(workspace + b.part_off[i]);
      sums.out[nsums] = out;
      sums.n[nsums] = (int64_t)b.mnk[i][0] * b.mnk[i][1];
      work += sums.n[nsums] / 8;
      sums.ksplit[nsums++] = ks;
      out = workspace + b.part_off[i];
    }
    d[n++] = {dy, b.is_dx[i] ? W1 : x, b.mnk[i][0], b.mnk[i][1], b.mnk[i][2], !b.is_dx[i], true, out, 1, ks};
  }
  const int st = b.plan.bn == 256 ? launch_pair<T, kEpiStore, MOE_ACT_NONE, 256>(d, n, nullptr, stream)
                                  : launch_pair<T, kEpiStore, MOE_ACT_NONE, 128>(d, n, nullptr, stream);
  if (st != MOE_LORA_OK || nsums == 0) return st;
  return launch_pdl(sum_shares_kernel<T>, (unsigned)std::min<int64_t>(ceil_div64(work, 256), 152 * 8), 256, 0, stream,
                    true, sums);
}

static int check_gated(int dtype, int act, int T, int H, int I) {
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_LORA_ERR_INVALID_ARG;
  if (act != MOE_ACT_SILU && act != MOE_ACT_GELU) return MOE_LORA_ERR_INVALID_ARG;
  if (T < 0 || H < 1 || I < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (H % 8 != 0 || I % 8 != 0 || T > (1 << 22) || H > (1 << 21) || I > (1 << 20))
    return MOE_LORA_ERR_UNSUPPORTED;
  return MOE_LORA_OK;
}

template <int kEpi>
static int launch_gated(int dtype, int act, const void* x, const void* W1, int T, int H, int I,
                        const void* dh, void* out, cudaStream_t stream) {
  if (T <= kFewTokens) return launch_gated_few(dtype, act, x, W1, T, H, I, dh, out, stream);
  const ProblemDesc d = {x, W1, T, I, H, false, false, out, kEpi == kEpiGrad ? 2 : 1, 1};
  if (dtype == MOE_DTYPE_BF16)
    return act == MOE_ACT_SILU ? launch_pair<__nv_bfloat16, kEpi, MOE_ACT_SILU, 256>(&d, 1, dh, stream)
                               : launch_pair<__nv_bfloat16, kEpi, MOE_ACT_GELU, 256>(&d, 1, dh, stream);
  return act == MOE_ACT_SILU ? launch_pair<__half, kEpi, MOE_ACT_SILU, 256>(&d, 1, dh, stream)
                             : launch_pair<__half, kEpi, MOE_ACT_GELU, 256>(&d, 1, dh, stream);
}

}  // namespace moe_lora

extern "C" int moe_ffn_get_error(moe_lora_stream_t stream, uint32_t* err) {
  using namespace moe_lora;
  if (!err) return MOE_LORA_ERR_INVALID_ARG;
  unsigned int* p = nullptr;
  const int st = ffn_error_word(&p);
  if (st != MOE_LORA_OK) return st;
  return moe_lora_get_error(p, stream, err);
}

extern "C" int moe_ffn_clear_error(moe_lora_stream_t stream) {
  using namespace moe_lora;
  unsigned int* p = nullptr;
  const int st = ffn_error_word(&p);
  return st == MOE_LORA_OK ? moe_lora_clear_error(p, stream) : st;
}

extern "C" int moe_ffn_set_wait_limit(int64_t ns) {
  using namespace moe_lora;
  t_wait_ns = ns == 0 ? kWaitLimitNs : ns < 0 ? 0ull : (unsigned long long)ns;
  return MOE_LORA_OK;
}

extern "C" int moe_gated_ffn(const void* x, const void* W1, int dtype, int act, int T, int H, int I,
                             void* h, moe_lora_stream_t stream) {
  using namespace moe_lora;
  int st = check_gated(dtype, act, T, H, I);
  if (st != MOE_LORA_OK) return st;
  if (T == 0) return MOE_LORA_OK;
  if (!x || !W1 || !h || !aligned16(x) || !aligned16(W1) || !aligned16(h)) return MOE_LORA_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  return launch_gated<kEpiGated>(dtype, act, x, W1, T, H, I, nullptr, h,
                                 reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_gated_ffn_backward_workspace_size(int T, int H, int I) {
  using namespace moe_lora;
  if (check_gated(MOE_DTYPE_BF16, MOE_ACT_SILU, T, H, I) != MOE_LORA_OK) return 0;
  return std::max<size_t>(plan_backward(T, H, I).bytes, 256);
}

extern "C" int moe_gated_ffn_backward(const void* dh, const void* x, const void* W1, int dtype,
                                      int act, int T, int H, int I, void* dx, void* dW1,
                                      void* workspace, size_t workspace_bytes,
                                      moe_lora_stream_t stream) {
  using namespace moe_lora;
  int st = check_gated(dtype, act, T, H, I);
  if (st != MOE_LORA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!aligned16(dx) || !aligned16(dW1)) return MOE_LORA_ERR_INVALID_ARG;
  if (!dx && !dW1) return MOE_LORA_OK;
  if (T == 0) {
    if ((st = check_device()) != MOE_LORA_OK) return st;
    if (dW1) ML_CHECK_CUDA(cudaMemsetAsync(dW1, 0, (size_t)2 * I * H * 2, s));
    return MOE_LORA_OK;
  }
  if (!dh || !x || !W1 || !aligned16(dh) || !aligned16(x) || !aligned16(W1)) return MOE_LORA_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return MOE_LORA_ERR_INVALID_ARG;
  if (workspace_bytes < moe_gated_ffn_backward_workspace_size(T, H, I)) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  // dy = [dg | du] [T, 2I] in the workspace, then both products of it
  if ((st = launch_gated<kEpiGrad>(dtype, act, x, W1, T, H, I, dh, workspace, s)) != MOE_LORA_OK) return st;
  if (dx && T <= kFewTokens) {
    if ((st = launch_dx_few(dtype, workspace, W1, T, H, I, dx, s)) != MOE_LORA_OK || !dW1) return st;
    dx = nullptr;
  }
  const BackwardPlan b = plan_backward(T, H, I);
  char* ws = static_cast<char*>(workspace);
  return dtype == MOE_DTYPE_BF16 ? launch_backward_products<__nv_bfloat16>(b, ws, ws, x, W1, dx, dW1, s)
                                 : launch_backward_products<__half>(b, ws, ws, x, W1, dx, dW1, s);
}
