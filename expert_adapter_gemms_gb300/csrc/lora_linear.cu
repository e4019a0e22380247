// The projection with adapters for many rows, on tcgen05 CTA pairs, and its C entry points.
//
// out = in M(e)^T + z U(e, l)^T over 256-row tiles of one expert's sorted rows (the align
// buffer's tiles) by up to 256 columns: persistent CTA pairs, tcgen05.mma.cta_group::2, operands by TMA
// (128-byte swizzle) in a ring of mbarriers, two TMEM accumulators so that a tile's epilogue
// overlaps the next tile's main loop. The same kernel computes y (M = W, U = B, summed over
// contiguous columns) and dx (M = W, U = A as they lie, read MN-major).
// * The adapters are further steps of the same sum, [in | z][M | U]^T, for each adapter of the
//   tile. A step's MMAs write only the TMEM lanes of the rows with that adapter
//   (disable-output-lane), so that no row meets another request's weights, not even times zero:
//   an infinity or NaN in one adapter stays with its own rows.
// * A tile's z is written once for all its adapters, by four warps of their own, from the fp32 z
//   that the pass before left, beside the ring and ahead of the base steps.
// * In sorted order, the base steps do not wait for that pass: it began only when everything
//   before it was complete, and so may they read it. In the tokens' order they wait where groups
//   of rows come from its copies.
// * A tile ends where its expert's rows end: rows past that are not stored.
// dx of 4096 rows by 4096 columns over 11008: 230 us (1.6 PFLOP/s, tensor pipe 89 % active); 16384
// rows of 32 experts and 16 adapters by 5760 over 2880: 440 us cold (1.25 PFLOP/s, 80 %: 81 row tiles
// for 64 tiles' rows); dense rows as many 300 us (1.8 PFLOP/s).
#include <algorithm>

#include "lora_linear.h"

namespace moe_lora {

constexpr int kLBM = 128;  // rows per CTA (256 per pair)
constexpr int kLBK = 64;   // summed columns per stage: 128 bytes
constexpr int kLEpiWarps = 8, kLZWarps = 4;
constexpr int kLThreads = 64 + 32 * (kLEpiWarps + kLZWarps);
constexpr int kLGroup = 8;  // row tiles per raster group

struct LinCfg {
  static constexpr int kABytes = kLBM * kLBK * 2;
  static constexpr int kBRows = 128;  // columns of the output per CTA, at most
  static constexpr int kStageBytes = kABytes + kBRows * kLBK * 2;
  // z of a step in one tile up to 32 ranks, else in two and a stage less
  static constexpr int kMostStages = 6;
  static constexpr int kOutBytes = kLEpiWarps * 2048;  // 32 rows of 32 columns per epilogue warp
  static constexpr int kBarBytes = 256;
  static constexpr int kSmemBytes = kMostStages * kStageBytes + kABytes + kOutBytes + kBarBytes + 1024;
  static constexpr uint32_t kAccCols = 256, kTmemCols = 2 * kAccCols;
  static_assert(kABytes <= kStageBytes, "the second z tile takes a stage's place");
  static_assert((2 * kMostStages + 7) * 8 + 8 <= kBarBytes, "barrier area");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

struct LinArgs {
  CUtensorMap tm_in[2], tm_sorted[2], tm_m, tm_u, tm_out;  // boxes of 128 rows and of a group's
  LinearRows rows;
  const float* z;
  void* out;
  int N, K, r;
  int width, tiles_n;  // columns per tile: a multiple of 32 (of 128 where mn), half of them per CTA
  int stages;
  int mn;  // M and U lie with the output's columns contiguous
  unsigned int* err;
  unsigned long long wait_ns;
};

// Row-grouped raster: kLGroup row tiles by every column tile, so that the pairs at work share
// rows and weights in L2. (At most 2^30 tiles: check_linear.)
__device__ __forceinline__ bool lin_tile(int i, int unit, int units, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int tile = unit + i * units;
  if (tile >= tiles_m * tiles_n) return false;
  const int per = kLGroup * tiles_n;
  const int grp = tile / per, in = tile - grp * per;
  const int rows = min(kLGroup, tiles_m - grp * kLGroup);
  tm = grp * kLGroup + in % rows;
  tn = in / rows;
  return true;
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, const void* src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

template <typename T>
__global__ void __launch_bounds__(kLThreads, 1) linear_pair_kernel(const __grid_constant__ LinArgs a) {
  using C = LinCfg;
  const int stages = a.stages, cta_cols = a.width / 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* z_tile = smem + stages * C::kStageBytes;
  const RankSteps rs(a.r);
  uint8_t* out_stage = z_tile + rs.tiles * C::kABytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_stage + C::kOutBytes);
  uint64_t* empty = full + C::kMostStages;
  uint64_t* tmem_full = empty + C::kMostStages;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* z_full = tmem_empty + 2;
  uint64_t* z_empty = z_full + 1;
  uint64_t* mma_done = z_empty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool leader = crank == 0;
  const int unit = blockIdx.x / 2, units = gridDim.x / 2;
  const int together = rs.together(), u_ranks = 64 / together, u_bytes = C::kBRows * u_ranks * 2;
  const int boxes = cta_cols / 64;  // of 64 columns, where M lies with its columns contiguous

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);   // the leader's arming; the copies of both CTAs complete on it
      mbar_init(&empty[s], 1);  // the commit, to both CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], 2 * kLEpiWarps);  // of both CTAs, on the leader's
    }
    mbar_init(z_full, 2 * kLZWarps);  // likewise
    mbar_init(z_empty, 1);            // the commit, to both CTAs
    mbar_init(mma_done, 1);
    *s_abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&a.tm_in[0]);
    if (a.rows.slots) {
      tma_prefetch_desc(&a.tm_in[1]);
      tma_prefetch_desc(&a.tm_sorted[0]);
      tma_prefetch_desc(&a.tm_sorted[1]);
    }
    tma_prefetch_desc(&a.tm_m);
    tma_prefetch_desc(&a.tm_u);
    tma_prefetch_desc(&a.tm_out);
  }
  cluster_sync();
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int tiles_m = __ldcg(a.rows.hdr + HDR_NTILES);
  const int nk = (a.K + kLBK - 1) / kLBK;

  auto set_abort = [&]() {
    *s_abort = 1;
    st_cluster_u32(smem_in_cta((const void*)s_abort, crank ^ 1u), 1u);
  };

  if (warp == 0) {
    // producer: the whole warp walks the loop, one elected lane copies
    const bool elected = elect_one();
    const uint64_t pol = l2_policy_evict_normal();
    const uint32_t full0 = smem_in_cta(full, 0);
    int s = 0, tm, tn;
    uint32_t ph = 1;  // of the stage's emptying
    bool filled = false, ok = true, waited = false;
    auto slot_free = [&]() {
      return !filled || __all_sync(0xffffffffu, mbar_wait_cluster(&empty[s], ph, a.wait_ns) && !*s_abort);
    };
    auto advance = [&]() {
      __syncwarp();
      if (++s == stages) {
        s = 0;
        ph ^= 1;
        filled = true;
      }
    };
    // A tile's place and where its rows come from, looked up while the tile before is under way:
    // the looks' latencies in a row would leave the ring empty.
    int4 t;  // expert, first row, rows
    Runs<8> runs;
    int from[4];     // where each group of this CTA's rows starts, in the tokens' order or in the copy
    bool copied[4];
    auto look = [&](int4 tile) {
      t = tile;
      runs.load(a.rows.row_adapter, t.y, t.z);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (a group past the tile's end: whatever follows the one before)
        from[j] = j ? from[j - 1] + kLinearGroup : 0;
        copied[j] = j && copied[j - 1];
        const int at = (int)crank * kLBM + j * kLinearGroup, n = min(kLinearGroup, t.z - at);
        if (a.rows.slots && n > 0) {
          from[j] = __shfl_sync(0xffffffffu, group_row(a.rows.slots, t.y + at, n, &copied[j]), 0);
          if (copied[j]) from[j] = t.y + at;
        }
      }
    };
    bool more = lin_tile(0, unit, units, tiles_m, a.tiles_n, tm, tn);
    if (more) look(__ldcg(a.rows.tiles + tm));
    for (int i = 0; ok && more; ++i) {
      const int n0 = tn * a.width + (int)crank * cta_cols;
      const int e = t.x;
      Runs<8> mine = runs;
      // one box where all rows follow one another (4 of a group each: 415 against 370 us for 16384
      // rows of 2880/5760)
      int at[4];
      const CUtensorMap* map[4];
      bool any_copied = false, one_box = true;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        at[j] = a.rows.slots ? from[j] : t.y + (int)crank * kLBM;
        map[j] = copied[j] ? &a.tm_sorted[1] : &a.tm_in[1];
        any_copied |= copied[j];
        if (a.rows.slots) one_box &= copied[j] == copied[0] && from[j] == from[0] + j * kLinearGroup;
      }
      if (one_box) map[0] = copied[0] ? &a.tm_sorted[0] : &a.tm_in[0];
      if (any_copied && !waited) {
        pdl_wait();
        waited = true;
      }
      int next_tm = 0, next_tn = 0;
      int4 next_t = {};
      auto copy_cols = [&](const CUtensorMap* m, uint8_t* sb, uint32_t bar, int k, int third, int block) {
        if (a.mn) {
          tma_load_3d_pair(sb, m, bar, n0, k, third, pol);
          if (boxes > 1) tma_load_3d_pair(sb + block, m, bar, n0 + 64, k, third, pol);
        } else {
          tma_load_3d_pair(sb, m, bar, k, n0, third, pol);
        }
      };
      for (int kb = 0; kb < nk; ++kb) {
        ok = slot_free();
        if (!ok) break;
        uint8_t* sa = smem + s * C::kStageBytes;
        const uint32_t bar = full0 + s * 8;
        if (elected) {
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * (C::kABytes + cta_cols * (kLBK * 2)));
          copy_cols(&a.tm_m, sa + C::kABytes, bar, kb * kLBK, e, 8192);
          tma_load_2d_pair(sa, map[0], bar, kb * kLBK, at[0], pol);
          if (!one_box)
#pragma unroll
            for (int j = 1; j < 4; ++j)
              tma_load_2d_pair(sa + j * (kLinearGroup * 128), map[j], bar, kb * kLBK, at[j], pol);
        }
        advance();
        if (kb == nk / 4) {
          more = lin_tile(i + 1, unit, units, tiles_m, a.tiles_n, next_tm, next_tn);
          if (more) next_t = __ldcg(a.rows.tiles + next_tm);
        }
        if (kb == nk / 2 && more) look(next_t);
      }
      for (int st = 0; ok && st < rs.steps; ++st) {
        mine.find();
        for (int l = mine.next(); l >= 0;) {
          ok = slot_free();
          if (!ok) break;
          // the next adapters' U one after the other in the stage
          int ls[4] = {l, -1, -1, -1}, n = 1;
#pragma unroll
          for (int j = 1; j < 4; ++j)
            if (j < together && ls[j - 1] >= 0) {
              ls[j] = mine.next();
              n += ls[j] >= 0;
            }
          l = n == together ? mine.next() : -1;
          if (elected) {
            if (leader) mbar_arrive_expect_tx(&full[s], (uint32_t)(2 * n * cta_cols * u_ranks * 2));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < n)
                copy_cols(&a.tm_u, smem + s * C::kStageBytes + C::kABytes + j * u_bytes, full0 + s * 8, 64 * st,
                          ls[j] * a.rows.E + e, u_ranks * 128);
          }
          advance();
        }
      }
      tm = next_tm;
      tn = next_tn;
    }
    if (!ok && lane == 0) set_abort();
  } else if (warp == 1) {
    // MMA issuer of the pair: a warp-uniform loop, one elected lane issues
    if (leader) {
      const bool elected = elect_one();
      const uint32_t idesc = (1u << 4) | (MmaType<T>::kFmt << 7) | (MmaType<T>::kFmt << 10) | ((uint32_t)a.mn << 16) |
                             ((uint32_t)(a.width >> 3) << 17) | ((256u >> 4) << 24);
      const uint32_t s0 = smem_u32(smem);
      const uint64_t da0 = smem_desc_sw128(s0), dz0 = smem_desc_sw128(smem_u32(z_tile));
      const uint64_t db0 = a.mn ? smem_desc_mn(s0 + C::kABytes) : smem_desc_sw128(s0 + C::kABytes);
      const uint32_t bstep = a.mn ? 2048 >> 4 : 32 >> 4;
      // U as it lies in its part of a stage: rows of u_ranks ranks under the swizzle of their
      // width, or blocks of u_ranks rows of 64 columns
      const uint64_t du0 = a.mn ? smem_desc_mn(s0 + C::kABytes, u_ranks * 128)
                           : u_ranks == 64 ? smem_desc_sw128(s0 + C::kABytes)
                           : u_ranks == 32 ? smem_desc_swz(s0 + C::kABytes, 4, 512)
                                           : smem_desc_swz(s0 + C::kABytes, 6, 256);
      int s = 0, tm, tn, zi = 0;
      uint32_t ph = 0;
      bool ok = true;
      auto advance = [&]() {
        __syncwarp();
        if (++s == stages) {
          s = 0;
          ph ^= 1;
        }
      };
      // (the adapters of the next tile's rows are looked up meanwhile, as the producer does)
      bool more = lin_tile(0, unit, units, tiles_m, a.tiles_n, tm, tn);
      Runs<8> runs, next;
      if (more) {
        const int4 t = __ldcg(a.rows.tiles + tm);
        next.load(a.rows.row_adapter, t.y, t.z);
      }
      for (int i = 0; ok && more; ++i) {
        const uint32_t acc = tmem + (uint32_t)(i & 1) * C::kAccCols;
        runs = next;
        int4 t = {};
        if (i >= 2) ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tmem_empty[i & 1], ((i >> 1) - 1) & 1, a.wait_ns));
        tc_fence_after();
        for (int kb = 0; ok && kb < nk; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(&full[s], ph, a.wait_ns) && !*s_abort);
          if (!ok) break;
          tc_fence_after();
          if (elected) {
            const uint64_t off = (uint64_t)((uint32_t)(s * C::kStageBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kLBK / 16; ++kk)
              tc_mma_bf16_pair(acc, da0 + off + kk * 2, db0 + off + kk * bstep, idesc, (kb | kk) != 0);
            tc_commit_pair_mc(&empty[s]);
          }
          advance();
          if (kb == nk / 4) {
            more = lin_tile(i + 1, unit, units, tiles_m, a.tiles_n, tm, tn);
            if (more) t = __ldcg(a.rows.tiles + tm);
          }
          if (kb == nk / 2) {
            runs.find();
            if (more) next.load(a.rows.row_adapter, t.y, t.z);
          }
        }
        for (int st = 0; ok && st < rs.steps; ++st) {
          if (st > 0) runs.find();
          if (!runs.any()) break;
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(z_full, zi & 1, a.wait_ns) && !*s_abort);
          const int nu = rs.u_mmas(st);
          const uint32_t low = rs.low(st, C::kABytes);
          for (int l = ok ? runs.next() : -1; l >= 0;) {
            ok = __all_sync(0xffffffffu, mbar_wait_cluster(&full[s], ph, a.wait_ns) && !*s_abort);
            if (!ok) break;
            tc_fence_after();
            uint64_t du = du0 + (uint64_t)((uint32_t)(s * C::kStageBytes) >> 4);
            for (int j = 0; j < together && l >= 0; ++j) {
              uint32_t off_rows[8];  // the lanes of the pair's rows that have another adapter
#pragma unroll
              for (int q = 0; q < 8; ++q) off_rows[q] = __ballot_sync(0xffffffffu, runs.ad[q] != l);
              if (elected)
                for (int kk = 0; kk < nu; ++kk) {
                  tc_mma_lanes_pair(acc, dz0 + kk * 2, du + kk * bstep, idesc, off_rows);
                  tc_mma_lanes_pair(acc, dz0 + low + kk * 2, du + kk * bstep, idesc, off_rows);
                }
              __syncwarp();
              du += (uint32_t)u_bytes >> 4;
              l = runs.next();
            }
            if (elected) tc_commit_pair_mc(&empty[s]);
            advance();
          }
          if (ok && elected) tc_commit_pair_mc(z_empty);
          __syncwarp();
          ++zi;
        }
        if (ok && elected) tc_commit_pair_mc(&tmem_full[i & 1]);
        __syncwarp();
      }
      if (!ok && lane == 0) set_abort();
    }
  } else if (warp >= 2 + kLEpiWarps) {
    // z writers: a thread per row of this CTA
    const int i0 = (int)threadIdx.x - 32 * (2 + kLEpiWarps);
    int tm, tn, zi = 0;
    bool ok = true;
    pdl_wait();  // z is the launch before's
    if (i0 == 0) pdl_trigger();
    for (int i = 0; ok && lin_tile(i, unit, units, tiles_m, a.tiles_n, tm, tn); ++i) {
      const int4 t = __ldcg(a.rows.tiles + tm);
      const int at = (int)crank * kLBM + i0;
      const bool mine = at < t.z && __ldcg(a.rows.row_adapter + t.y + at) >= 0;
      const float* zrow = a.z + (int64_t)(t.y + at) * a.r;
      Runs<8> runs;
      runs.load(a.rows.row_adapter, t.y, t.z);
      runs.find();
      if (!runs.any()) continue;
      for (int st = 0; st < rs.steps; ++st, ++zi) {
        if (zi > 0) ok = __all_sync(0xffffffffu, mbar_wait_cluster(z_empty, (zi - 1) & 1, a.wait_ns) && !*s_abort);
        if (!ok) break;
        write_z_row<T>(z_tile, C::kABytes, i0, zrow, mine, a.r, rs, st);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(smem_in_cta(z_full, 0));
      }
    }
    if (!ok && lane == 0) set_abort();
  } else {
    // Epilogue: warp w takes TMEM lanes [32 (w % 4), + 32) -- 32 rows -- and half of the
    // columns, 32 at a time. Rows that are neighbours in the output are laid out in shared memory
    // and stored by TMA (stored by their lanes, 16 bytes at a time, they held up the copies of
    // operands: 334 against 284 us without stores, for 16384 rows of 2880/5760); others, and
    // those of a tile's ragged end, by their lanes.
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* stage = out_stage + (warp - 2) * 2048;
    // the halves in whole chunks
    const int first_cols = (cta_cols + 31) / 32 * 32, col0 = half ? first_cols : 0, cols = half ? a.width - first_cols : first_cols;
    int tm, tn;
    for (int i = 0; lin_tile(i, unit, units, tiles_m, a.tiles_n, tm, tn); ++i) {
      const int4 t = __ldcg(a.rows.tiles + tm);
      const int at = (int)crank * kLBM + quad * 32;
      int row = t.y + at + lane;  // this lane's row of the output, -1: none
      if (at + lane >= t.z) row = -1;
      else if (a.rows.slots) row = __ldcg(a.rows.slots + row);
      const int row0 = __shfl_sync(0xffffffffu, row, 0);
      const bool together_out = __all_sync(0xffffffffu, row >= 0 && row == row0 + lane);
      const int n0 = tn * a.width + col0;
      const bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tmem_full[i & 1], (i >> 1) & 1, a.wait_ns) ? 1 : 0);
      if (!ok && lane == 0) set_abort();
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)(i & 1) * C::kAccCols + col0 + ((uint32_t)(quad * 32) << 16);
      T* to = static_cast<T*>(a.out) + (int64_t)row * a.N + n0;
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
        if (at >= t.z || n0 + c >= a.N) break;
        uint32_t v[2][16];
        tmem_ld_x16(acc + c, v[0]);
        tmem_ld_x16(acc + c + 16, v[1]);
        if (lane == 0) bulk_wait_read();  // the last store has read the staging
        tmem_ld_wait();
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t o[4];
#pragma unroll
          for (int p = 0; p < 4; ++p)
            o[p] = Elem<T>::r2(__uint_as_float(v[q / 2][q % 2 * 8 + 2 * p]), __uint_as_float(v[q / 2][q % 2 * 8 + 2 * p + 1]));
          if (together_out)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
          else if (row >= 0 && n0 + c + 8 * q < a.N)
            *reinterpret_cast<uint4*>(to + c + 8 * q) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (together_out && lane == 0) {
          tma_store_2d(&a.tm_out, stage, n0 + c, row0);
          bulk_commit();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(smem_in_cta(&tmem_empty[i & 1], 0));
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

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
int linear_map(CUtensorMap* m, const void* base, int64_t third, int64_t rows, int64_t cols, bool mn, int box_rows,
               int box_cols) {
  const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)third};
  const uint64_t strides[2] = {(uint64_t)cols * 2, (uint64_t)cols * rows * 2};
  const uint32_t box[3] = {mn ? 64u : (uint32_t)box_cols, (uint32_t)box_rows, 1};
  return make_tmap_bf16(m, base, 3, dims, strides, box,  // any 16-bit type: bytes are moved
                        mn || box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B
                        : box_cols == 32     ? CU_TENSOR_MAP_SWIZZLE_64B
                                             : CU_TENSOR_MAP_SWIZZLE_32B);
}

// Columns per tile: the width that ends soonest, by waves of tiles times a step's cycles (512 at 256
// columns, where the MMAs bound it; 320 at 128, where the copies do). 4096 rows by 4096 columns
// summed over 4096 in four even waves of 224 instead of 3.4 of 256: 140 -> 135 us. Where M lies with
// its columns contiguous a CTA copies whole boxes of 64 columns, and other widths only copy more
// (dx of 4096 rows by 4096 columns over 11008: 263 us in tiles of 256, 283 in tiles of 224).
static int pick_width(int tiles_m, int N, int pairs, bool mn) {
  int best = 256;
  int64_t best_cost = 0;
  for (int w = 256; w >= (mn ? 128 : 64); w -= mn ? 128 : 32) {
    const int64_t cost = ceil_div64((int64_t)tiles_m * ceil_div(N, w), pairs) * (256 + 3 * w);
    if (best_cost == 0 || cost < best_cost) {
      best = w;
      best_cost = cost;
    }
  }
  return best;
}

template <typename T>
static int launch_pair(const ProductArgs& p, cudaStream_t stream) {
  using C = LinCfg;
  auto kernel = linear_pair_kernel<T>;
  static std::atomic<uint64_t> seen[kMaxDevices];
  static std::atomic<int> resident[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_LORA_ERR_CUDA;
  int st = once_per_context(seen, [&] {
    ML_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)num_sms());
    cfg.blockDim = dim3(kLThreads);
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
  LinArgs a = {};
  const int E = p.rows.E;
  const int64_t pairs = (int64_t)E * p.rows.L;
  // (as many row tiles as there are experts' ragged ends more than full ones, about)
  const int tiles_m = std::min(p.rows.max_tiles, ceil_div(p.rows.S, 256) + (E - 1) / 2);
  a.width = pick_width(tiles_m, p.N, resident[dev].load(), p.mn);
  a.tiles_n = ceil_div(p.N, a.width);
  for (int i = 0; i < (p.rows.slots ? 2 : 1) && st == MOE_LORA_OK; ++i) {
    st = operand_map(&a.tm_in[i], p.in, p.rows.S, p.K, false, i ? kLinearGroup : kLBM);
    if (st == MOE_LORA_OK && p.rows.slots)
      st = operand_map(&a.tm_sorted[i], p.sorted, p.rows.S, p.K, false, i ? kLinearGroup : kLBM);
  }
  if (st == MOE_LORA_OK)
    st = p.mn ? linear_map(&a.tm_m, p.M, E, p.K, p.N, true, 64) : linear_map(&a.tm_m, p.M, E, p.N, p.K, false, a.width / 2);
  const int r16 = ceil_div(p.r, 16) * 16;
  if (st == MOE_LORA_OK)
    st = p.mn ? linear_map(&a.tm_u, p.U, pairs, p.r, p.N, true, r16 <= 32 ? r16 : 64)
              : linear_map(&a.tm_u, p.U, pairs, p.N, p.r, false, a.width / 2, r16 <= 32 ? r16 : 64);
  if (st == MOE_LORA_OK) {
    const uint64_t dims[2] = {(uint64_t)p.N, (uint64_t)p.rows.S};
    const uint64_t strides[1] = {(uint64_t)p.N * 2};
    const uint32_t box[2] = {32, 32};
    st = make_tmap_bf16(&a.tm_out, p.out, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
  }
  if (st == MOE_LORA_OK) st = ffn_error_word(&a.err);
  if (st != MOE_LORA_OK) return st;
  a.stages = C::kMostStages - (r16 <= 32 ? 0 : 1);
  a.rows = p.rows;
  a.z = p.z;
  a.out = p.out;
  a.N = p.N;
  a.K = p.K;
  a.r = p.r;
  a.mn = p.mn;
  a.wait_ns = ffn_wait_ns();
  const int units = std::min(p.rows.max_tiles * a.tiles_n, resident[dev].load());
  return launch_pdl_cluster(kernel, dim3(2 * (unsigned)units), kLThreads, C::kSmemBytes, stream, true, 2, a);
}

int launch_linear_product(const ProductArgs& p, int dtype, cudaStream_t stream) {
  if (p.rows.E == 1 && p.rows.S <= kLinearFewRows) return launch_linear_product_few(p, dtype, stream);
  return dtype == MOE_DTYPE_BF16 ? launch_pair<__nv_bfloat16>(p, stream) : launch_pair<__half>(p, stream);
}

// Whether the product takes copies of rows in sorted order.
static bool linear_copies(int E, int S, int row_flags) {
  return !(row_flags & MOE_ROWS_SORTED) && !(E == 1 && S <= kLinearFewRows);
}

// Arguments that do not depend on pointers, and the align buffer's layout.
static int check_linear(const moe_lora_align_t* al, int dtype, int N, int K, int r, int row_flags, int allowed,
                        AlignLayout* a) {
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_LORA_ERR_INVALID_ARG;
  const int st = check_align(al, a);
  if (st != MOE_LORA_OK) return st;
  if (N < 1 || K < 1 || r < 1 || al->L < 1 || (row_flags & ~allowed)) return MOE_LORA_ERR_INVALID_ARG;
  if (!(row_flags & MOE_ROWS_SORTED) && al->k != 1) return MOE_LORA_ERR_INVALID_ARG;
  if (N % 8 != 0 || K % 8 != 0 || r % 8 != 0 || r > 128 || N > (1 << 20) || K > (1 << 20) || al->adapter_ranks ||
      (int64_t)al->E * al->L > (1 << 20) || (int64_t)N * K >= (1ll << 39))
    return MOE_LORA_ERR_UNSUPPORTED;
  // the tiles of either direction's product, at the narrowest, are counted in 30 bits
  if ((int64_t)a->max_tiles * ceil_div(std::max(N, K), 64) >= (1 << 30)) return MOE_LORA_ERR_UNSUPPORTED;
  return MOE_LORA_OK;
}

static LinearRows linear_rows(const moe_lora_align_t* al, const AlignLayout& a, int row_flags) {
  const AlignView v = align_view(al->buf, a);
  LinearRows r = {};
  r.hdr = v.hdr;
  r.tiles = v.tiles;
  r.blocks = v.blocks;
  r.row_adapter = v.row_adapter;
  r.expert_begin = v.expert_begin;
  r.slots = row_flags & MOE_ROWS_SORTED ? nullptr : v.sorted_slots;
  r.slot_row = v.slot_row;
  r.S = a.S;
  r.E = al->E;
  r.L = al->L;
  r.max_tiles = a.max_tiles;
  r.max_blocks = a.max_blocks;
  return r;
}

// z [S, r]; for the backward v [S, r] and the pairs' first rows [E L]; in the tokens' order the
// rows that the product sums over, in sorted order.
struct LinearWorkspace {
  size_t v, seg, sorted, bytes;
};
static LinearWorkspace linear_workspace(const moe_lora_align_t* al, const AlignLayout& a, int N, int K, int r,
                                        int row_flags, bool backward) {
  const size_t one = round_up((size_t)a.S * r * 4, 256);
  LinearWorkspace w = {};
  w.v = one;
  w.seg = 2 * one;
  w.sorted = backward ? w.seg + round_up((size_t)al->E * al->L * 4, 256) : one;
  w.bytes = w.sorted;
  if (linear_copies(al->E, a.S, row_flags)) w.bytes += round_up((size_t)a.S * (backward ? N : K) * 2, 256);
  w.bytes = std::max<size_t>(w.bytes, 256);
  return w;
}

}  // namespace moe_lora

extern "C" size_t moe_lora_linear_workspace_size(const moe_lora_align_t* al, int N, int K, int r, int row_flags,
                                                 int backward) {
  using namespace moe_lora;
  AlignLayout a;
  if (!al) return 0;
  moe_lora_align_t shape = *al;
  shape.buf = reinterpret_cast<void*>(256);  // sizes only: the buffer may not be there yet
  if (check_linear(&shape, MOE_DTYPE_BF16, N, K, r, row_flags, MOE_ROWS_SORTED | MOE_ROWS_ZERO_DROPPED, &a) != MOE_LORA_OK)
    return 0;
  return linear_workspace(al, a, N, K, r, row_flags, backward != 0).bytes;
}

extern "C" int moe_lora_linear(const void* x, const void* W, const void* A, const void* B, int dtype,
                               const moe_lora_align_t* al, int N, int K, int r, int row_flags, void* y,
                               void* workspace, size_t workspace_bytes, moe_lora_stream_t stream) {
  using namespace moe_lora;
  AlignLayout a;
  int st = check_linear(al, dtype, N, K, r, row_flags, MOE_ROWS_SORTED | MOE_ROWS_ZERO_DROPPED, &a);
  if (st != MOE_LORA_OK) return st;
  if (a.S == 0) return MOE_LORA_OK;
  for (const void* p : {x, W, A, B, (const void*)y, (const void*)workspace})
    if (!p || !aligned16(p)) return MOE_LORA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return MOE_LORA_ERR_INVALID_ARG;
  const LinearWorkspace w = linear_workspace(al, a, N, K, r, row_flags, false);
  if (workspace_bytes < w.bytes) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  float* z = reinterpret_cast<float*>(ws);
  RowsPassArgs pass = {};
  pass.rows = linear_rows(al, a, row_flags);
  pass.part[0] = {x, A, z, K};
  pass.r = r;
  if (row_flags & MOE_ROWS_ZERO_DROPPED) {
    pass.zero_out = y;
    pass.zero_n = N;
  }
  if (linear_copies(al->E, a.S, row_flags)) {
    pass.copy_in = x;
    pass.copy_out = ws + w.sorted;
    pass.copy_n = K;
  }
  if ((st = launch_rows_pass(pass, dtype, s)) != MOE_LORA_OK) return st;
  return launch_linear_product({pass.rows, x, W, B, pass.copy_out, z, y, N, K, r, false}, dtype, s);
}

extern "C" int moe_lora_linear_backward(const void* dy, const void* x, const void* W, const void* A, const void* B,
                                        int dtype, const moe_lora_align_t* al, int N, int K, int r, int row_flags,
                                        void* dx, void* dA, void* dB, void* workspace, size_t workspace_bytes,
                                        moe_lora_stream_t stream) {
  using namespace moe_lora;
  AlignLayout a;
  int st = check_linear(al, dtype, N, K, r, row_flags, MOE_ROWS_SORTED | MOE_ROWS_ZERO_DROPPED, &a);
  if (st != MOE_LORA_OK) return st;
  if (!dx && !dA && !dB) return MOE_LORA_OK;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.S == 0) {  // no row: the adapters' gradients are zero
    if ((dA && !aligned16(dA)) || (dB && !aligned16(dB))) return MOE_LORA_ERR_INVALID_ARG;
    if (dA) ML_CHECK_CUDA(cudaMemsetAsync(dA, 0, (size_t)al->L * al->E * r * K * 2, s));
    if (dB) ML_CHECK_CUDA(cudaMemsetAsync(dB, 0, (size_t)al->L * al->E * r * N * 2, s));
    return MOE_LORA_OK;
  }
  for (const void* p : {dy, x, W, A, B, (const void*)workspace})
    if (!p || !aligned16(p)) return MOE_LORA_ERR_INVALID_ARG;
  for (const void* p : {dx, dA, dB})
    if (!aligned16(p)) return MOE_LORA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return MOE_LORA_ERR_INVALID_ARG;
  const LinearWorkspace w = linear_workspace(al, a, N, K, r, row_flags, true);
  if (workspace_bytes < w.bytes) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  char* ws = static_cast<char*>(workspace);
  float *z = reinterpret_cast<float*>(ws), *v = reinterpret_cast<float*>(ws + w.v);
  RowsPassArgs pass = {};
  pass.rows = linear_rows(al, a, row_flags);
  if (dB) pass.part[0] = {x, A, z, K};
  if (dx || dA) pass.part[1] = {dy, B, v, N};
  pass.r = r;
  if (dx && (row_flags & MOE_ROWS_ZERO_DROPPED)) {
    pass.zero_out = dx;
    pass.zero_n = K;
  }
  if (dA || dB) pass.seg_begin = reinterpret_cast<int*>(ws + w.seg);
  if (dx && linear_copies(al->E, a.S, row_flags)) {
    pass.copy_in = dy;
    pass.copy_out = ws + w.sorted;
    pass.copy_n = N;
  }
  if ((st = launch_rows_pass(pass, dtype, s)) != MOE_LORA_OK) return st;
  // The adapters' gradients before dx. Both orders timed in turn, four times each, in a graph: 4096 rows of
  // 11008/4096 327 against 331 us, 128 rows 15.5 against 15.7, 1021 rows no different (43.3 against 43.1).
  if (dA || dB) {
    st = launch_adapter_grads({pass.rows, x, dy, z, v, pass.seg_begin, dA, dB, K, N, r}, dtype, s);
    if (st != MOE_LORA_OK) return st;
  }
  return dx ? launch_linear_product({pass.rows, dy, W, A, pass.copy_out, v, dx, K, N, r, true}, dtype, s) : MOE_LORA_OK;
}
