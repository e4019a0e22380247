// The projection with adapters for up to kLinearFewRows rows of one expert (a decode batch, or
// its gradient), on tcgen05.
//
// The weights' stream bounds it. All rows are one 128-row tile, on the MMA's M side so that an
// adapter's steps can leave the other rows' TMEM lanes alone (lora_linear.cu); only the rows
// there are get copied, into as much shared memory as they take (the MMA reads what lies
// behind them for the lanes of rows that are not there, which are never stored), and the ring
// holds mostly weights.
// * A CTA takes as many columns, up to 128, as spread the weights evenly over the SMs in one
//   wave: a second wave of CTAs starts its stream anew (some 10 us). The sum is shared out over the
//   CTAs of a cluster where the column blocks alone would leave SMs idle, the adapters' steps in turn;
//   the CTAs add up through distributed shared memory in rank order, so no result depends on timing.
// * Weights stream while the pass before still makes z (see lora_linear.cu on what may be read
//   then); z tiles have a place of their own and are written once. Two CTAs per SM up to 64 rows.
// 64 rows of 8 adapters through 28672/4096: 46 us with the pass before (5.2 TB/s); one row through
// 4096/4096 12 us.
#include <algorithm>

#include "lora_linear.h"

namespace moe_lora {

constexpr int kLFThreads = 256;
constexpr int kLFCols = 128;  // output columns per cluster, at most

template <int ROWS>
struct LinFewCfg {
  static constexpr int kInBytes = ROWS * 64 * 2;
  static constexpr int kMostStages = 8;
  static constexpr int kBarBytes = 256 + 2 * 128 * 4;  // barriers, and the adapters for two roles
  static_assert((2 * kMostStages + 2) * 8 + 12 <= 256, "barrier area");
  // z tiles, ring, barriers; two CTAs on an SM up to 64 rows
  static constexpr int kRoom = (ROWS == 128 ? 226 * 1024 : 110 * 1024) - kBarBytes - 1024;
};

struct LinFewArgs {
  CUtensorMap tm_in, tm_m, tm_u;
  LinearRows rows;
  const float* z;
  void* out;
  int N, K, r;
  int cols;      // output columns per cluster: a multiple of 16, of 64 where mn
  int ks, kper;  // CTAs per cluster, 64-wide base steps of each
  int stages, stage_bytes;
  int mn;
  unsigned int* err;
  unsigned long long wait_ns;
};

template <typename T, int ROWS>
__global__ void __launch_bounds__(kLFThreads, ROWS == 128 ? 1 : 2) linear_few_kernel(const __grid_constant__ LinFewArgs a) {
  using C = LinFewCfg<ROWS>;
  constexpr int Q = ROWS / 32;
  const int stages = a.stages, stage_bytes = a.stage_bytes;
  const RankSteps rs(a.r);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem + rs.steps * rs.tiles * C::kInBytes;  // behind the z tiles
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + stages * stage_bytes);
  uint64_t* empty = full + C::kMostStages;
  uint64_t* z_full = empty + C::kMostStages;
  uint64_t* done = z_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_issued = reinterpret_cast<int*>(tmem_slot + 2);
  int* lists = reinterpret_cast<int*>(full) + 64;
  float* sums = reinterpret_cast<float*>(smem);  // [ROWS][128], after the ring is done

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.ks > 1 ? (int)cluster_ctarank() : 0;
  const int n0 = blockIdx.x / a.ks * a.cols;
  const int k0 = rank * a.kper;
  const int nk = min(a.kper, (a.K + 63) / 64 - k0);
  constexpr int kZWarps = ROWS / 32, kZWarp0 = 8 - kZWarps;

  // (no copy takes as long as one try: a limit of 0 tests)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return a.wait_ns ? mbar_wait_bounded(bar, parity, a.wait_ns) : mbar_test(bar, parity);
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(z_full, kZWarps);
    mbar_init(done, 1);
    *s_abort = 0;
    *s_issued = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&a.tm_m);
    tma_prefetch_desc(&a.tm_in);
    tma_prefetch_desc(&a.tm_u);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kLFCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_valid = __ldcg(a.rows.hdr + HDR_NVALID);
  // U of up to four adapters shares a stage. The stages go round the cluster's ranks, counted over
  // the adapters in order; each role lists the adapters for itself. fn(adapters, how many, step) ->
  // false to stop.
  const int together = rs.together(), u_ranks = 64 / together, u_bytes = a.cols * u_ranks * 2;
  auto list_adapters = [&](int* list) {
    Runs<Q> runs;
    runs.load(a.rows.row_adapter, 0, n_valid);
    runs.find();
    return runs.write(list);
  };
  auto adapter_stages = [&](const int* list, int n_runs, auto&& fn) {
    const int groups = (n_runs + together - 1) / together;
    for (int k = rank; k < groups * rs.steps; k += a.ks) {
      const int st = k / groups, first = (k - st * groups) * together;
      if (!fn(list + first, min(together, n_runs - first), st)) return;
    }
  };

  if (warp == 0) {
    // producer and, below, MMA issuer: warp-uniform loops, one elected lane issues
    const bool elected = elect_one();
    const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
    bool ok = true;
    int s = 0, i = 0;
    uint32_t ph = 1;
    auto slot_free = [&]() {
      ok = i < stages || __all_sync(0xffffffffu, wait(&empty[s], ph) && !*s_abort);
      return ok;
    };
    auto advance = [&]() {
      __syncwarp();
      ++i;
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    };
    auto copy_cols = [&](const CUtensorMap* m, uint8_t* sw, int k, int third, uint64_t pol, int block) {
      if (a.mn) {
        tma_load_3d(sw, m, &full[s], n0, k, third, pol);
        if (a.cols > 64) tma_load_3d(sw + block, m, &full[s], n0 + 64, k, third, pol);
      } else {
        tma_load_3d(sw, m, &full[s], k, n0, third, pol);
      }
    };
    while (i < nk && slot_free()) {
      if (elected) {
        mbar_arrive_expect_tx(&full[s], (uint32_t)((a.cols + a.rows.S) * 128));
        copy_cols(&a.tm_m, ring + s * stage_bytes + C::kInBytes, (k0 + i) * 64, 0, pol_w, 8192);
        tma_load_2d(ring + s * stage_bytes, &a.tm_in, &full[s], (k0 + i) * 64, 0, pol_x);
      }
      advance();
    }
    if (ok)
      adapter_stages(lists, list_adapters(lists), [&](const int* ls, int n, int st) {
        if (!slot_free()) return false;
        if (elected) {
          mbar_arrive_expect_tx(&full[s], (uint32_t)(n * u_bytes));
          for (int j = 0; j < n; ++j)
            copy_cols(&a.tm_u, ring + s * stage_bytes + C::kInBytes + j * u_bytes, 64 * st, ls[j], pol_w,
                      u_ranks * 128);
        }
        advance();
        return true;
      });
    if (lane == 0) {
      *s_issued = i;
      if (!ok) *s_abort = 1;
    }
  } else if (warp == 1) {
    const bool elected = elect_one();
    const uint32_t idesc = (1u << 4) | (MmaType<T>::kFmt << 7) | (MmaType<T>::kFmt << 10) | ((uint32_t)a.mn << 16) |
                           ((uint32_t)(a.cols >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t s0 = smem_u32(ring);
    const uint64_t da0 = smem_desc_sw128(s0), dz0 = smem_desc_sw128(smem_u32(smem));
    const uint64_t db0 = a.mn ? smem_desc_mn(s0 + C::kInBytes) : smem_desc_sw128(s0 + C::kInBytes);
    const uint32_t bstep = a.mn ? 2048 >> 4 : 32 >> 4;
    bool ok = true;
    int s = 0;
    uint32_t ph = 0;
    auto advance = [&]() {
      __syncwarp();
      if (++s == stages) {
        s = 0;
        ph ^= 1;
      }
    };
    for (int i = 0; i < nk; ++i) {
      ok = __all_sync(0xffffffffu, wait(&full[s], ph) && !*s_abort);
      if (!ok) break;
      tc_fence_after();
      if (elected) {
        const uint64_t off = (uint64_t)(s * (stage_bytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_bf16(tmem, da0 + off + kk * 2, db0 + off + kk * bstep, idesc, (i | kk) != 0);
        tc_commit(&empty[s]);
      }
      advance();
    }
    if (ok) {
      // the adapter of each row of the tile (which the operands' order may mix)
      int mine[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        int row = 32 * q + lane;
        if (a.rows.slots) row = row < a.rows.S ? __ldcg(a.rows.slot_row + row) : -1;
        mine[q] = row >= 0 && row < n_valid ? __ldcg(a.rows.row_adapter + row) : -1;
      }
      // U as it lies in its part of a stage (see linear_pair_kernel)
      const uint32_t u0 = s0 + C::kInBytes;
      const uint64_t du0 = a.mn            ? smem_desc_mn(u0, u_ranks * 128)
                           : u_ranks == 64 ? smem_desc_sw128(u0)
                           : u_ranks == 32 ? smem_desc_swz(u0, 4, 512)
                                           : smem_desc_swz(u0, 6, 256);
      adapter_stages(lists + 128, list_adapters(lists + 128), [&](const int* ls, int count, int st) {
        ok = __all_sync(0xffffffffu, wait(&full[s], ph) && wait(z_full, 0) && !*s_abort);
        if (!ok) return false;
        tc_fence_after();
        const uint64_t dz = dz0 + (uint64_t)(st * rs.tiles * (C::kInBytes >> 4));
        uint64_t du = du0 + (uint64_t)(s * (stage_bytes >> 4));
        const int nu = rs.u_mmas(st);
        const uint32_t low = rs.low(st, C::kInBytes);
        for (int j = 0; j < count; ++j) {
          uint32_t off_rows[4] = {~0u, ~0u, ~0u, ~0u};
#pragma unroll
          for (int q = 0; q < Q; ++q) off_rows[q] = __ballot_sync(0xffffffffu, mine[q] != ls[j]);
          if (elected)
            for (int kk = 0; kk < nu; ++kk) {
              tc_mma_lanes(tmem, dz + kk * 2, du + kk * bstep, idesc, off_rows);
              tc_mma_lanes(tmem, dz + low + kk * 2, du + kk * bstep, idesc, off_rows);
            }
          __syncwarp();
          du += (uint32_t)u_bytes >> 4;
        }
        if (elected) tc_commit(&empty[s]);
        advance();
        return true;
      });
    }
    if (!ok && lane == 0) *s_abort = 1;
    if (elected) tc_commit(done);  // also after a give-up: arrives once every MMA is over
    __syncwarp();
  } else if (warp >= kZWarp0) {
    // z writers: a thread per row of the tile
    const int i0 = (int)threadIdx.x - 32 * kZWarp0;
    int row = i0;
    if (a.rows.slots) row = i0 < a.rows.S ? __ldcg(a.rows.slot_row + i0) : -1;
    if (row >= n_valid) row = -1;
    const bool mine = row >= 0 && __ldcg(a.rows.row_adapter + row) >= 0;
    const float* zrow = a.z + (int64_t)max(row, 0) * a.r;
    pdl_wait();  // z is the launch before's
    if (i0 == 0) pdl_trigger();
    for (int st = 0; st < rs.steps; ++st) write_z_row<T>(smem + st * rs.tiles * C::kInBytes, C::kInBytes, i0, zrow, mine, a.r, rs, st);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(z_full);
  }
  // The sums of this CTA's share over the ring: every copy has landed and been consumed once
  // the last MMA is over (or, after a give-up, is waited for here).
  __syncwarp();
  if (!__all_sync(0xffffffffu, mbar_wait_bounded(done, 0, a.wait_ns + kWaitLimitNs)) && lane == 0) *s_abort = 1;
  __syncthreads();
  tc_fence_after();
  if (*s_abort) {
    if (threadIdx.x == 0) {
      for (int g = *s_issued - 1; g >= 0 && g >= *s_issued - stages; --g)
        mbar_wait_bounded(&full[g % stages], (g / stages) & 1);
      atomicOr(a.err, MOE_LORA_DEVERR_TIMEOUT);
    }
    __syncthreads();
  } else {
    // TMEM lanes [32 (w % 4), + 32), as many rows; the two warps of a quarter take half of the
    // columns each. A row's columns are rotated by its number, so that the lanes' stores meet
    // different banks.
    const int quad = warp & 3, half = warp >> 2;
    if (quad < Q && quad * 32 < a.rows.S) {
      const int row = quad * 32 + lane;
#pragma unroll 1
      for (int c = half * 64; c < min(half * 64 + 64, a.cols); c += 16) {
        uint32_t v[16];
        tmem_ld_x16(tmem + c + ((uint32_t)(quad * 32) << 16), v);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(sums + row * kLFCols + (((c / 4 + q) + row) & 31) * 4) =
              make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      }
    }
    tc_fence_before();
  }
  if (a.ks > 1) cluster_sync();
  else __syncthreads();
  // Every CTA finishes a share of the rows; a thread takes four columns at a time.
  const int rows = a.rows.S, per = (rows + a.ks - 1) / a.ks, t0 = rank * per, t1 = min(rows, t0 + per);
  const int quads = a.cols / 4;
#pragma unroll 1
  for (int i = threadIdx.x; i < (t1 - t0) * quads; i += kLFThreads) {
    const int row = t0 + i / quads, c4 = i % quads, n = n0 + c4 * 4;
    if (n >= a.N) continue;
    // a dropped slot's row is left as it is
    if (a.rows.slots ? __ldcg(a.rows.slot_row + row) < 0 : row >= n_valid) continue;
    float v[4] = {};
    const float* at = sums + row * kLFCols + ((c4 + row) & 31) * 4;
    for (int rk = 0; rk < a.ks; ++rk) {
      float4 p;
      if (a.ks > 1) {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w)
                     : "r"(smem_in_cta(at, (uint32_t)rk)));
      } else {
        p = *reinterpret_cast<const float4*>(at);
      }
      v[0] += p.x;
      v[1] += p.y;
      v[2] += p.z;
      v[3] += p.w;
    }
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (int64_t)row * a.N + n) =
        make_uint2(Elem<T>::r2(v[0], v[1]), Elem<T>::r2(v[2], v[3]));
  }
  if (a.ks > 1) cluster_sync();  // the sums are read before any CTA leaves
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kLFCols);
  }
}

template <typename T, int ROWS>
static int launch_few(LinFewArgs& a, const ProductArgs& product, cudaStream_t stream) {
  using C = LinFewCfg<ROWS>;
  auto kernel = linear_few_kernel<T, ROWS>;
  static std::atomic<uint64_t> seen[kMaxDevices];
  static std::atomic<int> resident[kMaxDevices][9];  // CTAs in clusters of that many at once
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return MOE_LORA_ERR_CUDA;
  int st = once_per_context(seen, [&] {
    ML_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kRoom + C::kBarBytes + 1024));
    for (int ks = 1; ks <= 8; ++ks) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * (unsigned)num_sms() / ks * ks);
      cfg.blockDim = dim3(kLFThreads);
      cfg.dynamicSmemBytes = C::kRoom + C::kBarBytes + 1024;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = ks;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      ML_CHECK_CUDA(cudaOccupancyMaxActiveClusters(&clusters, kernel, &cfg));
      // (the query counts one CTA an SM where tensor memory is allocated; two run. A tenth is left for
      // what keeps clusters from filling every place)
      resident[dev][ks].store(std::max(1, clusters) * ks * (ROWS == 128 ? 10 : 18) / 10);
    }
    return MOE_LORA_OK;
  });
  if (st != MOE_LORA_OK) return st;
  const int r16 = ceil_div(a.r, 16) * 16;
  const int z_bytes = (r16 <= 32 ? 1 : 2 * ceil_div(r16, 64)) * C::kInBytes;  // steps and tiles as RankSteps counts
  // Columns per CTA and CTAs per cluster (up to 8, four base steps each at least), so that the
  // SM with the most to stream has least: what its CTAs copy -- a third more where an SM has one
  // CTA, whose start and end nothing overlaps -- and for each further wave as long as some 400
  // KB take.
  // (32-bit divisions: the choice is made on every call)
  const int steps = ceil_div(a.K, 64), sms = num_sms();
  float best = 0.f;
  for (int ks = 1; ks <= 8 && (ks == 1 || ks * 4 <= steps); ++ks) {
    const int kper = ceil_div(steps, ks), n = ceil_div(steps, kper), places = resident[dev][n].load(std::memory_order_relaxed);
    for (int cols = kLFCols; cols >= (a.mn ? 64 : 48); cols -= a.mn ? 64 : 16) {
      const int ctas = ceil_div(a.N, cols) * n, per_sm = ceil_div(ctas, sms);
      const float bytes = (float)per_sm * kper * (cols + a.rows.S / 4) * 128;
      const float cost = (per_sm == 1 ? bytes * 4 / 3 : bytes) + (ceil_div(ctas, places) - 1) * 400000.f;
      if (best == 0.f || cost < best) {
        best = cost;
        a.cols = cols;
        a.kper = kper;
        a.ks = n;
      }
    }
  }
  // A stage: the rows there are and the weights' columns. An operand's 128 rows are read all the
  // same, wherever those that are there end: into its stage's weights, or from a z tile into the
  // ring behind it.
  a.stage_bytes = std::max(C::kInBytes + a.cols * 128, 128 * 128);
  a.stages = std::min(C::kMostStages, (C::kRoom - z_bytes) / a.stage_bytes);
  // the boxes of M and U have as many columns
  const ProductArgs& p = product;
  st = p.mn ? linear_map(&a.tm_m, p.M, 1, p.K, p.N, true, 64) : linear_map(&a.tm_m, p.M, 1, p.N, p.K, false, a.cols);
  if (st == MOE_LORA_OK)
    st = p.mn ? linear_map(&a.tm_u, p.U, p.rows.L, p.r, p.N, true, r16 <= 32 ? r16 : 64)
              : linear_map(&a.tm_u, p.U, p.rows.L, p.N, p.r, false, a.cols, r16 <= 32 ? r16 : 64);
  if (st != MOE_LORA_OK) return st;
  // (the sums, ROWS x 128 fp32, take the place of z tiles and ring: at least three stages)
  const int smem = z_bytes + a.stages * a.stage_bytes + C::kBarBytes + 1024;
  return launch_pdl_cluster(kernel, dim3((unsigned)(ceil_div(a.N, a.cols) * a.ks)), kLFThreads, smem, stream, true, a.ks, a);
}
template <typename T>
static int launch_few_rows(LinFewArgs& a, const ProductArgs& p, cudaStream_t s) {
  return a.rows.S <= 32   ? launch_few<T, 32>(a, p, s)
         : a.rows.S <= 64 ? launch_few<T, 64>(a, p, s)
                          : launch_few<T, 128>(a, p, s);
}

int launch_linear_product_few(const ProductArgs& p, int dtype, cudaStream_t stream) {
  LinFewArgs a = {};
  int st = operand_map(&a.tm_in, p.in, p.rows.S, p.K, false, p.rows.S);
  if (st == MOE_LORA_OK) st = ffn_error_word(&a.err);
  if (st != MOE_LORA_OK) return st;
  a.rows = p.rows;
  a.z = p.z;
  a.out = p.out;
  a.N = p.N;
  a.K = p.K;
  a.r = p.r;
  a.mn = p.mn;
  a.wait_ns = ffn_wait_ns();
  return dtype == MOE_DTYPE_BF16 ? launch_few_rows<__nv_bfloat16>(a, p, stream) : launch_few_rows<__half>(a, p, stream);
}

}  // namespace moe_lora
