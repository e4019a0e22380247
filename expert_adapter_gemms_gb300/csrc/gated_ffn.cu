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
#include "internal.h"

namespace moe_lora {

enum { kEpiStore = 0, kEpiGated = 1, kEpiGrad = 2 };

constexpr int kGBM = 128;         // rows per CTA (256 per pair)
constexpr int kGBK = 64;          // K per stage: 128 bytes
constexpr int kGThreads = 192;    // TMA warp, MMA warp, four epilogue warps
constexpr int kGGroup = 8;        // row tiles per raster group

template <int BN>
struct PairCfg {
  static constexpr int kABytes = kGBM * kGBK * 2;
  static constexpr int kBRows = BN / 2;  // rows (columns of the output) per CTA
  static constexpr int kBBytes = kBRows * kGBK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = BN == 256 ? 6 : BN == 128 ? 8 : 10;
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kSmemBytes = kBarOff + 256 + 1024;
  static constexpr uint32_t kTmemCols = 2 * BN;
  static_assert((2 * kStages + 5) * 8 + 16 <= 256, "barrier area");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// One product out[m, n] = sum_k A(m, k) B(n, k).
struct PairProblem {
  int M, N, K;         // N: columns of the output (features, for the gated forms)
  int tiles_m, tiles;  // 256-row tiles; all tiles
  int a_mn, b_mn;      // the operand lies with m (n) contiguous, not k
  int up_off;          // gated: rows of B between gate and up
  void* out;
  int64_t ldo;
};

struct PairArgs {
  CUtensorMap tm[2][2];  // [problem][A, B]
  PairProblem p[2];
  int nproblems;
  int light, extra;      // see unit_tile
  const void* dh;        // [M, N], kEpiGrad
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

// Row-grouped raster: kGGroup row tiles by every column tile, so that the pairs at work share
// rows of A and of B in L2.
__device__ __forceinline__ void tile_place(const PairProblem& p, int tile, int& tm, int& tn) {
  const int tiles_n = p.tiles / p.tiles_m;
  const int per = kGGroup * tiles_n;
  const int grp = tile / per, in = tile - grp * per;
  const int rows = min(kGGroup, p.tiles_m - grp * kGGroup);
  tm = grp * kGGroup + in % rows;
  tn = in / rows;
}

// Shared-memory matrix descriptor of an operand with m (n) contiguous: 64 x 64 boxes (64
// summed rows of 128 bytes, 128-byte swizzle), one after the other along m. Eight summed rows
// are 1024 bytes (stride offset), the next 64 of m one box (leading offset).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((uint32_t)(64 * 128) >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

template <typename T> struct MmaType;
template <> struct MmaType<__nv_bfloat16> { static constexpr uint32_t kFmt = 1; };
template <> struct MmaType<__half> { static constexpr uint32_t kFmt = 0; };

template <typename T, int kEpi, int kAct, int BN>
__global__ void __launch_bounds__(kGThreads, 1) pair_gemm_kernel(const __grid_constant__ PairArgs a) {
  using C = PairCfg<BN>;
  constexpr int STAGES = C::kStages;
  constexpr bool kGated = kEpi != kEpiStore;
  constexpr int kOutCols = kGated ? BN / 2 : BN;  // output columns per tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + STAGES;
  uint64_t* tmem_full = empty + STAGES;
  uint64_t* tmem_empty = tmem_full + 2;
  uint64_t* mma_done = tmem_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool leader = crank == 0;
  const int unit = blockIdx.x / 2, units = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);   // the leader's arming; the copies of both CTAs complete on it
      mbar_init(&empty[s], 1);  // the commit, to both CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tmem_full[i], 1);
      mbar_init(&tmem_empty[i], 8);  // the epilogue warps of both CTAs, on the leader's
    }
    mbar_init(mma_done, 1);
    *s_abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    for (int i = 0; i < a.nproblems; ++i) {
      tma_prefetch_desc(&a.tm[i][0]);
      tma_prefetch_desc(&a.tm[i][1]);
    }
  }
  cluster_sync();
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, C::kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_wait();  // every input may come from the launch before
  if (threadIdx.x == 0) pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
    int g = 0, prob, tile;
    bool ok = true;
    for (int i = 0; ok && unit_tile(a, unit, units, i, prob, tile); ++i) {
      const PairProblem& p = a.p[prob];
      const CUtensorMap *ta = &a.tm[prob][0], *tb = &a.tm[prob][1];
      int tm, tn;
      tile_place(p, tile, tm, tn);
      const int m0 = tm * 256 + (int)crank * kGBM;
      const int n0 = kGated ? tn * kOutCols + (int)crank * p.up_off : tn * BN + (int)crank * C::kBRows;
      const int nk = (p.K + kGBK - 1) / kGBK;
      const bool a_mn = p.a_mn != 0, b_mn = !kGated && p.b_mn != 0;
      for (int kb = 0; ok && kb < nk; ++kb, ++g) {
        const int s = g % STAGES;
        if (g >= STAGES)
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(&empty[s], ((g / STAGES) & 1) ^ 1, a.wait_ns) && !*s_abort);
        if (!ok) break;
        if (elected) {
          uint8_t* sa = smem + s * C::kStageBytes;
          uint8_t* sb = sa + C::kABytes;
          const uint32_t bar = full0 + s * 8;
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * C::kStageBytes);
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
      int g = 0, prob, tile;
      bool ok = true;
      for (int i = 0; ok && unit_tile(a, unit, units, i, prob, tile); ++i) {
        const PairProblem& p = a.p[prob];
        const int nk = (p.K + kGBK - 1) / kGBK;
        const uint32_t acc = tmem + (uint32_t)((i & 1) * BN);
        const uint32_t idesc = (1u << 4) | (MmaType<T>::kFmt << 7) | (MmaType<T>::kFmt << 10) |
                               ((uint32_t)p.a_mn << 15) | ((uint32_t)p.b_mn << 16) |
                               ((uint32_t)(BN >> 3) << 17) | ((256u >> 4) << 24);
        const uint32_t s0 = smem_u32(smem);
        const uint64_t da0 = p.a_mn ? smem_desc_mn(s0) : smem_desc_sw128(s0);
        const uint64_t db0 = p.b_mn ? smem_desc_mn(s0 + C::kABytes) : smem_desc_sw128(s0 + C::kABytes);
        // a K-major step of 16 is 32 bytes along the swizzled row; MN-major, 16 rows
        const uint32_t astep = p.a_mn ? 2048 >> 4 : 32 >> 4, bstep = p.b_mn ? 2048 >> 4 : 32 >> 4;
        if (i >= 2) ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tmem_empty[i & 1], ((i >> 1) - 1) & 1, a.wait_ns));
        tc_fence_after();
        for (int kb = 0; ok && kb < nk; ++kb, ++g) {
          const int s = g % STAGES;
          ok = __all_sync(0xffffffffu, mbar_wait_cluster(&full[s], (g / STAGES) & 1, a.wait_ns) && !*s_abort);
          if (!ok) break;
          tc_fence_after();
          if (elected) {
            const uint64_t off = (uint64_t)(s * (C::kStageBytes >> 4));
#pragma unroll
            for (int kk = 0; kk < kGBK / 16; ++kk)
              tc_mma_bf16_pair(acc, da0 + off + kk * astep, db0 + off + kk * bstep, idesc, (kb | kk) != 0);
            tc_commit_pair_mc(&empty[s]);
          }
          __syncwarp();
        }
        if (ok && elected) tc_commit_pair_mc(&tmem_full[i & 1]);
        __syncwarp();
      }
      if (!ok && lane == 0) set_abort();
    }
  } else {
    const int quad = warp & 3;
    int prob, tile;
    for (int i = 0; unit_tile(a, unit, units, i, prob, tile); ++i) {
      const PairProblem& p = a.p[prob];
      int tm, tn;
      tile_place(p, tile, tm, tn);
      bool ok = __all_sync(0xffffffffu, mbar_wait_cluster(&tmem_full[i & 1], (i >> 1) & 1, a.wait_ns) ? 1 : 0);
      if (!ok && lane == 0) set_abort();
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + (uint32_t)((i & 1) * BN) + ((uint32_t)(quad * 32) << 16);
      const int64_t m = (int64_t)tm * 256 + crank * kGBM + quad * 32 + lane;
      const int n0 = tn * kOutCols;
      T* orow = static_cast<T*>(p.out) + m * p.ldo;
      const bool row = m < p.M;
      // the output's columns in steps of 16 (N is a multiple of 8: whole 16-byte stores)
      for (int c = 0; c < kOutCols; c += 16) {
        const int n = n0 + c;
        uint32_t v[16], w[16];
        __syncwarp();
        tmem_ld_x16(acc + c, v);
        if (kGated) tmem_ld_x16(acc + BN / 2 + c, w);
        uint4 d[2] = {};
        if (kEpi == kEpiGrad && row) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.dh) + m * p.N + n);
          if (n < p.N) d[0] = __ldcg(src);
          if (n + 8 < p.N) d[1] = __ldcg(src + 1);
        }
        tmem_ld_wait();
        if (!row || n >= p.N) continue;
        uint32_t o[8], o2[8];
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
              const uint32_t dw = reinterpret_cast<const uint32_t*>(d)[q];
              const float2 e = Elem<T>::f2(dw);
              o[q] = Elem<T>::r2(e.x * u0 * d0, e.y * u1 * d1);
              o2[q] = Elem<T>::r2(e.x * a0, e.y * a1);
            }
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(orow + n);
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        if (n + 8 < p.N) dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        if (kEpi == kEpiGrad) {  // du beside dg: [dg | du] rows of 2N
          uint4* dst2 = reinterpret_cast<uint4*>(orow + p.N + n);
          dst2[0] = make_uint4(o2[0], o2[1], o2[2], o2[3]);
          if (n + 8 < p.N) dst2[1] = make_uint4(o2[4], o2[5], o2[6], o2[7]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(smem_in_cta(&tmem_empty[i & 1], 0));
    }
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
// The device address of the error word, per context.
static int ffn_error_word(unsigned int** out) {
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

// An operand: rows [rows, cols] with `cols` contiguous. Summed over cols (K-major) a box is
// 64 columns by `box_rows` rows; summed over rows (MN-major), 64 by 64.
static int operand_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, bool mn, int box_rows) {
  const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)cols * 2};
  const uint32_t box[2] = {64, (uint32_t)(mn ? 64 : box_rows)};
  return make_tmap_bf16(m, base, 2, dims, strides, box);  // any 16-bit type: bytes are moved
}

struct ProblemDesc {
  const void *A, *B;
  int M, N, K;
  bool a_mn, b_mn;
  void* out;
  int64_t ldo;
};

template <typename T, int kEpi, int kAct, int BN>
static int launch_pair(const ProblemDesc* d, int n, const void* dh, cudaStream_t stream) {
  using C = PairCfg<BN>;
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
    p.out = d[i].out;
    p.ldo = d[i].ldo;
    p.up_off = kGated ? p.N : 0;
    p.tiles_m = ceil_div(p.M, 256);
    const int64_t tiles = (int64_t)p.tiles_m * ceil_div(p.N, kGated ? BN / 2 : BN);
    if (tiles > (1 << 28)) return MOE_LORA_ERR_UNSUPPORTED;
    p.tiles = (int)tiles;
    all += tiles;
    st = operand_map(&a.tm[i][0], d[i].A, p.a_mn ? p.K : p.M, p.a_mn ? p.M : p.K, p.a_mn, kGBM);
    if (st != MOE_LORA_OK) return st;
    const int64_t bn_rows = kGated ? 2 * (int64_t)p.N : p.N;
    st = operand_map(&a.tm[i][1], d[i].B, p.b_mn ? p.K : bn_rows, p.b_mn ? bn_rows : p.K, p.b_mn, C::kBRows);
    if (st != MOE_LORA_OK) return st;
  }
  a.nproblems = n;
  a.dh = dh;
  a.wait_ns = kWaitLimitNs;
  if ((st = ffn_error_word(&a.err)) != MOE_LORA_OK) return st;
  const int units = (int)std::min<int64_t>(all, resident[dev].load());
  if (n == 2 && a.p[0].tiles % units) {
    a.light = units - a.p[0].tiles % units;
    a.extra = (a.p[0].K + a.p[1].K / 2) / a.p[1].K;
    a.extra = std::min(a.extra, a.p[1].tiles / a.light);
  }
  return launch_pdl_cluster(kernel, dim3(2 * (unsigned)units), kGThreads, C::kSmemBytes, stream, true, 2, a);
}

// Columns per tile: the most of 256 whose tiles still make a wave of the pairs, else fewer,
// so that more pairs share the work.
template <typename T, int kEpi, int kAct>
static int launch_products(const ProblemDesc* d, int n, const void* dh, cudaStream_t stream) {
  constexpr bool kGated = kEpi != kEpiStore;
  auto tiles = [&](int bn) {
    int64_t t = 0;
    for (int i = 0; i < n; ++i)
      t += (int64_t)ceil_div(d[i].M, 256) * ceil_div(d[i].N, kGated ? bn / 2 : bn);
    return t;
  };
  const int pairs = num_sms() / 2;
  if (tiles(256) >= pairs) return launch_pair<T, kEpi, kAct, 256>(d, n, dh, stream);
  return launch_pair<T, kEpi, kAct, 128>(d, n, dh, stream);
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
                        const void* dh, void* out, int64_t ldo, cudaStream_t stream) {
  const ProblemDesc d = {x, W1, T, I, H, false, false, out, ldo};
  if (dtype == MOE_DTYPE_BF16)
    return act == MOE_ACT_SILU ? launch_products<__nv_bfloat16, kEpi, MOE_ACT_SILU>(&d, 1, dh, stream)
                               : launch_products<__nv_bfloat16, kEpi, MOE_ACT_GELU>(&d, 1, dh, stream);
  return act == MOE_ACT_SILU ? launch_products<__half, kEpi, MOE_ACT_SILU>(&d, 1, dh, stream)
                             : launch_products<__half, kEpi, MOE_ACT_GELU>(&d, 1, dh, stream);
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

extern "C" int moe_gated_ffn(const void* x, const void* W1, int dtype, int act, int T, int H, int I,
                             void* h, moe_lora_stream_t stream) {
  using namespace moe_lora;
  int st = check_gated(dtype, act, T, H, I);
  if (st != MOE_LORA_OK) return st;
  if (T == 0) return MOE_LORA_OK;
  if (!x || !W1 || !h || !aligned16(x) || !aligned16(W1) || !aligned16(h)) return MOE_LORA_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  return launch_gated<kEpiGated>(dtype, act, x, W1, T, H, I, nullptr, h, I,
                                 reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t moe_gated_ffn_backward_workspace_size(int T, int H, int I) {
  using namespace moe_lora;
  if (check_gated(MOE_DTYPE_BF16, MOE_ACT_SILU, T, H, I) != MOE_LORA_OK) return 0;
  return round_up((size_t)T * 2 * I * 2 + 256, 256);
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
  if ((st = launch_gated<kEpiGrad>(dtype, act, x, W1, T, H, I, dh, workspace, 2 * (int64_t)I, s)) != MOE_LORA_OK)
    return st;
  ProblemDesc d[2];
  int n = 0;
  if (dx) d[n++] = {workspace, W1, T, H, 2 * I, false, true, dx, H};
  if (dW1) d[n++] = {workspace, x, 2 * I, H, T, true, true, dW1, H};
  if (n == 2 && d[1].K > d[0].K) std::swap(d[0], d[1]);  // the longer sums first
  return dtype == MOE_DTYPE_BF16 ? launch_products<__nv_bfloat16, kEpiStore, MOE_ACT_NONE>(d, n, nullptr, s)
                                 : launch_products<__half, kEpiStore, MOE_ACT_NONE>(d, n, nullptr, s);
}
