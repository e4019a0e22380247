// Products of up to kFewTokens rows with large weights, on tcgen05: the gated block (and its
// backward's dg and du), and dx = dy W1.
//
// The weights' stream bounds them: 4 I H bytes against 4 T I H operations. The weights take the
// MMA's M side (128 rows per CTA) and the tokens its N side, so no tensor-core row and no shared
// memory is spent on padding tokens to 128, and the token box holds exactly the T rows there
// are. One token of 4096/14336: 36 us (6.5 TB/s), 64: 38 us. (A kernel for single tokens that
// took the weights through registers into mma.sync was faster by 0.2 to 0.6 us at a few MB of
// weights and slower from 30 MB on, 9.1 against 8.1 us at 2880/2880.)
// * Gated: 64 gate rows and the 64 up rows of the same features make one 128-row operand.
//   dx: W1 is summed over its rows, and is staged as it lies in two 64 x 64 boxes that the MMA
//   reads MN-major.
// * The summed dimension is shared out over the CTAs of a cluster where the row blocks alone
//   would leave SMs idle. The CTAs add up through distributed shared memory: each takes a share
//   of the tokens and reads its columns of every CTA's sums, in rank order, so no result
//   depends on timing and no second launch is needed.
// * Two CTAs per SM (at most 113 KB of ring each): one's epilogue overlaps the other's stream.
#include <algorithm>

#include "activation.cuh"
#include "gated.h"

namespace moe_lora {

constexpr int kFewThreads = 256;
constexpr int kFewRows = 128;

template <int N>
struct FewCfg {
  static constexpr int kWBytes = kFewRows * 64 * 2;
  static constexpr int kStageBytes = kWBytes + N * 64 * 2;
  static constexpr int kStages = N == 32 ? 5 : N == 64 ? 4 : 3;
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kSmemBytes = kBarOff + 256 + 1024;
  static constexpr uint32_t kTmemCols = N;
  static_assert(N * kFewRows * 4 <= kBarOff, "the sums reuse the ring");
  static_assert(2 * (kSmemBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

struct FewArgs {
  CUtensorMap tm_w, tm_x;
  int T, rows, K;       // rows: features (gated) or columns of dx
  int ks, kper;         // CTAs per cluster, 64-wide steps of each
  int up_off;
  const void* dh;
  void* out;
  unsigned int* err;
  unsigned long long wait_ns;
};

// Four floats at `addr`'s offset in CTA `rank` of the cluster.
__device__ __forceinline__ float4 ld_peer(uint32_t addr, int rank) {
  float4 v;
  uint32_t peer;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(peer) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer));
  return v;
}
__device__ __forceinline__ void add4(float (&s)[4], const float4& v) {
  s[0] += v.x;
  s[1] += v.y;
  s[2] += v.z;
  s[3] += v.w;
}

template <typename T, int N, int kEpi, int kAct>
__global__ void __launch_bounds__(kFewThreads) few_tokens_kernel(const __grid_constant__ FewArgs a) {
  using C = FewCfg<N>;
  constexpr int STAGES = C::kStages;
  constexpr bool kGated = kEpi != kEpiStore;
  constexpr int kCols = kGated ? kFewRows / 2 : kFewRows;  // output columns per cluster
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + STAGES;
  uint64_t* done = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* s_abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_issued = reinterpret_cast<int*>(tmem_slot + 2);
  float* sums = reinterpret_cast<float*>(smem);  // [N][128], after the ring is done

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.ks > 1 ? (int)cluster_ctarank() : 0;
  const int block = blockIdx.x / a.ks;
  const int k0 = rank * a.kper;
  const int nk = min(a.kper, (a.K + 63) / 64 - k0);

  // (no copy takes as long as one try: a limit of 0 tests)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return a.wait_ns ? mbar_wait_bounded(bar, parity, a.wait_ns) : mbar_test(bar, parity);
  };
  // fn(box, c0, c1) for the two boxes of step i's weights: the gate's and the up's rows, or
  // two neighbours along dx's columns
  auto weight_boxes = [&](int i, auto&& fn) {
    const int k = (k0 + i) * 64, r0 = block * kCols;
    if (kGated) {
      fn(0, k, r0);
      fn(1, k, a.up_off + r0);
    } else {
      fn(0, r0, k);
      fn(1, r0 + 64, k);
    }
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *s_abort = 0;
    *s_issued = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&a.tm_w);
    tma_prefetch_desc(&a.tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  // Weights are pulled towards L2, as far as the ring goes, while earlier launches may still run,
  // and read only after the wait: one of those may be writing them. (Not the last launch alone: a
  // kernel that triggers its dependents before its own wait lets this one start while the
  // launches before it run too.) A prefetch delivers nothing but to L2, where such writes arrive as
  // well. Without it 8.9 against 8.1 us for one token of 2880/2880.
  if (warp == 0) {
    if (elect_one())
      for (int i = 0; i < min(STAGES, nk); ++i)
        weight_boxes(i, [&](int box, int c0, int c1) {
          if (kGated || box == 0 || c0 < a.rows) tma_prefetch_2d(&a.tm_w, c0, c1);
        });
    __syncwarp();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now, with the tensor memory in hand: a dependent CTA on this SM may take the rest
  if (threadIdx.x == 0) pdl_trigger();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // producer and, below, MMA issuer: warp-uniform loops, one elected lane issues
    const bool elected = elect_one();
    const uint64_t pol_w = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
    bool ok = true;
    int s = 0;
    uint32_t ph = 1;
    int i = 0;
    for (; i < nk; ++i) {
      if (i >= STAGES) {
        ok = __all_sync(0xffffffffu, wait(&empty[s], ph) && !*s_abort);
        if (!ok) break;
      }
      if (elected) {
        uint8_t* sw = smem + s * C::kStageBytes;
        mbar_arrive_expect_tx(&full[s], (uint32_t)(C::kWBytes + a.T * 128));
        weight_boxes(i, [&](int box, int c0, int c1) { tma_load_2d(sw + box * 8192, &a.tm_w, &full[s], c0, c1, pol_w); });
        tma_load_2d(sw + C::kWBytes, &a.tm_x, &full[s], (k0 + i) * 64, 0, pol_x);
      }
      __syncwarp();
      if (++s == STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
    if (lane == 0) {
      *s_issued = i;
      if (!ok) *s_abort = 1;
    }
  } else if (warp == 1) {
    const bool elected = elect_one();
    const uint32_t idesc = (1u << 4) | (MmaType<T>::kFmt << 7) | (MmaType<T>::kFmt << 10) |
                           ((kGated ? 0u : 1u) << 15) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t s0 = smem_u32(smem);
    const uint64_t da0 = kGated ? smem_desc_sw128(s0) : smem_desc_mn(s0);
    const uint64_t db0 = smem_desc_sw128(s0 + C::kWBytes);
    constexpr uint32_t kAStep = kGated ? 32 >> 4 : 2048 >> 4;
    bool ok = true;
    int s = 0;
    uint32_t ph = 0;
    for (int i = 0; i < nk; ++i) {
      ok = __all_sync(0xffffffffu, wait(&full[s], ph) && !*s_abort);
      if (!ok) break;
      tc_fence_after();
      if (elected) {
        const uint64_t off = (uint64_t)(s * (C::kStageBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_bf16(tmem, da0 + off + kk * kAStep, db0 + off + kk * 2, idesc, (i | kk) != 0);
        tc_commit(&empty[s]);
      }
      __syncwarp();
      if (++s == STAGES) {
        s = 0;
        ph ^= 1;
      }
    }
    if (!ok && lane == 0) *s_abort = 1;
    if (elected) tc_commit(done);  // also after a give-up: arrives once every MMA is over
    __syncwarp();
  }
  // The sums of this CTA's share, token by token, over the ring: every copy has landed and
  // been consumed once the last MMA is over (or, after a give-up, is waited for here).
  if (!__all_sync(0xffffffffu, mbar_wait_bounded(done, 0, a.wait_ns + kWaitLimitNs)) && lane == 0) *s_abort = 1;
  __syncthreads();
  tc_fence_after();
  if (*s_abort) {
    if (threadIdx.x == 0) {
      for (int g = *s_issued - 1; g >= 0 && g >= *s_issued - STAGES; --g)
        mbar_wait_bounded(&full[g % STAGES], (g / STAGES) & 1);
      atomicOr(a.err, MOE_LORA_DEVERR_TIMEOUT);
    }
    __syncthreads();
  } else {
    // TMEM lanes [32 (w % 4), + 32), as many weight rows, of every other 16 tokens
    const int quad = warp & 3;
    for (int c = (warp >> 2) * 16; c < N && c < a.T; c += 32) {
      uint32_t v[16];
      __syncwarp();
      tmem_ld_x16(tmem + c + ((uint32_t)(quad * 32) << 16), v);
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 16; ++q) sums[(c + q) * kFewRows + quad * 32 + lane] = __uint_as_float(v[q]);
    }
    tc_fence_before();
  }
  if (a.ks > 1) cluster_sync();
  else __syncthreads();
  // Every CTA finishes a share of the tokens; a thread takes four columns at a time (the
  // output's columns are a multiple of 8), consecutive threads consecutive columns.
  const int per = (a.T + a.ks - 1) / a.ks, t0 = rank * per, t1 = min(a.T, t0 + per);
  constexpr int kQuads = kCols / 4;
#pragma unroll 1
  for (int i = threadIdx.x; i < (t1 - t0) * kQuads; i += kFewThreads) {
    const int tok = t0 + i / kQuads, c = (i % kQuads) * 4, n = block * kCols + c;
    if (n >= a.rows) continue;
    uint2 e2 = make_uint2(0, 0);
    if (kEpi == kEpiGrad)
      e2 = __ldcg(reinterpret_cast<const uint2*>(static_cast<const T*>(a.dh) + (int64_t)tok * a.rows + n));
    float v[4] = {}, w[4] = {};
    const float* at = sums + tok * kFewRows + c;
    if (a.ks > 1) {
      const uint32_t addr = smem_u32(at);
      for (int r = 0; r < a.ks; ++r) {
        add4(v, ld_peer(addr, r));
        if (kGated) add4(w, ld_peer(addr + kFewRows / 2 * 4, r));
      }
    } else {
      add4(v, *reinterpret_cast<const float4*>(at));
      if (kGated) add4(w, *reinterpret_cast<const float4*>(at + kFewRows / 2));
    }
    if constexpr (kEpi == kEpiStore) {
      *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (int64_t)tok * a.rows + n) =
          make_uint2(Elem<T>::r2(v[0], v[1]), Elem<T>::r2(v[2], v[3]));
    } else {
      float ac[4], d[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) activation<kAct>(v[q], ac[q], d[q]);
      if (kEpi == kEpiGated) {
        *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (int64_t)tok * a.rows + n) =
            make_uint2(Elem<T>::r2(ac[0] * w[0], ac[1] * w[1]), Elem<T>::r2(ac[2] * w[2], ac[3] * w[3]));
      } else {
        const float2 ea = Elem<T>::f2(e2.x), eb = Elem<T>::f2(e2.y);
        T* o = static_cast<T*>(a.out) + (int64_t)tok * 2 * a.rows + n;
        *reinterpret_cast<uint2*>(o) = make_uint2(Elem<T>::r2(ea.x * w[0] * d[0], ea.y * w[1] * d[1]),
                                                  Elem<T>::r2(eb.x * w[2] * d[2], eb.y * w[3] * d[3]));
        *reinterpret_cast<uint2*>(o + a.rows) =
            make_uint2(Elem<T>::r2(ea.x * ac[0], ea.y * ac[1]), Elem<T>::r2(eb.x * ac[2], eb.y * ac[3]));
      }
    }
  }
  if (a.ks > 1) cluster_sync();  // the sums are read before any CTA leaves
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <typename T, int N, int kEpi, int kAct>
static int launch_few_n(FewArgs& a, int blocks, cudaStream_t stream) {
  using C = FewCfg<N>;
  auto kernel = few_tokens_kernel<T, N, kEpi, kAct>;
  static std::atomic<uint64_t> seen[kMaxDevices];
  const int st = once_per_context(seen, [&] {
    ML_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes));
    return MOE_LORA_OK;
  });
  if (st != MOE_LORA_OK) return st;
  return launch_pdl_cluster(kernel, dim3((unsigned)blocks * a.ks), kFewThreads, C::kSmemBytes, stream, true, a.ks, a);
}
template <typename T, int kEpi, int kAct>
static int launch_few_t(FewArgs& a, int blocks, cudaStream_t stream) {
  return a.T <= 32   ? launch_few_n<T, 32, kEpi, kAct>(a, blocks, stream)
         : a.T <= 64 ? launch_few_n<T, 64, kEpi, kAct>(a, blocks, stream)
                     : launch_few_n<T, 128, kEpi, kAct>(a, blocks, stream);
}

static int launch_few(FewArgs& a, int dtype, int act, int epi, int blocks, cudaStream_t s) {
  if (dtype == MOE_DTYPE_BF16) {
    using E = __nv_bfloat16;
    if (epi == kEpiStore) return launch_few_t<E, kEpiStore, MOE_ACT_NONE>(a, blocks, s);
    if (epi == kEpiGated)
      return act == MOE_ACT_SILU ? launch_few_t<E, kEpiGated, MOE_ACT_SILU>(a, blocks, s)
                                 : launch_few_t<E, kEpiGated, MOE_ACT_GELU>(a, blocks, s);
    return act == MOE_ACT_SILU ? launch_few_t<E, kEpiGrad, MOE_ACT_SILU>(a, blocks, s)
                               : launch_few_t<E, kEpiGrad, MOE_ACT_GELU>(a, blocks, s);
  }
  using E = __half;
  if (epi == kEpiStore) return launch_few_t<E, kEpiStore, MOE_ACT_NONE>(a, blocks, s);
  if (epi == kEpiGated)
    return act == MOE_ACT_SILU ? launch_few_t<E, kEpiGated, MOE_ACT_SILU>(a, blocks, s)
                               : launch_few_t<E, kEpiGated, MOE_ACT_GELU>(a, blocks, s);
  return act == MOE_ACT_SILU ? launch_few_t<E, kEpiGrad, MOE_ACT_SILU>(a, blocks, s)
                             : launch_few_t<E, kEpiGrad, MOE_ACT_GELU>(a, blocks, s);
}

// CTAs per cluster: enough to fill two CTAs on each of 152 SMs, four steps each at least.
static void split_few(FewArgs& a, int blocks) {
  const int steps = ceil_div(a.K, 64);
  int ks = std::min(8, std::max(1, 304 / blocks));
  ks = std::max(1, std::min(ks, steps / 4));
  a.kper = ceil_div(steps, ks);
  a.ks = ceil_div(steps, a.kper);
}

int launch_gated_few(int dtype, int act, const void* x, const void* W1, int T, int H, int I, const void* dh, void* out,
                     cudaStream_t stream) {
  FewArgs a = {};
  int st = operand_map(&a.tm_w, W1, 2 * (int64_t)I, H, false, 64);
  if (st == MOE_LORA_OK) st = operand_map(&a.tm_x, x, T, H, false, T);
  if (st == MOE_LORA_OK) st = ffn_error_word(&a.err);
  if (st != MOE_LORA_OK) return st;
  a.T = T;
  a.rows = I;
  a.K = H;
  a.up_off = I;
  a.dh = dh;
  a.out = out;
  a.wait_ns = ffn_wait_ns();
  const int blocks = ceil_div(I, kFewRows / 2);
  split_few(a, blocks);
  return launch_few(a, dtype, act, dh ? kEpiGrad : kEpiGated, blocks, stream);
}

int launch_dx_few(int dtype, const void* dy, const void* W1, int T, int H, int I, void* dx, cudaStream_t stream) {
  FewArgs a = {};
  int st = operand_map(&a.tm_w, W1, 2 * (int64_t)I, H, true, 64);
  if (st == MOE_LORA_OK) st = operand_map(&a.tm_x, dy, T, 2 * (int64_t)I, false, T);
  if (st == MOE_LORA_OK) st = ffn_error_word(&a.err);
  if (st != MOE_LORA_OK) return st;
  a.T = T;
  a.rows = H;
  a.K = 2 * I;
  a.out = dx;
  a.wait_ns = ffn_wait_ns();
  const int blocks = ceil_div(H, kFewRows);
  split_few(a, blocks);
  return launch_few(a, dtype, MOE_ACT_NONE, kEpiStore, blocks, stream);
}

}  // namespace moe_lora
