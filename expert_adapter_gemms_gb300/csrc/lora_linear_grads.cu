// The adapters' gradients dA = v^T x and dB = dy^T z over each (expert, adapter) pair's rows, on
// tcgen05.
//
// Bound by reading x and dy once. A unit is a pair and 128 columns of x (or dy): the product
// D [128 columns, ranks] = sum over the pair's rows of x^T v, 64 rows a step. x lies with its
// columns contiguous and is the MMA's M side as it lies (MN-major); so is v on the N side.
// * Rows are fetched by their numbers with cp.async (any order, none copied twice), rows past the
//   pair's last as zeros, so that no other pair's values meet this one.
// * v and z are fp32 and enter as two 16-bit values side by side on the N side, their first bits
//   and the remainder's: both products in one MMA, added when D is read. In fp16 the remainder is
//   scaled by 2^11, so that values below fp16's steps keep theirs: off by 2^-23 of v or 2^-36 (bf16:
//   2^-17 of it).
// * Three CTAs an SM (two or one at more ranks) of eight warps, which fetch, split and store in turn.
//   (Those jobs given to warps of their own in one or two CTAs were no faster.)
// * With few units the rows are shared out over a cluster whose CTAs add up through distributed
//   shared memory, in rank order. A pair without rows gets zeros.
// 4096 rows of 4096 and 11008 columns, 16 adapters of 32 ranks: 43 us cold (2.8 TB/s; rows are read in
// pieces of 256 bytes, and a kernel that only reads those takes 36). mma.sync in tf32 took 74.
#include <algorithm>

#include "lora_linear.h"

namespace moe_lora {

constexpr int kDThreads = 256, kDCols = 128, kDRows = 64;

// RB: blocks of 64 columns that both halves of the ranks take.
template <int RB>
struct GradCfg {
  static constexpr int kXBytes = kDRows * kDCols * 2;
  static constexpr int kStageBytes = kXBytes + RB * 8192;
  static constexpr int kStages = RB == 4 ? 4 : 3;
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kSmemBytes = kBarOff + 128 + 1024;
  static constexpr int kCtas = RB == 1 ? 3 : RB == 2 ? 2 : 1;  // per SM
  static constexpr int kVUnits = RB;                           // 8 ranks of a row, per thread
  static constexpr int kPitch = kDCols + 4;                    // floats between ranks of the sums
  static_assert(kDRows * RB * 4 == kVUnits * kDThreads, "v units");
  static_assert(RB * 32 * kPitch * 4 <= kBarOff, "the sums reuse the stages");
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "CTAs per SM");
};

struct GradArgs {
  AdapterGradArgs g;
  int chunks_a, chunks;  // 128-column chunks of x, and of x and dy
  int64_t units;
  int ks;                // CTAs per cluster
  unsigned int* err;
  unsigned long long wait_ns;
};

template <typename T> struct RestScale { static constexpr float up = 1.f, down = 1.f; };
template <> struct RestScale<__half> { static constexpr float up = 2048.f, down = 1.f / 2048.f; };

template <typename T, int RB>
__global__ void __launch_bounds__(kDThreads, GradCfg<RB>::kCtas) adapter_grads_kernel(const __grid_constant__ GradArgs p) {
  using C = GradCfg<RB>;
  const AdapterGradArgs& a = p.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* empty = reinterpret_cast<uint64_t*>(smem + C::kBarOff);  // per stage: its MMAs are over
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(empty + C::kStages);
  float* sums = reinterpret_cast<float*>(smem);  // [ranks][kPitch], after a unit's last MMA
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = p.ks > 1 ? (int)cluster_ctarank() : 0;
  const int r16 = (a.r + 15) & ~15;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(&empty[s], 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, RB * 64);
    tmem_relinquish();
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) pdl_trigger();  // with the tensor memory in hand
  const uint32_t tmem = *tmem_slot;
  const uint32_t idesc = (1u << 4) | (MmaType<T>::kFmt << 7) | (MmaType<T>::kFmt << 10) | (1u << 15) | (1u << 16) |
                         ((uint32_t)(2 * r16 >> 3) << 17) | ((128u >> 4) << 24);
  const uint64_t dx0 = smem_desc_mn(smem_u32(smem)), dv0 = smem_desc_mn(smem_u32(smem) + C::kXBytes);
  uint32_t used = 0;  // steps of all units before this one: with its own, a step's stage and phase
  bool ok = true, late = false;
  // Waits until the MMAs of step `u` (counted over all units) are over. One that takes longer than
  // the limit is reported, and still waited for by the default limit: the CTAs of a cluster go
  // through the same units to the end.
  auto free_of = [&](uint32_t u) {
    uint64_t* bar = &empty[u % C::kStages];
    const uint32_t parity = (u / C::kStages) & 1;
    if (!ok || (p.wait_ns ? mbar_wait_bounded(bar, parity, p.wait_ns) : mbar_test(bar, parity))) return;
    late = true;
    ok = mbar_wait_bounded(bar, parity);
  };

  for (int64_t unit = blockIdx.x / p.ks; unit < p.units; unit += gridDim.x / p.ks) {
    const int pair = (int)(unit / p.chunks), chunk = (int)(unit - (int64_t)pair * p.chunks);  // pair = e L + l
    const bool is_a = chunk < p.chunks_a;
    const int e = pair / a.rows.L, l = pair - e * a.rows.L;
    const int cols = is_a ? a.K : a.N, c0 = (is_a ? chunk : chunk - p.chunks_a) * kDCols;
    const T* in = static_cast<const T*>(is_a ? a.x : a.dy);
    const float* small = is_a ? a.v : a.z;
    const int seg0 = __ldcg(a.seg_begin + pair);
    const int seg1 = l + 1 < a.rows.L ? __ldcg(a.seg_begin + pair + 1) : __ldcg(a.rows.expert_begin + e + 1);
    // this CTA's share of the rows
    const int all = (seg1 - seg0 + kDRows - 1) / kDRows, per = p.ks > 1 ? (all + p.ks - 1) / p.ks : all;
    const int r0 = seg0 + min(all, rank * per) * kDRows, r1 = min(seg1, r0 + per * kDRows);
    const int steps = max(0, (r1 - r0 + kDRows - 1) / kDRows);

    // x of step i: thread -> 16 bytes of four rows; the rows' numbers are looked up a step ahead
    int at[4];
    auto look = [&](int i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = r0 + i * kDRows + j * 16 + tid / 16;
        at[j] = row < r1 ? (a.rows.slots ? __ldcg(a.rows.slots + row) : row) : -1;
      }
    };
    auto fetch = [&](uint32_t u) {
      uint8_t* sx = smem + u % C::kStages * C::kStageBytes + (tid % 16 / 8) * 8192;
      const int c = c0 + (tid % 16) * 8;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = j * 16 + tid / 16;
        const bool there = at[j] >= 0 && c < cols;
        cp_async16(sx + k * 128 + (((tid & 7) ^ (k & 7)) << 4), there ? in + (int64_t)at[j] * cols + c : in, there);
      }
    };
    // v of step i: 8 ranks of a row at a time, through registers
    float4 v[C::kVUnits][2];
    const int groups = r16 / 8;
    auto load_v = [&](int i) {
#pragma unroll
      for (int q = 0; q < C::kVUnits; ++q) {
        const int w = q * kDThreads + tid, k = w / groups, c = w % groups * 8, row = r0 + i * kDRows + k;
        v[q][0] = v[q][1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < kDRows && row < r1 && c < a.r) {
          const float4* src = reinterpret_cast<const float4*>(small + (int64_t)row * a.r + c);
          v[q][0] = __ldcg(src);
          v[q][1] = __ldcg(src + 1);
        }
      }
    };
    auto put_v = [&](uint32_t u) {
      uint8_t* sv = smem + u % C::kStages * C::kStageBytes + C::kXBytes;
#pragma unroll
      for (int q = 0; q < C::kVUnits; ++q) {
        const int w = q * kDThreads + tid, k = w / groups, g = w % groups;
        if (k >= kDRows) continue;
        uint4 hi, lo;
        split8<T>(v[q][0], v[q][1], hi, lo, RestScale<T>::up);
        const auto put = [&](int n8, const uint4& bits) {  // ranks 8 n8 .. of both halves' columns
          *reinterpret_cast<uint4*>(sv + n8 / 8 * 8192 + k * 128 + (((n8 & 7) ^ (k & 7)) << 4)) = bits;
        };
        put(g, hi);
        put(groups + g, lo);
      }
    };

    if (steps > 0) {
      look(0);
      load_v(0);
    }
    for (int i = 0; i < C::kStages - 1; ++i) {
      if (i < steps) {  // (a unit starts with its stages free)
        fetch(used + i);
        look(i + 1);
      }
      cp_async_commit();
    }
    for (int i = 0; i < steps; ++i) {
      put_v(used + i);
      if (i + 1 < steps) load_v(i + 1);
      cp_async_wait<C::kStages - 2>();
      fence_proxy_async_smem();
      __syncthreads();
      if (warp == 0) {
        if (elect_one()) {
          tc_fence_after();
          const uint64_t off = (uint64_t)((used + i) % C::kStages * (C::kStageBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < kDRows / 16; ++kk)
            tc_mma_bf16(tmem, dx0 + off + kk * (2048 >> 4), dv0 + off + kk * (2048 >> 4), idesc, (i | kk) != 0);
          tc_commit(&empty[(used + i) % C::kStages]);
        }
        __syncwarp();
      }
      // the stage to fill next is that of the step before this one
      const int nx = i + C::kStages - 1;
      if (i > 0) free_of(used + i - 1);
      if (nx < steps) {
        fetch(used + nx);
        look(nx + 1);
      }
      cp_async_commit();
    }
    if (steps > 0) free_of(used + steps - 1);
    used += steps;
    cp_async_wait<0>();
    __syncthreads();
    tc_fence_after();
    // D: lanes are columns; both halves of a rank added, [rank][column]
    for (int i = (warp >> 2) * 16; i < r16; i += 32) {
      const int quad = warp & 3;
      uint32_t hi[16] = {}, lo[16] = {};
      if (steps > 0) {
        tmem_ld_x16(tmem + i + ((uint32_t)(quad * 32) << 16), hi);
        tmem_ld_x16(tmem + r16 + i + ((uint32_t)(quad * 32) << 16), lo);
        tmem_ld_wait();
      }
      float* to = sums + i * C::kPitch + quad * 32 + lane;
#pragma unroll
      for (int q = 0; q < 16; ++q) to[q * C::kPitch] = __uint_as_float(hi[q]) + __uint_as_float(lo[q]) * RestScale<T>::down;
    }
    tc_fence_before();
    if (p.ks > 1) cluster_sync();
    else __syncthreads();
    const int64_t place = (int64_t)l * a.rows.E + e;
    // four columns of one rank, over the cluster
    auto sum4 = [&](int i, int c) {
      const float* mine = sums + i * C::kPitch + c;
      if (p.ks == 1) return *reinterpret_cast<const float4*>(mine);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < p.ks; ++k) {
        float4 t;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(t.x), "=f"(t.y), "=f"(t.z), "=f"(t.w)
                     : "r"(smem_in_cta(mine, (uint32_t)k)));
        s.x += t.x;
        s.y += t.y;
        s.z += t.z;
        s.w += t.w;
      }
      return s;
    };
    if (is_a) {
      T* out = static_cast<T*>(a.dA) + place * a.r * a.K + c0;
      for (int u = rank * kDThreads + tid; u < a.r * (kDCols / 4); u += p.ks * kDThreads) {
        const int i = u / (kDCols / 4), c = u % (kDCols / 4) * 4;
        if (c0 + c >= a.K) continue;
        const float4 s = sum4(i, c);
        *reinterpret_cast<uint2*>(out + (int64_t)i * a.K + c) = make_uint2(Elem<T>::r2(s.x, s.y), Elem<T>::r2(s.z, s.w));
      }
    } else {
      // dB [N, r]: four columns by four ranks a thread, neighbours along the ranks
      T* out = static_cast<T*>(a.dB) + (place * a.N + c0) * a.r;
      const int quads = a.r / 4;
      for (int u = rank * kDThreads + tid; u < quads * (kDCols / 4); u += p.ks * kDThreads) {
        const int i = u % quads * 4, c = u / quads * 4;
        if (c0 + c >= a.N) continue;
        const float4 s[4] = {sum4(i, c), sum4(i + 1, c), sum4(i + 2, c), sum4(i + 3, c)};
        const float* f = reinterpret_cast<const float*>(s);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<uint2*>(out + (int64_t)(c + j) * a.r + i) =
              make_uint2(Elem<T>::r2(f[j], f[4 + j]), Elem<T>::r2(f[8 + j], f[12 + j]));
      }
    }
    if (p.ks > 1) cluster_sync();  // the sums have been read: the stages are free again
    else __syncthreads();
  }
  if (late) atomicOr(p.err, MOE_LORA_DEVERR_TIMEOUT);
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, RB * 64);
  }
}

template <typename T, int RB>
static int launch_grads(const AdapterGradArgs& g, cudaStream_t stream) {
  using C = GradCfg<RB>;
  auto kernel = adapter_grads_kernel<T, RB>;
  static std::atomic<uint64_t> seen[kMaxDevices];
  int st = once_per_context(seen, [&] {
    ML_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes));
    return MOE_LORA_OK;
  });
  if (st != MOE_LORA_OK) return st;
  GradArgs p = {};
  p.g = g;
  p.chunks_a = g.dA ? ceil_div(g.K, kDCols) : 0;
  p.chunks = p.chunks_a + (g.dB ? ceil_div(g.N, kDCols) : 0);
  p.units = (int64_t)g.rows.E * g.rows.L * p.chunks;
  // rows shared out while that leaves places of the SMs free and a CTA four steps of them
  const int64_t places = (int64_t)num_sms() * C::kCtas;
  const int64_t steps = ceil_div64(g.rows.S, (int64_t)kDRows * g.rows.E * g.rows.L);  // on average
  p.ks = 1;
  while (p.ks < 8 && p.units * p.ks * 2 <= places && steps >= p.ks * 8) p.ks *= 2;
  p.wait_ns = ffn_wait_ns();
  if ((st = ffn_error_word(&p.err)) != MOE_LORA_OK) return st;
  const unsigned ctas = (unsigned)(std::min(p.units, places / p.ks) * p.ks);
  return launch_pdl_cluster(kernel, dim3(ctas), kDThreads, C::kSmemBytes, stream, true, p.ks, p);
}

int launch_adapter_grads(const AdapterGradArgs& a, int dtype, cudaStream_t stream) {
  const int n = 2 * ceil_div(a.r, 16) * 16;
  if (dtype == MOE_DTYPE_BF16)
    return n <= 64    ? launch_grads<__nv_bfloat16, 1>(a, stream)
           : n <= 128 ? launch_grads<__nv_bfloat16, 2>(a, stream)
                      : launch_grads<__nv_bfloat16, 4>(a, stream);
  return n <= 64    ? launch_grads<__half, 1>(a, stream)
         : n <= 128 ? launch_grads<__half, 2>(a, stream)
                    : launch_grads<__half, 4>(a, stream);
}

}  // namespace moe_lora
