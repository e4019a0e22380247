// The pass before the projection's products (lora_linear.cu): z = x A^T and v = dy B, and what else
// they need.
//
// It is bound by reading the rows and, where an adapter has many, its weights again from L2 for
// each 16 of them, at some tens of operations a byte, so mma.sync is fast enough and takes
// operands as they come. 16384 rows of 2880 with 512 pairs of rank 16: 30 us (4.4 TB/s); both
// shrinks of 4096 rows of 4096 and 11008, 16 adapters of rank 32: 48 us (0.4 GB through L2).
// * A CTA takes a LoRA block of the align buffer (at most 16 rows of one expert and adapter)
//   and up to 64 ranks; its warps split the long sum in steps of 32 and add up in a fixed order. Rows and A go from memory to the MMA's fragments in 16-byte loads: the
//   sum's order is free, so a lane's eight neighbouring columns serve as its columns of two
//   MMAs. B has its ranks contiguous, and its steps are transposed on the way through shared
//   memory (ldmatrix).
#include <algorithm>

#include "lora_linear.h"

namespace moe_lora {

// ---------------------------------------------------------------------------
// before the products
// ---------------------------------------------------------------------------
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&v)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}

// A shrink's shape: WARPS warps share the sum over 16 rows by NT x 8 ranks.
template <int NT, int WARPS>
struct ShrinkCfg {
  static constexpr int kThreads = WARPS * 32;
  // steps of 32 columns in flight per warp: as many as some 100 registers hold
  static constexpr int kSteps = NT == 1 ? 8 : NT == 2 ? 6 : NT == 4 ? 4 : 2;
  static constexpr int kTransSteps = NT == 8 ? 3 : 4;
  static constexpr int kPitch = NT * 16 + 16, kStage = 32 * kPitch;  // of B in shared memory
  static constexpr int kRedBytes = WARPS * 16 * NT * 8 * 4;
  static constexpr int kTransBytes = WARPS * kTransSteps * kStage;
  static constexpr int kSmemBytes = kTransBytes > kRedBytes ? kTransBytes : kRedBytes;
  static constexpr int kMinCtas = WARPS == 16 ? 1 : 2;
};

// The `n` sorted rows from r0 on, of one pair, times up to NT x 8 ranks from c0 on.
template <typename T, int NT, int WARPS, bool kTrans>
__device__ __forceinline__ void shrink_rows(const RowsPassArgs& a, const ShrinkPart& p, int r0, int n, int64_t pair, int c0,
                                            uint8_t* smem) {
  using S = ShrinkCfg<NT, WARPS>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int C = p.C, ranks = min(NT * 8, a.r - c0);
  const T* x[2];  // rows past the last one are it again, and are not stored
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = r0 + min(8 * i + g, n - 1);
    x[i] = static_cast<const T*>(p.in) + (int64_t)(a.rows.slots ? __ldcg(a.rows.slots + row) : row) * C + 8 * q;
  }
  float acc[NT][4] = {};
  const uint4 none = make_uint4(0, 0, 0, 0);
  auto ld = [](const T* at) { return __ldcg(reinterpret_cast<const uint4*>(at)); };
  auto mma = [&](float (&d)[4], const uint4& u0, const uint4& u1, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
    mma16816<T>(d, u0.x, u1.x, u0.y, u1.y, w0, w1);
    mma16816<T>(d, u0.z, u1.z, u0.w, u1.w, w2, w3);
  };
  constexpr int U = kTrans ? S::kTransSteps : S::kSteps, kStride = WARPS * 32;
  uint4 u[U][2];
  if constexpr (!kTrans) {
    const T* A = static_cast<const T*>(p.M) + (pair * a.r + c0) * C + 8 * q;
    uint4 w[U][NT];
    auto load = [&](int s, int k) {
      const bool in = k + 8 * q < C;
#pragma unroll
      for (int i = 0; i < 2; ++i) u[s][i] = in ? ld(x[i] + k) : none;
#pragma unroll
      for (int t = 0; t < NT; ++t) w[s][t] = in ? ld(A + (int64_t)min(t * 8 + g, ranks - 1) * C + k) : none;
    };
#pragma unroll
    for (int s = 0; s < U; ++s) load(s, (warp + WARPS * s) * 32);
    for (int k0 = warp * 32; k0 < C; k0 += U * kStride) {
#pragma unroll
      for (int s = 0; s < U; ++s) {
#pragma unroll
        for (int t = 0; t < NT; ++t) mma(acc[t], u[s][0], u[s][1], w[s][t].x, w[s][t].y, w[s][t].z, w[s][t].w);
        load(s, k0 + (U + s) * kStride);
      }
    }
  } else {
    const T* B = static_cast<const T*>(p.M) + pair * C * a.r + c0;
    uint8_t* mine = smem + warp * U * S::kStage;
    // Row k of a step lies where the eight rows that one 8 x 8 matrix takes are neighbours: lane
    // q's columns 8q + 2m, + 1 are rows 2q, 2q + 1 of matrix m.
    auto load = [&](int s, int k0) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int at = i * 32 + lane, k = at / NT, c = (at % NT) * 8;  // eight ranks of one row
        const int place = ((k & 7) >> 1) * 8 + (k >> 3) * 2 + (k & 1);
        const bool in = k0 + k < C && c < ranks;
        if (k0 < C) cp_async16(mine + s * S::kStage + place * S::kPitch + c * 2, in ? B + (int64_t)(k0 + k) * a.r + c : B, in);
      }
      cp_async_commit();
      const bool in = k0 + 8 * q < C;
#pragma unroll
      for (int i = 0; i < 2; ++i) u[s][i] = in ? ld(x[i] + k0) : none;
    };
#pragma unroll
    for (int s = 0; s < U; ++s) load(s, (warp + WARPS * s) * 32);
    for (int k0 = warp * 32; k0 < C; k0 += U * kStride) {
#pragma unroll
      for (int s = 0; s < U; ++s) {
        if (k0 + s * kStride >= C) break;
        cp_async_wait<U - 1>();
        __syncwarp();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t w[4];  // matrix m = lane / 8, its row lane % 8
          ldmatrix_x4_trans(w, smem_u32(mine + s * S::kStage + lane * S::kPitch + t * 16));
          mma(acc[t], u[s][0], u[s][1], w[0], w[1], w[2], w[3]);
        }
        __syncwarp();  // read before the next step's copies land here
        load(s, k0 + (U + s) * kStride);
      }
    }
    cp_async_wait<0>();
    __syncthreads();  // the stages' memory takes the partial sums
  }
  // [warp][16 rows][NT x 8 ranks]
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2*>(red + ((warp * 16 + g + 8 * h) * NT + t) * 8 + 2 * q) =
          make_float2(acc[t][2 * h], acc[t][2 * h + 1]);
  __syncthreads();
  for (int i = threadIdx.x; i < n * NT * 8; i += S::kThreads) {
    const int row = i / (NT * 8), c = i % (NT * 8);
    if (c >= ranks) continue;
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += red[w * 16 * NT * 8 + i];
    p.dst[(int64_t)(r0 + row) * a.r + c0 + c] = sum;
  }
}

// One LoRA block.
template <typename T, int NT, int WARPS, bool kTrans>
__device__ __forceinline__ void shrink_block(const RowsPassArgs& a, const ShrinkPart& p, int block, int c0, uint8_t* smem) {
  if (block >= __ldcg(a.rows.hdr + HDR_NBLOCKS)) return;
  const int4 b = __ldcg(a.rows.blocks + block);  // first row, rows, expert, adapter
  shrink_rows<T, NT, WARPS, kTrans>(a, p, b.x, b.y, (int64_t)b.w * a.rows.E + b.z, c0, smem);
}

// CTAs: for each part and NT x 8 ranks one per LoRA block; then one per group of rows to be
// copied in sorted order; those that zero dropped rows; those that look the pairs' first rows up.
struct RowsPassGrid {
  int chunks, shrink[2], copy, zero, seg;  // CTAs of each kind
};

template <typename T, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, ShrinkCfg<NT, WARPS>::kMinCtas)
    rows_pass_kernel(const RowsPassArgs a, const RowsPassGrid gr) {
  extern __shared__ __align__(16) uint8_t smem_pass[];
  pdl_wait();
  pdl_trigger();  // every CTA has waited: what an earlier launch wrote, the next one may read
  int id = blockIdx.x;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (id < gr.shrink[part]) {
      const int block = id / gr.chunks, c0 = id % gr.chunks * NT * 8;
      if (part == 0) shrink_block<T, NT, WARPS, false>(a, a.part[0], block, c0, smem_pass);
      else shrink_block<T, NT, WARPS, true>(a, a.part[1], block, c0, smem_pass);
      return;
    }
    id -= gr.shrink[part];
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (id < gr.copy) {
    constexpr int kPer = 256 / kLinearGroup;  // groups per tile
    if (id / kPer >= __ldcg(a.rows.hdr + HDR_NTILES)) return;
    const int4 t = __ldcg(a.rows.tiles + id / kPer);
    const int at = id % kPer * kLinearGroup, n = min(kLinearGroup, t.z - at);
    if (n <= 0) return;
    bool apart;
    const int from = group_row(a.rows.slots, t.y + at, n, &apart);
    if (!apart) return;
    const int units = a.copy_n / 8;
    for (int i = warp; i < n; i += WARPS) {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(a.copy_in) +
                                                        (int64_t)__shfl_sync(0xffffffffu, from, i) * a.copy_n);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.copy_out) + (int64_t)(t.y + at + i) * a.copy_n);
      for (int c = lane; c < units; c += 128) {
        uint4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c + 32 * u < units) v[u] = __ldcg(src + c + 32 * u);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c + 32 * u < units) dst[c + 32 * u] = v[u];
      }
    }
    return;
  }
  id -= gr.copy;
  const int n_valid = __ldcg(a.rows.hdr + HDR_NVALID);
  if (id < gr.zero) {
    if (n_valid == a.rows.S) return;
    for (int r0 = (id * WARPS + warp) * 32; r0 < a.rows.S; r0 += gr.zero * WARPS * 32) {
      const int row = r0 + lane;
      const bool drop = row < a.rows.S && (a.rows.slots ? __ldcg(a.rows.slot_row + row) < 0 : row >= n_valid);
      uint32_t set = __ballot_sync(0xffffffffu, drop);
      for (; set; set &= set - 1) {
        uint4* at = reinterpret_cast<uint4*>(static_cast<T*>(a.zero_out) + (int64_t)(r0 + __ffs(set) - 1) * a.zero_n);
        for (int c = lane; c < a.zero_n / 8; c += 32) at[c] = make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }
  id -= gr.zero;
  // pair (e, l): the first of expert e's rows, sorted by adapter, whose adapter is l or more
  const int64_t pair = (int64_t)id * (WARPS * 32) + threadIdx.x;
  if (pair >= (int64_t)a.rows.E * a.rows.L) return;
  const int e = (int)(pair / a.rows.L), l = (int)(pair % a.rows.L);
  int lo = __ldcg(a.rows.expert_begin + e), hi = __ldcg(a.rows.expert_begin + e + 1);
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldcg(a.rows.row_adapter + mid) < l) lo = mid + 1;
    else hi = mid;
  }
  a.seg_begin[pair] = lo;
}

template <typename T, int NT, int WARPS>
static int launch_rows_pass_n(const RowsPassArgs& a, cudaStream_t stream) {
  using S = ShrinkCfg<NT, WARPS>;
  auto kernel = rows_pass_kernel<T, NT, WARPS>;
  static std::atomic<uint64_t> seen[kMaxDevices];
  const int st = once_per_context(seen, [&] {
    ML_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes));
    return MOE_LORA_OK;
  });
  if (st != MOE_LORA_OK) return st;
  RowsPassGrid g = {};
  g.chunks = ceil_div(a.r, NT * 8);
  int64_t ctas = 0;
  for (int i = 0; i < 2; ++i) {
    if (a.part[i].in) g.shrink[i] = a.rows.max_blocks * g.chunks;
    ctas += g.shrink[i];
  }
  if (a.copy_out) g.copy = a.rows.max_tiles * (256 / kLinearGroup);
  if (a.zero_out) g.zero = std::min(ceil_div(a.rows.S, WARPS * 32), 152);
  if (a.seg_begin) g.seg = (int)ceil_div64((int64_t)a.rows.E * a.rows.L, WARPS * 32);
  ctas += g.copy + g.zero + g.seg;
  return launch_pdl(kernel, (unsigned)ctas, S::kThreads, a.part[1].in ? S::kSmemBytes : S::kRedBytes, stream, true, a, g);
}

// With few blocks the ranks are cut into chunks so that every SM (152: a fixed number, so that a sum's
// order goes by the shape alone) has some, and twice the warps share a sum's latency. With many
// each block reads its adapter again from L2; two blocks a CTA halved that and took longer (4096
// rows of 16 adapters 62 to 71 against 47 us: half the warps).
template <typename T>
static int launch_rows_pass_t(const RowsPassArgs& a, cudaStream_t s) {
  const int tiles = ceil_div(a.r, 8), blocks = a.rows.max_blocks;
  int nt = tiles == 1 ? 1 : tiles == 2 ? 2 : tiles <= 4 ? 4 : 8;
  while (nt > 2 && blocks * ceil_div(tiles, nt) < 152) nt /= 2;
  if (nt <= 2 && blocks * ceil_div(tiles, nt) <= 152)
    return nt == 1 ? launch_rows_pass_n<T, 1, 16>(a, s) : launch_rows_pass_n<T, 2, 16>(a, s);
  return nt == 1   ? launch_rows_pass_n<T, 1, 8>(a, s)
         : nt == 2 ? launch_rows_pass_n<T, 2, 8>(a, s)
         : nt == 4 ? launch_rows_pass_n<T, 4, 8>(a, s)
                   : launch_rows_pass_n<T, 8, 8>(a, s);
}

int launch_rows_pass(const RowsPassArgs& a, int dtype, cudaStream_t stream) {
  return dtype == MOE_DTYPE_BF16 ? launch_rows_pass_t<__nv_bfloat16>(a, stream) : launch_rows_pass_t<__half>(a, stream);
}

}  // namespace moe_lora
