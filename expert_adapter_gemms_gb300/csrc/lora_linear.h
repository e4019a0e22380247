// A projection with the low-rank adapters of many requests beside it, and its gradients: what
// its translation units share.
//   z = x A^T,  y = x W^T + z B^T              per row, with the row's expert and adapter
//   v = dy B,   dx = dy W + v A,   dA = v^T x,  dB = dy^T z
// z and v are fp32 [S, r] by sorted row.
#pragma once

#include "gated.h"

namespace moe_lora {

// The rows as the align buffer has them. slots null: the operands' rows are in sorted order;
// else row i of the sorted order is row slots[i] of the operands (and slot_row the inverse).
struct LinearRows {
  const int* hdr;
  const int4* tiles;
  const int4* blocks;
  const int* row_adapter;
  const int* expert_begin;
  const int* slots;
  const int* slot_row;
  int S, E, L, max_tiles, max_blocks;
};

// Rows in the tokens' order reach the pair kernel's tiles in groups of kLinearGroup sorted rows:
// by one box where the group's rows are neighbours in the tokens' order too (a request's tokens,
// mostly), else from a copy in sorted order that the pass before makes of such groups only.
// (Fetched four at a time by their numbers, tile::gather4, 4096 rows by 4096 summed over
// 11008 columns took 818 us: some 70 cycles for each of a step's 32 gathers.)
constexpr int kLinearGroup = 32;
// This lane's row of a group of n (1 to 32) sorted rows from `first` on -> its row in the
// tokens' order (the last one's for lanes past it); *apart: whether they are not neighbours.
__device__ __forceinline__ int group_row(const int* slots, int first, int n, bool* apart) {
  const int lane = threadIdx.x & 31;
  const int at = __ldcg(slots + first + min(lane, n - 1));
  const int base = __shfl_sync(0xffffffffu, at, 0);
  *apart = __any_sync(0xffffffffu, lane < n && at != base + lane);
  return at;
}

// Up to kLinearFewRows rows of a single expert go through one 128-row tile whose sum is shared
// by a cluster (lora_linear_few.cu); more, or several experts, through 256-row tiles on CTA
// pairs (lora_linear.cu).
constexpr int kLinearFewRows = 128;

// One shrink: dst[row, i] = sum_c in[row, c] M(i, c) over the rows that have an adapter. M is
// A [L, E, r, C] (sum over the contiguous dimension) or, `trans`, B [L, E, C, r].
struct ShrinkPart {
  const void* in;
  const void* M;
  float* dst;
  int C;
};

// The launch before the products: up to two shrinks (part[1] transposed), rows of dropped
// slots of `zero_out` [S, zero_n] set to zero, the first sorted row of each (expert, adapter)
// pair into seg_begin [E L] (null: not wanted), and the copies in sorted order.
struct RowsPassArgs {
  LinearRows rows;
  ShrinkPart part[2];
  int r;
  void* zero_out;
  int zero_n;
  int* seg_begin;
  const void* copy_in;  // the product's rows in the tokens' order [S, copy_n], and where groups
  void* copy_out;       // of them that are not neighbours go in sorted order (null: none)
  int copy_n;
};
int launch_rows_pass(const RowsPassArgs& a, int dtype, cudaStream_t stream);

// out [S, N] = in [S, K] M(e)^T + z (the adapter's U)^T, by rows: the forward with M = W [E, N, K]
// and U = B [L, E, N, r], or `mn` with M = W [E, K, N] and U = A [L, E, r, N] (N contiguous).
struct ProductArgs {
  LinearRows rows;
  const void *in, *M, *U;
  const void* sorted;  // the copies in sorted order (rows.slots given, more than kLinearFewRows rows)
  const float* z;
  void* out;
  int N, K, r;
  bool mn;
};
int launch_linear_product(const ProductArgs& a, int dtype, cudaStream_t stream);
int launch_linear_product_few(const ProductArgs& a, int dtype, cudaStream_t stream);
// The tensor map of M or U: [third][rows][cols] with cols contiguous, K-major boxes of box_cols
// (64, 32 or 16, under the swizzle of that width) columns by box_rows rows or (mn) of 64 by
// box_rows; what lies past an end reads zero.
int linear_map(CUtensorMap* m, const void* base, int64_t third, int64_t rows, int64_t cols, bool mn, int box_rows,
               int box_cols = 64);

// dA [L, E, r, K] = v^T x and dB [L, E, N, r] = dy^T z over each pair's rows (zero for a pair
// without rows); dA or dB may be null.
struct AdapterGradArgs {
  LinearRows rows;
  const void *x, *dy;
  const float *z, *v;
  const int* seg_begin;
  void *dA, *dB;
  int K, N, r;
};
int launch_adapter_grads(const AdapterGradArgs& a, int dtype, cudaStream_t stream);

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// D += A B with the TMEM lanes (rows of D) whose bit is set in `off` left as they are.
__device__ __forceinline__ void tc_mma_lanes(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             const uint32_t (&off)[4]) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7}, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
      : "memory");
}
__device__ __forceinline__ void tc_mma_lanes_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                  const uint32_t (&off)[8]) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.b32 p, 0, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]),
      "r"(off[5]), "r"(off[6]), "r"(off[7])
      : "memory");
}

// The adapters of up to 32 Q sorted rows, lane i of word q holding row 32 q + i (-1: none), and
// the walk over the distinct ones: equal adapters are neighbours.
template <int Q>
struct Runs {
  int ad[Q];
  uint32_t heads[Q];
  // Every lane of the warp calls these.
  __device__ __forceinline__ void load(const int* row_adapter, int first, int rows) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < Q; ++q) ad[q] = 32 * q + lane < rows ? __ldcg(row_adapter + first + 32 * q + lane) : -1;
  }
  __device__ __forceinline__ void find() {
    const int lane = threadIdx.x & 31;
    int last = -1;  // of the rows before
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      int before = __shfl_up_sync(0xffffffffu, ad[q], 1);
      if (lane == 0) before = last;
      heads[q] = __ballot_sync(0xffffffffu, ad[q] >= 0 && ad[q] != before);
      last = __shfl_sync(0xffffffffu, ad[q], 31);
    }
  }
  __device__ __forceinline__ bool any() const {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) m |= heads[q];
    return m != 0;
  }
  // All adapters in order, into `list` (32 Q words of this warp's); returns how many.
  __device__ __forceinline__ int write(int* list) const {
    const int lane = threadIdx.x & 31;
    int total = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      if (heads[q] >> lane & 1) list[total + __popc(heads[q] & ((1u << lane) - 1))] = ad[q];
      total += __popc(heads[q]);
    }
    __syncwarp();
    return total;
  }
  // The next adapter, or -1; each call takes one off.
  __device__ __forceinline__ int next() {
    int l = -1;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int v = __shfl_sync(0xffffffffu, ad[q], __ffs(heads[q]) - 1 & 31);
      if (l < 0 && heads[q]) {
        l = v;
        heads[q] &= heads[q] - 1;
      }
    }
    return l;
  }
};

// How z enters a product on the tensor cores: as two 16-bit values, its first bits and the
// rounding of the remainder (off by 2^-17 of z at most in bf16; in fp16 by 2^-23 of it or, below about
// 1/4, by fp16's least half step, 2^-25), against the same U. A step
// takes up to 64 ranks of it: their high and their low parts side by side in one 64-wide tile of z
// up to 32 ranks, else in a tile each.
struct RankSteps {
  int r16, steps, tiles;  // tiles of z per step
  __device__ __forceinline__ explicit RankSteps(int r) {
    r16 = (r + 15) & ~15;
    steps = (r16 + 63) / 64;
    tiles = r16 <= 32 ? 1 : 2;
  }
  // MMAs of 16 ranks that walk the step's U once: for the high parts, and again for the low ones
  __device__ __forceinline__ int u_mmas(int step) const { return min(4, r16 / 16 - 4 * step); }
  // where the low parts start, as the descriptor of z counts, tiles `tile_bytes` apart
  __device__ __forceinline__ uint32_t low(int step, int tile_bytes) const {
    return tiles == 1 ? 2 * u_mmas(step) : tile_bytes >> 4;
  }
  // adapters whose U share a 64-rank wide stage
  __device__ __forceinline__ int together() const { return r16 <= 32 ? 64 / r16 : 1; }
};

// hi and lo of two ranks as the tensor cores take them, lo times `scale`. The remainder is exact: its
// rounding is the error. A value that is infinite, or becomes so in hi (in fp16 past 65504), has no
// remainder: what subtraction leaves, NaN or the opposite infinity, would make NaN of it.
template <typename T>
__device__ __forceinline__ void split2(float f0, float f1, uint32_t& hi, uint32_t& lo, float scale) {
  hi = Elem<T>::r2(f0, f1);
  const float2 b = Elem<T>::f2(hi);
  lo = Elem<T>::r2(isinf(b.x) ? 0.f : (f0 - b.x) * scale, isinf(b.y) ? 0.f : (f1 - b.y) * scale);
}
template <typename T>
__device__ __forceinline__ void split8(const float4& a, const float4& b, uint4& hi, uint4& lo, float scale = 1.f) {
  split2<T>(a.x, a.y, hi.x, lo.x, scale);
  split2<T>(a.z, a.w, hi.y, lo.y, scale);
  split2<T>(b.x, b.y, hi.z, lo.z, scale);
  split2<T>(b.z, b.w, hi.w, lo.w, scale);
}

// Row `i` of the step's z tile or two, `tile_bytes` apart (128-byte rows, 128-byte swizzle): this
// row's z, or zeros. The tiles serve every adapter of their rows: an adapter's MMAs write its own
// rows' lanes only.
template <typename T>
__device__ __forceinline__ void write_z_row(uint8_t* tile, int tile_bytes, int i, const float* zrow, bool mine, int r,
                                            const RankSteps& rs, int step) {
  uint8_t* row = tile + i * 128;
  const auto put = [&](uint8_t* at, int unit, const uint4& v) { *reinterpret_cast<uint4*>(at + ((unit ^ (i & 7)) << 4)) = v; };
  const int units = rs.u_mmas(step) * 2, first = 64 * step;
  for (int u = 0; u < units; ++u) {
    float4 f0 = {}, f1 = {};
    const int c = first + 8 * u;
    if (mine && c < r) {
      f0 = __ldcg(reinterpret_cast<const float4*>(zrow + c));
      f1 = __ldcg(reinterpret_cast<const float4*>(zrow + c + 4));
    }
    uint4 hi, lo;
    split8<T>(f0, f1, hi, lo);
    put(row, u, hi);
    if (rs.tiles == 1) put(row, units + u, lo);
    else put(row + tile_bytes, u, lo);
  }
}

}  // namespace moe_lora
