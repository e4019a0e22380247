// Products of a few rows with 4-bit weights under group scales (moe_w4_*):
//   out[i, n] = sum_groups s[n, grp] * sum_{c in grp} (q[n, c] - z[n, grp]) x[i, c]
// dense, or for every routed expert the rows that moe_lora_align gave it; the gated form
// applies a(gate) * up to the two halves of the rows.
//
// At a few rows the weights' stream bounds the product (half a byte per weight against 2 R
// operations), and next to it the instructions that turn codes into operands.
// * The packed form makes the stream plain: rows in tiles of 16, columns in chunks of 128, and
//   each (tile, chunk) of 1 KiB holds, lane by lane, the codes that the lane feeds to
//   mma.sync.m16n8k16. A warp copies them into its own ring in shared memory with cp.async, two
//   chunks ahead: no register holds what is in flight, and no CTA-wide wait is in the loop.
// * The weights take the MMA's M side, 8 rows of x its N side. Which columns share an MMA step
//   is free as long as both operands agree: lane t of a quad takes columns 8t .. 8t+7 of every
//   32, so that the four lanes of a step never straddle a group of 32 and x's fragment is one
//   16-byte read of its row, which a CTA keeps in shared memory for all of its tiles.
// * A weight enters as the exact q - z, in three instructions for a pair: a shift, one three-input
//   logic instruction that makes the code the mantissa's low bits of a power of two, and a packed
//   add (of -(128 + z) or the like) that takes the excess off again. (Leaving the excess in and
//   starting a group's accumulators at -(16 + z) times the sum of x over the group was no faster,
//   17.9 against 18.0 us for one row of 28672/4096 and 27.9 against 22.8 for sixteen; and its error
//   grew with columns of x that a weight of zero ignores, up to 17 % of an output for outliers of a
//   million, and an infinity met its negative.) In bf16 the operand is (q - z) / 2048, so that no
//   sum over a group overflows where x does not; it is taken back in fp32 at the end. A group's sum
//   is scaled in fp32.
// * A tile's chunks are shared out over as many warps of a CTA as it takes to fill the GPU;
//   their sums meet in shared memory in a fixed order.
// 28672/4096 (66 MB) with one row 17.7 us, 3.7 TB/s, eight rows 18.3, sixteen 22.8, thirty-two 42,
// sixty-four 81; 5760/2880 with one row 6.5 us; 4096/14336 with one row 11.8, eight 21.6, sixteen 33;
// 64 tokens to 4 of 32 experts of 5760/2880 (300 MB) 81 to 83. The loop's instructions (38 per 512
// weights, everything counted, at six rows) bound it at four warps per scheduler, which use 45 to 62 %
// of the issue slots; eight warps with half the registers were slower. Loads alone run at 7.7 TB/s.
#include <algorithm>

#include "activation.cuh"
#include "internal.h"

namespace moe_lora {

constexpr int kTileRows = 16, kChunkCols = 128;
constexpr int kTileBytes = kTileRows * kChunkCols / 2;
constexpr int kW4Warps = 16;

// The columns that the product takes: rows of x are read by 16 bytes, and one has to fit into
// shared memory beside the ring. Packing other weights would lead nowhere.
constexpr int kW4MostK = 16384;
static bool w4_columns_ok(int K) { return K % 8 == 0 && K <= kW4MostK; }

// The packed form: codes, then scales, then zeros, each [E][tiles][chunks] of its block.
struct W4Layout {
  int half_rows;   // rows of a half (N unless gated)
  int half_tiles;  // tiles of a half
  int tiles;       // per expert
  int chunks;
  int gpc;         // groups per chunk
  int zero_bytes;  // per (tile, chunk) and row pair g, g + 8: 4 at least, a copy's smallest
  int64_t off_scales, off_zeros, bytes;
  bool valid;
};

static W4Layout w4_layout(int E, int N, int K, int group, int has_zeros, int gated) {
  W4Layout w = {};
  if (E < 1 || N < 1 || K < 1 || (group != 32 && group != 64 && group != 128) ||
      (gated && N % 2 != 0) || N > (1 << 24) || K > (1 << 24) || E > (1 << 20))
    return w;
  w.half_rows = gated ? N / 2 : N;
  w.half_tiles = ceil_div(w.half_rows, kTileRows);
  w.tiles = w.half_tiles * (gated ? 2 : 1);
  w.chunks = ceil_div(K, kChunkCols);
  w.gpc = kChunkCols / group;
  const int64_t blocks = (int64_t)E * w.tiles * w.chunks;
  if (blocks >= ((int64_t)1 << 31)) return w;
  w.off_scales = blocks * kTileBytes;
  w.off_zeros = w.off_scales + blocks * w.gpc * kTileRows * 2;
  w.zero_bytes = std::max(4, 2 * w.gpc);
  w.bytes = w.off_zeros + (has_zeros ? blocks * 8 * w.zero_bytes : 0);
  w.bytes = (int64_t)round_up((size_t)w.bytes, 16);
  w.valid = true;
  return w;
}

// ----------------------------------------------------------------------------
// quantise: one warp per group
// ----------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const T* __restrict__ W, int64_t rows, int K,
                                                          int group, int groups,
                                                          uint8_t* __restrict__ codes,
                                                          T* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t stride = (int64_t)gridDim.x * 8;
  const int kb = (K + 1) / 2;
  for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; i < rows * groups; i += stride) {
    const int64_t row = i / groups;
    const int c0 = (int)(i - row * groups) * group;
    float v[4];  // columns 2 lane, 2 lane + 1 of the group's first 64, and of its last
    float big = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int o = 2 * lane + (q & 1) + 64 * (q >> 1);
      v[q] = o < group && c0 + o < K ? Elem<T>::f(W[row * K + c0 + o]) : 0.f;
      big = fmaxf(big, fabsf(v[q]));
    }
    for (int off = 16; off > 0; off /= 2) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
    const T s = Elem<T>::r(__fdiv_rn(big, 7.f));
    const float sf = Elem<T>::f(s);
    if (lane == 0) scales[i] = s;
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const int o = 2 * lane + 32 * q;
      if (o >= group || c0 + o >= K) continue;
      int b = 0;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float z = sf > 0.f ? rintf(__fdiv_rn(v[q + p], sf)) : 0.f;
        z = fminf(fmaxf(z, -7.f), 7.f);
        b |= (int)(z + 8.f) << (4 * p);
      }
      codes[row * kb + (c0 + o) / 2] = (uint8_t)b;
    }
  }
}

// ----------------------------------------------------------------------------
// pack: one CTA per (tile, chunk), one thread per 32-bit word of codes and per scale
// ----------------------------------------------------------------------------
struct TileRows {
  int row0, rows;  // rows [row0, row0 + rows) of the expert's matrix
};
__device__ __forceinline__ TileRows tile_rows(int tile, int half_tiles, int half_rows) {
  const bool up = tile >= half_tiles;
  const int r = (up ? tile - half_tiles : tile) * kTileRows;
  TileRows t;
  t.row0 = (up ? half_rows : 0) + r;
  t.rows = min(half_rows - r, kTileRows);
  return t;
}

__global__ void __launch_bounds__(256) w4_pack_kernel(const uint8_t* __restrict__ codes,
                                                      const uint16_t* __restrict__ scales,
                                                      const uint8_t* __restrict__ zeros, int N, int K,
                                                      int groups, W4Layout w, int64_t blocks,
                                                      char* __restrict__ packed) {
  const int kb = (K + 1) / 2;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t et = b / w.chunks;
    const int chunk = (int)(b - et * w.chunks);
    const int64_t e = et / w.tiles;
    const TileRows tr = tile_rows((int)(et - e * w.tiles), w.half_tiles, w.half_rows);
    {  // thread = (row g or g + 8, lane, 32-column part j)
      const int i = threadIdx.x;
      const int j = i & 3, lane = (i >> 2) & 31, row = (lane >> 2) + 8 * (i >> 7);
      const int col = chunk * kChunkCols + j * 32 + (lane & 3) * 8;
      uint32_t word = 0;
      if (row < tr.rows) {
        const uint8_t* p = codes + (e * N + tr.row0 + row) * kb + col / 2;
        for (int q = 0; q < 8; ++q) {
          if (col + q >= K) break;
          const uint32_t c = (p[q / 2] >> (4 * (q & 1))) & 15u;
          word |= c << (4 * (q >> 1) + 16 * (q & 1));
        }
      }
      reinterpret_cast<uint32_t*>(packed + b * kTileBytes)[i] = word;
    }
    if (threadIdx.x < 16 * w.gpc) {  // [g][group of the chunk][row g, row g + 8]
      const int i = threadIdx.x;
      const int row = (i / (2 * w.gpc)) + 8 * (i & 1), grp = chunk * w.gpc + (i >> 1) % w.gpc;
      const bool in = row < tr.rows && grp < groups;
      const int64_t at = (e * N + tr.row0 + row) * groups + grp;
      reinterpret_cast<uint16_t*>(packed + w.off_scales)[b * 16 * w.gpc + i] = in ? scales[at] : 0;
      if (zeros)
        packed[w.off_zeros + (b * 8 + i / (2 * w.gpc)) * w.zero_bytes + i % (2 * w.gpc)] =
            (char)(in ? zeros[at] & 15 : 0);
    }
  }
}

// ----------------------------------------------------------------------------
// the product
// ----------------------------------------------------------------------------
// (v & mask) | base in one instruction. (Left to the compiler it was often two: 7.0 against 6.4 us
// for one row of 5760/2880.)
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t base) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(base));
  return r;
}

// What makes operands of codes. A word holds pair i of a row's codes in bits 4i .. 4i + 3 of its
// halves. For a row's zero point z (twice: z + (z << 16)): its constants, and the pairs' q - z times
// 1 / kUnit, exactly.
template <typename T> struct Codes;
template <> struct Codes<__nv_bfloat16> {
  static constexpr float kUnit = 2048.f;
  struct Zero {
    uint32_t c;  // -(128 + z) / 2048 twice
  };
  static __device__ __forceinline__ Zero zero(uint32_t zz) { return {zz | 0xBD80BD80u}; }
  static __device__ __forceinline__ void values(uint32_t w, const Zero& z, uint32_t (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 128 + q, then (128 + q) / 2048 - (128 + z) / 2048
      const uint32_t e = and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u);
      asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(v[i]) : "r"(e), "r"(0x3A003A00u), "r"(z.c));
    }
  }
};
template <> struct Codes<__half> {
  static constexpr float kUnit = 1.f;
  struct Zero {
    uint32_t lo, hi;  // -(1024 + z) and -(64 + z), each twice
  };
  static __device__ __forceinline__ Zero zero(uint32_t zz) { return {zz | 0xE400E400u, (zz << 4) | 0xD400D400u}; }
  static __device__ __forceinline__ void values(uint32_t w, const Zero& z, uint32_t (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // two pairs per shift: 1024 + q, and 64 + q from the next four bits
      const uint32_t u = w >> (8 * (i / 2));
      const uint32_t e = i % 2 == 0 ? and_or(u, 0x000F000Fu, 0x64006400u) : and_or(u, 0x00F000F0u, 0x54005400u);
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(e), "r"(i % 2 == 0 ? z.lo : z.hi));
    }
  }
};

__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
// kWords words of a row pair, at a multiple of their size.
template <int kWords>
__device__ __forceinline__ uint4 lds_words(uint32_t a) {
  if (kWords == 4) return lds128(a);
  if (kWords == 1) return make_uint4(lds32(a), 0, 0, 0);
  const uint2 v = lds64(a);
  return make_uint4(v.x, v.y, 0, 0);
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// One (tile, chunk) in the ring, as it is packed: 1 KiB of codes, then the scales (4 GPC bytes
// per row pair g, g + 8) and the zeros (8 bytes, or 4).
template <int GPC, bool kZeros>
struct W4Slot {
  static constexpr int kScales = 32 * GPC, kZerosAt = kTileBytes + kScales, kZ = GPC == 4 ? 64 : 32;
  static constexpr int kBytes = kZerosAt + (kZeros ? kZ : 0);
};
constexpr int kRingDepth = 2;  // chunks in a warp's ring: 16 warps have 18 to 39 KB in flight

struct W4Args {
  const void* x;
  const char* packed;
  W4Layout w;
  int N, K, R, act, out_fp32;
  int k, rows_sorted, zero_dropped, E;
  int share;           // warps per tile: 1, 2, 4, 8 or 16
  int stage_rows;      // rows of x that the shared memory holds
  int stage_stride;    // bytes from one to the next
  const int* expert_begin;  // null: one expert, R rows
  const int* sorted_slots;
  void* out;
};

// Where the experts' rows begin: in shared memory up to kListed experts.
constexpr int kListed = 1024;
struct ExpertList {
  const int* listed;  // null: too many
  const int* begin;
  __device__ __forceinline__ int at(int e) const { return listed ? listed[e] : __ldcg(begin + e); }
};

template <typename T, int GPC, bool kZeros, bool kPair>
struct W4Kernel {
  static constexpr int kTiles = kPair ? 2 : 1;
  static constexpr int kStepBytes = kTiles * W4Slot<GPC, kZeros>::kBytes;
  static constexpr int kPartPerGroup = 4 / GPC;  // 32-column parts per group
  using Slot = W4Slot<GPC, kZeros>;
  static constexpr int kRingBytes = kW4Warps * kRingDepth * kStepBytes;
  static constexpr int kRedBytes = kW4Warps * kTiles * 128 * 4;  // 16 x 8 sums of every warp

  // One pass: up to NT x 8 rows [r0, re) of expert e against tiles [tile0, tile1).
  template <int NT>
  static __device__ __forceinline__ void pass(const W4Args& p, char* smem, int e, int r0, int re, int tile0,
                                              int tile1) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int slots = kW4Warps / p.share;  // tiles at a time
    const int mine = warp / p.share, part = warp - mine * p.share;
    const int per = (p.w.chunks + p.share - 1) / p.share;
    const int first_c = part * per, n = max(0, min(p.w.chunks, first_c + per) - first_c);  // chunks of this warp
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kRingDepth * kStepBytes);
    float* red = reinterpret_cast<float*>(smem + kRingBytes);
    // Requests run two chunks ahead, through the tiles of this warp.
    // Lanes take 16 bytes of the scales (and of the zeros behind them) as far as those go.
    constexpr int kS = Slot::kScales, kZ = Slot::kZ;
    const char* const codes = p.packed + lane * 16;
    const bool meta = lane < (kS + (kZeros ? kZ : 0)) / 16;
    const bool zero_lane = lane >= kS / 16;
    const char* const metas = p.packed + (zero_lane ? p.w.off_zeros + (lane - kS / 16) * 16 : p.w.off_scales + lane * 16);
    const uint32_t meta_step = zero_lane ? kZ : kS;
    const uint32_t up = (uint32_t)p.w.half_tiles * p.w.chunks;  // blocks from a gate tile to its up tile
    const uint32_t next = (uint32_t)slots * p.w.chunks - n;
    uint32_t qb = ((uint32_t)e * p.w.tiles + tile0 + mine) * p.w.chunks + first_c;  // below 2^31 in all
    int left = n > 0 && tile0 + mine < tile1 ? ((tile1 - 1 - tile0 - mine) / slots + 1) * n : 0;
    int qc = n;
    auto request = [&](uint32_t slot) {
      if (left > 0) {
        --left;
#pragma unroll
        for (int tl = 0; tl < kTiles; ++tl) {
          const uint32_t dst = slot + (uint32_t)(tl * Slot::kBytes) + lane * 16;
          const uint32_t b = qb + (tl ? up : 0);
          const char* code = codes + (uint64_t)b * kTileBytes;
          copy_async16(dst, code);
          copy_async16(dst + 512, code + 512);
          if (meta) copy_async16(dst + 1024, metas + (uint64_t)b * meta_step);
        }
        ++qb;
        if (--qc == 0) {
          qc = n;
          qb += next;
        }
      }
      copy_commit();
    };
    request(ring);
    request(ring + kStepBytes);
    __syncthreads();        // the rows of the pass before are done with
    stage(p, smem + kRingBytes + kRedBytes, r0, re);
    __syncthreads();
    // x: this lane's columns of its row of each 8 (rows past the last repeat it, unused)
    uint32_t xr[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      xr[nt] = smem_u32(smem) + kRingBytes + kRedBytes + (uint32_t)(min(nt * 8 + g, re - r0 - 1) * p.stage_stride) +
               (uint32_t)(first_c * kChunkCols + t * 8) * 2;
    uint32_t rs = ring;
    for (int tb = tile0; tb < tile1; tb += slots) {
      const int tile = tb + mine;
      float tot[kTiles][NT][4] = {};
      if (tile < tile1) {
        for (int c = 0; c < n; ++c) {
          copy_wait<kRingDepth - 1>();
          __syncwarp();  // the scales came in by other lanes
          uint4 lo[kTiles], hi[kTiles], sc[kTiles], zr[kTiles];
#pragma unroll
          for (int tl = 0; tl < kTiles; ++tl) {
            const uint32_t at = rs + tl * Slot::kBytes;
            lo[tl] = lds128(at + lane * 16);
            hi[tl] = lds128(at + lane * 16 + 512);
            sc[tl] = lds_words<GPC>(at + kTileBytes + g * (4 * GPC));
            if (kZeros) zr[tl] = lds_words<GPC == 4 ? 2 : 1>(at + Slot::kZerosAt + g * (kZ / 8));
          }
          float acc[kTiles][NT][4];
          typename Codes<T>::Zero zl[kTiles], zh[kTiles];  // of the two rows, for a group
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int grp = j / kPartPerGroup;
            uint4 xv[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) xv[nt] = lds128(xr[nt] + (uint32_t)(c * kChunkCols * 2) + j * 64);
#pragma unroll
            for (int tl = 0; tl < kTiles; ++tl) {
              if (j % kPartPerGroup == 0) {
                // byte 2 grp of the row pair's zeros, and the next
                const uint32_t zw = kZeros ? word(zr[tl], grp >> 1) : 0u;
                const uint32_t by = 2 * (grp & 1);
                zl[tl] = Codes<T>::zero(kZeros ? __byte_perm(zw, 0, 0x4040u + by * 0x0101u) : 0x00080008u);
                zh[tl] = Codes<T>::zero(kZeros ? __byte_perm(zw, 0, 0x4141u + by * 0x0101u) : 0x00080008u);
              }
              uint32_t al[4], ah[4];
              Codes<T>::values(word(lo[tl], j), zl[tl], al);
              Codes<T>::values(word(hi[tl], j), zh[tl], ah);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float(&d)[4] = acc[tl][nt];
                if (j % kPartPerGroup == 0)
                  mma16816_from<T>(d, al[0], ah[0], al[1], ah[1], xv[nt].x, xv[nt].y, 0.f, 0.f, 0.f, 0.f);
                else
                  mma16816<T>(d, al[0], ah[0], al[1], ah[1], xv[nt].x, xv[nt].y);
                mma16816<T>(d, al[2], ah[2], al[3], ah[3], xv[nt].z, xv[nt].w);
              }
              if (j % kPartPerGroup == kPartPerGroup - 1) {
                const float2 sv = Elem<T>::f2(word(sc[tl], grp));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  tot[tl][nt][0] += sv.x * acc[tl][nt][0];
                  tot[tl][nt][1] += sv.x * acc[tl][nt][1];
                  tot[tl][nt][2] += sv.y * acc[tl][nt][2];
                  tot[tl][nt][3] += sv.y * acc[tl][nt][3];
                }
              }
            }
          }
          __syncwarp();
          request(rs);  // into the place whose contents every lane has used
          rs ^= ring ^ (ring + kStepBytes);
        }
      }
      const TileRows tr = tile_rows(min(tile, tile1 - 1), p.w.half_tiles, p.w.half_rows);
      if (p.share == 1) {
        if (tile < tile1)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              put(p, tr, g + 8 * (q >> 1), r0 + nt * 8 + 2 * t + (q & 1), re, tot[0][nt][q], tot[kTiles - 1][nt][q]);
        continue;
      }
      // the shares of each tile, 8 rows of x at a time
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        __syncthreads();
#pragma unroll
        for (int tl = 0; tl < kTiles; ++tl)
#pragma unroll
          for (int q = 0; q < 4; ++q) red[(warp * kTiles + tl) * 128 + q * 32 + lane] = tot[tl][nt][q];
        __syncthreads();
        for (int i = threadIdx.x; i < slots * 128; i += kW4Warps * 32) {
          const int slot = i >> 7, at = i & 127, ln = at & 31, q = at >> 5;
          if (tb + slot >= tile1) break;
          float v = 0.f, u = 0.f;
          for (int k = 0; k < p.share; ++k) {
            v += red[(slot * p.share + k) * kTiles * 128 + at];
            if (kPair) u += red[((slot * p.share + k) * kTiles + kTiles - 1) * 128 + at];
          }
          put(p, tile_rows(tb + slot, p.w.half_tiles, p.w.half_rows), (ln >> 2) + 8 * (q >> 1),
              r0 + nt * 8 + 2 * (ln & 3) + (q & 1), re, v, u);
        }
      }
    }
    copy_wait<0>();
  }

  static __device__ __forceinline__ void put(const W4Args& p, const TileRows& tr, int row, int r, int re, float v,
                                             float u) {
    if (row >= tr.rows || r >= re) return;
    v *= Codes<T>::kUnit;
    u *= Codes<T>::kUnit;
    const int n = tr.row0 + row;
    if (kPair) {
      float a, d;
      if (p.act == MOE_ACT_SILU) activation<MOE_ACT_SILU>(v, a, d);
      else activation<MOE_ACT_GELU>(v, a, d);
      static_cast<T*>(p.out)[(int64_t)r * (p.N / 2) + n] = Elem<T>::r(a * u);
    } else if (p.out_fp32) {
      static_cast<float*>(p.out)[(int64_t)r * p.N + n] = v;
    } else {
      static_cast<T*>(p.out)[(int64_t)r * p.N + n] = Elem<T>::r(v);
    }
  }

  // Rows [r0, r1) of x in shared memory, zero past K to the end of the last chunk.
  static __device__ __forceinline__ void stage(const W4Args& p, char* xs, int r0, int r1) {
    const int cols8 = p.w.chunks * (kChunkCols / 8), k8 = p.K / 8;
    // the source of row r0 + i in lane i: one look-up for all of them (32 at most)
    int from = min(r0 + (int)(threadIdx.x & 31), r1 - 1);
    if (p.expert_begin && !p.rows_sorted) from = __ldcg(p.sorted_slots + from) / p.k;
    for (int rb = r0; rb < r1; rb += 8) {  // eight rows' loads in flight
      const uint4* src[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        src[q] = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) +
                                                (int64_t)__shfl_sync(0xffffffffu, from, rb - r0 + q) * p.K);
      for (int c = threadIdx.x; c < cols8; c += kW4Warps * 32) {
        uint4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          v[q] = make_uint4(0, 0, 0, 0);
          if (c < k8 && rb + q < r1) v[q] = __ldcg(src[q] + c);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (rb + q >= r1) break;
          const int r = rb - r0 + q;
          *reinterpret_cast<uint4*>(xs + r * p.stage_stride + c * 16) = v[q];
        }
      }
    }
  }
};

// What a pass costs per tile by its rows: at 28672/4096 8, 16 and 32 rows take 18, 23 and 42 us,
// both halves of the gated form 18 and 23 (of either some 4 us are the launch's).
template <bool kPair>
__device__ __forceinline__ int pass_cost(int rows) {
  return rows <= 0 ? 0 : rows <= 8 ? 10 : kPair ? 14 : rows <= 16 ? 13 : 23;
}

// The tiles of all experts with rows, an expert's tiles weighted by its rows' passes, are shared
// evenly between the CTAs, in order. (With the same number of tiles each, the CTAs of the experts
// with many rows were the last: 227 against 110 us where 8 of 32 experts of 5760/2880 get most of
// 64 tokens' rows. Passes are counted as long as they are: counted as the longest that there are,
// though long rows of x leave room for fewer, 64 tokens to 2 of 16 experts of 4096/14336 took 274
// against 219 us.) kRows8: passes of at most 8 rows; else of up to 32 (16 of the gated form).
template <typename T, int GPC, bool kZeros, bool kPair, bool kRows8>
__global__ void __launch_bounds__(kW4Warps * 32, 1) w4_matvec_kernel(const W4Args p) {
  using Kern = W4Kernel<T, GPC, kZeros, kPair>;
  extern __shared__ __align__(16) char smem[];
  const int jobs = kPair ? p.w.half_tiles : p.w.tiles;
  const int unit = kW4Warps / p.share;  // tiles that the CTA works on together
  const int units = (jobs + unit - 1) / unit;  // per expert
  constexpr int kMost = kRows8 ? 8 : kPair ? 16 : 32;
  const int most = min(p.stage_rows, kMost);
  const bool routed = p.expert_begin;
  __shared__ int listed[kListed + 1];
  const ExpertList list = {p.E <= kListed ? listed : nullptr, p.expert_begin};
  const int lane = threadIdx.x & 31;
  auto weight = [&](int e) {
    const int n = e < p.E ? max(0, list.at(e + 1) - list.at(e)) : 0;
    const unsigned whole = (unsigned)n / (unsigned)most;
    return (int)whole * pass_cost<kPair>(most) + pass_cost<kPair>(n - (int)whole * most);
  };
  // the weights are a line of length `all`, [lo, hi) this CTA's part of it
  float lo = 0.f, hi = 0.f;
  // Nothing is read before every earlier launch is over, the weights neither: one may be writing
  // them still. (Pulling 2 to 32 chunks a warp into L2 meanwhile did not pay: 17.0 against 17.0 us
  // at 28672/4096 with 2, 18.0 from 8 on.)
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  if (routed) {
    if (p.E <= kListed) {
      for (int e = threadIdx.x; e <= p.E; e += kW4Warps * 32) listed[e] = __ldcg(p.expert_begin + e);
      __syncthreads();
    }
    int all = 0;
    for (int base = 0; base < p.E; base += 32) all += __reduce_add_sync(0xffffffffu, weight(base + lane));
    const float each = (float)all / (float)gridDim.x;
    lo = blockIdx.x == 0 ? -1.f : __fmul_rn(each, (float)blockIdx.x);
    hi = blockIdx.x == gridDim.x - 1 ? __int_as_float(0x7f800000) : __fmul_rn(each, (float)(blockIdx.x + 1));
  }
  int at = 0;  // the weights of the experts before e
  for (int e = 0;; ++e) {
    int rb = 0, re = p.R, u0, u1;
    if (!routed) {
      const unsigned n = (unsigned)units / gridDim.x, more = units - n * gridDim.x;
      u0 = (int)(blockIdx.x * n + min(blockIdx.x, more));
      u1 = u0 + (int)n + (blockIdx.x < more ? 1 : 0);
    } else {
      bool found = false;
      while (!found && e < p.E && (float)at < hi) {  // 32 experts at a time
        const int w = weight(e + lane);
        int end = w;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int v = __shfl_up_sync(0xffffffffu, end, o);
          if (lane >= o) end += v;
        }
        end += at;
        // an expert's units whose middles are before a place on the line: the CTAs on both its
        // sides agree on it
        const float per = __fdividef((float)units, (float)max(w, 1));
        auto before = [&](float x) {
          const float u = __fmul_rn(__fsub_rn(x, (float)(end - w)), per);
          return (int)ceilf(fminf(fmaxf(u, 0.f), (float)units) - 0.5f);
        };
        const int v0 = before(lo), v1 = w > 0 ? before(hi) : 0;
        const unsigned m = __ballot_sync(0xffffffffu, v0 < v1);
        const int src = m ? __ffs(m) - 1 : 31;
        found = m != 0;
        at = __shfl_sync(0xffffffffu, end, src);
        u0 = __shfl_sync(0xffffffffu, v0, src);
        u1 = __shfl_sync(0xffffffffu, v1, src);
        e += found ? src : 32;
      }
      if (!found) break;
      rb = list.at(e);
      re = list.at(e + 1);
    }
    const int t0 = u0 * unit, t1 = min(jobs, u1 * unit);
    for (int r0 = rb; r0 < re; r0 += most) {
      const int r1 = min(re, r0 + most), n = r1 - r0;
      // (32 rows of both halves of the gated form do not fit the registers)
      if (kRows8 || n <= 8) Kern::template pass<1>(p, smem, e, r0, r1, t0, t1);
      else if (kPair || n <= 16) Kern::template pass<kRows8 ? 1 : 2>(p, smem, e, r0, r1, t0, t1);
      else Kern::template pass<kRows8 ? 1 : kPair ? 2 : 4>(p, smem, e, r0, r1, t0, t1);
    }
    if (!routed) break;
  }
  if (p.zero_dropped) {  // the rows behind the last expert's
    const int n = kPair ? p.N / 2 : p.N;
    for (int64_t r = list.at(p.E) + (int)blockIdx.x; r < (int64_t)p.R * p.k; r += gridDim.x)
      for (int i = threadIdx.x; i < n; i += kW4Warps * 32) {
        if (p.out_fp32) static_cast<float*>(p.out)[r * n + i] = 0.f;
        else static_cast<uint16_t*>(p.out)[r * n + i] = 0;
      }
  }
}

template <typename T, int GPC, bool kZeros, bool kPair, bool kRows8>
static int launch_w4_k(W4Args& a, int rows, cudaStream_t stream) {
  using Kern = W4Kernel<T, GPC, kZeros, kPair>;
  auto kernel = w4_matvec_kernel<T, GPC, kZeros, kPair, kRows8>;
  constexpr int kMost = 222 * 1024;  // with the experts' list below 227 KB
  static std::atomic<uint64_t> seen[kMaxDevices];
  int st = once_per_context(seen, [&] {
    ML_CHECK_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost));
    return MOE_LORA_OK;
  });
  if (st != MOE_LORA_OK) return st;
  // x in shared memory: rows 64 bytes apart modulo 128, so that the two rows of a quarter-warp's
  // read take different banks
  a.stage_stride = a.w.chunks * kChunkCols * 2 + 64;
  auto bytes = [&](int r) { return Kern::kRingBytes + Kern::kRedBytes + r * a.stage_stride; };
  int most = a.expert_begin ? (kRows8 ? 8 : 32) : std::min(rows, kRows8 ? 8 : 32);
  if (bytes(most) > kMost && most > 16) most = 16;
  if (bytes(most) > kMost && most > 8) most = 8;
  while (most > 0 && bytes(most) > kMost) --most;
  if (most < 1) return MOE_LORA_ERR_UNSUPPORTED;
  a.stage_rows = most;
  const int smem = bytes(most);
  // Warps per tile: the fewest rounds of chunks on the busiest SM, where a round costs as much
  // as half a chunk more.
  const int64_t jobs = kPair ? a.w.half_tiles : a.w.tiles;
  const int experts = a.expert_begin ? (int)std::min<int64_t>(a.E, (int64_t)a.R * a.k) : 1;
  const int64_t ctas = num_sms();
  int64_t best = -1, groups = 0;
  for (int share = 1; share <= kW4Warps; share *= 2) {
    const int64_t n = experts * ceil_div64(jobs, kW4Warps / share);
    const int64_t cost = ceil_div64(n, ctas) * (ceil_div(a.w.chunks, share) * 2 + 1);
    if (best < 0 || cost < best) {
      best = cost;
      groups = n;
      a.share = share;
    }
  }
  return launch_pdl(kernel, (unsigned)std::min(groups, ctas), kW4Warps * 32, smem, stream, true, a);
}
template <typename T, int GPC, bool kZeros>
static int launch_w4_p(W4Args& a, int rows, cudaStream_t stream) {
  if (a.act != MOE_ACT_NONE)
    return rows <= 8 ? launch_w4_k<T, GPC, kZeros, true, true>(a, rows, stream)
                     : launch_w4_k<T, GPC, kZeros, true, false>(a, rows, stream);
  return rows <= 8 ? launch_w4_k<T, GPC, kZeros, false, true>(a, rows, stream)
                   : launch_w4_k<T, GPC, kZeros, false, false>(a, rows, stream);
}
template <typename T>
static int launch_w4(W4Args& a, bool zeros, int rows, cudaStream_t stream) {
  switch (a.w.gpc * 2 + (zeros ? 1 : 0)) {
    case 2: return launch_w4_p<T, 1, false>(a, rows, stream);
    case 3: return launch_w4_p<T, 1, true>(a, rows, stream);
    case 4: return launch_w4_p<T, 2, false>(a, rows, stream);
    case 5: return launch_w4_p<T, 2, true>(a, rows, stream);
    case 8: return launch_w4_p<T, 4, false>(a, rows, stream);
    default: return launch_w4_p<T, 4, true>(a, rows, stream);
  }
}

}  // namespace moe_lora

extern "C" int moe_w4_quantize(const void* W, int dtype, int E, int N, int K, int group, uint8_t* codes,
                               void* scales, moe_lora_stream_t stream) {
  using namespace moe_lora;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_LORA_ERR_INVALID_ARG;
  if (!w4_layout(E, N, K, group, 0, 0).valid) return MOE_LORA_ERR_UNSUPPORTED;
  if (!W || !codes || !scales) return MOE_LORA_ERR_INVALID_ARG;
  int st = check_device();
  if (st != MOE_LORA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t rows = (int64_t)E * N;
  const int groups = ceil_div(K, group);
  const unsigned ctas = (unsigned)std::min<int64_t>(ceil_div64(rows * groups, 8), 152 * 16);
  if (dtype == MOE_DTYPE_BF16)
    return launch_pdl(w4_quantize_kernel<__nv_bfloat16>, ctas, 256, 0, s, false,
                      static_cast<const __nv_bfloat16*>(W), rows, K, group, groups, codes,
                      static_cast<__nv_bfloat16*>(scales));
  return launch_pdl(w4_quantize_kernel<__half>, ctas, 256, 0, s, false, static_cast<const __half*>(W), rows, K,
                    group, groups, codes, static_cast<__half*>(scales));
}

extern "C" size_t moe_w4_packed_size(int E, int N, int K, int group, int has_zeros, int gated) {
  using namespace moe_lora;
  const W4Layout w = w4_layout(E, N, K, group, has_zeros, gated);
  return w.valid ? (size_t)w.bytes : 0;
}

extern "C" int moe_w4_pack(const uint8_t* codes, const void* scales, const uint8_t* zeros, int E, int N, int K,
                           int group, int gated, void* packed, moe_lora_stream_t stream) {
  using namespace moe_lora;
  const W4Layout w = w4_layout(E, N, K, group, zeros != nullptr, gated);
  if (!w.valid || !w4_columns_ok(K)) return MOE_LORA_ERR_UNSUPPORTED;
  if (!codes || !scales || !packed || !aligned16(packed)) return MOE_LORA_ERR_INVALID_ARG;
  int st = check_device();
  if (st != MOE_LORA_OK) return st;
  const int64_t blocks = (int64_t)E * w.tiles * w.chunks;
  return launch_pdl(w4_pack_kernel, (unsigned)std::min<int64_t>(blocks, 152 * 16), 256, 0,
                    reinterpret_cast<cudaStream_t>(stream), false, codes, static_cast<const uint16_t*>(scales),
                    zeros, N, K, ceil_div(K, group), w, blocks, static_cast<char*>(packed));
}

extern "C" int moe_w4_matvec(const void* x, int dtype, const void* packed, int E, int N, int K, int group,
                             int has_zeros, int gated, int act, int T, const moe_lora_align_t* al, int row_flags,
                             void* out, int out_fp32, moe_lora_stream_t stream) {
  using namespace moe_lora;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_LORA_ERR_INVALID_ARG;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SILU && act != MOE_ACT_GELU) return MOE_LORA_ERR_INVALID_ARG;
  if (act != MOE_ACT_NONE && (!gated || out_fp32)) return MOE_LORA_ERR_INVALID_ARG;
  if (T < 0 || T > (1 << 22) || (row_flags & ~(MOE_W4_ROWS_SORTED | MOE_W4_ZERO_DROPPED))) return MOE_LORA_ERR_INVALID_ARG;
  W4Args a = {};
  a.w = w4_layout(E, N, K, group, has_zeros, gated);
  if (!a.w.valid || !w4_columns_ok(K)) return MOE_LORA_ERR_UNSUPPORTED;
  int rows = T, st;
  if (al) {
    AlignLayout lay;
    if ((st = check_align(al, &lay)) != MOE_LORA_OK) return st;
    if (al->E != E || al->T != T) return MOE_LORA_ERR_INVALID_ARG;
    const AlignView v = align_view(al->buf, lay);
    a.expert_begin = v.expert_begin;
    a.sorted_slots = v.sorted_slots;
    a.k = al->k;
    a.rows_sorted = row_flags & MOE_W4_ROWS_SORTED;
    a.zero_dropped = row_flags & MOE_W4_ZERO_DROPPED;
    // an expert's rows, as far as the shared memory is planned: twice the mean at most
    rows = (int)std::min<int64_t>(T, 2 * ceil_div64(lay.S, E));
  } else if (E != 1) {
    return MOE_LORA_ERR_INVALID_ARG;
  }
  if (T == 0) return MOE_LORA_OK;
  if (!x || !packed || !out || !aligned16(x) || !aligned16(packed)) return MOE_LORA_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(out) & (out_fp32 ? 3 : 1)) return MOE_LORA_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  a.x = x;
  a.packed = static_cast<const char*>(packed);
  a.N = N;
  a.K = K;
  a.R = T;
  a.E = E;
  a.act = act;
  a.out_fp32 = out_fp32;
  a.out = out;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == MOE_DTYPE_BF16 ? launch_w4<__nv_bfloat16>(a, has_zeros != 0, rows, s)
                                 : launch_w4<__half>(a, has_zeros != 0, rows, s);
}
