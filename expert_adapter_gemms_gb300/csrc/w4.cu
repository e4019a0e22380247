// Products of a few rows with 4-bit weights under group scales (moe_w4_*):
//   out[i, n] = sum_groups s[n, grp] * sum_{c in grp} (q[n, c] - z[n, grp]) x[i, c]
// dense, or for every routed expert the rows that moe_lora_align gave it; the gated form
// applies a(gate) * up to the two halves of the rows.
//
// At a few rows the weights' stream bounds the product (half a byte per weight against 2 R
// operations). The packed form makes that stream plain: rows in tiles of 16, columns in
// chunks of 128, and each (tile, chunk) of 1 KiB holds, lane by lane, the codes that the
// lane feeds to mma.sync.m16n8k16 -- 16-byte loads, 512 contiguous bytes per warp, no shared
// memory. The weights take the MMA's M side, up to 8 rows of x its N side. Which columns
// share an MMA step is free as long as both operands agree: lane t of a quad takes columns
// 8t .. 8t+7 of every 32, so that the four lanes of a step never straddle a group of 32 and
// x's fragment is one 16-byte load of its row.
// A code enters exactly: OR-ed into the mantissa of 128 (bf16) or 1024 (fp16) it is 128 + q,
// less 128 + z it is q - z, with no rounding; products are summed in fp32 over a group, and
// the group's sum is scaled in fp32.
// The warps of a CTA share out the chunks and add up through shared memory in a fixed order.
#include <algorithm>

#include "activation.cuh"
#include "internal.h"

namespace moe_lora {

constexpr int kTileRows = 16, kChunkCols = 128;
constexpr int kTileBytes = kTileRows * kChunkCols / 2;
constexpr int kW4Warps = 8;

// The packed form: codes, then scales, then zeros, each [E][tiles][chunks] of its block.
struct W4Layout {
  int half_rows;   // rows of a half (N unless gated)
  int half_tiles;  // tiles of a half
  int tiles;       // per expert
  int chunks;
  int gpc;         // groups per chunk
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
  if (blocks > ((int64_t)1 << 40)) return w;
  w.off_scales = blocks * kTileBytes;
  w.off_zeros = w.off_scales + blocks * w.gpc * kTileRows * 2;
  w.bytes = w.off_zeros + (has_zeros ? blocks * w.gpc * kTileRows : 0);
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
  const int half = tile / half_tiles, r = (tile - half * half_tiles) * kTileRows;
  TileRows t;
  t.row0 = half * half_rows + r;
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
        reinterpret_cast<uint8_t*>(packed + w.off_zeros)[b * 16 * w.gpc + i] = in ? zeros[at] & 15 : 0;
    }
  }
}

// ----------------------------------------------------------------------------
// the product
// ----------------------------------------------------------------------------
// 8 codes of a row -> 4 registers of 2 values q - z, in column order.
template <typename T>
__device__ __forceinline__ void dequant8(uint32_t w, uint32_t base, uint32_t (&v)[4]) {
  using T2 = typename Elem<T>::T2;
  const T2 b = *reinterpret_cast<const T2*>(&base);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) | Elem<T>::kOne;
    const T2 r = __hsub2(*reinterpret_cast<const T2*>(&u), b);
    v[i] = *reinterpret_cast<const uint32_t*>(&r);
  }
}

struct W4Args {
  const void* x;
  const char* packed;
  W4Layout w;
  int N, K, R, act, out_fp32;
  int k, rows_sorted;
  const int* expert_begin;  // null: one expert, R rows
  const int* sorted_slots;
  void* out;
};

// NT tiles of 8 rows of x per pass; GPC groups per chunk; kPair: a gate tile and its up tile
// per warp.
template <typename T, int NT, int GPC, bool kZeros, bool kPair>
__global__ void __launch_bounds__(kW4Warps * 32) w4_matvec_kernel(const W4Args p) {
  constexpr int kTiles = kPair ? 2 : 1;
  constexpr int kPartPerGroup = 4 / GPC;  // 32-column parts per group
  __shared__ float red[kW4Warps][kTiles][kTileRows][NT * 8 + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int jobs = kPair ? p.w.half_tiles : p.w.tiles;
  const int e = blockIdx.x / jobs, tile0 = blockIdx.x - e * jobs;
  int rb = 0, re = p.R;
  if (p.expert_begin) {
    rb = p.expert_begin[e];
    re = p.expert_begin[e + 1];
  }
  const T* x = static_cast<const T*>(p.x);
  for (int r0 = rb; r0 < re; r0 += NT * 8) {
    const T* xr[NT];  // this lane's row of each 8; null past the last
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + g;
      xr[nt] = nullptr;
      if (r < re) {
        const int64_t src = p.expert_begin && !p.rows_sorted ? p.sorted_slots[r] / p.k : r;
        xr[nt] = x + src * p.K;
      }
    }
    float tot[kTiles][NT][4] = {};
    for (int c = warp; c < p.w.chunks; c += kW4Warps) {
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl) {
        const int64_t b = ((int64_t)e * p.w.tiles + tile0 + tl * p.w.half_tiles) * p.w.chunks + c;
        const uint4* cw = reinterpret_cast<const uint4*>(p.packed + b * kTileBytes);
        const uint4 lo = cw[lane], hi = cw[32 + lane];
        const uint32_t* sw = reinterpret_cast<const uint32_t*>(p.packed + p.w.off_scales) + (b * 8 + g) * GPC;
        const uint16_t* zw = reinterpret_cast<const uint16_t*>(p.packed + p.w.off_zeros) + (b * 8 + g) * GPC;
        const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
        float acc[NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int grp = j / kPartPerGroup;
          if (j % kPartPerGroup == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
          uint32_t bl = Elem<T>::kOne + 0x00080008u, bh = bl;
          if (kZeros) {
            const uint32_t z = zw[grp];
            bl = Elem<T>::kOne + (z & 15u) * 0x00010001u;
            bh = Elem<T>::kOne + (z >> 8) * 0x00010001u;
          }
          uint32_t al[4], ah[4];
          dequant8<T>(lw[j], bl, al);
          dequant8<T>(hw[j], bh, ah);
          const int col = c * kChunkCols + j * 32 + t * 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint4 xv = make_uint4(0, 0, 0, 0);
            if (xr[nt] && col < p.K) xv = *reinterpret_cast<const uint4*>(xr[nt] + col);
            mma16816<T>(acc[nt], al[0], ah[0], al[1], ah[1], xv.x, xv.y);
            mma16816<T>(acc[nt], al[2], ah[2], al[3], ah[3], xv.z, xv.w);
          }
          if (j % kPartPerGroup == kPartPerGroup - 1) {
            const uint32_t s = sw[grp];
            const float s0 = Elem<T>::f((uint16_t)s), s1 = Elem<T>::f((uint16_t)(s >> 16));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              tot[tl][nt][0] += s0 * acc[nt][0];
              tot[tl][nt][1] += s0 * acc[nt][1];
              tot[tl][nt][2] += s1 * acc[nt][2];
              tot[tl][nt][3] += s1 * acc[nt][3];
            }
          }
        }
      }
    }
#pragma unroll
    for (int tl = 0; tl < kTiles; ++tl)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        red[warp][tl][g][nt * 8 + 2 * t] = tot[tl][nt][0];
        red[warp][tl][g][nt * 8 + 2 * t + 1] = tot[tl][nt][1];
        red[warp][tl][g + 8][nt * 8 + 2 * t] = tot[tl][nt][2];
        red[warp][tl][g + 8][nt * 8 + 2 * t + 1] = tot[tl][nt][3];
      }
    __syncthreads();
    for (int i = threadIdx.x; i < kTileRows * NT * 8; i += kW4Warps * 32) {
      const int row = i % kTileRows, r = r0 + i / kTileRows;
      const TileRows tr = tile_rows(tile0, p.w.half_tiles, p.w.half_rows);
      if (row >= tr.rows || r >= re) continue;
      float v[kTiles];
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl) {
        v[tl] = 0.f;
        for (int q = 0; q < kW4Warps; ++q) v[tl] += red[q][tl][row][i / kTileRows];
      }
      const int n = tr.row0 + row;
      if (kPair) {
        float a, d;
        if (p.act == MOE_ACT_SILU) activation<MOE_ACT_SILU>(v[0], a, d);
        else activation<MOE_ACT_GELU>(v[0], a, d);
        static_cast<T*>(p.out)[(int64_t)r * (p.N / 2) + n] = Elem<T>::r(a * v[kTiles - 1]);
      } else if (p.out_fp32) {
        static_cast<float*>(p.out)[(int64_t)r * p.N + n] = v[0];
      } else {
        static_cast<T*>(p.out)[(int64_t)r * p.N + n] = Elem<T>::r(v[0]);
      }
    }
    __syncthreads();
  }
}

template <typename T, int NT, int GPC, bool kZeros>
static int launch_w4_p(const W4Args& a, int E, cudaStream_t stream) {
  const bool pair = a.act != MOE_ACT_NONE;
  const int64_t ctas = (int64_t)E * (pair ? a.w.half_tiles : a.w.tiles);
  if (ctas > 0x7fffffff) return MOE_LORA_ERR_UNSUPPORTED;
  if (pair)
    return launch_pdl(w4_matvec_kernel<T, NT, GPC, kZeros, true>, (unsigned)ctas, kW4Warps * 32, 0, stream, false, a);
  return launch_pdl(w4_matvec_kernel<T, NT, GPC, kZeros, false>, (unsigned)ctas, kW4Warps * 32, 0, stream, false, a);
}
template <typename T, int NT>
static int launch_w4_n(const W4Args& a, int E, bool zeros, cudaStream_t stream) {
  switch (a.w.gpc * 2 + (zeros ? 1 : 0)) {
    case 2: return launch_w4_p<T, NT, 1, false>(a, E, stream);
    case 3: return launch_w4_p<T, NT, 1, true>(a, E, stream);
    case 4: return launch_w4_p<T, NT, 2, false>(a, E, stream);
    case 5: return launch_w4_p<T, NT, 2, true>(a, E, stream);
    case 8: return launch_w4_p<T, NT, 4, false>(a, E, stream);
    default: return launch_w4_p<T, NT, 4, true>(a, E, stream);
  }
}
template <typename T>
static int launch_w4(const W4Args& a, int E, bool zeros, int rows, cudaStream_t stream) {
  return rows <= 8    ? launch_w4_n<T, 1>(a, E, zeros, stream)
         : rows <= 16 ? launch_w4_n<T, 2>(a, E, zeros, stream)
                      : launch_w4_n<T, 4>(a, E, zeros, stream);
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
  if (!w.valid) return MOE_LORA_ERR_UNSUPPORTED;
  if (!codes || !scales || !packed || !aligned16(packed)) return MOE_LORA_ERR_INVALID_ARG;
  int st = check_device();
  if (st != MOE_LORA_OK) return st;
  const int64_t blocks = (int64_t)E * w.tiles * w.chunks;
  return launch_pdl(w4_pack_kernel, (unsigned)std::min<int64_t>(blocks, 152 * 16), 256, 0,
                    reinterpret_cast<cudaStream_t>(stream), false, codes, static_cast<const uint16_t*>(scales),
                    zeros, N, K, ceil_div(K, group), w, blocks, static_cast<char*>(packed));
}

extern "C" int moe_w4_matvec(const void* x, int dtype, const void* packed, int E, int N, int K, int group,
                             int has_zeros, int gated, int act, int T, const moe_lora_align_t* al, int rows_sorted,
                             void* out, int out_fp32, moe_lora_stream_t stream) {
  using namespace moe_lora;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_LORA_ERR_INVALID_ARG;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SILU && act != MOE_ACT_GELU) return MOE_LORA_ERR_INVALID_ARG;
  if (act != MOE_ACT_NONE && (!gated || out_fp32)) return MOE_LORA_ERR_INVALID_ARG;
  if (T < 0 || T > (1 << 22)) return MOE_LORA_ERR_INVALID_ARG;
  W4Args a = {};
  a.w = w4_layout(E, N, K, group, has_zeros, gated);
  if (!a.w.valid || K % 8 != 0) return MOE_LORA_ERR_UNSUPPORTED;
  int rows = T, st;
  if (al) {
    AlignLayout lay;
    if ((st = check_align(al, &lay)) != MOE_LORA_OK) return st;
    if (al->E != E || al->T != T) return MOE_LORA_ERR_INVALID_ARG;
    const AlignView v = align_view(al->buf, lay);
    a.expert_begin = v.expert_begin;
    a.sorted_slots = v.sorted_slots;
    a.k = al->k;
    a.rows_sorted = rows_sorted;
    // the pass that most experts fit in: twice the mean rows of an expert
    rows = (int)std::min<int64_t>(lay.S, 2 * ceil_div64(lay.S, E));
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
  a.act = act;
  a.out_fp32 = out_fp32;
  a.out = out;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == MOE_DTYPE_BF16 ? launch_w4<__nv_bfloat16>(a, E, has_zeros != 0, rows, s)
                                 : launch_w4<__half>(a, E, has_zeros != 0, rows, s);
}
