// Launchers and device pieces shared between the gated block's translation units.
#pragma once

#include "activation.cuh"
#include "internal.h"

namespace moe_lora {

// What a product's epilogue does: store it; a(g) * u of a gate and an up product; or the
// backward's dg and du of them.
enum { kEpiStore = 0, kEpiGated = 1, kEpiGrad = 2 };

// Up to kFewTokens tokens gated_few_tokens.cu computes the gated block (dh null: h [T, I]) or
// its backward's dy = [dg | du] [T, 2I], with the weights on the MMA's M side: 128 tokens of
// 4096/14336 in 42 us, where the 256-row tiles of gated_ffn.cu, for more tokens, take 50 us.
constexpr int kFewTokens = 128;
int launch_gated_few(int dtype, int act, const void* x, const void* W1, int T, int H, int I, const void* dh, void* out,
                     cudaStream_t stream);
// dx [T, H] = dy [T, 2I] W1 for at most kFewTokens tokens.
int launch_dx_few(int dtype, const void* dy, const void* W1, int T, int H, int I, void* dx, cudaStream_t stream);

// The device address of the sticky error word, per context.
int ffn_error_word(unsigned int** out);

// The main loops' wait limit that the calling thread has set (moe_ffn_set_wait_limit).
unsigned long long ffn_wait_ns();

// An operand: rows [rows, cols] with `cols` contiguous. Summed over cols (K-major) a box is
// 64 columns by `box_rows` rows; summed over rows (MN-major), 64 by 64.
int operand_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, bool mn, int box_rows);

// Shared-memory matrix descriptor of an operand with m (n) contiguous: 64 x 64 boxes (64
// summed rows of 128 bytes, 128-byte swizzle), one after the other along m. Eight summed rows
// are 1024 bytes (stride offset), the next 64 of m one box of `block` bytes (leading offset).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr, uint32_t block = 64 * 128) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(block >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

template <typename T> struct MmaType;
template <> struct MmaType<__nv_bfloat16> { static constexpr uint32_t kFmt = 1; };
template <> struct MmaType<__half> { static constexpr uint32_t kFmt = 0; };

}  // namespace moe_lora
