// The gated feed-forward block and its gradients, dense, in bf16 or fp16:
//   h = a(x Wg^T) * (x Wu^T)                                (moe_gated_ffn)
//   dg = dh u a'(g), du = dh a(g);  dx = [dg du] W1, dW1 = [dg du]^T x   (the backward)
//
// Plain tiles: a CTA computes a 64 x 64 tile of a product (two of them, gate and up, where
// the activation follows) from 64 x 16 slices of both operands staged in shared memory as
// fp32; 256 threads hold 4 x 4 outputs each. Operands are addressed by two strides, so one
// kernel serves every transposition.
#include "activation.cuh"
#include "internal.h"

namespace moe_lora {

enum { kEpiStore = 0, kEpiGated = 1, kEpiGrad = 2 };

template <typename T, int kEpi, int kAct>
__global__ void __launch_bounds__(256) tile_product_kernel(
    const T* A, int64_t sam, int64_t sak, const T* B, int64_t sbn, int64_t sbk, int64_t up_off, int M, int N,
    int K, const T* dh, T* out, int64_t ldo) {
  constexpr bool kTwo = kEpi != kEpiStore;
  __shared__ float sa[16][65], sb[kTwo ? 2 : 1][16][65];
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tm = threadIdx.x / 16, tn = threadIdx.x % 16;
  float acc[2][4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 16) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int r = i / 16, k = i % 16;
      const bool kin = k0 + k < K;
      sa[k][r] = kin && m0 + r < M ? Elem<T>::f(A[(m0 + r) * sam + (k0 + k) * sak]) : 0.f;
      for (int q = 0; q < (kTwo ? 2 : 1); ++q)
        sb[q][k][r] = kin && n0 + r < N ? Elem<T>::f(B[q * up_off + (n0 + r) * sbn + (k0 + k) * sbk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[0][i][j] += sa[k][tm + 16 * i] * sb[0][k][tn + 16 * j];
          if (kTwo) acc[1][i][j] += sa[k][tm + 16 * i] * sb[kTwo ? 1 : 0][k][tn + 16 * j];
        }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + tm + 16 * i;
      const int n = n0 + tn + 16 * j;
      if (m >= M || n >= N) continue;
      if (kEpi == kEpiStore) {
        out[m * ldo + n] = Elem<T>::r(acc[0][i][j]);
        continue;
      }
      float a, d;
      activation<kAct>(acc[0][i][j], a, d);
      if (kEpi == kEpiGated) {
        out[m * ldo + n] = Elem<T>::r(a * acc[1][i][j]);
      } else {
        const float g = Elem<T>::f(dh[m * N + n]);
        out[m * ldo + n] = Elem<T>::r(g * acc[1][i][j] * d);
        out[m * ldo + N + n] = Elem<T>::r(g * a);
      }
    }
}

template <typename T, int kEpi, int kAct>
static int launch_tile_product(const void* A, int64_t sam, int64_t sak, const void* B, int64_t sbn,
                               int64_t sbk, int64_t up_off, int M, int N, int K, const void* dh,
                               void* out, int64_t ldo, cudaStream_t stream) {
  if (ceil_div(M, 64) > 65535) return MOE_LORA_ERR_UNSUPPORTED;
  return launch_pdl(tile_product_kernel<T, kEpi, kAct>, dim3(ceil_div(N, 64), ceil_div(M, 64)), 256, 0,
                    stream, false, static_cast<const T*>(A), sam, sak, static_cast<const T*>(B), sbn, sbk,
                    up_off, M, N, K, static_cast<const T*>(dh), static_cast<T*>(out), ldo);
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
  const int64_t up = (int64_t)I * H;
  auto go = [&](auto f) { return f(x, H, 1, W1, H, 1, up, T, I, H, dh, out, ldo, stream); };
  if (dtype == MOE_DTYPE_BF16)
    return act == MOE_ACT_SILU ? go(launch_tile_product<__nv_bfloat16, kEpi, MOE_ACT_SILU>)
                               : go(launch_tile_product<__nv_bfloat16, kEpi, MOE_ACT_GELU>);
  return act == MOE_ACT_SILU ? go(launch_tile_product<__half, kEpi, MOE_ACT_SILU>)
                             : go(launch_tile_product<__half, kEpi, MOE_ACT_GELU>);
}

}  // namespace moe_lora

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
  if ((st = launch_gated<kEpiGrad>(dtype, act, x, W1, T, H, I, dh, workspace, 2 * (int64_t)I, s)) != MOE_LORA_OK)
    return st;
  auto product = [&](auto f) {
    if (dx) {
      const int e = f(workspace, 2 * (int64_t)I, 1, W1, 1, H, 0, T, H, 2 * I, nullptr, dx, H, s);
      if (e != MOE_LORA_OK) return e;
    }
    if (dW1) return f(workspace, 1, 2 * (int64_t)I, x, 1, H, 0, 2 * I, H, T, nullptr, dW1, H, s);
    return (int)MOE_LORA_OK;
  };
  return dtype == MOE_DTYPE_BF16 ? product(launch_tile_product<__nv_bfloat16, kEpiStore, MOE_ACT_SILU>)
                                 : product(launch_tile_product<__half, kEpiStore, MOE_ACT_SILU>);
}
