// The gated block for single tokens: h = a(x Wg^T) * (x Wu^T) at up to kFewMaxTokens rows of x.
//
// The weights' stream bounds it: 4 I H bytes against 4 T I H operations. The weights take the
// M side of mma.sync.m16n8k16 and 8 tokens its N side, so that a weight is read once and no
// tensor-core row is padding of tokens to 128. Which columns share an MMA step is free as long
// as both operands agree: lane t of a quad takes columns 8t .. 8t+7 of every 32, and both
// fragments are plain 16-byte loads of a row as it lies -- no shared memory, no transposition.
// A warp owns 16 features, gate and up rows both, over its share of the columns, and keeps
// kDepth steps of weights in flight in registers; the warps of a CTA share out the columns and
// add up through shared memory in a fixed order, where g and u of an output meet.
#include <algorithm>

#include "activation.cuh"
#include "gated.h"

namespace moe_lora {

constexpr int kFewWarps = 8;

struct FewArgs {
  const void *x, *W1;
  void* out;  // h [T, I]
  int T, H, I;
};

template <typename T, int kAct>
__global__ void __launch_bounds__(kFewWarps * 32) gated_few_kernel(const FewArgs p) {
  constexpr int kDepth = 4;  // steps of 32 columns per batch, two batches in flight
  __shared__ float red[kFewWarps][32][kFewMaxTokens + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int i0 = blockIdx.x * 16;
  const T* W = static_cast<const T*>(p.W1);
  // the lane's rows: gate g, g + 8, up g, g + 8; rows past the last feature read
  // the last one, their sums are not used
  const uint4* w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t r = min(i0 + g + 8 * (q & 1), p.I - 1) + (q >> 1 ? (int64_t)p.I : 0);
    w[q] = reinterpret_cast<const uint4*>(W + r * p.H);
  }
  const int n8 = p.H / 8;             // 16-byte groups of a row
  const int steps = (p.H + 31) / 32;  // steps of 4 groups
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load = [&](uint4 (&v)[kDepth][4], int s0) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int c = (s0 + d * kFewWarps) * 4 + t;
#pragma unroll
      for (int q = 0; q < 4; ++q) v[d][q] = c < n8 ? ld_stream(w[q] + c) : zero;
    }
  };
  constexpr int kBatch = kFewWarps * kDepth;
  uint4 v0[kDepth][4], v1[kDepth][4];
  load(v0, warp);  // weights do not depend on a launch, x does
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  // tokens past the last repeat it, unused
  const uint4* xr = reinterpret_cast<const uint4*>(static_cast<const T*>(p.x) + (int64_t)min(g, p.T - 1) * p.H);
  float acc[2][4] = {};
  auto mul = [&](const uint4 (&v)[kDepth][4], int s0) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      const int c = (s0 + d * kFewWarps) * 4 + t;
      const uint4 xv = c < n8 ? __ldcg(xr + c) : zero;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 &a = v[d][2 * h], &b = v[d][2 * h + 1];
        mma16816<T>(acc[h], a.x, b.x, a.y, b.y, xv.x, xv.y);
        mma16816<T>(acc[h], a.z, b.z, a.w, b.w, xv.z, xv.w);
      }
    }
  };
  for (int s0 = warp; s0 < steps; s0 += 2 * kBatch) {
    load(v1, s0 + kBatch);
    mul(v0, s0);
    load(v0, s0 + 2 * kBatch);
    mul(v1, s0 + kBatch);
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* a = &red[warp][16 * h + g][2 * t];
    float* b = &red[warp][16 * h + g + 8][2 * t];
    a[0] = acc[h][0];
    a[1] = acc[h][1];
    b[0] = acc[h][2];
    b[1] = acc[h][3];
  }
  __syncthreads();
  if (threadIdx.x >= 16 * kFewMaxTokens) return;
  const int f = threadIdx.x % 16, tok = threadIdx.x / 16, n = i0 + f;
  if (n >= p.I || tok >= p.T) return;
  float gv = 0.f, uv = 0.f;
#pragma unroll
  for (int q = 0; q < kFewWarps; ++q) {
    gv += red[q][f][tok];
    uv += red[q][16 + f][tok];
  }
  float a, d;
  activation<kAct>(gv, a, d);
  static_cast<T*>(p.out)[(int64_t)tok * p.I + n] = Elem<T>::r(a * uv);
}

template <typename T>
static int launch_few_t(const FewArgs& p, int act, cudaStream_t stream) {
  const unsigned ctas = (unsigned)ceil_div(p.I, 16);
  return act == MOE_ACT_SILU
             ? launch_pdl(gated_few_kernel<T, MOE_ACT_SILU>, ctas, kFewWarps * 32, 0, stream, true, p)
             : launch_pdl(gated_few_kernel<T, MOE_ACT_GELU>, ctas, kFewWarps * 32, 0, stream, true, p);
}

int launch_gated_few(int dtype, int act, const void* x, const void* W1, int T, int H, int I, void* out,
                     cudaStream_t stream) {
  const FewArgs p = {x, W1, out, T, H, I};
  return dtype == MOE_DTYPE_BF16 ? launch_few_t<__nv_bfloat16>(p, act, stream) : launch_few_t<__half>(p, act, stream);
}

}  // namespace moe_lora
