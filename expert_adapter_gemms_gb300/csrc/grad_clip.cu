// The global norm of many gradient tensors and the gradients scaled to a bound
// (moe_grad_clip): norm = sqrt(sum_i |g_i|^2), out_i = g_i * min(1, max_norm / (norm + 1e-6)).
//
// Two launches, bound by memory: the gradients are read twice and written once (whether
// they are scaled is known only when all of them are read). The tensors are cut into chunks of
// 32 KB, counted through all tensors; the table of tensors travels in the kernels'
// parameters (no copy, so a call can be captured), in a table of 48 tensors where that is
// enough: 29 KB of parameters cost 2 us a launch. The first kernel sums squares, a CTA taking
// every gridDim-th chunk with all of a thread's loads in flight and the next chunk looked up
// meanwhile: fp32 per thread (64 terms a chunk, the chunks' sums with their rounding carried
// along) and in a tree per CTA, fp64 over the CTAs' partial sums. In the second every CTA adds
// those up in the same order, so that all of them scale by the same number without a third
// launch or an atomic; it takes the chunks backwards, so that the last ones read are found in
// L2. 100 M bf16 elements: 34 us (5.9 TB/s) and 60 us; 300 M fp32: 174 us (6.9) and 380 (6.3).
//
// Up to 1 MB in all (the adapters of a layer) one launch does: a cluster of eight CTAs holds the
// gradients in registers, the CTAs' sums meet in distributed shared memory, and nothing is
// read twice.
#include <algorithm>

#include "activation.cuh"
#include "internal.h"

namespace moe_lora {

constexpr int kClipThreads = 256;
constexpr int kChunkGroups = 2048;  // 16-byte groups of a chunk: 8 per thread
constexpr int kTableMax = 1024;  // tensors per launch (kernel parameters hold 32764 bytes)
constexpr int kTableFew = 48;    // or of the small table
constexpr int kClipCtas = 152 * 4;
constexpr float kNormEps = 1e-6f;

template <int kMax>
struct ClipTable {
  int n, chunks;         // tensors and chunks of this launch
  int first[kMax + 1];   // chunks before tensor i
  const void* in[kMax];
  void* out[kMax];
  int64_t numel[kMax];   // times 4, plus the type
};
static_assert(sizeof(ClipTable<kTableMax>) <= 32000, "kernel parameters");

// Elements between `p` and the 16-byte boundary at or before it: chunks are cut at
// boundaries, so that whole 16-byte groups stay whole.
__host__ __device__ __forceinline__ int clip_lead(const void* p, int type) {
  return (int)((reinterpret_cast<uintptr_t>(p) & 15) >> (type == MOE_DTYPE_FP32 ? 2 : 1));
}

__host__ __device__ __forceinline__ int clip_chunk(int type) {  // elements of a chunk
  return kChunkGroups * (type == MOE_DTYPE_FP32 ? 4 : 8);
}

// one(p, k): element k, read from L2 as the whole groups are (an earlier launch wrote it).
template <int kType> struct ClipType;
template <typename T>
struct ClipType16 : Elem<T> {
  static constexpr int kPer = 8;
  using E = T;
  static __device__ __forceinline__ float one(const void* p, int64_t k) {
    return Elem<T>::f(__ldcg(static_cast<const uint16_t*>(p) + k));
  }
};
template <> struct ClipType<MOE_DTYPE_BF16> : ClipType16<__nv_bfloat16> {};
template <> struct ClipType<MOE_DTYPE_FP16> : ClipType16<__half> {};
template <> struct ClipType<MOE_DTYPE_FP32> {
  static constexpr int kPer = 4;
  using E = float;
  static __device__ __forceinline__ float f(float v) { return v; }
  static __device__ __forceinline__ float r(float v) { return v; }
  static __device__ __forceinline__ float one(const void* p, int64_t k) {
    return __ldcg(static_cast<const float*>(p) + k);
  }
};

struct ClipChunk {
  const void* in;       // the 16-byte boundary at or before the tensor
  void* out;            // the output less the same number of elements
  int64_t lo, hi;       // the chunk's elements, counted from that boundary
  int64_t g0, w0, w1;   // its first 16-byte group, and its whole groups [w0, w1)
  int type;
  bool vec;             // the output's boundary is a 16-byte boundary too
};

constexpr int kGroups = kChunkGroups / kClipThreads;  // a thread's groups of a chunk

// A thread's whole groups of the chunk, all in flight.
__device__ __forceinline__ void load_chunk(const ClipChunk& c, uint4 (&v)[kGroups]) {
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int64_t g = c.g0 + i * kClipThreads + threadIdx.x % kClipThreads;
    if (g >= c.w0 && g < c.w1) v[i] = __ldcg(static_cast<const uint4*>(c.in) + g);
  }
}
// fn(group, value) for the thread's whole groups; edge(element) for the elements of groups that
// are cut at an end of the tensor, by the threads that would have taken them.
template <typename C, typename Fn, typename Edge>
__device__ __forceinline__ void use_chunk(const ClipChunk& c, uint4 (&v)[kGroups], Fn&& fn, Edge&& edge) {
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int64_t g = c.g0 + i * kClipThreads + threadIdx.x % kClipThreads;
    if (g >= c.w0 && g < c.w1) fn(g, v[i]);
  }
  if (c.w0 * C::kPer == c.lo && c.w1 * C::kPer == c.hi) return;
  for (int i = 0; i < kGroups; ++i) {
    const int64_t g = c.g0 + i * kClipThreads + threadIdx.x % kClipThreads;
    if (g >= c.w0 && g < c.w1) continue;
    for (int64_t k = g * C::kPer; k < (g + 1) * C::kPer; ++k)
      if (k >= c.lo && k < c.hi) edge(k);
  }
}

template <int kType>
__device__ __forceinline__ float chunk_squares(const ClipChunk& c, uint4 (&v)[kGroups]) {
  using C = ClipType<kType>;
  using E = typename C::E;
  float sum = 0.f;
  use_chunk<C>(
      c, v,
      [&](int64_t, const uint4& u) {
        const E* e = reinterpret_cast<const E*>(&u);
#pragma unroll
        for (int i = 0; i < C::kPer; ++i) sum += C::f(e[i]) * C::f(e[i]);
      },
      [&](int64_t k) {
        const float f = C::one(c.in, k);
        sum += f * f;
      });
  return sum;
}

template <int kType>
__device__ __forceinline__ void chunk_scale(const ClipChunk& c, uint4 (&v)[kGroups], float scale) {
  using C = ClipType<kType>;
  using E = typename C::E;
  E* q = static_cast<E*>(c.out);
  use_chunk<C>(
      c, v,
      [&](int64_t g, uint4& u) {
        E* e = reinterpret_cast<E*>(&u);
#pragma unroll
        for (int i = 0; i < C::kPer; ++i) e[i] = C::r(C::f(e[i]) * scale);
        if (c.vec) {
          __stcs(static_cast<uint4*>(c.out) + g, u);
        } else {
          for (int i = 0; i < C::kPer; ++i) q[g * C::kPer + i] = e[i];
        }
      },
      [&](int64_t k) { q[k] = C::r(C::one(c.in, k) * scale); });
}

template <int kMax>
__device__ __forceinline__ ClipChunk find_chunk(const ClipTable<kMax>& t, int c) {
  int a = 0, b = t.n - 1;  // the last tensor with first[] <= c
  while (a < b) {
    const int m = (a + b + 1) / 2;
    if (t.first[m] <= c) a = m;
    else b = m - 1;
  }
  ClipChunk k;
  k.type = (int)(t.numel[a] & 3);
  const int size = k.type == MOE_DTYPE_FP32 ? 4 : 2;
  const int lead = clip_lead(t.in[a], k.type);
  k.in = static_cast<const char*>(t.in[a]) - lead * size;
  k.out = static_cast<char*>(t.out[a]) - lead * size;
  k.vec = (reinterpret_cast<uintptr_t>(k.out) & 15) == 0;
  const int64_t end = lead + (t.numel[a] >> 2);
  const int chunk = clip_chunk(k.type);
  const int64_t at = (int64_t)(c - t.first[a]) * chunk;
  k.lo = at > lead ? at : lead;
  k.hi = at + chunk < end ? at + chunk : end;
  const int shift = k.type == MOE_DTYPE_FP32 ? 2 : 3;  // elements of a group
  k.g0 = at >> shift;
  k.w0 = (k.lo + (1 << shift) - 1) >> shift;
  k.w1 = k.hi >> shift;
  return k;
}

__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
  if (isinf(max_norm)) return 1.f;  // no bound, though the ratio to an infinite norm is none
  const float ratio = max_norm / (norm + kNormEps);
  return ratio >= 1.f ? 1.f : ratio;  // a NaN norm's ratio stays NaN
}

// Sum over the CTA, in a fixed tree, in thread 0.
template <int kThreads>
__device__ __forceinline__ float cta_sum(float v) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float part[kWarps];
#pragma unroll
  for (int off = 16; off > 0; off /= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < kWarps ? part[threadIdx.x] : 0.f;
#pragma unroll
    for (int off = kWarps / 2; off > 0; off /= 2) v += __shfl_xor_sync(0xffffffffu, v, off);
  }
  return v;
}

template <int kMax>
__global__ void __launch_bounds__(kClipThreads)
    clip_squares_kernel(const __grid_constant__ ClipTable<kMax> t, double* __restrict__ partial) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  float sum = 0.f, lost = 0.f;  // over the chunks, with the rounding carried along
  ClipChunk k;
  int c = blockIdx.x;
  if (c < t.chunks) k = find_chunk(t, c);
  while (c < t.chunks) {
    uint4 v[kGroups];
    load_chunk(k, v);
    c += gridDim.x;
    ClipChunk next = k;  // looked up while the loads are in flight
    if (c < t.chunks) next = find_chunk(t, c);
    float more;
    if (k.type == MOE_DTYPE_BF16) more = chunk_squares<MOE_DTYPE_BF16>(k, v);
    else if (k.type == MOE_DTYPE_FP16) more = chunk_squares<MOE_DTYPE_FP16>(k, v);
    else more = chunk_squares<MOE_DTYPE_FP32>(k, v);
    const float add = more - lost, to = sum + add;
    lost = isfinite(to) ? (to - sum) - add : 0.f;  // an infinite sum stays infinite
    sum = to;
    k = next;
  }
  sum = cta_sum<kClipThreads>(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <int kMax>
__global__ void __launch_bounds__(kClipThreads)
    clip_scale_kernel(const __grid_constant__ ClipTable<kMax> t, const double* __restrict__ partial, int nparts,
                      float max_norm, float* __restrict__ norm_out) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  __shared__ float s_scale;
  if (threadIdx.x < 32) {  // one warp adds the partial sums up, the same way in every CTA
    double sum = 0;
    for (int i = threadIdx.x; i < nparts; i += 32) sum += __ldcg(partial + i);
    for (int off = 16; off > 0; off /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (threadIdx.x == 0) {
      const float norm = sqrtf((float)sum);
      if (norm_out && blockIdx.x == 0) *norm_out = norm;
      s_scale = clip_factor(norm, max_norm);
    }
  }
  __syncthreads();
  const float scale = s_scale;
  int c = t.chunks - 1 - (int)blockIdx.x;
  ClipChunk k;
  if (c >= 0) k = find_chunk(t, c);
  while (c >= 0) {
    uint4 v[kGroups];
    const bool skip = scale == 1.f && k.in == k.out;  // in place and within the bound
    if (!skip) load_chunk(k, v);
    c -= gridDim.x;
    ClipChunk next = k;
    if (c >= 0) next = find_chunk(t, c);
    if (!skip) {
      if (k.type == MOE_DTYPE_BF16) chunk_scale<MOE_DTYPE_BF16>(k, v, scale);
      else if (k.type == MOE_DTYPE_FP16) chunk_scale<MOE_DTYPE_FP16>(k, v, scale);
      else chunk_scale<MOE_DTYPE_FP32>(k, v, scale);
    }
    k = next;
  }
}

// The whole of it in one cluster: a chunk to every 256 threads, which keep it in registers
// between the sum and the scaling.
constexpr int kSmallCtas = 8, kSmallChunks = 4;  // CTAs, and chunks of each
__global__ void __launch_bounds__(kSmallChunks * kClipThreads, 1)
    clip_small_kernel(const __grid_constant__ ClipTable<kTableFew> t, float max_norm, float* __restrict__ norm_out,
                      int scale_out) {
  __shared__ float s_sum;
  __shared__ float s_scale;
  pdl_wait();
  if (threadIdx.x == 0) pdl_trigger();
  const int c = blockIdx.x + (threadIdx.x / kClipThreads) * kSmallCtas;
  const bool mine = c < t.chunks;
  ClipChunk k = {};
  uint4 v[kGroups];
  float squares = 0.f;
  if (mine) {
    k = find_chunk(t, c);
    load_chunk(k, v);
    if (k.type == MOE_DTYPE_BF16) squares = chunk_squares<MOE_DTYPE_BF16>(k, v);
    else if (k.type == MOE_DTYPE_FP16) squares = chunk_squares<MOE_DTYPE_FP16>(k, v);
    else squares = chunk_squares<MOE_DTYPE_FP32>(k, v);
  }
  squares = cta_sum<kSmallChunks * kClipThreads>(squares);
  if (threadIdx.x == 0) s_sum = squares;
  cluster_sync();
  if (threadIdx.x < 32) {  // every CTA's, a lane each, then one tree
    float part = 0.f;
    if (threadIdx.x < kSmallCtas)
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(part) : "r"(smem_in_cta(&s_sum, threadIdx.x)) : "memory");
    double sum = part;
#pragma unroll
    for (int off = kSmallCtas / 2; off > 0; off /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (threadIdx.x == 0) {
      const float norm = sqrtf((float)sum);
      if (blockIdx.x == 0) *norm_out = norm;
      s_scale = clip_factor(norm, max_norm);
    }
  }
  cluster_sync();  // read by all before any leaves
  const float scale = s_scale;
  if (!scale_out || !mine || (scale == 1.f && k.in == k.out)) return;
  if (k.type == MOE_DTYPE_BF16) chunk_scale<MOE_DTYPE_BF16>(k, v, scale);
  else if (k.type == MOE_DTYPE_FP16) chunk_scale<MOE_DTYPE_FP16>(k, v, scale);
  else chunk_scale<MOE_DTYPE_FP32>(k, v, scale);
}

// Takes down the tensors from `at` on, as far as the table holds; `at` becomes the first left.
template <int kMax>
static void fill_table(ClipTable<kMax>& t, const void* const* grads, void* const* outs, const int64_t* numels,
                       const int32_t* dtypes, int n, int& at) {
  t.n = 0;
  int64_t chunks = 0;
  for (; at < n && t.n < kMax; ++at) {
    if (numels[at] == 0) continue;
    t.first[t.n] = (int)chunks;
    t.in[t.n] = grads[at];
    t.out[t.n] = outs ? outs[at] : nullptr;
    t.numel[t.n] = numels[at] * 4 + dtypes[at];
    chunks += ceil_div64(numels[at] + clip_lead(grads[at], dtypes[at]), clip_chunk(dtypes[at]));
    ++t.n;
  }
  t.first[t.n] = (int)chunks;
  t.chunks = (int)chunks;
}

// Both passes over the tensors, kMax to a launch.
template <int kMax>
static int run_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int32_t* dtypes, int n,
                    float max_norm, float* norm, double* partial, cudaStream_t s) {
  int nparts = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int at = 0, parts = 0;
    do {
      ClipTable<kMax> t;
      fill_table(t, grads, outs, numels, dtypes, n, at);
      const int ctas = (int)std::min<int64_t>(std::max<int64_t>(t.chunks, 1), kClipCtas);
      int st;
      if (pass == 0) {
        st = launch_pdl(clip_squares_kernel<kMax>, ctas, kClipThreads, 0, s, true, t, partial + parts);
      } else {
        if (!outs) t.chunks = 0;
        st = launch_pdl(clip_scale_kernel<kMax>, outs ? ctas : 1, kClipThreads, 0, s, true, t,
                        (const double*)partial, nparts, max_norm, parts == 0 ? norm : (float*)nullptr);
      }
      if (st != MOE_LORA_OK) return st;
      parts += ctas;
      if (pass == 1 && !outs) break;
    } while (at < n);
    nparts = parts;
  }
  return MOE_LORA_OK;
}

}  // namespace moe_lora

extern "C" size_t moe_grad_clip_workspace_size(int n, const int64_t* numels) {
  using namespace moe_lora;
  if (n < 0 || (n > 0 && !numels)) return 0;
  for (int i = 0; i < n; ++i)
    if (numels[i] < 0) return 0;
  return (size_t)std::max(1, ceil_div(n, kTableMax)) * kClipCtas * sizeof(double);
}

extern "C" int moe_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels,
                             const int32_t* dtypes, int n, float max_norm, float* norm,
                             void* workspace, size_t workspace_bytes, moe_lora_stream_t stream) {
  using namespace moe_lora;
  if (n < 0 || !norm || !(max_norm >= 0.f)) return MOE_LORA_ERR_INVALID_ARG;
  if (n > 0 && (!grads || !numels || !dtypes)) return MOE_LORA_ERR_INVALID_ARG;
  int64_t all_chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (numels[i] < 0 || dtypes[i] < 0 || dtypes[i] > MOE_DTYPE_FP32) return MOE_LORA_ERR_INVALID_ARG;
    if (numels[i] > ((int64_t)1 << 40)) return MOE_LORA_ERR_UNSUPPORTED;
    const uintptr_t mask = dtypes[i] == MOE_DTYPE_FP32 ? 3 : 1;
    if (numels[i] == 0) continue;
    if (!grads[i] || (reinterpret_cast<uintptr_t>(grads[i]) & mask)) return MOE_LORA_ERR_INVALID_ARG;
    if (outs && (!outs[i] || (reinterpret_cast<uintptr_t>(outs[i]) & mask))) return MOE_LORA_ERR_INVALID_ARG;
    all_chunks += ceil_div64(numels[i] + 7, clip_chunk(dtypes[i]));
    if (all_chunks > 0x7fff0000) return MOE_LORA_ERR_UNSUPPORTED;
  }
  if (!workspace || !aligned16(workspace)) return MOE_LORA_ERR_INVALID_ARG;
  if (workspace_bytes < moe_grad_clip_workspace_size(n, numels)) return MOE_LORA_ERR_WORKSPACE_TOO_SMALL;
  int st = check_device();
  if (st != MOE_LORA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  if (n <= kTableFew && all_chunks <= kSmallCtas * kSmallChunks) {
    ClipTable<kTableFew> t;
    int at = 0;
    fill_table(t, grads, outs, numels, dtypes, n, at);
    return launch_pdl_cluster(clip_small_kernel, kSmallCtas, kSmallChunks * kClipThreads, 0, s, true, kSmallCtas, t, max_norm, norm,
                              outs ? 1 : 0);
  }
  return n <= kTableFew ? run_clip<kTableFew>(grads, outs, numels, dtypes, n, max_norm, norm, partial, s)
                        : run_clip<kTableMax>(grads, outs, numels, dtypes, n, max_norm, norm, partial, s);
}
