// Tokens' rows laid out by expert and brought back, with their gradients, and the gradient of
// the router's softmax:
//   permute             xs[i] = x[slot(i) / k]
//   unpermute           y[t] = sum_j w[t, j] o[row(t, j)]   (without weights: permute's gradient)
//   unpermute backward  do[row(t, j)] = w[t, j] dy[t],  dw[t, j] = <o[row(t, j)], dy[t]>
//   top-k softmax       dl[t, ids[t, j]] = w_j (dw_j - sum_i w_i dw_i)
//
// All of them walk the tokens, not the sorted rows: a token's x is read once for its k rows, a
// token's sum or dot products stay in one thread group, so nothing is added with atomics and no
// order varies. A group of a power of two threads, up to a CTA, takes a token, and a thread as
// wide a piece of a row as its length and the pointers' alignment allow (16 bytes for most
// models' widths). The bound is HBM, or a few launches' latency for few tokens: every byte comes
// from HBM once and is written once. (dy is read again, from L2, for every four choices of a
// token, two up to k = 2; the rows back read a token's last row again in place of those that fill
// 2, 4 or 8 up.) 4096 tokens' rows of 4 x 2880 bf16 back: 25 us (4.7 TB/s), of 1, 3, 6 and 8: 13, 22,
// 37 and 42 us for 7, 14, 24 and 31 at the rate of a copy; gradients of 2 x 4096 fp32 for as many: 58 us
// (5.8 TB/s); 4096 tokens out to 4: 20 us (5.9 TB/s), 64 tokens: 4 us. Few tokens of wide rows are
// bound by the rounds of a token's one CTA: 8 x 8191 bf16 back 42 us, 8 x 8192 5 us.
#include "activation.cuh"
#include "internal.h"

namespace moe_lora {

// V bytes of a row as fp32 values and back.
template <int V> struct Raw;
template <> struct Raw<16> { using T = uint4; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<2> { using T = uint16_t; };

template <typename E, int V>
struct Piece {
  static constexpr int N = V / (int)sizeof(E);
  typename Raw<V>::T raw;
  __device__ __forceinline__ void load(const void* row, int64_t i) {
    raw = __ldcg(static_cast<const typename Raw<V>::T*>(row) + i);
  }
  __device__ __forceinline__ void store(void* row, int64_t i) const { static_cast<typename Raw<V>::T*>(row)[i] = raw; }
  __device__ __forceinline__ void zero() { raw = typename Raw<V>::T{}; }
  __device__ __forceinline__ void to(float (&f)[N]) const {
    if constexpr (V == 2) {
      f[0] = Elem<E>::f(raw);
    } else {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        if constexpr (sizeof(E) == 4) {
          f[i] = __uint_as_float(u[i]);
        } else {
          const float2 t = Elem<E>::f2(u[i]);
          f[2 * i] = t.x;
          f[2 * i + 1] = t.y;
        }
      }
    }
  }
  __device__ __forceinline__ void from(const float (&f)[N]) {
    if constexpr (V == 2) {
      const E e = Elem<E>::r(f[0]);
      raw = *reinterpret_cast<const uint16_t*>(&e);
    } else {
      uint32_t* u = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        if constexpr (sizeof(E) == 4) u[i] = __float_as_uint(f[i]);
        else u[i] = Elem<E>::r2(f[2 * i], f[2 * i + 1]);
      }
    }
  }
};

constexpr int kPThreads = 256;

struct RowsArgs {
  const void* in;        // x or o
  const void* dy;
  const float* w;        // null: every weight is 1
  const int* hdr;
  const int* slot_row;
  void* out;             // xs, y or do
  float* dw;
  int T, k, group;       // threads per token (a power of two)
  int n;                 // pieces per row
  int zero;              // rows past the last kept one are set to zero
};

// The token of this thread's group and its place in it; false past the last token.
__device__ __forceinline__ bool group_token(const RowsArgs& a, int& t, int& c0) {
  const int per = kPThreads / a.group;
  const int64_t tok = (int64_t)blockIdx.x * per + threadIdx.x / a.group;
  c0 = threadIdx.x % a.group;
  t = (int)tok;
  return tok < a.T;
}

// Rows [n_valid, S) hold no slot; the token whose slots would be numbered so zeroes them.
template <typename E, int V>
__device__ __forceinline__ void zero_tail(const RowsArgs& a, int t, int c0) {
  if (!a.zero) return;
  const int64_t end = ((int64_t)t + 1) * a.k;
  Piece<E, V> p;
  p.zero();
  for (int64_t row = max((int64_t)__ldcg(a.hdr + HDR_NVALID), (int64_t)t * a.k); row < end; ++row)
    for (int c = c0; c < a.n; c += a.group) p.store(a.out, row * a.n + c);
}

// Bytes are moved, whatever the type.
template <int V>
__global__ void __launch_bounds__(kPThreads) permute_kernel(const RowsArgs a) {
  using P = Piece<uint16_t, V>;
  pdl_wait();
  pdl_trigger();
  int t, c0;
  if (!group_token(a, t, c0)) return;
  const int* rows = a.slot_row + (int64_t)t * a.k;
  constexpr int U = 4;  // loads in flight
  for (int c = c0; c < a.n; c += U * a.group) {
    P p[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * a.group < a.n) p[u].load(a.in, (int64_t)t * a.n + c + u * a.group);
    for (int j = 0; j < a.k; ++j) {
      const int row = __ldcg(rows + j);
      if (row < 0) continue;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (c + u * a.group < a.n) p[u].store(a.out, (int64_t)row * a.n + c + u * a.group);
    }
  }
  zero_tail<uint16_t, V>(a, t, c0);
}

// J rows of a token at a time and U pieces of each. Every load is made, so that all are in flight
// together (a branch around each kept them apart: 33 -> 39 us for 4099 tokens of 8 x 2048): in
// place of a row that is not there its neighbour again, dropped where it would be added.
template <typename E, int V, int J, int U>
__global__ void __launch_bounds__(kPThreads) unpermute_kernel(const RowsArgs a) {
  using P = Piece<E, V>;
  pdl_wait();
  pdl_trigger();
  int t, c0;
  if (!group_token(a, t, c0)) return;
  const int64_t s0 = (int64_t)t * a.k;
  int from[J];
  float w[J];
  bool there[J];
  auto places = [&](int j0) {
    int last = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = j0 + j < a.k ? __ldcg(a.slot_row + s0 + j0 + j) : -1;
      there[j] = row >= 0;
      from[j] = there[j] ? row : last;
      last = from[j];
      w[j] = a.w && j0 + j < a.k ? __ldcg(a.w + s0 + j0 + j) : 1.f;
    }
  };
  places(0);
  for (int c = c0; c < a.n; c += U * a.group) {
    float acc[U][P::N] = {};
    for (int j0 = 0; j0 < a.k; j0 += J) {
      if (a.k > J) places(j0);
      P p[U][J];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          p[u][j].load(a.in, (int64_t)from[j] * a.n + min(c + u * a.group, a.n - 1));
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          float f[P::N];
          p[u][j].to(f);
#pragma unroll
          for (int i = 0; i < P::N; ++i) acc[u][i] += there[j] ? w[j] * f[i] : 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      P p;
      p.from(acc[u]);
      if (c + u * a.group < a.n) p.store(a.out, (int64_t)t * a.n + c + u * a.group);
    }
  }
}

// The dot products are summed in fp32: in a thread over its columns, then over the group's
// threads in a tree of fixed shape.
template <typename E, int V, int J, int U>
__global__ void __launch_bounds__(kPThreads) unpermute_backward_kernel(const RowsArgs a) {
  using P = Piece<E, V>;
  __shared__ float part[kPThreads / 32][J];
  pdl_wait();
  pdl_trigger();
  int t, c0;
  const bool mine = group_token(a, t, c0);
  const int64_t s0 = (int64_t)t * a.k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int j0 = 0; j0 < a.k; j0 += J) {
    float dot[J] = {};
    if (mine) {
      int row[J];
      float w[J];
#pragma unroll
      for (int j = 0; j < J; ++j) row[j] = j0 + j < a.k ? __ldcg(a.slot_row + s0 + j0 + j) : -1;
#pragma unroll
      for (int j = 0; j < J; ++j) w[j] = row[j] >= 0 && a.w ? __ldcg(a.w + s0 + j0 + j) : 1.f;
      for (int c = c0; c < a.n; c += U * a.group) {
        P d[U], o[U][J];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int cu = c + u * a.group;
          d[u].zero();
          if (cu < a.n) d[u].load(a.dy, (int64_t)t * a.n + cu);
          if (a.dw)
#pragma unroll
            for (int j = 0; j < J; ++j) {
              o[u][j].zero();
              if (row[j] >= 0 && cu < a.n) o[u][j].load(a.in, (int64_t)row[j] * a.n + cu);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int cu = c + u * a.group;
          float g[P::N];
          d[u].to(g);
          if (a.out)
#pragma unroll
            for (int j = 0; j < J; ++j) {
              if (row[j] < 0 || cu >= a.n) continue;
              float f[P::N];
#pragma unroll
              for (int i = 0; i < P::N; ++i) f[i] = w[j] * g[i];
              P p;
              p.from(f);
              p.store(a.out, (int64_t)row[j] * a.n + cu);
            }
          if (a.dw)
#pragma unroll
            for (int j = 0; j < J; ++j) {
              float f[P::N];
              o[u][j].to(f);
#pragma unroll
              for (int i = 0; i < P::N; ++i) dot[j] += row[j] >= 0 ? f[i] * g[i] : 0.f;
            }
        }
      }
    }
    if (a.dw) {
#pragma unroll
      for (int j = 0; j < J; ++j)
        for (int m = min(a.group, 32) / 2; m; m /= 2) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], m);
      if (a.group > 32) {
        __syncthreads();  // the sums of the rows before have been read
        if (lane == 0)
#pragma unroll
          for (int j = 0; j < J; ++j) part[warp][j] = dot[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < J; ++j) {
          dot[j] = 0.f;
          if (c0 == 0)
            for (int q = 0; q < a.group / 32; ++q) dot[j] += part[warp + q][j];
        }
      }
      if (mine && c0 == 0)
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (j0 + j < a.k) a.dw[s0 + j0 + j] = dot[j];
    }
  }
  if (mine && a.out) zero_tail<E, V>(a, t, c0);
}

// A warp per token. An expert's logit takes every choice that names it, so that ids that are
// not distinct add up, as the formula says; ids outside [0, E) take no part.
__global__ void __launch_bounds__(256) topk_softmax_backward_kernel(const float* dw, const int* ids, const float* w,
                                                                    int T, int E, int k, float* dl) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= T) return;
  int id = -1;
  float p = 0.f, d = 0.f;  // choice `lane`
  if (lane < k) {
    const int v = __ldcg(ids + t * k + lane);
    if (v >= 0 && v < E) {
      id = v;
      p = __ldcg(w + t * k + lane);
      d = __ldcg(dw + t * k + lane);
    }
  }
  float mean = p * d;
  for (int m = 16; m; m /= 2) mean += __shfl_xor_sync(0xffffffffu, mean, m);
  const float g = p * (d - mean);
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    float s = 0.f;
    for (int j = 0; j < k; ++j) {
      const int ij = __shfl_sync(0xffffffffu, id, j);
      const float gj = __shfl_sync(0xffffffffu, g, j);
      if (ij == e) s += gj;
    }
    if (e < E) dl[t * E + e] = s;
  }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
static int elem_size(int dtype) { return dtype == MOE_DTYPE_FP32 ? 4 : 2; }

// The widest piece that divides a row and that every pointer is aligned to.
static int piece_bytes(int64_t row_bytes, std::initializer_list<const void*> ptrs) {
  int v = 16;
  for (const void* p : ptrs)
    while (reinterpret_cast<uintptr_t>(p) % v) v /= 2;
  while (row_bytes % v) v /= 2;
  return v;
}

static int check_rows(const moe_lora_align_t* al, int dtype, int H, AlignLayout* a) {
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16 && dtype != MOE_DTYPE_FP32) return MOE_LORA_ERR_INVALID_ARG;
  if (H < 1) return MOE_LORA_ERR_INVALID_ARG;
  if (H > (1 << 24)) return MOE_LORA_ERR_UNSUPPORTED;
  return check_align(al, a);
}

static RowsArgs rows_args(const moe_lora_align_t* al, const AlignLayout& a, int dtype, int H, int v) {
  const AlignView view = align_view(al->buf, a);
  RowsArgs r = {};
  r.hdr = view.hdr;
  r.slot_row = view.slot_row;
  r.T = al->T;
  r.k = al->k;
  r.n = (int)((int64_t)H * elem_size(dtype) / v);
  // threads per token: as many as a row has pieces, up to a CTA; with enough tokens for every SM
  // (two for each of 152: a fixed number, so that dw's order goes by the shape alone) the fewest
  // rounds' worth of idle threads, the larger group where equal
  r.group = 1;
  while (r.group < kPThreads && r.group < r.n) r.group *= 2;
  const auto threads = [&](int g) { return ceil_div(r.n, g) * g; };
  for (int g = r.group / 2; g >= 32 && r.T >= 304; g /= 2)
    if (threads(g) < threads(r.group)) r.group = g;
  return r;
}

template <typename K>
static int launch_rows(K kernel, const RowsArgs& a, cudaStream_t stream) {
  return launch_pdl(kernel, (unsigned)ceil_div(a.T, kPThreads / a.group), kPThreads, 0, stream, true, a);
}

// Rows in flight by the choices per token; widths that no 16-byte piece divides have one form.
template <typename E>
static int launch_unpermute(const RowsArgs& a, int v, cudaStream_t s) {
  constexpr int kLeast = sizeof(E) == 4 ? 4 : 2;
  if (v == 16)
    return a.k <= 2   ? launch_rows(unpermute_kernel<E, 16, 2, 2>, a, s)
           : a.k <= 4 ? launch_rows(unpermute_kernel<E, 16, 4, 2>, a, s)
                      : launch_rows(unpermute_kernel<E, 16, 8, 1>, a, s);
  if (v == 8) return launch_rows(unpermute_kernel<E, 8, 8, 1>, a, s);
  if (v == 4 || sizeof(E) == 4) return launch_rows(unpermute_kernel<E, 4, 8, 1>, a, s);
  return launch_rows(unpermute_kernel<E, kLeast, 8, 1>, a, s);
}
template <typename E>
static int launch_unpermute_backward(const RowsArgs& a, int v, cudaStream_t s) {
  constexpr int kLeast = sizeof(E) == 4 ? 4 : 2;
  if (v == 16)
    return a.k <= 2 ? launch_rows(unpermute_backward_kernel<E, 16, 2, 2>, a, s)
                    : launch_rows(unpermute_backward_kernel<E, 16, 4, 1>, a, s);
  if (v == 8) return launch_rows(unpermute_backward_kernel<E, 8, 4, 1>, a, s);
  if (v == 4 || sizeof(E) == 4) return launch_rows(unpermute_backward_kernel<E, 4, 4, 1>, a, s);
  return launch_rows(unpermute_backward_kernel<E, kLeast, 4, 1>, a, s);
}

static bool misaligned(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % elem_size(dtype) != 0; }

}  // namespace moe_lora

extern "C" int moe_permute(const void* x, int dtype, const moe_lora_align_t* al, int H, int row_flags, void* xs,
                           moe_lora_stream_t stream) {
  using namespace moe_lora;
  AlignLayout a;
  int st = check_rows(al, dtype, H, &a);
  if (st != MOE_LORA_OK) return st;
  if (row_flags & ~MOE_ROWS_ZERO_DROPPED) return MOE_LORA_ERR_INVALID_ARG;
  if (al->T == 0) return MOE_LORA_OK;
  if (!x || !xs || misaligned(x, dtype) || misaligned(xs, dtype)) return MOE_LORA_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  const int v = piece_bytes((int64_t)H * elem_size(dtype), {x, xs});
  RowsArgs r = rows_args(al, a, dtype, H, v);
  r.in = x;
  r.out = xs;
  r.zero = row_flags & MOE_ROWS_ZERO_DROPPED;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return v == 16  ? launch_rows(permute_kernel<16>, r, s)
         : v == 8 ? launch_rows(permute_kernel<8>, r, s)
         : v == 4 ? launch_rows(permute_kernel<4>, r, s)
                  : launch_rows(permute_kernel<2>, r, s);
}

extern "C" int moe_unpermute(const void* o, int dtype, const moe_lora_align_t* al, const float* w, int H, void* y,
                             moe_lora_stream_t stream) {
  using namespace moe_lora;
  AlignLayout a;
  int st = check_rows(al, dtype, H, &a);
  if (st != MOE_LORA_OK) return st;
  if (al->T == 0) return MOE_LORA_OK;
  if (!o || !y || misaligned(o, dtype) || misaligned(y, dtype) || misaligned(w, MOE_DTYPE_FP32))
    return MOE_LORA_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  const int v = piece_bytes((int64_t)H * elem_size(dtype), {o, y});
  RowsArgs r = rows_args(al, a, dtype, H, v);
  r.in = o;
  r.w = w;
  r.out = y;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == MOE_DTYPE_BF16   ? launch_unpermute<__nv_bfloat16>(r, v, s)
         : dtype == MOE_DTYPE_FP16 ? launch_unpermute<__half>(r, v, s)
                                   : launch_unpermute<float>(r, v, s);
}

extern "C" int moe_unpermute_backward(const void* dy, const void* o, int dtype, const moe_lora_align_t* al,
                                      const float* w, int H, int row_flags, void* d_o, float* dw,
                                      moe_lora_stream_t stream) {
  using namespace moe_lora;
  AlignLayout a;
  int st = check_rows(al, dtype, H, &a);
  if (st != MOE_LORA_OK) return st;
  if (row_flags & ~MOE_ROWS_ZERO_DROPPED) return MOE_LORA_ERR_INVALID_ARG;
  if (al->T == 0 || (!d_o && !dw)) return MOE_LORA_OK;
  if (!dy || (dw && !o) || misaligned(dy, dtype) || misaligned(o, dtype) || misaligned(d_o, dtype) ||
      misaligned(w, MOE_DTYPE_FP32) || misaligned(dw, MOE_DTYPE_FP32))
    return MOE_LORA_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  const int v = piece_bytes((int64_t)H * elem_size(dtype), {dy, dw ? o : nullptr, d_o});
  RowsArgs r = rows_args(al, a, dtype, H, v);
  r.in = o;
  r.dy = dy;
  r.w = w;
  r.out = d_o;
  r.dw = dw;
  r.zero = row_flags & MOE_ROWS_ZERO_DROPPED;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dtype == MOE_DTYPE_BF16   ? launch_unpermute_backward<__nv_bfloat16>(r, v, s)
         : dtype == MOE_DTYPE_FP16 ? launch_unpermute_backward<__half>(r, v, s)
                                   : launch_unpermute_backward<float>(r, v, s);
}

extern "C" int moe_topk_softmax_backward(const float* dw, const int32_t* ids, const float* w, int T, int E, int k,
                                         float* dlogits, moe_lora_stream_t stream) {
  using namespace moe_lora;
  int st = check_route_args(dlogits, T, E, k, ids, w);
  if (st != MOE_LORA_OK) return st;
  if (T == 0) return MOE_LORA_OK;
  if (!dw) return MOE_LORA_ERR_INVALID_ARG;
  if ((st = check_device()) != MOE_LORA_OK) return st;
  return launch_pdl(topk_softmax_backward_kernel, (unsigned)ceil_div(T, 8), 256, 0,
                    reinterpret_cast<cudaStream_t>(stream), true, dw, ids, w, T, E, k, dlogits);
}
