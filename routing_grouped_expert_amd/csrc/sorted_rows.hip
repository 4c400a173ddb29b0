// Token rows into expert-sorted order and back with the routing weights
// applied, and the gradients: what surrounds expert products that run outside
// this library (the sort-by-expert dispatch and the weighted sum back of the
// minimind issue #835 page, "It is removable in plain PyTorch", and "Summary").
//
//   dispatch          x_sorted[p] = x[t],               p = row_sorted[t k + j]
//   weighted combine  out[t] = sum_j w[t, j] y[p]       (fp32, slot order, one rounding)
//   its gradient      d_y[p] = w[t, j] d_out[t];  d_w[t, j] = <d_out[t], y[p]>
//   softmax gradient  d_logits[t, e_j] = w_j (d_w_j - sum_i w_i d_w_i), 0 elsewhere
//
// The gradient of the dispatch is the plain combine (combine.hip).  Every
// kernel walks tokens, not sorted rows: a token's row is then read (or written)
// once while its k sorted rows, each contiguous, are touched once, and since
// row_sorted is a bijection no two threads write the same place, so there are
// no atomics and the results are the same on every run.  Slots whose position
// is outside [0, M) (-1 for experts outside an expert-parallel share) move and
// add nothing.
#include "rows.h"

#include <type_traits>

namespace moe {
namespace {

constexpr int kThreads = 256;

// The token and the 16-byte chunk of its row that a thread of a flat grid over
// all n * nch chunks owns.  The block's first token is found by one uniform
// 64-bit division; a thread's own offset stays small.
__device__ __forceinline__ bool own_chunk(int64_t n, int nch, int64_t &t, int &c) {
  const int64_t base = (int64_t)blockIdx.x * kThreads;
  const int64_t t0 = base / nch;
  const uint32_t r = (uint32_t)(base - t0 * nch) + threadIdx.x;
  const uint32_t dt = r / (uint32_t)nch;
  t = t0 + dt;
  c = (int)(r - dt * (uint32_t)nch);
  return t < n;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const T *__restrict__ x,
                                                            const int32_t *__restrict__ row_sorted,
                                                            T *__restrict__ xs, int64_t N, int K,
                                                            int H) {
  constexpr int CH = chunk_elems<T>();
  int64_t t;
  int c;
  if (!own_chunk(N, H / CH, t, c)) return;
  const uint32_t M = (uint32_t)(N * K);
  const u32x4_t v = *reinterpret_cast<const u32x4_t *>(x + t * H + (int64_t)c * CH);
  for (int j = 0; j < K; ++j) {
    const uint32_t p = (uint32_t)row_sorted[t * K + j];
    if (p < M) *reinterpret_cast<u32x4_t *>(xs + (int64_t)p * H + (int64_t)c * CH) = v;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void combine_weighted_kernel(
    const T *__restrict__ y, const int32_t *__restrict__ row_sorted, const void *__restrict__ w,
    bool w_bf16, T *__restrict__ out, int64_t N, int K, int H) {
  constexpr int CH = chunk_elems<T>();
  int64_t t;
  int c;
  if (!own_chunk(N, H / CH, t, c)) return;
  const uint32_t M = (uint32_t)(N * K);
  float acc[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) acc[i] = 0.f;
  for (int j = 0; j < K; ++j) {
    const uint32_t p = (uint32_t)row_sorted[t * K + j];
    if (p < M) {
      const float wj = weight_at(w, w_bf16, t * K + j);
      float f[CH];
      unpack(*reinterpret_cast<const u32x4_t *>(y + (int64_t)p * H + (int64_t)c * CH), f);
#pragma unroll
      for (int i = 0; i < CH; ++i) acc[i] = fmaf(wj, f[i], acc[i]);
    }
  }
  *reinterpret_cast<u32x4_t *>(out + t * H + (int64_t)c * CH) = pack(acc);
}

// One wave a token: it keeps a piece of d_out in registers while it passes
// over the same piece of the token's k expert rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void combine_weighted_backward_kernel(
    const T *__restrict__ d_out, const T *__restrict__ y, const int32_t *__restrict__ row_sorted,
    const void *__restrict__ w, bool w_bf16, T *__restrict__ dy, float *__restrict__ dw, int64_t N,
    int K, int H) {
  constexpr int CH = chunk_elems<T>();
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (t >= N) return;  // a whole wave
  const uint32_t M = (uint32_t)(N * K);
  const int nch = H / CH;
  for (int j = 0; j < K; ++j) {
    const uint32_t p = (uint32_t)row_sorted[t * K + j];
    float dot = 0.f;
    if (p < M) {  // the same for the whole wave
      const float wj = weight_at(w, w_bf16, t * K + j);
      for (int c = lane; c < nch; c += 64) {
        float d[CH], f[CH];
        unpack(*reinterpret_cast<const u32x4_t *>(d_out + t * H + (int64_t)c * CH), d);
        unpack(*reinterpret_cast<const u32x4_t *>(y + (int64_t)p * H + (int64_t)c * CH), f);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          dot = fmaf(d[i], f[i], dot);
          d[i] *= wj;
        }
        *reinterpret_cast<u32x4_t *>(dy + (int64_t)p * H + (int64_t)c * CH) = pack(d);
      }
    }
    dot = wave_sum_f32(dot);
    if (lane == 0) dw[t * K + j] = dot;
  }
}

// One thread per element of d_logits.
template <typename W>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const float *__restrict__ dw, const int32_t *__restrict__ topk_idx, const W *__restrict__ w,
    W *__restrict__ d_logits, int64_t N, int E, int K) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= N * E) return;
  const int64_t t = i / E;
  const int e = (int)(i - t * E);
  float s = 0.f, wm = 0.f, dm = 0.f;
  for (int j = 0; j < K; ++j) {
    const float wj = to_f32(w[t * K + j]), dj = dw[t * K + j];
    s = fmaf(wj, dj, s);
    if (topk_idx[t * K + j] == e) {
      wm = wj;
      dm = dj;
    }
  }
  d_logits[i] = from_f32<W>(wm * (dm - s));
}

template <typename T> int64_t chunk_blocks(int64_t n, int hidden) {
  return (n * (hidden / (16 / (int)sizeof(T))) + kThreads - 1) / kThreads;
}

}  // namespace

hipError_t launch_dispatch(const void *x, const int32_t *row_sorted, void *x_sorted,
                           moe_dtype_t dt, int64_t n_tokens, int topk, int hidden, hipStream_t s) {
  auto go = [&](auto tag) {
    using T = decltype(tag);
    hipLaunchKernelGGL(dispatch_kernel<T>, dim3((unsigned)chunk_blocks<T>(n_tokens, hidden)),
                       dim3(kThreads), 0, s, reinterpret_cast<const T *>(x), row_sorted,
                       reinterpret_cast<T *>(x_sorted), n_tokens, topk, hidden);
  };
  if (dt == MOE_BF16) go(bf16_t()); else go(float());
  return hipGetLastError();
}

hipError_t launch_combine_weighted(const void *y_sorted, const int32_t *row_sorted,
                                   const void *topk_w, moe_dtype_t w_dt, void *out, moe_dtype_t dt,
                                   int64_t n_tokens, int topk, int hidden, hipStream_t s) {
  auto go = [&](auto tag) {
    using T = decltype(tag);
    hipLaunchKernelGGL(combine_weighted_kernel<T>,
                       dim3((unsigned)chunk_blocks<T>(n_tokens, hidden)), dim3(kThreads), 0, s,
                       reinterpret_cast<const T *>(y_sorted), row_sorted, topk_w,
                       w_dt == MOE_BF16, reinterpret_cast<T *>(out), n_tokens, topk, hidden);
  };
  if (dt == MOE_BF16) go(bf16_t()); else go(float());
  return hipGetLastError();
}

hipError_t launch_combine_weighted_backward(const void *d_out, const void *y_sorted,
                                            const int32_t *row_sorted, const void *topk_w,
                                            moe_dtype_t w_dt, void *d_y_sorted, float *d_topk_w,
                                            moe_dtype_t dt, int64_t n_tokens, int topk, int hidden,
                                            hipStream_t s) {
  const unsigned blocks = (unsigned)((n_tokens + kThreads / 64 - 1) / (kThreads / 64));
  auto go = [&](auto tag) {
    using T = decltype(tag);
    hipLaunchKernelGGL(combine_weighted_backward_kernel<T>, dim3(blocks), dim3(kThreads), 0, s,
                       reinterpret_cast<const T *>(d_out), reinterpret_cast<const T *>(y_sorted),
                       row_sorted, topk_w, w_dt == MOE_BF16, reinterpret_cast<T *>(d_y_sorted),
                       d_topk_w, n_tokens, topk, hidden);
  };
  if (dt == MOE_BF16) go(bf16_t()); else go(float());
  return hipGetLastError();
}

hipError_t launch_route_backward(const float *d_topk_w, const int32_t *topk_idx,
                                 const void *topk_w, void *d_logits, moe_dtype_t w_dt,
                                 int64_t n_tokens, int n_experts, int topk, hipStream_t s) {
  const unsigned blocks = (unsigned)((n_tokens * n_experts + kThreads - 1) / kThreads);
  auto go = [&](auto tag) {
    using W = decltype(tag);
    hipLaunchKernelGGL(route_backward_kernel<W>, dim3(blocks), dim3(kThreads), 0, s, d_topk_w,
                       topk_idx, reinterpret_cast<const W *>(topk_w),
                       reinterpret_cast<W *>(d_logits), n_tokens, n_experts, topk);
  };
  if (w_dt == MOE_BF16) go(bf16_t()); else go(float());
  return hipGetLastError();
}

}  // namespace moe
