// Token rows into expert-sorted order and back with the routing weights
// applied, and the gradients: what surrounds expert products that run outside
// this library (the sort-by-expert dispatch and the weighted sum back of the
// minimind issue #835 page, "It is removable in plain PyTorch", and "Summary").
//
//   dispatch          x_sorted[p] = x[t],               p = row_sorted[t k + j]
//   weighted combine  out[t] = sum_j w[t, j] y[p]       (fp32, slot order, one rounding)
//   its gradient      d_y[p] = w[t, j] d_out[t];  d_w[t, j] = <d_out[t], y[p]>
//   softmax gradient  d_logits[t, e_j] = w_j (d_w_j - sum_i w_i d_w_i), 0 elsewhere
//                     (summed where several slots name one expert)
//
// The gradient of the dispatch is the plain combine (combine.hip).  Every
// kernel walks tokens, not sorted rows: a token's row is then read (or written)
// once while its k sorted rows, each contiguous, are touched once, and since
// row_sorted is a bijection no two threads write the same place, so there are
// no atomics and the results are the same on every run.  Slots whose position
// is outside [0, M) (-1 for experts outside an expert-parallel share) move and
// add nothing.  A token's slots are taken up to eight at a time, their
// positions and then their rows all in flight.  All of it is bound by HBM, at
// the rate of a large copy (5.1 - 5.4 TB/s): 16384 tokens x 4096 bf16, 8 slots:
// dispatch (1.2 GB) 230 us, 5.3 TB/s; gradient (2.3 GB) 452 us, 5.1 TB/s; 4096
// x 2880, 4 slots: weighted combine (118 MB, above a copy's rate, so partly from
// a cache) 21 us.  Small batches cost 2.2 - 5.8 us a kernel.
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

template <typename T> __device__ __forceinline__ u32x4_t load16(const T *p) {
  return *reinterpret_cast<const u32x4_t *>(p);
}
template <typename T> __device__ __forceinline__ void store16(T *p, u32x4_t v) {
  *reinterpret_cast<u32x4_t *>(p) = v;
}

// Positions of the slots j0 .. j0 + JB - 1 of token t; kNone past the last
// slot and for slots that point nowhere.
constexpr uint32_t kNone = 0xffffffffu;
template <int JB>
__device__ __forceinline__ void slot_rows(const int32_t *__restrict__ row_sorted, int64_t t, int K,
                                          int j0, uint32_t M, uint32_t (&p)[JB]) {
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    p[j] = j0 + j < K ? (uint32_t)row_sorted[t * K + j0 + j] : kNone;
    if (p[j] >= M) p[j] = kNone;
  }
}

template <typename T, int JB>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(const T *__restrict__ x,
                                                            const int32_t *__restrict__ row_sorted,
                                                            T *__restrict__ xs, int64_t N, int K,
                                                            int H) {
  constexpr int CH = chunk_elems<T>();
  int64_t t;
  int c;
  if (!own_chunk(N, H / CH, t, c)) return;
  const u32x4_t v = load16(x + t * H + (int64_t)c * CH);
  for (int j0 = 0; j0 < K; j0 += JB) {
    uint32_t p[JB];
    slot_rows<JB>(row_sorted, t, K, j0, (uint32_t)(N * K), p);
#pragma unroll
    for (int j = 0; j < JB; ++j)
      if (p[j] != kNone) store16(xs + (int64_t)p[j] * H + (int64_t)c * CH, v);
  }
}

template <typename T, int JB>
__global__ __launch_bounds__(kThreads) void combine_weighted_kernel(
    const T *__restrict__ y, const int32_t *__restrict__ row_sorted, const void *__restrict__ w,
    bool w_bf16, T *__restrict__ out, int64_t N, int K, int H) {
  constexpr int CH = chunk_elems<T>();
  int64_t t;
  int c;
  if (!own_chunk(N, H / CH, t, c)) return;
  float acc[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < K; j0 += JB) {
    uint32_t p[JB];
    slot_rows<JB>(row_sorted, t, K, j0, (uint32_t)(N * K), p);
    u32x4_t v[JB];
    float wj[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      wj[j] = p[j] != kNone ? weight_at(w, w_bf16, t * K + j0 + j) : 0.f;
      v[j] = p[j] != kNone ? load16(y + (int64_t)p[j] * H + (int64_t)c * CH)
                           : u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      float f[CH];
      unpack(v[j], f);
#pragma unroll
      for (int i = 0; i < CH; ++i) acc[i] = fmaf(wj[j], f[i], acc[i]);
    }
  }
  store16(out + t * H + (int64_t)c * CH, pack(acc));
}

// The expert rows are read once and past the caches (fp32, 4095 tokens x 1416, 6
// slots: 66 -> 60 us); non-temporal stores made it 68, and changed nothing or
// lost up to 6 % elsewhere.  WPT waves a token: each keeps a piece of d_out in
// registers while it passes over the same piece of the token's expert rows, JB
// at a time.
template <typename T, int JB, int WPT>
__global__ __launch_bounds__(kThreads) void combine_weighted_backward_kernel(
    const T *__restrict__ d_out, const T *__restrict__ y, const int32_t *__restrict__ row_sorted,
    const void *__restrict__ w, bool w_bf16, T *__restrict__ dy, float *__restrict__ dw, int64_t N,
    int K, int H) {
  constexpr int CH = chunk_elems<T>(), TPB = kThreads / 64 / WPT;  // tokens a workgroup
  __shared__ float part[kThreads / 64][JB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * TPB + wave / WPT;
  const bool live = t < N;  // (waves past the last token still reach the barriers)
  const int nch = H / CH, first = wave % WPT * 64 + lane;
  for (int j0 = 0; j0 < K; j0 += JB) {
    uint32_t p[JB];
    slot_rows<JB>(row_sorted, t, live ? K : 0, j0, (uint32_t)(N * K), p);
    float wj[JB], dot[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      wj[j] = p[j] != kNone ? weight_at(w, w_bf16, t * K + j0 + j) : 0.f;
      dot[j] = 0.f;
    }
    for (int c = first; live && c < nch; c += 64 * WPT) {
      const int64_t at = (int64_t)c * CH;
      const u32x4_t dv = *reinterpret_cast<const u32x4_t *>(d_out + t * H + at);
      u32x4_t v[JB];
#pragma unroll
      for (int j = 0; j < JB; ++j)
        v[j] = p[j] != kNone ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(
                                   y + (int64_t)p[j] * H + at))
                             : u32x4_t{0u, 0u, 0u, 0u};
      float d[CH];
      unpack(dv, d);
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        if (p[j] == kNone) continue;  // the same for the whole wave
        float f[CH];
        unpack(v[j], f);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          dot[j] = fmaf(d[i], f[i], dot[j]);
          f[i] = wj[j] * d[i];
        }
        store16(dy + (int64_t)p[j] * H + at, pack(f));
      }
    }
#pragma unroll
    for (int j = 0; j < JB; ++j) dot[j] = wave_sum_f32(dot[j]);
    if constexpr (WPT == 1) {
#pragma unroll
      for (int j = 0; j < JB; ++j)
        if (live && lane == 0 && j0 + j < K) dw[t * K + j0 + j] = dot[j];
    } else {
      if (j0 > 0) __syncthreads();
#pragma unroll
      for (int j = 0; j < JB; ++j)
        if (lane == 0) part[wave][j] = dot[j];
      __syncthreads();
      if (live && wave % WPT == 0 && lane < JB && j0 + lane < K) {
        float s = part[wave][lane];
#pragma unroll
        for (int q = 1; q < WPT; ++q) s += part[wave + q][lane];
        dw[t * K + j0 + lane] = s;
      }
    }
  }
}

// C consecutive elements of one token's d_logits a thread: 16 bytes where rows
// are whole 16-byte chunks, else one element (16384 tokens x 64 experts bf16, 8
// slots: 4.0 us against 7.0).
template <typename W, int C>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const float *__restrict__ dw, const int32_t *__restrict__ topk_idx, const W *__restrict__ w,
    W *__restrict__ d_logits, int64_t N, int E, int K) {
  int64_t t;
  int c;
  if (!own_chunk(N, E / C, t, c)) return;
  float s = 0.f;
  for (int j = 0; j < K; ++j) s = fmaf(to_f32(w[t * K + j]), dw[t * K + j], s);
  float v[C];
#pragma unroll
  for (int i = 0; i < C; ++i) v[i] = 0.f;
  for (int j = 0; j < K; ++j) {
    const int e = topk_idx[t * K + j] - c * C;
    const float d = to_f32(w[t * K + j]) * (dw[t * K + j] - s);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] += e == i ? d : 0.f;
  }
  W *out = d_logits + t * E + (int64_t)c * C;
  if constexpr (C == 1) *out = from_f32<W>(v[0]);
  else store16(out, pack(v));
}

template <typename T> int64_t chunk_blocks(int64_t n, int hidden) {
  return (n * (hidden / (16 / (int)sizeof(T))) + kThreads - 1) / kThreads;
}

// Calls go(T(), JB) for the row type and the number of slots taken at a time.
template <typename F> void by_slots(moe_dtype_t dt, int topk, F go) {
  auto jb = [&](auto tag) {
    if (topk == 1) go(tag, std::integral_constant<int, 1>());
    else if (topk == 2) go(tag, std::integral_constant<int, 2>());
    else if (topk <= 4) go(tag, std::integral_constant<int, 4>());
    else go(tag, std::integral_constant<int, 8>());
  };
  if (dt == MOE_BF16) jb(bf16_t()); else jb(float());
}

}  // namespace

hipError_t launch_dispatch(const void *x, const int32_t *row_sorted, void *x_sorted,
                           moe_dtype_t dt, int64_t n_tokens, int topk, int hidden, hipStream_t s) {
  by_slots(dt, topk, [&](auto tag, auto jb) {
    using T = decltype(tag);
    hipLaunchKernelGGL((dispatch_kernel<T, decltype(jb)::value>),
                       dim3((unsigned)chunk_blocks<T>(n_tokens, hidden)), dim3(kThreads), 0, s,
                       reinterpret_cast<const T *>(x), row_sorted,
                       reinterpret_cast<T *>(x_sorted), n_tokens, topk, hidden);
  });
  return hipGetLastError();
}

hipError_t launch_combine_weighted(const void *y_sorted, const int32_t *row_sorted,
                                   const void *topk_w, moe_dtype_t w_dt, void *out, moe_dtype_t dt,
                                   int64_t n_tokens, int topk, int hidden, hipStream_t s) {
  by_slots(dt, topk, [&](auto tag, auto jb) {
    using T = decltype(tag);
    hipLaunchKernelGGL((combine_weighted_kernel<T, decltype(jb)::value>),
                       dim3((unsigned)chunk_blocks<T>(n_tokens, hidden)), dim3(kThreads), 0, s,
                       reinterpret_cast<const T *>(y_sorted), row_sorted, topk_w,
                       w_dt == MOE_BF16, reinterpret_cast<T *>(out), n_tokens, topk, hidden);
  });
  return hipGetLastError();
}

hipError_t launch_combine_weighted_backward(const void *d_out, const void *y_sorted,
                                            const int32_t *row_sorted, const void *topk_w,
                                            moe_dtype_t w_dt, void *d_y_sorted, float *d_topk_w,
                                            moe_dtype_t dt, int64_t n_tokens, int topk, int hidden,
                                            hipStream_t s) {
  by_slots(dt, topk, [&](auto tag, auto jb) {
    using T = decltype(tag);
    constexpr int JB = decltype(jb)::value;
    auto run = [&](auto wpt) {
      constexpr int WPT = decltype(wpt)::value, TPB = kThreads / 64 / WPT;
      hipLaunchKernelGGL((combine_weighted_backward_kernel<T, JB, WPT>),
                         dim3((unsigned)((n_tokens + TPB - 1) / TPB)), dim3(kThreads), 0, s,
                         reinterpret_cast<const T *>(d_out), reinterpret_cast<const T *>(y_sorted),
                         row_sorted, topk_w, w_dt == MOE_BF16, reinterpret_cast<T *>(d_y_sorted),
                         d_topk_w, n_tokens, topk, hidden);
    };
    // as many waves as cover the row once: 33 tokens of 2880 bf16 values 5.8 us
    // with four and 7.9 with one; 8000 of 512 (one wave's width) 49 and 31
    const int nch = hidden / (16 / (int)sizeof(T));
    if (nch <= 64) run(std::integral_constant<int, 1>());
    else if (nch <= 128) run(std::integral_constant<int, 2>());
    else run(std::integral_constant<int, 4>());
  });
  return hipGetLastError();
}

hipError_t launch_route_backward(const float *d_topk_w, const int32_t *topk_idx,
                                 const void *topk_w, void *d_logits, moe_dtype_t w_dt,
                                 int64_t n_tokens, int n_experts, int topk, hipStream_t s) {
  auto go = [&](auto tag, auto chunk) {
    using W = decltype(tag);
    constexpr int C = decltype(chunk)::value;
    const int64_t total = n_tokens * (n_experts / C);
    hipLaunchKernelGGL((route_backward_kernel<W, C>),
                       dim3((unsigned)((total + kThreads - 1) / kThreads)), dim3(kThreads), 0, s,
                       d_topk_w, topk_idx, reinterpret_cast<const W *>(topk_w),
                       reinterpret_cast<W *>(d_logits), n_tokens, n_experts, topk);
  };
  auto by_chunk = [&](auto tag) {
    constexpr int C = chunk_elems<decltype(tag)>();
    if (n_experts % C == 0) go(tag, std::integral_constant<int, C>());
    else go(tag, std::integral_constant<int, 1>());
  };
  if (w_dt == MOE_BF16) by_chunk(bf16_t()); else by_chunk(float());
  return hipGetLastError();
}

}  // namespace moe
