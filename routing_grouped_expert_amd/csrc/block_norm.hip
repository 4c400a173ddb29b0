// RMS norms around a block of layers in one pass over the token rows: the norm
// of the block's output with its gate, the residual scale and the residual sum,
// and the norm ahead of the next block; and the gradient of that step.
//
//   z = y * rstd(y) * w_post        rstd(u) = 1 / sqrt(mean(u^2) + eps)
//   x_out = x + residual_scale * gate * z
//   n_out = x_out * rstd(x_out) * w_pre
//
// Without w_post z is y itself, without y x_out is x, without w_pre there is no
// n_out.  The gate is one value a token or one a channel.
//
// Gradient, with xh = x_out * rstd_pre, yh = y * rstd_post, <> the mean over
// the row, g1 = d_n_out * w_pre, g2 = residual_scale * gate * d_x * w_post:
//   d_x = d_x_out + rstd_pre * (g1 - xh * <g1 xh>)
//   d_y = rstd_post * (g2 - yh * <g2 yh>)
//   d_w_pre = sum_t d_n_out * xh    d_w_post = sum_t residual_scale * gate * d_x * yh
//   d_gate = sum of residual_scale * d_x * z over the token's row, or over the tokens
// x_out is formed again from x and y in fp32, so the gradient sees the value
// the norm saw and not its rounding.
//
// A row is read once into registers (TPR threads a row, V 16-byte chunks a
// thread), summed across its threads in fp32 and written once; the step is
// bound by HBM: forward 16384 x 4096 bf16 (537 MB) 102 us, 5.2 TB/s, a copy's
// rate; backward (805 MB) 158 us, 5.1 TB/s; one token 3.2 us.  That holds for the
// backward pass up to 8192 values: the wider kernels pass the 128 registers that
// 1024 threads leave each, 114 (bf16) and 156 (fp32) of them go through scratch,
// and 2048 x 16384 takes 368 us in bf16 (1.1 TB/s) and 466 in fp32 (1.7 TB/s).
// Loading the next row ahead of the sums measured no faster (backward 164 -> 167
// us).  A workgroup takes rows in turn, so that the weights are loaded once and the
// column sums of the gradient are added up in registers; the workgroups' sums are
// then added in a fixed order by a second kernel, with no atomics.
#include "rows.h"

#include <type_traits>

namespace moe {
namespace {

// Sum over the TPR threads of a row.  Rows of more than a wave go through LDS;
// the two halves of `red` are used in turn, so one barrier a sum is enough.
// Every thread of the workgroup must call it.
template <int TPR, int WAVES, int NV>
__device__ __forceinline__ void row_sum(float (&v)[NV], float (&red)[2][WAVES][NV], int &half) {
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int m = (TPR < 64 ? TPR : 64) / 2; m >= 1; m >>= 1) v[i] += __shfl_xor(v[i], m);
  if constexpr (TPR > 64) {
    constexpr int WPR = TPR / 64;  // waves a row
    const int wave = threadIdx.x >> 6, first = wave / WPR * WPR;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) red[half][wave][i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < WPR; ++q) s += red[half][first + q][i];
      v[i] = s;
    }
    half ^= 1;
  }
}

template <typename T>
__device__ __forceinline__ u32x4_t load_chunk(const void *p, int64_t row, int H, int c) {
  return *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const T *>(p) + row * H +
                                            (int64_t)c * chunk_elems<T>());
}
template <typename T>
__device__ __forceinline__ void store_chunk(void *p, int64_t row, int H, int c, u32x4_t v) {
  *reinterpret_cast<u32x4_t *>(reinterpret_cast<T *>(p) + row * H +
                               (int64_t)c * chunk_elems<T>()) = v;
}
template <typename T> __device__ __forceinline__ float load_scalar(const void *p, int64_t i) {
  return to_f32(reinterpret_cast<const T *>(p)[i]);
}

constexpr int block_threads(int tpr) { return tpr > 256 ? tpr : 256; }

template <typename T, int TPR, int V>
__global__ __launch_bounds__(block_threads(TPR)) void block_norm_kernel(BlockNormArgs g) {
  constexpr int CH = chunk_elems<T>(), BT = block_threads(TPR), RPB = BT / TPR;
  __shared__ float red[2][BT / 64][1];
  int half = 0;
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int H = g.hidden, nch = H / CH;
  const float inv_h = 1.f / (float)H;
  const u32x4_t zero = {0u, 0u, 0u, 0u};

  u32x4_t wpost[V], wpre[V], gate[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane + i * TPR;
    const bool ok = c < nch;
    wpost[i] = ok && g.w_post ? load_chunk<T>(g.w_post, 0, H, c) : zero;
    wpre[i] = ok && g.w_pre ? load_chunk<T>(g.w_pre, 0, H, c) : zero;
    gate[i] = ok && g.gate_kind == MOE_GATE_CHANNEL ? load_chunk<T>(g.gate, 0, H, c) : zero;
  }

  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < g.n_tokens;
       row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + group;
    const bool live = row < g.n_tokens;
    u32x4_t xr[V], yr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = lane + i * TPR;
      const bool ok = live && c < nch;
      xr[i] = ok ? load_chunk<T>(g.x, row, H, c) : zero;
      yr[i] = ok && g.y ? load_chunk<T>(g.y, row, H, c) : zero;
    }
    float xv[V][CH];
#pragma unroll
    for (int i = 0; i < V; ++i) unpack(xr[i], xv[i]);
    if (g.y) {
      float ry = 1.f;
      if (g.w_post) {
        float ss[1] = {0.f};
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float yv[CH];
          unpack(yr[i], yv);
#pragma unroll
          for (int q = 0; q < CH; ++q) ss[0] = fmaf(yv[q], yv[q], ss[0]);
        }
        row_sum<TPR>(ss, red, half);
        ry = 1.f / sqrtf(fmaf(ss[0], inv_h, g.eps));
        if (g.rstd_post && live && lane == 0) g.rstd_post[row] = ry;
      }
      float sg = g.residual_scale;
      if (g.gate_kind == MOE_GATE_TOKEN && live) sg *= load_scalar<T>(g.gate, row);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = lane + i * TPR;
        float yv[CH], wv[CH], gv[CH];
        unpack(yr[i], yv);
        unpack(wpost[i], wv);
        unpack(gate[i], gv);
#pragma unroll
        for (int q = 0; q < CH; ++q) {
          float z = yv[q];
          if (g.w_post) z *= ry * wv[q];
          if (g.gate_kind == MOE_GATE_CHANNEL) z *= gv[q];
          xv[i][q] = fmaf(sg, z, xv[i][q]);
        }
        if (live && c < nch) store_chunk<T>(g.x_out, row, H, c, pack(xv[i]));
      }
    }
    if (g.w_pre) {
      float ss[1] = {0.f};
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < CH; ++q) ss[0] = fmaf(xv[i][q], xv[i][q], ss[0]);
      row_sum<TPR>(ss, red, half);
      const float rx = 1.f / sqrtf(fmaf(ss[0], inv_h, g.eps));
      if (g.rstd_pre && live && lane == 0) g.rstd_pre[row] = rx;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = lane + i * TPR;
        float wv[CH];
        unpack(wpre[i], wv);
#pragma unroll
        for (int q = 0; q < CH; ++q) xv[i][q] *= rx * wv[q];
        if (live && c < nch) store_chunk<T>(g.n_out, row, H, c, pack(xv[i]));
      }
    }
  }
}

template <typename T, int TPR, int V>
__global__ __launch_bounds__(block_threads(TPR)) void block_norm_backward_kernel(
    BlockNormArgs g) {
  constexpr int CH = chunk_elems<T>(), BT = block_threads(TPR), RPB = BT / TPR;
  __shared__ float red1[2][BT / 64][1];
  __shared__ float red2[2][BT / 64][2];
  __shared__ float cols[RPB > 1 ? BT * V * CH : 1];
  int half1 = 0, half2 = 0;
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int H = g.hidden, nch = H / CH;
  const float inv_h = 1.f / (float)H;
  const u32x4_t zero = {0u, 0u, 0u, 0u};

  u32x4_t wpost[V], wpre[V], gate[V];
  float a_pre[V][CH], a_post[V][CH], a_gate[V][CH];  // column sums of this thread's rows
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = lane + i * TPR;
    const bool ok = c < nch;
    wpost[i] = ok && g.w_post ? load_chunk<T>(g.w_post, 0, H, c) : zero;
    wpre[i] = ok && g.w_pre ? load_chunk<T>(g.w_pre, 0, H, c) : zero;
    gate[i] = ok && g.gate_kind == MOE_GATE_CHANNEL ? load_chunk<T>(g.gate, 0, H, c) : zero;
#pragma unroll
    for (int q = 0; q < CH; ++q) a_pre[i][q] = a_post[i][q] = a_gate[i][q] = 0.f;
  }

  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < g.n_tokens;
       row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + group;
    const bool live = row < g.n_tokens;
    u32x4_t xr[V], yr[V], nr[V], dr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = lane + i * TPR;
      const bool ok = live && c < nch;
      xr[i] = ok ? load_chunk<T>(g.x, row, H, c) : zero;
      yr[i] = ok && g.y ? load_chunk<T>(g.y, row, H, c) : zero;
      nr[i] = ok && g.w_pre ? load_chunk<T>(g.d_n_out, row, H, c) : zero;
      dr[i] = ok && g.d_x_out ? load_chunk<T>(g.d_x_out, row, H, c) : zero;
    }
    const float ry = live && g.w_post ? g.rstd_post[row] : 1.f;
    const float rx = live && g.w_pre ? g.rstd_pre[row] : 0.f;
    const float gt = live && g.gate_kind == MOE_GATE_TOKEN ? load_scalar<T>(g.gate, row) : 1.f;

    // xv: x_out * rstd_pre (with w_pre); dv: the gradient of x_out, which is that of x
    float xv[V][CH], dv[V][CH];
    float c1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float yv[CH], wv[CH], gv[CH], nv[CH], pv[CH];
      unpack(xr[i], xv[i]);
      unpack(yr[i], yv);
      unpack(wpost[i], wv);
      unpack(gate[i], gv);
      unpack(nr[i], nv);
      unpack(wpre[i], pv);
#pragma unroll
      for (int q = 0; q < CH; ++q) {
        if (g.y) {
          float z = yv[q];
          if (g.w_post) z *= ry * wv[q];
          if (g.gate_kind == MOE_GATE_CHANNEL) z *= gv[q];
          xv[i][q] = fmaf(g.residual_scale * gt, z, xv[i][q]);
        }
        if (g.w_pre) {
          xv[i][q] *= rx;
          c1[0] = fmaf(nv[q] * pv[q], xv[i][q], c1[0]);
          a_pre[i][q] = fmaf(nv[q], xv[i][q], a_pre[i][q]);
        }
      }
    }
    if (g.w_pre) row_sum<TPR>(c1, red1, half1);
    const float m1 = c1[0] * inv_h;
    float c2[2] = {0.f, 0.f};  // <g2 yh>, and the token's gate gradient
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = lane + i * TPR;
      float yv[CH], wv[CH], gv[CH], nv[CH], pv[CH];
      unpack(dr[i], dv[i]);
      unpack(nr[i], nv);
      unpack(wpre[i], pv);
      if (g.w_pre) {
#pragma unroll
        for (int q = 0; q < CH; ++q)
          dv[i][q] = fmaf(rx, fmaf(-m1, xv[i][q], nv[q] * pv[q]), dv[i][q]);
      }
      if (live && c < nch) store_chunk<T>(g.d_x, row, H, c, pack(dv[i]));
      if (g.y) {
        unpack(yr[i], yv);
        unpack(wpost[i], wv);
        unpack(gate[i], gv);
#pragma unroll
        for (int q = 0; q < CH; ++q) {
          const float yh = yv[q] * ry;               // y itself without a norm
          const float z = g.w_post ? yh * wv[q] : yh;
          const float sd = g.residual_scale * dv[i][q];
          c2[1] = fmaf(sd, z, c2[1]);
          a_gate[i][q] = fmaf(sd, z, a_gate[i][q]);
          float dz = sd * gt;
          if (g.gate_kind == MOE_GATE_CHANNEL) dz *= gv[q];
          a_post[i][q] = fmaf(dz, yh, a_post[i][q]);
          if (g.w_post) dz *= wv[q];
          c2[0] = fmaf(dz, yh, c2[0]);
          dv[i][q] = dz;
        }
      }
    }
    if (g.y) {
      if (g.w_post || g.gate_kind == MOE_GATE_TOKEN) row_sum<TPR>(c2, red2, half2);
      if (g.gate_kind == MOE_GATE_TOKEN && live && lane == 0) g.d_gate[row] = c2[1];
      const float m2 = c2[0] * inv_h;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = lane + i * TPR;
        if (g.w_post) {  // (without the norm d_y does not depend on y, which may be infinite)
          float yv[CH];
          unpack(yr[i], yv);
#pragma unroll
          for (int q = 0; q < CH; ++q) dv[i][q] = ry * fmaf(-m2 * ry, yv[q], dv[i][q]);
        }
        if (live && c < nch) store_chunk<T>(g.d_y, row, H, c, pack(dv[i]));
      }
    }
  }

  // this workgroup's column sums, its row groups added in order
  auto put = [&](const float (&a)[V][CH], int which) {
    float *out = g.partial + ((int64_t)which * gridDim.x + blockIdx.x) * H;
    if constexpr (RPB == 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = lane + i * TPR;
        if (c < nch)
#pragma unroll
          for (int q = 0; q < CH; ++q) out[c * CH + q] = a[i][q];
      }
    } else {
      constexpr int W = TPR * V * CH;  // columns a group holds
      __syncthreads();
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < CH; ++q)
          cols[group * W + (lane + i * TPR) * CH + q] = a[i][q];
      __syncthreads();
      for (int col = threadIdx.x; col < H; col += BT) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < RPB; ++r) s += cols[r * W + col];
        out[col] = s;
      }
    }
  };
  if (g.w_pre) put(a_pre, 0);
  if (g.w_post) put(a_post, 1);
  if (g.gate_kind == MOE_GATE_CHANNEL) put(a_gate, 2);
}

// out[which][col] = sum over the workgroups' partial sums, in a fixed order: a
// workgroup takes 64 columns, its threads every 16th partial row (a norm of 16384
// x 4096: 25 MB in 5.7 us).
constexpr int kSumCols = 64;
__global__ __launch_bounds__(1024) void column_sum_kernel(const float *__restrict__ partial,
                                                          int blocks, int H, ColumnSums out) {
  constexpr int R = 1024 / kSumCols, U = 8;  // rows at a time, loads in flight
  __shared__ float part[R][kSumCols];
  const int c = threadIdx.x % kSumCols, r = threadIdx.x / kSumCols;
  const int col = (int)blockIdx.x * kSumCols + c, which = blockIdx.y;
  float *o = which == 0 ? out.d_w_pre : which == 1 ? out.d_w_post : out.d_gate;
  if (!o) return;  // the same for the whole workgroup
  float s = 0.f;
  if (col < H) {
    const float *p = partial + (int64_t)which * blocks * H + col;
    for (int b = r; b < blocks; b += R * U) {
      float v[U];
#pragma unroll
      for (int q = 0; q < U; ++q) v[q] = b + R * q < blocks ? p[(int64_t)(b + R * q) * H] : 0.f;
#pragma unroll
      for (int q = 0; q < U; ++q) s += v[q];
    }
  }
  part[r][c] = s;
  __syncthreads();
  if (r == 0 && col < H) {
#pragma unroll
    for (int q = 1; q < R; ++q) s += part[q][c];
    o[col] = s;
  }
}

// Calls go(TPR, V) for the number of 16-byte chunks in a row of T.  V = 2 up to
// 512 chunks where one wave or 256 threads then cover the row; from there on the
// backward pass, whose bf16 row, weights and column sums are 190 registers at V = 2
// (two waves a SIMD) and 110 - 140 at V = 1 (three or four), takes V = 1 as far as
// 1024 threads reach.  Only what a row of up to kMaxNormHidden values can ask for
// is built.
template <bool kBackward, typename T, typename F> void by_width(int nch, F go) {
  using std::integral_constant;
  integral_constant<int, 1> one;
  integral_constant<int, 2> two;
  integral_constant<int, 4> four;
  if (nch <= 16) return go(integral_constant<int, 16>(), one);
  if (nch <= 64) return go(integral_constant<int, 64>(), one);
  if (nch <= 128) return go(integral_constant<int, 64>(), two);
  if (nch <= 256) return go(integral_constant<int, 256>(), one);
  if constexpr (kBackward) {
    if (nch <= 384) return go(integral_constant<int, 384>(), one);
    if (nch <= 512) return go(integral_constant<int, 256>(), two);
    if (nch <= 768) return go(integral_constant<int, 768>(), one);
    if (nch <= 1024) return go(integral_constant<int, 1024>(), one);
  } else {
    if (nch <= 512) return go(integral_constant<int, 256>(), two);
    if (nch <= 1024) return go(integral_constant<int, 256>(), four);
  }
  if constexpr (kMaxNormHidden / chunk_elems<T>() <= 2048) {
    go(integral_constant<int, 1024>(), two);
  } else {
    if (nch <= 2048) return go(integral_constant<int, 1024>(), two);
    go(integral_constant<int, 1024>(), four);
  }
}

int chunks_of(int hidden, moe_dtype_t dt) { return hidden / (dt == MOE_BF16 ? 8 : 4); }

// Rows a workgroup takes at a time (as by_width has them, either direction).
int rows_at_a_time(int nch) { return nch <= 16 ? 16 : nch <= 128 ? 4 : 1; }

// Workgroups of a launch: enough to fill the chip, few enough that the weights
// are loaded (and the column sums written) seldom.  Backward, 16384 x 4096: 256
// workgroups 232 us, 512 164, 1024 177 (their column sums are 3 x 16 MB more);
// forward within 2 % from 1024 on.
int64_t norm_blocks(int64_t n, int nch, int most) {
  const int64_t b = (n + rows_at_a_time(nch) - 1) / rows_at_a_time(nch);
  return b < most ? b : most;
}
constexpr int kForwardBlocks = 2048, kBackwardBlocks = 512;

}  // namespace

size_t block_norm_scratch_bytes(int64_t n_tokens, int hidden, moe_dtype_t dt) {
  return (size_t)3 * norm_blocks(n_tokens, chunks_of(hidden, dt), kBackwardBlocks) * hidden *
         sizeof(float);
}

hipError_t launch_block_norm(const BlockNormArgs &g, moe_dtype_t dt, hipStream_t s) {
  const int nch = chunks_of(g.hidden, dt);
  const dim3 grid((unsigned)norm_blocks(g.n_tokens, nch, kForwardBlocks));
  auto run = [&](auto tag) {
    using T = decltype(tag);
    by_width<false, T>(nch, [&](auto tpr, auto v) {
      constexpr int TPR = decltype(tpr)::value, V = decltype(v)::value;
      hipLaunchKernelGGL((block_norm_kernel<T, TPR, V>), grid, dim3(block_threads(TPR)), 0, s, g);
    });
  };
  if (dt == MOE_BF16) run(bf16_t()); else run(float());
  return hipGetLastError();
}

hipError_t launch_block_norm_backward(const BlockNormArgs &g, const ColumnSums &sums,
                                      moe_dtype_t dt, hipStream_t s) {
  const int nch = chunks_of(g.hidden, dt);
  const int blocks = (int)norm_blocks(g.n_tokens, nch, kBackwardBlocks);
  if (blocks > 0) {
    auto run = [&](auto tag) {
      using T = decltype(tag);
      by_width<true, T>(nch, [&](auto tpr, auto v) {
        constexpr int TPR = decltype(tpr)::value, V = decltype(v)::value;
        hipLaunchKernelGGL((block_norm_backward_kernel<T, TPR, V>), dim3(blocks),
                           dim3(block_threads(TPR)), 0, s, g);
      });
    };
    if (dt == MOE_BF16) run(bf16_t()); else run(float());
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  // (with no tokens the sums are zeros)
  if (sums.d_w_pre || sums.d_w_post || sums.d_gate)
    hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((g.hidden + kSumCols - 1) / kSumCols), 3), dim3(1024), 0,
                       s, g.partial, blocks, g.hidden, sums);
  return hipGetLastError();
}

}  // namespace moe
