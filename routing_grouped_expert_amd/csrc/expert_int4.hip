// Expert FFN of decode-sized batches with 4-bit weights: codes of 4 bits, one
// bf16 scale and one zero point per group of G = 32, 64 or 128 consecutive
// weights along K,
//
//   w[n, k] = s[k / G, n] * (q[n, k] - z[k / G, n])          (z = 8 if absent)
//
// the matrix-vector form of the expert FFN of grouped_gemm.hip (w13 with the
// fused activation, or w2 with the routing weight; activations and w13 layouts
// as the vLLM PR #47106 report describes them).  With a few rows an expert the
// layer is a stream of weights, half a byte each, so what counts is bytes in
// flight and few instructions a weight.
//
// Mathematics.  Over one group the scale is a factor of the whole sum:
//   sum_k a_k w_k = sum over groups of s * (sum_k a_k (q_k - z)),
// and the inner sum is taken exactly as products of small integers with bf16
// activations, on the matrix cores: a code q put into the low mantissa bits of
// bf16 128.0 (0x4300 | q) is the number 128 + q, one AND and one OR for two
// weights, and a second product with the constant -(128 + z), also exact in
// bf16, takes the offset and the zero point off again.  Sums are fp32; the
// scale enters in fp32 once a group.  Nothing is rounded to bf16 but the
// activation rows between the two products (the bf16 layer's own type).
//
// One workgroup of four waves computes 16 output columns (16 weight rows, or
// 16 gate and 16 up rows) of one expert that has rows; the waves split K and
// add up through LDS.  A 16x16x32 product takes the expert's token rows as its
// 16 rows (missing ones are zeros and cost no traffic) and the weight rows as
// its 16 columns, so a lane holds codes, scale and zero point of one weight
// row.  A lane loads 16 bytes of codes, 32 weights of its row; the four lanes
// of a row hold 128 weights, and a 4 x 4 transpose of dwords between the lane
// groups (four lane swaps) gives each of the four products 32 consecutive
// weights, so that no product mixes two groups.
#include "gemm_common.h"
#include "lds_dma.h"
#include "rows.h"

namespace moe {
namespace {

constexpr int kWaves = 4;

struct Int4Args {
  const void *A;               // w13: x [N, K]; w2: activation rows [M, K]
  const uint8_t *q;            // [E, NSETS * Nout, K / 2]
  const bf16_t *s;             // [E, K / G, NSETS * Nout]
  const uint8_t *z;            // [E, K / G, NSETS * Nout] or NULL (8)
  void *C;                     // w13: [M, Nout] bf16; w2: [M, Nout] fp32 or [N, Nout] bf16
  const int32_t *offsets;      // [E + 1]
  const int32_t *col_sorted;   // [M]
  const void *gate_scal;       // [M] (w2)
  uint32_t a_bytes;
  int gate_bf16, E, K, Nout, topk, gather, interleaved;
  ActParams prm;
};

// Eight codes of a dword (element i in nibble i) as bf16 128 + q, in the order
// (0, 4), (1, 5), (2, 6), (3, 7) that token_order gives the token rows.
__device__ __forceinline__ bf16x8_t codes_plus_128(uint32_t w) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ((w >> (4 * i)) & 0x000f000fu) | 0x43004300u;
  return __builtin_bit_cast(bf16x8_t, v);
}
__device__ __forceinline__ bf16x8_t token_order(u32x4_t a) {
  u32x4_t v;
  v[0] = __builtin_amdgcn_perm(a[2], a[0], 0x05040100u);  // low halves: elements 0, 4
  v[1] = __builtin_amdgcn_perm(a[2], a[0], 0x07060302u);  // high halves: 1, 5
  v[2] = __builtin_amdgcn_perm(a[3], a[1], 0x05040100u);
  v[3] = __builtin_amdgcn_perm(a[3], a[1], 0x07060302u);
  return __builtin_bit_cast(bf16x8_t, v);
}

// Dword d of lane group c (of four groups of 16 lanes) becomes dword c of lane
// group d.
__device__ __forceinline__ void transpose_groups(u32x4_t &v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false));
  const u32x2 c = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false));
  const u32x2 d = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false));
  v[0] = c[0];
  v[1] = c[1];
  v[2] = d[0];
  v[3] = d[1];
}

// The blockIdx.y-th expert with rows and its range of sorted rows, found by
// one wave (four experts a lane); expert -1 if there are fewer.  sel: LDS.
__device__ __forceinline__ void find_expert(const int32_t *offsets, int E, int want, int *sel) {
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    int o[5], c[4], n = 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) o[i] = offsets[min(lane * 4 + i, E)];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = lane * 4 + i < E ? o[i + 1] - o[i] : 0;
      n += c[i] > 0;
    }
    const int incl = wave_inclusive_sum(n);
    int before = incl - n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c[i] > 0 && before++ == want) {
        sel[0] = lane * 4 + i;
        sel[1] = o[i];
        sel[2] = c[i];
      }
    }
    if (lane == 63 && incl <= want) sel[0] = -1;
  }
  __syncthreads();
}

// GS = G / 32; NT: tiles of 16 token rows held at a time.
template <int NSETS, int EPI, int GS, int NT>
__global__ __launch_bounds__(64 * kWaves) void expert_int4_kernel(Int4Args g) {
  __shared__ int sel[3];
  __shared__ float red[kWaves][NSETS][NT][16][17];
  find_expert(g.offsets, g.E, (int)blockIdx.y, sel);
  const int e = __builtin_amdgcn_readfirstlane(sel[0]);
  if (e < 0) return;  // the whole workgroup
  const int row0 = __builtin_amdgcn_readfirstlane(sel[1]);
  const int cnt = __builtin_amdgcn_readfirstlane(sel[2]);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;  // this lane's row in a tile, its lane group
  const int K = g.K, Nout = g.Nout, nrows = NSETS * Nout;
  const int n0 = (int)blockIdx.x * 16;
  const int nblk = (K + 127) / 128, per = (nblk + kWaves - 1) / kWaves;
  const int b0 = wave * per, b1 = min(b0 + per, nblk);

  // this expert's weights (Nout is a multiple of 32); a group past K reads
  // zeros: code 0 and zero point 0 are a weight of 128 - 128, and scale 0
  const uint32_t qbytes = (uint32_t)nrows * (uint32_t)(K / 2);
  const uint32_t groups = (uint32_t)(K / (32 * GS));
  const uint32_t sn = groups * (uint32_t)nrows;
  const __amdgpu_buffer_rsrc_t rq = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(g.q) + (size_t)e * qbytes, (short)0, (int)qbytes, kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<bf16_t *>(g.s) + (size_t)e * sn, (short)0, (int)(2 * sn), kRsrcWord3);
  const __amdgpu_buffer_rsrc_t rz = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t *>(g.z) + (g.z ? (size_t)e * sn : 0), (short)0, g.z ? (int)sn : 0,
      kRsrcWord3);
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void *>(g.A), (short)0, (int)g.a_bytes, kRsrcWord3);
  uint32_t wrow[NSETS];
#pragma unroll
  for (int s = 0; s < NSETS; ++s)
    wrow[s] = NSETS == 1 ? n0 + r : g.interleaved ? 2 * (n0 + r) + s : s * Nout + n0 + r;

  for (int a0 = 0; a0 < cnt; a0 += 16 * NT) {
    uint32_t arow[NT];  // byte offset of this lane's token row in each tile
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int i = a0 + 16 * t + r;
      uint32_t row = 0;
      if (i < cnt) row = g.gather ? (uint32_t)g.col_sorted[row0 + i] / (uint32_t)g.topk : row0 + i;
      arow[t] = i < cnt ? row * (uint32_t)(2 * K) : kOOB;
    }
    f32x4_t acc[NSETS][NT];
#pragma unroll
    for (int s = 0; s < NSETS; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[s][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    for (int b = b0; b < b1; ++b) {
      u32x4_t cw[NSETS], tok[NT][4];
      uint32_t sc[NSETS][4 / GS], zp[NSETS][4 / GS];
#pragma unroll
      for (int s = 0; s < NSETS; ++s) {
        const int k = b * 128 + h * 32;
        const uint32_t off =
            k < K ? wrow[s] * (uint32_t)(K / 2) + (uint32_t)(k / 2) : kOOB;
        cw[s] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, (int)off, 0, 0));
#pragma unroll
        for (int i = 0; i < 4 / GS; ++i) {
          const uint32_t gi = (uint32_t)(b * (4 / GS) + i);
          const uint32_t at = gi < groups ? gi * (uint32_t)nrows + wrow[s] : kOOB / 2;
          sc[s][i] = (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, (int)(2 * at), 0, 0);
          zp[s][i] = g.z ? (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rz, (int)at, 0, 0)
                     : gi < groups ? 8u : 0u;
        }
      }
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = b * 128 + i * 32 + h * 8;
          const uint32_t off = arow[t] != kOOB && k < K ? arow[t] + (uint32_t)(2 * k) : kOOB;
          tok[t][i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(ra, (int)off, 0, 0));
        }
#pragma unroll
      for (int s = 0; s < NSETS; ++s) transpose_groups(cw[s]);
      f32x4_t sum[NSETS][NT];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int s = 0; s < NSETS; ++s) {
          const uint32_t zz = zp[s][i / GS] * 0x00010001u | 0xc300c300u;
          const bf16x8_t wz = __builtin_bit_cast(bf16x8_t, u32x4_t{zz, zz, zz, zz});
          const bf16x8_t wv = codes_plus_128(cw[s][i]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const bf16x8_t av = token_order(tok[t][i]);
            if (i % GS == 0) sum[s][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            sum[s][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, wv, sum[s][t], 0, 0, 0);
            sum[s][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, wz, sum[s][t], 0, 0, 0);
            if (i % GS == GS - 1) {
              const float f = __uint_as_float(sc[s][i / GS] << 16);
#pragma unroll
              for (int q = 0; q < 4; ++q) acc[s][t][q] = fmaf(f, sum[s][t][q], acc[s][t][q]);
            }
          }
        }
      }
    }

    // the waves' parts: lane (h, r) holds column r of token rows 4 h .. 4 h + 3
    if (a0 > 0) __syncthreads();
#pragma unroll
    for (int s = 0; s < NSETS; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) red[wave][s][t][4 * h + q][r] = acc[s][t][q];
    __syncthreads();
    const int col = threadIdx.x & 15, trow = threadIdx.x >> 4;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int i = a0 + 16 * t + trow;
      if (i >= cnt) continue;
      float v[NSETS];
#pragma unroll
      for (int s = 0; s < NSETS; ++s) {
        v[s] = red[0][s][t][trow][col];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v[s] += red[w][s][t][trow][col];
      }
      const size_t p = (size_t)(row0 + i);
      if constexpr (EPI == EPI_Y || EPI == EPI_OUT) {
        const float y = v[0] * weight_at(g.gate_scal, g.gate_bf16, (int64_t)p);
        if (EPI == EPI_Y)  // summed over the slots by sum_slots_kernel, in fp32
          reinterpret_cast<float *>(g.C)[p * Nout + n0 + col] = y;
        else               // one slot a token: entry == token
          reinterpret_cast<bf16_t *>(g.C)[(size_t)g.col_sorted[p] * Nout + n0 + col] = bf16_rne(y);
      } else {
        const float nal = -g.prm.alpha * 1.44269504088896341f;
        float a = act_val<EPI>(v[0], v[NSETS - 1], nal, g.prm);
        // the clamps and the rectifier drop a NaN; the token's row shall show it
        if (__builtin_isnan(v[0]) || __builtin_isnan(v[NSETS - 1])) a = __builtin_nanf("");
        reinterpret_cast<bf16_t *>(g.C)[p * Nout + n0 + col] = bf16_rne(a);
      }
    }
  }
}

// out[t] = sum over the token's slots of its fp32 rows, rounded once.
__global__ __launch_bounds__(256) void sum_slots_kernel(const float *__restrict__ y,
                                                        const int32_t *__restrict__ row_sorted,
                                                        bf16_t *__restrict__ out, int64_t N, int K,
                                                        int H) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int nch = H / 8;
  if (i >= N * nch) return;
  const int64_t t = i / nch;
  const int c = (int)(i - t * nch) * 8;
  float acc[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] = 0.f;
  for (int j = 0; j < K; ++j) {
    const uint32_t p = (uint32_t)row_sorted[t * K + j];
    if (p >= (uint32_t)(N * K)) continue;
    const f32x4_t lo = *reinterpret_cast<const f32x4_t *>(y + (int64_t)p * H + c);
    const f32x4_t hi = *reinterpret_cast<const f32x4_t *>(y + (int64_t)p * H + c + 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[q] += lo[q];
      acc[q + 4] += hi[q];
    }
  }
  *reinterpret_cast<u32x4_t *>(out + t * H + c) = pack(acc);
}

template <int NSETS, int EPI, int GS>
void launch_tiles(const Int4Args &a, int64_t n_tokens, int64_t M, hipStream_t s) {
  const dim3 grid((unsigned)(a.Nout / 16), (unsigned)(M < a.E ? M : a.E));
  // an expert holds at most one row a token
  if (n_tokens <= 16)
    hipLaunchKernelGGL((expert_int4_kernel<NSETS, EPI, GS, 1>), grid, dim3(64 * kWaves), 0, s, a);
  else
    hipLaunchKernelGGL((expert_int4_kernel<NSETS, EPI, GS, 2>), grid, dim3(64 * kWaves), 0, s, a);
}

template <int NSETS, int EPI>
hipError_t launch_groups(const Int4Args &a, int group, int64_t n_tokens, int64_t M,
                         hipStream_t s) {
  if (group == 32) launch_tiles<NSETS, EPI, 1>(a, n_tokens, M, s);
  else if (group == 64) launch_tiles<NSETS, EPI, 2>(a, n_tokens, M, s);
  else launch_tiles<NSETS, EPI, 4>(a, n_tokens, M, s);
  return hipGetLastError();
}

// One thread per group of one row.  Division and rounding are IEEE fp32, so
// the codes are the same everywhere.
template <typename T>
__global__ __launch_bounds__(256) void quantize_int4_kernel(const T *__restrict__ w, int64_t nrows,
                                                            int rows, int K, int G,
                                                            uint32_t *__restrict__ q,
                                                            bf16_t *__restrict__ s,
                                                            uint8_t *__restrict__ z) {
  const int ng = K / G;
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (idx >= nrows * ng) return;
  const int64_t row = idx / ng;
  const int gi = (int)(idx - row * ng);
  const T *src = w + row * K + (int64_t)gi * G;
  float lo = 0.f, hi = 0.f;
  for (int i = 0; i < G; ++i) {
    const float v = to_f32(src[i]);
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  const bf16_t sb = bf16_rne(z ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f);
  const float sc = to_f32(sb);
  float zero = 8.f;
  if (z) zero = sc > 0.f ? fminf(fmaxf(rintf(-lo / sc), 0.f), 15.f) : 0.f;
  uint32_t *dst = q + (row * K + (int64_t)gi * G) / 8;
  for (int i = 0; i < G; i += 8) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = sc > 0.f ? rintf(to_f32(src[i + j]) / sc) : 0.f;
      word |= (uint32_t)fminf(fmaxf(v + zero, 0.f), 15.f) << (4 * j);
    }
    dst[i / 8] = word;
  }
  const int64_t e = row / rows, r = row - e * rows;
  s[(e * ng + gi) * rows + r] = sb;
  if (z) z[(e * ng + gi) * rows + r] = (uint8_t)zero;
}

// Eight weights a thread: s * (q - z), exact in fp32, rounded once to bf16.
__global__ __launch_bounds__(256) void dequantize_int4_kernel(const uint32_t *__restrict__ q,
                                                              const bf16_t *__restrict__ s,
                                                              const uint8_t *__restrict__ z,
                                                              int64_t nrows, int rows, int K,
                                                              int G, bf16_t *__restrict__ w) {
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int nw = K / 8;
  if (idx >= nrows * nw) return;
  const int64_t row = idx / nw, e = row / rows, r = row - e * rows;
  const int c = (int)(idx - row * nw);
  const int64_t at = (e * (K / G) + c * 8 / G) * rows + r;
  const float sc = to_f32(s[at]), zero = z ? (float)z[at] : 8.f;
  const uint32_t word = q[idx];
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = sc * ((float)((word >> (4 * j)) & 15u) - zero);
  *reinterpret_cast<u32x4_t *>(w + row * K + c * 8) = pack(v);
}

}  // namespace

hipError_t launch_experts_int4(const Int4Weights &w13, const Int4Weights &w2, const void *x,
                               const moe_routing_t *r, void *out, void *act, void *y,
                               int64_t n_tokens, int topk, int n_experts, int hidden, int inter,
                               int group, moe_act_t kind, moe_w13_layout_t layout, ActParams prm,
                               hipStream_t s) {
  const int64_t M = n_tokens * topk;
  Int4Args a{x, reinterpret_cast<const uint8_t *>(w13.q), reinterpret_cast<const bf16_t *>(w13.s),
             reinterpret_cast<const uint8_t *>(w13.z), act, r->offsets, r->col_sorted, nullptr,
             (uint32_t)(n_tokens * hidden * 2), 0, n_experts, hidden, inter, topk, 1,
             layout == MOE_W13_INTERLEAVED, prm};
  const bool clamp = __builtin_isfinite(prm.limit);
  hipError_t err = kind == MOE_ACT_RELU2 ? launch_groups<1, EPI_RELU2>(a, group, n_tokens, M, s)
                   : clamp ? launch_groups<2, EPI_GATED_CLAMP>(a, group, n_tokens, M, s)
                           : launch_groups<2, EPI_GATED>(a, group, n_tokens, M, s);
  if (err != hipSuccess) return err;
  const bool direct = topk == 1;
  Int4Args b{act, reinterpret_cast<const uint8_t *>(w2.q), reinterpret_cast<const bf16_t *>(w2.s),
             reinterpret_cast<const uint8_t *>(w2.z), direct ? out : y, r->offsets, r->col_sorted,
             r->gate_scal, (uint32_t)(M * inter * 2), r->w_dtype == MOE_BF16, n_experts, inter,
             hidden, topk, 0, 0, prm};
  if (direct) return launch_groups<1, EPI_OUT>(b, group, n_tokens, M, s);
  if ((err = launch_groups<1, EPI_Y>(b, group, n_tokens, M, s)) != hipSuccess) return err;
  const int64_t total = n_tokens * (hidden / 8);
  hipLaunchKernelGGL(sum_slots_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, s,
                     reinterpret_cast<const float *>(y), r->row_sorted,
                     reinterpret_cast<bf16_t *>(out), n_tokens, topk, hidden);
  return hipGetLastError();
}

hipError_t launch_quantize_int4(const void *w, moe_dtype_t dt, int n_experts, int rows, int k,
                                int group, const Int4Weights &out, hipStream_t s) {
  const int64_t nrows = (int64_t)n_experts * rows, total = nrows * (k / group);
  const dim3 grid((unsigned)((total + 255) / 256));
  uint32_t *q = reinterpret_cast<uint32_t *>(const_cast<void *>(out.q));
  bf16_t *sc = reinterpret_cast<bf16_t *>(const_cast<void *>(out.s));
  uint8_t *z = reinterpret_cast<uint8_t *>(const_cast<void *>(out.z));
  if (dt == MOE_BF16)
    hipLaunchKernelGGL(quantize_int4_kernel<bf16_t>, grid, dim3(256), 0, s,
                       reinterpret_cast<const bf16_t *>(w), nrows, rows, k, group, q, sc, z);
  else
    hipLaunchKernelGGL(quantize_int4_kernel<float>, grid, dim3(256), 0, s,
                       reinterpret_cast<const float *>(w), nrows, rows, k, group, q, sc, z);
  return hipGetLastError();
}

hipError_t launch_dequantize_int4(const Int4Weights &in, int n_experts, int rows, int k, int group,
                                  void *w, hipStream_t s) {
  const int64_t nrows = (int64_t)n_experts * rows, total = nrows * (k / 8);
  hipLaunchKernelGGL(dequantize_int4_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0,
                     s, reinterpret_cast<const uint32_t *>(in.q),
                     reinterpret_cast<const bf16_t *>(in.s),
                     reinterpret_cast<const uint8_t *>(in.z), nrows, rows, k, group,
                     reinterpret_cast<bf16_t *>(w));
  return hipGetLastError();
}

}  // namespace moe
