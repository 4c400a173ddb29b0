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
// bf16 128.0 (0x4300 | q) is the number 128 + q, a shift and one AND-OR for two
// weights.  A product with ones gives the group's sum of a, once for all the
// weight rows of the wave, and s * (sum_k a_k (128 + q_k) - (128 + z) sum_k a_k)
// enters the result in fp32 once a group.  The activation rows between the two
// products are kept as two bf16 parts, a = hi + lo with hi = bf16(a) and lo =
// bf16(a - hi), off by 2^-16 of a value at most; the second product takes both
// parts into the same sums.  So the only rounding to bf16 of a whole call is
// that of its output (one part would add as much error as that rounding again:
// 0.0022 instead of 0.0017 in the 2-norm).
//
// A wave streams 32 weight rows of one expert (16 gate and 16 up rows, or 32
// plain ones) and no other wave reads them, so they go straight to registers,
// two steps of 256 weights a row ahead of the products.  The expert's token
// rows stand in LDS, read by all waves of the workgroup.  A 16x16x32 product
// takes token rows as its 16 rows (missing ones may be anything: their sums are
// not used) and weight rows as its 16 columns, so a lane holds codes, scale and
// zero point of one weight row and no sum leaves its lane until the end.
//
// Four neighbouring lanes load 64 bytes of a row (lanes that are rows apart
// measured 3.1 TB/s instead of 4.4 on the 64-expert layer); a lane permutation
// and, for groups of 32 and 64, lane swaps bring the dwords to the lanes whose
// product they belong to, so that no product mixes two groups.
//
// What bounds it: the rate of the loads, and about 235 vector instructions (of
// the whole kernel, counted) and 24 products a step of 8192 weights in w13, 300 and
// 48 in w2 with both parts; at one token the start of three kernels and of their
// loads.  Measured against the bytes of the touched experts: 64 experts (H 4096, I
// 1536, k 8), 32 tokens, groups of 128: 151 us, 4.1 TB/s; 128 experts (H = I =
// 2880, k 4), groups of 64 with zero points: 128 tokens 431 us, 4.0 TB/s, 33 tokens
// 370 us, 3.1 TB/s (rows of 1440 bytes straddle cache lines: 2816 wide 3.6 TB/s;
// the loads alone 319 us), one token 26.6 us (the loads alone 21, three empty
// kernels 10).  The second parts cost what w2 has more of: with one part those five
// took 148, 432, 355, 293 (2816 wide) and 25.3 us, and where experts hold 16 rows and
// more the whole 15 % less (8 experts, 64 tokens 112 us for 129).
#include "gemm_common.h"
#include "lds_dma.h"
#include "rows.h"

#include <type_traits>

namespace moe {
namespace {

struct Int4Args {
  const void *A;               // w13: x [N, K]; w2: activation rows [M, 2, K] (hi, lo)
  const uint8_t *q;            // [E, NSETS * Nout, K / 2]
  const bf16_t *s;             // [E, K / G, NSETS * Nout]
  const uint8_t *z;            // [E, K / G, NSETS * Nout] or NULL (8)
  void *C;                     // w13: [M, 2, Nout] bf16; w2: [M, Nout] fp32 or [N, Nout] bf16
  const int32_t *offsets;      // [E + 1]
  const int32_t *col_sorted;   // [M]
  const void *gate_scal;       // [M] (w2)
  int gate_bf16, E, K, Nout, topk, gather, interleaved;
  ActParams prm;
};

// Eight codes of a dword (element i in nibble i) as bf16 128 + q, in the order
// (0, 4), (1, 5), (2, 6), (3, 7) that token_order gives the token rows: a shift
// and one v_and_or_b32 for two codes.  mask and magic are 0x000f000f and
// 0x43004300 in registers (known constants become an AND and an OR instead).
__device__ __forceinline__ bf16x8_t codes_plus_128(uint32_t w, uint32_t mask, uint32_t magic) {
  u32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = ((w >> (4 * i)) & mask) | magic;
  return __builtin_bit_cast(bf16x8_t, v);
}
__device__ __forceinline__ u32x4_t token_order(u32x4_t a) {
  u32x4_t v;
  v[0] = __builtin_amdgcn_perm(a[2], a[0], 0x05040100u);  // low halves: elements 0, 4
  v[1] = __builtin_amdgcn_perm(a[2], a[0], 0x07060302u);  // high halves: 1, 5
  v[2] = __builtin_amdgcn_perm(a[3], a[1], 0x05040100u);
  v[3] = __builtin_amdgcn_perm(a[3], a[1], 0x07060302u);
  return v;
}

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x2_t swap32(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(a, b, false, false));
}
__device__ __forceinline__ u32x2_t swap16(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(a, b, false, false));
}

// Four dwords of lane group c (of four groups of 16 lanes) are 32 weights of
// piece c.  For groups of 128 weights they stay: product j takes dword j of
// all four pieces.  For 64 the halves are exchanged, so that products 0 and 1
// take pieces 0 and 1 (lane group h: piece h % 2, dword 2 (h / 2) + j % 2) and
// 2 and 3 the other two.  For 32, the full transpose: product j takes piece j
// (lane group h: dword h).
template <int GS> __device__ __forceinline__ void arrange(u32x4_t &v) {
  if constexpr (GS < 4) {
    const u32x2_t a = swap32(v[0], v[2]), b = swap32(v[1], v[3]);
    if constexpr (GS == 2) {
      v = u32x4_t{a[0], b[0], a[1], b[1]};
    } else {
      const u32x2_t c = swap16(a[0], b[0]), d = swap16(a[1], b[1]);
      v = u32x4_t{c[0], c[1], d[0], d[1]};
    }
  }
}
// The 8-weight piece of a 128-weight block that lane group h gives product j.
template <int GS> __device__ __forceinline__ int eighth(int j, int h) {
  return GS == 4 ? 4 * h + j : GS == 2 ? 8 * (j >> 1) + 4 * (h & 1) + 2 * (h >> 1) + (j & 1)
                                       : 4 * j + h;
}

// Sends lane group i's value to every lane, for i = 0 .. 3.
__device__ __forceinline__ void spread_groups(uint32_t v, uint32_t (&out)[4]) {
  const u32x2_t a = swap32(v, v), b = swap16(a[0], a[0]), c = swap16(a[1], a[1]);
  out[0] = b[0];
  out[1] = b[1];
  out[2] = c[0];
  out[3] = c[1];
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

// The workgroup's place among all, so that neighbouring column tiles, which
// share cache lines of the scales and zero points, run on one XCD (workgroups
// go to the eight XCDs in turn).
__device__ __forceinline__ void place(int &x, int &y) {
  const uint32_t gx = gridDim.x, total = gx * gridDim.y, lin = blockIdx.y * gx + blockIdx.x;
  const uint32_t per = total / 8, rest = total % 8, xcd = lin % 8;
  const uint32_t at = xcd * per + min(xcd, rest) + lin / 8;
  x = (int)(at % gx);
  y = (int)(at / gx);
}

constexpr int kStepK = 256;  // weights of a row a step: one 128-byte line of codes
constexpr int kStepBytes = 2 * kStepK;  // a token row's part of a step in LDS

// One expert's weight arrays as a wave reads them.
template <int GS> struct ExpertArrays {
  __amdgpu_buffer_rsrc_t rq, rs, rz;  // (without zero points rz is empty: loads give 0)
  bool has_z;
  uint32_t nrows, magic, mask;
  int lane, K;

  __device__ __forceinline__ void open(const Int4Args &g, int e, int rows) {
    lane = threadIdx.x & 63;
    K = g.K;
    nrows = (uint32_t)rows;
    has_z = g.z != nullptr;
    const uint32_t qbytes = nrows * (uint32_t)(K / 2), sn = (uint32_t)(K / (32 * GS)) * nrows;
    rq = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(g.q) + (size_t)e * qbytes,
                                           (short)0, (int)qbytes, kRsrcWord3);
    rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<bf16_t *>(g.s) + (size_t)e * sn, (short)0,
                                           (int)(2 * sn), kRsrcWord3);
    rz = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(g.z) + (has_z ? (size_t)e * sn : 0),
                                           (short)0, has_z ? (int)sn : 0, kRsrcWord3);
    magic = 0x43004300u;
    mask = 0x000f000fu;
    asm("" : "+v"(magic));  // (no instruction: hides the values, see codes_plus_128)
    asm("" : "+s"(mask));
  }
  __device__ __forceinline__ u32x4_t codes(uint32_t at) const {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, (int)at, 0, 0));
  }
  __device__ __forceinline__ uint32_t scale(uint32_t at) const {  // bf16 bits
    return (uint32_t)(uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, (int)(2 * at), 0, 0);
  }
  __device__ __forceinline__ uint32_t zero(uint32_t at) const {
    return (uint32_t)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rz, (int)at, 0, 0);
  }
};

// One wave's 32 weight rows (two tiles of 16) of one expert: where they are,
// and the products of a step of them with the token rows in LDS.
template <int GS> struct WaveRows : ExpertArrays<GS> {
  using A = ExpertArrays<GS>;
  static constexpr int NM = GS == 1 ? 2 : 1;  // loads of four groups' scales a step and tile

  struct Codes {  // a step of the rows
    u32x4_t w[2][2];
    uint32_t s[2][NM], z[2][NM];
  };

  uint32_t qoff[2], moff[2];

  // memrow(t, x): memory row of row x of tile t.  Codes: four lanes a row, 64
  // bytes; a lane permutation puts them where the products want them.  Scales
  // and zero points: lane group h loads the step's groups h (and h + 4).  Loads
  // past K bring other rows' data, or zeros past the array's end; they are not
  // used.
  template <typename F> __device__ __forceinline__ void init(const Int4Args &g, int e, int rows,
                                                             F memrow) {
    A::open(g, e, rows);
    const int lane = A::lane;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      qoff[t] = (uint32_t)memrow(t, lane >> 2) * (uint32_t)(A::K / 2) + (uint32_t)((lane & 3) * 16);
      moff[t] = (uint32_t)(lane >> 4) * A::nrows + (uint32_t)memrow(t, lane & 15);
    }
  }

  __device__ __forceinline__ void load(Codes &c, int step) const {
    const uint32_t k0 = (uint32_t)step * kStepK, g0 = k0 / (32 * GS) * A::nrows;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int b = 0; b < 2; ++b) c.w[t][b] = A::codes(qoff[t] + k0 / 2 + 64 * b);
#pragma unroll
      for (int m = 0; m < NM; ++m) {
        const uint32_t at = moff[t] + g0 + 4 * m * A::nrows;
        c.s[t][m] = A::scale(at);
        c.z[t][m] = A::has_z ? A::zero(at) : 8u;
      }
    }
  }

  // acc[t] += this step's products with the lane's token row, whose part of the
  // step is at `tok` (16-byte piece c at place c ^ swz); with TILES = 2 also with
  // the row's second part, right behind; with kWhole = false only the groups
  // ahead of K.
  template <int TILES, bool kWhole>
  __device__ __forceinline__ void work(const Codes &c, int step, const char *tok, int swz,
                                       f32x4_t (&acc)[2]) const {
    const int h = A::lane >> 4, from = (4 * (A::lane & 15) + h) * 4;
    const int ngroups = kWhole ? 8 / GS : (A::K - step * kStepK) / (32 * GS);
    const bf16x8_t ones = __builtin_bit_cast(
        bf16x8_t, u32x4_t{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u});
    uint32_t mt[2][4];  // scale << 16 | zero point of the groups (of this half for NM = 2)
    f32x4_t sum[2], tot;
    const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      u32x4_t cw[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (NM == 2 || b == 0) {
          const int m = NM == 2 ? b : 0;
          spread_groups(c.s[t][m] << 16 | c.z[t][m], mt[t]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          cw[t][q] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)c.w[t][b][q]);
        arrange<GS>(cw[t]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int gr = (4 * b + j) / GS;
        if (!kWhole && gr >= ngroups) break;
        bf16x8_t wv[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) wv[t] = codes_plus_128(cw[t][j], A::mask, A::magic);
#pragma unroll
        for (int u = 0; u < TILES; ++u) {
          const bf16x8_t av = *reinterpret_cast<const bf16x8_t *>(
              tok + u * kStepBytes + 256 * b + ((eighth<GS>(j, h) ^ swz) * 16));
          const bool begins = j % GS == 0 && u == 0;
          tot = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, ones, begins ? zero : tot, 0, 0, 0);
#pragma unroll
          for (int t = 0; t < 2; ++t)
            sum[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, wv[t], begins ? zero : sum[t], 0,
                                                             0, 0);
        }
        // (keeps the second parts' loads from being moved up past the registers: up to 18
        // spilled without, 8 for groups of 32 with)
        if constexpr (TILES == 2) __builtin_amdgcn_sched_barrier(0);
        if (j % GS == GS - 1) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float f = __uint_as_float(mt[t][gr & 3] & 0xffff0000u);
            const float z = 128.f + (float)(mt[t][gr & 3] & 0xffu);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[t][q] = fmaf(f, fmaf(-z, tot[q], sum[t][q]), acc[t][q]);
          }
        }
      }
    }
  }

  // Steps first .. last - 1, the first two already in c0 and c1, two ahead;
  // tok0: the lane's token row at step s0, a step every PARTS * kStepBytes.
  template <int TILES, int PARTS>
  __device__ __forceinline__ void stream(Codes &c0, Codes &c1, int first, int last, int s0,
                                         const char *tok0, int swz, f32x4_t (&acc)[2]) const {
    auto run = [&](const Codes &c, int step) {
      const char *tok = tok0 + (step - s0) * (PARTS * kStepBytes);
      if ((step + 1) * kStepK <= A::K) work<TILES, true>(c, step, tok, swz, acc);
      else work<TILES, false>(c, step, tok, swz, acc);
    };
    for (int step = first; step < last; step += 2) {
      run(c0, step);
      if (step + 1 >= last) break;
      if (step + 2 < last) load(c0, step + 2);
      run(c1, step + 1);
      if (step + 3 < last) load(c1, step + 3);
    }
  }
};

// acc + a.lo * b.lo + a.hi * b.hi on packed bf16 pairs (v_dot2_f32_bf16).
__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float acc) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, a),
                                         __builtin_bit_cast(bf16x2_t, b), acc, false);
}

// The same rows for a single token row, where a product of 16 token rows would
// compute one: dot products, every lane its own 32 weights of a row (lane l:
// row l / 4 of a tile, piece l % 4 of 128 weights) with the token's values at
// those places, the scale and zero point of the lane's own group, and one sum
// over the four lanes of a row at the end.  The lanes keep what they load: no
// permutation, no swaps (one token of 128 experts, groups of 64: 28.7 us by the
// products, 27.1 this way; of 32 experts, groups of 32: 32.1 and 27.2).
template <int GS> struct DotRows : ExpertArrays<GS> {
  using A = ExpertArrays<GS>;
  struct Codes {  // a step of the rows
    u32x4_t w[2][2];
    uint32_t s[2][2], z[2][2];
  };

  uint32_t qoff[2], mrow[2];

  template <typename F> __device__ __forceinline__ void init(const Int4Args &g, int e, int rows,
                                                             F memrow) {
    A::open(g, e, rows);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mrow[t] = (uint32_t)memrow(t, A::lane >> 2);
      qoff[t] = mrow[t] * (uint32_t)(A::K / 2) + (uint32_t)((A::lane & 3) * 16);
    }
  }

  __device__ __forceinline__ void load(Codes &c, int step) const {
    const uint32_t k0 = (uint32_t)step * kStepK;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t piece = k0 + 128 * b + 32 * (uint32_t)(A::lane & 3);
        c.w[t][b] = A::codes(qoff[t] + k0 / 2 + 64 * b);
        c.s[t][b] = A::scale(piece / (32 * GS) * A::nrows + mrow[t]);
        c.z[t][b] = A::zero(piece / (32 * GS) * A::nrows + mrow[t]);
      }
  }

  // acc[t] += the lane's part of row lane / 4 of tile t; tok: the token row at
  // this step (with PARTS = 2 its second part `part` bytes further on), sums: the
  // sums of its pieces of 32.
  template <int PARTS>
  __device__ __forceinline__ void work(const Codes &c, int step, const char *tok, int part,
                                       const float *sums, float (&acc)[2]) const {
    const float zero0 = A::has_z ? 128.f : 136.f;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // (a piece past K: the loads brought anything, nothing is added)
      const bool in = step * kStepK + 128 * b + 32 * (A::lane & 3) < A::K;
      const float total = sums[4 * b + (A::lane & 3)];
      float dot[2] = {0.f, 0.f};
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        u32x4_t av[PARTS];
#pragma unroll
        for (int u = 0; u < PARTS; ++u)
          av[u] = *reinterpret_cast<const u32x4_t *>(tok + u * part + 256 * b +
                                                     (A::lane & 3) * 64 + 16 * d);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const u32x4_t wv =
              __builtin_bit_cast(u32x4_t, codes_plus_128(c.w[t][b][d], A::mask, A::magic));
#pragma unroll
          for (int u = 0; u < PARTS; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) dot[t] = dot2(wv[i], av[u][i], dot[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float f = __uint_as_float(c.s[t][b] << 16), z = zero0 + (float)c.z[t][b];
        const float v = fmaf(f, fmaf(-z, total, dot[t]), acc[t]);
        acc[t] = in ? v : acc[t];
      }
    }
  }

  template <int PARTS>
  __device__ __forceinline__ void stream(Codes &c0, Codes &c1, int first, int last, int s0,
                                         const char *tok0, int part, const float *sums0,
                                         float (&acc)[2]) const {
    auto run = [&](const Codes &c, int step) {
      work<PARTS>(c, step, tok0 + (step - s0) * (2 * kStepK), part,
                  sums0 + (step - s0) * (kStepK / 32), acc);
    };
    for (int step = first; step < last; step += 2) {
      run(c0, step);
      if (step + 1 >= last) break;
      if (step + 2 < last) load(c0, step + 2);
      run(c1, step + 1);
      if (step + 3 < last) load(c1, step + 3);
    }
  }
};

// Token rows into LDS by the whole workgroup: values kb .. kb + klen - 1 of the
// rows row(0) .. row(n - 1), rowb bytes apart, 16-byte piece c of row i at place c
// ^ (i % 8).  With PARTS = 2 row i is memory rows 2 row(i) and 2 row(i) + 1, a step
// of the second behind each step of the first.  U loads of a thread in flight.
template <int U, int PARTS, typename F>
__device__ __forceinline__ void stage_rows(const Int4Args &g, char *lds, int rowb, int n, int kb,
                                           int klen, F row) {
  const int np = klen / 8, total = PARTS * n * np, stride = blockDim.x;
  for (int i0 = threadIdx.x; i0 < total; i0 += U * stride) {
    int at[U], to[U];
    u32x4_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u * stride, total - 1), c = i % np, lo = i / np >= n;
      const int t = i / np - lo * n;
      at[u] = PARTS * row(t) + lo;
      to[u] = t * rowb + (c / 32 * PARTS + lo) * kStepBytes + ((c % 32 ^ (t & 7)) * 16);
      v[u][0] = (uint32_t)c;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const bf16_t *>(g.A) +
                                                (size_t)at[u] * g.K + kb + 8 * (int)v[u][0]);
#pragma unroll
    for (int u = 0; u < U; ++u)  // (past the last piece: the last one again)
      *reinterpret_cast<u32x4_t *>(lds + to[u]) = token_order(v[u]);
  }
}

// The epilogue of sorted row p's column: v0 (gated: and v1, the up value) are
// the products.
template <int EPI>
__device__ __forceinline__ void finish(const Int4Args &g, int p, int col, float v0, float v1) {
  if constexpr (EPI == EPI_Y || EPI == EPI_OUT) {
    const float y = v0 * weight_at(g.gate_scal, g.gate_bf16, p);
    if (EPI == EPI_Y)  // summed over the slots by sum_slots_kernel, in fp32
      reinterpret_cast<float *>(g.C)[(size_t)p * g.Nout + col] = y;
    else               // one slot a token: entry == token
      reinterpret_cast<bf16_t *>(g.C)[(size_t)g.col_sorted[p] * g.Nout + col] = bf16_rne(y);
  } else {
    const float nal = -g.prm.alpha * 1.44269504088896341f;
    float a = act_val<EPI>(v0, v1, nal, g.prm);
    // the clamps and the rectifier drop a NaN; the token's row shall show it
    if (__builtin_isnan(v0) || __builtin_isnan(v1)) a = __builtin_nanf("");
    const bf16_t hi = bf16_rne(a);
    bf16_t *c = reinterpret_cast<bf16_t *>(g.C) + (size_t)2 * p * g.Nout + col;
    c[0] = hi;
    c[g.Nout] = bf16_rne(a - to_f32(hi));
  }
}

// Parts of a token row: w2 takes the activation rows as hi and lo.
template <int EPI> constexpr int parts() { return EPI == EPI_Y || EPI == EPI_OUT ? 2 : 1; }

// LDS for token rows: 128 KB leaves one workgroup a compute unit (8 experts, 64
// tokens 134 -> 173 us, 32 tokens of 64 experts 151 -> 167); 32 KB takes more parts of
// a row (136 and 159).
constexpr int kTokenLds = 64 * 1024;

// Values of a token row that LDS holds at a time where it holds `rows` rows: all
// of K, or equal parts of it in whole steps.
__host__ __device__ inline int staged_values(int K, int rows) {
  const int most = kTokenLds / (2 * rows);
  const int nstep = (K + kStepK - 1) / kStepK, parts = (K + most - 1) / most;
  return (nstep + parts - 1) / parts * kStepK;
}

// GS = G / 32.  A wave streams 32 weight rows; ks waves share them and split the
// steps; the workgroup's waves / ks column groups share the token rows in LDS.
//
// Up to `most` token rows of the expert are taken at a time, past those its weights
// are read again.  How many rows LDS is laid out for follows from the expert's own
// count, not from the average: routing is skewed, and the expert that most tokens
// take sets the layer's time (128 experts 2880 wide, groups of 64, 33 tokens, Zipf-like
// routing with exponent 1.1: 389 us, against 595 with 4 rows a pass for all because
// there are less than two an expert on average; even routing 366 and 352).
//
// w2 takes the activation rows as two parts each.  With TILES = 1 the second parts
// are the other 8 rows of the products (8 token rows a pass, nothing computed
// twice), with TILES = 2 products of their own (16 token rows a pass).
template <int EPI, int GS, int TILES>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(4))) void
expert_int4_kernel(Int4Args g, int ks, int most) {
  constexpr bool kPlain = EPI == EPI_Y || EPI == EPI_OUT || EPI == EPI_RELU2;
  constexpr int COLS = kPlain ? 32 : 16;  // output columns of a wave's 32 weight rows
  constexpr int PARTS = parts<EPI>();
  __shared__ int sel[3];
  // the token rows, kc values of each; then the waves' sums
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int place_x, want;
  place(place_x, want);
  find_expert(g.offsets, g.E, want, sel);
  const int e = __builtin_amdgcn_readfirstlane(sel[0]);
  if (e < 0) return;  // the whole workgroup
  const int row0 = __builtin_amdgcn_readfirstlane(sel[1]);
  const int cnt = __builtin_amdgcn_readfirstlane(sel[2]);

  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h = lane >> 4;  // this lane's row in a tile, its lane group
  const int K = g.K, Nout = g.Nout;
  const int cg = wave / ks, kw = wave % ks;  // column group, share of the steps
  const int n0 = (place_x * (waves / ks) + cg) * COLS;
  const bool live = n0 < Nout;  // (the last workgroup's last groups may be past the last column)

  // Gated: tile 0 the gate rows of 16 columns, tile 1 their up rows; plain: two
  // runs of 16 columns.
  WaveRows<GS> rows;
  rows.init(g, e, kPlain ? Nout : 2 * Nout, [&](int t, int x) {
    return kPlain ? n0 + 16 * t + x : g.interleaved ? 2 * (n0 + x) + t : t * Nout + n0 + x;
  });

  for (int a0 = 0; a0 < cnt; a0 += most) {
    const int na = min(most, cnt - a0);
    // token rows LDS has room for, rows of a product (the last ones may hold
    // anything: their sums are not used)
    const int room = na <= 4 ? 4 : na <= 8 ? 8 : 16, tile = PARTS / TILES * room;
    const int kc = staged_values(K, PARTS * room), rowb = PARTS * 2 * kc;
    const int x = r & (room - 1), second = TILES < PARTS && (r & room) ? kStepBytes : 0;
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int kb = 0; kb < K; kb += kc) {
      const int klen = min(kc, K - kb);
      const int s0 = kb / kStepK, ns = (klen + kStepK - 1) / kStepK, per = (ns + ks - 1) / ks;
      const int first = s0 + min(kw * per, ns), last = live ? s0 + min(kw * per + per, ns) : first;
      typename WaveRows<GS>::Codes c0, c1;
      if (first < last) rows.load(c0, first);
      if (first + 1 < last) rows.load(c1, first + 1);
      if (a0 > 0 || kb > 0) __syncthreads();
      // (four loads in flight where rows are many: 8 experts, 64 tokens 138 -> 128 us;
      // few rows gain nothing by them, one token each of four 71 -> 73)
      auto row = [&](int i) {
        const int p = row0 + a0 + i;
        return g.gather ? g.col_sorted[p] / g.topk : p;
      };
      if (PARTS * room < 16) stage_rows<1, PARTS>(g, lds, rowb, na, kb, klen, row);
      else stage_rows<4, PARTS>(g, lds, rowb, na, kb, klen, row);
      __syncthreads();
      rows.template stream<TILES, PARTS>(c0, c1, first, last, s0, lds + x * rowb + second, x & 7,
                                         acc);
    }

    // the waves' parts, through LDS that the token rows no longer need: lane
    // (h, r) holds row r of a tile for rows 4 h .. 4 h + 3 of the product
    float *red = reinterpret_cast<float *>(lds);  // [wave][tile of weights][row][17]
    __syncthreads();
    if (4 * h < tile) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) red[((wave * 2 + t) * tile + 4 * h + q) * 17 + r] = acc[t][q];
    }
    __syncthreads();
    for (int i = kw * 64 + lane; i < na * COLS && live; i += ks * 64) {
      const int col = i % COLS, trow = i / COLS;
      auto part = [&](int t, int c) {
        float v = 0.f;
        for (int w = cg * ks; w < cg * ks + ks; ++w) {
          const float *p = red + ((w * 2 + t) * tile + trow) * 17 + c;
          v += p[0];
          if (TILES < PARTS) v += p[room * 17];  // the row's second part
        }
        return v;
      };
      finish<EPI>(g, row0 + a0 + trow, n0 + col, part(kPlain ? col >> 4 : 0, col & 15),
                  kPlain ? 0.f : part(1, col & 15));
    }
  }
}

// One token: as expert_int4_kernel, on DotRows.  An expert has one row, or more in a
// routing of the caller's own that names it in several slots.
template <int EPI, int GS>
__global__ __launch_bounds__(512) void expert_int4_one_kernel(Int4Args g, int ks, int kc) {
  constexpr bool kPlain = EPI == EPI_Y || EPI == EPI_OUT || EPI == EPI_RELU2;
  constexpr int COLS = kPlain ? 32 : 16, PARTS = parts<EPI>();
  __shared__ int sel[3];
  __shared__ float red[8][2][16];
  // [PARTS][kc] bf16, [kc / 32] fp32
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int place_x, want;
  place(place_x, want);
  find_expert(g.offsets, g.E, want, sel);
  const int e = __builtin_amdgcn_readfirstlane(sel[0]);
  if (e < 0) return;  // the whole workgroup
  const int row0 = __builtin_amdgcn_readfirstlane(sel[1]);
  const int cnt = __builtin_amdgcn_readfirstlane(sel[2]);

  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int K = g.K, Nout = g.Nout;
  const int cg = wave / ks, kw = wave % ks;
  const int n0 = (place_x * (waves / ks) + cg) * COLS;
  const bool live = n0 < Nout;
  DotRows<GS> rows;
  rows.init(g, e, kPlain ? Nout : 2 * Nout, [&](int t, int x) {
    return kPlain ? n0 + 16 * t + x : g.interleaved ? 2 * (n0 + x) + t : t * Nout + n0 + x;
  });
  float *sums = reinterpret_cast<float *>(lds + PARTS * 2 * kc);
  for (int p = row0; p < row0 + cnt; ++p) {
    float acc[2] = {0.f, 0.f};
    for (int kb = 0; kb < K; kb += kc) {
      const int klen = min(kc, K - kb);
      const int s0 = kb / kStepK, ns = (klen + kStepK - 1) / kStepK, per = (ns + ks - 1) / ks;
      const int first = s0 + min(kw * per, ns), last = live ? s0 + min(kw * per + per, ns) : first;
      typename DotRows<GS>::Codes c0, c1;
      if (first < last) rows.load(c0, first);
      if (first + 1 < last) rows.load(c1, first + 1);
      if (p > row0 || kb > 0) __syncthreads();
      const int row = g.gather ? g.col_sorted[p] / g.topk : p;
      for (int c = threadIdx.x; c < klen / 8; c += blockDim.x) {
        u32x4_t v[PARTS];
#pragma unroll
        for (int u = 0; u < PARTS; ++u)
          v[u] = *reinterpret_cast<const u32x4_t *>(reinterpret_cast<const bf16_t *>(g.A) +
                                                    (size_t)(PARTS * row + u) * K + kb + 8 * c);
        float s = 0.f;  // sums of 32: four neighbouring lanes
#pragma unroll
        for (int u = 0; u < PARTS; ++u) {
          *reinterpret_cast<u32x4_t *>(lds + u * 2 * kc + 16 * c) = token_order(v[u]);
          float f[8];
          unpack(v[u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s += f[i];
        }
        s += __shfl_xor(s, 1);
        s += __shfl_xor(s, 2);
        if ((c & 3) == 0) sums[c >> 2] = s;
      }
      __syncthreads();
      rows.template stream<PARTS>(c0, c1, first, last, s0, lds, 2 * kc, sums, acc);
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      acc[t] += __shfl_xor(acc[t], 1);
      acc[t] += __shfl_xor(acc[t], 2);
    }
    if ((lane & 3) == 0) {
      red[wave][0][lane >> 2] = acc[0];
      red[wave][1][lane >> 2] = acc[1];
    }
    __syncthreads();
    if (kw != 0 || lane >= COLS || !live) continue;
    auto part = [&](int t, int c) {
      float v = 0.f;
      for (int w = wave; w < wave + ks; ++w) v += red[w][t][c];
      return v;
    };
    finish<EPI>(g, p, n0 + lane, part(kPlain ? lane >> 4 : 0, lane & 15),
                kPlain ? 0.f : part(1, lane & 15));
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

// Waves a workgroup and waves that split K, by the number of column groups of
// all experts (G): fewer waves are left to wait for memory when G is small, and
// each further wave on the same rows costs its start and a share of the sum at
// the end.  Measured (us a call, split in 4 / 2 / 1): G = 720, one token of 128
// experts, 26.6 / 27.5 / 31.8; G = 2880, four tokens, 79.5 / 69.0 / 77.4; G =
// 2048, 8 experts, 64 tokens, 176 / 128 / 142; G = 23040, 33 tokens, 420 / 392 /
// 368.  Eight waves share the token rows of one workgroup from 2048 groups on (8
// experts, 64 tokens: 123 us against 161 with four); with fewer groups four spread
// over more compute units (one token: 26.6 against 30.8).
template <int EPI, int GS>
void launch_rows(const Int4Args &a, int64_t n_tokens, int64_t M, hipStream_t s) {
  constexpr int cols = EPI == EPI_Y || EPI == EPI_OUT || EPI == EPI_RELU2 ? 32 : 16;
  constexpr int PARTS = parts<EPI>();
  const int64_t experts = M < a.E ? M : a.E, groups = (a.Nout / cols) * experts;
  const int waves = groups < 2048 ? 4 : 8;
  const int ks = groups < 1024 ? 4 : groups < 4096 ? 2 : 1;
  const int wide = cols * (waves / ks);
  const dim3 grid((unsigned)((a.Nout + wide - 1) / wide), (unsigned)experts), block(64 * waves);
  auto bytes = [&](int rows) { return (size_t)rows * staged_values(a.K, rows) * 2; };
  if (n_tokens == 1) {
    const int kc = staged_values(a.K, PARTS);
    hipLaunchKernelGGL((expert_int4_one_kernel<EPI, GS>), grid, block,
                       bytes(PARTS) + (size_t)kc / 32 * sizeof(float), s, a, ks, kc);
    return;
  }
  auto run = [&](auto tiles) {
    constexpr int TILES = decltype(tiles)::value;
    // Token rows a pass: an expert has about one a token at most, and LDS that it
    // cannot fill keeps other workgroups away.
    int most = 4;
    while (most < n_tokens && most < 16 * TILES / PARTS) most *= 2;
    size_t lds = sizeof(float) * waves * 2 * 16 * 17;
    for (int rows = 4; rows <= most; rows *= 2)
      if (bytes(PARTS * rows) > lds) lds = bytes(PARTS * rows);
    hipLaunchKernelGGL((expert_int4_kernel<EPI, GS, TILES>), grid, block, lds, s, a, ks, most);
  };
  // Products of their own for the second parts wherever an expert can have more rows
  // than a pass holds without: even routing loses up to 2 % by them (33 tokens of 128
  // experts 359 -> 366 us; groups of 32, which spill 8 registers, 427 -> 447), skewed routing and more rows
  // an expert gain (the same 33 tokens with exponent 1.1 404 -> 389, 128 tokens 912 ->
  // 773; 8 experts, 64 tokens 141 -> 128).
  if (PARTS == 2 && n_tokens > 8) run(std::integral_constant<int, PARTS>());
  else run(std::integral_constant<int, 1>());
}

template <int EPI>
hipError_t launch_groups(const Int4Args &a, int group, int64_t n_tokens, int64_t M,
                         hipStream_t s) {
  if (group == 32) launch_rows<EPI, 1>(a, n_tokens, M, s);
  else if (group == 64) launch_rows<EPI, 2>(a, n_tokens, M, s);
  else launch_rows<EPI, 4>(a, n_tokens, M, s);
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
             0, n_experts, hidden, inter, topk, 1, layout == MOE_W13_INTERLEAVED, prm};
  const bool clamp = __builtin_isfinite(prm.limit);
  hipError_t err = kind == MOE_ACT_RELU2 ? launch_groups<EPI_RELU2>(a, group, n_tokens, M, s)
                   : clamp ? launch_groups<EPI_GATED_CLAMP>(a, group, n_tokens, M, s)
                           : launch_groups<EPI_GATED>(a, group, n_tokens, M, s);
  if (err != hipSuccess) return err;
  const bool direct = topk == 1;
  Int4Args b{act, reinterpret_cast<const uint8_t *>(w2.q), reinterpret_cast<const bf16_t *>(w2.s),
             reinterpret_cast<const uint8_t *>(w2.z), direct ? out : y, r->offsets, r->col_sorted,
             r->gate_scal, r->w_dtype == MOE_BF16, n_experts, inter, hidden, topk, 0, 0, prm};
  if (direct) return launch_groups<EPI_OUT>(b, group, n_tokens, M, s);
  if ((err = launch_groups<EPI_Y>(b, group, n_tokens, M, s)) != hipSuccess) return err;
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
