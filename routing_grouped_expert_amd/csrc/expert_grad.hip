// Gradient of the grouped expert FFN, MFMA on gfx950.
//
// With h[p] = W13[e] x[t], a[p] = act(h[p]) and out[t] = sum_p w[p] W2[e] a[p]
// (p: sorted row, t: its token, e: its expert, w: its routing weight) and
// u[p] = W2[e]^T d_out[t]:
//
//   d_w[p]  = <u[p], a[p]>              d_x[t]  = sum_p W13[e]^T dh[p]
//   dh[p]   = w[p] act'(h[p]) u[p]      dW13[e] = sum_p dh[p] x[t]^T
//                                       dW2[e]  = sum_p d_out[t] (w[p] a[p])^T
//
// Four grouped products in three kernel forms.  Two data gradients run over row
// tiles as the forward products do, but contract over the weights' row index;
// the first one's epilogue turns u (never stored) into dh, w a and d_w from the
// saved h.  The weight gradients contract over an expert's rows, so their K is
// ragged and an expert without rows gets zeros.
//
// An operand that is contracted over its row index lies in LDS as it lies in
// memory: BK rows (one K each) of the tile's columns.  bf16 fragments are then
// read with the transposing LDS load (ds_read_b64_tr_b16): in each 16-lane
// group lane t addresses four columns of K row t / 4 and receives column t of
// all four rows, so two of them give the eight consecutive K of a lane's MFMA
// fragment.  No transposed copy of a weight or an activation is ever written.
// fp32 fragments are single elements and need no transposition.
//
// Loads go straight into LDS (buffer_load ... lds) through an S-stage ring; rows
// and columns outside an operand get an out-of-range offset, so the hardware
// fills in zeros.  Workgroups are persistent: their tiles form one stream of
// K-slices and the ring runs on across tile ends.
#include <cmath>
#include <type_traits>

#include "gemm_common.h"
#include "lds_dma.h"
#include "rows.h"

namespace moe {
namespace {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

template <typename T> struct Mma;
template <> struct Mma<bf16_t> {
  static constexpr int KS = 16;  // K per instruction
  typedef bf16x8_t Frag;
  __device__ static f32x16_t mma(Frag a, Frag b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
};
template <> struct Mma<float> {
  static constexpr int KS = 2;
  typedef float Frag;
  __device__ static f32x16_t mma(Frag a, Frag b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(a, b, c, 0, 0, 0);
  }
};

// ---- LDS tiles of one K-slice (RB bytes of K: 64 bf16 or 32 fp32) -------------

constexpr int RB = 128;
template <typename T> constexpr int kBK = RB / (int)sizeof(T);

// Rows of K: operand row r is RB bytes, its 16-byte chunks XOR-swizzled by r / 2
// so that the 16-byte reads of 16 consecutive rows hit distinct banks.
__device__ __forceinline__ int row_key(int r) { return (r >> 1) & 7; }

// Columns of K: K row r is COLS elements.  A bf16 transposing read takes, from
// each of four K rows, 64 bytes at the same columns (two 16-lane groups), which
// the key spreads over the 256-byte bank line; an fp32 read takes 128 bytes from
// each of two K rows.
template <typename T> __device__ __forceinline__ int col_key(int r) {
  return std::is_same<T, bf16_t>::value ? (r & 3) << 2 : (r & 1) << 3;
}

// Operand tile of ROWS rows, K contiguous, NW waves loading.
template <typename T, int ROWS, int NW> struct RowTile {
  static constexpr int BYTES = ROWS * RB, J = BYTES / 1024 / NW;
  static_assert(J * NW * 1024 == BYTES, "whole loads a wave");
  // line (here: operand row) and byte inside it that load j of a wave brings to its lane
  __device__ static int line(int wave, int lane, int j) { return (wave * J + j) * 8 + (lane >> 3); }
  __device__ static int byte(int wave, int lane, int j) {
    return ((lane & 7) ^ row_key(line(wave, lane, j))) << 4;
  }
  __device__ static typename Mma<T>::Frag frag(const char *p, int ks, int r, int lane) {
    constexpr int EPL = sizeof(typename Mma<T>::Frag) / sizeof(T);
    const int b = (ks * Mma<T>::KS + (lane >> 5) * EPL) * (int)sizeof(T);
    r += lane & 31;
    return *reinterpret_cast<const typename Mma<T>::Frag *>(
        p + r * RB + (((b >> 4) ^ row_key(r)) << 4) + (b & 15));
  }
};

// Operand tile of COLS columns, K rows, NW waves loading.
template <typename T, int COLS, int NW> struct ColTile {
  static constexpr int BYTES = COLS * RB, J = BYTES / 1024 / NW;
  static constexpr int ROWB = COLS * (int)sizeof(T), CPR = ROWB / 16;
  static_assert(J * NW * 1024 == BYTES, "whole loads a wave");
  static_assert(CPR >= 16, "a K row spans the banks");
  __device__ static int line(int wave, int lane, int j) {  // (here: K row)
    return ((wave * J + j) * 64 + lane) / CPR;
  }
  __device__ static int byte(int wave, int lane, int j) {
    return ((lane % CPR) ^ col_key<T>(line(wave, lane, j))) << 4;
  }
  __device__ static typename Mma<T>::Frag frag(const char *p, int ks, int c, int lane) {
    if constexpr (std::is_same<T, bf16_t>::value) {
      typedef short s16x4_t __attribute__((ext_vector_type(4)));
      typedef short s16x8_t __attribute__((ext_vector_type(8)));
      typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
      // K row t / 4 of four (its key is that of every ks), columns 4 (t % 4) ..
      const int t = lane & 15, k = ks * 16 + (lane >> 5) * 8 + (t >> 2);
      const int b = (c + ((lane >> 4) & 1) * 16 + (t & 3) * 4) * 2;
      const char *q = p + k * ROWB + (((b >> 4) ^ ((t >> 2) << 2)) << 4) + (b & 15);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t *)q);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t *)(q + 4 * ROWB));
      const s16x8_t v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      return __builtin_bit_cast(bf16x8_t, v);
    } else {
      const int k = ks * 2 + (lane >> 5), b = (c + (lane & 31)) * 4;
      return *reinterpret_cast<const float *>(p + k * ROWB +
                                              (((b >> 4) ^ col_key<T>(k)) << 4) + (b & 15));
    }
  }
};

// ---- arguments -------------------------------------------------------------------

struct GradArgs {
  const void *A;                // data gradients: rows [.., K]; weight gradients: [rows, M]
  const void *B;                // data gradients: weights [E, K, N]; weight gradients: [rows, N]
  void *C;                      // [rows, N] / [E, M, N]
  const int32_t *offsets;       // [E + 1]
  const int32_t *col_sorted;    // [rows]
  uint32_t a_bytes, b_bytes;    // buffer ranges (b_bytes: of one expert's weights)
  uint32_t c_bytes;             // (of one expert in the weight gradients)
  int E, K, M, N;
  uint32_t div_mul, div_shift;  // f / topk = (f * div_mul) >> div_shift
  // epilogue of the first data gradient
  const void *h;                // [rows, sets * N]
  void *dh, *wa;                // [rows, sets * N], [rows, N]
  float *part;                  // [column slabs, rows]: parts of d_w
  const void *gate_scal;        // [rows]
  int64_t rows;                 // n_tokens * topk
  uint32_t h_bytes;
  int gate_bf16, interleaved;
  ActParams prm;
};

__device__ __forceinline__ uint32_t token_of(const GradArgs &g, int f) {
  return (uint32_t)(((uint64_t)(uint32_t)f * g.div_mul) >> g.div_shift);
}

// Gradient kinds, and whose rows are gathered: row p of A (1) or B (2) is that of
// token col_sorted[p] / topk.
enum { GRAD_ACT = 0, GRAD_ROWS = 1, GRAD_WEIGHT = 2 };
// Activation kinds of GRAD_ACT.
enum { ACT_GATED = 0, ACT_RELU2 = 1 };

// a, and the derivatives of a with respect to the gate and up products.
template <int ACT>
__device__ __forceinline__ void act_grad(float g, float v, const ActParams &p, float &a, float &dg,
                                         float &dv) {
  if constexpr (ACT == ACT_RELU2) {
    const float r = fmaxf(g, 0.f);
    a = r * r;
    dg = 2.f * r;
    dv = 0.f;
  } else {
    const bool gin = g <= p.limit, vin = fabsf(v) <= p.limit;
    g = fminf(g, p.limit);
    v = fminf(fmaxf(v, -p.limit), p.limit);
    // the logistic function as 1 / (1 + 2^(-alpha log2(e) g)), as the forward pass
    const float ag = p.alpha * g;
    const float s =
        __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * ag));
    const float gs = g * s, vb = v + p.beta;
    a = gs * vb;
    dg = gin ? s * (1.f + ag * (1.f - s)) * vb : 0.f;
    dv = vin ? gs : 0.f;
  }
}

// ---- tiles -----------------------------------------------------------------------

// Tiles of an expert are walked in blocks of GM x GN (n-block outer, m-block
// inner, m-tile fastest inside a block), so the workgroups an XCD runs at a time
// share both operands' tiles in its L2.
constexpr int GM = 8, GN = 4;

struct Tile {
  int e, row0, rows, m0, n0;  // expert, its rows of this tile, output position
};

__device__ __forceinline__ void tile_place(int l, int mt_all, int nt_all, int &mt, int &nt) {
  const int nb = l / (GN * mt_all);
  const int gn = min(GN, nt_all - nb * GN);
  const int r = l - nb * GN * mt_all;
  const int mb = r / (GM * gn);
  const int gm = min(GM, mt_all - mb * GM);
  const int r2 = r - mb * GM * gn;
  mt = mb * GM + r2 % gm;
  nt = nb * GN + r2 / gm;
}

// A value that every lane holds, in a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Last e in [0, E) with s[e] <= v (s ascending, s[0] <= v).
__device__ __forceinline__ int find_expert(const int *s, int E, int v) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (uniform(s[mid]) <= v) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// One expert's units (row tiles, or K-slices: at least `least`) summed up to each
// expert, and the routing offsets, in LDS; one wave, four experts a lane.
template <int UNIT>
__device__ __forceinline__ void expert_units(const GradArgs &g, int least, int *s_unit, int *s_off,
                                             int lane) {
  int v[4], s = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = lane * 4 + q;
    const int o0 = e < g.E ? g.offsets[e] : 0;
    const int o1 = e < g.E ? g.offsets[e + 1] : 0;
    if (e < g.E) s_off[e] = o0;
    v[q] = e < g.E ? max(least, (o1 - o0 + UNIT - 1) / UNIT) : 0;
    s += v[q];
  }
  const int incl = wave_inclusive_sum(s);
  int run = incl - s;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = lane * 4 + q;
    if (e < g.E) s_unit[e] = run;
    run += v[q];
  }
  if (lane == 63) {
    s_unit[g.E] = incl;
    s_off[g.E] = g.offsets[g.E];
  }
}

// ---- the kernel --------------------------------------------------------------------
//
// Tile of BM x BN outputs, WM x WN waves, S-stage ring.  Eight waves run the
// ping-pong schedule: waves 0-3 and 4-7 (one of each a SIMD) alternate between a
// memory phase (next slice's loads out, this slice's fragments into registers)
// and an MFMA phase, one group a barrier behind the other.  Four waves read the
// fragments of the next k-step while the current one multiplies; with 256-row
// tiles (one wave a SIMD, 128 x 128 each) every memory instruction is placed
// behind an MFMA by hand.
//
// The MFMA takes the N-side fragment first: lane l ends with output row l % 32 of
// a 32 x 32 sub-tile and, in register group q, columns 8 q + 4 (l / 32) + [0, 4).
template <typename T, int KIND, int ACT, int GATHER, int BM, int BN, int WM, int WN, int S>
__device__ __forceinline__ void grad_body(const GradArgs &g) {
  using Mm = Mma<T>;
  using Frag = typename Mm::Frag;
  constexpr bool BF = std::is_same<T, bf16_t>::value;
  constexpr int NW = WM * WN, BK = kBK<T>, NKS = BK / Mm::KS, ES = (int)sizeof(T);
  constexpr bool WG = KIND == GRAD_WEIGHT;
  using TA = typename std::conditional<WG, ColTile<T, BM, NW>, RowTile<T, BM, NW>>::type;
  using TB = ColTile<T, BN, NW>;
  constexpr int STAGE = TA::BYTES + TB::BYTES, JA = TA::J, JB = TB::J, PER = JA + JB;
  constexpr int TM = BM / WM / 32, TN = BN / WN / 32, WC = BN / WN;
  constexpr int SETS = KIND == GRAD_ACT && ACT == ACT_GATED ? 2 : 1;
  // stores a wave's epilogue issues at least (the ring's waits count them)
  constexpr int NPART = BF ? 2 : 4;  // pieces of a sub-tile row a lane
  constexpr int NST = TM * TN * NPART * (KIND == GRAD_ACT ? SETS + 1 : 1);
  constexpr bool PP = NW == 8;
  constexpr bool BIG = NW == 4 && BM == 256;  // one wave a SIMD
  static_assert(!BIG || (BF && S == 2 && NKS >= 4), "four-wave tiles");
  static_assert(TM * 32 * WM == BM && TN * 32 * WN == BN && S >= 2 && (S - 2) * PER < 64, "tile");

  __shared__ __attribute__((aligned(16))) char smem[S * STAGE];
  __shared__ int s_unit[kMaxExperts + 1], s_off[kMaxExperts + 1];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  if (wave == 0) expert_units<WG ? BK : BM>(g, WG ? 1 : 0, s_unit, s_off, lane);
  __syncthreads();

  // this workgroup's tiles: first, first + stride, ... below end.  The tile order
  // is cut into one run for each XCD (workgroup b runs on XCD b % 8): of equal
  // tile counts, or in the weight gradients of equal K-slice counts
  const int n_nt = (g.N + BN - 1) / BN, n_mt = WG ? (g.M + BM - 1) / BM : 0;
  const int per_e = n_mt * n_nt, stride = (int)gridDim.x / 8, xcd = (int)blockIdx.x % 8;
  auto cut = [&](int c) -> int {
    if constexpr (WG) {
      if (c == 8) return g.E * per_e;
      const int64_t want = (int64_t)uniform(s_unit[g.E]) * per_e * c / 8;
      const int e = find_expert(s_unit, g.E, (int)(want / per_e));
      const int before = uniform(s_unit[e]), nk = uniform(s_unit[e + 1]) - before;
      return e * per_e + (int)((want - (int64_t)before * per_e) / nk);
    } else {
      const int total = uniform(s_unit[g.E]) * n_nt;
      return min(total, c * ((total + 7) / 8));
    }
  };
  const int first = cut(xcd) + (int)blockIdx.x / 8, end = cut(xcd + 1);
  if (first >= end) return;

  auto tile_of = [&](int L) -> Tile {
    Tile t;
    int mt, nt;
    if constexpr (WG) {
      t.e = L / per_e;
      tile_place(L - t.e * per_e, n_mt, n_nt, mt, nt);
      t.row0 = uniform(s_off[t.e]);
      t.rows = uniform(s_off[t.e + 1]) - t.row0;
      t.m0 = mt * BM;
    } else {
      t.e = find_expert(s_unit, g.E, L / n_nt);
      const int before = uniform(s_unit[t.e]);
      tile_place(L - before * n_nt, uniform(s_unit[t.e + 1]) - before, n_nt, mt, nt);
      t.row0 = uniform(s_off[t.e]) + mt * BM;
      t.rows = min(BM, uniform(s_off[t.e + 1]) - t.row0);
      t.m0 = 0;
    }
    t.n0 = nt * BN;
    return t;
  };
  auto slices = [&](const Tile &t) { return ((WG ? max(t.rows, 1) : g.K) + BK - 1) / BK; };

  // ---- loading side: slice k_in of tile L_in is the next to load ----------------
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void *>(g.A), (short)0, (int)g.a_bytes, kRsrcWord3);
  __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<void *>(g.B), (short)0, (int)g.b_bytes, kRsrcWord3);
  const uint32_t arow = (uint32_t)((WG ? g.M : g.K) * ES), brow = (uint32_t)(g.N * ES);
  uint32_t va[JA], vb[JB];  // a lane's offsets that hold for the whole tile
  uint32_t oa[JA], ob[JB];  // and those of the next slice
  // col_sorted of the gathered operand's rows in the next slice (weight gradients) or
  // tile, read ahead of their use (rows past the end read any valid entry)
  constexpr bool GA = GATHER == 1, GB = GATHER == 2;
  int ia[GA ? JA : 1], ib[GB ? JB : 1];
  Tile in{};
  int L_in = first, k_in = 0, nk_in = 0, z_in = 0;  // z_in: slices loaded so far
  auto fetch = [&](const Tile &t, int k0) {
    const int last = t.row0 + t.rows - 1;
    if (t.rows == 0) return;
    if constexpr (GA) {
#pragma unroll
      for (int j = 0; j < JA; ++j)
        ia[j] = g.col_sorted[min(t.row0 + k0 + TA::line(wave, lane, j), last)];
    }
    if constexpr (GB) {
#pragma unroll
      for (int j = 0; j < JB; ++j)
        ib[j] = g.col_sorted[min(t.row0 + k0 + TB::line(wave, lane, j), last)];
    }
  };
  // Offsets of tile L_in, whose gather indices are there.
  auto begin_tile = [&]() {
    in = tile_of(L_in);
    nk_in = slices(in);
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      if constexpr (WG) {
        const int b = in.m0 * ES + TA::byte(wave, lane, j);
        va[j] = b < (int)arow ? (uint32_t)b : kOOB;
      } else {
        const int r = TA::line(wave, lane, j);
        const uint32_t row = GA ? token_of(g, ia[GA ? j : 0]) : (uint32_t)(in.row0 + r);
        va[j] = r < in.rows ? row * arow + TA::byte(wave, lane, j) : kOOB;
      }
    }
    if constexpr (!WG)
      rb = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char *>(reinterpret_cast<const char *>(g.B)) + (size_t)in.e * g.b_bytes,
          (short)0, (int)g.b_bytes, kRsrcWord3);
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int b = in.n0 * ES + TB::byte(wave, lane, j);
      vb[j] = b < (int)brow ? (uint32_t)b : kOOB;
      // (out of range it stays so: an expert's weights are below 2^31 bytes)
      if constexpr (!WG) vb[j] += (uint32_t)TB::line(wave, lane, j) * brow;
    }
    if constexpr (GA && !WG)
      if (L_in + stride < end) fetch(tile_of(L_in + stride), 0);
  };
  // Offset of load j of the next slice, A and B; past the last tile out of range.
  auto prep_a = [&](int j) {
    if constexpr (WG) {
      const int k = k_in * BK + TA::line(wave, lane, j);
      const uint32_t row = GA ? token_of(g, ia[GA ? j : 0]) : (uint32_t)(in.row0 + k);
      oa[j] = L_in < end && k < in.rows && va[j] != kOOB ? row * arow + va[j] : kOOB;
    } else {
      const int kb = k_in * RB;  // (a row is a whole number of 16-byte chunks)
      const bool past = L_in >= end || kb + TA::byte(wave, lane, j) >= (int)arow;
      oa[j] = past ? kOOB : va[j] + (uint32_t)kb;
    }
  };
  auto prep_b = [&](int j) {
    const int k = k_in * BK + TB::line(wave, lane, j);
    if constexpr (WG) {
      const uint32_t row = GB ? token_of(g, ib[GB ? j : 0]) : (uint32_t)(in.row0 + k);
      ob[j] = L_in < end && k < in.rows && vb[j] != kOOB ? row * brow + vb[j] : kOOB;
    } else {
      ob[j] = L_in >= end || k >= g.K ? kOOB : vb[j] + (uint32_t)(k_in * BK) * brow;
    }
  };
  auto load_a = [&](char *base, int j) { dma16(ra, base + (wave * JA + j) * 1024, oa[j]); };
  auto load_b = [&](char *base, int j) {
    dma16(rb, base + TA::BYTES + (wave * JB + j) * 1024, ob[j]);
  };
  // The gather indices of the slice after the next one (the next one's are in use).
  auto ahead = [&]() {
    if constexpr (WG && GATHER) {
      if (k_in + 1 < nk_in) fetch(in, (k_in + 1) * BK);
      else if (L_in + stride < end) fetch(tile_of(L_in + stride), 0);
    }
  };
  // On to the slice after this one, whose loads are out.
  auto advance = [&]() {
    ++z_in;
    if (++k_in < nk_in) return;
    k_in = 0;
    L_in += stride;
    if (L_in < end) begin_tile();
  };
  auto issue = [&]() {
    char *base = smem + (z_in % S) * STAGE;
#pragma unroll
    for (int j = 0; j < JB; ++j) prep_b(j);
#pragma unroll
    for (int j = 0; j < JA; ++j) prep_a(j);
    ahead();
#pragma unroll
    for (int j = 0; j < JB; ++j) load_b(base, j);
#pragma unroll
    for (int j = 0; j < JA; ++j) load_a(base, j);
    advance();
  };

  // ---- multiplying side ------------------------------------------------------------
  f32x16_t acc[TM][TN];
  auto zero_acc = [&]() {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  };
  int st_until = -1;  // last slice whose wait must also cover the latest epilogue's stores
  // slice w is in LDS as far as this wave's loads go (and its LDS reads are done)
  auto wait_slice = [&](int w) {
    wait_pending<PER, NST, S - 2>(min(S - 2, z_in - 1 - w), w <= st_until);
  };
  // Piece c of a lane's share of sub-tile (i, j): NV consecutive columns of its
  // row, from column piece_col(c).  In bf16 register groups 2c and 2c + 1 hold 4
  // of 8 + 8 columns each in lanes l and l + 32; exchanging the halves gives
  // each lane 8 consecutive ones, a 16-byte piece.
  constexpr int NV = 16 / ES;
  auto piece = [&](int i, int j, int c, float (&v)[NV]) {
    if constexpr (BF) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[i][j][8 * c + t]),
                                                        __float_as_uint(acc[i][j][8 * c + 4 + t]),
                                                        false, false);
        v[t] = __uint_as_float(s[0]);
        v[4 + t] = __uint_as_float(s[1]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < 4; ++t) v[t] = acc[i][j][4 * c + t];
    }
  };
  // (four-wave tiles: the accumulators stay in AGPRs up to their sub-tile, and the
  // sub-tiles apart: reading them all early would need 256 more registers)
  auto hold = [&](int i, int j) {
    if constexpr (BIG) {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" : "+a"(acc[i][j]));
    }
  };
  auto piece_col = [&](int c) { return BF ? 16 * c + 8 * (lane >> 5) : 8 * c + 4 * (lane >> 5); };
  auto put = [&](__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[NV]) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4_t, pack(v)), r, (int)off, 0, 0);
  };

  auto epilogue = [&](const Tile &t, int z) {
    if constexpr (KIND == GRAD_ACT) {
      const __amdgpu_buffer_rsrc_t rh = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<void *>(g.h), (short)0, (int)g.h_bytes, kRsrcWord3);
      const __amdgpu_buffer_rsrc_t rdh =
          __builtin_amdgcn_make_buffer_rsrc(g.dh, (short)0, (int)g.h_bytes, kRsrcWord3);
      const __amdgpu_buffer_rsrc_t rwa =
          __builtin_amdgcn_make_buffer_rsrc(g.wa, (short)0, (int)g.c_bytes, kRsrcWord3);
      const int slab = (t.n0 + wn * WC) / WC;
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int m = wm * (BM / WM) + i * 32 + (lane & 31);
        const bool ok = m < t.rows;
        const uint32_t p = (uint32_t)(t.row0 + (ok ? m : 0));
        const float w = weight_at(g.gate_scal, g.gate_bf16, p);
        float sum = 0.f;  // this lane's part of d_w
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          hold(i, j);
#pragma unroll
          for (int c = 0; c < NPART; ++c) {
            const int col = t.n0 + wn * WC + j * 32 + piece_col(c);
            const bool in_range = ok && col < g.N;
            const uint32_t row_h = p * (uint32_t)(SETS * g.N);
            // the gate and up chunks, or the pairs of columns [0, NV / 2) and the rest
            const uint32_t c0 = SETS == 1 ? (uint32_t)col
                                : g.interleaved ? (uint32_t)(2 * col) : (uint32_t)col;
            const uint32_t c1 = g.interleaved ? (uint32_t)(2 * col + NV) : (uint32_t)(g.N + col);
            const uint32_t o0 = in_range ? (row_h + c0) * ES : kOOB;
            const uint32_t o1 = in_range ? (row_h + c1) * ES : kOOB;
            float u[NV], h0[NV], h1[NV], gate[NV], up[NV], a[NV], dg[NV], dv[NV];
            piece(i, j, c, u);
            unpack(__builtin_bit_cast(u32x4_t,
                                      __builtin_amdgcn_raw_buffer_load_b128(rh, (int)o0, 0, 0)), h0);
            if constexpr (SETS == 2)
              unpack(__builtin_bit_cast(
                         u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rh, (int)o1, 0, 0)), h1);
#pragma unroll
            for (int q = 0; q < NV; ++q) {
              gate[q] = h0[q];
              up[q] = SETS == 2 ? h1[q] : 0.f;
              if (SETS == 2 && g.interleaved) {
                gate[q] = q < NV / 2 ? h0[(2 * q) % NV] : h1[(2 * q) % NV];
                up[q] = q < NV / 2 ? h0[(2 * q + 1) % NV] : h1[(2 * q + 1) % NV];
              }
              act_grad<ACT>(gate[q], up[q], g.prm, a[q], dg[q], dv[q]);
              sum += in_range ? u[q] * a[q] : 0.f;
              const float wu = w * u[q];
              a[q] *= w;
              dg[q] *= wu;
              dv[q] *= wu;
            }
            put(rwa, in_range ? (p * (uint32_t)g.N + (uint32_t)col) * ES : kOOB, a);
            if constexpr (SETS == 1) {
              put(rdh, o0, dg);
            } else {
#pragma unroll
              for (int q = 0; q < NV; ++q) {
                h0[q] = dg[q];
                h1[q] = dv[q];
                if (g.interleaved) {
                  h0[q] = q % 2 ? dv[q / 2] : dg[q / 2];
                  h1[q] = q % 2 ? dv[NV / 2 + q / 2] : dg[NV / 2 + q / 2];
                }
              }
              put(rdh, o0, h0);
              put(rdh, o1, h1);
            }
          }
        }
        sum += __shfl_xor(sum, 32);
        if (ok && lane < 32 && slab * WC < g.N) g.part[(int64_t)slab * g.rows + p] = sum;
      }
    } else {
      const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
          reinterpret_cast<char *>(g.C) + (WG ? (size_t)t.e * g.c_bytes : 0), (short)0,
          (int)g.c_bytes, kRsrcWord3);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const int m = wm * (BM / WM) + i * 32 + (lane & 31);
        const bool ok = WG ? t.m0 + m < g.M : m < t.rows;
        const uint32_t row = (uint32_t)((WG ? t.m0 : t.row0) + m);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          hold(i, j);
#pragma unroll
          for (int c = 0; c < NPART; ++c) {
            const int col = t.n0 + wn * WC + j * 32 + piece_col(c);
            float v[NV];
            piece(i, j, c, v);
            put(rc, ok && col < g.N ? (row * (uint32_t)g.N + (uint32_t)col) * ES : kOOB, v);
          }
        }
      }
    }
    st_until = z + S - 1 + (BIG ? 1 : 0);  // (four waves load a slice further ahead)
  };

  if constexpr (GA && !WG) fetch(tile_of(first), 0);
  begin_tile();
  if constexpr (WG && GATHER) fetch(in, 0);
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (L_in < end) issue();

  Tile cur = tile_of(first);
  int nk = slices(cur), kt = 0, L = first;
  auto frag_a = [&](const char *p, int ks, int i) {
    return TA::frag(p, ks, wm * (BM / WM) + i * 32, lane);
  };
  auto frag_b = [&](const char *p, int ks, int j) {
    return TB::frag(p + TA::BYTES, ks, wn * WC + j * 32, lane);
  };
  auto bar = [&]() {  // workgroup barrier; MFMAs may cross it
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  auto next = [&]() {  // the slice after this one (its tile's first: the next tile)
    if (++kt < nk) return;
    kt = 0;
    L += stride;
    cur = tile_of(L);
    nk = slices(cur);
  };

  if constexpr (PP) {
    const int grp = wave >> 2;
    Frag fa[NKS][TM], fb[NKS][TN];
    wait_slice(0);
    barrier();
    if (grp) barrier();  // group 1 runs one phase behind group 0
    for (int z = 0;; ++z) {
      const bool done = kt + 1 == nk && L + stride >= end;
      if (L_in < end) issue();
      const char *p = smem + (z % S) * STAGE;
#pragma unroll
      for (int ks = 0; ks < NKS; ++ks) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[ks][i] = frag_a(p, ks, i);
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[ks][j] = frag_b(p, ks, j);
      }
      if (grp && !done) wait_slice(z + 1);
      barrier();
      __builtin_amdgcn_s_setprio(1);
      if (kt == 0) zero_acc();
#pragma unroll
      for (int ks = 0; ks < NKS; ++ks)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = Mm::mma(fb[ks][j], fa[ks][i], acc[i][j]);
      __builtin_amdgcn_s_setprio(0);
      if (kt + 1 == nk) epilogue(cur, z);
      if (!grp && !done) wait_slice(z + 1);
      barrier();
      if (done) break;
      next();
    }
    if (!grp) barrier();
  } else if constexpr (BIG) {
    // One wave a SIMD: nothing else fills the matrix core while this wave issues
    // other work, so each memory instruction follows an MFMA.
    //  * k-step 0: the load offsets of slice z + 2; k-step 1: the gather indices of
    //    slice z + 3 (the wait in k-step NKS - 2 covers them).
    //  * k-steps before the last: the fragments of the next k-step.
    //  * k-step NKS - 2, once its reads are out: the wait for slice z + 1 and the
    //    barrier (after which no wave reads slot z % 2 again), then the first loads
    //    of slice z + 2 into that slot.
    //  * last k-step: its other loads, then slice z + 1's first fragments.
    constexpr int NM = TM * TN, NF = TM + TN, NL = JA + JB;
    static_assert(!BIG || NL <= NM, "a load offset after each MFMA");
    Frag fa[2][TM], fb[2][TN];
    auto read = [&](int buf, const char *p, int ks, int f) {
      if (f < TM) fa[buf][f] = frag_a(p, ks, f);
      else fb[buf][f - TM] = frag_b(p, ks, f - TM);
    };
    auto load = [&](char *base, int q) {
      if (q < JB) load_b(base, q);
      else load_a(base, q - JB);
    };
    wait_vm<0>();
    barrier();
    issue();  // (past the last slice: zeros)
#pragma unroll
    for (int f = 0; f < NF; ++f) read(0, smem, 0, f);
    int z = 0;
#pragma nounroll
    for (;;) {
      zero_acc();
#pragma nounroll
      for (int k = 0; k < nk; ++k, ++z) {
        char *here = smem + (z & 1) * STAGE, *other = smem + ((z + 1) & 1) * STAGE;
#pragma unroll
        for (int ks = 0; ks < NKS; ++ks) {
          constexpr int D0 = NM - NF - 1;   // loads that k-step NKS - 2 has room for
          constexpr int NQ = NL - D0 + NF;  // memory instructions of the last k-step
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            const int i = m / TN, j = m % TN;
            acc[i][j] = Mm::mma(fb[ks & 1][j], fa[ks & 1][i], acc[i][j]);
            if (ks == 0 && m < NL) {
              if (m < JB) prep_b(m);
              else prep_a(m - JB);
            }
            if (ks == 1 && m == 0) ahead();
            if (ks + 2 < NKS) {
              if (m % 2 == 0) read((ks + 1) & 1, here, ks + 1, m / 2);
            } else if (ks + 2 == NKS) {
              if (m < NF) {
                read((ks + 1) & 1, here, ks + 1, m);
              } else if (m == NF) {
                if (!(WG && GATHER) && z + 1 <= st_until) wait_vm<vm_cap(NST)>();
                else wait_vm<0>();
                bar();
              } else {
                load(here, m - NF - 1);
              }
            } else {
#pragma unroll
              for (int q = 0; q < NQ; ++q) {
                if (q * NM / NQ != m) continue;
                if (q < NL - D0) load(here, D0 + q);
                else read((ks + 1) & 1, other, 0, q - (NL - D0));
              }
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        advance();
      }
      epilogue(cur, z - 1);
      L += stride;
      if (L >= end) break;
      cur = tile_of(L);
      nk = slices(cur);
    }
    wait_vm<0>();  // the loads past the last slice have landed
  } else {
    for (int z = 0;; ++z) {
      const bool done = kt + 1 == nk && L + stride >= end;
      wait_slice(z);
      barrier();
      if (L_in < end) issue();
      if (kt == 0) zero_acc();
      const char *p = smem + (z % S) * STAGE;
      Frag fa[2][TM], fb[2][TN];
      auto load = [&](int ks) {
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[ks & 1][i] = frag_a(p, ks, i);
#pragma unroll
        for (int j = 0; j < TN; ++j) fb[ks & 1][j] = frag_b(p, ks, j);
      };
      load(0);
#pragma unroll
      for (int ks = 0; ks < NKS; ++ks) {
        if (ks + 1 < NKS) load(ks + 1);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = Mm::mma(fb[ks & 1][j], fa[ks & 1][i], acc[i][j]);
      }
      if (kt + 1 == nk) epilogue(cur, z);
      if (done) break;
      next();
    }
  }
}

template <typename T, int KIND, int ACT, int GATHER, int BM, int BN, int WM, int WN, int S>
__global__ __launch_bounds__(64 * WM * WN) void grad_gemm(GradArgs g) {
  grad_body<T, KIND, ACT, GATHER, BM, BN, WM, WN, S>(g);
}

// The four-wave 256-row tiles: one wave a SIMD, which may then hold the whole
// register file (256 accumulator registers for its 128 x 128 outputs).
template <typename T, int KIND, int ACT, int GATHER>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void grad_gemm_w4(
    GradArgs g) {
  grad_body<T, KIND, ACT, GATHER, 256, 256, 2, 2, 2>(g);
}

// d_topk_w of entry f: the column slabs' parts of its sorted row, added in order;
// 0 for a slot outside an expert share.
__global__ __launch_bounds__(256) void join_weight_grad(const float *__restrict__ part,
                                                        const int32_t *__restrict__ row_sorted,
                                                        float *__restrict__ d_topk_w, int64_t rows,
                                                        int slabs) {
  const int64_t f = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (f >= rows) return;
  const int p = row_sorted[f];
  float s = 0.f;
  if (p >= 0)
    for (int i = 0; i < slabs; ++i) s += part[i * rows + p];
  d_topk_w[f] = s;
}

// Weight gradients of a call without tokens.
__global__ __launch_bounds__(256) void zero_kernel(u32x4_t *__restrict__ p, int64_t chunks) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < chunks; i += (int64_t)gridDim.x * 256)
    p[i] = u32x4_t{0u, 0u, 0u, 0u};
}

// Activation rows of the forward pass from its saved products: one 16-byte chunk
// of act a thread.
template <typename T, int ACT>
__global__ __launch_bounds__(256) void activation_kernel(const T *__restrict__ h,
                                                         T *__restrict__ act,
                                                         const int32_t *__restrict__ offsets,
                                                         int E, int inter, int interleaved,
                                                         int64_t chunks, ActParams prm) {
  constexpr int NV = 16 / (int)sizeof(T);
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int nch = inter / NV;
  if (idx >= chunks) return;
  const int64_t p = idx / nch;
  const int c = (int)(idx - p * nch);
  if (p >= offsets[E]) return;
  const u32x4_t *row = reinterpret_cast<const u32x4_t *>(h + p * (ACT == ACT_RELU2 ? 1 : 2) * inter);
  float h0[NV], h1[NV], a[NV], dg, dv;
  unpack(row[interleaved ? 2 * c : c], h0);
  if constexpr (ACT == ACT_GATED) unpack(row[interleaved ? 2 * c + 1 : nch + c], h1);
#pragma unroll
  for (int q = 0; q < NV; ++q) {
    float gate = h0[q], up = ACT == ACT_GATED ? h1[q] : 0.f;
    if (ACT == ACT_GATED && interleaved) {
      gate = q < NV / 2 ? h0[(2 * q) % NV] : h1[(2 * q) % NV];
      up = q < NV / 2 ? h0[(2 * q + 1) % NV] : h1[(2 * q + 1) % NV];
    }
    act_grad<ACT>(gate, up, prm, a[q], dg, dv);
  }
  reinterpret_cast<u32x4_t *>(act + p * inter)[c] = pack(a);
}

// ---- launches ------------------------------------------------------------------------

int device_cus() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      cus <= 0)
    cus = 256;
  return cus;
}

template <typename T, int KIND, int ACT, int GATHER, int BM, int BN, int WM, int WN, int S>
hipError_t launch(const GradArgs &g, int64_t tiles, hipStream_t s) {
  constexpr int LDS = S * RB * (BM + BN) + 2 * (kMaxExperts + 1) * 4;
  static_assert(LDS <= 160 * 1024, "LDS budget");
  constexpr int per_cu = 160 * 1024 / LDS < 2 ? 1 : 2;
  int64_t grid = (int64_t)device_cus() * per_cu;
  if (grid > tiles) grid = tiles;
  grid = (grid + 7) / 8 * 8;  // whole XCD rounds; surplus workgroups get no tiles
  if constexpr (BM == 256 && WM * WN == 4)
    hipLaunchKernelGGL((grad_gemm_w4<T, KIND, ACT, GATHER>), dim3((unsigned)grid), dim3(256), 0, s,
                       g);
  else
    hipLaunchKernelGGL((grad_gemm<T, KIND, ACT, GATHER, BM, BN, WM, WN, S>), dim3((unsigned)grid),
                       dim3(64 * WM * WN), 0, s, g);
  return hipGetLastError();
}

inline int64_t cover(int64_t n, int64_t unit) { return (n + unit - 1) / unit; }

// Data gradients: tiles of 256 rows where they cover the compute units, of 128
// rows below that, and of 32 rows where experts hold fewer than 48 rows.
// Returns the columns of a slab of d_w parts in *slab.
template <typename T, int KIND, int ACT, int GATHER>
hipError_t launch_rows(const GradArgs &g, hipStream_t s, int *slab) {
  const int64_t cus = device_cus(), most = g.rows < g.E ? g.rows : g.E;
  auto expected = [&](int bm, int bn) {
    return (g.rows / bm + (most + 1) / 2) * cover(g.N, bn);
  };
  auto tiles = [&](int bm, int bn) { return (g.rows / bm + most) * cover(g.N, bn); };
  if (g.rows < 48 * (int64_t)g.E || expected(128, 128) < cus / 2) {
    *slab = 32;
    return launch<T, KIND, ACT, GATHER, 32, 128, 1, 4, 4>(g, tiles(32, 128), s);
  }
  if (expected(256, 256) >= cus) {
    *slab = 128;
    // (fp32 accumulates at a sixteenth of the rate: nothing to place by hand)
    constexpr int WM = std::is_same<T, bf16_t>::value ? 2 : 4;
    return launch<T, KIND, ACT, GATHER, 256, 256, WM, 2, 2>(g, tiles(256, 256), s);
  }
  *slab = 32;
  return launch<T, KIND, ACT, GATHER, 128, 128, 2, 4, 3>(g, tiles(128, 128), s);
}

// Weight gradients: 256 x 256 tiles where they cover the compute units.
template <typename T, int GATHER> hipError_t launch_weights(const GradArgs &g, hipStream_t s) {
  const int64_t big = g.E * cover(g.M, 256) * cover(g.N, 256);
  constexpr int WM = std::is_same<T, bf16_t>::value ? 2 : 4;
  if (big >= device_cus()) return launch<T, GRAD_WEIGHT, 0, GATHER, 256, 256, WM, 2, 2>(g, big, s);
  return launch<T, GRAD_WEIGHT, 0, GATHER, 128, 128, 2, 4, 3>(
      g, g.E * cover(g.M, 128) * cover(g.N, 128), s);
}

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T>
hipError_t run(const ExpertGradArgs &a, GradArgs g, hipStream_t s) {
  constexpr size_t ES = sizeof(T);
  const int rows13 = (a.act == MOE_ACT_RELU2 ? 1 : 2) * a.inter;
  const size_t m = (size_t)g.rows;
  char *ws = reinterpret_cast<char *>(a.workspace);
  void *dh = ws;
  void *wa = ws += align256(m * rows13 * ES);
  void *dx = ws += align256(m * a.inter * ES);
  float *part = reinterpret_cast<float *>(ws += align256(m * a.hidden * ES));
  const uint32_t token_bytes = (uint32_t)(a.n_tokens * a.hidden * ES);
  const uint32_t h_bytes = (uint32_t)(m * rows13 * ES), wa_bytes = (uint32_t)(m * a.inter * ES);
  const uint32_t w13_bytes = (uint32_t)((size_t)rows13 * a.hidden * ES);
  const uint32_t w2_bytes = (uint32_t)((size_t)a.inter * a.hidden * ES);
  hipError_t err;

  // u = d_out W2, to dh, w a and the parts of d_w
  GradArgs q = g;
  q.A = a.d_out, q.a_bytes = token_bytes, q.K = a.hidden;
  q.B = a.w2, q.b_bytes = w2_bytes, q.N = a.inter;
  q.h = a.h, q.dh = dh, q.wa = wa, q.part = part, q.h_bytes = h_bytes, q.c_bytes = wa_bytes;
  int slab = 32, unused;
  err = a.act == MOE_ACT_RELU2 ? launch_rows<T, GRAD_ACT, ACT_RELU2, 1>(q, s, &slab)
                               : launch_rows<T, GRAD_ACT, ACT_GATED, 1>(q, s, &slab);
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(join_weight_grad, dim3((unsigned)cover(g.rows, 256)), dim3(256), 0, s, part,
                     a.routing->row_sorted, a.d_topk_w, g.rows, (int)cover(a.inter, slab));
  if ((err = hipGetLastError()) != hipSuccess) return err;

  // dW2 = d_out^T (w a)
  q = g;
  q.A = a.d_out, q.a_bytes = token_bytes, q.M = a.hidden;
  q.B = wa, q.b_bytes = wa_bytes, q.N = a.inter, q.C = a.d_w2, q.c_bytes = w2_bytes;
  if ((err = launch_weights<T, 1>(q, s)) != hipSuccess) return err;

  // rows of d_x = dh W13, added up by token
  q = g;
  q.A = dh, q.a_bytes = h_bytes, q.K = rows13;
  q.B = a.w13, q.b_bytes = w13_bytes, q.N = a.hidden;
  q.C = dx, q.c_bytes = (uint32_t)(m * a.hidden * ES);
  if ((err = launch_rows<T, GRAD_ROWS, 0, 0>(q, s, &unused)) != hipSuccess) return err;
  err = launch_combine(dx, a.routing->row_sorted, a.d_x, a.dtype, a.n_tokens, a.topk, a.hidden, s);
  if (err != hipSuccess) return err;

  // dW13 = dh^T x
  q = g;
  q.A = dh, q.a_bytes = h_bytes, q.M = rows13;
  q.B = a.x, q.b_bytes = token_bytes, q.N = a.hidden;
  q.C = a.d_w13, q.c_bytes = w13_bytes;
  return launch_weights<T, 2>(q, s);
}

}  // namespace

hipError_t launch_zero(void *p, size_t bytes, hipStream_t s) {
  const int64_t chunks = (int64_t)(bytes / 16), blocks = cover(chunks, 256);
  hipLaunchKernelGGL(zero_kernel, dim3((unsigned)(blocks < 8192 ? blocks : 8192)), dim3(256), 0, s,
                     reinterpret_cast<u32x4_t *>(p), chunks);
  return hipGetLastError();
}

hipError_t launch_activation(const void *h, void *act, const int32_t *offsets, int n_experts,
                             moe_dtype_t dt, int64_t rows, int inter, moe_act_t kind,
                             moe_w13_layout_t layout, ActParams prm, hipStream_t s) {
  const int64_t chunks = rows * (inter / (dt == MOE_BF16 ? 8 : 4));
  auto go = [&](auto t, auto k) {
    using T = decltype(t);
    hipLaunchKernelGGL((activation_kernel<T, decltype(k)::value>),
                       dim3((unsigned)cover(chunks, 256)), dim3(256), 0, s,
                       reinterpret_cast<const T *>(h), reinterpret_cast<T *>(act), offsets,
                       n_experts, inter, layout == MOE_W13_INTERLEAVED, chunks, prm);
  };
  std::integral_constant<int, ACT_GATED> gated;
  std::integral_constant<int, ACT_RELU2> relu2;
  if (dt == MOE_BF16) kind == MOE_ACT_RELU2 ? go(bf16_t(), relu2) : go(bf16_t(), gated);
  else kind == MOE_ACT_RELU2 ? go(float(), relu2) : go(float(), gated);
  return hipGetLastError();
}

size_t experts_backward_scratch_bytes(int64_t n_tokens, int topk, int hidden, int inter,
                                      moe_dtype_t dt) {
  const size_t m = (size_t)n_tokens * topk, es = dt == MOE_BF16 ? 2 : 4;
  // dh (as for a gated activation), w a, the rows of d_x, the parts of d_w
  return align256(2 * m * inter * es) + align256(m * inter * es) + align256(m * hidden * es) +
         align256(m * (size_t)cover(inter, 32) * 4);
}

hipError_t launch_experts_backward(const ExpertGradArgs &a, hipStream_t s) {
  GradArgs g{};
  g.offsets = a.routing->offsets;
  g.col_sorted = a.routing->col_sorted;
  g.gate_scal = a.routing->gate_scal;
  g.gate_bf16 = a.routing->w_dtype == MOE_BF16;
  g.E = a.n_experts;
  g.rows = a.n_tokens * a.topk;
  g.interleaved = a.layout == MOE_W13_INTERLEAVED;
  g.prm = a.prm;
  // exact for f below 2^31: mul = ceil(2^(31 + l) / topk), 2^l >= topk
  int l = 0;
  while ((1 << l) < a.topk) ++l;
  g.div_shift = 31 + l;
  g.div_mul = (uint32_t)(((1ull << (31 + l)) + a.topk - 1) / a.topk);
  return a.dtype == MOE_BF16 ? run<bf16_t>(a, g, s) : run<float>(a, g, s);
}

}  // namespace moe
