// The experts' products of an expert-parallel MoE step, between dispatch and
// combine, and their gradients.
//
// Rows arrive grouped by expert (the dispatch layout): group e's rows are
// offsets[e] .. offsets[e+1] of one arena, and each group has weights of its
// own.  With X a group's rows, W its weight [out][in]:
//   linear   Y = act(X W^T + b) + R
//   gated    H = act(X Wg^T) * (X Wu^T)
// and, with dZ the gradient before the activation,
//   dX = dZ W,  dW = dZ^T X,  db = the column sums of dZ.
// All of it is matrix products over ragged groups, computed by one tiled
// kernel in three forms that differ in which side has the reduction index
// contiguous in memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "rrb_internal.h"
#include "rrb_kernels.h"

namespace rrb {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

// Groups that a wave counts, 64 at a time, before it starts on its tile.
constexpr int kMaxGroups = 4096;
// Row widths whose tile offsets fit 32 bits.
constexpr int64_t kMaxWidth = int64_t(1) << 20;

// ---- activations ------------------------------------------------------------
//
// In fp32.  The sigmoid is v_rcp_f32 of 1 + v_exp_f32: about 2 ulp of fp32,
// where every result is rounded to bf16 (2^16 ulp of fp32) afterwards.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }

// Argument of the tanh form's sigmoid: gelu_tanh(x) = x sigmoid(2u),
// u = sqrt(2/pi) (x + 0.044715 x^3).
__device__ __forceinline__ float gelu_2u(float x) {
  return 1.5957691216057308f * (x + 0.044715f * x * x * x);
}

// Phi(x) = erfc(-x / sqrt 2) / 2 with erfc(z) = t P(t) e^(-z^2), t = 1 / (1 +
// 0.38 z), z >= 0: P of degree 6, fitted to the smallest relative error of
// e^(z^2) erfc(z) on 0 <= z <= 10.5, 1.1e-6.  Relative, because x Phi(x) is
// rounded relative to itself however far out x is: with z^2 rounded to fp32
// before the exponential Phi stays within 2^-14 down to x = -13, below which it
// leaves fp32's normal range (a fit of the absolute error, 1.5e-7, was 0.4% off
// at -6 and 1% at -8).  About 17 instructions where the library's erfc takes
// some 100 (it was an eighth of a 4096-deep product's time).
// e receives e^(-x^2 / 2), of which the density is made.
__device__ __forceinline__ float normal_cdf(float x, float &e) {
  const float z = 0.70710678118654752f * fabsf(x);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.38f, z, 1.f));
  float q = __builtin_fmaf(-0.12530328f, t, 0.33559692f);
  q = __builtin_fmaf(q, t, -0.069232336f);
  q = __builtin_fmaf(q, t, 0.24729234f);
  q = __builtin_fmaf(q, t, 0.18082708f);
  q = __builtin_fmaf(q, t, 0.21652655f);
  q = __builtin_fmaf(q, t, 0.21429171f);
  e = __expf(-z * z);
  const float half = 0.5f * q * t * e;
  return x < 0.f ? half : 1.f - half;
}

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if (ACT == RRB_ACT_SILU) return x * sigmoid(x);
  if (ACT == RRB_ACT_GELU) {
    float e;
    return x * normal_cdf(x, e);
  }
  if (ACT == RRB_ACT_GELU_TANH) return x * sigmoid(gelu_2u(x));
  if (ACT == RRB_ACT_RELU) return x < 0.f ? 0.f : x;
  return x;
}

// act(x) and act'(x).
template <int ACT>
__device__ __forceinline__ void activate_grad(float x, float &f, float &df) {
  if (ACT == RRB_ACT_SILU) {
    const float s = sigmoid(x);
    f = x * s;
    df = s * (1.f + x * (1.f - s));
  } else if (ACT == RRB_ACT_GELU) {
    float e;
    const float c = normal_cdf(x, e);
    f = x * c;
    df = c + x * (0.3989422804014327f * e);
  } else if (ACT == RRB_ACT_GELU_TANH) {
    const float s = sigmoid(gelu_2u(x));
    const float t = s * (1.f - s);
    f = x * s;
    // Where the sigmoid is flat the slope's term is 0, also where x^2
    // overflows.
    df = t == 0.f ? s : s + x * t * 1.5957691216057308f * (1.f + 0.134145f * x * x);
  } else if (ACT == RRB_ACT_RELU) {
    f = x < 0.f ? 0.f : x;
    df = x > 0.f ? 1.f : 0.f;
  } else {
    f = x;
    df = 1.f;
  }
}

// ---- arguments --------------------------------------------------------------

// Forms of the tiled product C[m][n] = sum over k of A(m, k) B(n, k).
//   kForward  A = X rows, B = weight rows: both have k contiguous
//   kGradX    A = dZ rows (k contiguous), B(n, k) = W[k][n] (n contiguous);
//             gated: k runs over dG with Wg, then over dU with Wu
//   kGradW    A(m, k) = dZ[k][m], B(n, k) = X[k][n]: k is the group's rows
enum Form { kForward = 0, kGradX = 1, kGradW = 2 };

struct ProductArgs {
  const uint16_t *a[2];  // kGradX: per phase; kGradW: per output; else a[0]
  const uint16_t *b[2];  // kForward gated: gate, up; kGradX: per phase
  uint16_t *c[2];        // kGradW gated: dWg, dWu; else c[0]
  uint16_t *save[2];     // kForward: pre-activation values to keep, or NULL
  const uint16_t *bias, *residual;
  const int32_t *offsets;  // [groups + 1], or NULL: one group of all rows
  int32_t rows;
  int64_t lda, ldb, ldc;  // row pitches, in elements
  int64_t bstride;        // kForward, kGradX: weight elements per group (kGradW: dW's)
  int32_t groups;
  int32_t m, n, k;        // m: kGradW only; k: kForward, kGradX only
  int32_t mtiles;         // kGradW: m tiles of both outputs
  int32_t ntiles;
  int32_t bm, bn;         // tiles of one XCD's block: bm slots x bn column tiles, or bm in a row
  int32_t halves;         // kGradX: phases; kGradW: outputs
  int32_t act;
};

// Offsets as the kernels read them: inside the arena whatever the array
// holds.
__device__ __forceinline__ int32_t offset_at(const ProductArgs &p, int e) {
  if (!p.offsets) return e == 0 ? 0 : p.rows;
  const int32_t v = p.offsets[e];
  return v < 0 ? 0 : v > p.rows ? p.rows : v;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const uint16_t *uniform(const uint16_t *q) {
  const uint64_t v = reinterpret_cast<uint64_t>(q);
  const uint32_t lo = uniform(static_cast<int>(v)), hi = uniform(static_cast<int>(v >> 32));
  // As a global address: through a plain one the loads would be flat, which
  // wait with the LDS's.
  typedef __attribute__((address_space(1))) const uint16_t *global;
  return (const uint16_t *)(global)(static_cast<uint64_t>(hi) << 32 | lo);
}

// ---- operand tiles in LDS -----------------------------------------------------
//
// kStep reduction indexes per step.  A row tile (k contiguous) is [rows][64]
// bf16: 128-byte rows of eight 16-byte chunks, chunk c of row r stored at
// chunk c ^ (r / 2 % 8), so that the 16 rows of a fragment read land on 16
// different bank groups.  A column tile (k across rows) is [64][cols]: rows of
// 32-byte slots, slot s of row k stored at slot s ^ (k % 4 + 4 * (k / 8 % 2)),
// so that the eight rows that half a wave reads transposed (ds_read_b64_tr_b16)
// land on eight different bank groups.
constexpr int kStep = 64;

__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }
template <int COLS>
__device__ __forceinline__ int col_swizzle(int k) {
  // 64 columns are four slots, and two rows span the banks.
  if (COLS == 64) return ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
  return (k & 3) | ((k >> 3) & 1) << 2;
}

// Fragment of 16 rows x 32 k from a row tile: lane l holds row l % 16, k =
// 8 (l / 16) .. + 7.
__device__ __forceinline__ bf16x8_t row_fragment(const unsigned char *tile, int row, int kk) {
  const int lane = threadIdx.x & 63;
  const int r = row + (lane & 15);
  const int c = (kk * 4 + (lane >> 4)) ^ row_swizzle(r);
  return *reinterpret_cast<const bf16x8_t *>(tile + r * 128 + c * 16);
}

// The same fragment from a column tile of `cols` columns: two transposed
// reads, each giving lane l column l % 16 of four rows k.
template <int COLS>
__device__ __forceinline__ bf16x8_t col_fragment(const unsigned char *tile, int col, int kk) {
  const int lane = threadIdx.x & 63;
  const int k = kk * 32 + (lane >> 4) * 8 + ((lane >> 2) & 3);
  const int at = k * (COLS * 2) + (((col >> 4) ^ col_swizzle<COLS>(k)) << 5) + (lane & 3) * 8;
  typedef __attribute__((address_space(3))) s16x4_t *lds_ptr;
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + at));
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(tile + at + 4 * COLS * 2));
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Eight bf16 from `src`, of which the first `have` exist (the others are 0).  A
// partial chunk is read as eight single elements, the last one again for those
// that are not there, so that its loads go out together.
__device__ __forceinline__ u32x4_t load_chunk(const uint16_t *src, int64_t have) {
  u32x4_t v = {0, 0, 0, 0};
  if (have >= 8) {
    __builtin_memcpy(&v, src, 16);
  } else if (have > 0) {
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = src[i < have ? i : have - 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (2 * i < have ? e[2 * i] : 0) | (2 * i + 1 < have ? e[2 * i + 1] << 16 : 0);
  }
  return v;
}

// W consecutive columns of one row, W = 4 or 8, as fp32; `have` of them exist.
template <int W>
__device__ __forceinline__ void load_cols(const uint16_t *src, int have, float (&v)[W]) {
  if (have >= W) {
    uint32_t w[W / 2];
    __builtin_memcpy(w, src, sizeof w);
#pragma unroll
    for (int q = 0; q < W; ++q) v[q] = q & 1 ? bf16_hi(w[q >> 1]) : bf16_lo(w[q >> 1]);
  } else {
#pragma unroll
    for (int q = 0; q < W; ++q) v[q] = q < have ? bf16_to_f32(src[q]) : 0.f;
  }
}
template <int W>
__device__ __forceinline__ void store_cols(uint16_t *dst, int have, const float (&v)[W]) {
  uint32_t w[W / 2];
#pragma unroll
  for (int q = 0; q < W / 2; ++q) w[q] = cvt_pk_bf16(v[2 * q], v[2 * q + 1]);
  if (have >= W) {
    __builtin_memcpy(dst, w, sizeof w);
  } else {
#pragma unroll
    for (int q = 0; q < W; ++q)
      if (q < have) dst[q] = static_cast<uint16_t>(w[q >> 1] >> (16 * (q & 1)));
  }
}

// ---- epilogue -------------------------------------------------------------------
//
// The fragments are computed as B x A, so lane l holds row l % 16 and four
// consecutive columns of each 16 x 16 block: 4 (l / 16) .. + 3, or, where two
// blocks were dealt together (WIDE), the first or second half of eight at
// 8 (l / 16).  Gated: blocks are gate and up by turns.
// The second half of a wave's blocks of rows begins `down` rows behind the first
// block, and of columns `right` columns.  Rows may start at any element: vector
// loads and stores need no alignment.  `stage` (256 x 256 tiles, not gated): 128
// KiB of LDS through which results leave as whole rows of the tile instead of
// 32- or 64-byte pieces (a weight gradient's 268 MB of zeros: 77 -> 56 us);
// 16-byte chunk c of row r is kept at c ^ r % 16, so that neither side meets its
// own banks.  Then save0 is NULL: the stage holds one output at a time.
struct Spot {
  int m, n;         // the wave's first row and output column in the tile
  int down, right;
};

template <int ACT, bool GATED, bool WIDE, int FM, int FN>
__device__ __forceinline__ void store_tile(const ProductArgs &p, const f32x4_t (&acc)[FM][FN], uint16_t *c,
                                           uint16_t *save0, uint16_t *save1, const uint16_t *bias,
                                           const uint16_t *residual, Spot spot, int mvalid, int n0,
                                           unsigned char *stage) {
  constexpr int W = WIDE ? 8 : 4;                           // consecutive columns per lane
  constexpr int BLOCKS = (GATED ? 2 : 1) * (WIDE ? 2 : 1);  // blocks that make them
  const int lane = threadIdx.x & 63;
  auto row_at = [&](int i) { return spot.m + (i >= FM / 2 ? spot.down + (i - FM / 2) * 16 : i * 16) + (lane & 15); };
  auto col_at = [&](int j) {
    const int g = j / BLOCKS, halves = FN / BLOCKS / 2;
    return spot.n + (halves && g >= halves ? spot.right + (g - halves) * W * 4 : g * W * 4) + (lane >> 4) * W;
  };
  // To `to` directly, or into the stage.
  auto put = [&](uint16_t *to, int m, int n, const float (&v)[W]) {
    if (!GATED && stage) {
      unsigned char *q = stage + m * 512 + ((n >> 3) ^ (m & 15)) * 16 + (n & 7) * 2;
      *reinterpret_cast<uint2 *>(q) = make_uint2(cvt_pk_bf16(v[0], v[1]), cvt_pk_bf16(v[2], v[3]));
      if (W == 8)
        *reinterpret_cast<uint2 *>(q + 8) = make_uint2(cvt_pk_bf16(v[W - 4], v[W - 3]), cvt_pk_bf16(v[W - 2], v[W - 1]));
    } else {
      store_cols<W>(to + m * p.ldc + n0 + n, p.n - n0 - n, v);
    }
  };
  // The staged tile to `to`, 32 rows per wave.
  auto flush = [&](uint16_t *to) {
    if (GATED || !stage) return;
    __syncthreads();
    const int n = n0 + (lane & 31) * 8;
#pragma unroll
    for (int b = 0; b < 16; ++b) {
      const int m = (threadIdx.x >> 6) * 32 + b * 2 + (lane >> 5);
      const u32x4_t v = *reinterpret_cast<const u32x4_t *>(stage + m * 512 + ((lane & 31) ^ (m & 15)) * 16);
      if (m >= mvalid) continue;
      if (n + 8 <= p.n) {
        __builtin_memcpy(to + m * p.ldc + n, &v, 16);
      } else {
#pragma unroll
        for (int q = 0; q < 7; ++q)
          if (n + q < p.n) to[m * p.ldc + n + q] = static_cast<uint16_t>(v[q >> 1] >> (16 * (q & 1)));
      }
    }
    __syncthreads();
  };
#pragma unroll
  for (int j = 0; j < FN; j += BLOCKS) {
    const int n = col_at(j), have = p.n - n0 - n;
    if (have <= 0) continue;
    float b[W];
    if (!GATED && bias) load_cols<W>(bias + n0 + n, have, b);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int m = row_at(i);
      if (m >= mvalid) continue;
      float v[W];
      if (GATED) {
        float u[W];
#pragma unroll
        for (int q = 0; q < W; ++q) {
          v[q] = acc[i][j + (q >> 2) * 2][q & 3];
          u[q] = acc[i][j + (q >> 2) * 2 + (GATED ? 1 : 0)][q & 3];
        }
        if (save0) {
          put(save0, m, n, v);
          put(save1, m, n, u);
        }
#pragma unroll
        for (int q = 0; q < W; ++q) v[q] = activate<ACT>(v[q]) * u[q];
      } else {
#pragma unroll
        for (int q = 0; q < W; ++q) v[q] = acc[i][j + (q >> 2)][q & 3] + (bias ? b[q] : 0.f);
        if (save0) put(save0, m, n, v);
#pragma unroll
        for (int q = 0; q < W; ++q) v[q] = activate<ACT>(v[q]);
        if (residual) {
          float r[W];
          load_cols<W>(residual + m * p.ldc + n0 + n, have, r);
#pragma unroll
          for (int q = 0; q < W; ++q) v[q] += r[q];
        }
      }
      put(c, m, n, v);
    }
  }
  flush(c);
}

// ---- the tiled product ------------------------------------------------------------

// Where a workgroup's tile lies: operand bases at the tile's first row (or
// column) and extents.  All uniform, and kept in scalar registers.
struct Place {
  const uint16_t *a[2], *b[2];
  uint16_t *c;
  int32_t row0, klen;   // klen: reduction length (per phase)
  int32_t e, n0, m0, mvalid;
  bool empty;
};

// Tile (mt, nt) of group e, whose rows are first .. last - 1; BM x NCOLS
// outputs.  kGradW: mt counts the tiles of both outputs.
template <int BM, int NCOLS, int FORM>
__device__ __forceinline__ Place place_at(const ProductArgs &p, int e, int first, int last, int mt, int nt) {
  Place t;
  t.e = e;
  t.n0 = nt * NCOLS;
  t.empty = false;
  if (FORM == kGradW) {
    const int tiles = p.mtiles / p.halves;
    const int half = mt / tiles;
    t.row0 = 0;
    t.m0 = (mt - half * tiles) * BM;
    t.klen = last > first ? last - first : 0;
    t.mvalid = p.m - t.m0;
    t.a[0] = t.a[1] = uniform(p.a[half] + first * p.lda + t.m0);
    t.b[0] = t.b[1] = uniform(p.b[0] + first * p.ldb + t.n0);
    t.c = p.c[half] + e * p.bstride + t.m0 * p.ldc;
  } else {
    t.m0 = 0;
    t.row0 = first + mt * BM;
    t.mvalid = uniform(last - t.row0 < BM ? last - t.row0 : BM);
    t.klen = p.k;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      t.a[h] = uniform(p.a[FORM == kGradX ? h : 0] + t.row0 * p.lda);
      t.b[h] = uniform(p.b[h] + e * p.bstride + (FORM == kForward ? t.n0 * p.ldb : t.n0));
    }
    t.c = p.c[0] + t.row0 * p.ldc;
  }
  return t;
}

// Workgroup i runs on XCD i % 8.  A weight gradient's tiles: every group has
// the same ones, and each XCD takes blocks of bm x bn of them, every eighth
// block, so that tiles that share operand rows at the same time share an L2.
template <int BM, int NCOLS>
__device__ __forceinline__ Place place_weight(const ProductArgs &p) {
  Place none;
  none.empty = true;
  const int xcd = blockIdx.x & 7, at = blockIdx.x >> 3;
  const int size = p.bm * p.bn;
  int block = at / size * 8 + xcd;
  const int in = at % size;
  const int down = (p.mtiles + p.bm - 1) / p.bm, across = (p.ntiles + p.bn - 1) / p.bn;
  const int e = block / (down * across);
  block -= e * (down * across);
  const int mt = block / across * p.bm + in % p.bm;
  const int nt = block % across * p.bn + in / p.bm;
  if (mt >= p.mtiles || nt >= p.ntiles || e >= p.groups) return none;
  return place_at<BM, NCOLS, kGradW>(p, e, uniform(offset_at(p, e)), uniform(offset_at(p, e + 1)), mt, nt);
}

// The other forms' tiles.  How many row tiles a group has is known on the
// device alone: they are counted, so that the tiles come without gaps (with
// workgroups that only exit between them, taking their turns on the CUs, other
// CUs got two tiles to do: 512 rows in each of 16 groups, one tile per CU, 185
// -> 105 us).  Every wave counts by itself, 64 groups at a time.  LIGHT: tiles
// of at most so many rows cost half of a whole one and come last, where they
// fill the CUs that the whole ones leave (an input gradient of 12007 rows in
// seven groups: 522 -> 498 us).  Tiles are ordered in bands of four row tiles,
// columns in turn, and dealt to the XCDs in runs of p.bm.
template <int BM, int NCOLS, int LIGHT, int FORM>
__device__ __forceinline__ Place place_counted(const ProductArgs &p) {
  Place none;
  none.empty = true;
  const int lane = threadIdx.x & 63;
  struct Group {
    int first, last, whole, all;  // rows; tiles that are not light, and all
  };
  auto group = [&](int e) {
    Group g = {0, 0, 0, 0};
    if (e < p.groups) {
      g.first = offset_at(p, e);
      g.last = offset_at(p, e + 1);
      const int n = g.last > g.first ? g.last - g.first : 0;
      g.all = (n + BM - 1) / BM;
      g.whole = n == 0 ? 0 : (n - 1) / BM + ((n - 1) % BM >= LIGHT ? 1 : 0);
    }
    return g;
  };
  int whole = 0, all = 0;
  for (int e = lane; e < p.groups; e += 64) {
    const Group g = group(e);
    whole += g.whole;
    all += g.all;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    whole += __shfl_xor(whole, d, 64);
    all += __shfl_xor(all, d, 64);
  }
  whole = uniform(whole);
  all = uniform(all);
  const int xcd = blockIdx.x & 7, turn = blockIdx.x >> 3;
  const int at = (turn / p.bm * 8 + xcd) * p.bm + turn % p.bm;
  const int band = at / (4 * p.ntiles) * 4;
  if (band >= all) return none;
  const int high = all - band < 4 ? all - band : 4;
  const int in = at - band * p.ntiles;
  if (in >= high * p.ntiles) return none;
  int row = band + in % high;
  const int nt = in / high;
  const bool light = row >= whole;
  if (light) row -= whole;
  for (int base = 0, done = 0; base < p.groups; base += 64) {
    const Group g = group(base + lane);
    const int n = light ? g.all - g.whole : g.whole;
    int upto = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    // The group whose tiles include this one: those below it end before.
    const int l = __popcll(__ballot(done + upto <= row));
    if (l < 64) {
      const int before = done + __shfl(upto - n, l, 64);
      const int mt = row - before + (light ? __shfl(g.whole, l, 64) : 0);
      return place_at<BM, NCOLS, FORM>(p, base + l, uniform(__shfl(g.first, l, 64)), uniform(__shfl(g.last, l, 64)),
                                       uniform(mt), nt);
    }
    done += uniform(__shfl(upto, 63, 64));
  }
  return none;
}

template <int BM, int NCOLS, int LIGHT, int FORM>
__device__ __forceinline__ Place place_tile(const ProductArgs &p) {
  if (FORM == kGradW) return place_weight<BM, NCOLS>(p);
  return place_counted<BM, NCOLS, LIGHT, FORM>(p);
}

// Stores a wave's part of the tile.  DEALT: row regions were dealt for eight
// columns per lane.
template <int FORM, bool GATED, bool DEALT, int FM, int FN>
__device__ __forceinline__ void finish_tile(const ProductArgs &p, const Place &t, const f32x4_t (&acc)[FM][FN],
                                            Spot spot, unsigned char *stage) {
  constexpr bool WIDE = DEALT && FORM == kForward;
  uint16_t *s0 = nullptr, *s1 = nullptr;
  const uint16_t *bias = nullptr, *res = nullptr;
  if (FORM == kForward) {
    if (p.save[0]) s0 = p.save[0] + t.row0 * p.ldc;
    if (p.save[1]) s1 = p.save[1] + t.row0 * p.ldc;
    if (p.bias) bias = p.bias + static_cast<int64_t>(t.e) * p.n;
    if (p.residual) res = p.residual + t.row0 * p.ldc;
  }
#define RRB_STORE(A) store_tile<A, GATED, WIDE>(p, acc, t.c, s0, s1, bias, res, spot, t.mvalid, t.n0, stage);
  if (FORM != kForward) {
    RRB_STORE(RRB_ACT_NONE)
    return;
  }
  // Staged, the pre-activation goes by itself: the stage holds one output.
  if (!GATED && stage && s0) {
    store_tile<RRB_ACT_NONE, GATED, WIDE>(p, acc, s0, nullptr, nullptr, bias, nullptr, spot, t.mvalid, t.n0, stage);
    s0 = nullptr;
  }
  switch (p.act) {
#define RRB_CASE(A)  \
  case A:            \
    RRB_STORE(A)     \
    break;
    RRB_CASE(RRB_ACT_SILU) RRB_CASE(RRB_ACT_GELU) RRB_CASE(RRB_ACT_GELU_TANH) RRB_CASE(RRB_ACT_RELU)
#undef RRB_CASE
    default: RRB_STORE(RRB_ACT_NONE)
  }
#undef RRB_STORE
}

template <int FM, int FN>
__device__ __forceinline__ void clear_tile(f32x4_t (&acc)[FM][FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

// Row j of a gated B tile: blocks of 16 gate rows and 16 up rows by turns, so
// that a lane holds both projections of its outputs.
__device__ __forceinline__ int gated_row(int j) { return (j >> 5) * 16 + (j & 15); }
__device__ __forceinline__ bool gated_up(int j) { return j & 16; }

// Operands whose rows do not start on 16-byte boundaries: tiles go through
// registers, with 16-byte loads that need no alignment and the last, partial
// chunk of a row read element by element.  Bound by those loads and the one
// step that they are ahead: 0.5 PFLOP/s on 8 groups of 1024 rows, 4095 x 4096
// (1.2 where rows are aligned).
template <int BM, int BN, int WR, int WC, int FORM, bool GATED>
__global__ void __launch_bounds__(WR *WC * 64) product_kernel(ProductArgs p) {
  constexpr int NT = WR * WC * 64;
  constexpr int FM = BM / WR / 16, FN = BN / WC / 16;
  constexpr int A_BYTES = BM * kStep * 2, B_BYTES = BN * kStep * 2;
  constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT;  // 16-byte chunks per thread
  constexpr bool A_COL = FORM == kGradW, B_COL = FORM != kForward;
  __shared__ __align__(16) unsigned char lds[2 * (A_BYTES + B_BYTES)];

  const int tid = threadIdx.x;
  const int wave = uniform(tid >> 6);
  const Place t = place_tile<BM, GATED ? BN / 2 : BN, 0, FORM>(p);
  if (t.empty) return;
  const int klen = t.klen;
  const int per = (klen + kStep - 1) / kStep;  // steps per phase
  const int steps = FORM == kGradX ? per * p.halves : per;

  u32x4_t ra[CA], rb[CB];
  // Elements of a column tile's chunk to read in row k, of whose `cols` columns
  // `have` are left there.  A chunk over the row's end is read whole, into the
  // next rows, while the group's matrix has that many elements left: its
  // columns past the end are of outputs that are not stored.
  auto there = [&](int64_t k, int have, int cols, int64_t ld) {
    if (k >= klen) return 0;
    return have > 0 && (klen - k) * ld - (cols - have) >= 8 ? 8 : have;
  };
  // Loads of one step's chunks into registers.
  auto fetch = [&](int step) {
    const int h = FORM == kGradX && step >= per ? 1 : 0;
    const int64_t k0 = static_cast<int64_t>(step - h * per) * kStep;
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const int id = i * NT + tid;
      if (A_COL) {
        const int kr = id / (BM / 8), pos = id % (BM / 8);
        const int ch = pos ^ (col_swizzle<BM>(kr) << 1);
        ra[i] = load_chunk(t.a[0] + (k0 + kr) * p.lda + ch * 8, there(k0 + kr, p.m - t.m0 - ch * 8, p.m, p.lda));
      } else {
        const int r = id >> 3, ch = (id & 7) ^ row_swizzle(r);
        const int64_t have = klen - k0 - ch * 8;
        ra[i] = load_chunk(t.a[h] + r * p.lda + k0 + ch * 8, r < t.mvalid ? have : 0);
      }
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int id = i * NT + tid;
      if (B_COL) {
        const int kr = id / (BN / 8), pos = id % (BN / 8);
        const int ch = pos ^ (col_swizzle<BN>(kr) << 1);
        rb[i] = load_chunk(t.b[h] + (k0 + kr) * p.ldb + ch * 8, there(k0 + kr, p.n - t.n0 - ch * 8, p.n, p.ldb));
      } else {
        const int r = id >> 3, ch = (id & 7) ^ row_swizzle(r);
        const int64_t have = klen - k0 - ch * 8;
        const int n = GATED ? gated_row(r) : r;
        const uint16_t *src = GATED && gated_up(r) ? t.b[1] : t.b[0];
        rb[i] = load_chunk(src + n * p.ldb + k0 + ch * 8, t.n0 + n < p.n ? have : 0);
      }
    }
  };
  auto commit = [&](int buf) {
    unsigned char *ta = lds + buf * (A_BYTES + B_BYTES), *tb = ta + A_BYTES;
#pragma unroll
    for (int i = 0; i < CA; ++i) *reinterpret_cast<u32x4_t *>(ta + (i * NT + tid) * 16) = ra[i];
#pragma unroll
    for (int i = 0; i < CB; ++i) *reinterpret_cast<u32x4_t *>(tb + (i * NT + tid) * 16) = rb[i];
  };

  const int wm = wave / WC * (BM / WR), wn = wave % WC * (BN / WC);
  f32x4_t acc[FM][FN];
  clear_tile(acc);
  if (steps > 0) {
    fetch(0);
    commit(0);
  }
  for (int s = 0; s < steps; ++s) {
    __syncthreads();
    if (s + 1 < steps) fetch(s + 1);
    const unsigned char *ta = lds + (s & 1) * (A_BYTES + B_BYTES), *tb = ta + A_BYTES;
#pragma unroll
    for (int kk = 0; kk < kStep / 32; ++kk) {
      bf16x8_t fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[i] = A_COL ? col_fragment<BM>(ta, wm + i * 16, kk) : row_fragment(ta, wm + i * 16, kk);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[j] = B_COL ? col_fragment<BN>(tb, wn + j * 16, kk) : row_fragment(tb, wn + j * 16, kk);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    if (s + 1 < steps) commit((s + 1) & 1);
  }
  finish_tile<FORM, GATED, false>(p, t, acc, Spot{wm, GATED ? wn / 2 : wn, FM * 8, FN * (GATED ? 4 : 8)}, nullptr);
}

// ---- the tiled product, loads straight to LDS -----------------------------------
//
// Operands with rows on 16-byte boundaries.  Each lane moves 16-byte chunks
// from memory to LDS without a register (buffer_load_dwordx4 ... lds): a wave
// fills 1 KiB in lane order, so the swizzle is applied to the address each
// lane reads.  Rows past a tile's last valid one read that row again (their
// results are not stored); chunks past the reduction's end, and rows of a
// column tile past it, lie outside the descriptor and arrive as zeros, on both
// sides, so that nothing behind a group reaches its sums.  The range check is of
// a lane's own offset, the scalar offset left out or taken off the descriptor's
// size first; so that an empty descriptor holds either way (0 less an offset
// must not wrap to a large size), loads through one have a scalar offset of 0.
//
// Small tiles, for few rows or few tiles: STAGES - 1 steps of loads in flight
// and one barrier a step.  64 x 64 in five stages (two workgroups a CU) streams
// the weights of 24 single-row groups at 6.1 TB/s (7168 -> 2048 gated, 231 us;
// the 256 x 256 kernel 335); 64 x 256 in three stages covers 64 rows in each of
// 16 groups, 4096 -> 2048, in 58 us (64 x 64 79, 256 x 256 74).  Four stages of
// 32 x 128, eight to twelve of 32 x 64 and 128 x 256 in three were within 10% of
// these or behind.

__device__ __forceinline__ u32x4_t descriptor(const uint16_t *base, int bytes) {
  const uint64_t v = reinterpret_cast<uint64_t>(uniform(base));
  return u32x4_t{static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32), static_cast<uint32_t>(uniform(bytes)),
                 0x00020000u};
}
constexpr int kOutside = 0x7fffffff;

// Address of a workgroup's LDS as the loads below take it.
__device__ __forceinline__ int lds_address(const unsigned char *lds) {
  return static_cast<int>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const unsigned char *)lds));
}

// 16 bytes per lane from `d` at voffset + soffset to LDS address `at` (the
// wave's first byte, uniform) + 16 * lane.  As assembly, because the compiler
// would wait for every such load in flight before it reads any LDS
// transposed; the kernels wait themselves, by count.  (m0 is reserved: the
// compiler keeps nothing in it from one use to the next.  The five wait states
// stand between a vector instruction that may just have written the scalar
// operands and the load that reads them; the compiler sees to that only for
// instructions of its own.)
__device__ __forceinline__ void load_to_lds(u32x4_t d, int at, int voffset, int soffset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(uniform(at)), "v"(voffset), "s"(d), "s"(uniform(soffset))
               : "memory");
}

// Two such loads, 8 KiB apart in LDS, behind one set of wait states.
__device__ __forceinline__ void load_two_to_lds(u32x4_t d, int at, int voffset0, int voffset1, int soffset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %4, %5 offen lds\n\t"
      "s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %4, %5 offen lds"
      :
      : "s"(uniform(at)), "s"(uniform(at + 8192)), "v"(voffset0), "v"(voffset1), "s"(d), "s"(uniform(soffset))
      : "memory");
}

template <int BM, int BN, int WR, int WC, int STAGES, int FORM, bool GATED>
__global__ void __launch_bounds__(WR *WC * 64) product_direct_kernel(ProductArgs p) {
  constexpr int NT = WR * WC * 64;
  constexpr int FM = BM / WR / 16, FN = BN / WC / 16;
  constexpr int A_BYTES = BM * kStep * 2, B_BYTES = BN * kStep * 2;
  constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT, NCOLS = GATED ? BN / 2 : BN;
  constexpr bool A_COL = FORM == kGradW, B_COL = FORM != kForward;
  __shared__ __align__(16) unsigned char lds[STAGES * (A_BYTES + B_BYTES)];

  const int tid = threadIdx.x;
  const int wave = uniform(tid >> 6);
  const Place t = place_tile<BM, GATED ? BN / 2 : BN, 0, FORM>(p);
  if (t.empty) return;
  const int klen = t.klen;
  const int per = (klen + kStep - 1) / kStep;  // steps per phase
  const int steps = FORM == kGradX ? per * p.halves : per;
  const int lda2 = static_cast<int>(p.lda * 2), ldb2 = static_cast<int>(p.ldb * 2);

  // Byte offsets of this thread's chunks in a step's tile.
  int va[CA], vb[CB];
#pragma unroll
  for (int i = 0; i < CA; ++i) {
    const int id = i * NT + tid;
    if (A_COL) {
      const int kr = id / (BM / 8), pos = id % (BM / 8);
      va[i] = kr * lda2 + (pos ^ (col_swizzle<BM>(kr) << 1)) * 16;
    } else {
      const int r = id >> 3;
      va[i] = (r < t.mvalid ? r : t.mvalid - 1) * lda2 + ((id & 7) ^ row_swizzle(r)) * 16;
    }
  }
#pragma unroll
  for (int i = 0; i < CB; ++i) {
    const int id = i * NT + tid;
    if (B_COL) {
      const int kr = id / (BN / 8), pos = id % (BN / 8);
      vb[i] = kr * ldb2 + (pos ^ (col_swizzle<BN>(kr) << 1)) * 16;
    } else {
      const int r = id >> 3;
      const int n = GATED ? gated_row(r) : r;
      vb[i] = (t.n0 + n < p.n ? n : p.n - 1 - t.n0) * ldb2 + ((id & 7) ^ row_swizzle(r)) * 16;
    }
  }

  // Starts one step's loads into buffer `buf`; past the end through an empty
  // descriptor, so that every step counts the same.
  auto issue = [&](int step, int buf) {
    const int h = FORM == kGradX && step >= per ? 1 : 0;
    const int kstep = step - h * per;
    const int k0 = kstep * kStep;
    const int left = klen - k0;
    const bool live = step < steps;
    const int along = live ? kstep * 128 : 0;
    const int rows = left < kStep ? left : kStep;  // of the column tiles
    const int ta = lds_address(lds) + buf * (A_BYTES + B_BYTES) + wave * 1024, tb = ta + A_BYTES;
    if (A_COL) {
      const auto d = descriptor(t.a[0] + k0 * p.lda, live ? rows * lda2 - t.m0 * 2 : 0);
#pragma unroll
      for (int i = 0; i < CA; ++i)
        load_to_lds(d, ta + i * NT * 16, va[i], 0);
    } else {
      const auto d = descriptor(t.a[h], live ? t.mvalid * lda2 : 0);
#pragma unroll
      for (int i = 0; i < CA; ++i) {
        int v = va[i];
        if (left < kStep) {
          const int id = i * NT + tid;
          if (((id & 7) ^ row_swizzle(id >> 3)) * 8 >= left) v = kOutside;
        }
        load_to_lds(d, ta + i * NT * 16, v, along);
      }
    }
    if (B_COL) {
      const auto d = descriptor(t.b[h] + k0 * p.ldb, live ? rows * ldb2 - t.n0 * 2 : 0);
#pragma unroll
      for (int i = 0; i < CB; ++i)
        load_to_lds(d, tb + i * NT * 16, vb[i], 0);
    } else {
      const int bytes = live ? (p.n - t.n0 < NCOLS ? p.n - t.n0 : NCOLS) * ldb2 : 0;
      const auto d0 = descriptor(t.b[0], bytes);
      const auto d1 = descriptor(GATED ? t.b[1] : t.b[0], bytes);
#pragma unroll
      for (int i = 0; i < CB; ++i) {
        int v = vb[i];
        if (left < kStep) {
          const int id = i * NT + tid;
          if (((id & 7) ^ row_swizzle(id >> 3)) * 8 >= left) v = kOutside;
        }
        // The wave's eight rows are all gate rows or all up rows.
        const bool up = GATED && gated_up((i * NT + wave * 64) >> 3);
        load_to_lds(up ? d1 : d0, tb + i * NT * 16, v, along);
      }
    }
  };

  const int wm = wave / WC * (BM / WR), wn = wave % WC * (BN / WC);
  f32x4_t acc[FM][FN];
  clear_tile(acc);
  if (steps > 0) {
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) issue(s, s);
  }
  int buf = 0, free = STAGES - 1;
  for (int s = 0; s < steps; ++s) {
    // This step's loads have landed, and every wave is done with the buffer
    // that is loaded next.
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * (CA + CB)) : "memory");
    issue(s + STAGES - 1, free);
    free = buf;
    const unsigned char *ta = lds + buf * (A_BYTES + B_BYTES), *tb = ta + A_BYTES;
    buf = buf + 1 == STAGES ? 0 : buf + 1;
#pragma unroll
    for (int kk = 0; kk < kStep / 32; ++kk) {
      bf16x8_t fa[FM], fb[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[j] = B_COL ? col_fragment<BN>(tb, wn + j * 16, kk) : row_fragment(tb, wn + j * 16, kk);
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[i] = A_COL ? col_fragment<BM>(ta, wm + i * 16, kk) : row_fragment(ta, wm + i * 16, kk);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  finish_tile<FORM, GATED, false>(p, t, acc, Spot{wm, GATED ? wn / 2 : wn, FM * 8, FN * (GATED ? 4 : 8)}, nullptr);
}

// ---- the tiled product, two wave groups by turns -----------------------------------
//
// 256 x 256 tiles, for products that are bound by the matrix cores.  Eight waves
// (2 x 4, 128 x 64 outputs each) in two groups of one wave per SIMD: while one
// group issues 16 matrix instructions (a quarter of its step) the other reads
// fragments and starts loads, so a SIMD's matrix core and the LDS work at the
// same time.  A step's tiles are kept as four regions of 16 KiB, the first and
// second 128 rows (A0, A1; a group has 64 of each) and columns (B0, B1; a wave
// has 32 of each, gated: half of the rows dealt to its 32 outputs), two steps
// deep.  In phase p a group reads and starts
//   0  reads B0, half of A1;            starts A1 of step s + 1;    A0 x B0
//   1  reads the rest of A1;                                        A0 x B1
//   2  reads half of A0 of s + 1;       starts A0, B0 of s + 2;     A1 x B1
//   3  reads the rest of it, B1 of s + 1; starts B1 of s + 2;       A1 x B0
// then a barrier, the products, a barrier; the second group runs one barrier
// behind.  Only B0 is read in the phase that uses it.  A region is loaded again
// no earlier than a whole phase after both groups have used its fragments: A0
// and B0 by products 0, B1 by products 1, A1 by products 2.  A wave lets at most
// six of its loads be in flight when it passes phase 1, 2 or 3, which leaves
// what the next phase reads (A0; B1; A1 and B0) complete in every wave before
// the barrier between.  Steps past the end load through an empty descriptor
// (zeros, no memory access), so the count holds to the last step.  A tile of at
// most 128 valid rows loads nothing for A1 and leaves out its reads and
// products, so it costs half the matrix instructions of a whole one.
// Measured: 1.24 to 1.34 PFLOP/s (8192 x 8192 outputs, 8192 and 4096 deep, random
// data; 1.74 on zeros: the clock falls to 2.0 GHz under load), matrix cores busy
// 60% of the time in a 4096-deep gated forward; tiles of few steps are bound by
// their first loads and results, about 13 us a tile together.

// Row of B (column of the output) that sits at row r of half h of a row region.
// Sixteen rows make a fragment and a lane holds four consecutive ones of each;
// rows are dealt so that two fragments give a lane eight consecutive columns.
template <bool GATED>
__device__ __forceinline__ int dealt_row(int r, int h) {
  if (GATED) return (r >> 5) * 32 + ((r >> 2) & 3) * 8 + h * 4 + (r & 3);  // gate and up rows of the same outputs
  return h * 128 + (r >> 5) * 32 + ((r >> 2) & 3) * 8 + ((r >> 4) & 1) * 4 + (r & 3);
}

template <int FORM, bool GATED>
__device__ __forceinline__ void product_turns_tile(const ProductArgs &p, const Place &t, unsigned char *lds) {
  constexpr int REGION = 16384, BUFFER = 4 * REGION, NCOLS = GATED ? 128 : 256;
  constexpr bool A_COL = FORM == kGradW, B_COL = FORM != kForward;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int klen = t.klen;
  const int per = (klen + kStep - 1) / kStep;
  const int steps = FORM == kGradX ? per * p.halves : per;
  const int lda2 = static_cast<int>(p.lda * 2), ldb2 = static_cast<int>(p.ldb * 2);

  // Byte offsets of this thread's two chunks in each region.
  int va[2][2], vb[2][2];
  const int ch = (tid & 7) ^ row_swizzle(tid >> 3);  // row regions: the chunk of the row
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int id = i * 512 + tid;
      const int kr = id >> 4, c = (id & 15) ^ (col_swizzle<128>(kr) << 1);
      const int r = id >> 3;
      if (A_COL) {
        va[h][i] = kr * lda2 + (h * 128 + c * 8) * 2;
      } else {
        const int m = h * 128 + r;
        va[h][i] = m < t.mvalid ? m * lda2 + ch * 16 : kOutside;
      }
      if (B_COL) {
        vb[h][i] = kr * ldb2 + (h * 128 + c * 8) * 2;
      } else {
        const int n = dealt_row<GATED>(r, h);
        vb[h][i] = (t.n0 + n < p.n ? n : p.n - 1 - t.n0) * ldb2 + ch * 16;
      }
    }
  }
  const int to = lds_address(lds) + wave * 1024;
  const bool both = t.mvalid > 128;  // rows in A1

  auto start_a = [&](int step, int h) {
    const int ph = FORM == kGradX && step >= per ? 1 : 0;
    const int ks = step - ph * per;
    const int k0 = ks * kStep, left = klen - k0;
    const int rows = left < kStep ? left : kStep;
    const int dst = to + (step & 1) * BUFFER + h * REGION;
    const bool live = step < steps;
    if (A_COL) {
      const auto d = descriptor(t.a[0] + k0 * p.lda, live && (h == 0 || both) ? rows * lda2 - t.m0 * 2 : 0);
      load_two_to_lds(d, dst, va[h][0], va[h][1], 0);
    } else {
      const bool any = live && (h == 0 || both);
      const auto d = descriptor(t.a[ph], any ? t.mvalid * lda2 : 0);
      const bool out = left < kStep && ch * 8 >= left;
      load_two_to_lds(d, dst, out ? kOutside : va[h][0], out ? kOutside : va[h][1], any ? ks * 128 : 0);
    }
  };
  auto start_b = [&](int step, int h) {
    const int ph = FORM == kGradX && step >= per ? 1 : 0;
    const int ks = step - ph * per;
    const int k0 = ks * kStep, left = klen - k0;
    const int rows = left < kStep ? left : kStep;
    const int dst = to + (step & 1) * BUFFER + (2 + h) * REGION;
    const bool live = step < steps;
    if (B_COL) {
      const auto d = descriptor(t.b[ph] + k0 * p.ldb, live ? rows * ldb2 - t.n0 * 2 : 0);
      load_two_to_lds(d, dst, vb[h][0], vb[h][1], 0);
    } else {
      // The wave's eight rows are all gate rows or all up rows.
      const bool up = GATED && (wave & 2);
      const int cols = p.n - t.n0 < NCOLS ? p.n - t.n0 : NCOLS;
      const auto d = descriptor(up ? t.b[1] : t.b[0], live ? cols * ldb2 : 0);
      const bool out = left < kStep && ch * 8 >= left;
      load_two_to_lds(d, dst, out ? kOutside : vb[h][0], out ? kOutside : vb[h][1], live ? ks * 128 : 0);
    }
  };

  // Fragment addresses within a region: by kk for rows (the swizzle moves
  // with the chunk), by fragment for columns (it moves with the slot).
  const int wr = wave >> 2, wc = wave & 3;
  int fa_at[4], fb_at[2];
  if (A_COL) {
    const int k = (lane >> 4) * 8 + ((lane >> 2) & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) fa_at[i] = k * 256 + (((wr * 4 + i) ^ col_swizzle<128>(k)) << 5) + (lane & 3) * 8;
  } else {
    const int r = wr * 64 + (lane & 15);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) fa_at[kk] = r * 128 + ((kk * 4 + (lane >> 4)) ^ row_swizzle(r)) * 16;
  }
  if (B_COL) {
    const int k = (lane >> 4) * 8 + ((lane >> 2) & 3);
#pragma unroll
    for (int j = 0; j < 2; ++j) fb_at[j] = k * 256 + (((wc * 2 + j) ^ col_swizzle<128>(k)) << 5) + (lane & 3) * 8;
  } else {
    const int r = wc * 32 + (lane & 15);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) fb_at[kk] = r * 128 + ((kk * 4 + (lane >> 4)) ^ row_swizzle(r)) * 16;
  }
  auto rows_at = [](const unsigned char *q) { return *reinterpret_cast<const bf16x8_t *>(q); };
  auto cols_at = [](const unsigned char *q) {
    typedef __attribute__((address_space(3))) s16x4_t *lds_ptr;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)q);
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(q + 1024));
    return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  bf16x8_t fa[2][2][4], fb[2][2][2];  // [half][kk][block]
  auto read_a = [&](const unsigned char *buf, int h, int kk) {
    const unsigned char *region = buf + h * REGION;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      fa[h][kk][i] = A_COL ? cols_at(region + fa_at[i] + kk * 8192) : rows_at(region + fa_at[kk] + i * 2048);
  };
  auto read_b = [&](const unsigned char *buf, int h) {
    const unsigned char *region = buf + (2 + h) * REGION;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        fb[h][kk][j] = B_COL ? cols_at(region + fb_at[j] + kk * 8192) : rows_at(region + fb_at[kk] + j * 2048);
  };
  f32x4_t acc[8][4];
  clear_tile(acc);
#define RRB_BARRIER()                       \
  __builtin_amdgcn_sched_barrier(0);        \
  asm volatile("s_barrier" ::: "memory");   \
  __builtin_amdgcn_sched_barrier(0)
  auto multiply = [&](int ah, int bh) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[ah * 4 + i][bh * 2 + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              fb[bh][kk][j], fa[ah][kk][i], acc[ah * 4 + i][bh * 2 + j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
  };

  if (steps > 0) {
    start_a(0, 0);
    start_b(0, 0);
    start_b(0, 1);
    start_a(0, 1);
    start_a(1, 0);
    start_b(1, 0);
    start_b(1, 1);
    asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
    RRB_BARRIER();
    read_a(lds, 0, 0);
    read_a(lds, 0, 1);
    read_b(lds, 1);
    if (wr) {
      RRB_BARRIER();
    }
    // Two loops, so that each one's waits count the reads it makes.
    auto run = [&](auto whole) {
      constexpr bool BOTH = decltype(whole)::value;
      for (int s = 0; s < steps; ++s) {
        const unsigned char *buf = lds + (s & 1) * BUFFER, *next = lds + (~s & 1) * BUFFER;
        read_b(buf, 0);
        if (BOTH) read_a(buf, 1, 0);
        start_a(s + 1, 1);
        RRB_BARRIER();
        multiply(0, 0);
        RRB_BARRIER();
        if (BOTH) read_a(buf, 1, 1);
        asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
        RRB_BARRIER();
        multiply(0, 1);
        RRB_BARRIER();
        read_a(next, 0, 0);
        start_a(s + 2, 0);
        start_b(s + 2, 0);
        asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
        RRB_BARRIER();
        if (BOTH) multiply(1, 1);
        RRB_BARRIER();
        read_a(next, 0, 1);
        read_b(next, 1);
        start_b(s + 2, 1);
        asm volatile("s_waitcnt vmcnt(6)" ::: "memory");
        RRB_BARRIER();
        if (BOTH) multiply(1, 0);
        RRB_BARRIER();
      }
    };
    if (both)
      run(std::true_type{});
    else
      run(std::false_type{});
    if (!wr) {
      RRB_BARRIER();
    }
    // The last loads (of steps past the end) have landed in every wave: the
    // epilogue takes the LDS over.
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    RRB_BARRIER();
  }
#undef RRB_BARRIER
  finish_tile<FORM, GATED, true>(p, t, acc, Spot{wr * 64, wc * 32, 128, GATED ? 16 : 128}, GATED ? nullptr : lds);
}

template <int FORM, bool GATED>
__global__ void __launch_bounds__(512, 2) product_turns_kernel(ProductArgs p) {
  __shared__ __align__(16) unsigned char lds[131072];
  const Place t = place_tile<256, GATED ? 128 : 256, 128, FORM>(p);
  if (t.empty) return;
  product_turns_tile<FORM, GATED>(p, t, lds);
}

// ---- gradients before the activation -------------------------------------------

struct ActGradArgs {
  const uint16_t *dout, *gate, *up;  // linear: gate is the pre-activation (or NULL), up NULL
  uint16_t *dgate, *dup;             // pitch ldo, columns n .. ldc padded with 0
  const int32_t *offsets;
  int64_t rows, ldo;
  int32_t n, groups;
};

// dG = dH * U * act'(G), dU = dH * act(G) (linear: dZ = dY * act'(pre)), one
// 8-column chunk per thread, rows of groups only.  Memory-bound: 12007 x 2001
// gated, 240 MB in 48 us (5.0 TB/s).  The results are rounded to bf16, as the
// matrix instructions take them.  Columns up to
// the pitch are written as 0, so the products that reduce over them read
// zeros and not what the workspace held.
template <int ACT, bool GATED>
__global__ void __launch_bounds__(256) act_grad_kernel(ActGradArgs p) {
  const int64_t chunks = p.ldo / 8;
  int64_t first = 0, last = p.rows;
  if (p.offsets) {
    first = p.offsets[0], last = p.offsets[p.groups];
    if (first < 0) first = 0;
    if (last > p.rows) last = p.rows;
  }
  const int64_t total = (last - first) * chunks;
  for (int64_t id = blockIdx.x * 256ll + threadIdx.x; id < total; id += gridDim.x * 256ll) {
    const int64_t r = first + id / chunks;
    const int c0 = static_cast<int>(id % chunks) * 8;
    const int have = p.n - c0;
    const int64_t at = r * p.n + c0;
    u32x4_t d = load_chunk(p.dout + at, have), g = {0, 0, 0, 0}, u = {0, 0, 0, 0};
    if (ACT != RRB_ACT_NONE || GATED) g = load_chunk(p.gate + at, have);
    if (GATED) u = load_chunk(p.up + at, have);
    u32x4_t og, ou;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f0, df0, f1, df1;
      activate_grad<ACT>(bf16_lo(g[q]), f0, df0);
      activate_grad<ACT>(bf16_hi(g[q]), f1, df1);
      const float d0 = bf16_lo(d[q]), d1 = bf16_hi(d[q]);
      if (GATED) {
        og[q] = cvt_pk_bf16(d0 * bf16_lo(u[q]) * df0, d1 * bf16_hi(u[q]) * df1);
        ou[q] = cvt_pk_bf16(d0 * f0, d1 * f1);
      } else {
        og[q] = cvt_pk_bf16(d0 * df0, d1 * df1);
      }
    }
    const int64_t to = r * p.ldo + c0;
    *reinterpret_cast<u32x4_t *>(p.dgate + to) = og;
    if (GATED) *reinterpret_cast<u32x4_t *>(p.dup + to) = ou;
  }
}

// db[e][n] = the sum over group e's rows of dZ = dY * act'(pre), which is taken
// from dY and pre in fp32 and not from its bf16 copy for the matrix
// instructions: one rounding, of the sum.  It writes that copy too where one is
// needed, in act_grad_kernel's place.  64 columns per workgroup, eight lanes
// wide and 32 rows deep.  A group's rows are split over workgroups where the
// columns alone make few; their sums are then joined in order by
// bias_join_kernel.  8192 x 7168 in 16 groups (1792 workgroups): bound by reading
// dY, 117 MB in 31 us.  32768 x 64 in one group: 196 us whole and 12.5 split;
// with silu's slope 590 and 14.
struct BiasGradArgs {
  const uint16_t *dout, *pre;  // pre: NULL without an activation
  uint16_t *db;
  float *part;   // [splits][groups][n], or NULL: one split, straight to db
  uint16_t *dz;  // COPY; pitch ldo, columns n .. ldo padded with 0
  int64_t ldo;
  ProductArgs p;  // offsets, rows, groups
  int32_t n, splits;
};

template <int ACT, bool COPY>
__global__ void __launch_bounds__(256) bias_grad_kernel(BiasGradArgs a) {
  __shared__ float part[32][64 + 1];
  const int e = blockIdx.z, lane8 = threadIdx.x & 7, deep = threadIdx.x >> 3;
  const int c0 = blockIdx.x * 64 + lane8 * 8;
  const int32_t first = offset_at(a.p, e), last = offset_at(a.p, e + 1);
  const uint32_t rows = last > first ? last - first : 0, z = blockIdx.y;
  const uint32_t each = a.splits == 1 ? rows : (rows + a.splits - 1) / static_cast<uint32_t>(a.splits);
  const int64_t s = first + min(rows, each * z), t = first + min(rows, each * (z + 1));
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t r = s + deep; r < t; r += 32) {
    const u32x4_t v = load_chunk(a.dout + r * a.n + c0, a.n - c0);
    u32x4_t x = {0, 0, 0, 0};
    if (ACT != RRB_ACT_NONE) x = load_chunk(a.pre + r * a.n + c0, a.n - c0);
    float d[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      float f, df;
      activate_grad<ACT>(q & 1 ? bf16_hi(x[q >> 1]) : bf16_lo(x[q >> 1]), f, df);
      d[q] = df * (q & 1 ? bf16_hi(v[q >> 1]) : bf16_lo(v[q >> 1]));
      sum[q] += d[q];
    }
    if (COPY && c0 < a.ldo) store_cols<8>(a.dz + r * a.ldo + c0, 8, d);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) part[deep][lane8 * 8 + q] = sum[q];
  __syncthreads();
  if (threadIdx.x < 64) {
    float total = 0.f;
    for (int d = 0; d < 32; ++d) total += part[d][threadIdx.x];
    const int col = blockIdx.x * 64 + threadIdx.x;
    const int64_t at = static_cast<int64_t>(e) * a.n + col;
    if (col >= a.n) return;
    if (a.part)
      a.part[static_cast<int64_t>(z) * a.p.groups * a.n + at] = total;
    else
      a.db[at] = f32_to_bf16_rne(total);
  }
}

__global__ void __launch_bounds__(256) bias_join_kernel(BiasGradArgs a) {
  const int64_t all = static_cast<int64_t>(a.p.groups) * a.n, at = blockIdx.x * 256ll + threadIdx.x;
  if (at >= all) return;
  float total = 0.f;
#pragma unroll 8
  for (int i = 0; i < a.splits; ++i) total += a.part[i * all + at];
  a.db[at] = f32_to_bf16_rne(total);
}

// ---- launchers -------------------------------------------------------------------

rrb_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? RRB_OK : fail(RRB_EHIP, "%s launch: %s", what, hipGetErrorString(e));
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Row tiles that the groups' rows can make at most: each group that has rows
// adds at most one partial tile.
int64_t most_row_tiles(const ProductArgs &p, int bm) {
  return p.rows / bm + (p.groups < p.rows ? p.groups : p.rows);
}

// Launches the form over BM x BN tiles with the given kernel.
template <int BM, int BN, int FORM, bool GATED>
rrb_status launch_tiles(void (*kernel)(ProductArgs), int threads, ProductArgs p, hipStream_t s) {
  constexpr int cols = GATED ? BN / 2 : BN;
  p.ntiles = (p.n + cols - 1) / cols;
  int64_t grid;
  if (FORM == kGradW) {
    p.mtiles = (p.m + BM - 1) / BM * p.halves;
    // Blocks of 4 x 8 tiles (one per CU of an XCD) where there are enough to
    // go round, smaller ones for fewer tiles.
    const int64_t tiles = static_cast<int64_t>(p.mtiles) * p.ntiles * p.groups;
    p.bm = tiles >= 512 ? 4 : tiles >= 128 ? 2 : 1;
    p.bn = tiles >= 1024 ? 8 : tiles >= 256 ? 4 : tiles >= 128 ? 2 : 1;
    const int64_t blocks =
        static_cast<int64_t>((p.mtiles + p.bm - 1) / p.bm) * ((p.ntiles + p.bn - 1) / p.bn) * p.groups;
    grid = (blocks + 7) / 8 * 8 * p.bm * p.bn;
  } else {
    // Runs of 32 tiles (an XCD's CUs) where there are many, shorter ones so
    // that few tiles spread over the XCDs.
    const int64_t tiles = most_row_tiles(p, BM) * p.ntiles;
    p.bm = tiles >= 4096 ? 32 : tiles >= 1024 ? 16 : tiles >= 256 ? 8 : 1;
    grid = (tiles + 8 * p.bm - 1) / (8 * p.bm) * (8 * p.bm);
  }
  // A launch's threads are counted in 32 bits.
  if (grid * threads > 0xffffffffLL) return fail(RRB_EUNSUPPORTED, "too many tiles for one launch");
  hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, s, p);
  return launched("expert product");
}

// Estimated time (us) of the form over BM x BN tiles, `resident` of them per CU
// at a time: rounds of tiles of so many steps, `step` each, and `rest` per tile
// (first loads, results); no less than moving the operands from the L2s takes
// at 10 TB/s, nor than moving the weights (or their gradients) from or to HBM
// at 5.5 TB/s.  The rates are measured; what counts is which shape comes out
// first.
template <int FORM, bool GATED>
double estimate(const ProductArgs &p, int bm, int bn, int resident, double step, double rest) {
  constexpr double kCus = 256;
  const double live = p.groups < p.rows ? p.groups : p.rows;
  const int cols = GATED ? bn / 2 : bn;
  const double across = (p.n + cols - 1) / cols;
  const double weights = 2.0 * p.n * (GATED ? 2 : 1) * p.halves * (FORM == kGradW ? p.groups : live) *
                         (FORM == kGradW ? p.m : p.k);
  double down, steps, moved;
  if (FORM == kGradW) {
    down = static_cast<double>((p.m + bm - 1) / bm) * p.halves * p.groups;
    steps = live > 0 ? p.rows / live / kStep : 0;
    moved = down * across * steps * (bm + bn);
  } else {
    down = static_cast<double>(p.rows) / bm + live / 2;
    if (down < live) down = live;
    steps = static_cast<double>((p.k + kStep - 1) / kStep) * (FORM == kGradX ? p.halves : 1);
    moved = across * steps * (down * bn + p.rows);
  }
  const double rounds = down * across / (kCus * resident);
  // Rounds that are not whole: about half a one more where tiles come and go
  // by themselves, up to a whole one where one fills a CU.
  const double more = rounds <= 1 ? 1 : rounds + 0.5;
  const double whole = rounds <= 1 ? 1 : (resident > 1 ? more : std::ceil(rounds)) / rounds;
  const double matrix = more * (steps * step + rest);
  return std::max(matrix, std::max(moved * kStep * 2 / 10e6, weights / 5.5e6 * whole));
}

// Three tile shapes.  256 x 256 is the fastest by far where there are enough
// tiles to fill the CUs (1.3 PFLOP/s; 64 x 256 reaches 0.7, 64 x 64 0.5), but
// few tiles leave CUs idle, and few rows leave a tile empty.  Measured (us;
// 256 x 256, 64 x 256, 64 x 64), products of `rows` in each of G groups:
//   G 1, 1 row, 4096 x 4096: 61, 41, 20     G 16, 64, 4096 x 2048: 74, 58, 79
//   G 1, 512, 8192 x 1024: 147, 76, 37      G 1, 2048, 4096 x 2048: 85, 50, 57
//   G 32, 1, 7168 x 2048: 158, 155, 152     G 8, 512, 2048 x 2048: 57, 69, 63
//   G 2, 1024, 4096 x 4096: 94, 132, 121    G 32, 160, 2048 x 1024: 46, 51, 51
template <int FORM, bool GATED>
rrb_status launch_product(const ProductArgs &p, hipStream_t s) {
  bool direct = p.lda % 8 == 0 && p.ldb % 8 == 0;
  for (int h = 0; h < 2; ++h) direct = direct && aligned(p.a[h], 16) && aligned(p.b[h], 16);
  if (!direct) {
    if (estimate<FORM, GATED>(p, 128, 128, 2, 1.7, 2) <= estimate<FORM, GATED>(p, 64, 64, 4, 1.1, 1))
      return launch_tiles<128, 128, FORM, GATED>(product_kernel<128, 128, 2, 2, FORM, GATED>, 256, p, s);
    return launch_tiles<64, 64, FORM, GATED>(product_kernel<64, 64, 2, 2, FORM, GATED>, 256, p, s);
  }
  // A tile of at most 128 valid rows takes about half a 256-row step.
  const bool half = FORM != kGradW && static_cast<int64_t>(p.groups) * 128 >= p.rows;
  const double big = estimate<FORM, GATED>(p, 256, 256, 1, half ? 0.9 : 1.55, 8);
  const double mid = estimate<FORM, GATED>(p, 64, 256, 1, 0.66, 4);
  const double low = estimate<FORM, GATED>(p, 64, 64, 2, 0.42, 2);
  if (big <= mid && big <= low)
    return launch_tiles<256, 256, FORM, GATED>(product_turns_kernel<FORM, GATED>, 512, p, s);
  if (mid <= low)
    return launch_tiles<64, 256, FORM, GATED>(product_direct_kernel<64, 256, 2, 4, 3, FORM, GATED>, 512, p, s);
  return launch_tiles<64, 64, FORM, GATED>(product_direct_kernel<64, 64, 2, 2, 5, FORM, GATED>, 256, p, s);
}

int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }

// What every entry point checks of its sizes.
rrb_status check_spec(const rrb_expert_spec *s, const int32_t *offsets) {
  if (!s) return fail(RRB_EINVAL, "NULL spec");
  if (s->rows < 0 || s->in < 1 || s->out < 1 || s->groups < 1)
    return fail(RRB_EINVAL, "rows %lld, in %lld, out %lld, groups %d: rows >= 0 and the others >= 1 needed",
                (long long)s->rows, (long long)s->in, (long long)s->out, s->groups);
  if (s->activation < RRB_ACT_NONE || s->activation > RRB_ACT_RELU)
    return fail(RRB_EINVAL, "unknown activation %d", s->activation);
  if (!offsets && s->groups != 1) return fail(RRB_EINVAL, "NULL offsets with %d groups", s->groups);
  if (s->rows >= 1LL << 30) return fail(RRB_EUNSUPPORTED, "rows %lld >= 2^30", (long long)s->rows);
  if (s->in > kMaxWidth || s->out > kMaxWidth)
    return fail(RRB_EUNSUPPORTED, "in %lld, out %lld: at most 2^20", (long long)s->in, (long long)s->out);
  if (s->groups > kMaxGroups) return fail(RRB_EUNSUPPORTED, "groups %d: at most %d", s->groups, kMaxGroups);
  return RRB_OK;
}

// Bytes of the arrays that the sizes name.
struct Bytes {
  int64_t x, y, w, bias, offsets;
  explicit Bytes(const rrb_expert_spec &s)
      : x(s.rows * s.in * 2), y(s.rows * s.out * 2), w(s.groups * s.in * s.out * 2), bias(s.groups * s.out * 2),
        offsets((s.groups + 1ll) * 4) {}
};

ProductArgs base_args(const rrb_expert_spec &s, const int32_t *offsets) {
  ProductArgs p;
  std::memset(&p, 0, sizeof p);
  p.offsets = offsets;
  p.rows = static_cast<int32_t>(s.rows);
  p.groups = s.groups;
  p.halves = 1;
  p.bstride = s.in * s.out;
  return p;
}

template <bool GATED>
rrb_status launch_act_grad(const ActGradArgs &a, int act, hipStream_t s) {
  if (a.rows == 0) return RRB_OK;
  const int64_t blocks = (a.rows * (a.ldo / 8) + 255) / 256;
  const dim3 grid(static_cast<unsigned>(blocks < 8192 ? blocks : 8192));
  switch (act) {
#define RRB_CASE(A)                                                                         \
  case A:                                                                                   \
    hipLaunchKernelGGL((act_grad_kernel<A, GATED>), grid, dim3(256), 0, s, a);              \
    break;
    RRB_CASE(RRB_ACT_NONE) RRB_CASE(RRB_ACT_SILU) RRB_CASE(RRB_ACT_GELU) RRB_CASE(RRB_ACT_GELU_TANH)
    RRB_CASE(RRB_ACT_RELU)
#undef RRB_CASE
  }
  return launched("activation gradient");
}

// Splits of each group's rows for the bias gradient, towards eight workgroups per
// CU, and at most 64, which one thread then joins.  The join is a launch of 2 us.
// Without an activation a turn of 32 rows takes 0.2 us, and groups of fewer than
// 512 rows on average stay whole.  With one it takes up to 0.7, and the rows of
// the whole arena count, as they may all be one group's (32768 x 64, silu, all in
// one of 256 groups: the whole backward 428 us at four splits in the order
// groups, splits; 247 at eight in this one).
int64_t bias_splits(const rrb_expert_spec &s, bool act) {
  const int64_t mean = s.rows / s.groups, most = act ? s.rows / 256 : mean < 512 ? 1 : mean / 128;
  return std::max<int64_t>(1, std::min<int64_t>(64, std::min(2048 / ((s.out + 63) / 64 * s.groups), most)));
}

rrb_status launch_bias_grad(const BiasGradArgs &a, int act, hipStream_t s) {
  // Splits before groups: a group's then run on different XCDs.
  const dim3 grid(static_cast<unsigned>((a.n + 63) / 64), static_cast<unsigned>(a.splits),
                  static_cast<unsigned>(a.p.groups));
  switch (act) {
#define RRB_CASE(A)                                                              \
  case A:                                                                        \
    if (a.dz)                                                                    \
      hipLaunchKernelGGL((bias_grad_kernel<A, true>), grid, dim3(256), 0, s, a); \
    else                                                                         \
      hipLaunchKernelGGL((bias_grad_kernel<A, false>), grid, dim3(256), 0, s, a); \
    break;
    RRB_CASE(RRB_ACT_NONE) RRB_CASE(RRB_ACT_SILU) RRB_CASE(RRB_ACT_GELU) RRB_CASE(RRB_ACT_GELU_TANH)
    RRB_CASE(RRB_ACT_RELU)
#undef RRB_CASE
  }
  const rrb_status st = launched("bias gradient");
  if (st != RRB_OK || !a.part) return st;
  const int64_t blocks = (static_cast<int64_t>(a.p.groups) * a.n + 255) / 256;
  hipLaunchKernelGGL(bias_join_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a);
  return launched("bias gradient's join");
}

const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }
uint16_t *u16(void *p) { return static_cast<uint16_t *>(p); }

}  // namespace
}  // namespace rrb

using namespace rrb;

extern "C" {

rrb_status rrb_expert_gated(const rrb_expert_spec *spec, const void *d_x, const int32_t *d_offsets,
                            const void *d_w_gate, const void *d_w_up, void *d_out, void *d_save_gate,
                            void *d_save_up, rrb_stream_t stream) {
  clear_error();
  rrb_status st = check_spec(spec, d_offsets);
  if (st != RRB_OK) return st;
  if (spec->rows == 0) return RRB_OK;
  if (!d_x || !d_w_gate || !d_w_up || !d_out) return fail(RRB_EINVAL, "NULL x, w_gate, w_up or out");
  if (!d_save_gate != !d_save_up) return fail(RRB_EINVAL, "save_gate and save_up go together");
  const Bytes z(*spec);
  const Span spans[] = {{d_x, z.x, "x", false}, {d_offsets, z.offsets, "offsets", false},
                        {d_w_gate, z.w, "w_gate", false}, {d_w_up, z.w, "w_up", false},
                        {d_out, z.y, "out", true}, {d_save_gate, z.y, "save_gate", true},
                        {d_save_up, z.y, "save_up", true}};
  if ((st = check_disjoint(spans)) != RRB_OK) return st;
  ProductArgs p = base_args(*spec, d_offsets);
  p.a[0] = p.a[1] = u16(d_x);
  p.b[0] = u16(d_w_gate);
  p.b[1] = u16(d_w_up);
  p.c[0] = u16(d_out);
  p.save[0] = u16(d_save_gate);
  p.save[1] = u16(d_save_up);
  p.lda = p.ldb = spec->in;
  p.ldc = spec->out;
  p.n = static_cast<int32_t>(spec->out);
  p.k = static_cast<int32_t>(spec->in);
  p.act = spec->activation;
  return launch_product<kForward, true>(p, static_cast<hipStream_t>(stream));
}

rrb_status rrb_expert_linear(const rrb_expert_spec *spec, const void *d_x, const int32_t *d_offsets,
                             const void *d_w, const void *d_bias, const void *d_residual, void *d_out,
                             void *d_save_pre, rrb_stream_t stream) {
  clear_error();
  rrb_status st = check_spec(spec, d_offsets);
  if (st != RRB_OK) return st;
  if (spec->rows == 0) return RRB_OK;
  if (!d_x || !d_w || !d_out) return fail(RRB_EINVAL, "NULL x, w or out");
  const Bytes z(*spec);
  // A tile's residual is read before any of the tile is written, and by no
  // other workgroup: it may be the output itself.
  const Span spans[] = {{d_x, z.x, "x", false}, {d_offsets, z.offsets, "offsets", false}, {d_w, z.w, "w", false},
                        {d_bias, z.bias, "bias", false},
                        {d_residual == d_out ? nullptr : d_residual, z.y, "residual", false},
                        {d_out, z.y, "out", true}, {d_save_pre, z.y, "save_pre", true}};
  if ((st = check_disjoint(spans)) != RRB_OK) return st;
  ProductArgs p = base_args(*spec, d_offsets);
  p.a[0] = p.a[1] = u16(d_x);
  p.b[0] = p.b[1] = u16(d_w);
  p.c[0] = u16(d_out);
  p.save[0] = u16(d_save_pre);
  p.bias = u16(d_bias);
  p.residual = u16(d_residual);
  p.lda = p.ldb = spec->in;
  p.ldc = spec->out;
  p.n = static_cast<int32_t>(spec->out);
  p.k = static_cast<int32_t>(spec->in);
  p.act = spec->activation;
  return launch_product<kForward, false>(p, static_cast<hipStream_t>(stream));
}

rrb_status rrb_expert_gated_backward_workspace(const rrb_expert_spec *spec, size_t *bytes) {
  clear_error();
  if (!bytes) return fail(RRB_EINVAL, "NULL bytes");
  *bytes = 0;
  static const int32_t any = 0;
  rrb_status st = check_spec(spec, &any);
  if (st != RRB_OK) return st;
  *bytes = static_cast<size_t>(2 * spec->rows * padded(spec->out) * 2);
  return RRB_OK;
}

rrb_status rrb_expert_linear_backward_workspace(const rrb_expert_spec *spec, size_t *bytes) {
  clear_error();
  if (!bytes) return fail(RRB_EINVAL, "NULL bytes");
  *bytes = 0;
  static const int32_t any = 0;
  rrb_status st = check_spec(spec, &any);
  if (st != RRB_OK) return st;
  // dZ, and the bias gradient's partial sums where its rows are split (the more
  // of them with an activation: one size serves all).
  const int64_t splits = std::max(bias_splits(*spec, false), bias_splits(*spec, true));
  *bytes = static_cast<size_t>(spec->rows * padded(spec->out) * 2 +
                               (splits > 1 ? splits * spec->groups * spec->out * 4 : 0));
  return RRB_OK;
}

rrb_status rrb_expert_gated_backward(const rrb_expert_spec *spec, const void *d_dout, const void *d_x,
                                     const int32_t *d_offsets, const void *d_w_gate, const void *d_w_up,
                                     const void *d_gate, const void *d_up, void *d_dx, void *d_dw_gate,
                                     void *d_dw_up, void *d_workspace, size_t workspace_bytes,
                                     rrb_stream_t stream) {
  clear_error();
  rrb_status st = check_spec(spec, d_offsets);
  if (st != RRB_OK) return st;
  // (Without rows dx is empty, and its address may be NULL.)
  if (spec->rows > 0 && !d_dx && !d_dw_gate) return fail(RRB_EINVAL, "no gradient asked for");
  if (!d_dw_gate != !d_dw_up) return fail(RRB_EINVAL, "dw_gate and dw_up go together");
  size_t need = 0;
  st = rrb_expert_gated_backward_workspace(spec, &need);
  if (st != RRB_OK) return st;
  if (spec->rows > 0) {
    if (!d_dout || !d_gate || !d_up) return fail(RRB_EINVAL, "NULL dout, gate or up");
    if (d_dx && (!d_w_gate || !d_w_up)) return fail(RRB_EINVAL, "NULL w_gate or w_up");
    if (d_dw_gate && !d_x) return fail(RRB_EINVAL, "NULL x");
    if (!d_workspace || workspace_bytes < need || !aligned(d_workspace, 16))
      return fail(RRB_EINVAL, "workspace of %zu bytes, 16-byte aligned, needed", need);
  }
  const Bytes z(*spec);
  const Span spans[] = {{d_dout, z.y, "dout", false}, {d_x, z.x, "x", false}, {d_offsets, z.offsets, "offsets", false},
                        {d_w_gate, z.w, "w_gate", false}, {d_w_up, z.w, "w_up", false}, {d_gate, z.y, "gate", false},
                        {d_up, z.y, "up", false}, {d_dx, z.x, "dx", true}, {d_dw_gate, z.w, "dw_gate", true},
                        {d_dw_up, z.w, "dw_up", true}, {d_workspace, static_cast<int64_t>(need), "workspace", true}};
  if ((st = check_disjoint(spans)) != RRB_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t pitch = padded(spec->out);
  uint16_t *dgate = u16(d_workspace);
  uint16_t *dup = dgate ? dgate + spec->rows * pitch : nullptr;
  ActGradArgs g;
  std::memset(&g, 0, sizeof g);
  g.dout = u16(d_dout);
  g.gate = u16(d_gate);
  g.up = u16(d_up);
  g.dgate = dgate;
  g.dup = dup;
  g.offsets = d_offsets;
  g.rows = spec->rows;
  g.ldo = pitch;
  g.n = static_cast<int32_t>(spec->out);
  g.groups = spec->groups;
  if ((st = launch_act_grad<true>(g, spec->activation, s)) != RRB_OK) return st;
  ProductArgs p = base_args(*spec, d_offsets);
  p.a[0] = dgate;
  p.a[1] = dup;
  p.lda = g.ldo;
  p.halves = 2;
  p.n = static_cast<int32_t>(spec->in);
  if (d_dx && spec->rows > 0) {
    ProductArgs q = p;
    q.b[0] = u16(d_w_gate);
    q.b[1] = u16(d_w_up);
    q.c[0] = u16(d_dx);
    q.ldb = q.ldc = spec->in;
    q.k = static_cast<int32_t>(spec->out);
    if ((st = launch_product<kGradX, false>(q, s)) != RRB_OK) return st;
  }
  if (d_dw_gate) {
    p.b[0] = p.b[1] = u16(d_x);
    p.c[0] = u16(d_dw_gate);
    p.c[1] = u16(d_dw_up);
    p.ldb = p.ldc = spec->in;
    p.m = static_cast<int32_t>(spec->out);
    if ((st = launch_product<kGradW, false>(p, s)) != RRB_OK) return st;
  }
  return RRB_OK;
}

rrb_status rrb_expert_linear_backward(const rrb_expert_spec *spec, const void *d_dout, const void *d_x,
                                      const int32_t *d_offsets, const void *d_w, const void *d_pre, void *d_dx,
                                      void *d_dw, void *d_dbias, void *d_workspace, size_t workspace_bytes,
                                      rrb_stream_t stream) {
  clear_error();
  rrb_status st = check_spec(spec, d_offsets);
  if (st != RRB_OK) return st;
  if (spec->rows > 0 && !d_dx && !d_dw && !d_dbias) return fail(RRB_EINVAL, "no gradient asked for");
  size_t need = 0;
  st = rrb_expert_linear_backward_workspace(spec, &need);
  if (st != RRB_OK) return st;
  const bool act = spec->activation != RRB_ACT_NONE;
  if (spec->rows > 0) {
    if (!d_dout) return fail(RRB_EINVAL, "NULL dout");
    if (act && !d_pre) return fail(RRB_EINVAL, "an activation's gradient needs pre");
    if (d_dx && !d_w) return fail(RRB_EINVAL, "NULL w");
    if (d_dw && !d_x) return fail(RRB_EINVAL, "NULL x");
    if (!d_workspace || workspace_bytes < need || !aligned(d_workspace, 16))
      return fail(RRB_EINVAL, "workspace of %zu bytes, 16-byte aligned, needed", need);
  }
  const Bytes z(*spec);
  const Span spans[] = {{d_dout, z.y, "dout", false}, {d_x, z.x, "x", false}, {d_offsets, z.offsets, "offsets", false},
                        {d_w, z.w, "w", false}, {act ? d_pre : nullptr, z.y, "pre", false}, {d_dx, z.x, "dx", true},
                        {d_dw, z.w, "dw", true}, {d_dbias, z.bias, "dbias", true},
                        {d_workspace, static_cast<int64_t>(need), "workspace", true}};
  if ((st = check_disjoint(spans)) != RRB_OK) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  ProductArgs p = base_args(*spec, d_offsets);
  p.a[0] = p.a[1] = u16(d_dout);
  p.lda = spec->out;
  // Without an activation dZ is dY itself; rows that do not start on 16-byte
  // boundaries are copied into padded ones first.
  const bool copy = (d_dx || d_dw) && (act || spec->out % 8 || !aligned(d_dout, 16));
  if (d_dbias) {
    BiasGradArgs b;
    std::memset(&b, 0, sizeof b);
    b.dout = u16(d_dout);
    b.pre = act ? u16(d_pre) : nullptr;
    b.db = u16(d_dbias);
    b.dz = copy ? u16(d_workspace) : nullptr;
    b.ldo = padded(spec->out);
    b.splits = static_cast<int32_t>(bias_splits(*spec, act));
    if (b.splits > 1) b.part = reinterpret_cast<float *>(u16(d_workspace) + spec->rows * b.ldo);
    b.p = p;
    b.n = static_cast<int32_t>(spec->out);
    if ((st = launch_bias_grad(b, spec->activation, s)) != RRB_OK) return st;
  } else if (copy) {
    ActGradArgs g;
    std::memset(&g, 0, sizeof g);
    g.dout = u16(d_dout);
    g.gate = u16(d_pre);
    g.dgate = u16(d_workspace);
    g.offsets = d_offsets;
    g.rows = spec->rows;
    g.ldo = padded(spec->out);
    g.n = static_cast<int32_t>(spec->out);
    g.groups = spec->groups;
    if ((st = launch_act_grad<false>(g, spec->activation, s)) != RRB_OK) return st;
  }
  if (copy) {
    p.a[0] = p.a[1] = u16(d_workspace);
    p.lda = padded(spec->out);
  }
  p.n = static_cast<int32_t>(spec->in);
  if (d_dx && spec->rows > 0) {
    ProductArgs q = p;
    q.b[0] = q.b[1] = u16(d_w);
    q.c[0] = u16(d_dx);
    q.ldb = q.ldc = spec->in;
    q.k = static_cast<int32_t>(spec->out);
    if ((st = launch_product<kGradX, false>(q, s)) != RRB_OK) return st;
  }
  if (d_dw) {
    ProductArgs q = p;
    q.b[0] = q.b[1] = u16(d_x);
    q.c[0] = q.c[1] = u16(d_dw);
    q.ldb = q.ldc = spec->in;
    q.m = static_cast<int32_t>(spec->out);
    if ((st = launch_product<kGradW, false>(q, s)) != RRB_OK) return st;
  }
  return RRB_OK;
}

}  // extern "C"
