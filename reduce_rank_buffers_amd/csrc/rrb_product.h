// The tiled product behind the experts' calls: C[m][n] = sum over k of
// A(m, k) B(n, k) over ragged groups of rows, with the calls' epilogues, and
// its launcher.  Elements are bf16, summed in fp32 (rrb_experts.hip: the
// products and their gradients), or 8-bit integers, summed exactly in 32 bits
// and scaled by row and column (rrb_experts_int8.hip: kForward alone).  The
// two differ in the matrix instruction, which takes 16 bytes of each of 16
// rows per lane group either way, and in how a sum becomes a value; tiles,
// loads and orders are the same in bytes.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "rrb_activations.h"
#include "rrb_internal.h"
#include "rrb_kernels.h"
#include "rrb_lds.h"

namespace rrb {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Groups that a wave counts, 64 at a time, before it starts on its tile.
constexpr int kMaxGroups = 4096;
// Row widths whose tile offsets fit 32 bits.
constexpr int64_t kMaxWidth = int64_t(1) << 20;

// ---- arguments --------------------------------------------------------------

// Forms of the tiled product C[m][n] = sum over k of A(m, k) B(n, k).
//   kForward  A = X rows, B = weight rows: both have k contiguous
//   kGradX    A = dZ rows (k contiguous), B(n, k) = W[k][n] (n contiguous);
//             gated: k runs over dG with Wg, then over dU with Wu
//   kGradW    A(m, k) = dZ[k][m], B(n, k) = X[k][n]: k is the group's rows
enum Form { kForward = 0, kGradX = 1, kGradW = 2 };

// What an element type brings: its fragment of 16 rows, the sums, and the
// matrix instruction.
template <typename EL>
struct Element;
template <>
struct Element<uint16_t> {  // bf16
  typedef bf16x8_t Fragment;
  typedef f32x4_t Sum;
  static __device__ __forceinline__ Sum multiply(Fragment a, Fragment b, Sum c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Element<int8_t> {
  typedef i32x4_t Fragment;
  typedef i32x4_t Sum;
  static __device__ __forceinline__ Sum multiply(Fragment a, Fragment b, Sum c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};

// Scales of integer operands: per arena row, and per group and output column
// (gated: gate, up).
template <typename EL>
struct Scales {};
template <>
struct Scales<int8_t> {
  const float *row, *col[2];
};

template <typename EL>
struct ProductArgs : Scales<EL> {
  const EL *a[2];  // kGradX: per phase; kGradW: per output; else a[0]
  const EL *b[2];  // kForward gated: gate, up; kGradX: per phase
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
template <typename EL>
__device__ __forceinline__ int32_t offset_at(const ProductArgs<EL> &p, int e) {
  if (!p.offsets) return e == 0 ? 0 : p.rows;
  const int32_t v = p.offsets[e];
  return v < 0 ? 0 : v > p.rows ? p.rows : v;
}

// ---- operand tiles in LDS -----------------------------------------------------
//
// A step's reduction indexes are 128 bytes of a row: 64 of bf16 (kStep), 128 of
// 8-bit integers.  A row tile (k contiguous) has 128-byte rows of eight 16-byte
// chunks, chunk c of row r stored at
// chunk c ^ (r / 2 % 8), so that the 16 rows of a fragment read land on 16
// different bank groups.  A column tile (k across rows) is [64][cols]: rows of
// 32-byte slots, slot s of row k stored at slot s ^ (k % 4 + 4 * (k / 8 % 2)),
// so that the eight rows that half a wave reads transposed (ds_read_b64_tr_b16)
// land on eight different bank groups.
constexpr int kStep = 64;
template <typename EL>
constexpr int kPer = 16 / static_cast<int>(sizeof(EL));  // elements of a 16-byte chunk
template <typename EL>
constexpr int kSteps = 8 * kPer<EL>;  // reduction indexes per step

__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }
template <int COLS>
__device__ __forceinline__ int col_swizzle(int k) {
  // 64 columns are four slots, and two rows span the banks.
  if (COLS == 64) return ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
  return (k & 3) | ((k >> 3) & 1) << 2;
}

// Fragment of 16 rows x 32 k from a row tile: lane l holds row l % 16, k =
// 8 (l / 16) .. + 7 (8-bit integers: 64 k, 16 a lane).
template <typename EL>
__device__ __forceinline__ typename Element<EL>::Fragment row_fragment(const unsigned char *tile, int row, int kk) {
  const int lane = threadIdx.x & 63;
  const int r = row + (lane & 15);
  const int c = (kk * 4 + (lane >> 4)) ^ row_swizzle(r);
  return *reinterpret_cast<const typename Element<EL>::Fragment *>(tile + r * 128 + c * 16);
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

// Either one; tiles of integers are row tiles.
template <bool COL, int COLS, typename EL>
__device__ __forceinline__ typename Element<EL>::Fragment fragment(const unsigned char *tile, int at, int kk) {
  if constexpr (COL)
    return col_fragment<COLS>(tile, at, kk);
  else
    return row_fragment<EL>(tile, at, kk);
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

// The same of 16 8-bit integers, of a row of `length`, whose end the chunk may pass.
__device__ __forceinline__ u32x4_t load_chunk(const int8_t *src, int64_t have, int length) {
  u32x4_t v = {0, 0, 0, 0};
  if (have >= 16) {
    __builtin_memcpy(&v, src, 16);
  } else if (have > 0 && length >= 16) {
    uint64_t w[2];
    load_last(src, static_cast<int>(have), w);
    __builtin_memcpy(&v, w, 16);
  } else if (have > 0) {
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < have) v[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(src[i])) << (8 * (i & 3));
  }
  return v;
}
__device__ __forceinline__ u32x4_t load_chunk(const uint16_t *src, int64_t have, int) { return load_chunk(src, have); }

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

// Scales of W consecutive columns, of which `have` exist.
template <int W>
__device__ __forceinline__ void load_scales(const float *src, int have, float (&v)[W]) {
  if (have >= W) {
    __builtin_memcpy(v, src, sizeof v);
  } else {
#pragma unroll
    for (int q = 0; q < W; ++q) v[q] = q < have ? src[q] : 0.f;
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

// Where an integer tile's scales begin: its first row's and its group's.
struct TileScales {
  const float *row, *col[2];
};

template <int ACT, bool GATED, bool WIDE, typename EL, int FM, int FN>
__device__ __forceinline__ void store_tile(const ProductArgs<EL> &p, const typename Element<EL>::Sum (&acc)[FM][FN],
                                           uint16_t *c, uint16_t *save0, uint16_t *save1, const uint16_t *bias,
                                           const uint16_t *residual, const TileScales &scales, Spot spot, int mvalid,
                                           int n0, unsigned char *stage) {
  constexpr bool INT = sizeof(EL) == 1;
  constexpr int W = WIDE ? 8 : 4;                           // consecutive columns per lane
  constexpr int BLOCKS = (GATED ? 2 : 1) * (WIDE ? 2 : 1);  // blocks that make them
  static_assert(FN % BLOCKS == 0, "a wave has whole outputs");
  const int lane = threadIdx.x & 63;
  auto row_at = [&](int i) {
    return spot.m + (FM > 1 && i >= FM / 2 ? spot.down + (i - FM / 2) * 16 : i * 16) + (lane & 15);
  };
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
  // An integer sum (exact) becomes a value as fl(fl(fl(sum) row) column): scales of
  // any size in either order of magnitude keep the product in range where the
  // value is.
  [[maybe_unused]] float rs[FM];
  if constexpr (INT) {
#pragma unroll
    for (int i = 0; i < FM; ++i) rs[i] = row_at(i) < mvalid ? scales.row[row_at(i)] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < FN; j += BLOCKS) {
    const int n = col_at(j), have = p.n - n0 - n;
    if (have <= 0) continue;
    float b[W];
    [[maybe_unused]] float cs[W], us[W];
    if (!GATED && bias) load_cols<W>(bias + n0 + n, have, b);
    if constexpr (INT) load_scales<W>(scales.col[0] + n0 + n, have, cs);
    if constexpr (INT && GATED) load_scales<W>(scales.col[1] + n0 + n, have, us);
    // Integers: the residual of all rows is asked for before any is needed (8000 x
    // 4096 -> 8192, us, gelu with the whole epilogue: 298 -> 286, silu 287 -> 267; row
    // by row each load was waited for).
    constexpr bool EARLY = INT && !GATED;
    [[maybe_unused]] uint32_t early[EARLY ? FM : 1][W / 2];
    if constexpr (EARLY) {
      if (residual && have >= W) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
          if (row_at(i) < mvalid) __builtin_memcpy(early[i], residual + row_at(i) * p.ldc + n0 + n, W * 2);
      }
    }
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
          if constexpr (INT) {
            v[q] = v[q] * rs[i] * cs[q];
            u[q] = u[q] * rs[i] * us[q];
          }
        }
        if (save0) {
          put(save0, m, n, v);
          put(save1, m, n, u);
        }
#pragma unroll
        for (int q = 0; q < W; ++q) v[q] = activate<ACT>(v[q]) * u[q];
      } else {
#pragma unroll
        for (int q = 0; q < W; ++q) {
          v[q] = acc[i][j + (q >> 2)][q & 3];
          if constexpr (INT) v[q] = v[q] * rs[i] * cs[q];
          v[q] += bias ? b[q] : 0.f;
        }
        if (save0) put(save0, m, n, v);
#pragma unroll
        for (int q = 0; q < W; ++q) v[q] = activate<ACT>(v[q]);
        if (residual) {
          float r[W];
          if (EARLY && have >= W) {
#pragma unroll
            for (int q = 0; q < W; ++q)
              r[q] = q & 1 ? bf16_hi(early[EARLY ? i : 0][q >> 1]) : bf16_lo(early[EARLY ? i : 0][q >> 1]);
          } else {
            load_cols<W>(residual + m * p.ldc + n0 + n, have, r);
          }
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
template <typename EL>
struct Place {
  const EL *a[2], *b[2];
  uint16_t *c;
  int32_t row0, klen;   // klen: reduction length (per phase)
  int32_t e, n0, m0, mvalid;
  bool empty;
  bool single;  // the group's only row tile (not kGradW)
};

// Tile (mt, nt) of group e, whose rows are first .. last - 1; BM x NCOLS
// outputs.  kGradW: mt counts the tiles of both outputs.
template <int BM, int NCOLS, int FORM, typename EL>
__device__ __forceinline__ Place<EL> place_at(const ProductArgs<EL> &p, int e, int first, int last, int mt, int nt) {
  Place<EL> t;
  t.e = e;
  t.n0 = nt * NCOLS;
  t.empty = false;
  t.single = false;
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
    t.single = last - first <= BM;
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
template <int BM, int NCOLS, typename EL>
__device__ __forceinline__ Place<EL> place_weight(const ProductArgs<EL> &p) {
  Place<EL> none;
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
template <int BM, int NCOLS, int LIGHT, int FORM, typename EL>
__device__ __forceinline__ Place<EL> place_counted(const ProductArgs<EL> &p) {
  Place<EL> none;
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

template <int BM, int NCOLS, int LIGHT, int FORM, typename EL>
__device__ __forceinline__ Place<EL> place_tile(const ProductArgs<EL> &p) {
  if (FORM == kGradW) return place_weight<BM, NCOLS>(p);
  return place_counted<BM, NCOLS, LIGHT, FORM>(p);
}

// Stores a wave's part of the tile.  DEALT: row regions were dealt for eight
// columns per lane.
template <int FORM, bool GATED, bool DEALT, typename EL, int FM, int FN>
__device__ __forceinline__ void finish_tile(const ProductArgs<EL> &p, const Place<EL> &t,
                                            const typename Element<EL>::Sum (&acc)[FM][FN], Spot spot,
                                            unsigned char *stage) {
  constexpr bool WIDE = DEALT && FORM == kForward;
  uint16_t *s0 = nullptr, *s1 = nullptr;
  const uint16_t *bias = nullptr, *res = nullptr;
  if (FORM == kForward) {
    if (p.save[0]) s0 = p.save[0] + t.row0 * p.ldc;
    if (p.save[1]) s1 = p.save[1] + t.row0 * p.ldc;
    if (p.bias) bias = p.bias + static_cast<int64_t>(t.e) * p.n;
    if (p.residual) res = p.residual + t.row0 * p.ldc;
  }
  TileScales scales = {nullptr, {nullptr, nullptr}};
  if constexpr (sizeof(EL) == 1) {
    scales.row = p.row + t.row0;
    for (int h = 0; h < 2; ++h) scales.col[h] = p.col[h] + static_cast<int64_t>(t.e) * p.n;
  }
#define RRB_STORE(A) store_tile<A, GATED, WIDE>(p, acc, t.c, s0, s1, bias, res, scales, spot, t.mvalid, t.n0, stage);
  if (FORM != kForward) {
    RRB_STORE(RRB_ACT_NONE)
    return;
  }
  // Staged, the pre-activation goes by itself: the stage holds one output.
  if (!GATED && stage && s0) {
    store_tile<RRB_ACT_NONE, GATED, WIDE>(p, acc, s0, nullptr, nullptr, bias, nullptr, scales, spot, t.mvalid, t.n0,
                                          stage);
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

template <typename SUM, int FM, int FN>
__device__ __forceinline__ void clear_tile(SUM (&acc)[FM][FN]) {
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = SUM{0, 0, 0, 0};
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
template <int BM, int BN, int WR, int WC, int FORM, bool GATED, typename EL>
__global__ void __launch_bounds__(WR *WC * 64) product_kernel(ProductArgs<EL> p) {
  constexpr int PER = kPer<EL>, STEP = kSteps<EL>;
  constexpr int NT = WR * WC * 64;
  constexpr int FM = BM / WR / 16, FN = BN / WC / 16;
  constexpr int A_BYTES = BM * kStep * 2, B_BYTES = BN * kStep * 2;
  constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT;  // 16-byte chunks per thread
  constexpr bool A_COL = FORM == kGradW, B_COL = FORM != kForward;
  __shared__ __align__(16) unsigned char lds[2 * (A_BYTES + B_BYTES)];

  const int tid = threadIdx.x;
  const int wave = uniform(tid >> 6);
  const Place<EL> t = place_tile<BM, GATED ? BN / 2 : BN, 0, FORM>(p);
  if (t.empty) return;
  const int klen = t.klen;
  const int per = (klen + STEP - 1) / STEP;  // steps per phase
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
    const int64_t k0 = static_cast<int64_t>(step - h * per) * STEP;
#pragma unroll
    for (int i = 0; i < CA; ++i) {
      const int id = i * NT + tid;
      if constexpr (A_COL) {
        const int kr = id / (BM / 8), pos = id % (BM / 8);
        const int ch = pos ^ (col_swizzle<BM>(kr) << 1);
        ra[i] = load_chunk(t.a[0] + (k0 + kr) * p.lda + ch * 8, there(k0 + kr, p.m - t.m0 - ch * 8, p.m, p.lda));
      } else {
        const int r = id >> 3, ch = (id & 7) ^ row_swizzle(r);
        const int64_t have = klen - k0 - ch * PER;
        ra[i] = load_chunk(t.a[h] + r * p.lda + k0 + ch * PER, r < t.mvalid ? have : 0, klen);
      }
    }
#pragma unroll
    for (int i = 0; i < CB; ++i) {
      const int id = i * NT + tid;
      if constexpr (B_COL) {
        const int kr = id / (BN / 8), pos = id % (BN / 8);
        const int ch = pos ^ (col_swizzle<BN>(kr) << 1);
        rb[i] = load_chunk(t.b[h] + (k0 + kr) * p.ldb + ch * 8, there(k0 + kr, p.n - t.n0 - ch * 8, p.n, p.ldb));
      } else {
        const int r = id >> 3, ch = (id & 7) ^ row_swizzle(r);
        const int64_t have = klen - k0 - ch * PER;
        const int n = GATED ? gated_row(r) : r;
        const EL *src = GATED && gated_up(r) ? t.b[1] : t.b[0];
        rb[i] = load_chunk(src + n * p.ldb + k0 + ch * PER, t.n0 + n < p.n ? have : 0, klen);
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
  typename Element<EL>::Sum acc[FM][FN];
  clear_tile(acc);
  if constexpr (sizeof(EL) == 1) {
    // Integers: two steps ahead while whole steps last, in two sets of registers that
    // are loaded without a branch, so that a wait for one lets the other's loads be
    // under way (9 groups of 334 rows, 2001 x 1111: 31.5 -> 27.2 us; one of 1000, 4001 x
    // 4001: 51 -> 41).
    const EL *from[CA + CB];
#pragma unroll
    for (int i = 0; i < CA + CB; ++i) {
      const int id = (i < CA ? i : i - CA) * NT + tid, r = id >> 3;
      const int n = GATED ? gated_row(r) : r, last = p.n - 1 - t.n0;
      from[i] = (i < CA ? t.a[0] + (r < t.mvalid ? r : t.mvalid - 1) * p.lda
                        : (GATED && gated_up(r) ? t.b[1] : t.b[0]) + (n < last ? n : last) * p.ldb) +
                ((id & 7) ^ row_swizzle(r)) * PER;
    }
    u32x4_t set[2][CA + CB];
    auto load = [&](u32x4_t (&v)[CA + CB], int step) {
#pragma unroll
      for (int i = 0; i < CA + CB; ++i) __builtin_memcpy(&v[i], from[i] + step * STEP, 16);
    };
    auto store = [&](const u32x4_t (&v)[CA + CB], int buf) {
#pragma unroll
      for (int i = 0; i < CA + CB; ++i)
        *reinterpret_cast<u32x4_t *>(lds + buf * (A_BYTES + B_BYTES) + (i * NT + tid) * 16) = v[i];
    };
    auto multiply = [&](int buf) {
      const unsigned char *ta = lds + buf * (A_BYTES + B_BYTES), *tb = ta + A_BYTES;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        typename Element<EL>::Fragment fa[FM], fb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i) fa[i] = row_fragment<EL>(ta, wm + i * 16, kk);
#pragma unroll
        for (int j = 0; j < FN; ++j) fb[j] = row_fragment<EL>(tb, wn + j * 16, kk);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = Element<EL>::multiply(fb[j], fa[i], acc[i][j]);
      }
    };
    const int whole = klen / STEP;
    int s = 0;
    if (whole >= 2) {
      load(set[0], 0);
      load(set[1], 1);
      store(set[0], 0);
      for (; s + 3 < whole; s += 2) {
        __syncthreads();
        load(set[0], s + 2);
        multiply(0);
        store(set[1], 1);
        __syncthreads();
        load(set[1], s + 3);
        multiply(1);
        store(set[0], 0);
      }
      __syncthreads();
      multiply(0);
      store(set[1], 1);
      __syncthreads();
      multiply(1);
      s += 2;
    }
    for (; s < steps; ++s) {
      fetch(s);
      commit(0);
      __syncthreads();
      multiply(0);
      __syncthreads();
    }
  } else {
    if (steps > 0) {
      fetch(0);
      commit(0);
    }
    for (int s = 0; s < steps; ++s) {
      __syncthreads();
      if (s + 1 < steps) fetch(s + 1);
      const unsigned char *ta = lds + (s & 1) * (A_BYTES + B_BYTES), *tb = ta + A_BYTES;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        typename Element<EL>::Fragment fa[FM], fb[FN];
#pragma unroll
        for (int i = 0; i < FM; ++i)
          fa[i] = fragment<A_COL, BM, EL>(ta, wm + i * 16, kk);
#pragma unroll
        for (int j = 0; j < FN; ++j)
          fb[j] = fragment<B_COL, BN, EL>(tb, wn + j * 16, kk);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            acc[i][j] = Element<EL>::multiply(fb[j], fa[i], acc[i][j]);
      }
      if (s + 1 < steps) commit((s + 1) & 1);
    }
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

// Two such loads, 8 KiB apart in LDS, behind one set of wait states.
__device__ __forceinline__ void load_two_to_lds(u32x4_t d, int at, int voffset0, int voffset1, int soffset) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %2, %4, %5 offen lds\n\t"
      "s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %4, %5 offen lds"
      :
      : "s"(uniform(at)), "s"(uniform(at + 8192)), "v"(voffset0), "v"(voffset1), "s"(d), "s"(uniform(soffset))
      : "memory");
}

// ONCE: the weights of a group that has one row of tiles go past the caches.
template <int BM, int BN, int WR, int WC, int STAGES, int FORM, bool GATED, typename EL, bool ONCE = false>
__global__ void __launch_bounds__(WR *WC * 64) product_direct_kernel(ProductArgs<EL> p) {
  constexpr int PER = kPer<EL>, STEP = kSteps<EL>;
  constexpr int NT = WR * WC * 64;
  constexpr int FM = BM / WR / 16, FN = BN / WC / 16;
  constexpr int A_BYTES = BM * kStep * 2, B_BYTES = BN * kStep * 2;
  constexpr int CA = BM * 8 / NT, CB = BN * 8 / NT, NCOLS = GATED ? BN / 2 : BN;
  constexpr bool A_COL = FORM == kGradW, B_COL = FORM != kForward;
  __shared__ __align__(16) unsigned char lds[STAGES * (A_BYTES + B_BYTES)];

  const int tid = threadIdx.x;
  const int wave = uniform(tid >> 6);
  const Place<EL> t = place_tile<BM, GATED ? BN / 2 : BN, 0, FORM>(p);
  if (t.empty) return;
  const int klen = t.klen;
  const int per = (klen + STEP - 1) / STEP;  // steps per phase
  const int steps = FORM == kGradX ? per * p.halves : per;
  const int lda2 = static_cast<int>(p.lda * sizeof(EL)), ldb2 = static_cast<int>(p.ldb * sizeof(EL));  // bytes

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
  auto issue = [&](auto past, int step, int buf) {
    const int h = FORM == kGradX && step >= per ? 1 : 0;
    const int kstep = step - h * per;
    const int k0 = kstep * STEP;
    const int left = klen - k0;
    const bool live = step < steps;
    const int along = live ? kstep * 128 : 0;
    const int rows = left < STEP ? left : STEP;  // of the column tiles
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
        if (left < STEP) {
          const int id = i * NT + tid;
          if (((id & 7) ^ row_swizzle(id >> 3)) * PER >= left) v = kOutside;
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
        if (left < STEP) {
          const int id = i * NT + tid;
          if (((id & 7) ^ row_swizzle(id >> 3)) * PER >= left) v = kOutside;
        }
        // The wave's eight rows are all gate rows or all up rows.
        const bool up = GATED && gated_up((i * NT + wave * 64) >> 3);
        load_to_lds<decltype(past)::value>(up ? d1 : d0, tb + i * NT * 16, v, along);
      }
    }
  };

  const int wm = wave / WC * (BM / WR), wn = wave % WC * (BN / WC);
  typename Element<EL>::Sum acc[FM][FN];
  clear_tile(acc);
  // The steps, once for each way of the weights' loads (as a lambda they made the
  // compiler order the other kernels' instructions anew).
#define RRB_STEPS(PAST)                                                                                     \
  constexpr std::integral_constant<bool, PAST> past;                                                        \
  if (steps > 0) {                                                                                          \
    _Pragma("unroll") for (int s = 0; s < STAGES - 1; ++s) issue(past, s, s);                               \
  }                                                                                                         \
  int buf = 0, free = STAGES - 1;                                                                           \
  for (int s = 0; s < steps; ++s) {                                                                         \
    /* This step's loads have landed, and every wave is done with the buffer that is loaded next. */        \
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * (CA + CB)) : "memory"); \
    issue(past, s + STAGES - 1, free);                                                                      \
    free = buf;                                                                                             \
    const unsigned char *ta = lds + buf * (A_BYTES + B_BYTES), *tb = ta + A_BYTES;                          \
    buf = buf + 1 == STAGES ? 0 : buf + 1;                                                                  \
    _Pragma("unroll") for (int kk = 0; kk < 2; ++kk) {                                                      \
      typename Element<EL>::Fragment fa[FM], fb[FN];                                                        \
      _Pragma("unroll") for (int j = 0; j < FN; ++j) fb[j] = fragment<B_COL, BN, EL>(tb, wn + j * 16, kk);  \
      _Pragma("unroll") for (int i = 0; i < FM; ++i) fa[i] = fragment<A_COL, BM, EL>(ta, wm + i * 16, kk);  \
      _Pragma("unroll") for (int i = 0; i < FM; ++i)                                                        \
        _Pragma("unroll") for (int j = 0; j < FN; ++j)                                                      \
          acc[i][j] = Element<EL>::multiply(fb[j], fa[i], acc[i][j]);                                       \
    }                                                                                                       \
  }
  if (ONCE && t.single) {
    RRB_STEPS(ONCE)
  } else {
    RRB_STEPS(false)
  }
#undef RRB_STEPS
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

template <int FORM, bool GATED, typename EL>
__device__ __forceinline__ void product_turns_tile(const ProductArgs<EL> &p, const Place<EL> &t, unsigned char *lds) {
  typedef typename Element<EL>::Fragment Fragment;
  constexpr int PER = kPer<EL>, STEP = kSteps<EL>;
  constexpr int REGION = 16384, BUFFER = 4 * REGION, NCOLS = GATED ? 128 : 256;
  constexpr bool A_COL = FORM == kGradW, B_COL = FORM != kForward;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = uniform(tid >> 6);
  const int klen = t.klen;
  const int per = (klen + STEP - 1) / STEP;
  const int steps = FORM == kGradX ? per * p.halves : per;
  const int lda2 = static_cast<int>(p.lda * sizeof(EL)), ldb2 = static_cast<int>(p.ldb * sizeof(EL));  // bytes

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
    const int k0 = ks * STEP, left = klen - k0;
    const int rows = left < STEP ? left : STEP;
    const int dst = to + (step & 1) * BUFFER + h * REGION;
    const bool live = step < steps;
    if (A_COL) {
      const auto d = descriptor(t.a[0] + k0 * p.lda, live && (h == 0 || both) ? rows * lda2 - t.m0 * 2 : 0);
      load_two_to_lds(d, dst, va[h][0], va[h][1], 0);
    } else {
      const bool any = live && (h == 0 || both);
      const auto d = descriptor(t.a[ph], any ? t.mvalid * lda2 : 0);
      const bool out = left < STEP && ch * PER >= left;
      load_two_to_lds(d, dst, out ? kOutside : va[h][0], out ? kOutside : va[h][1], any ? ks * 128 : 0);
    }
  };
  auto start_b = [&](int step, int h) {
    const int ph = FORM == kGradX && step >= per ? 1 : 0;
    const int ks = step - ph * per;
    const int k0 = ks * STEP, left = klen - k0;
    const int rows = left < STEP ? left : STEP;
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
      const bool out = left < STEP && ch * PER >= left;
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
  auto rows_at = [](const unsigned char *q) { return *reinterpret_cast<const Fragment *>(q); };
  auto cols_at = [](const unsigned char *q) {
    typedef __attribute__((address_space(3))) s16x4_t *lds_ptr;
    const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)q);
    const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(q + 1024));
    return __builtin_bit_cast(Fragment, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  Fragment fa[2][2][4], fb[2][2][2];  // [half][kk][block]
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
  typename Element<EL>::Sum acc[8][4];
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
          acc[ah * 4 + i][bh * 2 + j] = Element<EL>::multiply(
              fb[bh][kk][j], fa[ah][kk][i], acc[ah * 4 + i][bh * 2 + j]);
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

template <int FORM, bool GATED, typename EL>
__global__ void __launch_bounds__(512, 2) product_turns_kernel(ProductArgs<EL> p) {
  __shared__ __align__(16) unsigned char lds[131072];
  const Place<EL> t = place_tile<256, GATED ? 128 : 256, 128, FORM>(p);
  if (t.empty) return;
  product_turns_tile<FORM, GATED>(p, t, lds);
}

// ---- launchers -------------------------------------------------------------------

inline rrb_status launched(const char *what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? RRB_OK : fail(RRB_EHIP, "%s launch: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// Row tiles that the groups' rows can make at most: each group that has rows
// adds at most one partial tile.
template <typename EL>
int64_t most_row_tiles(const ProductArgs<EL> &p, int bm) {
  return p.rows / bm + (p.groups < p.rows ? p.groups : p.rows);
}

// Launches the form over BM x BN tiles with the given kernel.
template <int BM, int BN, int FORM, bool GATED, typename EL>
rrb_status launch_tiles(void (*kernel)(ProductArgs<EL>), int threads, ProductArgs<EL> p, hipStream_t s) {
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
template <int FORM, bool GATED, typename EL>
double estimate(const ProductArgs<EL> &p, int bm, int bn, int resident, double step, double rest) {
  constexpr double kCus = 256;
  const double live = p.groups < p.rows ? p.groups : p.rows;
  const int cols = GATED ? bn / 2 : bn;
  const double across = (p.n + cols - 1) / cols;
  const double weights = 1.0 * sizeof(EL) * p.n * (GATED ? 2 : 1) * p.halves * (FORM == kGradW ? p.groups : live) *
                         (FORM == kGradW ? p.m : p.k);
  double down, steps, moved;
  if (FORM == kGradW) {
    down = static_cast<double>((p.m + bm - 1) / bm) * p.halves * p.groups;
    steps = live > 0 ? p.rows / live / kStep : 0;
    moved = down * across * steps * (bm + bn);
  } else {
    down = static_cast<double>(p.rows) / bm + live / 2;
    if (down < live) down = live;
    steps = static_cast<double>((p.k + kSteps<EL> - 1) / kSteps<EL>) * (FORM == kGradX ? p.halves : 1);
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

// Whether one launch (2^32 threads, at most 512 a tile, and the run of tiles that a
// grid is rounded up to) holds the integer product's tiles of that shape.
template <bool GATED>
bool fits(const ProductArgs<int8_t> &p, int bm, int bn) {
  const int cols = GATED ? bn / 2 : bn;
  return most_row_tiles(p, bm) * ((p.n + cols - 1) / cols) <= (1 << 23) - 512;
}

// Estimated time (us) of an integer product over BM x BN tiles: rounds of tiles as
// above, or the weights from HBM.  In whole tiles where one group has all rows; where
// there are more how many tiles are partial is not known, and rounds come out a
// third longer.
template <bool GATED>
double estimate_integers(const ProductArgs<int8_t> &p, int bm, int bn, int resident, double step, double rest) {
  const double live = p.groups < p.rows ? p.groups : p.rows;
  const int cols = GATED ? bn / 2 : bn;
  if (!fits<GATED>(p, bm, bn)) return INFINITY;
  const double across = (p.n + cols - 1) / cols, steps = (p.k + kSteps<int8_t> - 1) / kSteps<int8_t>;
  double down = static_cast<double>(p.rows) / bm + live / 2;
  if (down < live) down = live;
  if (p.groups == 1) down = (p.rows + bm - 1) / bm;
  double rounds = down * across / (256.0 * resident);
  rounds = rounds <= 1 ? 1 : p.groups == 1 ? std::ceil(rounds) : rounds + 0.35;
  return std::max(3 + rounds * (steps * step + rest), live * p.n * (GATED ? 2.0 : 1.0) * p.k / 5.2e6);
}

// Integer products have half the steps of bf16 ones, so what a tile takes besides
// its steps weighs more, and shapes between 64 x 64 and 256 x 256 are worth their
// place.  Measured (us; 256 x 256, 128 x 256, 64 x 128, 64 x 64), products of `rows`
// in each of G groups:
//   G 1, 8000 rows, 4096 x 8192: 239, 313, 428, 548   G 1, 2048, 4096 x 2048: 52, 40, 30, 38
//   G 2, 1024, 4096 x 4096: 57, 45, 57, 71            G 1, 512, 8192 x 1024: 96, 64, 40, 27
//   G 9, 334, 2000 x 1112: 35, 28, 26, 31             G 32, 160, 2048 x 1024: 34, 30, 36, 39
//   G 16, 64, 4096 x 2048: 49, 45, 41, 36             gated, G 32, 74 to 410, 7168 x 2048: 244, 223, 296, 350
// Groups of few rows, on average, take 32 x 64 tiles, three workgroups a CU.  How many
// rows each has the device knows: a group of one row of tiles has its weights past
// the caches (G 24, 1 row, 2048 x 7168: 75 at 64 x 64, 71 past the caches, 61 at 32 x
// 64, 5.8 TB/s; 7168 x 2048 gated: 119, 110, 105; G 32, 16 rows, 7168 x 2048: 88, 81,
// 75; G 1, 1 row, 4096 x 4096: 17, 17, 13), in one of more the tiles share them (always
// past the caches, through them for all, and by group; G 32, 800 rows of which 500 in
// one, 2048 x 7168: 116, 112, 105; 7168 x 2048 gated: 193, 193, 173; all 1024 rows in one
// of 32: 67, 52, 53 and 116, 73, 73).
// Rows off 16-byte boundaries: 128 x 128 by eight waves where there are enough (one
// step ahead, G 9, 334 rows, 2001 x 1111: 43 -> 31, gated 72 -> 42; G 1, 4000, 4001 x
// 4001: 241 -> 136), else 64 x 64 (G 16, 1 row, 2001 x 1111: 24 and 21).
template <bool GATED>
rrb_status launch_integers(const ProductArgs<int8_t> &p, bool direct, hipStream_t s) {
  const int64_t rows = p.rows, groups = p.groups;
  if (!direct) {
    const int64_t tiles = (rows / 128 + std::min(groups, rows) / 2) * ((p.n + (GATED ? 63 : 127)) / (GATED ? 64 : 128));
    if ((rows > 64 * groups && tiles >= 128) || !fits<GATED>(p, 64, 64))
      return launch_tiles<128, 128, kForward, GATED>(product_kernel<128, 128, 2, 4, kForward, GATED, int8_t>, 512, p,
                                                     s);
    return launch_tiles<64, 64, kForward, GATED>(product_kernel<64, 64, 2, 2, kForward, GATED, int8_t>, 256, p, s);
  }
#define RRB_DIRECT(BM, BN, WR, WC, STAGES, ONCE)                                                                   \
  launch_tiles<BM, BN, kForward, GATED>(                                                                           \
      product_direct_kernel<BM, BN, WR, WC, STAGES, kForward, GATED, int8_t, ONCE>, WR * WC * 64, p, s)
  if (rows <= 32 * groups && fits<GATED>(p, 32, 64)) return RRB_DIRECT(32, 64, 2, 2, 4, true);
  const double big = estimate_integers<GATED>(p, 256, 256, 1, 1.4, 12);
  const double wide = estimate_integers<GATED>(p, 128, 256, 1, 0.95, 8.6);
  const double mid = estimate_integers<GATED>(p, 64, 128, 2, 0.58, 9);
  const double low = estimate_integers<GATED>(p, 64, 64, 2, 0.35, 6.3);
  const double best = std::min(std::min(big, wide), std::min(mid, low));
  if (std::isfinite(low) && (low == best || rows <= 64 * groups)) return RRB_DIRECT(64, 64, 2, 2, 5, false);
  if (std::isfinite(mid) && mid == best) return RRB_DIRECT(64, 128, 2, 2, 3, false);
  if (std::isfinite(wide) && wide == best) return RRB_DIRECT(128, 256, 2, 4, 3, false);
#undef RRB_DIRECT
  return launch_tiles<256, 256, kForward, GATED>(product_turns_kernel<kForward, GATED, int8_t>, 512, p, s);
}

// Three tile shapes.  256 x 256 is the fastest by far where there are enough
// tiles to fill the CUs (1.3 PFLOP/s; 64 x 256 reaches 0.7, 64 x 64 0.5), but
// few tiles leave CUs idle, and few rows leave a tile empty.  Measured (us;
// 256 x 256, 64 x 256, 64 x 64), products of `rows` in each of G groups:
//   G 1, 1 row, 4096 x 4096: 61, 41, 20     G 16, 64, 4096 x 2048: 74, 58, 79
//   G 1, 512, 8192 x 1024: 147, 76, 37      G 1, 2048, 4096 x 2048: 85, 50, 57
//   G 32, 1, 7168 x 2048: 158, 155, 152     G 8, 512, 2048 x 2048: 57, 69, 63
//   G 2, 1024, 4096 x 4096: 94, 132, 121    G 32, 160, 2048 x 1024: 46, 51, 51
template <int FORM, bool GATED, typename EL>
rrb_status launch_product(const ProductArgs<EL> &p, hipStream_t s) {
  bool direct = p.lda % kPer<EL> == 0 && p.ldb % kPer<EL> == 0;
  for (int h = 0; h < 2; ++h) direct = direct && aligned(p.a[h], 16) && aligned(p.b[h], 16);
  if constexpr (sizeof(EL) == 1) {
    return launch_integers<GATED>(p, direct, s);
  } else {
    if (!direct) {
      if (estimate<FORM, GATED>(p, 128, 128, 2, 1.7, 2) <= estimate<FORM, GATED>(p, 64, 64, 4, 1.1, 1))
        return launch_tiles<128, 128, FORM, GATED>(product_kernel<128, 128, 2, 2, FORM, GATED, EL>, 256, p, s);
      return launch_tiles<64, 64, FORM, GATED>(product_kernel<64, 64, 2, 2, FORM, GATED, EL>, 256, p, s);
    }
    // A tile of at most 128 valid rows takes about half a 256-row step.
    const bool half = FORM != kGradW && static_cast<int64_t>(p.groups) * 128 >= p.rows;
    const double big = estimate<FORM, GATED>(p, 256, 256, 1, half ? 0.9 : 1.55, 8);
    const double mid = estimate<FORM, GATED>(p, 64, 256, 1, 0.66, 4);
    const double low = estimate<FORM, GATED>(p, 64, 64, 2, 0.42, 2);
    if (big <= mid && big <= low)
      return launch_tiles<256, 256, FORM, GATED>(product_turns_kernel<FORM, GATED, EL>, 512, p, s);
    if (mid <= low)
      return launch_tiles<64, 256, FORM, GATED>(product_direct_kernel<64, 256, 2, 4, 3, FORM, GATED, EL>, 512, p, s);
    return launch_tiles<64, 64, FORM, GATED>(product_direct_kernel<64, 64, 2, 2, 5, FORM, GATED, EL>, 256, p, s);
  }
}

// What every entry point checks of its sizes.
inline rrb_status check_spec(const rrb_expert_spec *s, const int32_t *offsets) {
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

template <typename EL>
ProductArgs<EL> base_args(const rrb_expert_spec &s, const int32_t *offsets) {
  ProductArgs<EL> p;
  std::memset(static_cast<void *>(&p), 0, sizeof p);
  p.offsets = offsets;
  p.rows = static_cast<int32_t>(s.rows);
  p.groups = s.groups;
  p.halves = 1;
  p.bstride = s.in * s.out;
  return p;
}

inline const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }
inline uint16_t *u16(void *p) { return static_cast<uint16_t *>(p); }

}  // namespace
}  // namespace rrb
