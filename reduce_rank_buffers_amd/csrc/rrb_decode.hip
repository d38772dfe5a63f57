// The expert layer of an MoE for a few tokens, whole, in two kernels.  For token
// t with choices e_j and weights w_j
//   y_t = sum over j of w_j Wd[e_j] h_j,  h_j = act(Wg[e_j] x_t) * (Wu[e_j] x_t)
// The first kernel computes the h of every choice, the second the products with
// Wd and the sum.  Weights are bf16, or 8-bit integers with a scale for each
// output channel; x, h and y are bf16, and sums fp32.
//
// With few tokens the time is the weights' bytes: every weight of an expert that
// some token chose is read once, for all of its tokens (so long as they are not
// many).  A wave computes sixteen output channels, rows of a weight matrix, for up to
// sixteen columns at a time, the tokens; which tokens chose which experts each
// workgroup finds for itself from the choices.  h is kept in two bf16 parts: rounded
// to one it would cost more than the result's own rounding (0.0024 of the result's
// norm off instead of 0.0017), and the matrix instruction has columns to spare.
#include <hip/hip_runtime.h>

#include "rrb_activations.h"
#include "rrb_internal.h"
#include "rrb_kernels.h"
#include "rrb_lds.h"

namespace rrb {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kMaxTokens = 64;
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int kUpWaves = 4, kDownWaves = 8;
// Experts of layers whose weights go through LDS, which holds the tables too.
constexpr int direct_experts(int tokens) { return tokens <= 8 ? kRouteMaxExperts : 512; }

struct DecodeArgs {
  const uint16_t *x;
  const int32_t *idx;
  const float *w;
  const void *gate, *up, *down;
  const float *sgate, *sup, *sdown;  // integers' scales
  uint16_t *h;                       // [rows][2][pitch]: bf16 parts whose sum is h
  uint16_t *y;
  int32_t tokens, topk, experts, hidden, inner, pitch, act, tiles;
};

// ---- which experts have tokens -----------------------------------------------
//
// Every workgroup reads the choices and makes the same tables: each expert's tokens
// as a mask, and the experts that have any, ascending, each with the row of h at
// which its tokens' rows begin (one for each, in the tokens' order).

template <int TOKENS, int EXPERTS>
struct Choices {
  static constexpr int BITS = TOKENS <= 8 ? 8 : TOKENS <= 16 ? 16 : 64;
  static constexpr int ROWS = TOKENS * kRouteMaxTopk;
  uint32_t mask[EXPERTS * BITS / 32];
  uint32_t list[ROWS < EXPERTS ? ROWS : EXPERTS];  // expert | its first row << 16

  __device__ __forceinline__ void add(int e, int t) {
    if (BITS == 8)
      atomicOr(&mask[e >> 2], 1u << (8 * (e & 3) + t));
    else if (BITS == 16)
      atomicOr(&mask[e >> 1], 1u << (16 * (e & 1) + t));
    else
      atomicOr(&mask[2 * e + (t >> 5)], 1u << (t & 31));
  }
  __device__ __forceinline__ uint64_t tokens(int e) const {
    if (BITS == 8) return mask[e >> 2] >> (8 * (e & 3)) & 0xff;
    if (BITS == 16) return mask[e >> 1] >> (16 * (e & 1)) & 0xffff;
    return mask[2 * e] | static_cast<uint64_t>(mask[2 * e + 1]) << 32;
  }
};

// What the second kernel needs besides: each row's weight.
template <int TOKENS, int EXPERTS>
struct Weights {
  int16_t idx[TOKENS * kRouteMaxTopk];  // the choices: experts that are here, or -1
  uint16_t row_of[EXPERTS];
  float row[TOKENS * kRouteMaxTopk];
};

struct Live {
  int experts;   // in the list
  int turns[4];  // sum over them of tokens / 4, / 8, / 16 and / 32, rounded up
};

__device__ __forceinline__ uint64_t below(int lane) { return (uint64_t(1) << lane) - 1; }

// Fills `c`, and `weights` if it is there (NT threads).
template <int NT, int TOKENS, int EXPERTS>
__device__ __forceinline__ Live find_experts(const DecodeArgs &a, Choices<TOKENS, EXPERTS> &c,
                                             Weights<TOKENS, EXPERTS> *weights) {
  constexpr int EACH = (TOKENS * kRouteMaxTopk + NT - 1) / NT;
  const int tid = threadIdx.x, lane = tid & 63, n = a.tokens * a.topk;
  int e[EACH], t[EACH];
  float w[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int at = i * NT + tid;
    e[i] = at < n ? a.idx[at] : -1;
    w[i] = weights && at < n ? a.w[at] : 0.f;
    t[i] = at / a.topk;
    if (e[i] < 0 || e[i] >= a.experts) e[i] = -1;
  }
  for (int i = tid; i < (a.experts * c.BITS + 31) / 32; i += NT) c.mask[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int at = i * NT + tid;
    if (weights && at < n) weights->idx[at] = e[i];
    if (e[i] >= 0) c.add(e[i], t[i]);
  }
  __syncthreads();
  // Every wave makes the whole list, so that none waits for another's part.
  Live live = {0, {0, 0, 0, 0}};
  int rows = 0, fours = 0, sixteens = 0;  // turns of four and (upper half) eight, ..
  for (int first = 0; first < a.experts; first += 64) {
    const int x = first + lane;
    const int many = x < a.experts ? __popcll(c.tokens(x)) : 0;
    const uint64_t set = __ballot(many > 0);
    if (!set) continue;
    int upto = many;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(upto, d, 64);
      if (lane >= d) upto += v;
    }
    const int row = rows + upto - many;
    if (many) {
      c.list[live.experts + __popcll(set & below(lane))] = x | row << 16;
      if (weights) weights->row_of[x] = row;
    }
    live.experts += __popcll(set);
    rows += __shfl(upto, 63, 64);
    fours += (many + 3) / 4 | (many + 7) / 8 << 16;
    sixteens += (many + 15) / 16 | (many + 31) / 32 << 16;
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    fours += __shfl_xor(fours, d, 64);
    sixteens += __shfl_xor(sixteens, d, 64);
  }
  live.turns[0] = uniform(fours) & 0xffff;
  live.turns[1] = uniform(fours) >> 16;
  live.turns[2] = uniform(sixteens) & 0xffff;
  live.turns[3] = uniform(sixteens) >> 16;
  if (weights) {
    // A token's first choice of an expert brings those of the same one with it.
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      if (e[i] < 0) continue;
      const int j = i * NT + tid - t[i] * a.topk;
      bool first = true;
      for (int k = 0; k < a.topk; ++k) {
        if (k == j || weights->idx[t[i] * a.topk + k] != e[i]) continue;
        if (k < j) first = false;
        w[i] += a.w[t[i] * a.topk + k];
      }
      if (first) weights->row[weights->row_of[e[i]] + __popcll(c.tokens(e[i]) & below(t[i]))] = w[i];
    }
    __syncthreads();
  }
  live.experts = uniform(live.experts);
  return live;
}

// Lane i receives the lane of the i-th set bit of `set` (the others' follow).
__device__ __forceinline__ int in_order(uint64_t set) {
  const int lane = threadIdx.x & 63;
  const int at = set >> lane & 1 ? __popcll(set & below(lane)) : __popcll(set) + __popcll(~set & below(lane));
  return __builtin_amdgcn_ds_permute(at * 4, lane);
}

// An expert of the list and its tokens.
struct Expert {
  int e, row;    // and its tokens' first row of h
  uint64_t set;  // its tokens
  int many;

  template <int TOKENS, int EXPERTS>
  __device__ __forceinline__ void find(const Choices<TOKENS, EXPERTS> &c, int slot) {
    const int entry = uniform(static_cast<int>(c.list[slot]));
    e = entry & 0xffff;
    row = entry >> 16;
    const uint64_t tokens = c.tokens(e);
    set = static_cast<uint32_t>(uniform(static_cast<int>(tokens)));
    if (c.BITS > 32) set |= static_cast<uint64_t>(static_cast<uint32_t>(uniform(static_cast<int>(tokens >> 32)))) << 32;
    many = __popcll(set);
  }
};

// ---- operands --------------------------------------------------------------------

// A fragment of 16 weight rows is 16 bytes per lane: lane l holds row l % 16, from
// chunk l / 16 on.  bf16: 32 k, one matrix instruction; integers: 64 k, two, the
// lower and the upper half of each lane's sixteen.
template <bool INT>
constexpr int kFragment = INT ? 64 : 32;  // k

__device__ __forceinline__ bf16x8_t as_bf16(u32x4_t v) { return __builtin_bit_cast(bf16x8_t, v); }

// Eight integers (exact in bf16): a conversion that takes its byte, and half of
// one that packs two, for each.
__device__ __forceinline__ bf16x8_t as_bf16(uint32_t lo, uint32_t hi) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int v = static_cast<int>(i < 2 ? lo : hi), at = 16 * (i & 1);
    r[i] = cvt_pk_bf16(static_cast<float>(static_cast<int>(__builtin_amdgcn_sbfe(v, at, 8))),
                       static_cast<float>(static_cast<int>(__builtin_amdgcn_sbfe(v, at + 8, 8))));
  }
  return as_bf16(r);
}

// 16 bytes from `src` in a row of `length` elements, of which `have` are left there;
// the others are 0.
template <typename T>
__device__ __forceinline__ u32x4_t load_part(const T *src, int have, int length) {
  constexpr int N = 16 / sizeof(T), PER = 4 / sizeof(T);
  u32x4_t v = {0, 0, 0, 0};
  if (have >= N) {
    __builtin_memcpy(&v, src, 16);
  } else if (have > 0 && length >= N) {
    uint64_t w[2];
    load_last(src, have * static_cast<int>(sizeof(T)), w);
    __builtin_memcpy(&v, w, 16);
  } else if (have > 0) {
    for (int i = 0; i < have; ++i) {
      const uint32_t e = static_cast<uint32_t>(src[i]) << (8 * static_cast<int>(sizeof(T)) * (i % PER));
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] |= i / PER == q ? e : 0u;
    }
  }
  return v;
}

template <bool INT>
struct Element {
  typedef uint16_t T;
};
template <>
struct Element<true> {
  typedef uint8_t T;
};

// One block of k: U fragments of each of M matrices' 16 rows, and of NC x 16 rows
// of the other operand.
template <bool INT, int M, int NC, int U>
struct Block {
  static constexpr int K = U * kFragment<INT>;
  static constexpr int XS = INT ? 2 : 1;  // 16-byte chunks of the other operand per fragment
  typedef typename Element<INT>::T T;
  u32x4_t w[M][U], x[NC][U][XS];

  __device__ __forceinline__ void load(const T *const (&rows)[M], const uint16_t *const (&xrows)[NC], int k0) {
    const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kFragment<INT> + q * (kFragment<INT> / 4);
#pragma unroll
      for (int m = 0; m < M; ++m) __builtin_memcpy(&w[m][u], rows[m] + k, 16);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int h = 0; h < XS; ++h) __builtin_memcpy(&x[c][u][h], xrows[c] + k + h * 8, 16);
    }
  }
  // The same where the rows end at k = `end`.
  __device__ __forceinline__ void load_end(const T *const (&rows)[M], const uint16_t *const (&xrows)[NC], int k0,
                                           int end) {
    const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kFragment<INT> + q * (kFragment<INT> / 4);
#pragma unroll
      for (int m = 0; m < M; ++m) w[m][u] = load_part(rows[m] + k, end - k, end);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int h = 0; h < XS; ++h) x[c][u][h] = load_part(xrows[c] + k + h * 8, end - k - h * 8, end);
    }
  }
  __device__ __forceinline__ void multiply(f32x4_t (&acc)[M][NC]) const {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < XS; ++h) {
          const bf16x8_t wf = INT ? as_bf16(w[m][u][2 * h], w[m][u][2 * h + 1]) : as_bf16(w[m][u]);
#pragma unroll
          for (int c = 0; c < NC; ++c)
            acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, as_bf16(x[c][u][h]), acc[m][c], 0, 0, 0);
        }
  }
};

// acc += rows x xrows over the blocks first, first + step, .. below `last` of k, one
// block ahead, two blocks a turn (with the loop's ends behind each, the compiler kept
// copies of both: up to 512 bytes of scratch a lane, and 64 tokens on 16 experts, 2001
// x 1001, took 122 us, integers 119, where these are 114 and 73).  Only the last block
// of a row may be partial.
template <bool INT, int M, int NC, int U>
__device__ __forceinline__ void sum_blocks(f32x4_t (&acc)[M][NC],
                                           const typename Element<INT>::T *const (&rows)[M],
                                           const uint16_t *const (&xrows)[NC], int first, int step, int last, int end) {
  typedef Block<INT, M, NC, U> B;
  const int whole = min(last, end / B::K);
  int b = first;
  if (b < whole) {
    B even, odd;
    even.load(rows, xrows, b * B::K);
    for (; b + 2 * step < whole; b += 2 * step) {
      odd.load(rows, xrows, (b + step) * B::K);
      even.multiply(acc);
      even.load(rows, xrows, (b + 2 * step) * B::K);
      odd.multiply(acc);
    }
    const bool more = b + step < whole;
    if (more) odd.load(rows, xrows, (b + step) * B::K);
    even.multiply(acc);
    if (more) odd.multiply(acc);
    b += more ? 2 * step : step;
  }
  if (b < last) {
    // (At once where the registers have room.)
    typedef Block<INT, M, NC, NC == 1 ? U : 1> P;
    P part;
    for (int k = b * B::K; k < end; k += P::K) {
      part.load_end(rows, xrows, k, end);
      part.multiply(acc);
    }
  }
}

// Fragments per block, so that two blocks leave registers for two waves a SIMD and
// more (integers have twice the columns' bytes per fragment: at bf16's depths 193 to
// 272 registers, and 64 tokens on 16 experts, 2001 x 1001, took 83 us; at these 119
// to 206, and 73).
template <bool INT, int NC>
constexpr int kDepth = INT ? (NC == 1 ? 2 : 1) : NC == 1 ? 4 : NC == 2 ? 2 : 1;

// Calls `run` with NC = 1, 2 or 4 tiles of 16, whichever holds `tiles` first; MOST
// bounds what is compiled.
template <int MOST, typename F>
__device__ __forceinline__ void with_tiles(int tiles, F run) {
  if (MOST == 1 || tiles <= 1) {
    run(std::integral_constant<int, 1>{});
  } else if constexpr (MOST >= 2) {
    if (MOST == 2 || tiles <= 2)
      run(std::integral_constant<int, 2>{});
    else if constexpr (MOST >= 4)
      run(std::integral_constant<int, 4>{});
  }
}

// ---- h ------------------------------------------------------------------------------

template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
  return activate<ACT>(g) * u;
}
__device__ __forceinline__ float gated(int act, float g, float u) {
  switch (act) {
    case RRB_ACT_SILU: return gated<RRB_ACT_SILU>(g, u);
    case RRB_ACT_GELU: return gated<RRB_ACT_GELU>(g, u);
    case RRB_ACT_GELU_TANH: return gated<RRB_ACT_GELU_TANH>(g, u);
    case RRB_ACT_RELU: return gated<RRB_ACT_RELU>(g, u);
    default: return g * u;
  }
}

// Channels n .. n + 3 of a row of h from its two projections.
__device__ __forceinline__ void store_h(const DecodeArgs &a, int n, int row, f32x4_t gate, f32x4_t up) {
  uint16_t *to = a.h + static_cast<int64_t>(row) * 2 * a.pitch + n;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (n + q >= a.inner) continue;
    const float h = gated(a.act, gate[q], up[q]);
    const uint16_t first = f32_to_bf16_rne(h);
    const float value = bf16_to_f32(first);
    to[q] = first;
    // (An infinity, h's or by its rounding, has no remainder, nor has a NaN.)
    to[a.pitch + q] = f32_to_bf16_rne(fabsf(value) < INFINITY ? h - value : 0.f);
  }
}

// Scales of four of an expert's channels, n of them all.
__device__ __forceinline__ f32x4_t load_scales(const float *scales, int e, int n, int at) {
  f32x4_t v;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = scales[static_cast<int64_t>(e) * n + min(at + q, n - 1)];
  return v;
}

// Sixteen channels of one expert per workgroup at a time: its waves take blocks of
// k by turns, and wave 0 joins their sums in order.  For rows off 16-byte boundaries,
// whose weights go straight into the matrix instruction's registers: bound by the
// loads in flight and their alignment (5 tokens, 1001 x 333: 10 us and the second kernel
// 9, mostly latency; 64 tokens on 16 experts, 2001 x 1001: 61 and 52, 1.7 TB/s, integers
// 37 and 35, 1.3).
template <bool INT, int MOST>
__global__ void __launch_bounds__(kUpWaves * 64) decode_up_kernel(DecodeArgs a) {
  typedef typename Element<INT>::T T;
  __shared__ Choices<kMaxTokens, kRouteMaxExperts> choices;
  __shared__ f32x4_t part[kUpWaves - 1][2][MOST][64];
  const int items = a.tiles * find_experts<kUpWaves * 64, kMaxTokens, kRouteMaxExperts>(a, choices, nullptr).experts;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int slot = item / a.tiles, n0 = (item - slot * a.tiles) * 16;
    Expert who;
    who.find(choices, slot);
    const int e = who.e, order = in_order(who.set);
    const int64_t row = min(n0 + (lane & 15), a.inner - 1) + static_cast<int64_t>(e) * a.inner;
    const T *const rows[2] = {static_cast<const T *>(a.gate) + row * a.hidden,
                              static_cast<const T *>(a.up) + row * a.hidden};
    with_tiles<MOST>((who.many + 15) / 16, [&](auto tiles) {
      constexpr int NC = decltype(tiles)::value, U = kDepth<INT, NC>, K = U * kFragment<INT>;
      const uint16_t *xrows[NC];
      int to[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = c * 16 + (lane & 15);
        xrows[c] = a.x + static_cast<int64_t>(__shfl(order, i < who.many ? i : 0, 64)) * a.hidden;
        to[c] = i < who.many ? who.row + i : -1;
      }
      f32x4_t acc[2][NC];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      sum_blocks<INT, 2, NC, U>(acc, rows, xrows, wave, kUpWaves, (a.hidden + K - 1) / K, a.hidden);
      if (wave) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int c = 0; c < NC; ++c) part[wave - 1][m][c][lane] = acc[m][c];
      }
      __syncthreads();
      if (wave) return;
      const int n = n0 + (lane >> 4) * 4;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
          for (int i = 0; i < kUpWaves - 1; ++i) acc[m][c] += part[i][m][c][lane];
        if (INT) {
          acc[0][c] *= load_scales(a.sgate, e, a.inner, n);
          acc[1][c] *= load_scales(a.sup, e, a.inner, n);
        }
        if (to[c] >= 0) store_h(a, n, to[c], acc[0][c], acc[1][c]);
      }
    });
    __syncthreads();
  }
}

// ---- y ------------------------------------------------------------------------------

// Adds an expert's sixteen channels of a token to its sums: those of both parts of
// h, which are two columns, HALF apart.  Where an infinite weight (or a NaN) has made
// the first part's sum infinite it stands alone: the second part, 0 or of either
// sign, would turn it into a NaN.
template <int HALF>
__device__ __forceinline__ void add_expert(f32x4_t acc, bool scaled, f32x4_t scale, int token, float share,
                                           f32x4_t *sums) {
  f32x4_t z;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // row_ror by 16 - HALF: lane i of a row receives lane (i + HALF) % 16.
    const int other = __builtin_amdgcn_mov_dpp(__float_as_int(acc[q]), 0x120 + 16 - HALF, 0xf, 0xf, false);
    z[q] = fabsf(acc[q]) < INFINITY ? acc[q] + __int_as_float(other) : acc[q];
    if (scaled) z[q] *= scale[q];
  }
  if (token < 0) return;
  f32x4_t &s = sums[token * 4 + ((threadIdx.x & 63) >> 4)];
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] += share * z[q];
}

// y of the workgroup's sixteen channels from its waves' sums, [wave][token][16].
template <int WAVES>
__device__ __forceinline__ void store_y(const DecodeArgs &a, int n0, const float *all) {
  for (int i = threadIdx.x; i < a.tokens * 16; i += WAVES * 64) {
    float v = 0.f;
    for (int s = 0; s < WAVES; ++s) v += all[s * a.tokens * 16 + i];
    const int n = n0 + (i & 15);
    if (n < a.hidden) a.y[static_cast<int64_t>(i >> 4) * a.hidden + n] = f32_to_bf16_rne(v);
  }
}

// Sixteen channels of y per workgroup, of every token: its waves share the blocks
// of all experts' k evenly, each a run of them, and add what an expert gives to
// sums of their own, which are joined in order at the end.  The two parts of a
// token's h are two columns of the matrix instruction, which has sixteen whether
// they are used or not: eight tokens at a time.
template <bool INT, int WAVES, int MOST>
__global__ void __launch_bounds__(WAVES * 64) decode_down_kernel(DecodeArgs a) {
  typedef typename Element<INT>::T T;
  constexpr int NT = WAVES * 64;
  __shared__ Choices<kMaxTokens, kRouteMaxExperts> choices;
  __shared__ Weights<kMaxTokens, kRouteMaxExperts> weights;
  extern __shared__ __align__(16) unsigned char dynamic[];
  f32x4_t *const all = reinterpret_cast<f32x4_t *>(dynamic);  // [wave][token][channel / 4]
  const int n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  f32x4_t *const sums = all + wave * a.tokens * 4;
  for (int t = lane; t < a.tokens * 4; t += 64) sums[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int count = find_experts<NT, kMaxTokens, kRouteMaxExperts>(a, choices, &weights).experts;
  constexpr int K = kFragment<INT> * kDepth<INT, 1>;  // a unit of the waves' shares: whole blocks of every depth
  const int per = (a.inner + K - 1) / K;         // units per expert
  int b = static_cast<int>(static_cast<int64_t>(count) * per * wave / WAVES);
  const int end = static_cast<int>(static_cast<int64_t>(count) * per * (wave + 1) / WAVES);
  while (b < end) {
    const int slot = b / per, from = b - slot * per, to = min(per, from + end - b);
    Expert who;
    who.find(choices, slot);
    const int e = who.e, order = in_order(who.set);
    const int64_t row = min(n0 + (lane & 15), a.hidden - 1) + static_cast<int64_t>(e) * a.hidden;
    const T *const rows[1] = {static_cast<const T *>(a.down) + row * a.inner};
    for (int base = 0; base < who.many; base += 8 * MOST) {
      with_tiles<MOST>((who.many - base + 7) / 8, [&](auto tiles) {
        constexpr int NC = decltype(tiles)::value, U = kDepth<INT, NC>, PER = kDepth<INT, 1> / U;
        const uint16_t *xrows[NC];
        int token[NC];
        float share[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int i = min(base + c * 8 + (lane & 7), who.many - 1), t = __shfl(order, i, 64);
          xrows[c] = a.h + (static_cast<int64_t>(who.row + i) * 2 + (lane >> 3 & 1)) * a.pitch;
          share[c] = weights.row[who.row + i];
          token[c] = base + c * 8 + (lane & 7) < who.many && !(lane & 8) ? t : -1;
        }
        f32x4_t acc[1][NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[0][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        constexpr int B = U * kFragment<INT>;
        sum_blocks<INT, 1, NC, U>(acc, rows, xrows, from * PER, 1, min(to * PER, (a.inner + B - 1) / B), a.inner);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          f32x4_t scale = {1.f, 1.f, 1.f, 1.f};
          if (INT) scale = load_scales(a.sdown, e, a.hidden, n0 + (lane >> 4) * 4);
          add_expert<8>(acc[0][c], INT, scale, token[c], share[c], sums);
        }
      });
    }
    b += to - from;
  }
  __syncthreads();
  store_y<WAVES>(a, n0, reinterpret_cast<const float *>(all));
}

// ---- weights through LDS -------------------------------------------------------------
//
// Rows on 16-byte boundaries go from memory to LDS without a register
// (buffer_load_dwordx4 ... lds), eight lanes to 128 bytes of a row: memory is read
// in whole lines, and once, so past the caches.  A wave has a ring of stages of its
// own and waits for nobody but its loads: a stage is 128 bytes of each of 16 rows of
// the M matrices and, as rows of the same kind, what they are multiplied by, of NX
// groups of eight columns.  Row r keeps its 16-byte chunk c at c ^ (r / 2 % 8), so
// that a fragment's reads meet all banks.  Rings do not empty between experts or
// tiles: the loads run ahead into the next segment.
//
// Bound by HBM where rows are long: a pure read of such rows reaches 6.0 TB/s
// through the caches and 6.65 past them (whole lines; 5.6 in halves, as the matrix
// instruction's own layout reads them).  Measured, us (first kernel and second):
// one token, 8 of 32 experts, 7168 x 2048 bf16: 70 (6.7 TB/s) and 44 (5.3), where loads
// into registers took 79 and 48; int8 39 and 24 (integers are converted at 1.5
// operations each, and the columns' bytes are twice as many beside the weights'); 64
// tokens on 28 of 32 experts, bf16: 277 (5.9) and 151 (5.4); one token, 2048 x 1024
// (100 MB): 14 and 11, of which launch, tables and the first loads are 4 to 5 each.

constexpr int kStageBytes = 128;  // of a weight row
__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }

// What a stage's loads start from: a segment's matrices and columns.
template <int M, int NX>
struct Source {
  u32x4_t wd[M], xd;
  int wv[2], xv[NX];  // this lane's bytes in the buffers: of its weight rows, of its columns

  // Of every matrix `rows` rows exist, `pitch` bytes apart.  This lane's column of
  // group g begins `at[g]` bytes into the buffer xd, or is not there (-1).
  __device__ __forceinline__ void begin(int pitch, int rows, const int (&at)[NX]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = h * 8 + (lane >> 3);
      wv[h] = r < rows ? r * pitch + ((lane & 7) ^ row_swizzle(r)) * 16 : kOutside;
    }
#pragma unroll
    for (int g = 0; g < NX; ++g)
      xv[g] = at[g] < 0 ? kOutside : at[g] + ((lane & 7) ^ row_swizzle(g * 8 + (lane >> 3))) * 16;
  }
};

template <bool INT, int M, int NX, int RING>
struct Stream {
  static constexpr int XB = INT ? 2 : 1;                    // 128-byte blocks of a column per stage
  static constexpr int NC = NX <= 2 ? 1 : NX / 2;           // tiles of 16 columns
  static constexpr int LOADS = 2 * M + NX * XB;             // of 1 KiB
  static constexpr int STAGE = LOADS * 1024;
  static constexpr int STAGES = RING / STAGE < 8 ? RING / STAGE : 8;
  static_assert(STAGES >= 2 && (STAGES - 2) * LOADS < 64, "stages in the ring, loads that can be counted");

  // Starts stage `s` (128 bytes at s * 128 of rows of `end` bytes) into the ring at
  // LDS address `to`; where it is not live nothing is read.
  static __device__ __forceinline__ void start(const Source<M, NX> &from, int s, bool live, int end, int to) {
    const int lane = threadIdx.x & 63;
    const int along = s * kStageBytes;
    if (live && along + kStageBytes <= end) {
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) load_to_lds<true>(from.wd[m], to + (m * 2 + h) * 1024, from.wv[h], along);
#pragma unroll
      for (int g = 0; g < NX; ++g)
#pragma unroll
        for (int b = 0; b < XB; ++b)
          load_to_lds(from.xd, to + (2 * M + g * XB + b) * 1024, from.xv[g], along * XB + b * kStageBytes);
      return;
    }
    // The row's last bytes, or nothing: chunks past the end lie outside the buffers.
    const int first = live ? along : end;
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int chunk = (lane & 7) ^ row_swizzle(h * 8 + (lane >> 3));
        load_to_lds<true>(from.wd[m], to + (m * 2 + h) * 1024, first + chunk * 16 >= end ? kOutside : from.wv[h],
                          live ? along : 0);
      }
#pragma unroll
    for (int g = 0; g < NX; ++g)
#pragma unroll
      for (int b = 0; b < XB; ++b) {
        // (Integers: a stage's 128 elements are 256 bytes of a column.)
        const int chunk = b * 8 + ((lane & 7) ^ row_swizzle(g * 8 + (lane >> 3)));
        load_to_lds(from.xd, to + (2 * M + g * XB + b) * 1024, first + chunk * (16 / XB) >= end ? kOutside : from.xv[g],
                    live ? along * XB + b * kStageBytes : 0);
      }
  }

  static __device__ __forceinline__ void multiply(const unsigned char *stage, f32x4_t (&acc)[M][NC]) {
    const int lane = threadIdx.x & 63, q = lane >> 4;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      u32x4_t w[M], x[NC][XB];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int r = lane & 15;
        w[m] = *reinterpret_cast<const u32x4_t *>(stage + m * 2048 + r * 128 + ((kk * 4 + q) ^ row_swizzle(r)) * 16);
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        // One group of eight columns stands in both halves of the sixteen.
        const int col = NX == 1 ? lane & 7 : c * 16 + (lane & 15);
        const unsigned char *row = stage + (2 * M + (col >> 3) * XB) * 1024 + (col & 7) * 128;
#pragma unroll
        for (int h = 0; h < XB; ++h) {
          const int chunk = (INT ? 2 * q + h : kk * 4 + q) ^ row_swizzle(col);
          x[c][h] = *reinterpret_cast<const u32x4_t *>(row + (INT ? kk * 1024 : 0) + chunk * 16);
        }
      }
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < XB; ++h) {
          const bf16x8_t wf = INT ? as_bf16(w[m][2 * h], w[m][2 * h + 1]) : as_bf16(w[m]);
#pragma unroll
          for (int c = 0; c < NC; ++c)
            acc[m][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, as_bf16(x[c][h]), acc[m][c], 0, 0, 0);
        }
    }
  }

  // Goes through the segments from `segment` on, the loads of the next ones ahead
  // of the sums of this one: for each, `finish` gets the sums of its stages from,
  // from + step, .. below to (rows of `end` bytes).
  template <typename S, typename F>
  static __device__ __forceinline__ void run(unsigned char *ring, S segment, int step, int end, F finish) {
    // (A wave without any segment has no buffers to load through.)
    if (!segment.valid()) return;
    const int at = lds_address(ring);
    S ahead = segment;
    Source<M, NX> source;
    int s = 0, to = 0;
    auto begin = [&] {
      if (ahead.valid()) {
        ahead.template begin<M, NX>(source);
        s = ahead.from();
        to = ahead.to();
      }
    };
    auto next = [&](int buf) {
      while (ahead.valid() && s >= to) {
        ahead.next();
        begin();
      }
      start(source, s, ahead.valid(), end, at + buf * STAGE);
      s += step;
    };
    begin();
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) next(i);
    int buf = 0, free = STAGES - 1;
    for (; segment.valid(); segment.next()) {
      f32x4_t acc[M][NC];
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      for (int i = segment.from(); i < segment.to(); i += step) {
        // This stage's loads have landed, and what was read of the one that is
        // loaded next has arrived.
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((STAGES - 2) * LOADS) : "memory");
        next(free);
        free = buf;
        multiply(ring + buf * STAGE, acc);
        buf = buf + 1 == STAGES ? 0 : buf + 1;
      }
      finish(segment, acc);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  }
};

// Groups of eight columns, 1 .. MOST, that make the least work: an expert with more
// tokens than they hold goes by turns, each of which reads its weights again (W KiB a
// stage), and every group is read and multiplied for every expert (X KiB, from the
// L2, at about half the cost).  live.turns[FIRST] is that of one group.
template <int W, int X, int MOST, int FIRST>
__device__ __forceinline__ int best_groups(const Live &live) {
  int best = 1, cost = live.turns[FIRST] * (2 * W + X);
#pragma unroll
  for (int i = 1; 1 << i <= MOST; ++i) {
    const int c = live.turns[FIRST + i < 4 ? FIRST + i : 3] * (2 * W + (X << i));
    if (c < cost) best = 1 << i, cost = c;
  }
  return best;
}

// Calls `run` with NX = 1, 2, 4 or 8; MOST bounds what is compiled.
template <int MOST, typename F>
__device__ __forceinline__ void with_groups(int groups, F run) {
  if (MOST == 1 || groups <= 1) {
    run(std::integral_constant<int, 1>{});
  } else if constexpr (MOST >= 2) {
    if (MOST == 2 || groups <= 2) {
      run(std::integral_constant<int, 2>{});
    } else if constexpr (MOST >= 4) {
      if (MOST == 4 || groups <= 4)
        run(std::integral_constant<int, 4>{});
      else if constexpr (MOST >= 8)
        run(std::integral_constant<int, 8>{});
    }
  }
}

// Sixteen scales of an integer matrix's rows, of which this lane gets its four;
// through scalar registers, whose loads are not counted with the stages'.
__device__ __forceinline__ f32x4_t four_scales(const float *scales, int64_t at) {
  typedef __attribute__((address_space(4))) const float *constant;
  const constant s = (constant)(reinterpret_cast<uintptr_t>(uniform(scales + at)));
  // (Pinned to scalars: a lane's own four would be a vector load.)
  auto scalar = [](float v) {
    asm volatile("" : "+s"(v));
    return v;
  };
  const int q = (threadIdx.x & 63) >> 4;
  f32x4_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v0 = scalar(s[i]), v1 = scalar(s[4 + i]), v2 = scalar(s[8 + i]), v3 = scalar(s[12 + i]);
    const float lo = q & 1 ? v1 : v0, hi = q & 1 ? v3 : v2;
    v[i] = q & 2 ? hi : lo;
  }
  return v;
}

__device__ __forceinline__ void barrier_without_loads() {
  // What was written to LDS is there; the stages under way stay so.
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A segment of the first kernel: sixteen channels of one expert for up to 8 NX of
// its tokens; every wave of the workgroup has stages of it.
template <typename C, int NX>
struct UpSegment {
  const DecodeArgs &a;
  const C &choices;
  int item, items, size, wave;  // 16 channels of an expert each, `gridDim.x` apart
  int n0, base;
  Expert who;

  __device__ __forceinline__ void enter() {
    if (!valid()) return;
    const int slot = item / a.tiles;
    n0 = (item - slot * a.tiles) * 16;
    base = 0;
    who.find(choices, slot);
  }
  __device__ __forceinline__ bool valid() const { return item < items; }
  __device__ __forceinline__ void next() {
    base += 8 * NX;
    if (base < who.many) return;
    item += gridDim.x;
    enter();
  }
  __device__ __forceinline__ int from() const { return wave; }
  __device__ __forceinline__ int to() const { return (a.hidden * size + kStageBytes - 1) / kStageBytes; }
  template <int M, int G>
  __device__ __forceinline__ void begin(Source<M, G> &s) const {
    const int rows = min(16, a.inner - n0), pitch = a.hidden * size;
    const int64_t row = (static_cast<int64_t>(who.e) * a.inner + n0) * pitch;
    s.wd[0] = descriptor(static_cast<const uint8_t *>(a.gate) + row, rows * pitch);
    s.wd[1] = descriptor(static_cast<const uint8_t *>(a.up) + row, rows * pitch);
    s.xd = descriptor(a.x, a.tokens * a.hidden * 2);
    const int order = in_order(who.set);
    int at[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int i = base + g * 8 + ((threadIdx.x & 63) >> 3), t = __shfl(order, i & 63, 64);
      at[g] = i < who.many ? t * a.hidden * 2 : -1;
    }
    s.begin(pitch, rows, at);
  }
};

// decode_up_kernel's work.  TOKENS: what the launch is for; MOST: groups of eight
// tokens at a time.
template <bool INT, int TOKENS, int MOST, int RING>
__global__ void __launch_bounds__(kUpWaves * 64) decode_up_direct_kernel(DecodeArgs a) {
  constexpr int TILES = (MOST + 1) / 2;
  typedef Choices<TOKENS, direct_experts(TOKENS)> C;
  __shared__ C choices;
  __shared__ __align__(16) unsigned char rings[kUpWaves][RING];
  // One group of columns stands twice in the sixteen, and is kept once.
  constexpr int LANES = MOST == 1 ? 32 : 64;
  __shared__ f32x4_t parts[kUpWaves - 1][2 * TILES][LANES];
  const Live live = find_experts<kUpWaves * 64, TOKENS, direct_experts(TOKENS)>(a, choices, nullptr);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int at = MOST == 1 ? (lane >> 4) * 8 + (lane & 7) : lane;
  with_groups<MOST>(best_groups<4, INT ? 2 : 1, MOST, 1>(live), [&](auto groups) {
    constexpr int NX = decltype(groups)::value;
    typedef Stream<INT, 2, NX, RING> S;
    typedef UpSegment<C, NX> Segment;
    Segment first{a, choices, static_cast<int>(blockIdx.x), live.experts * a.tiles, INT ? 1 : 2, wave, 0, 0, {}};
    first.enter();
    int turn = 0;
    S::run(rings[wave], first, kUpWaves, a.hidden * (INT ? 1 : 2), [&](const Segment &s, f32x4_t (&acc)[2][S::NC]) {
      // The waves' sums meet in LDS, but for those of the wave whose turn it is to
      // join them, in the waves' order.
      const int joins = turn++ & (kUpWaves - 1);
      if (wave != joins) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int c = 0; c < S::NC; ++c) parts[wave - (wave > joins)][m * S::NC + c][at] = acc[m][c];
      }
      barrier_without_loads();
      f32x4_t sum[2][S::NC];
      if (wave == joins) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int c = 0; c < S::NC; ++c) {
            f32x4_t all = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kUpWaves; ++i)
              all += i == wave ? acc[m][c] : parts[min(i - (i > wave), kUpWaves - 2)][m * S::NC + c][at];
            sum[m][c] = all;
          }
      }
      barrier_without_loads();
      if (wave != joins) return;
      if (INT) {
        const int64_t row = static_cast<int64_t>(s.who.e) * a.inner + s.n0;
        const f32x4_t gate = four_scales(a.sgate, row), up = four_scales(a.sup, row);
#pragma unroll
        for (int c = 0; c < S::NC; ++c) sum[0][c] *= gate, sum[1][c] *= up;
      }
#pragma unroll
      for (int c = 0; c < S::NC; ++c) {
        const int i = s.base + c * 16 + (lane & 15);
        if (i < s.who.many && (NX > 1 || !(lane & 8)))
          store_h(a, s.n0 + (lane >> 4) * 4, s.who.row + i, sum[0][c], sum[1][c]);
      }
    });
  });
}

// A segment of the second kernel: this wave's stages of one expert for up to
// 4 NX of its tokens.
template <typename C, int NX>
struct DownSegment {
  static constexpr int HALF = NX == 1 ? 4 : 8;  // columns between a token's two
  const DecodeArgs &a;
  const C &choices;
  int slot, first, end, size, per;  // this wave's stages, counted over all experts
  int base;
  Expert who;

  __device__ __forceinline__ void enter() {
    if (!valid()) return;
    base = 0;
    who.find(choices, slot);
  }
  __device__ __forceinline__ bool valid() const { return slot * per < end; }
  __device__ __forceinline__ void next() {
    base += 4 * NX;
    if (base < who.many) return;
    ++slot;
    enter();
  }
  __device__ __forceinline__ int from() const { return max(0, first - slot * per); }
  __device__ __forceinline__ int to() const { return min(per, end - slot * per); }
  template <int M, int G>
  __device__ __forceinline__ void begin(Source<M, G> &s) const {
    const int n0 = blockIdx.x * 16, rows = min(16, a.hidden - n0), pitch = a.inner * size;
    s.wd[0] = descriptor(static_cast<const uint8_t *>(a.down) + (static_cast<int64_t>(who.e) * a.hidden + n0) * pitch,
                         rows * pitch);
    s.xd = descriptor(a.h, a.tokens * a.topk * 2 * a.pitch * 2);
    int at[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int col = g * 8 + ((threadIdx.x & 63) >> 3), i = base + col / (2 * HALF) * HALF + col % HALF;
      at[g] = i < who.many ? ((who.row + i) * 2 + col / HALF % 2) * a.pitch * 2 : -1;
    }
    s.begin(pitch, rows, at);
  }
};

// decode_down_kernel's work.  MOST: groups of eight columns at a time.
template <bool INT, int TOKENS, int WAVES, int MOST, int RING>
__global__ void __launch_bounds__(WAVES * 64) decode_down_direct_kernel(DecodeArgs a) {
  typedef Choices<TOKENS, direct_experts(TOKENS)> C;
  __shared__ C choices;
  __shared__ Weights<TOKENS, direct_experts(TOKENS)> weights;
  __shared__ __align__(16) unsigned char rings[WAVES][RING];
  __shared__ f32x4_t all[WAVES * TOKENS * 4];  // [wave][token][channel / 4]
  const int n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  f32x4_t *const sums = all + wave * a.tokens * 4;
  for (int t = lane; t < a.tokens * 4; t += 64) sums[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const Live live = find_experts<WAVES * 64, TOKENS, direct_experts(TOKENS)>(a, choices, &weights);
  with_groups<MOST>(best_groups<2, INT ? 2 : 1, MOST, 0>(live), [&](auto groups) {
    constexpr int NX = decltype(groups)::value;
    typedef Stream<INT, 1, NX, RING> S;
    typedef DownSegment<C, NX> Segment;
    const int pitch = a.inner * (INT ? 1 : 2), per = (pitch + kStageBytes - 1) / kStageBytes;
    const int64_t total = static_cast<int64_t>(live.experts) * per;
    const int from = static_cast<int>(total * wave / WAVES), to = static_cast<int>(total * (wave + 1) / WAVES);
    Segment first{a, choices, from / per, from, to, INT ? 1 : 2, per, 0, {}};
    if (from == to) first.slot = live.experts, first.end = 0;
    first.enter();
    S::run(rings[wave], first, 1, pitch, [&](const Segment &s, f32x4_t (&acc)[1][S::NC]) {
      f32x4_t scale = {1.f, 1.f, 1.f, 1.f};
      if (INT) scale = four_scales(a.sdown, static_cast<int64_t>(s.who.e) * a.hidden + n0);
      const int order = in_order(s.who.set);
#pragma unroll
      for (int c = 0; c < S::NC; ++c) {
        const int i = s.base + c * 8 + (lane & (Segment::HALF - 1)), t = __shfl(order, i & 63, 64);
        const bool there = i < s.who.many && (lane & 15) < Segment::HALF;
        add_expert<Segment::HALF>(acc[0][c], INT, scale, there ? t : -1, weights.row[there ? s.who.row + i : 0], sums);
      }
    });
  });
  __syncthreads();
  store_y<WAVES>(a, n0, reinterpret_cast<const float *>(all));
}

// ---- launchers -------------------------------------------------------------------

int64_t pitch_of(const rrb_decode_spec &s) { return (s.inner + 7) / 8 * 8; }

rrb_status check_spec(const rrb_decode_spec *s) {
  if (!s) return fail(RRB_EINVAL, "NULL spec");
  if (s->tokens < 0 || s->hidden < 1 || s->inner < 1 || s->experts < 1 || s->topk < 1)
    return fail(RRB_EINVAL,
                "tokens %lld, hidden %lld, inner %lld, experts %d, topk %d: tokens >= 0 and the others >= 1 needed",
                (long long)s->tokens, (long long)s->hidden, (long long)s->inner, s->experts, s->topk);
  if (s->activation < RRB_ACT_NONE || s->activation > RRB_ACT_RELU)
    return fail(RRB_EINVAL, "unknown activation %d", s->activation);
  if (s->tokens > kMaxTokens)
    return fail(RRB_EUNSUPPORTED, "tokens %lld: at most %d", (long long)s->tokens, kMaxTokens);
  if (s->hidden > kMaxWidth || s->inner > kMaxWidth)
    return fail(RRB_EUNSUPPORTED, "hidden %lld, inner %lld: at most 2^20", (long long)s->hidden, (long long)s->inner);
  if (s->experts > kRouteMaxExperts || s->topk > kRouteMaxTopk)
    return fail(RRB_EUNSUPPORTED, "experts %d, topk %d: at most %d and %d", s->experts, s->topk, kRouteMaxExperts,
                kRouteMaxTopk);
  return RRB_OK;
}

// Tiles that the kernels are compiled for: 1, 2 or 4, of which one token's expert
// can fill `tiles`.
template <bool INT>
auto up_kernel(int tiles) {
  return tiles <= 1 ? decode_up_kernel<INT, 1> : tiles <= 2 ? decode_up_kernel<INT, 2> : decode_up_kernel<INT, 4>;
}
template <bool INT>
auto down_kernel(int tiles) {
  return tiles <= 1   ? decode_down_kernel<INT, kDownWaves, 1>
         : tiles <= 2 ? decode_down_kernel<INT, kDownWaves, 2>
                      : decode_down_kernel<INT, kDownWaves, 4>;
}

template <bool INT>
rrb_status launch_decode(const DecodeArgs &a, hipStream_t s) {
  const int most = a.experts < a.tokens * a.topk ? a.experts : a.tokens * a.topk;
  dim3 up_grid(static_cast<unsigned>(most * a.tiles)), down_grid(static_cast<unsigned>((a.hidden + 15) / 16));
  // Weights go through LDS where the rows that a kernel reads start on 16-byte
  // boundaries (integers: and both widths are of whole sixteens, as their scales are
  // read), the tables have room, and (all but widths near 2^20) offsets into h fit the
  // buffers' 31 bits.
  auto whole = [](const void *p, int width) { return width % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  const bool room = a.experts <= direct_experts(a.tokens) && (!INT || (a.hidden % 16 == 0 && a.inner % 16 == 0));
  const bool up_direct = room && whole(a.gate, a.hidden) && whole(a.up, a.hidden) && whole(a.x, a.hidden);
  const bool down_direct = room && whole(a.down, a.inner) &&
                           static_cast<int64_t>(a.tokens) * a.topk * 4 * a.pitch < (1LL << 31);
  void (*up)(DecodeArgs), (*down)(DecodeArgs);
  int down_waves = kDownWaves;
  unsigned lds = 0;
  const int t = a.tokens;
  if (up_direct) {
    // The first kernel's workgroups stay, two a CU, or one with deeper rings and tables
    // for up to 64 tokens (us, both kernels, 64 tokens on 8 experts, top-2, 4096 x 4096:
    // 249 at two a CU, where an expert's tokens go sixteen at a time, and 220; 64
    // tokens, an eighth of them here, on 32 experts, 7168 x 2048: 371 either way).
    int there = 512;
    if (t <= 8)
      up = decode_up_direct_kernel<INT, 8, 1, 18432>;
    else if (t <= 16)
      up = decode_up_direct_kernel<INT, 16, 2, 18432>;
    else
      up = decode_up_direct_kernel<INT, 64, 4, 34816>, there = 256;
    if (up_grid.x > static_cast<unsigned>(there)) up_grid.x = there;
  } else {
    if (up_grid.x > 1 << 20) up_grid.x = 1 << 20;
    up = up_kernel<INT>((t + 15) / 16);
  }
  if (down_direct) {
    // The second kernel's are as many as there are tiles of 16 channels: two of four
    // waves a CU, or one of eight where they are at most the CUs.  Tokens that all
    // meet on few experts want all columns at once, and the LDS for it.
    const bool wide = down_grid.x > 256, dense = t > 16 && t * a.topk > 16 * a.experts;
    constexpr int MOST = INT ? 2 : 4;
    if (t <= 8)
      down = wide ? decode_down_direct_kernel<INT, 8, 4, 2, 18432> : decode_down_direct_kernel<INT, 8, 8, 2, 18432>;
    else if (t <= 16)
      down = wide ? decode_down_direct_kernel<INT, 16, 4, MOST, 17408>
                  : decode_down_direct_kernel<INT, 16, 8, MOST, 17408>;
    else if (dense)
      down = decode_down_direct_kernel<INT, 64, 4, 2 * MOST, 32768>;
    else
      down = wide ? decode_down_direct_kernel<INT, 64, 4, MOST, 12288>
                  : decode_down_direct_kernel<INT, 64, 8, MOST, 12288>;
    down_waves = wide || dense ? 4 : 8;
  } else {
    down = down_kernel<INT>((t + 7) / 8);
    lds = kDownWaves * t * 64;
  }
  hipLaunchKernelGGL(up, up_grid, dim3(kUpWaves * 64), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(RRB_EHIP, "decode launch: %s", hipGetErrorString(e));
  hipLaunchKernelGGL(down, down_grid, dim3(down_waves * 64), lds, s, a);
  e = hipGetLastError();
  return e == hipSuccess ? RRB_OK : fail(RRB_EHIP, "decode launch: %s", hipGetErrorString(e));
}

}  // namespace
}  // namespace rrb

using namespace rrb;

extern "C" {

rrb_status rrb_moe_decode_workspace(const rrb_decode_spec *spec, size_t *bytes) {
  clear_error();
  if (!bytes) return fail(RRB_EINVAL, "NULL bytes");
  *bytes = 0;
  const rrb_status st = check_spec(spec);
  if (st != RRB_OK) return st;
  *bytes = static_cast<size_t>(spec->tokens * spec->topk * 2 * pitch_of(*spec) * 2);
  return RRB_OK;
}

rrb_status rrb_moe_decode(const rrb_decode_spec *spec, const void *d_x, const int32_t *d_topk_idx,
                          const float *d_topk_w, const void *d_w_gate, const void *d_w_up, const void *d_w_down,
                          const float *d_gate_scale, const float *d_up_scale, const float *d_down_scale, void *d_out,
                          void *d_workspace, size_t workspace_bytes, rrb_stream_t stream) {
  clear_error();
  size_t need = 0;
  rrb_status st = rrb_moe_decode_workspace(spec, &need);
  if (st != RRB_OK) return st;
  if (spec->tokens == 0) return RRB_OK;
  if (!d_x || !d_topk_idx || !d_topk_w || !d_w_gate || !d_w_up || !d_w_down || !d_out)
    return fail(RRB_EINVAL, "NULL x, topk_idx, topk_w, w_gate, w_up, w_down or out");
  const bool integers = d_gate_scale != nullptr;
  if (integers != (d_up_scale != nullptr) || integers != (d_down_scale != nullptr))
    return fail(RRB_EINVAL, "the three scales go together");
  if (!d_workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(d_workspace) & 15))
    return fail(RRB_EINVAL, "workspace of %zu bytes, 16-byte aligned, needed", need);
  const int64_t x = spec->tokens * spec->hidden * 2, choices = spec->tokens * spec->topk * 4;
  const int64_t w = spec->experts * spec->hidden * spec->inner * (integers ? 1 : 2);
  const int64_t in = spec->experts * spec->inner * 4, out = spec->experts * spec->hidden * 4;
  const Span spans[] = {{d_x, x, "x", false}, {d_topk_idx, choices, "topk_idx", false},
                        {d_topk_w, choices, "topk_w", false}, {d_w_gate, w, "w_gate", false},
                        {d_w_up, w, "w_up", false}, {d_w_down, w, "w_down", false},
                        {d_gate_scale, in, "gate_scale", false}, {d_up_scale, in, "up_scale", false},
                        {d_down_scale, out, "down_scale", false}, {d_out, x, "out", true},
                        {d_workspace, static_cast<int64_t>(need), "workspace", true}};
  if ((st = check_disjoint(spans)) != RRB_OK) return st;
  DecodeArgs a{};
  a.x = static_cast<const uint16_t *>(d_x);
  a.idx = d_topk_idx;
  a.w = d_topk_w;
  a.gate = d_w_gate;
  a.up = d_w_up;
  a.down = d_w_down;
  a.sgate = d_gate_scale;
  a.sup = d_up_scale;
  a.sdown = d_down_scale;
  a.h = static_cast<uint16_t *>(d_workspace);
  a.y = static_cast<uint16_t *>(d_out);
  a.tokens = static_cast<int32_t>(spec->tokens);
  a.topk = spec->topk;
  a.experts = spec->experts;
  a.hidden = static_cast<int32_t>(spec->hidden);
  a.inner = static_cast<int32_t>(spec->inner);
  a.pitch = static_cast<int32_t>(pitch_of(*spec));
  a.act = spec->activation;
  a.tiles = (a.inner + 15) / 16;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return integers ? launch_decode<true>(a, s) : launch_decode<false>(a, s);
}

}  // extern "C"
