// The expert layer of an MoE for a few tokens, whole, in two kernels.  For token
// t with choices e_j and weights w_j
//   y_t = sum over j of w_j Wd[e_j] h_j,  h_j = act(Wg[e_j] x_t) * (Wu[e_j] x_t)
// The first kernel computes the h of every choice, the second the products with
// Wd and the sum.  Weights are bf16, or 8-bit integers with a scale for each
// output channel; x, h and y are bf16, and sums fp32.
//
// With few tokens the time is the weights' bytes: every weight of an expert that
// some token chose is read once, by one wave, for all of its tokens.  A wave
// computes sixteen output channels (rows of a weight matrix, straight from memory
// into the matrix instruction's registers) for up to sixteen tokens at a time;
// which tokens chose which experts each workgroup finds for itself from the
// choices.
#include <hip/hip_runtime.h>

#include "rrb_activations.h"
#include "rrb_internal.h"
#include "rrb_kernels.h"

namespace rrb {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kMaxTokens = 64;
constexpr int kMaxChoices = kMaxTokens * kRouteMaxTopk;
constexpr int64_t kMaxWidth = int64_t(1) << 20;
constexpr int kUpWaves = 4, kDownWaves = 8;

struct DecodeArgs {
  const uint16_t *x;
  const int32_t *idx;
  const float *w;
  const void *gate, *up, *down;
  const float *sgate, *sup, *sdown;  // integers' scales
  uint16_t *h;                       // [tokens * topk][pitch]
  uint16_t *y;
  int32_t tokens, topk, experts, hidden, inner, pitch, act, tiles;
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// ---- which experts have tokens -----------------------------------------------

struct Choices {
  int32_t idx[kMaxChoices];
  uint32_t mask[kRouteMaxExperts / 32];
  uint16_t list[kRouteMaxExperts];  // experts with tokens, ascending
};

// Fills `c` (NT threads) and returns the number of experts in its list.
template <int NT>
__device__ __forceinline__ int find_experts(const DecodeArgs &a, Choices &c) {
  const int tid = threadIdx.x, n = a.tokens * a.topk;
  if (tid < kRouteMaxExperts / 32) c.mask[tid] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += NT) {
    const int e = a.idx[i];
    c.idx[i] = e;
    if (e >= 0 && e < a.experts) atomicOr(&c.mask[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  const int words = (a.experts + 31) >> 5;
  int count = 0;
  for (int i = 0; i < words; ++i) count += __popc(c.mask[i]);
  for (int e = tid; e < a.experts; e += NT) {
    if (!(c.mask[e >> 5] >> (e & 31) & 1)) continue;
    int at = __popc(c.mask[e >> 5] & ((1u << (e & 31)) - 1));
    for (int i = 0; i < e >> 5; ++i) at += __popc(c.mask[i]);
    c.list[at] = e;
  }
  __syncthreads();
  return uniform(count);
}

// The tokens of expert e, by lane: lane l < 64 is token l.  Of each its first
// choice that is e, or -1.
__device__ __forceinline__ int choice_of(const DecodeArgs &a, const Choices &c, int e, int t) {
  int found = -1;
  if (t < a.tokens) {
    for (int j = a.topk - 1; j >= 0; --j)
      if (c.idx[t * a.topk + j] == e) found = t * a.topk + j;
  }
  return found;
}

// Lane i receives the lane of the i-th set bit of `set` (the others' follow).
__device__ __forceinline__ int in_order(uint64_t set) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int at = set >> lane & 1 ? __popcll(set & below) : __popcll(set) + __popcll(~set & below);
  return __builtin_amdgcn_ds_permute(at * 4, lane);
}

// ---- operands --------------------------------------------------------------------

// A fragment of 16 weight rows is 16 bytes per lane: lane l holds row l % 16, from
// chunk l / 16 on.  bf16: 32 k, one matrix instruction; integers: 64 k, two, the
// lower and the upper half of each lane's sixteen.
template <bool INT>
constexpr int kFragment = INT ? 64 : 32;  // k

__device__ __forceinline__ bf16x8_t as_bf16(u32x4_t v) { return __builtin_bit_cast(bf16x8_t, v); }

// Eight integers (exact in bf16).
__device__ __forceinline__ bf16x8_t as_bf16(uint32_t lo, uint32_t hi) {
  bf16x8_t r;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    r[i] = static_cast<__bf16>(static_cast<float>(static_cast<int8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)))));
  return r;
}

// 16 bytes from `src`, of which the first `have` elements exist, the others 0.
template <typename T>
__device__ __forceinline__ u32x4_t load_part(const T *src, int have) {
  constexpr int N = 16 / sizeof(T), PER = 4 / sizeof(T);
  u32x4_t v = {0, 0, 0, 0};
  if (have >= N) {
    __builtin_memcpy(&v, src, 16);
  } else if (have > 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t e = src[i < have ? i : have - 1];
      v[i / PER] |= i < have ? e << (8 * static_cast<int>(sizeof(T)) * (i % PER)) : 0u;
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
      for (int m = 0; m < M; ++m) w[m][u] = load_part(rows[m] + k, end - k);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int h = 0; h < XS; ++h) x[c][u][h] = load_part(xrows[c] + k + h * 8, end - k - h * 8);
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
// block ahead.  Only the last block of a row may be partial.
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
    for (;;) {
      b += step;
      if (b >= whole) {
        even.multiply(acc);
        break;
      }
      odd.load(rows, xrows, b * B::K);
      even.multiply(acc);
      b += step;
      if (b >= whole) {
        odd.multiply(acc);
        break;
      }
      even.load(rows, xrows, b * B::K);
      odd.multiply(acc);
    }
  }
  if (b < last) {
    B part;
    part.load_end(rows, xrows, b * B::K, end);
    part.multiply(acc);
  }
}

// Fragments per block, so that two blocks fit the registers.
template <int NC>
constexpr int kDepth = NC == 4 ? 2 : 4;

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

// Sixteen channels of one expert per workgroup: its waves take blocks of k by
// turns, and wave 0 joins their sums in order.
template <bool INT>
__global__ void __launch_bounds__(kUpWaves * 64) decode_up_kernel(DecodeArgs a) {
  typedef typename Element<INT>::T T;
  __shared__ Choices choices;
  __shared__ f32x4_t part[kUpWaves - 1][2][4][64];
  const int slot = blockIdx.x / a.tiles, n0 = (blockIdx.x - slot * a.tiles) * 16;
  const int count = find_experts<kUpWaves * 64>(a, choices);
  if (slot >= count) return;
  const int e = uniform(choices.list[slot]);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int mine = choice_of(a, choices, e, lane);
  const uint64_t set = __ballot(mine >= 0);
  const int tokens = __popcll(set), order = in_order(set);
  const int64_t row = min(n0 + (lane & 15), a.inner - 1) + static_cast<int64_t>(e) * a.inner;
  const T *const rows[2] = {static_cast<const T *>(a.gate) + row * a.hidden, static_cast<const T *>(a.up) + row * a.hidden};
  auto run = [&](auto tiles) {
    constexpr int NC = decltype(tiles)::value, U = kDepth<NC>, K = U * kFragment<INT>;
    const uint16_t *xrows[NC];
    int choice[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int i = c * 16 + (lane & 15), t = __shfl(order, i < tokens ? i : 0, 64);
      xrows[c] = a.x + static_cast<int64_t>(t) * a.hidden;
      const int from = __shfl(mine, t, 64);  // by every lane, before any is left out
      choice[c] = i < tokens ? from : -1;
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
      if (choice[c] < 0) continue;
      uint16_t *to = a.h + static_cast<int64_t>(choice[c]) * a.pitch + n;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (n + q >= a.inner) continue;
        float g = acc[0][c][q], u = acc[1][c][q];
        if (INT) {
          const int64_t at = static_cast<int64_t>(e) * a.inner + n + q;
          g *= a.sgate[at];
          u *= a.sup[at];
        }
        to[q] = f32_to_bf16_rne(gated(a.act, g, u));
      }
    }
  };
  if (tokens <= 16)
    run(std::integral_constant<int, 1>{});
  else if (tokens <= 32)
    run(std::integral_constant<int, 2>{});
  else
    run(std::integral_constant<int, 4>{});
}

// ---- y ------------------------------------------------------------------------------

// Sixteen channels of y per workgroup, of every token: its waves share the blocks
// of all experts' k evenly, each a run of them, and add what an expert gives to
// sums of their own, which are joined in order at the end.
template <bool INT>
__global__ void __launch_bounds__(kDownWaves * 64) decode_down_kernel(DecodeArgs a) {
  typedef typename Element<INT>::T T;
  constexpr int NT = kDownWaves * 64;
  __shared__ Choices choices;
  __shared__ f32x4_t sums[kDownWaves][kMaxTokens][4];  // [wave][token][channel / 4]
  const int n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  for (int t = lane; t < a.tokens * 4; t += 64) sums[wave][t >> 2][t & 3] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int count = find_experts<NT>(a, choices);
  constexpr int K = 2 * kFragment<INT>;  // the smallest block
  const int per = (a.inner + K - 1) / K;  // blocks per expert
  int b = static_cast<int>(static_cast<int64_t>(count) * per * wave / kDownWaves);
  const int end = static_cast<int>(static_cast<int64_t>(count) * per * (wave + 1) / kDownWaves);
  while (b < end) {
    const int slot = b / per, from = b - slot * per, to = min(per, from + end - b);
    const int e = uniform(choices.list[slot]);
    const int mine = choice_of(a, choices, e, lane);
    float weight = 0.f;
    if (mine >= 0) {
      for (int j = 0; j < a.topk; ++j)
        if (choices.idx[lane * a.topk + j] == e) weight += a.w[lane * a.topk + j];
    }
    const uint64_t set = __ballot(mine >= 0);
    const int tokens = __popcll(set), order = in_order(set);
    const int64_t row = min(n0 + (lane & 15), a.hidden - 1) + static_cast<int64_t>(e) * a.hidden;
    const T *const rows[1] = {static_cast<const T *>(a.down) + row * a.inner};
    auto run = [&](auto tiles) {
      constexpr int NC = decltype(tiles)::value;
      const uint16_t *xrows[NC];
      int token[NC];
      float share[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int i = c * 16 + (lane & 15), t = __shfl(order, i < tokens ? i : 0, 64);
        xrows[c] = a.h + static_cast<int64_t>(__shfl(mine, t, 64)) * a.pitch;
        share[c] = __shfl(weight, t, 64);
        token[c] = i < tokens ? t : -1;
      }
      f32x4_t acc[1][NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[0][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      sum_blocks<INT, 1, NC, 2>(acc, rows, xrows, from, 1, to, a.inner);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (token[c] < 0) continue;
        f32x4_t z = acc[0][c];
        if (INT) {
          const int n = n0 + (lane >> 4) * 4;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            z[q] *= a.sdown[static_cast<int64_t>(e) * a.hidden + min(n + q, a.hidden - 1)];
        }
        f32x4_t &s = sums[wave][token[c]][lane >> 4];
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += share[c] * z[q];
      }
    };
    if (tokens <= 16)
      run(std::integral_constant<int, 1>{});
    else if (tokens <= 32)
      run(std::integral_constant<int, 2>{});
    else
      run(std::integral_constant<int, 4>{});
    b += to - from;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.tokens * 16; i += NT) {
    const int t = i >> 4, c = i & 15;
    float v = 0.f;
    for (int s = 0; s < kDownWaves; ++s) v += sums[s][t][c >> 2][c & 3];
    if (n0 + c < a.hidden) a.y[static_cast<int64_t>(t) * a.hidden + n0 + c] = f32_to_bf16_rne(v);
  }
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

template <bool INT>
rrb_status launch_decode(const DecodeArgs &a, hipStream_t s) {
  const int most = a.experts < a.tokens * a.topk ? a.experts : a.tokens * a.topk;
  hipLaunchKernelGGL(decode_up_kernel<INT>, dim3(static_cast<unsigned>(most * a.tiles)), dim3(kUpWaves * 64), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(RRB_EHIP, "decode launch: %s", hipGetErrorString(e));
  hipLaunchKernelGGL(decode_down_kernel<INT>, dim3(static_cast<unsigned>((a.hidden + 15) / 16)), dim3(kDownWaves * 64),
                     0, s, a);
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
  *bytes = static_cast<size_t>(spec->tokens * spec->topk * pitch_of(*spec) * 2);
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
