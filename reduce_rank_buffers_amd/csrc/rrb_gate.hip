// The gate of an MoE layer: from scores [tokens][experts], each token's top-k
// experts and their softmax weights, as rrb_moe_route takes them, and the
// gradient of the scores.
//
// L lanes of a wave share a token, each with V of its scores.  The experts are
// chosen on the scores themselves (the softmax keeps their order, and rounding
// a probability could only merge two): k rounds of a maximum over integers
// that order as the scores do, ties to the lower expert, so the choice is
// exact.  Weights are fp32: w_i = e^(l_i - m) / sum, over all experts, or over
// the chosen ones.
#include <hip/hip_runtime.h>

#include "rrb_internal.h"
#include "rrb_kernels.h"

namespace rrb {
namespace {

struct GateArgs {
  const void *logits;
  int32_t *idx;        // forward: written; backward: read
  float *w;            // forward: written
  const float *dw;     // backward
  void *dlogits;       // backward
  int64_t tokens;
  int32_t experts, topk, renorm;
};

// Tokens up to which a wave takes one token (kernel times, us, whole wave and
// 16 lanes, top-8: 1024 x 256 fp32 4.9, 6.8; 4096 x 256 fp32 7.1, 7.1; 4096 x 64
// fp32 7.1, 4.6; 4096 x 256 bf16 6.6, 5.8).
constexpr int64_t kFewTokens = 1024;

// Scores that one 16-byte load brings.
template <typename T>
constexpr int kPerLoad = 16 / sizeof(T);

__device__ __forceinline__ float score(float v) { return v; }
__device__ __forceinline__ float score(uint16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ void store_score(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_score(uint16_t *p, float v) { *p = f32_to_bf16_rne(v); }

// Orders scores as unsigned integers: -inf lowest, both zeros equal, every
// NaN above +inf (so a row with a NaN has it among its experts and shows it
// in its weights).  Always above 0.
__device__ __forceinline__ uint32_t score_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.f);  // -0 + 0 is +0
  const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
  return f != f ? 0xffffffffu : k;
}
__device__ __forceinline__ float key_score(uint32_t k) {
  return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);  // NaN keeps being one
}

// e^(l - m), where an expert masked out by -inf has no share (also where all
// are) and scores of +inf share equally.  e^x = 2^t (1 + r ln 2) with
// t = fl(x log2 e) and r what t lost of x log2 e, so the product's rounding
// does not grow with |x|: 2 ulp, and 0 below 2^-126.
__device__ __forceinline__ float share(float l, float m) {
  const float x = l - m;
  const float t = x * 1.4426950408889634f;
  const float r = __builtin_fmaf(x, 1.4426950408889634f, -t) + x * 1.925963033500e-8f;
  const float e = __builtin_amdgcn_exp2f(t);
  const float v = __builtin_fmaf(e, r * 0.6931471805599453f, e);
  return l == -INFINITY ? 0.f : l == m ? 1.f : e == 0.f ? 0.f : v;
}

// All-reduce over the L = 16 or 64 lanes of a token: within 16 lanes by DPP
// (two quad permutations, two row rotations), across rows through scalar
// registers.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, false);
}
template <int L, typename F>
__device__ __forceinline__ int across(int v, F f) {
  v = f(v, dpp<0xb1>(v));   // quad_perm [1,0,3,2]
  v = f(v, dpp<0x4e>(v));   // quad_perm [2,3,0,1]
  v = f(v, dpp<0x124>(v));  // row_ror:4
  v = f(v, dpp<0x128>(v));  // row_ror:8
  if (L == 64) {
    const int a = f(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16));
    const int b = f(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48));
    v = f(a, b);
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t most(uint32_t v) {
  return across<L>(static_cast<int>(v), [](int a, int b) {
    return static_cast<int>(max(static_cast<uint32_t>(a), static_cast<uint32_t>(b)));
  });
}
template <int L>
__device__ __forceinline__ uint32_t least(uint32_t v) {
  return ~most<L>(~v);
}
template <int L>
__device__ __forceinline__ float sum_of(float v) {
  return __int_as_float(across<L>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}
template <int L>
__device__ __forceinline__ float max_of(float v) {
  return __int_as_float(across<L>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
}

// The expert of score i of lane `lane`: W consecutive ones per load.
template <int L, int W>
__device__ __forceinline__ int expert_of(int i, int lane) {
  return (i / W * L + lane) * W + i % W;
}

// A lane's V scores of a row; -inf past its end.  W = 1, or a whole load's.
template <typename T, int L, int V, int W>
__device__ __forceinline__ void load_scores(const T *row, int experts, int lane, float (&l)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += W) {
    const int e = expert_of<L, W>(i, lane);
    if (W > 1) {
      T part[W];
      if (e < experts) __builtin_memcpy(part, __builtin_assume_aligned(row + e, 16), sizeof part);
#pragma unroll
      for (int q = 0; q < W; ++q) l[i + q] = e < experts ? score(part[q]) : -INFINITY;
    } else {
      l[i] = e < experts ? score(row[e]) : -INFINITY;
    }
  }
}

// Bound by its operations, the rounds' and the sum's (which renormalised weights
// do not need): 32768 x 256 bf16, top-8, 13 us (45 with a whole wave per token
// and 64-bit keys through shuffles; the scores alone move in 4); 16 x 256 fp32
// 4.2 us, of which the launch is 2.
template <typename T, int L, int V, int W>
__global__ void __launch_bounds__(256) gate_kernel(GateArgs a) {
  constexpr bool kShort = sizeof(T) == 2;
  const int lane = threadIdx.x & (L - 1);
  const int64_t t = blockIdx.x * (256ll / L) + threadIdx.x / L;
  if (t >= a.tokens) return;  // whole tokens leave: the others' lanes are all there
  float l[V];
  load_scores<T, L, V, W>(static_cast<const T *>(a.logits) + t * a.experts, a.experts, lane, l);
  // bf16 scores: the key's upper half and the expert in one word, so a round
  // is one maximum.  fp32: a maximum, then the lowest expert that has it.
  uint32_t key[V];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = expert_of<L, W>(i, lane);
    const uint32_t k = score_key(l[i]);
    key[i] = e >= a.experts ? 0 : kShort ? (k & 0xffff0000u) | (0xffffu - e) : k;
    m = fmaxf(m, l[i]);
  }
  m = max_of<L>(m);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += share(l[i], m);
  float mine = 0.f;
  int chosen = 0;
  uint32_t best = 0;
  for (int j = 0; j < a.topk; ++j) {
    int e;
    float le;
    if (kShort) {
      // Keys differ, so the next one is the largest below the last: as
      // key - best wraps, the keys below best come out above the others, in
      // their order.  (At first best is 0 and every key above it.)
      uint32_t d = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) d = max(d, key[i] - best);
      best += most<L>(d);
      e = static_cast<int>(0xffffu - (best & 0xffffu));
      // the key of a negative score is complemented: its lower half is ones
      le = best >= 0xff810000u ? NAN : key_score(best >> 31 ? best & 0xffff0000u : best | 0xffffu);
    } else {
      best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) best = max(best, key[i]);
      best = most<L>(best);
      uint32_t low = 0xffffffffu;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const uint32_t x = expert_of<L, W>(i, lane);
        low = key[i] == best ? min(low, x) : low;
      }
      low = least<L>(low);
      e = static_cast<int>(low);
      le = key_score(best);
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = expert_of<L, W>(i, lane) == e ? 0 : key[i];
    }
    if (lane == j) {
      chosen = e;
      mine = share(le, m);
    }
  }
  sum = sum_of<L>(a.renorm ? mine : sum);
  if (lane < a.topk) {
    a.idx[t * a.topk + lane] = chosen;
    a.w[t * a.topk + lane] = sum == 0.f ? 0.f : mine / sum;
  }
}

// With p the softmax over all experts and c the chosen ones' sum of p_i dw_i:
//   dl_j = [j chosen] p_j dw_j - p_j c;
// renormalised, with w over the chosen ones alone, dl_i = w_i (dw_i - sum w dw)
// for these and 0 for the others.  Lane j takes the j-th chosen expert: the
// chosen ones' terms meet the row through LDS.  16384 x 128 fp32, top-6: 5.6 us
// for 17 MB.  A masked expert takes no part: its dw is not used.  Indices outside the experts are passed over.
template <typename T, int L, int V, int W>
__global__ void __launch_bounds__(256) gate_backward_kernel(GateArgs a) {
  __shared__ float term[256 * V];  // [token][expert]
  const int lane = threadIdx.x & (L - 1), local = threadIdx.x / L;
  const int64_t t = blockIdx.x * (256ll / L) + local;
  if (t >= a.tokens) return;
  const T *row = static_cast<const T *>(a.logits) + t * a.experts;
  T *out = static_cast<T *>(a.dlogits) + t * a.experts;
  float *mine = term + local * (L * V);
  int32_t e = lane < a.topk ? a.idx[t * a.topk + lane] : -1;
  float dw = lane < a.topk ? a.dw[t * a.topk + lane] : 0.f;
  if (e >= a.experts) e = -1;
  const float le = e >= 0 ? score(row[e]) : -INFINITY;
  if (le == -INFINITY) dw = 0.f;
  float l[V];
  load_scores<T, L, V, W>(row, a.experts, lane, l);
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    m = fmaxf(m, l[i]);
    mine[expert_of<L, W>(i, lane)] = 0.f;
  }
  // Renormalised, the chosen ones' own largest: theirs need not be the row's.
  m = max_of<L>(a.renorm ? le : m);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) sum += l[i] = share(l[i], m);
  const float se = share(le, m);
  sum = sum_of<L>(a.renorm ? se : sum);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const float pe = se * inv;
  const float c = sum_of<L>(pe * dw);
  // A token's lanes are of one wave, whose LDS accesses keep their order; the
  // fence keeps the compiler's.
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (se != 0.f) mine[e] = a.renorm ? pe * (dw - c) : pe * dw;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int i = 0; i < V; i += W) {
    const int x = expert_of<L, W>(i, lane);
    if (x >= a.experts) continue;
    T part[W];
#pragma unroll
    for (int q = 0; q < W; ++q) {
      float d = mine[x + q];
      if (!a.renorm) d = l[i + q] == 0.f ? d : d - l[i + q] * inv * c;
      store_score(part + q, d);
    }
    if (W > 1)
      __builtin_memcpy(__builtin_assume_aligned(out + x, 16), part, sizeof part);
    else
      out[x] = part[0];
  }
}

using GateFn = void (*)(GateArgs);

// Sixteen lanes per token where that leaves at most 16 scores a lane, the
// whole wave otherwise, and where tokens are few: a lane's rounds are then a
// quarter as long, and there is room for the waves.
template <typename T, int W>
GateFn gate_pick(const GateArgs &a, bool back, int *lanes) {
#define RRB_PICK(LANES, n)                                                       \
  if (a.experts <= LANES * (n)) {                                                \
    *lanes = LANES;                                                              \
    return back ? gate_backward_kernel<T, LANES, n, W> : gate_kernel<T, LANES, n, W>; \
  }
  if (a.tokens > kFewTokens) {
    RRB_PICK(16, 4 < W ? W : 4) RRB_PICK(16, 8) RRB_PICK(16, 16)
  }
  RRB_PICK(64, 4 < W ? W : 4) RRB_PICK(64, 8) RRB_PICK(64, 16)
#undef RRB_PICK
  return nullptr;
}

rrb_status gate(const GateArgs &a, int32_t dtype, uint32_t flags, bool back, rrb_stream_t stream) {
  if (a.tokens < 0 || a.experts < 1 || a.topk < 1 || a.topk > a.experts)
    return fail(RRB_EINVAL, "tokens %lld, experts %d, topk %d: tokens >= 0, 1 <= topk <= experts needed",
                (long long)a.tokens, a.experts, a.topk);
  if (dtype != RRB_BF16 && dtype != RRB_F32) return fail(RRB_EINVAL, "unknown dtype %d", dtype);
  if (flags & ~RRB_GATE_RENORMALIZE) return fail(RRB_EINVAL, "unknown flags 0x%x", flags);
  if (a.experts > kRouteMaxExperts || a.topk > kRouteMaxTopk)
    return fail(RRB_EUNSUPPORTED, "experts %d, topk %d: at most %d and %d", a.experts, a.topk, kRouteMaxExperts,
                kRouteMaxTopk);
  if (a.tokens >= 1LL << 26) return fail(RRB_EUNSUPPORTED, "tokens %lld >= 2^26", (long long)a.tokens);
  if (a.tokens == 0) return RRB_OK;
  if (!a.logits || !a.idx || (back ? !a.dw || !a.dlogits : !a.w)) return fail(RRB_EINVAL, "NULL array");
  const int64_t row = a.experts * static_cast<int64_t>(elem_size(dtype));
  const int64_t scores = a.tokens * row, chosen = a.tokens * a.topk * 4;
  // A token's scores are read before its gradients are written, by one wave:
  // the gradients may take the scores' place.
  const Span spans[] = {{a.dlogits == a.logits ? nullptr : a.logits, scores, "logits", false},
                        {a.idx, chosen, "topk_idx", !back},
                        {a.w, chosen, "topk_w", true},
                        {a.dw, chosen, "dtopk_w", false},
                        {a.dlogits, scores, "dlogits", true}};
  const rrb_status st = check_disjoint(spans);
  if (st != RRB_OK) return st;
  // Whole 16-byte loads where every row starts on such a boundary.
  const int per = dtype == RRB_F32 ? kPerLoad<float> : kPerLoad<uint16_t>;
  const bool wide = a.experts % per == 0 &&
                    ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits)) & 15) == 0;
  int lanes = 64;
  const GateFn fn = dtype == RRB_F32 ? (wide ? gate_pick<float, kPerLoad<float>>(a, back, &lanes)
                                             : gate_pick<float, 1>(a, back, &lanes))
                                     : (wide ? gate_pick<uint16_t, kPerLoad<uint16_t>>(a, back, &lanes)
                                             : gate_pick<uint16_t, 1>(a, back, &lanes));
  // A launch's threads are counted in 32 bits: 2^23 tokens (at most 2^29
  // threads) at a time.
  constexpr int64_t kMost = 1 << 23;
  for (int64_t first = 0; first < a.tokens; first += kMost) {
    GateArgs b = a;
    b.tokens = a.tokens - first < kMost ? a.tokens - first : kMost;
    b.logits = static_cast<const char *>(a.logits) + first * row;
    b.idx += first * a.topk;
    if (back) {
      b.dw += first * a.topk;
      b.dlogits = static_cast<char *>(a.dlogits) + first * row;
    } else {
      b.w += first * a.topk;
    }
    const int64_t blocks = (b.tokens + 256 / lanes - 1) / (256 / lanes);
    hipLaunchKernelGGL(fn, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, static_cast<hipStream_t>(stream), b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(RRB_EHIP, "gate launch: %s", hipGetErrorString(e));
  }
  return RRB_OK;
}

}  // namespace
}  // namespace rrb

using namespace rrb;

extern "C" {

rrb_status rrb_moe_gate(int64_t tokens, int32_t experts, int32_t topk, int32_t dtype, uint32_t flags,
                        const void *d_logits, int32_t *d_topk_idx, float *d_topk_w, rrb_stream_t stream) {
  clear_error();
  GateArgs a{};
  a.logits = d_logits;
  a.idx = d_topk_idx;
  a.w = d_topk_w;
  a.tokens = tokens;
  a.experts = experts;
  a.topk = topk;
  a.renorm = flags & RRB_GATE_RENORMALIZE ? 1 : 0;
  return gate(a, dtype, flags, false, stream);
}

rrb_status rrb_moe_gate_backward(int64_t tokens, int32_t experts, int32_t topk, int32_t dtype, uint32_t flags,
                                 const void *d_logits, const int32_t *d_topk_idx, const float *d_dtopk_w,
                                 void *d_dlogits, rrb_stream_t stream) {
  clear_error();
  GateArgs a{};
  a.logits = d_logits;
  a.idx = const_cast<int32_t *>(d_topk_idx);
  a.dw = d_dtopk_w;
  a.dlogits = d_dlogits;
  a.tokens = tokens;
  a.experts = experts;
  a.topk = topk;
  a.renorm = flags & RRB_GATE_RENORMALIZE ? 1 : 0;
  return gate(a, dtype, flags, true, stream);
}

}  // extern "C"
